"""GPU checks of the operators around the recurrence at the edges of what their
documentation allows: offsets past 32 bits, very many columns, heads and tiles,
repeated (stride 0) gradients, poison in one row, positions out of order."""
import numpy as np
import pytest

import around_ref as ref
from test_gpu_around import _close, _draw, _nan, _pdn, _scan_case, _up
from gpu_util import torch_mod

pytestmark = pytest.mark.gpu
f64 = lambda v: None if v is None else np.asarray(v, np.float64)


def _far(buf, first, shape, strides):
    """A view whose last row starts past 2^31 elements of `buf`."""
    return buf.as_strided(shape, strides, first)


def test_scan_rows_past_32_bits():
    pdn = _pdn()
    torch = torch_mod()
    B, T, D = 2, 5, 64
    st, sb = 248_000_000, 1_240_000_000      # last row at 2.23e9 elements
    buf = torch.empty(2_480_000_000, device="cuda", dtype=torch.bfloat16)
    x, la, h0, dh, dhT = _scan_case((B, T, D, "bf16", "bf16", 2, True, True), 300)
    views = [_far(buf, 64 * i, (B, T, D), (sb, st, 1)) for i in range(6)]
    xd, lad, h, dhd, dx, dla = views
    xd.copy_(_up(x, "bf16"))
    lad.copy_(_up(la, "bf16"))
    dhd.copy_(_up(dh, "bf16"))
    dh0 = _nan((B, D))
    pdn.pdn_scan_fwd(xd, lad, h, h0=_up(h0), gain=2)
    want, bound = ref.scan_fwd(f64(x), f64(la), f64(h0), 2)
    _close("far scan h", h, want, bound, "bf16")
    pdn.pdn_scan_bwd(xd, lad, dhd, dx, dla, h0=_up(h0), dhT=_up(dhT), dh0=dh0, gain=2)
    refs = ref.scan_bwd(f64(x), f64(la), f64(h0), f64(dh), f64(dhT), 2)
    _close("far scan dx", dx, *refs[0], "bf16")
    _close("far scan dlog_a", dla, *refs[1], "bf16")
    _close("far scan dh0", dh0, *refs[2])


def test_norm_rows_past_32_bits():
    pdn = _pdn()
    torch = torch_mod()
    B, T, H, d = 2, 4, 2, 128
    sb, st, sh = 1_240_000_000, 300_000_000, 100_000_000
    buf = torch.empty(2_480_000_000, device="cuda", dtype=torch.bfloat16)
    rng = np.random.default_rng(301)
    x, z = _draw(rng, (B, T, H, d), "bf16"), _draw(rng, (B, T, H, d), "bf16")
    g, o = rng.standard_normal((B, H, T, d)).astype(np.float32), rng.standard_normal((B, H, T, d)).astype(np.float32)
    w = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    xd, zd, dx, y = (_far(buf, 128 * i, (B, T, H, d), (sb, st, sh, 1)) for i in range(4))
    xd.copy_(_up(x, "bf16"))
    zd.copy_(_up(z, "bf16"))
    q, k = _nan((B, H, T, d), "bf16"), _nan((B, H, T, d), "bf16")
    eps = float(np.float32(1e-6))
    pdn.pdn_qk_norm_fwd(xd, zd, q, k, norm=1)
    for t, v in ((q, x), (k, z)):
        want, bound = ref.qk_one(f64(v), None, 1.0, H, 1, eps, None)
        _close("far q/k", t, want, bound, "bf16")
    near = _nan((B, T, H, d), "bf16")
    pdn.pdn_qk_norm_bwd(xd, zd, _up(g), _up(g), dx, near, norm=1)
    for t, v in ((dx, x), (near, z)):
        want, bound, _, _ = ref.qk_one_bwd(f64(v), None, 1.0, f64(g), 1, eps, None)
        _close("far dx", t, want, bound, "bf16")
    pdn.pdn_out_norm_fwd(_up(o), y, z=zd, w=_up(w))
    want, bound = ref.out_fwd(f64(o), f64(w), f64(z), 1, eps)
    _close("far y", y, want, bound, "bf16")
    # the gate's gradient over the far rows of y
    do, dw = _nan((B, H, T, d)), _nan((d,))
    pdn.pdn_out_norm_bwd(_up(o), xd, do, z=zd, dz=y, w=_up(w), dw=dw)
    wdo, wdz, wdw = ref.out_bwd(f64(o), f64(w), f64(z), f64(x), 1, eps)
    _close("far do", do, *wdo)
    _close("far dz", y, *wdz, "bf16")
    _close("far dw", dw, *wdw)


@pytest.mark.parametrize("case", [
    (20000, 150, 8, "fp32", "fp32", 0, True, False),      # very many columns
    (1, 100003, 8, "fp32", "fp32", 1, True, True),        # very many tiles of one
    (3, 2, 4096, "bf16", "bf16", 2, True, False),
    (1, 385, 2040, "bf16", "fp32", 1, False, True),       # a strip's last channels missing
], ids=lambda c: "B%d-T%d-D%d" % c[:3])
def test_scan_shapes(case):
    pdn = _pdn()
    B, T, D, dt, lt, kind, state, _ = case
    x, la, h0, dh, dhT = _scan_case(case, 302)
    h0d, dhTd = (_up(h0), _up(dhT)) if state else (None, None)
    h, hT = _nan((B, T, D), dt), _nan((B, D))
    dx, dla, dh0 = _nan((B, T, D), dt), _nan((B, T, D), lt), _nan((B, D))
    xd, lad = _up(x, dt), _up(la, lt)
    pdn.pdn_scan_fwd(xd, lad, h, h0=h0d, hT=hT, gain=kind)
    want, bound = ref.scan_fwd(f64(x), f64(la), f64(h0), kind)
    _close("scan h", h, want, bound, dt)
    _close("scan hT", hT, want[:, -1], bound[:, -1])
    pdn.pdn_scan_bwd(xd, lad, _up(dh, dt), dx, dla, h0=h0d, dhT=dhTd, dh0=dh0, gain=kind)
    refs = ref.scan_bwd(f64(x), f64(la), f64(h0), f64(dh), f64(dhT), kind)
    _close("scan dx", dx, *refs[0], dt)
    _close("scan dlog_a", dla, *refs[1], lt)
    _close("scan dh0", dh0, *refs[2])


def test_repeated_gradients():
    """The gradient of a sum: one value for all, stride 0 throughout but the last dimension."""
    pdn = _pdn()
    torch = torch_mod()
    x, la, h0, _, _ = _scan_case((2, 300, 64, "fp32", "fp32", 0, True, False), 303)
    one = torch.ones((1, 1, 64), device="cuda").expand(2, 300, 64)
    got, want = [], []
    for out, dh in ((got, one), (want, one.contiguous())):
        out += [_nan((2, 300, 64)), _nan((2, 300, 64))]
        pdn.pdn_scan_bwd(_up(x), _up(la), dh, *out, h0=_up(h0))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    o = torch.randn((2, 3, 5, 32), device="cuda")
    dy = torch.ones((1, 1, 1, 32), device="cuda").expand(2, 5, 3, 32)
    a, b = _nan((2, 3, 5, 32)), _nan((2, 3, 5, 32))
    pdn.pdn_out_norm_bwd(o, dy, a)
    pdn.pdn_out_norm_bwd(o, dy.contiguous(), b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,H", [(3, 4096), (1, 70000)])
def test_very_many_heads(T, H):
    pdn = _pdn()
    B, d = 1, 64
    rng = np.random.default_rng(304)
    x = _draw(rng, (B, T, H, d), "bf16")
    q, k = _nan((B, H, T, d), "bf16"), _nan((B, H, T, d), "bf16")
    one = _draw(rng, (B, T, 1, d), "bf16")
    pdn.pdn_qk_norm_fwd(_up(x, "bf16"), _up(one, "bf16"), q, k)
    eps = float(np.float32(1e-6))
    for t, v in ((q, x), (k, one)):
        want, bound = ref.qk_one(f64(v), None, 1.0, H, 2, eps, None)
        _close("many heads", t, want, bound, "bf16")
    g = rng.standard_normal((B, H, T, d)).astype(np.float32)
    dx, done = _nan((B, T, H, d), "bf16"), _nan((B, T, 1, d), "bf16")
    w = np.ones(d, np.float32)
    dw = [_nan((d,)), _nan((d,))]
    pdn.pdn_qk_norm_bwd(_up(x, "bf16"), _up(one, "bf16"), _up(g), _up(g), dx, done, wq=_up(w), wk=_up(w), dwq=dw[0], dwk=dw[1])
    for t, v, s in ((dx, x, dw[0]), (done, one, dw[1])):
        want, bound, dww, dwb = ref.qk_one_bwd(f64(v), f64(w), 1.0, f64(g), 2, eps, None)
        _close("many heads dx", t, want, bound, "bf16")
        _close("many heads dw", s, dww, dwb)


def test_poison_stays_in_its_row():
    """NaN and infinities in one head of one token leave every other row's bits."""
    pdn = _pdn()
    torch = torch_mod()
    B, T, H, d = 2, 37, 4, 128
    gen = torch.Generator(device="cuda").manual_seed(305)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x, z, g, o = rnd(B, T, H, d), rnd(B, T, H, d), rnd(B, H, T, d), rnd(B, H, T, d)
    inv = torch.rand(32, generator=gen, device="cuda", dtype=torch.float64)

    def run(x, z, o):
        q, k, y = _nan((B, H, T, d)), _nan((B, H, T, d)), _nan((B, T, H, d))
        pdn.pdn_qk_norm_fwd(x, z, q, k, inv_freq=inv)
        pdn.pdn_out_norm_fwd(o, y, z=z)
        dx, dz, do, dg = _nan((B, T, H, d)), _nan((B, T, H, d)), _nan((B, H, T, d)), _nan((B, T, H, d))
        pdn.pdn_qk_norm_bwd(x, z, g, g, dx, dz, inv_freq=inv)
        pdn.pdn_out_norm_bwd(o, x, do, z=z, dz=dg)
        return [q.transpose(1, 2), k.transpose(1, 2), y, dx, dz, do.transpose(1, 2), dg]

    good = run(x, z, o)
    bx, bz, bo = x.clone(), z.clone(), o.clone()
    bx[1, 20, 2, 5], bz[1, 20, 2, 100], bo[1, 2, 20, 77] = float("nan"), float("inf"), float("-inf")
    bad = run(bx, bz, bo)
    keep = torch.ones((B, T, H), dtype=torch.bool, device="cuda")
    keep[1, 20, 2] = False
    for a, b in zip(bad, good):
        assert torch.equal(a[keep], b[keep])
        assert not torch.isfinite(a[1, 20, 2]).all()


def test_positions_in_any_order():
    pdn = _pdn()
    B, T, H, d = 2, 50, 2, 64
    rng = np.random.default_rng(306)
    x = _draw(rng, (B, T, H, d), "fp32")
    pos = rng.integers(-(1 << 30), 1 << 30, (B, T))
    pos[0, :10] = 7                       # the same position many times
    pos[1, 0] = (1 << 40) + 1             # past what 32 bits hold
    inv = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    q, k = _nan((B, H, T, d)), _nan((B, H, T, d))
    pdn.pdn_qk_norm_fwd(_up(x), _up(x), q, k, inv_freq=_up(inv), positions=_up(pos), rope_layout=1)
    small = np.abs(pos) < (1 << 31)       # 64-bit angles of larger ones are off by more than fp32 rounds
    turn = ref.rotation(np.where(small, pos, 0), inv, d, 1, 1.0)
    want, bound = ref.qk_one(f64(x), None, 1.0, H, 2, float(np.float32(1e-6)), turn)
    # |angle| 2^31 in 64 bits: 2^31 x 2^-53 x 3 roundings on each side, under 24 U of a radian
    bound = bound * 2
    for t in (q, k):
        sel = np.broadcast_to(small[:, None, :], (B, H, T))
        _close("q/k at any position", t[torch_mod().from_numpy(sel.copy()).to("cuda")], want[sel], bound[sel])


@pytest.mark.parametrize("which", ["q", "k"])
def test_weights_on_one_side(which):
    pdn = _pdn()
    B, T, H, d = 2, 40, 3, 64
    rng = np.random.default_rng(307)
    x = {n: _draw(rng, (B, T, H, d), "fp32") for n in "qk"}
    g = {n: rng.standard_normal((B, H, T, d)).astype(np.float32) for n in "qk"}
    w = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    out = {n: _nan((B, H, T, d)) for n in "qk"}
    kw = {"w" + which: _up(w), "norm": 1}
    pdn.pdn_qk_norm_fwd(_up(x["q"]), _up(x["k"]), out["q"], out["k"], **kw)
    dx, dw = {n: _nan((B, T, H, d)) for n in "qk"}, _nan((d,))
    pdn.pdn_qk_norm_bwd(_up(x["q"]), _up(x["k"]), _up(g["q"]), _up(g["k"]), dx["q"], dx["k"], **{"dw" + which: dw}, **kw)
    eps = float(np.float32(1e-6))
    for n in "qk":
        wn = f64(w) if n == which else None
        want, bound = ref.qk_one(f64(x[n]), wn, 1.0, H, 1, eps, None)
        _close("one side " + n, out[n], want, bound)
        want, bound, dww, dwb = ref.qk_one_bwd(f64(x[n]), wn, 1.0, f64(g[n]), 1, eps, None)
        _close("one side dx" + n, dx[n], want, bound)
        if n == which:
            _close("one side dw" + n, dw, dww, dwb)


def test_heads_before_tokens():
    """Strided tensors in the other order: [B,H,T,d] memory seen as [B,T,H,d]."""
    pdn = _pdn()
    torch = torch_mod()
    B, T, H, d = 2, 37, 3, 128
    gen = torch.Generator(device="cuda").manual_seed(308)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x, z, o, g = rnd(B, H, T, d), rnd(B, H, T, d), rnd(B, H, T, d), rnd(B, H, T, d)
    got, want = [], []
    for order, out in ((lambda t: t.transpose(1, 2), got), (lambda t: t.transpose(1, 2).contiguous(), want)):
        new = lambda: _nan((B, H, T, d)).transpose(1, 2) if order(x).stride(1) == d else _nan((B, T, H, d))
        q, k, y, dx, dz, dg, do = _nan((B, H, T, d)), _nan((B, H, T, d)), new(), new(), new(), new(), _nan((B, H, T, d))
        pdn.pdn_qk_norm_fwd(order(x), order(z), q, k)
        pdn.pdn_out_norm_fwd(o, y, z=order(z))
        pdn.pdn_qk_norm_bwd(order(x), order(z), g, g, dx, dz)
        pdn.pdn_out_norm_bwd(o, order(x), do, z=order(z), dz=dg)
        out += [q, k, y, dx, dz, dg, do]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_with_workspaces_made_inside():
    pdn = _pdn()
    torch = torch_mod()
    x, la, h0, dh, dhT = _scan_case((2, 1100, 1160, "bf16", "bf16", 0, True, True), 309)
    ins = [_up(x, "bf16"), _up(la, "bf16"), _up(dh, "bf16")]
    outs = [torch.zeros_like(ins[0]) for _ in range(3)]

    def run():
        pdn.pdn_scan_fwd(ins[0], ins[1], outs[0])
        pdn.pdn_scan_bwd(ins[0], ins[1], ins[2], outs[1], outs[2])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t in outs:
            t.zero_()
        junk = torch.full((1 << 22,), 5.0, device="cuda")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        del junk


def test_calls_from_two_threads():
    import threading
    pdn = _pdn()
    torch = torch_mod()
    cases = [_scan_case((2, 1500, 264, "fp32", "fp32", 1, True, False), s) for s in (310, 311)]
    ins = [(_up(x), _up(la), _up(h0)) for x, la, h0, _, _ in cases]
    want = []
    for x, la, h0 in ins:
        want.append(torch.empty_like(x))
        pdn.pdn_scan_fwd(x, la, want[-1], h0=h0, gain=1)
    torch.cuda.synchronize()
    got = [[] for _ in ins]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                h = torch.zeros_like(ins[i][0])
                pdn.pdn_scan_fwd(ins[i][0], ins[i][1], h, h0=ins[i][2], gain=1)
                got[i].append(h)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 20 and all(torch.equal(h, want[i]) for h in got[i])


def test_very_many_tokens():
    """40 million rows of 16, some of them looked at."""
    pdn = _pdn()
    torch = torch_mod()
    n, d = 40_000_003, 16
    gen = torch.Generator(device="cuda").manual_seed(312)
    o = torch.randn((1, 1, n, d), generator=gen, device="cuda", dtype=torch.float32)
    y = torch.full((1, n, 1, d), float("nan"), device="cuda")
    pdn.pdn_out_norm_fwd(o, y)
    at = torch.cat([torch.arange(100), torch.randint(0, n, (5000,)), torch.arange(n - 100, n)]).to("cuda")
    want, bound = ref.out_fwd(o[:, :, at].double().cpu().numpy(), None, None, 0, float(np.float32(1e-6)))
    _close("many tokens", y[:, at], want, bound)
    assert bool(torch.isfinite(y).all())
