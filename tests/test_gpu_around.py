"""GPU checks of the operators around the recurrence (q/k norm and rotation,
gated output norm, vector-state scan), forward and backward, element by
element against 64-bit references with bounds counted in roundings
(around_ref.py): sizes from one token up, ragged tails, shared heads, strided
views, both layouts and types, resets, NaN and infinities before a reset,
streams, graphs, and all of them in one training step."""
import numpy as np
import pytest

import around_ref as ref
from around_ref import HALF, U
from gpu_util import torch_mod

pytestmark = pytest.mark.gpu
TINY = 1e-37   # fp32 results below 2^-126 may be flushed to zero


def _pdn():
    import gated_delta_rule_77_amd as pdn
    return pdn


def _up(x, dtype="fp32"):
    torch = torch_mod()
    t = torch.from_numpy(np.ascontiguousarray(x)).to("cuda")
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def _down(t):
    return t.detach().double().cpu().numpy()


def _draw(rng, shape, dtype, scale=1.0):
    x = (scale * rng.standard_normal(shape)).astype(np.float32)
    return ref.bf16(x) if dtype == "bf16" else x


def _close(name, got, want, bound, dtype="fp32"):
    got = _down(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if not want.size:
        return
    assert np.isfinite(got).all(), "%s: not finite" % name
    room = bound + HALF[dtype] * (np.abs(want) + bound) + TINY
    over = np.abs(got - want) / room
    print("[around] %s: worst error %.2f of its bound" % (name, over.max()), flush=True)
    assert over.max() <= 1.0, "%s: %.3g times its bound at %s" % (name, over.max(), np.unravel_index(over.argmax(), over.shape))


def _nan(shape, dtype="fp32"):
    torch = torch_mod()
    return torch.full(shape, float("nan"), device="cuda", dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)


# ---------------------------------------------------------------------------
# q/k norm and rotation
# ---------------------------------------------------------------------------

QK = [  # B, T, Hq, Hk, H, d, dtype, norm, weights, rot, layout, positions
    (1, 1, 1, 1, 1, 64, "fp32", 2, False, 0, 0, None),
    (1, 1, 4, 4, 4, 128, "bf16", 2, False, 128, 0, 123456789),
    (3, 5, 6, 2, 6, 128, "bf16", 1, True, 64, 0, 0),
    (2, 17, 3, 3, 3, 128, "fp32", 1, True, 128, 1, 7),
    (2, 33, 5, 1, 5, 64, "bf16", 2, True, 16, 1, 1 << 20),
    (1, 67, 2, 4, 8, 64, "fp32", 0, False, 48, 0, 1 << 24),
    (2, 131, 16, 4, 16, 128, "bf16", 2, False, 0, 0, None),
    (1, 1000, 4, 4, 4, 128, "bf16", 1, True, 96, 0, None),
    (70, 1, 8, 8, 8, 128, "bf16", 2, False, 128, 0, 60000),
    (1, 40, 1, 1, 12, 128, "fp32", 2, True, 32, 0, 5),
]


def _qk_case(case, seed):
    B, T, Hq, Hk, H, d, dtype, norm, weights, rot, layout, at = case
    rng = np.random.default_rng(seed)
    rows = _draw(rng, (B, T, (Hq + Hk + H) * d), dtype)
    if T > 2:
        rows[0, 1] = 0          # a row of zeros
        rows[0, 2] *= 2.0 ** -40
    w = [(1 + 0.2 * rng.standard_normal(d)).astype(np.float32) if weights else None for _ in range(2)]
    inv = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot) if rot else None
    pos = None
    if rot and at is not None:
        pos = (at + 3 * np.arange(B)[:, None] + np.arange(T)[None]).astype(np.int64)
        pos[-1, -1] = 0         # a sequence that starts within the row
    scale = (d ** -0.5, 1.25)
    rs = 1.1 if rot else 1.0
    dev = _up(rows, dtype)
    xq = dev[:, :, :Hq * d].unflatten(2, (Hq, d))
    xk = dev[:, :, Hq * d:(Hq + Hk) * d].unflatten(2, (Hk, d))
    kw = dict(norm=norm, eps=1e-6, wq=None if w[0] is None else _up(w[0]), wk=None if w[1] is None else _up(w[1]),
              q_scale=scale[0], k_scale=scale[1])
    if rot:
        kw.update(inv_freq=_up(inv), positions=None if pos is None else _up(pos), rope_layout=layout, rope_scale=rs)
        turn = ref.rotation(pos if pos is not None else np.broadcast_to(np.arange(T), (B, T)), inv, d, layout, float(np.float32(rs)))
    else:
        turn = None
    host = rows.astype(np.float64)
    hq, hk = host[..., :Hq * d].reshape(B, T, Hq, d), host[..., Hq * d:(Hq + Hk) * d].reshape(B, T, Hk, d)
    f64 = lambda v: None if v is None else v.astype(np.float64)
    sides = [(hq, f64(w[0]), float(np.float32(scale[0]))), (hk, f64(w[1]), float(np.float32(scale[1])))]
    return (xq, xk), kw, sides, turn, float(np.float32(1e-6)), rng


@pytest.mark.parametrize("case", QK, ids=lambda c: "B%d-T%d-%d.%d.%d-d%d-%s-n%d%s-r%d.%d" % (c[:8] + ("w" if c[8] else "",) + c[9:11]))
def test_qk_norm_fwd(case):
    pdn = _pdn()
    B, T, Hq, Hk, H, d, dtype, norm = case[:8]
    (xq, xk), kw, sides, turn, eps, _ = _qk_case(case, 200)
    q, k = _nan((B, H, T, d), dtype), _nan((B, H, T, d), dtype)
    pdn.pdn_qk_norm_fwd(xq, xk, q, k, **kw)
    for name, t, (x, w, scale) in zip("qk", (q, k), sides):
        want, bound = ref.qk_one(x, w, scale, H, norm, eps, turn)
        _close("qk_norm " + name, t, want, bound, dtype)


@pytest.mark.parametrize("case", QK, ids=lambda c: "B%d-T%d-%d.%d.%d-d%d-%s-n%d%s-r%d.%d" % (c[:8] + ("w" if c[8] else "",) + c[9:11]))
def test_qk_norm_bwd(case):
    pdn = _pdn()
    torch = torch_mod()
    B, T, Hq, Hk, H, d, dtype, norm = case[:8]
    (xq, xk), kw, sides, turn, eps, rng = _qk_case(case, 201)
    g = [_draw(rng, (B, H, T, d), "fp32") for _ in range(2)]
    # the gradients go into a projection's gradient, side by side; the rest of it stays as it was
    rows = torch.full((B, T, (Hq + Hk + H) * d), 7.0, device="cuda", dtype=xq.dtype)
    dxq = rows[:, :, :Hq * d].unflatten(2, (Hq, d))
    dxk = rows[:, :, Hq * d:(Hq + Hk) * d].unflatten(2, (Hk, d))
    dw = {"dwq": _nan((d,)), "dwk": _nan((d,))} if case[8] else {}
    pdn.pdn_qk_norm_bwd(xq, xk, _up(g[0]), _up(g[1]), dxq, dxk, **dw, **kw)
    again = {n: t.clone() for n, t in dw.items()}
    for name, dx, gs, (x, w, scale) in zip("qk", (dxq, dxk), g, sides):
        want, bound, dww, dwb = ref.qk_one_bwd(x, w, scale, gs.astype(np.float64), norm, eps, turn)
        _close("qk_norm dx" + name, dx, want, bound, dtype)
        if dw:
            _close("qk_norm dw" + name, dw["dw" + name], dww, dwb)
    assert bool((rows[:, :, (Hq + Hk) * d:] == 7.0).all())
    pdn.pdn_qk_norm_bwd(xq, xk, _up(g[0]), _up(g[1]), dxq, dxk, **dw, **kw)
    for n in dw:
        assert torch.equal(dw[n], again[n]), n + " differs between two calls"


def test_qk_norm_gradient_by_differences():
    """The backward against central differences of the forward (fp32): their
    own error is about U |L| / step plus step^2 times a third derivative of
    order one, over sums of 512 terms."""
    pdn = _pdn()
    rng = np.random.default_rng(202)
    B, T, H, d = 1, 4, 2, 64
    x = rng.standard_normal((B, T, 2, d)).astype(np.float32)
    g = rng.standard_normal((2, B, H, T, d)).astype(np.float32)
    inv = _up(10000.0 ** (-2.0 * np.arange(16) / 32))
    w = _up((1 + 0.1 * rng.standard_normal(d)).astype(np.float32))
    kw = dict(norm=1, wq=w, wk=w, inv_freq=inv, rope_layout=0)

    def loss(xs):
        xd = _up(xs.astype(np.float32))
        q, k = _nan((B, H, T, d)), _nan((B, H, T, d))
        pdn.pdn_qk_norm_fwd(xd[:, :, :1], xd[:, :, 1:], q, k, **kw)
        return float((_down(q) * g[0]).sum() + (_down(k) * g[1]).sum())

    xd = _up(x)
    dx, dw = _nan((B, T, 2, d)), [_nan((d,)), _nan((d,))]
    pdn.pdn_qk_norm_bwd(xd[:, :, :1], xd[:, :, 1:], _up(g[0]), _up(g[1]), dx[:, :, :1], dx[:, :, 1:], dwq=dw[0], dwk=dw[1], **kw)
    got = _down(dx)
    for _ in range(6):
        v = rng.standard_normal(x.shape)
        v /= np.linalg.norm(v)
        step = 2.0 ** -7
        diff = (loss(x + step * v) - loss(x - step * v)) / (2 * step)
        assert abs(diff - (got * v).sum()) < 5e-3 * max(1.0, np.linalg.norm(got)), (diff, (got * v).sum())


def test_qk_norm_without_tokens():
    pdn = _pdn()
    torch = torch_mod()
    e = lambda *s: torch.empty(s, device="cuda")
    pdn.pdn_qk_norm_fwd(e(2, 0, 4, 64), e(2, 0, 2, 64), e(2, 4, 0, 64), e(2, 4, 0, 64))
    w, dw = torch.ones(64, device="cuda"), [_nan((64,)), _nan((64,))]
    pdn.pdn_qk_norm_bwd(e(2, 0, 4, 64), e(2, 0, 2, 64), e(2, 4, 0, 64), e(2, 4, 0, 64), e(2, 0, 4, 64), e(2, 0, 2, 64),
                        dwq=dw[0], dwk=dw[1], wq=w, wk=w)
    assert all(bool((t == 0).all()) for t in dw)


# ---------------------------------------------------------------------------
# gated output norm
# ---------------------------------------------------------------------------

OUT = [  # B, H, T, dv, o type, type, act, weights
    (1, 1, 1, 16, "fp32", "fp32", 0, False),
    (2, 3, 5, 128, "fp32", "bf16", 1, True),
    (1, 2, 33, 96, "bf16", "bf16", 2, True),
    (2, 1, 70, 256, "fp32", "fp32", 1, True),
    (1, 5, 17, 48, "fp32", "bf16", 1, False),
    (3, 4, 1, 64, "bf16", "fp32", 2, True),
    (1, 16, 300, 128, "fp32", "bf16", 1, True),
    (1, 1, 9, 240, "fp32", "bf16", 0, True),
    (1, 2, 1000, 32, "fp32", "fp32", 1, True),
]


def _out_case(case, seed):
    B, H, T, dv, od, dt, kind, weights = case
    rng = np.random.default_rng(seed)
    o = _draw(rng, (B, H, T, dv), od, 0.3)
    if T > 1:
        o[0, 0, 1] = 0
    z = _draw(rng, (B, T, 2 * H * dv), dt, 3.0) if kind else None
    if kind:
        z[0, 0, H * dv:H * dv + 4] = [-100.0, 100.0, -20.0, 0.0]
    w = (1 + 0.2 * rng.standard_normal(dv)).astype(np.float32) if weights else None
    zd = _up(z, dt)[:, :, H * dv:].unflatten(2, (H, dv)) if kind else None
    zh = z[:, :, H * dv:].reshape(B, T, H, dv).astype(np.float64) if kind else None
    return o, zd, zh, w, rng


def _out_ids(c):
    return "B%d-H%d-T%d-%d-%s-%s-a%d%s" % (c[:7] + ("w" if c[7] else "",))


@pytest.mark.parametrize("case", OUT, ids=_out_ids)
def test_out_norm_fwd(case):
    pdn = _pdn()
    B, H, T, dv, od, dt, kind, weights = case
    o, zd, zh, w, _ = _out_case(case, 210)
    torch = torch_mod()
    wide = torch.full((B, T, H + 1, dv), 7.0, device="cuda", dtype=torch.bfloat16 if dt == "bf16" else torch.float32)
    y = wide[:, :, :H]
    pdn.pdn_out_norm_fwd(_up(o, od), y, z=zd, w=None if w is None else _up(w), act=kind)
    want, bound = ref.out_fwd(o.astype(np.float64), None if w is None else w.astype(np.float64), zh, kind, float(np.float32(1e-6)))
    _close("out_norm y", y, want, bound, dt)
    assert bool((wide[:, :, H] == 7.0).all())


@pytest.mark.parametrize("case", OUT, ids=_out_ids)
def test_out_norm_bwd(case):
    pdn = _pdn()
    torch = torch_mod()
    B, H, T, dv, od, dt, kind, weights = case
    o, zd, zh, w, rng = _out_case(case, 211)
    dy = _draw(rng, (B, T, H, dv), dt)
    do = _nan((B, H, T, dv))
    dz = _nan((B, T, H, dv), dt) if kind else None
    wd, dw = (_up(w), _nan((dv,))) if weights else (None, None)
    pdn.pdn_out_norm_bwd(_up(o, od), _up(dy, dt), do, z=zd, dz=dz, w=wd, dw=dw, act=kind)
    wdo, wdz, wdw = ref.out_bwd(o.astype(np.float64), None if w is None else w.astype(np.float64), zh, dy.astype(np.float64),
                                kind, float(np.float32(1e-6)))
    _close("out_norm do", do, *wdo)
    if kind:
        _close("out_norm dz", dz, *wdz, dt)
    if weights:
        _close("out_norm dw", dw, *wdw)
        first = dw.clone()
        pdn.pdn_out_norm_bwd(_up(o, od), _up(dy, dt), do, z=zd, dz=dz, w=wd, dw=dw, act=kind)
        assert torch.equal(dw, first)


def test_out_norm_gradient_by_differences():
    pdn = _pdn()
    rng = np.random.default_rng(212)
    B, H, T, dv = 1, 2, 3, 48
    o, z = rng.standard_normal((B, H, T, dv)).astype(np.float32), rng.standard_normal((B, T, H, dv)).astype(np.float32)
    g, w = rng.standard_normal((B, T, H, dv)).astype(np.float32), _up((1 + 0.1 * rng.standard_normal(dv)).astype(np.float32))

    def loss(os, zs):
        y = _nan((B, T, H, dv))
        pdn.pdn_out_norm_fwd(_up(os.astype(np.float32)), y, z=_up(zs.astype(np.float32)), w=w)
        return float((_down(y) * g).sum())

    do, dz, dw = _nan((B, H, T, dv)), _nan((B, T, H, dv)), _nan((dv,))
    pdn.pdn_out_norm_bwd(_up(o), _up(g), do, z=_up(z), dz=dz, w=w, dw=dw)
    step = 2.0 ** -7
    for _ in range(6):
        v, u = rng.standard_normal(o.shape), rng.standard_normal(z.shape)
        v, u = v / np.linalg.norm(v), u / np.linalg.norm(u)
        diff = (loss(o + step * v, z + step * u) - loss(o - step * v, z - step * u)) / (2 * step)
        mine = (_down(do) * v).sum() + (_down(dz) * u).sum()
        assert abs(diff - mine) < 5e-3 * max(1.0, np.linalg.norm(_down(do))), (diff, mine)


def test_out_norm_without_tokens():
    pdn = _pdn()
    torch = torch_mod()
    e = lambda *s: torch.empty(s, device="cuda")
    pdn.pdn_out_norm_fwd(e(2, 3, 0, 64), e(2, 0, 3, 64))
    dw = _nan((64,))
    pdn.pdn_out_norm_bwd(e(2, 3, 0, 64), e(2, 0, 3, 64), e(2, 3, 0, 64), w=torch.ones(64, device="cuda"), dw=dw)
    assert bool((dw == 0).all())


# ---------------------------------------------------------------------------
# scan
# ---------------------------------------------------------------------------

SCAN = [  # B, T, D, type, type of log_a, gain, h0 / dhT, resets
    (1, 1, 8, "fp32", "fp32", 0, True, False),
    (2, 7, 64, "bf16", "bf16", 2, True, False),
    (1, 127, 72, "bf16", "fp32", 1, False, True),
    (3, 128, 520, "fp32", "fp32", 2, True, False),
    (1, 129, 64, "bf16", "bf16", 0, True, True),
    (2, 256, 136, "bf16", "fp32", 2, True, False),
    (1, 257, 8, "fp32", "fp32", 1, True, False),
    (2, 1000, 200, "bf16", "bf16", 2, True, True),
    (1, 2049, 136, "fp32", "fp32", 0, True, False),
    (5, 515, 64, "bf16", "fp32", 1, False, False),
    (1, 20011, 64, "bf16", "bf16", 2, True, False),
    (2, 9000, 24, "fp32", "fp32", 0, True, True),
    (3, 700, 520, "bf16", "fp32", 1, True, True),      # more columns than have carriers
    (9, 3001, 72, "fp32", "fp32", 2, True, False),
    # a bf16 forward tile, one token less and more, and lengths that are multiples of both directions'
    (1, 191, 64, "bf16", "bf16", 1, True, False),
    (2, 192, 136, "bf16", "fp32", 2, True, True),
    (1, 193, 72, "bf16", "bf16", 0, True, False),
    (3, 576, 520, "bf16", "bf16", 2, True, True),
    (1, 6145, 64, "bf16", "fp32", 0, True, False),     # 32 whole tiles and a token: a carrier's round and one more
]


def _scan_ids(c):
    return "B%d-T%d-D%d-%s-%s-g%d%s%s" % (c[:6] + ("-state" if c[6] else "", "-resets" if c[7] else ""))


def _scan_case(case, seed):
    B, T, D, dt, lt, kind, state, resets = case
    rng = np.random.default_rng(seed)
    x, dh = _draw(rng, (B, T, D), dt), _draw(rng, (B, T, D), dt)
    # channels from short memories to nearly none lost
    rate = np.exp(rng.uniform(np.log(2e-4), np.log(3.0), D))
    la = -(rate * rng.uniform(0.1, 1.0, (B, T, D))).astype(np.float32)
    if resets:
        for b in range(B):
            at = rng.integers(0, T, 1 + T // 300)
            la[b, at] = -np.inf
        la[rng.random((B, T, D)) < 0.002] = -200.0     # e^-200 is zero in fp32
    if lt == "bf16":
        la = ref.bf16(la)
    h0 = rng.standard_normal((B, D)).astype(np.float32) if state else None
    dhT = rng.standard_normal((B, D)).astype(np.float32) if state else None
    return x, la, h0, dh, dhT


def _views(t, pad, lead):
    """t [B,T,D] as a view into wider rows, `lead` elements in."""
    torch = torch_mod()
    B, T, D = t.shape
    wide = torch.full((B, T, D + pad), 7.0, device="cuda", dtype=t.dtype)
    v = wide[:, :, lead:lead + D]
    v.copy_(t)
    return v, wide


@pytest.mark.parametrize("case", SCAN, ids=_scan_ids)
def test_scan(case):
    """Forward (state, marks) and backward, with the forward's marks and without."""
    pdn = _pdn()
    torch = torch_mod()
    B, T, D, dt, lt, kind, state, _ = case
    x, la, h0, dh, dhT = _scan_case(case, 220)
    f64 = lambda v: None if v is None else v.astype(np.float64)
    xd, _w = _views(_up(x, dt), 24, 8)
    lad, _w2 = _views(_up(la, lt), 8, 0)
    h, wide = _views(_nan((B, T, D), dt), 16, 8)
    h0d = _up(h0) if state else None
    hT, marks = _nan((B, D)), _nan((B, pdn.pdn_scan_marks(T), D))
    print("[around] scan forward %s" % (case,), flush=True)
    pdn.pdn_scan_fwd(xd, lad, h, h0=h0d, hT=hT, marks=marks, gain=kind)
    want, bound = ref.scan_fwd(f64(x), f64(la), f64(h0), kind)
    _close("scan h", h, want, bound, dt)
    _close("scan hT", hT, want[:, -1], bound[:, -1])
    assert bool((wide[:, :, :8] == 7.0).all()) and bool((wide[:, :, 8 + D:] == 7.0).all())
    at = np.arange(0, T, pdn.PDN_SCAN_MARK)
    first = np.zeros((B, 1, D)) if h0 is None else f64(h0)[:, None]
    before, beforeb = (np.concatenate([f, v[:, :-1]], 1)[:, at] for f, v in ((first, want), (0 * first, bound)))
    _close("scan marks", marks, before, beforeb)

    refs = ref.scan_bwd(f64(x), f64(la), f64(h0), f64(dh), f64(dhT), kind)
    dhd, _w3 = _views(_up(dh, dt), 8, 8)
    got = []
    for given in (marks, None):
        dx, dxw = _views(_nan((B, T, D), dt), 8, 0)
        dla, _w4 = _views(_nan((B, T, D), lt), 16, 8)
        dh0 = _nan((B, D))
        print("[around] scan backward, marks %s" % ("given" if given is not None else "formed"), flush=True)
        pdn.pdn_scan_bwd(xd, lad, dhd, dx, dla, h0=h0d, dhT=_up(dhT) if state else None, dh0=dh0, marks=given, gain=kind)
        for name, t, (w, b), ty in (("dx", dx, refs[0], dt), ("dlog_a", dla, refs[1], lt), ("dh0", dh0, refs[2], "fp32")):
            _close("scan " + name, t, w, b, ty)
        assert bool((dxw[:, :, D:] == 7.0).all())
        got.append((dx.clone(), dla.clone(), dh0))
    for a, b in zip(*got):
        assert torch.equal(a, b), "the backward depends on who formed the marks"


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_scan_step_is_the_scan(kind):
    """Steps one after another, in place, give the scan's states."""
    pdn = _pdn()
    case = (3, 9, 136, "bf16", "fp32", kind, True, True)
    x, la, h0, _, _ = _scan_case(case, 221)
    want, bound = ref.scan_fwd(x.astype(np.float64), la.astype(np.float64), h0.astype(np.float64), kind)
    s, xd, lad = _up(h0), _up(x, "bf16"), _up(la)
    for t in range(9):
        h = _nan((3, 136), "bf16")
        pdn.pdn_scan_step(xd[:, t], lad[:, t], h, s, s, gain=kind)
        _close("step %d h" % t, h, want[:, t], bound[:, t], "bf16")
        _close("step %d state" % t, s, want[:, t], bound[:, t])


def test_scan_reset_drops_infinities_and_nan():
    """Nothing from before a zero decay, in either direction, whatever it holds."""
    pdn = _pdn()
    case = (2, 700, 64, "fp32", "fp32", 0, True, False)
    x, la, h0, dh, dhT = _scan_case(case, 222)
    at = 401
    la[:, at] = -np.inf
    bad_x, bad_dh, bad_h0 = x.copy(), dh.copy(), h0.copy()
    bad_x[0, 17], bad_x[1, 399], bad_h0[0, :9] = np.nan, np.inf, np.inf
    bad_dh[0, 500], bad_dh[1, 699] = np.nan, -np.inf
    la[1, 350, 5] = np.nan
    good_la = np.where(np.isnan(la), -0.5, la)

    def both(xv, lav, hv, gv):
        xd, lad, hd, gd = _up(xv), _up(lav), _up(hv), _up(gv)
        h, hT, dx, dla, dh0 = _nan((2, 700, 64)), _nan((2, 64)), _nan((2, 700, 64)), _nan((2, 700, 64)), _nan((2, 64))
        pdn.pdn_scan_fwd(xd, lad, h, h0=hd, hT=hT)
        pdn.pdn_scan_bwd(xd, lad, gd, dx, dla, h0=hd, dhT=_up(dhT), dh0=dh0)
        return [_down(t) for t in (h, hT, dx, dla, dh0)]

    good = both(x, good_la, h0, dh)
    bad = both(bad_x, la, bad_h0, dh)           # poison before the reset: the forward after it is untouched
    np.testing.assert_array_equal(bad[0][:, at:], good[0][:, at:])
    np.testing.assert_array_equal(bad[1], good[1])
    assert not np.isfinite(bad[0][0, 20]).any() and not np.isfinite(bad[0][1, 399]).any()
    np.testing.assert_array_equal(bad[2][:, at:], good[2][:, at:])
    np.testing.assert_array_equal(bad[3][:, at:], good[3][:, at:])
    assert (good[3][:, at] == 0).all()          # the reset's own decay has no gradient
    bad = both(x, good_la, h0, bad_dh)          # poison behind it: the gradients before it are untouched
    np.testing.assert_array_equal(bad[2][:, :at], good[2][:, :at])
    np.testing.assert_array_equal(bad[3][:, :at], good[3][:, :at])
    np.testing.assert_array_equal(bad[4], good[4])
    assert not np.isfinite(bad[2][0, 450]).any()


def test_scan_packed_row_equals_its_sequences():
    pdn = _pdn()
    torch = torch_mod()
    lengths = [1, 255, 3, 600, 128]
    T, D = sum(lengths), 72
    x, la, _, _, _ = _scan_case((1, T, D, "bf16", "fp32", 2, False, False), 223)
    starts = np.cumsum([0] + lengths[:-1])
    packed = la.copy()
    packed[:, starts] = -np.inf
    h = _nan((1, T, D), "bf16")
    pdn.pdn_scan_fwd(_up(x, "bf16"), _up(packed), h, gain=2)
    want = np.concatenate([ref.scan_fwd(x[:, s:s + n].astype(np.float64), packed[:, s:s + n].astype(np.float64), None, 2)[0]
                           for s, n in zip(starts, lengths)], 1)
    bound = ref.scan_fwd(x.astype(np.float64), packed.astype(np.float64), None, 2)[1]
    _close("packed h", h, want, bound, "bf16")
    assert torch.equal(h, h.clone())


def test_scan_without_tokens_and_states_in_place():
    pdn = _pdn()
    torch = torch_mod()
    e = lambda *s: torch.empty(s, device="cuda")
    h0, hT, dh0 = torch.randn(2, 16, device="cuda"), _nan((2, 16)), _nan((2, 16))
    pdn.pdn_scan_fwd(e(2, 0, 16), e(2, 0, 16), e(2, 0, 16), h0=h0, hT=hT, marks=e(2, 0, 16))
    assert torch.equal(hT, h0)
    pdn.pdn_scan_fwd(e(2, 0, 16), e(2, 0, 16), e(2, 0, 16), hT=hT)
    assert bool((hT == 0).all())
    pdn.pdn_scan_bwd(e(2, 0, 16), e(2, 0, 16), e(2, 0, 16), e(2, 0, 16), e(2, 0, 16), dhT=h0, dh0=dh0)
    assert torch.equal(dh0, h0)
    x, la, h0n, dh, dhT = _scan_case((2, 900, 64, "fp32", "fp32", 1, True, False), 224)
    xd, lad, s, c = _up(x), _up(la), _up(h0n), _up(dhT)
    h, dx, dla, out, dh0 = _nan((2, 900, 64)), _nan((2, 900, 64)), _nan((2, 900, 64)), _nan((2, 64)), _nan((2, 64))
    pdn.pdn_scan_fwd(xd, lad, h, h0=_up(h0n), hT=out, gain=1)
    pdn.pdn_scan_fwd(xd, lad, h, h0=s, hT=s, gain=1)
    assert torch.equal(out, s)
    pdn.pdn_scan_bwd(xd, lad, _up(dh), dx, dla, h0=_up(h0n), dhT=c, dh0=dh0, gain=1)
    pdn.pdn_scan_bwd(xd, lad, _up(dh), dx, dla, h0=_up(h0n), dhT=c, dh0=c, gain=1)
    assert torch.equal(dh0, c)


def test_scan_repeats_bit_for_bit_and_splits():
    """Many columns and tiles, several times: the same bits whatever the
    timing; and a row cut in two with the state carried over, within bounds."""
    pdn = _pdn()
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(225)
    B, T, D = 2, 6000, 1032
    x = torch.randn((B, T, D), generator=gen, device="cuda").to(torch.bfloat16)
    la = -0.05 * torch.rand((B, T, D), generator=gen, device="cuda")
    h0 = torch.randn((B, D), generator=gen, device="cuda")
    first = None
    for _ in range(5):
        h, hT = torch.full_like(x, float("nan")), _nan((B, D))
        dx, dla, dh0 = torch.full_like(x, float("nan")), torch.full_like(la, float("nan")), _nan((B, D))
        pdn.pdn_scan_fwd(x, la, h, h0=h0, hT=hT, gain=2)
        pdn.pdn_scan_bwd(x, la, x, dx, dla, h0=h0, dhT=h0, dh0=dh0, gain=2)
        out = [h, hT, dx, dla, dh0]
        if first is None:
            first = out
        for a, b in zip(out, first):
            assert torch.equal(a, b)
    cut, s = 2500, _nan((B, D))
    h = torch.full_like(x, float("nan"))
    pdn.pdn_scan_fwd(x[:, :cut], la[:, :cut], h[:, :cut], h0=h0, hT=s, gain=2)
    pdn.pdn_scan_fwd(x[:, cut:], la[:, cut:], h[:, cut:], h0=s, hT=s, gain=2)
    # both within some 32 U of sums of about 40 states' worth of terms
    assert float((s - first[1]).abs().max()) < 1e-4
    assert float((h.float() - first[0].float()).abs().max()) < 2.0 ** -5


def test_scan_gradient_by_differences():
    pdn = _pdn()
    x, la, h0, dh, dhT = _scan_case((1, 300, 8, "fp32", "fp32", 2, True, False), 226)
    la = np.minimum(la, -0.02)   # away from the gain's unbounded slope

    def loss(xs, ls, hs):
        h, hT = _nan((1, 300, 8)), _nan((1, 8))
        pdn.pdn_scan_fwd(_up(xs.astype(np.float32)), _up(ls.astype(np.float32)), h, h0=_up(hs.astype(np.float32)), hT=hT, gain=2)
        return float((_down(h) * dh).sum() + (_down(hT) * dhT).sum())

    dx, dla, dh0 = _nan((1, 300, 8)), _nan((1, 300, 8)), _nan((1, 8))
    pdn.pdn_scan_bwd(_up(x), _up(la), _up(dh), dx, dla, h0=_up(h0), dhT=_up(dhT), dh0=dh0, gain=2)
    rng, step = np.random.default_rng(227), 2.0 ** -6
    for _ in range(6):
        v = [rng.standard_normal(a.shape) for a in (x, la, h0)]
        v = [a / np.linalg.norm(a) for a in v]
        v[1] *= 0.05
        diff = (loss(x + step * v[0], la + step * v[1], h0 + step * v[2]) - loss(x - step * v[0], la - step * v[1], h0 - step * v[2])) / (2 * step)
        mine = (_down(dx) * v[0]).sum() + (_down(dla) * v[1]).sum() + (_down(dh0) * v[2]).sum()
        size = np.linalg.norm(_down(dx)) + 0.05 * np.linalg.norm(_down(dla)) + np.linalg.norm(_down(dh0))
        assert abs(diff - mine) < 5e-3 * max(1.0, size), (diff, mine)


# ---------------------------------------------------------------------------
# streams, graphs, refusals, and the operators together
# ---------------------------------------------------------------------------

def test_another_stream_and_its_workspace():
    """Calls on a stream that is not torch's current one, given as an object and
    as a handle, their workspaces made here."""
    pdn = _pdn()
    torch = torch_mod()
    x, la, h0, dh, dhT = _scan_case((2, 3001, 264, "bf16", "fp32", 2, True, False), 230)
    xd, lad, h0d, dhd = _up(x, "bf16"), _up(la), _up(h0), _up(dh, "bf16")
    want = [_nan((2, 3001, 264), "bf16"), _nan((2, 3001, 264), "bf16"), _nan((2, 3001, 264))]
    pdn.pdn_scan_fwd(xd, lad, want[0], h0=h0d, gain=2)
    pdn.pdn_scan_bwd(xd, lad, dhd, want[1], want[2], h0=h0d, gain=2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0, torch.cuda.default_stream()):
        got = [torch.zeros_like(t) for t in want]
        side.wait_stream(torch.cuda.current_stream())
        pdn.pdn_scan_fwd(xd, lad, got[0], h0=h0d, gain=2, stream=stream)
        pdn.pdn_scan_bwd(xd, lad, dhd, got[1], got[2], h0=h0d, gain=2, stream=stream)
        # the current stream allocates and writes meanwhile
        junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del junk


def test_two_scans_at_once():
    """Two calls on two streams, a workspace each."""
    pdn = _pdn()
    torch = torch_mod()
    ins = [_scan_case((1, 8000, 520, "bf16", "bf16", 0, True, False), s) for s in (231, 232)]
    ins = [(_up(x, "bf16"), _up(la, "bf16"), _up(h0)) for x, la, h0, _, _ in ins]
    want = []
    for x, la, h0 in ins:
        want.append(torch.empty_like(x))
        pdn.pdn_scan_fwd(x, la, want[-1], h0=h0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(3):
        got = [torch.zeros_like(x) for x, _, _ in ins]
        torch.cuda.synchronize()
        for (x, la, h0), out, s in zip(ins, got, streams):
            pdn.pdn_scan_fwd(x, la, out, h0=h0, stream=s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_graphs_sharing_a_workspace():
    """Each call captured and replayed, two graphs on one workspace in turn,
    with eager work between the replays."""
    pdn = _pdn()
    torch = torch_mod()
    x, la, h0, dh, dhT = _scan_case((2, 1500, 136, "bf16", "bf16", 2, True, True), 233)
    xd, lad, h0d, dhd, dhTd = _up(x, "bf16"), _up(la, "bf16"), _up(h0), _up(dh, "bf16"), _up(dhT)
    h, hT = _nan((2, 1500, 136), "bf16"), _nan((2, 136))
    dx, dla, dh0 = _nan((2, 1500, 136), "bf16"), _nan((2, 1500, 136), "bf16"), _nan((2, 136))
    (xq, xk), kw, _, _, _, rng = _qk_case(QK[2], 234)
    B, T, Hq, Hk, H, d = QK[2][:6]
    q, k = _nan((B, H, T, d), "bf16"), _nan((B, H, T, d), "bf16")
    gq, gk = _up(_draw(rng, (B, H, T, d), "fp32")), _up(_draw(rng, (B, H, T, d), "fp32"))
    dxq, dxk = _nan((B, T, Hq, d), "bf16"), _nan((B, T, Hk, d), "bf16")
    dwq, dwk = _nan((d,)), _nan((d,))
    o, zd, _, w, rng = _out_case(OUT[1], 235)
    od, wd, y = _up(o), _up(w), _nan((2, 5, 3, 128), "bf16")
    dyd, do, dz, dw = _up(_draw(rng, (2, 5, 3, 128), "bf16"), "bf16"), _nan((2, 3, 5, 128)), _nan((2, 5, 3, 128), "bf16"), _nan((128,))
    n = max(pdn.pdn_scan_bwd_workspace_size(xd, lad, dhd, dx, dla, h0=h0d, dhT=dhTd, dh0=dh0, gain=2),
            pdn.pdn_qk_norm_bwd_workspace_size(xq, xk, gq, gk, dxq, dxk, dwq=dwq, dwk=dwk, **kw),
            pdn.pdn_out_norm_bwd_workspace_size(od, dyd, do, z=zd, dz=dz, w=wd, dw=dw))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def forward():
        pdn.pdn_scan_fwd(xd, lad, h, h0=h0d, hT=hT, gain=2, workspace=ws)
        pdn.pdn_qk_norm_fwd(xq, xk, q, k, **kw)
        pdn.pdn_out_norm_fwd(od, y, z=zd, w=wd)

    def backward():
        pdn.pdn_scan_bwd(xd, lad, dhd, dx, dla, h0=h0d, dhT=dhTd, dh0=dh0, gain=2, workspace=ws)
        pdn.pdn_qk_norm_bwd(xq, xk, gq, gk, dxq, dxk, dwq=dwq, dwk=dwk, workspace=ws, **kw)
        pdn.pdn_out_norm_bwd(od, dyd, do, z=zd, dz=dz, w=wd, dw=dw, workspace=ws)

    outs = [h, hT, q, k, y, dx, dla, dh0, dxq, dxk, dwq, dwk, do, dz, dw]
    forward()
    backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward()
        backward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for call in (forward, backward):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for rep in range(4):
        for t in outs:
            t.fill_(float("nan"))
        ws.fill_(rep * 85)
        torch.cuda.synchronize()
        for g in graphs if rep % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), "replay %d, output %d" % (rep, i)


def test_decode_layouts_meet():
    """One token: q and k as pdn_decode_step takes them, o as it leaves it."""
    pdn = _pdn()
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(236)
    B, H, d = 5, 4, 128
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    rows = rnd(B, 1, 4 * H * d).to(torch.bfloat16)
    part = lambda i: rows[:, :, i * H * d:(i + 1) * H * d].unflatten(2, (H, d))
    q, k = (torch.empty((B, H, 1, d), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    pdn.pdn_qk_norm_fwd(part(0), part(1), q, k, q_scale=d ** -0.5)
    S, o = rnd(B, H, d, d) * 0.1, torch.empty((B, H, d), device="cuda")
    S64 = S.double()
    beta, la = torch.rand((B, H), generator=gen, device="cuda"), -torch.rand((B, H), generator=gen, device="cuda")
    v = part(2)[:, 0].contiguous()
    pdn.pdn_decode_step(q[:, :, 0], k[:, :, 0], v, o, S, log_alpha=la, beta=beta)
    y, w = torch.empty((B, 1, H, d), device="cuda"), torch.ones(d, device="cuda")
    pdn.pdn_out_norm_fwd(o.unsqueeze(2), y, z=part(3).float(), w=w)
    q64, k64, v64 = q[:, :, 0].double(), k[:, :, 0].double(), v.double()
    A = S64 * la.double().exp()[..., None, None]
    kt, vt = k64 * beta.double().sqrt()[..., None], v64 * beta.double().sqrt()[..., None]
    S1 = A + kt[..., None] * (vt - (A * kt[..., None]).sum(2))[:, :, None]
    o64 = (S1 * q64[..., None]).sum(2)
    n = o64 / (o64.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    z = part(3)[:, 0].double()
    want = n * z * torch.sigmoid(z)
    err = float((y[:, 0].double() - want).norm() / want.norm())
    print("[around] decode chain rel %.2e" % err, flush=True)
    assert err < 1e-5   # the bound of the recurrence's fp32 decode


def test_a_layer_trains():
    """The operators as a layer uses them: the vector-state scan mixes the
    projected stream in time, q and k are normed and rotated out of it, the
    delta rule runs, its output goes through the gated norm; then backward
    through all of it, against fp64 autograd of the whole (token by token)."""
    pdn = _pdn()
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(237)
    B, T, H, d = 1, 150, 2, 128
    D = 2 * H * d
    rnd = lambda *s, sc=1.0: (torch.randn(s, generator=gen, device="cuda") * sc)
    x, la = rnd(B, T, D), -0.3 * torch.rand((B, T, D), generator=gen, device="cuda") - 0.01
    v, z = rnd(B, H, T, d), rnd(B, T, H, d)
    beta = torch.rand((B, H, T), generator=gen, device="cuda") * 0.8 + 0.1
    log_alpha = -0.2 * torch.rand((B, H, T), generator=gen, device="cuda")
    wq, wk, w = 1 + rnd(d, sc=0.1), 1 + rnd(d, sc=0.1), 1 + rnd(d, sc=0.1)
    dy = rnd(B, T, H, d)
    freqs, rs = pdn.pdn_rope_freqs(64, 10000.0, pdn.PDN_ROPE_BY_PARTS, 4.0, 64)
    inv = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    e = lambda *s: torch.full(s, float("nan"), device="cuda")
    kw = dict(norm=pdn.PDN_NORM_L2, wq=wq, wk=wk, q_scale=d ** -0.5, inv_freq=inv, rope_scale=rs)

    h, marks = e(B, T, D), e(B, pdn.pdn_scan_marks(T), D)
    pdn.pdn_scan_fwd(x, la, h, marks=marks, gain=pdn.PDN_GAIN_NORM)
    xq, xk = h[..., :H * d].unflatten(2, (H, d)), h[..., H * d:].unflatten(2, (H, d))
    q, k, o, y = e(B, H, T, d), e(B, H, T, d), e(B, H, T, d), e(B, T, H, d)
    pdn.pdn_qk_norm_fwd(xq, xk, q, k, **kw)
    pdn.pdn_chunk_fwd(q, k, v, o, log_alpha=log_alpha, beta=beta)
    pdn.pdn_out_norm_fwd(o, y, z=z, w=w)
    do, dz, dw = e(B, H, T, d), e(B, T, H, d), e(d)
    pdn.pdn_out_norm_bwd(o, dy, do, z=z, dz=dz, w=w, dw=dw)
    dq, dk, dv, dbeta, dlog = e(B, H, T, d), e(B, H, T, d), e(B, H, T, d), e(B, H, T), e(B, H, T)
    pdn.pdn_chunk_bwd(q, k, v, do, dq, dk, dv, dlog_alpha=dlog, dbeta=dbeta, log_alpha=log_alpha, beta=beta)
    dh, dwq, dwk = e(B, T, D), e(d), e(d)
    pdn.pdn_qk_norm_bwd(xq, xk, dq, dk, dh[..., :H * d].unflatten(2, (H, d)), dh[..., H * d:].unflatten(2, (H, d)),
                        dwq=dwq, dwk=dwk, **kw)
    dx, dla = e(B, T, D), e(B, T, D)
    pdn.pdn_scan_bwd(x, la, dh, dx, dla, marks=marks, gain=pdn.PDN_GAIN_NORM)
    torch.cuda.synchronize()

    names = "x la v z beta log_alpha wq wk w".split()
    t64 = {n: t.double().cpu().requires_grad_() for n, t in zip(names, (x, la, v, z, beta, log_alpha, wq, wk, w))}
    a = t64["la"].exp()
    b = torch.sqrt(-torch.expm1(2 * t64["la"])) * t64["x"]
    s, hs = torch.zeros(B, D, dtype=torch.float64), []
    for t in range(T):
        s = a[:, t] * s + b[:, t]
        hs.append(s)
    hh = torch.stack(hs, 1)
    ang = torch.arange(T, dtype=torch.float64)[:, None, None] * inv.cpu()
    cos, sin = ang.cos() * np.float32(rs).item(), ang.sin() * np.float32(rs).item()

    def head(u, wt, sc):
        n = u / torch.sqrt(u.square().sum(-1, keepdim=True) + 1e-6) * wt * sc
        i, j = n[..., :32], n[..., 32:64]
        return torch.cat([i * cos - j * sin, j * cos + i * sin, n[..., 64:]], -1).transpose(1, 2)

    qq = head(hh[..., :H * d].unflatten(2, (H, d)), t64["wq"], d ** -0.5)
    kk = head(hh[..., H * d:].unflatten(2, (H, d)), t64["wk"], 1.0)
    S, oo = torch.zeros(B, H, d, d, dtype=torch.float64), []
    for t in range(T):
        A = S * t64["log_alpha"][:, :, t].exp()[..., None, None]
        g = t64["beta"][:, :, t].sqrt()[..., None]
        kt, vt = kk[:, :, t] * g, t64["v"][:, :, t] * g
        S = A + kt[..., None] * (vt - (A * kt[..., None]).sum(2))[:, :, None]
        oo.append((S * qq[:, :, t, :, None]).sum(2))
    ob = torch.stack(oo, 1)
    yy = ob / torch.sqrt(ob.square().mean(-1, keepdim=True) + 1e-6) * t64["w"] * t64["z"] * torch.sigmoid(t64["z"])
    yy.backward(dy.double().cpu())
    got = dict(zip(names, (dx, dla, dv, dz, dbeta, dlog, dwq, dwk, dw)))
    rel = lambda p, r: float((p.double().cpu() - r).norm() / r.norm())
    errs = {"y": rel(y, yy.detach())}
    errs.update((n, rel(got[n], t64[n].grad)) for n in names)
    print("[around] layer: " + " ".join("%s=%.1e" % kv for kv in errs.items()), flush=True)
    # fp32 throughout: the recurrence's own fp32 bound, through four operators
    assert all(v < 4e-5 for v in errs.values()), errs


def test_tensors_are_refused():
    pdn = _pdn()
    torch = torch_mod()
    e = lambda *s, **k: torch.zeros(s, device="cuda", **k)
    with pytest.raises(ValueError, match="shape"):
        pdn.pdn_qk_norm_fwd(e(1, 4, 2, 64), e(1, 4, 2, 64), e(1, 2, 4, 64), e(1, 2, 5, 64))
    with pytest.raises(ValueError, match="last dimension"):
        pdn.pdn_scan_fwd(e(1, 8, 4).transpose(1, 2), e(1, 4, 8), e(1, 4, 8))
    with pytest.raises(ValueError, match="must be torch.float32"):
        pdn.pdn_scan_fwd(e(1, 4, 8), e(1, 4, 8), e(1, 4, 8), h0=e(1, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="device memory"):
        pdn.pdn_scan_fwd(e(1, 4, 8), torch.zeros(1, 4, 8), e(1, 4, 8))
    with pytest.raises(pdn.PdnError) as x:   # rows not 16-byte aligned
        pdn.pdn_scan_fwd(e(1, 4, 9)[:, :, :8], e(1, 4, 8), e(1, 4, 8))
    assert x.value.code == pdn.PDN_EINVAL
    with pytest.raises(pdn.PdnError) as x:   # an output whose rows lie on each other
        pdn.pdn_scan_fwd(e(1, 4, 8), e(1, 4, 8), e(1, 1, 8).expand(1, 4, 8))
    assert x.value.code == pdn.PDN_EINVAL
    with pytest.raises(pdn.PdnError) as x:
        pdn.pdn_scan_fwd(e(1, 4, 12), e(1, 4, 12), e(1, 4, 12))
    assert x.value.code == pdn.PDN_EUNSUPPORTED
    with pytest.raises(pdn.PdnError) as x:
        pdn.pdn_scan_fwd(e(1, 400, 8), e(1, 400, 8), e(1, 400, 8), workspace=e(4))
    assert x.value.code == pdn.PDN_EWORKSPACE
    with pytest.raises(pdn.PdnError) as x:
        pdn.pdn_out_norm_fwd(e(1, 1, 4, 64), e(1, 4, 1, 64), act=pdn.PDN_ACT_SILU)
    assert x.value.code == pdn.PDN_EINVAL


def test_repeated_inputs_are_read_in_place():
    """Stride 0: one decay row for all tokens, one input row for all sequences."""
    pdn = _pdn()
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(238)
    x, la = torch.randn((1, 300, 64), generator=gen, device="cuda"), -torch.rand((1, 1, 64), generator=gen, device="cuda")
    got, want = _nan((3, 300, 64)), _nan((3, 300, 64))
    pdn.pdn_scan_fwd(x.expand(3, 300, 64), la.expand(3, 300, 64), got)
    pdn.pdn_scan_fwd(x.expand(3, 300, 64).contiguous(), la.expand(3, 300, 64).contiguous(), want)
    assert torch.equal(got, want)
