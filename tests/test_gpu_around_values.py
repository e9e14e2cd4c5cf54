"""GPU checks of the operators around the recurrence at values, views and sizes that
the other suites pass over: decays of exactly one, infinities beside a rotation,
gates far from zero, slices of a longer buffer of positions, as many columns as a
launch holds, packed rows against their sequences alone."""
import numpy as np
import pytest

import around_ref as ref
from around_ref import U
from test_gpu_around import TINY, _close, _down, _nan, _pdn, _scan_case, _up
from gpu_util import torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 300])
def test_normed_gain_slope_at_a_decay_of_one(dtype, T):
    """sqrt(1 - a^2) falls ever steeper towards a = 1, where its derivative by
    log_a is -inf whichever zero log_a is: dlog_a is -inf times the sign of x G."""
    pdn = _pdn()
    rng = np.random.default_rng(400)
    D = 16
    x = rng.choice([-1.0, 2.0], (1, T, D)).astype(np.float32)
    la = np.full((1, T, D), -0.25, np.float32)
    at = T // 2
    la[:, at, ::2], la[:, at, 1::2] = 0.0, -0.0
    sign = rng.choice([-1.0, 1.0], (1, 1, D)).astype(np.float32)
    dh = np.broadcast_to(sign, x.shape).copy()       # every G of a channel has its sign
    xd, lad = _up(x, dtype), _up(la, dtype)
    dx, dla = _nan(x.shape, dtype), _nan(x.shape, dtype)
    pdn.pdn_scan_bwd(xd, lad, _up(dh, dtype), dx, dla, gain=pdn.PDN_GAIN_NORM)
    got = _down(dla)
    np.testing.assert_array_equal(got[:, at], -np.inf * (x * dh)[:, at])
    assert np.isfinite(np.delete(got, at, 1)).all()
    dx = _down(dx)
    assert (dx[:, at] == 0).all() and np.isfinite(dx).all()
    h = _nan(x.shape, dtype)
    pdn.pdn_scan_fwd(xd, lad, h, gain=pdn.PDN_GAIN_NORM)
    h = _down(h)
    np.testing.assert_array_equal(h[:, at], h[:, at - 1] if at else 0 * h[:, 0])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d,rot", [(64, 16), (128, 64), (128, 112)])
@pytest.mark.parametrize("layout", [0, 1])
def test_elements_behind_the_rotation_stay(layout, d, rot, dtype):
    """Without a norm an element behind rot_dim is its input times the scale, and
    no other element sees it: infinities and NaN there, forward and backward."""
    pdn = _pdn()
    rng = np.random.default_rng(401)
    B, T, H = 2, 19, 3
    x = rng.standard_normal((B, T, H, d)).astype(np.float32)
    if dtype == "bf16":
        x = ref.bf16(x)
    g = rng.standard_normal((B, H, T, d)).astype(np.float32)
    bad_x, bad_g = x.copy(), g.copy()
    for bad in (bad_x, bad_g):
        bad[0, 1, 2, rot + 3], bad[1, 2, 0, rot + 8], bad[1, 0, 1, d - 1] = np.inf, -np.inf, np.nan
    kw = dict(norm=pdn.PDN_NORM_NONE, q_scale=0.5, k_scale=2.0, rope_layout=layout,
              inv_freq=_up(10000.0 ** (-2.0 * np.arange(rot // 2) / rot)))

    def both(xv, gv):
        xd = _up(xv, dtype)
        q, k = _nan((B, H, T, d), dtype), _nan((B, H, T, d), dtype)
        pdn.pdn_qk_norm_fwd(xd, xd, q, k, **kw)
        dxq, dxk = _nan((B, T, H, d), dtype), _nan((B, T, H, d), dtype)
        pdn.pdn_qk_norm_bwd(xd, xd, _up(gv), _up(gv), dxq, dxk, **kw)
        return [_down(t) for t in (q, k, dxq, dxk)]

    for xv, gv in ((bad_x, g), (x, bad_g)):
        good, bad = both(x, g), both(xv, gv)
        for i, (a, b) in enumerate(zip(good, bad)):
            source, given = (xv.transpose(0, 2, 1, 3), x.transpose(0, 2, 1, 3)) if i < 2 else (gv.transpose(0, 2, 1, 3), g.transpose(0, 2, 1, 3))
            hit = ~np.isfinite(source)
            np.testing.assert_array_equal(b[hit], source[hit])      # inf stays inf, NaN NaN
            np.testing.assert_array_equal(b[~hit], a[~hit])
            behind = given[..., rot:].astype(np.float64) * (0.5, 2.0)[i % 2]
            if i >= 2 and dtype == "bf16":
                behind = ref.bf16(behind.astype(np.float32)).astype(np.float64)
            np.testing.assert_array_equal(a[..., rot:], behind)


def test_sigmoid_gate_gradient_far_from_zero():
    """dz = n f (1 - f) w dy keeps its relative accuracy where f is near one:
    2 |z| for the exponent's argument (its constant and its product), 12 for exp2,
    add and reciprocal of f and of 1 - f, 13 for the row's norm, 5 products."""
    pdn = _pdn()
    rng = np.random.default_rng(402)
    B, H, T, dv = 1, 2, 40, 32
    o = rng.standard_normal((B, H, T, dv)).astype(np.float32)
    z = rng.uniform(-80.0, 80.0, (B, T, H, dv)).astype(np.float32)
    z[0, 0, 0, :4] = [17.5, 20.0, 60.0, -60.0]
    dy = rng.choice([-1.0, 1.0], (B, T, H, dv)).astype(np.float32) * rng.uniform(0.5, 2.0, (B, T, H, dv)).astype(np.float32)
    w = (1 + 0.2 * rng.standard_normal(dv)).astype(np.float32)
    do, dz, dw = _nan((B, H, T, dv)), _nan((B, T, H, dv)), _nan((dv,))
    pdn.pdn_out_norm_bwd(_up(o), _up(dy), do, z=_up(z), dz=dz, w=_up(w), dw=dw, act=pdn.PDN_ACT_SIGMOID)
    x, z64 = o.astype(np.float64).transpose(0, 2, 1, 3), z.astype(np.float64)
    r = ref.norm_factor(x, 1, float(np.float32(1e-6)))[0]
    want = dy * x * r * w.astype(np.float64) / (1 + np.exp(-z64)) / (1 + np.exp(z64))
    _close("sigmoid dz", dz, want, np.abs(want) * (32 + 2 * np.abs(z64)) * U)


@pytest.mark.parametrize("B,H,d,dtype", [(1, 4, 128, "bf16"), (1, 2, 64, "fp32")])
def test_positions_sliced_from_a_longer_buffer(B, H, d, dtype):
    """A generation loop takes positions[:, t:t + 1] of one buffer, a prefill in
    parts positions[:, s:e]: such slices are contiguous and begin anywhere."""
    pdn = _pdn()
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(403)
    T = 9
    x = torch.randn((B, T, 2, H, d), generator=gen, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    g = torch.randn((2, B, H, T, d), generator=gen, device="cuda")
    positions = 1000 + 7 * torch.arange(T, device="cuda")[None]
    table = torch.tensor([0.0] + pdn.pdn_rope_freqs(d)[0], dtype=torch.float64, device="cuda")
    w = torch.ones(d, device="cuda")

    def run(s, e, inv, stream=None):
        kw = dict(norm=pdn.PDN_NORM_RMS, inv_freq=inv, positions=positions[:, s:e], wq=w, wk=w)
        xq, xk = x[:, s:e, 0], x[:, s:e, 1]
        q, k = (torch.full((B, H, e - s, d), float("nan"), device="cuda", dtype=x.dtype) for _ in range(2))
        dxq, dxk = (torch.full((B, e - s, H, d), float("nan"), device="cuda", dtype=x.dtype) for _ in range(2))
        dq, dk = g[0][:, :, s:e].contiguous(), g[1][:, :, s:e].contiguous()
        dwq, dwk = _nan((d,)), _nan((d,))
        if stream is not None:
            torch.cuda.synchronize()
        pdn.pdn_qk_norm_fwd(xq, xk, q, k, stream=stream, **kw)
        assert pdn.pdn_qk_norm_bwd_workspace_size(xq, xk, dq, dk, dxq, dxk, dwq=dwq, dwk=dwk, **kw) > 0
        pdn.pdn_qk_norm_bwd(xq, xk, dq, dk, dxq, dxk, dwq=dwq, dwk=dwk, stream=stream, **kw)
        if stream is not None:
            junk = [torch.full((64,), -1, device="cuda", dtype=torch.int64) for _ in range(16)]  # nothing of the call's is free yet
            torch.cuda.synchronize()
            del junk
        return q, k, dxq, dxk

    inv = table[1:].clone()
    whole = run(0, T, inv)
    side = torch.cuda.Stream()
    parts = [(t, t + 1) for t in range(T)] + [(1, 4), (3, T), (2, 8)]
    for s, e in parts:
        for iv, stream in ((inv, None), (table[1:], None), (inv, side), (inv, side.cuda_stream), (table[1:], 0)):
            got = run(s, e, iv, stream)
            for name, a, b in zip(("q", "k"), got, whole):
                assert torch.equal(a, b[:, :, s:e]), (name, s, e)
            for name, a, b in zip(("dxq", "dxk"), got[2:], whole[2:]):
                assert torch.equal(a, b[:, s:e]), (name, s, e)


def test_sliced_positions_captured():
    """The call in a graph reads the slice at every replay."""
    pdn = _pdn()
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(404)
    H, d = 2, 64
    x = torch.randn((1, 1, 2, H, d), generator=gen, device="cuda")
    buf = torch.zeros((1, 4), dtype=torch.int64, device="cuda")
    inv = torch.tensor(pdn.pdn_rope_freqs(d)[0], dtype=torch.float64, device="cuda")
    q, k, wq, wk = (_nan((1, H, 1, d)) for _ in range(4))
    call = lambda pos, a, b: pdn.pdn_qk_norm_fwd(x[:, :, 0], x[:, :, 1], a, b, inv_freq=inv, positions=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(buf[:, 1:2], q, k)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(buf[:, 1:2], q, k)
    for pos in (0, 5, 123456, 7):
        buf.fill_(-3)
        buf[0, 1] = pos
        q.fill_(float("nan"))
        k.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        call(torch.full((1, 1), pos, dtype=torch.int64, device="cuda"), wq, wk)
        assert torch.equal(q, wq) and torch.equal(k, wk), pos


@pytest.mark.parametrize("B", [5_000_000, (1 << 23) - 1])
def test_scan_of_as_many_columns_as_a_launch_holds(B):
    """One token of very many sequences: a workgroup each, and no other."""
    pdn = _pdn()
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(406)
    x, dh = (torch.randn((B, 1, 8), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    la = -torch.rand((B, 1, 8), generator=gen, device="cuda")
    h0, dhT = (torch.randn((B, 8), generator=gen, device="cuda") for _ in range(2))
    h, hT = torch.full_like(x, float("nan")), torch.full_like(h0, float("nan"))
    print("[around] scan of %d columns" % B, flush=True)
    pdn.pdn_scan_fwd(x, la, h, h0=h0, hT=hT, gain=pdn.PDN_GAIN_NORM)
    step_h, step = torch.empty_like(x[:, 0]), torch.empty_like(h0)
    pdn.pdn_scan_step(x[:, 0], la[:, 0], step_h, h0, step, gain=pdn.PDN_GAIN_NORM)
    assert torch.equal(hT, step) and torch.equal(h[:, 0], step_h)
    dx, dla, dh0 = torch.full_like(x, float("nan")), torch.full_like(la, float("nan")), torch.full_like(h0, float("nan"))
    pdn.pdn_scan_bwd(x, la, dh, dx, dla, h0=h0, dhT=dhT, dh0=dh0)
    assert torch.equal(dx[:, 0], (dh[:, 0].float() + dhT).to(torch.bfloat16))     # one addition, one rounding
    # dlog_a = h0 dh0.  dlog_a: a h0, dh + dhT and their product are rounded, 3 U |a h0 (dh + dhT)|; dh0:
    # a dh is rounded before dhT joins it, U |a dh| whatever the sum cancels to, then their sum; a <= 1
    h0, dh, dhT = h0.double(), dh[:, 0].double(), dhT.double()
    room = U * h0.abs() * (5 * (dh + dhT).abs() + 2 * dh.abs()) + TINY
    assert bool(((dla[:, 0].double() - dh0.double() * h0).abs() <= room).all())


@pytest.mark.parametrize("D,lengths", [(72, [1, 255, 3, 600, 128]), (1160, [192, 96, 5, 700]), (8, [97, 1, 1, 400])])
def test_packed_row_against_its_sequences_alone(D, lengths):
    """A packed row's states are those of its sequences run one by one, each
    within the bounds of the definition: forward and backward."""
    pdn = _pdn()
    T = sum(lengths)
    x, la, _, dh, _ = _scan_case((1, T, D, "fp32", "fp32", 2, False, False), 405)
    starts = np.cumsum([0] + lengths[:-1])
    la[:, starts] = -np.inf
    f64 = lambda v: v.astype(np.float64)
    names = ("h", "dx", "dlog_a")

    def run(s, e):
        xd, lad = _up(x[:, s:e]), _up(la[:, s:e])
        h, dx, dla = (_nan((1, e - s, D)) for _ in names)
        pdn.pdn_scan_fwd(xd, lad, h, gain=2)
        pdn.pdn_scan_bwd(xd, lad, _up(dh[:, s:e]), dx, dla, gain=2)
        return h, dx, dla

    packed = run(0, T)
    bounds = (ref.scan_fwd(f64(x), f64(la), None, 2)[1],) + tuple(
        b for _, b in ref.scan_bwd(f64(x), f64(la), None, f64(dh), None, 2)[:2])
    for s, n in zip(starts, lengths):
        for name, a, b, bound in zip(names, run(s, s + n), packed, bounds):
            # each is off by its bound and its own rounding at most
            _close("packed " + name, b[:, s:s + n], _down(a), 2 * bound[:, s:s + n] + U * (np.abs(_down(a)) + bound[:, s:s + n]))
