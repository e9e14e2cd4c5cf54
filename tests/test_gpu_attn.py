"""GPU checks of causal softmax attention, forward and backward, element by element
against 64-bit references with bounds counted in roundings (block_ref.py): one query
to several tiles, shared heads, windows, packed and padded rows, queries that see
nothing, what is not finite and not seen, views, streams, graphs."""
import numpy as np
import pytest

import block_ref as ref
from block_ref import HALF
from gpu_util import torch_mod

pytestmark = pytest.mark.gpu
TINY = 1e-37


def _pdn():
    import gated_delta_rule_77_amd as pdn
    return pdn


def _dt(name):
    torch = torch_mod()
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rand(gen, *shape, dtype="fp32", scale=1.0):
    return (torch_mod().randn(shape, generator=gen) * scale).to(_dt(dtype)).cuda()


def _host(t):
    return t.detach().cpu().double()


def _close(name, got, want, bound, dtype):
    got = _host(got)
    torch = torch_mod()
    assert got.shape == want.shape
    if not want.numel():
        return
    same = torch.isinf(want) & (got == want)
    room = bound + HALF[dtype] * (want.abs() + bound) + TINY
    over = torch.where(same, torch.zeros_like(want), (got - want).abs() / room).max().item()
    print("[attn] %s: worst error %.2f of its bound" % (name, over), flush=True)
    assert np.isfinite(over) and over <= 1.0, "%s: %.3g times its bound" % (name, over)


def _nan(shape, dtype="fp32"):
    return torch_mod().full(shape, float("nan"), device="cuda", dtype=_dt(dtype))


# B, H, Hk, Tq, Tk, d, dtype, o and dO, gradients, window, first
CASES = [
    (1, 1, 1, 1, 1, 64, "bf16", "bf16", "bf16", 0, None),
    (1, 1, 1, 1, 1, 128, "fp32", "fp32", "fp32", 0, None),
    (2, 4, 2, 1, 333, 128, "bf16", "bf16", "bf16", 0, None),
    (2, 2, 1, 5, 5, 64, "bf16", "fp32", "fp32", 0, None),
    (1, 3, 1, 31, 33, 128, "bf16", "bf16", "bf16", 0, None),
    (1, 4, 4, 64, 64, 64, "bf16", "bf16", "bf16", 0, None),
    (2, 6, 2, 65, 65, 128, "bf16", "bf16", "fp32", 0, None),
    (1, 8, 1, 129, 129, 64, "fp32", "fp32", "fp32", 0, None),
    (1, 2, 2, 257, 300, 128, "bf16", "bf16", "bf16", 0, None),
    (1, 2, 1, 513, 513, 128, "bf16", "fp32", "bf16", 0, None),
    (1, 4, 2, 385, 385, 128, "fp32", "fp32", "fp32", 0, None),
    (1, 4, 2, 700, 700, 64, "bf16", "bf16", "bf16", 0, None),
    (2, 4, 2, 200, 200, 128, "bf16", "bf16", "bf16", 1, None),
    (1, 2, 2, 300, 300, 64, "bf16", "bf16", "bf16", 16, None),
    (1, 3, 3, 400, 460, 128, "fp32", "fp32", "fp32", 100, None),
    (1, 2, 1, 520, 520, 128, "bf16", "bf16", "bf16", 130, None),
    (2, 2, 1, 300, 300, 128, "bf16", "bf16", "bf16", 0, "packed"),
    (2, 4, 4, 333, 333, 64, "fp32", "fp32", "fp32", 50, "packed"),
    (3, 2, 2, 150, 170, 128, "bf16", "bf16", "bf16", 0, "padded"),
    (2, 2, 1, 190, 190, 64, "bf16", "fp32", "fp32", 20, "padded"),
    (1, 2, 2, 140, 140, 128, "bf16", "bf16", "bf16", 0, "any"),
    (1, 2, 2, 90, 40, 64, "bf16", "bf16", "bf16", 0, None),      # queries before the first key
    (1, 2, 1, 300, 10, 128, "fp32", "fp32", "fp32", 4, None),
    (1, 2, 1, 3, 2500, 128, "bf16", "bf16", "bf16", 0, None),    # keys dealt to several workgroups
    (1, 4, 2, 40, 1500, 64, "bf16", "bf16", "bf16", 0, "packed"),
    (1, 1, 1, 70, 1100, 128, "fp32", "fp32", "fp32", 900, None),
    (1, 12, 2, 37, 800, 64, "fp32", "fp32", "fp32", 0, "padded"),
]


def _first(kind, B, Tq, Tk, rng):
    """First keys: of packed sequences, of a padded batch (left padding, and queries that
    see nothing at the end), or anything at all."""
    if kind is None:
        return None
    out = np.zeros((B, Tq), np.int32)
    off = Tk - Tq
    for b in range(B):
        if kind == "packed":
            at = 0
            while at < Tk:
                n = int(rng.integers(1, 90))
                out[b, max(0, at - off):max(0, at - off + n)] = at
                at += n
        elif kind == "padded":
            out[b] = int(rng.integers(0, Tk // 2))
            out[b, Tq - int(rng.integers(0, Tq // 2)):] = Tk + b
        else:
            out[b] = rng.choice([-2 ** 31, -5, 0, 3, 31, 32, 64, 100, Tk - 1, Tk, Tk + 9, 2 ** 31 - 1], Tq)
    return out


def _make(case, seed):
    torch = torch_mod()
    B, H, Hk, Tq, Tk, d, dtype, odtype, gdtype, window, kind = case
    gen = torch.Generator().manual_seed(seed)
    # q and k as the recurrence's layout, v and o in the projection's
    q, k = _rand(gen, B, H, Tq, d, dtype=dtype, scale=1.5), _rand(gen, B, Hk, Tk, d, dtype=dtype)
    v = _rand(gen, B, Tk, 2 * Hk, d, dtype=dtype)[:, :, Hk:].transpose(1, 2)
    do = _rand(gen, B, Tq, H, d, dtype=odtype).transpose(1, 2)
    first = _first(kind, B, Tq, Tk, np.random.default_rng(seed))
    f = None if first is None else torch.from_numpy(first)
    mask = ref.seen(Tq, Tk, window, f)
    return gen, q, k, v, do, None if f is None else f.cuda(), mask


ids = lambda c: "B%d-H%d.%d-T%d.%d-d%d-%s-%s-%s-w%d-%s" % c  # noqa: E731


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_attn(case):
    torch, pdn = torch_mod(), _pdn()
    B, H, Hk, Tq, Tk, d, dtype, odtype, gdtype, window, kind = case
    gen, q, k, v, do, first, mask = _make(case, 21)
    scale = 0.11
    o, lse = _nan((B, Tq, H, d), odtype).transpose(1, 2), _nan((B, H, Tq))
    same = dict(scale=scale, window=window, first=first)
    ws = torch.full((pdn.pdn_attn_fwd_workspace_size(q, k, v, o, lse=lse, **same),), 255, dtype=torch.uint8, device="cuda")
    pdn.pdn_attn_fwd(q, k, v, o, lse=lse, workspace=ws, **same)
    torch.cuda.synchronize()
    s32 = float(np.float32(scale))
    want = ref.attn(_host(q), _host(k), _host(v), s32, mask, dtype)
    _close("o", o, want["o"], want["bo"], odtype)
    _close("lse", lse, want["lse"], want["bl"], "fp32")
    o2 = torch.empty_like(o)
    pdn.pdn_attn_fwd(q, k, v, o2, **same)  # no lse, no workspace of the caller's: the same bits
    assert torch.equal(o, o2)

    dq, dk, dv = _nan((B, H, Tq, d), gdtype), _nan((B, Hk, Tk, d), gdtype), _nan((B, Tk, Hk, d), gdtype).transpose(1, 2)
    ws = torch.full((pdn.pdn_attn_bwd_workspace_size(q, k, v, o, do, lse, dq, dk, dv, **same),), 255, dtype=torch.uint8, device="cuda")
    pdn.pdn_attn_bwd(q, k, v, o, do, lse, dq, dk, dv, workspace=ws, **same)
    torch.cuda.synchronize()
    # the gradient through the o that the forward kept
    want = ref.attn_bwd(_host(q), _host(k), _host(v), _host(o), _host(do), s32, mask, dtype, dtype == "bf16" and odtype == "fp32", odtype)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _close(n, t, *want[n], gdtype)
    again = [torch.empty_like(t) for t in (dq, dk, dv)]
    pdn.pdn_attn_bwd(q, k, v, o, do, lse, *again, **same)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dv)))


def test_no_queries_and_no_keys():
    torch, pdn = torch_mod(), _pdn()
    e = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    pdn.pdn_attn_fwd(e(1, 2, 0, 64), e(1, 2, 9, 64), e(1, 2, 9, 64), e(1, 2, 0, 64))
    dq, dk, dv = e(1, 2, 0, 64), e(1, 2, 9, 64), e(1, 2, 9, 64)
    pdn.pdn_attn_bwd(e(1, 2, 0, 64), e(1, 2, 9, 64), e(1, 2, 9, 64), e(1, 2, 0, 64), e(1, 2, 0, 64), torch.empty(1, 2, 0, device="cuda"), dq, dk, dv)
    assert not dk.any() and not dv.any()
    o, lse = e(1, 2, 5, 64), torch.ones(1, 2, 5, device="cuda")
    none = e(1, 1, 0, 64)
    pdn.pdn_attn_fwd(e(1, 2, 5, 64), none, none, o, lse=lse)
    assert not o.any() and (lse == -float("inf")).all()
    dq = e(1, 2, 5, 64)
    pdn.pdn_attn_bwd(e(1, 2, 5, 64), none, none, o, e(1, 2, 5, 64), lse, dq, e(1, 1, 0, 64), e(1, 1, 0, 64))
    assert not dq.any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_what_is_not_seen_has_no_part(dtype, d, bad):
    """Keys, values, queries and dO that are not finite, where a mask hides them: after
    a query, before its window or its first key, or of queries that see nothing."""
    torch, pdn = torch_mod(), _pdn()
    bad = float(bad)
    T, at, window = 230, 117, 60
    gen = torch.Generator().manual_seed(31)
    q, k, v, do = (_rand(gen, 1, 2, T, d, dtype=dtype) for _ in range(4))
    first = torch.zeros(1, T, dtype=torch.int32, device="cuda")
    first[0, 200:] = T  # these see nothing

    def both(q, k, v, do):
        o, lse = torch.empty_like(q), torch.empty(1, 2, T, device="cuda")
        pdn.pdn_attn_fwd(q, k, v, o, lse=lse, window=window, first=first)
        g = [torch.empty_like(q) for _ in range(3)]
        pdn.pdn_attn_bwd(q, k, v, o, do, lse, *g, window=window, first=first)
        return [o, lse, *g]

    clean = both(q, k, v, do)
    blind = torch.arange(T, device="cuda") >= 200
    # a key and its value that only the queries at .. at + window - 1 see
    for which in (1, 2):
        args = [t.clone() for t in (q, k, v, do)]
        args[which][:, :, at, 3] = bad
        got = both(*args)
        hit = torch.zeros(T, dtype=torch.bool, device="cuda")
        hit[at:at + window] = True
        assert torch.equal(got[0][:, :, ~hit], clean[0][:, :, ~hit])
        if which == 2 or bad != bad:
            assert not torch.isfinite(got[0][:, :, hit][..., 3]).any()
        assert torch.equal(got[2][:, :, ~hit], clean[2][:, :, ~hit])  # dq of those that do not see it
        far = torch.zeros(T, dtype=torch.bool, device="cuda")
        far[at - window + 1:at + window] = True                        # keys that share a query with it
        for n in (3, 4):
            assert torch.equal(got[n][:, :, ~far], clean[n][:, :, ~far])
    # a query, or its dO: keys at - window + 1 .. at see it
    for which in (0, 3):
        args = [t.clone() for t in (q, k, v, do)]
        args[which][:, :, at, 5] = bad
        got = both(*args)
        hit = torch.zeros(T, dtype=torch.bool, device="cuda")
        hit[at - window + 1:at + 1] = True
        others = torch.arange(T, device="cuda") != at
        assert torch.equal(got[0][:, :, others], clean[0][:, :, others]) and torch.equal(got[2][:, :, others], clean[2][:, :, others])
        for n in (3, 4):
            assert torch.equal(got[n][:, :, ~hit], clean[n][:, :, ~hit])
        if bad != bad:
            assert not torch.isfinite(got[4][:, :, hit][..., 5]).any()
    # queries that see nothing: whatever they and their dO hold
    args = [t.clone() for t in (q, k, v, do)]
    args[0][:, :, blind] = bad
    args[3][:, :, blind] = bad
    got = both(*args)
    for a, b in zip(got, clean):
        assert torch.equal(a, b)
    assert not got[0][:, :, blind].any() and not got[2][:, :, blind].any() and (got[1][:, :, blind] == -float("inf")).all()


def test_scores_far_apart():
    """Scores of thousands, rising along the keys (the running maximum moves at every
    tile) and falling: no exponential leaves its range."""
    torch, pdn = torch_mod(), _pdn()
    T, d = 600, 64
    for sign in (1.0, -1.0):
        q = torch.zeros(1, 1, T, d)
        k = torch.zeros(1, 1, T, d)
        q[..., 0], k[0, 0, :, 0] = 100.0, sign * torch.arange(T) * 0.5
        gen = torch.Generator().manual_seed(6)
        v = torch.randn(1, 1, T, d, generator=gen)
        for dtype in ("fp32", "bf16"):
            a = [t.to(_dt(dtype)).cuda() for t in (q, k, v)]
            o, lse = torch.empty_like(a[0]), torch.empty(1, 1, T, device="cuda")
            pdn.pdn_attn_fwd(*a, o, lse=lse, scale=1.0)
            want = ref.attn(*(_host(t) for t in a), 1.0, ref.seen(T, T, 0, None), dtype)
            _close("o", o, want["o"], want["bo"], dtype)
            _close("lse", lse, want["lse"], want["bl"], "fp32")


def test_shared_heads_by_views_of_repeated_keys():
    """The keys that pdn_qk_norm_fwd repeats for the recurrence, taken back by a view; one
    key head for a whole batch (stride 0)."""
    torch, pdn = torch_mod(), _pdn()
    gen = torch.Generator().manual_seed(41)
    q, k, v = _rand(gen, 2, 6, 77, 64, dtype="bf16"), _rand(gen, 2, 2, 77, 64, dtype="bf16"), _rand(gen, 2, 2, 77, 64, dtype="bf16")
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    pdn.pdn_attn_fwd(q, k, v, o)
    wide = k.repeat_interleave(3, 1)
    pdn.pdn_attn_fwd(q, wide[:, ::3], v, o2)
    assert torch.equal(o, o2)
    pdn.pdn_attn_fwd(q, k[:1, :1].expand(2, 6, -1, -1), v[:1, :1].expand(2, 6, -1, -1), o)
    pdn.pdn_attn_fwd(q, k[:1, :1].repeat(2, 6, 1, 1), v[:1, :1].repeat(2, 6, 1, 1), o2)
    assert torch.equal(o, o2)


def test_streams_workspaces_and_graphs():
    """Two calls at once on two streams, and two graphs captured one after the other (their
    workspaces from one pool), replayed several times with eager calls between."""
    torch, pdn = torch_mod(), _pdn()
    gen = torch.Generator().manual_seed(51)
    cases = [(1, 4, 2, 9, 3000, 64), (2, 4, 2, 300, 300, 128)]
    data = []
    for B, H, Hk, Tq, Tk, d in cases:
        q, do = _rand(gen, B, H, Tq, d, dtype="bf16"), _rand(gen, B, H, Tq, d)
        k, v = _rand(gen, B, Hk, Tk, d, dtype="bf16"), _rand(gen, B, Hk, Tk, d, dtype="bf16")
        out = [torch.empty(B, H, Tq, d, device="cuda"), torch.empty(B, H, Tq, device="cuda"), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)]
        data.append((q, k, v, do, out))

    def step(q, k, v, do, out, stream=None):
        pdn.pdn_attn_fwd(q, k, v, out[0], lse=out[1], stream=stream)
        pdn.pdn_attn_bwd(q, k, v, out[0], do, out[1], *out[2:], stream=stream)

    def eager():
        torch.cuda.synchronize()
        for x in data:
            step(*x)
        torch.cuda.synchronize()
        return [[t.clone() for t in x[-1]] for x in data]

    want = eager()
    for x in data:
        for t in x[-1]:
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for x, s in zip(data, streams):
        step(*x, stream=s)
    torch.cuda.synchronize()
    for x, w in zip(data, want):
        assert all(torch.equal(a, b) for a, b in zip(x[-1], w))
    graphs = []
    for x in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            step(*x)
        graphs.append(g)
    for n in range(4):
        for x in data:
            x[0].mul_(-1.5 if n % 2 else 0.5)
            for t in x[-1]:
                t.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in x[-1]] for x in data]
        want = eager()
        assert all(torch.equal(a, b) for x, w in zip(got, want) for a, b in zip(x, w))


def test_far_strides():
    """Offsets past 32 bits: rows of a long cache's layout."""
    torch, pdn = torch_mod(), _pdn()
    T, d, step = 300, 64, 1 << 24   # 300 * 2^24 bf16 elements span 10 GB
    base = torch.empty(T * step, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(61)
    q, do = _rand(gen, 1, 1, T, d, dtype="bf16"), _rand(gen, 1, 1, T, d, dtype="bf16")
    far = [base.as_strided((1, 1, T, d), (T * step, T * step, step, 1), i * d) for i in range(6)]
    k, v, dk, dv, o, dq = far
    near = [_rand(gen, 1, 1, T, d, dtype="bf16") for _ in range(2)]
    k.copy_(near[0])
    v.copy_(near[1])
    lse, lse2 = torch.empty(1, 1, T, device="cuda"), torch.empty(1, 1, T, device="cuda")
    want = [torch.empty_like(q) for _ in range(4)]
    pdn.pdn_attn_fwd(q, *near, want[0], lse=lse)
    pdn.pdn_attn_bwd(q, *near, want[0], do, lse, *want[1:])
    pdn.pdn_attn_fwd(q, k, v, o, lse=lse2)
    pdn.pdn_attn_bwd(q, k, v, o, do, lse2, dq, dk, dv)
    assert torch.equal(lse, lse2)
    for a, b in zip((o, dq, dk, dv), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("big", [3.4028234e38, -3.3962e38])
def test_the_largest_numbers_count_as_infinite(d, big):
    """fp32 numbers from 3.396e38 on: no part in what does not see them either."""
    torch, pdn = torch_mod(), _pdn()
    T, at = 150, 77
    gen = torch.Generator().manual_seed(64)
    q, k, v, do = (_rand(gen, 1, 1, T, d) for _ in range(4))

    def both(q, k, v, do):
        o, lse = torch.empty_like(q), torch.empty(1, 1, T, device="cuda")
        pdn.pdn_attn_fwd(q, k, v, o, lse=lse)
        g = [torch.empty_like(q) for _ in range(3)]
        pdn.pdn_attn_bwd(q, k, v, o, do, lse, *g)
        return [o, *g]

    clean = both(q, k, v, do)
    for which in range(4):
        args = [t.clone() for t in (q, k, v, do)]
        args[which][:, :, at, 2] = big
        got = both(*args)
        assert torch.equal(got[0][:, :, :at], clean[0][:, :, :at]) and torch.equal(got[1][:, :, :at], clean[1][:, :, :at])
        if which in (0, 3):   # keys behind the query see nothing of it
            assert torch.equal(got[2][:, :, at + 1:], clean[2][:, :, at + 1:]) and torch.equal(got[3][:, :, at + 1:], clean[3][:, :, at + 1:])


@pytest.mark.parametrize("d", [64, 128])
def test_one_key_gives_its_value(d):
    """fp32 values of every size and of 24 bits come back.  The key's weight w is one but for the
    rounding of its exponent, and leaves by o = (w v) / w: in halves of a step (2^-24) one of
    w v's parts that are left out, six of its sums, one each of 1 / w and the last product,
    and one for the second order."""
    torch, pdn = torch_mod(), _pdn()
    gen = torch.Generator().manual_seed(63)
    T = 200
    q, k, v = (_rand(gen, 1, 1, T, d) for _ in range(3))
    v *= torch.exp2(torch.randint(-100, 120, v.shape, generator=gen).float().cuda())
    v[..., 0], v[..., 1] = 3.39e38, -3.39e38
    first = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    o = torch.empty_like(q)
    pdn.pdn_attn_fwd(q, k, v, o, first=first)
    assert ((o.double() - v.double()).abs() <= 10 * 2.0 ** -24 * v.double().abs()).all()


def test_furthest_token_steps():
    """Whole tiles whose lanes' offsets use all of their 32 bits."""
    torch, pdn = torch_mod(), _pdn()
    T, d, step = 64, 64, 1 << 28
    base = torch.empty((T - 1) * step + 8 * d, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(62)
    near = [_rand(gen, 1, 1, T, d, dtype="bf16") for _ in range(4)]
    far = [base.as_strided((1, 1, T, d), (T * step, T * step, step, 1), i * d) for i in range(4)]
    for a, b in zip(far, near):
        a.copy_(b)
    got = []
    for q, k, v, do in (near, far):
        out, lse = [torch.empty_like(near[0]) for _ in range(4)], torch.empty(1, 1, T, device="cuda")
        pdn.pdn_attn_fwd(q, k, v, out[0], lse=lse)
        pdn.pdn_attn_bwd(q, k, v, out[0], do, lse, *out[1:])
        got.append(out + [lse])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_gradient_against_differences():
    """dq, dk and dv of the fp32 kernel against differences of its own forward."""
    torch, pdn = torch_mod(), _pdn()
    gen = torch.Generator().manual_seed(71)
    q, k, v, do = (_rand(gen, 1, 2, 70, 64, scale=0.7) for _ in range(4))
    k, v = k[:, :1].contiguous(), v[:, :1].contiguous()
    o, lse = torch.empty_like(q), torch.empty(1, 2, 70, device="cuda")
    pdn.pdn_attn_fwd(q, k, v, o, lse=lse, window=40)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    pdn.pdn_attn_bwd(q, k, v, o, do, lse, *grads, window=40)
    for n, t in enumerate((q, k, v)):
        way = _rand(gen, *t.shape)
        slope = (grads[n].double() * way.double()).sum().item()
        ends = []
        for h in (2.0 ** -7, -2.0 ** -7):
            args = [q, k, v]
            args[n] = t + h * way
            pdn.pdn_attn_fwd(*args, o, window=40)
            ends.append((o.double() * do.double()).sum().item())
        # a third derivative of order one leaves h^2 of it; the forward's own error, 1e-6 of a
        # sum of some 9000 terms of order one over 2 h, is smaller
        assert abs((ends[0] - ends[1]) / 2.0 ** -6 - slope) < 2e-2 * max(1.0, abs(slope))


def test_binding_refusals():
    torch, pdn = torch_mod(), _pdn()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    q, k, v, o = z(1, 4, 8, 64), z(1, 2, 8, 64), z(1, 2, 8, 64), z(1, 4, 8, 64)
    ok = dict(q=q, k=k, v=v, o=o)
    pdn.pdn_attn_fwd(**ok)
    f32 = torch.float32
    for bad in (dict(k=z(1, 3, 8, 64), v=z(1, 3, 8, 64)), dict(k=k.float()), dict(v=z(1, 2, 9, 64)), dict(o=z(1, 4, 8, 128)), dict(scale=-1.0),
                dict(scale=0.0), dict(window=-1), dict(first=z(1, 8, dtype=torch.int64)), dict(first=z(8, dtype=torch.int32)),
                dict(lse=z(1, 4, 8)), dict(lse=z(1, 4, 9, dtype=f32)), dict(q=q.transpose(2, 3)), dict(q=z(4, 8, 64)), dict(o=z(1, 4, 8, 64, dtype=torch.float16)),
                dict(o=z(1, 1, 8, 64).expand(1, 4, 8, 64)), dict(q=q.half(), k=k.half(), v=v.half()), dict(k=k.cpu()),
                dict(q=z(1, 4, 8, 96), k=z(1, 2, 8, 96), v=z(1, 2, 8, 96), o=z(1, 4, 8, 96))):
        with pytest.raises((ValueError, pdn.PdnError)):
            pdn.pdn_attn_fwd(**{**ok, **bad})
    lse = z(1, 4, 8, dtype=f32)
    g = dict(do=o, lse=lse, dq=q.clone(), dk=k.clone(), dv=v.clone())
    pdn.pdn_attn_bwd(**ok, **g)
    for bad in (dict(lse=None), dict(do=o.float()), dict(dq=q.float()), dict(dk=z(1, 4, 8, 64)), dict(dv=z(1, 2, 7, 64)), dict(dq=z(1, 4, 8, 64, dtype=torch.float16)),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, pdn.PdnError)):
            pdn.pdn_attn_bwd(**ok, **{**g, **bad})
