"""GPU checks of attention, contiguous and paged, at the ends of its range: scores of any
size, rows whose scores are all -inf, keys and queries that are not finite, keys dealt to many
workgroups, pages by the hundred, D of rows with keys in several blocks."""
import numpy as np
import pytest

import block_ref as ref
import test_gpu_attn as contiguous
import test_gpu_paged as paged
from block_ref import HALF, U
from gpu_util import torch_mod
from test_gpu_attn import _close, _dt, _host, _make, _nan, _pdn, _rand

pytestmark = pytest.mark.gpu


# -- scores of any size -------------------------------------------------------

def _peaks(gen, H, Hk, Tq, Tk, dtype, power, sign, low=None):
    """q, k, v of one sequence whose scores are one product each, exact in either type: 2^power
    (1 + n / 128) for n = 0 .. 127, or from 2^low to 2^power along the keys."""
    torch = torch_mod()
    d = 64
    q, k = torch.zeros(1, H, Tq, d), torch.zeros(1, Hk, Tk, d)
    q[..., 5] = sign * 2.0 ** (power // 2)
    if low is None:
        k[..., 5] = 2.0 ** (power - power // 2) * (1 + torch.randint(0, 128, (1, Hk, Tk), generator=gen) / 128)
    else:
        k[..., 5] = torch.exp2(torch.linspace(low, power, Tk).round() - power // 2)
    v = torch.randn(1, Hk, Tk, d, generator=gen)
    return [t.to(_dt(dtype)).cuda() for t in (q, k, v)]


def _peaked(o, lse, q, k, v, scale, dtype):
    """Against the softmax in 64 bits.  Scores are exact, and a difference of two is off by its own
    rounding only: an exponential that counts by 2^-18 at most (its exponent is above -30 there,
    the scale's rounding and its own two), which is nothing where scores are equal."""
    torch = torch_mod()
    q, k, v = _host(q), _host(k), _host(v)
    rep = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    seen = ref.seen(q.shape[2], k.shape[2], 0, None)[:, None]
    s = ((q @ k.mT) * scale).masked_fill(~seen, -torch.inf)
    p = torch.softmax(s, -1)
    size, n = p @ v.abs(), k.shape[2]
    half = HALF["bf16"] if dtype == "bf16" else 0.0
    _close("o", o, p @ v, size * (half + 2.0 ** -17 + 2 * (n + 8) * U), dtype)
    want = torch.logsumexp(s, -1)
    _close("lse", lse, want, want.abs() * 6 * U + 2.0 ** -18 + 2 * (n + 8) * U, "fp32")


# few and many rows, one workgroup and several, joined by lanes and by workgroups
@pytest.mark.parametrize("H,Hk,Tq,Tk", [(1, 1, 1, 1), (2, 1, 200, 200), (2, 1, 3, 2500), (2, 2, 1, 6000), (1, 1, 300, 2600)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scores_of_any_size(dtype, H, Hk, Tq, Tk):
    """Finite scores from 1e7 to 1e30, of either sign: the largest key's value comes out, the mean
    where several are the largest."""
    torch, pdn = torch_mod(), _pdn()
    gen = torch.Generator().manual_seed(91)
    for power, low in ((24, None), (31, None), (34, None), (60, None), (100, None), (100, -10), (40, 10)):
        for sign in (1.0, -1.0):
            for scale in (0.125, 0.11, 3.0):
                q, k, v = _peaks(gen, H, Hk, Tq, Tk, dtype, power, sign, low)
                o, lse = torch.empty_like(q), _nan((1, H, Tq))
                pdn.pdn_attn_fwd(q, k, v, o, lse=lse, scale=scale)
                _peaked(o, lse, q, k, v, float(np.float32(scale)), dtype)


@pytest.mark.parametrize("news,lens", [([1], [700]), ([1], [6000]), ([90], [2000])])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scores_of_any_size_over_pages(dtype, news, lens):
    torch, pdn = torch_mod(), _pdn()
    gen, kp, vp, table, dlens, starts, _ = paged._paged_case(1, 1, 64, dtype, 16, news, lens, 92)
    for power, sign in ((34, 1.0), (34, -1.0), (100, 1.0)):
        q, k, v = _peaks(gen, 2, 1, news[0], lens[0], dtype, power, sign)
        j = torch.arange(lens[0], device="cuda")
        at = table[0, j // 16].long(), j % 16
        kp[at], vp[at] = k[0].transpose(0, 1), v[0].transpose(0, 1)
        rows = q[0].transpose(0, 1).contiguous()
        o, lse = torch.empty_like(rows), _nan((news[0], 2))
        pdn.pdn_attn_paged(rows, o, kp, vp, table, dlens, starts=starts, max_new=news[0], lse=lse, scale=0.125)
        _peaked(o.transpose(0, 1)[None], lse.T[None], q, k, v, 0.125, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_whose_scores_are_all_minus_infinity(dtype):
    """q and k finite, their products not: such a query gives o = 0 and lse = -inf, as one that
    sees nothing, and passes nothing on."""
    torch, pdn = torch_mod(), _pdn()
    gen = torch.Generator().manual_seed(93)
    B, H, Hk, T, d = 1, 4, 2, 300, 64
    q, k, v = _rand(gen, B, H, T, d, dtype=dtype), _rand(gen, B, Hk, T, d, dtype=dtype), _rand(gen, B, Hk, T, d, dtype=dtype)
    do = _rand(gen, B, H, T, d, dtype=dtype)
    q[..., 7], k[..., 7] = 0.0, -2.0 ** 80
    none = torch.tensor([0, 3, 40, 64, 130, 131, 299], device="cuda")
    q[:, :, none] = 0.0
    q[:, :, none, 7] = 2.0 ** 80

    o, lse = torch.empty_like(q), _nan((B, H, T))
    pdn.pdn_attn_fwd(q, k, v, o, lse=lse)
    g = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    pdn.pdn_attn_bwd(q, k, v, o, do, lse, *g)
    assert not o[:, :, none].any() and (lse[:, :, none] == -float("inf")).all() and not g[0][:, :, none].any()
    # as where these queries see nothing by their mask
    first = torch.zeros(B, T, dtype=torch.int32)
    first[:, none.cpu()] = T
    mask, scale = ref.seen(T, T, 0, first), float(np.float32(d ** -0.5))
    want = ref.attn(_host(q), _host(k), _host(v), scale, mask, dtype)
    _close("o", o, want["o"], want["bo"], dtype)
    _close("lse", lse, want["lse"], want["bl"], "fp32")
    want = ref.attn_bwd(_host(q), _host(k), _host(v), _host(o), _host(do), scale, mask, dtype, False, dtype)
    for n, t in zip(("dq", "dk", "dv"), g):
        _close(n, t, *want[n], dtype)


# -- what is not finite and is seen ------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_keys_and_queries_reach_the_gradients(dtype, d):
    """A key or query with an infinity, its scores -inf (in fp32 NaN), a value or dO with one:
    wherever a tile ends, the gradients of what it has a part in are not finite, the others' as
    ever."""
    torch, pdn = torch_mod(), _pdn()
    gen = torch.Generator().manual_seed(94)
    T = 300
    q, k, v, do = (_rand(gen, 1, 2, T, d, dtype=dtype) for _ in range(4))
    q[..., 3], k[..., 3] = 0.5, 0.25

    def both(q, k, v, do):
        o, lse = torch.empty_like(q), _nan((1, 2, T))
        pdn.pdn_attn_fwd(q, k, v, o, lse=lse)
        g = [torch.empty_like(t) for t in (q, k, v)]
        pdn.pdn_attn_bwd(q, k, v, o, do, lse, *g)
        return [o, *g]

    clean = both(q, k, v, do)
    for at in (5, 31, 70, 128, 290):
        for which in range(4):
            args = [t.clone() for t in (q, k, v, do)]
            args[which][:, :, at, 3] = -float("inf")
            o, dq, dk, dv = both(*args)
            if which in (1, 2):
                assert torch.equal(o[:, :, :at], clean[0][:, :, :at]) and torch.equal(dq[:, :, :at], clean[1][:, :, :at])
                assert not torch.isfinite(dq[:, :, at:, 3]).any()     # of all that see it
                if which == 1 and dtype == "bf16":
                    assert torch.isfinite(o.float()).all()            # a probability of zero
            else:
                others = torch.arange(T, device="cuda") != at
                assert torch.equal(o[:, :, others], clean[0][:, :, others]) and torch.equal(dq[:, :, others], clean[1][:, :, others])
                for got, was in ((dk, clean[2]), (dv, clean[3])):
                    assert not torch.isfinite(got[:, :, :at + 1, 3]).any()   # of all that it sees
                    assert torch.equal(got[:, :, at + 1:], was[:, :, at + 1:])


@pytest.mark.parametrize("H,Hk,Tq,Tk", [(2, 1, 200, 200), (2, 1, 3, 2500), (2, 2, 1, 6000), (1, 1, 300, 2600)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_a_seen_value_that_is_not_finite_shows(dtype, H, Hk, Tq, Tk, bad):
    """Also where its key's probability is zero, and its workgroup's part of the sum with it."""
    torch, pdn = torch_mod(), _pdn()
    gen = torch.Generator().manual_seed(95)
    q, k, v = _rand(gen, 1, H, Tq, 64, dtype=dtype), _rand(gen, 1, Hk, Tk, 64, dtype=dtype), _rand(gen, 1, Hk, Tk, 64, dtype=dtype)
    q[..., 0] = 64.0
    k[..., 0] = 0.0
    k[:, :, :2 * Tk // 3, 0] = -512.0     # these count for nothing beside the rest
    v[:, :, 9, 2] = float(bad)
    o = torch.empty_like(q)
    pdn.pdn_attn_fwd(q, k, v, o)
    see = torch.arange(Tq, device="cuda") + Tk - Tq >= 9
    assert not torch.isfinite(o[:, :, see, 2].float()).any() and torch.isfinite(o[:, :, ~see].float()).all()


# -- paths that depend on a call's sizes --------------------------------------

MANY = [  # keys dealt to more than eight workgroups, and to more than a wave's 64
    (1, 2, 1, 1, 5200, 64, "bf16", "bf16", "bf16", 0, None),
    (1, 1, 1, 1, 34000, 128, "bf16", "bf16", "bf16", 0, None),
    (1, 2, 1, 1, 34000, 64, "bf16", "fp32", "fp32", 0, None),
    (1, 2, 1, 2, 3000, 64, "fp32", "fp32", "fp32", 0, None),
    (1, 2, 1, 1, 2600, 128, "fp32", "fp32", "fp32", 0, None),
]


@pytest.mark.parametrize("case", MANY, ids=contiguous.ids)
def test_keys_dealt_to_many_workgroups(case):
    B, H, Hk, Tq, Tk, d, dtype, odtype = case[:8]
    e = lambda *s, t=dtype: torch_mod().empty(s, dtype=_dt(t), device="cuda")  # noqa: E731
    size = _pdn().pdn_attn_fwd_workspace_size(e(B, H, Tq, d), e(B, Hk, Tk, d), e(B, Hk, Tk, d), e(B, H, Tq, d, t=odtype))
    assert size > (64 if Tk > 32768 else 8) * B * H * Tq * (d + 2) * 4
    contiguous.test_attn(case)


_long = lambda n, every, far: [far if b % every == 1 else 1 + (7 * b) % 40 for b in range(n)]  # noqa: E731
PAGES = [
    (1, 4, 1, 64, "bf16", "bf16", 64, [1], [5000], 0),
    (1, 2, 1, 64, "fp32", "fp32", 16, [1], [2600], 0),
    (1, 2, 1, 128, "fp32", "fp32", 32, [2], [2600], 0),
    (1, 2, 1, 128, "bf16", "bf16", 128, [1], [34000], 0),
    # every unit has a workgroup by the heads alone
    (128, 4, 2, 64, "bf16", "bf16", 32, [1] * 128, [1 + (397 * b) % 2100 for b in range(128)], 0),
    # hundreds of pages to one workgroup, one token and several of a sequence
    (130, 2, 1, 64, "bf16", "bf16", 16, [1] * 130, _long(130, 40, 5000), 0),
    (256, 4, 4, 64, "bf16", "bf16", 16, [40 if b == 41 else 1 for b in range(256)], _long(256, 40, 3300), 0),
]


@pytest.mark.parametrize("case", PAGES, ids=lambda c: "B%d-H%d.%d-d%d-%s-p%d-L%d" % (*c[:5], c[6], max(c[8])))
def test_pages_by_the_hundred_and_parts_by_the_dozen(case):
    paged.test_paged(case)


# -- D ------------------------------------------------------------------------

@pytest.mark.parametrize("case", [(1, 2, 1, 200, 240, 128, "bf16", "bf16", "fp32", 0, None), (1, 2, 2, 150, 250, 64, "bf16", "fp32", "fp32", 40, None),
                                  (2, 4, 2, 90, 1500, 64, "bf16", "bf16", "fp32", 0, None), (1, 2, 1, 200, 240, 64, "fp32", "fp32", "fp32", 0, None)],
                         ids=contiguous.ids)
def test_rows_of_several_blocks_take_d_from_o(case):
    """Every query sees more than 32 keys, so that no block of 32 holds them all: D is <dO, o> of
    the o that is given, without the rounding of P that a D formed from P would bring.  An o that
    is off by more than that shows it: the gradients are those of this o."""
    torch, pdn = torch_mod(), _pdn()
    B, H, Hk, Tq, Tk, d, dtype, odtype, gdtype, window, kind = case
    gen, q, k, v, do, first, mask = _make(case, 96)
    assert mask.sum(-1).min() > 32
    o, lse = _nan((B, H, Tq, d), odtype), _nan((B, H, Tq))
    pdn.pdn_attn_fwd(q, k, v, o, lse=lse, window=window)
    o = (o.float() + 0.25).to(o.dtype)
    grads = [_nan(t.shape, gdtype) for t in (q, k, v)]
    pdn.pdn_attn_bwd(q, k, v, o, do, lse, *grads, window=window)
    scale = float(np.float32(d ** -0.5))
    f = ref.attn(_host(q), _host(k), _host(v), scale, mask, dtype)
    p, kk, vv, rep = f["p"], f["k"], f["v"], H // Hk
    h, hd = HALF["bf16"] if dtype == "bf16" else 0.0, HALF["bf16"] if dtype == "bf16" and odtype == "fp32" else 0.0
    dof, of = _host(do), _host(o)
    dp, size_p = dof @ vv.mT, dof.abs() @ vv.abs().mT
    delta, size_d = (dof * of).sum(-1, keepdim=True), (dof * of).abs().sum(-1, keepdim=True)
    ds = p * (dp - delta)
    # as block_ref.attn_bwd counts, with D's own sum of d products in the place of what P would add
    e = 2 * f["e"] + 2 * (Tk + 8) * U + 4 * U * f["lse"].abs()[..., None]
    eds = p * (size_p * (hd + 2 * (d + 2) * U) + size_d * 2 * (d + 2) * U) + ds.abs() * (e + 4 * U)
    eds = eds * (1 + h) + ds.abs() * h
    fold = lambda t: t.unflatten(1, (Hk, rep)).sum(2)  # noqa: E731
    qf, sums = _host(q), 2 * (max(Tk, Tq * rep) + 8) * U
    _close("dq", grads[0], scale * (ds @ kk), scale * (eds @ kk.abs() + sums * (ds.abs() @ kk.abs())), gdtype)
    _close("dk", grads[1], scale * fold(ds.mT @ qf), scale * fold(eds.mT @ qf.abs() + sums * (ds.abs().mT @ qf.abs())), gdtype)


# -- the largest values --------------------------------------------------------

@pytest.mark.parametrize("H,Hk,Tq,Tk", [(2, 1, 200, 200), (2, 1, 3, 2500), (1, 1, 300, 2600)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_values_up_to_the_limit(dtype, H, Hk, Tq, Tk):
    """|v| of 3.4e38 / (2^8 Tk), and scores that rise along the keys by less than moves the
    maximum at every one: finite, and as the softmax gives it."""
    torch, pdn = torch_mod(), _pdn()
    gen = torch.Generator().manual_seed(97)
    q, k = torch.zeros(1, H, Tq, 64), torch.zeros(1, Hk, Tk, 64)
    q[..., 0], k[..., 0] = 1.0, (torch.arange(Tk) % 128) / 32.0
    v = torch.full((1, Hk, Tk, 64), 3.39e38 / (256 * Tk))
    v[..., 1::2] *= torch.rand(1, Hk, Tk, 32, generator=gen)
    q, k, v = (t.to(_dt(dtype)).cuda() for t in (q, k, v))
    o = torch.empty_like(q)
    pdn.pdn_attn_fwd(q, k, v, o, scale=1.0)
    f = ref.attn(_host(q), _host(k), _host(v), 1.0, ref.seen(Tq, Tk, 0, None), dtype)
    _close("o", o, f["o"], f["bo"], dtype)


# -- numbers past 32 bits -------------------------------------------------------

def test_numbers_past_32_bits_are_refused():
    """Sizes, windows and bounds that the library's 32-bit fields would take for others."""
    torch, pdn = torch_mod(), _pdn()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    q, o = z(1, 2, 8, 64), z(1, 2, 8, 64)
    for window in (2 ** 31, 2 ** 32 + 3, -2 ** 32):
        with pytest.raises((ValueError, pdn.PdnError)):
            pdn.pdn_attn_fwd(q, q, q, o, window=window)
    many = z(1, 1, 1, 64).expand(1, 1, 2 ** 32 + 8, 64)
    with pytest.raises((ValueError, pdn.PdnError)):
        pdn.pdn_attn_fwd(q, many, many, o)
    lse = z(1, 2, 8, dtype=torch.float32)
    with pytest.raises((ValueError, pdn.PdnError)):
        pdn.pdn_attn_bwd(q, many, many, o, o, lse, q.clone(), many, many)
    rows = z(1, 1, 8).expand(1, 2 ** 32 + 1, 8)
    with pytest.raises((ValueError, pdn.PdnError)):
        pdn.pdn_add_norm_fwd(rows, z(1, 1, 8).expand(rows.shape))
    with pytest.raises((ValueError, pdn.PdnError)):
        pdn.pdn_add_norm_bwd(rows, rows, z(1, 1, 8).expand(rows.shape))
    pages, table, lens, starts = z(3, 16, 2, 64), z(2, 3, dtype=torch.int32), z(2, dtype=torch.int32), z(3, dtype=torch.int32)
    for bound in (2 ** 31, 2 ** 32 + 4, -2 ** 32):
        with pytest.raises((ValueError, pdn.PdnError)):
            pdn.pdn_attn_paged(z(4, 2, 64), z(4, 2, 64), pages, pages, table, lens, starts=starts, max_new=bound)
        with pytest.raises((ValueError, pdn.PdnError)):
            pdn.pdn_cache_append(z(4, 2, 64), z(4, 2, 64), pages, pages.clone(), table, lens, starts=starts, max_new=bound)
