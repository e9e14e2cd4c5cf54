"""GPU checks of the paged cache: the writes into it and the attention over it,
against 64-bit references and against the contiguous attention, and the operators of
a hybrid stack's layers together, forward and backward."""
import numpy as np
import pytest

import block_ref as ref
from block_ref import HALF
from gpu_util import torch_mod
from test_gpu_attn import _close, _dt, _host, _pdn, _rand

pytestmark = pytest.mark.gpu


def _paged_case(B, Hk, d, dtype, page, news, lens, seed, spare=3, fill=None):
    """A pool whose unused slots are NaN, sequences' pages scattered over it."""
    torch = torch_mod()
    gen = torch.Generator().manual_seed(seed)
    pages = [-(-t // page) for t in lens]
    pool, width = sum(pages) + spare, max(1, *pages)
    order = torch.randperm(pool, generator=gen).int()
    table = torch.full((B, width), -1 if fill is None else fill, dtype=torch.int32)
    kp, vp = (torch.full((pool, page, Hk, d), float("nan"), dtype=_dt(dtype)) for _ in range(2))
    at, seqs = 0, []
    for b, t in enumerate(lens):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
        k, v = _rand(gen, t, Hk, d, dtype=dtype).cpu(), _rand(gen, t, Hk, d, dtype=dtype).cpu()
        j = torch.arange(t)
        kp[table[b, j // page].long(), j % page] = k
        vp[table[b, j // page].long(), j % page] = v
        seqs.append((k, v))
    starts = torch.tensor([0] + np.cumsum(news).tolist(), dtype=torch.int32)
    return gen, kp.cuda(), vp.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), starts.cuda(), seqs


# B, H, Hk, d, dtype, o, page, new, lens, window
PAGED = [
    (1, 1, 1, 64, "bf16", "bf16", 16, [1], [1], 0),
    (3, 4, 2, 128, "bf16", "bf16", 16, [1, 1, 1], [1, 17, 300], 0),
    (4, 8, 1, 64, "bf16", "fp32", 64, [1, 1, 1, 1], [64, 65, 63, 700], 0),
    (2, 6, 2, 128, "fp32", "fp32", 32, [1, 1], [33, 900], 0),
    (1, 4, 1, 128, "bf16", "bf16", 128, [1], [5000], 0),
    (1, 4, 4, 64, "fp32", "fp32", 16, [1], [3001], 500),
    (3, 4, 2, 128, "bf16", "bf16", 16, [5, 0, 31], [5, 40, 200], 0),
    (3, 3, 1, 64, "bf16", "bf16", 32, [100, 1, 7], [150, 260, 7], 0),
    (2, 2, 2, 128, "bf16", "fp32", 64, [300, 12], [300, 2012], 0),
    (2, 4, 2, 64, "fp32", "fp32", 16, [70, 33], [90, 1033], 64),
    (2, 4, 2, 128, "bf16", "bf16", 16, [90, 140], [400, 140], 33),
    (2, 16, 1, 128, "bf16", "bf16", 1024, [3, 2], [1500, 9], 0),
    (5, 2, 1, 64, "bf16", "bf16", 16, [2, 0, 0, 1, 3], [2, 0, 9, 4, 3], 0),
]
PAGED += [  # chunks of many sequences, with equal lengths among them: in order of length, and (33) as given
    (n, 4, 2, 64, "bf16", "bf16", 16, [(7 * b) % 31 for b in range(n)], [(7 * b) % 31 + 64 * (b % 3) + (b % 2) for b in range(n)], 0)
    for n in (31, 32, 33)
]
ids = lambda c: "B%d-H%d.%d-d%d-%s-%s-p%d-n%s-L%s-w%d" % (c[:7] + (".".join(map(str, c[7])), ".".join(map(str, c[8])), c[9]))  # noqa: E731


@pytest.mark.parametrize("case", PAGED, ids=ids)
def test_paged(case):
    torch, pdn = torch_mod(), _pdn()
    B, H, Hk, d, dtype, odtype, page, news, lens, window = case
    gen, kp, vp, table, dlens, starts, seqs = _paged_case(B, Hk, d, dtype, page, news, lens, 81)
    N, behind = sum(news), 4
    q = _rand(gen, N + behind, H, d, dtype=dtype, scale=1.5)
    o = torch.full((N + behind, H, d), 7.0, dtype=_dt(odtype), device="cuda")
    lse = torch.full((N + behind, H), 7.0, device="cuda")
    same = dict(starts=starts, max_new=max(news), scale=0.13, window=window)
    size = pdn.pdn_attn_paged_workspace_size(q, o, kp, vp, table, dlens, lse=lse, **same)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    pdn.pdn_attn_paged(q, o, kp, vp, table, dlens, lse=lse, workspace=ws, **same)
    torch.cuda.synchronize()
    assert (o[N:] == 7.0).all() and (lse[N:] == 7.0).all()   # rows behind the last sequence
    row = 0
    for b in range(B):
        n, t = news[b], lens[b]
        if n == 0:
            continue
        k, v = (x.double().permute(1, 0, 2)[None] for x in seqs[b])
        f = ref.attn(_host(q[row:row + n]).permute(1, 0, 2)[None], k, v, float(np.float32(0.13)), ref.seen(n, t, window, None), dtype)
        _close("o", o[row:row + n].permute(1, 0, 2)[None], f["o"], f["bo"], odtype)
        _close("lse", lse[row:row + n].T[None], f["lse"], f["bl"], "fp32")
        row += n
    # a larger bound on the new tokens, more table, no lse: the same rows
    o2 = torch.full_like(o, 7.0)
    wide = torch.cat([table, torch.full((B, 3), 2 ** 31 - 1, dtype=torch.int32, device="cuda")], 1)
    pdn.pdn_attn_paged(q, o2, kp, vp, wide, dlens, starts=starts, scale=0.13, window=window)
    row = 0
    for b in range(B):
        n, t = news[b], lens[b]
        if n:
            k, v = (x.double().permute(1, 0, 2)[None] for x in seqs[b])
            f = ref.attn(_host(q[row:row + n]).permute(1, 0, 2)[None], k, v, float(np.float32(0.13)), ref.seen(n, t, window, None), dtype)
            _close("o", o2[row:row + n].permute(1, 0, 2)[None], f["o"], f["bo"], odtype)
        row += n
    assert (o2[N:] == 7.0).all()


def test_uniform_chunks_and_strides():
    """No starts: every sequence brings as many; pages of keys and values in one tensor,
    q and o as views."""
    torch, pdn = torch_mod(), _pdn()
    B, H, Hk, d, page = 3, 4, 2, 64, 32
    gen, kp, vp, table, lens, starts, _ = _paged_case(B, Hk, d, "bf16", page, [4] * B, [40, 4, 133], 82)
    q = _rand(gen, 12, H, d, dtype="bf16")
    o = torch.empty_like(q)
    pdn.pdn_attn_paged(q, o, kp, vp, table, lens, starts=starts)
    both = torch.stack([kp, vp], 1)                       # [pages, 2, page, Hk, d]
    heads_first = both.permute(0, 1, 3, 2, 4).contiguous().permute(0, 1, 3, 2, 4)
    wide = torch.zeros(12, 3 * H, d, dtype=torch.bfloat16, device="cuda")
    wide[:, H:2 * H] = q
    for pages in (both, heads_first):
        out = torch.zeros(H, 12, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        pdn.pdn_attn_paged(wide[:, H:2 * H], out, pages[:, 0], pages[:, 1], table, lens)
        assert torch.equal(out, o)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 64), ("bf16", 8), ("fp32", 256)])
def test_append(dtype, d):
    torch, pdn = torch_mod(), _pdn()
    news, lens, page, Hk = [5, 0, 70, 1], [5, 9, 100, 64], 16, 3
    gen, kp, vp, table, dlens, starts, _ = _paged_case(4, Hk, d, dtype, page, news, lens, 83)
    kp.zero_(), vp.zero_()
    N = sum(news)
    rows = _rand(gen, N + 3, 2 * Hk, d, dtype=dtype)
    k, v = rows[:, :Hk], rows[:, Hk:]
    wk, wv = kp.clone(), vp.clone()
    row = 0
    for b in range(4):
        for i in range(news[b]):
            at = lens[b] - news[b] + i
            wk[table[b, at // page], at % page], wv[table[b, at // page], at % page] = k[row], v[row]
            row += 1
    pdn.pdn_cache_append(k, v, kp, vp, table, dlens, starts=starts)
    assert torch.equal(kp, wk) and torch.equal(vp, wv)
    # what is appended is what the next call sees: one token more each, no starts
    k1, v1 = _rand(gen, 4, Hk, d, dtype=dtype), _rand(gen, 4, Hk, d, dtype=dtype)
    table = torch.cat([table, torch.arange(4, dtype=torch.int32, device="cuda")[:, None]], 1)
    lens1 = torch.tensor([6, 10, 101, 64], dtype=torch.int32, device="cuda")
    pdn.pdn_cache_append(k1, v1, kp, vp, table, lens1)
    for b, t in enumerate((6, 10, 101, 64)):
        assert torch.equal(kp[table[b, (t - 1) // page], (t - 1) % page], k1[b])
        assert torch.equal(vp[table[b, (t - 1) // page], (t - 1) % page], v1[b])


def test_numbers_that_lead_nowhere():
    """Pages that are not there, lengths past the table, rows past N: appended tokens
    without a place are left out, the others written; attention stays inside (what such
    a sequence gives means nothing) and the others' rows are as ever."""
    torch, pdn = torch_mod(), _pdn()
    B, H, Hk, d, page = 3, 2, 1, 64, 16
    gen, kp, vp, table, lens, starts, _ = _paged_case(B, Hk, d, "bf16", page, [2, 2, 2], [40, 33, 20], 84, fill=0)
    q, o = _rand(gen, 6, H, d, dtype="bf16"), torch.empty(6, H, d, dtype=torch.bfloat16, device="cuda")
    pdn.pdn_attn_paged(q, o, kp, vp, table, lens, starts=starts, max_new=2)
    k, v = _rand(gen, 6, Hk, d, dtype="bf16"), _rand(gen, 6, Hk, d, dtype="bf16")
    ok = (kp.clone(), vp.clone())
    pdn.pdn_cache_append(k, v, *ok, table, lens, starts=starts)
    for entry in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = table.clone()
        bad[1] = entry
        o2 = torch.empty_like(o)
        pdn.pdn_attn_paged(q, o2, kp, vp, bad, lens, starts=starts, max_new=2)
        assert torch.equal(o2[:2], o[:2]) and torch.equal(o2[4:], o[4:])
        a = (kp.clone(), vp.clone())
        pdn.pdn_cache_append(k, v, *a, bad, lens, starts=starts)
        want = (kp.clone(), vp.clone())
        for b, t in ((0, 40), (2, 20)):
            for i in (0, 1):
                at = t - 2 + i
                want[0][table[b, at // page], at % page], want[1][table[b, at // page], at % page] = k[2 * b + i], v[2 * b + i]
        for x, y in zip(a, want):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    for length in (0, 1, -5, 49, 2 ** 31 - 1, -2 ** 31):
        n = lens.clone()
        n[1] = length
        o2 = torch.empty_like(o)
        pdn.pdn_attn_paged(q, o2, kp, vp, table, n, starts=starts, max_new=2)
        assert torch.equal(o2[:2], o[:2]) and torch.equal(o2[4:], o[4:])
        if length == 0:
            assert not o2[2:4].any()
        a = (kp.clone(), vp.clone())
        pdn.pdn_cache_append(k, v, *a, table, n, starts=starts)
    for wrong in ([0, 2, 2 ** 31 - 1, 2 ** 31 - 1], [0, 2, -7, 6], [0, 2, 9, 1]):
        s = torch.tensor(wrong, dtype=torch.int32, device="cuda")
        o2 = torch.empty_like(o)
        pdn.pdn_attn_paged(q, o2, kp, vp, table, lens, starts=s, max_new=2)
        assert torch.equal(o2[:2], o[:2])
        pdn.pdn_cache_append(k, v, kp.clone(), vp.clone(), table, lens, starts=s)
    torch.cuda.synchronize()


def test_chunks_equal_the_whole():
    """A prompt in chunks through the cache, then token by token, against the contiguous
    attention of the same tokens, with captured decode steps."""
    torch, pdn = torch_mod(), _pdn()
    B, H, Hk, d, page, T, dtype = 2, 4, 2, 128, 16, 90, "bf16"
    gen = torch.Generator().manual_seed(85)
    q, k, v = _rand(gen, B, H, T, d, dtype=dtype), _rand(gen, B, Hk, T, d, dtype=dtype), _rand(gen, B, Hk, T, d, dtype=dtype)
    f = ref.attn(_host(q), _host(k), _host(v), d ** -0.5, ref.seen(T, T, 0, None), dtype)
    width = -(-T // page)
    kp, vp = (torch.full((B * width, page, Hk, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.randperm(B * width, generator=gen).int().view(B, width).cuda()
    out = torch.empty_like(q)
    at = 0
    for n in (1, 33, 40):
        rows = lambda x: x[:, :, at:at + n].transpose(1, 2).flatten(0, 1).contiguous()  # noqa: B023, E731
        lens = torch.full((B,), at + n, dtype=torch.int32, device="cuda")
        pdn.pdn_cache_append(rows(k), rows(v), kp, vp, table, lens)
        o = torch.empty(B * n, H, d, dtype=torch.bfloat16, device="cuda")
        pdn.pdn_attn_paged(rows(q), o, kp, vp, table, lens)
        out[:, :, at:at + n] = o.unflatten(0, (B, n)).transpose(1, 2)
        at += n
    lens = torch.full((B,), at, dtype=torch.int32, device="cuda")
    q1, k1, v1 = (torch.empty(B, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hk, Hk))
    o1 = torch.empty_like(q1)

    def step():
        lens.add_(1)
        pdn.pdn_cache_append(k1, v1, kp, vp, table, lens)
        pdn.pdn_attn_paged(q1, o1, kp, vp, table, lens)

    for x, y in ((q1, q), (k1, k), (v1, v)):
        x.copy_(y[:, :, at])
    step()
    out[:, :, at] = o1
    at += 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    while at < T:
        for x, y in ((q1, q), (k1, k), (v1, v)):
            x.copy_(y[:, :, at])
        graph.replay()
        torch.cuda.synchronize()
        out[:, :, at] = o1
        at += 1
    assert int(lens[0]) == T
    _close("o", out, f["o"], f["bo"], dtype)


def test_far_pages():
    """Pages past 32-bit offsets."""
    torch, pdn = torch_mod(), _pdn()
    page, Hk, d = 16, 1, 64
    step = 1 << 27   # elements between pages: 20 pages span 5 GB
    base = torch.empty(20 * step + 4096, dtype=torch.bfloat16, device="cuda")
    kp = base.as_strided((20, page, Hk, d), (step, d, d, 1))
    vp = base.as_strided((20, page, Hk, d), (step, d, d, 1), 2048)
    gen = torch.Generator().manual_seed(86)
    near_k, near_v = torch.zeros(20, page, Hk, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(20, page, Hk, d, dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(20, generator=gen).int()[None].cuda()
    lens = torch.tensor([317], dtype=torch.int32, device="cuda")
    k, v, q = _rand(gen, 317, Hk, d, dtype="bf16"), _rand(gen, 317, Hk, d, dtype="bf16"), _rand(gen, 317, 2, d, dtype="bf16")
    pdn.pdn_cache_append(k, v, near_k, near_v, table, lens)
    pdn.pdn_cache_append(k, v, kp, vp, table, lens)
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    pdn.pdn_attn_paged(q, o, near_k, near_v, table, lens)
    pdn.pdn_attn_paged(q, o2, kp, vp, table, lens)
    assert torch.equal(o, o2) and torch.isfinite(o.float()).all()


def test_layer_of_a_hybrid_stack():
    """The seam, q/k norm with rotation, attention and the output norm of one layer,
    forward and backward through the library's calls, against the same in 64 bits
    with autograd; the projections are plain products."""
    torch, pdn = torch_mod(), _pdn()
    B, T, H, Hk, d, D, window = 2, 75, 4, 2, 64, 256, 40
    gen = torch.Generator().manual_seed(87)
    x, res = _rand(gen, B, T, D), _rand(gen, B, T, D)
    w, wq, wk, wo = (1 + _rand(gen, n, scale=0.1) for n in (D, d, d, d))
    proj, back = _rand(gen, D, (H + 2 * Hk) * d, scale=D ** -0.5), _rand(gen, H * d, D, scale=(H * d) ** -0.5)
    key = torch.tensor([17, 4], dtype=torch.int64, device="cuda")
    drop, rot = 0.1, 64
    freqs, _ = pdn.pdn_rope_freqs(rot)
    inv = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    first = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    first[1, 30:] = 30
    positions = (torch.arange(T, device="cuda") - first).contiguous()
    dout, ds_in = _rand(gen, B, T, D), _rand(gen, B, T, D)
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731

    # forward
    s, y = e(B, T, D), e(B, T, D)
    pdn.pdn_add_norm_fwd(x, y, res=res, s=s, w=w, drop_p=drop, seed=key)
    rows = (y @ proj).unflatten(2, (-1, d))
    xq, xk, v = rows[:, :, :H], rows[:, :, H:H + Hk], rows[:, :, H + Hk:].transpose(1, 2)
    q, k = e(B, H, T, d), e(B, H, T, d)
    qk = dict(norm=pdn.PDN_NORM_RMS, wq=wq, wk=wk, inv_freq=inv, positions=positions)
    pdn.pdn_qk_norm_fwd(xq, xk, q, k, **qk)
    kk = k[:, ::H // Hk]
    o, lse = e(B, H, T, d), e(B, H, T)
    at = dict(window=window, first=first)
    pdn.pdn_attn_fwd(q, kk, v, o, lse=lse, **at)
    z = e(B, T, H, d)
    pdn.pdn_out_norm_fwd(o, z, w=wo)
    out = z.flatten(2) @ back

    # backward
    dz = (dout @ back.T).unflatten(2, (H, d))
    do, dwo = e(B, H, T, d), e(d)
    pdn.pdn_out_norm_bwd(o, dz, do, w=wo, dw=dwo)
    dq, dk = e(B, H, T, d), torch.zeros(B, H, T, d, device="cuda")
    drows = e(B, T, H + 2 * Hk, d)
    pdn.pdn_attn_bwd(q, kk, v, o, do, lse, dq, dk[:, ::H // Hk], drows[:, :, H + Hk:].transpose(1, 2), **at)
    dwq, dwk = e(d), e(d)
    pdn.pdn_qk_norm_bwd(xq, xk, dq, dk, drows[:, :, :H], drows[:, :, H:H + Hk], dwq=dwq, dwk=dwk, **qk)
    dy = drows.flatten(2) @ proj.T
    dres, dx, dw = e(B, T, D), e(B, T, D), e(D)
    pdn.pdn_add_norm_bwd(s, dy, dres, ds=ds_in, dx=dx, w=w, dw=dw, drop_p=drop, seed=key)
    torch.cuda.synchronize()

    # the same in 64 bits
    g = {n: _host(t).requires_grad_() for n, t in dict(x=x, res=res, w=w, wq=wq, wk=wk, wo=wo).items()}
    keep, factor = ref.philox_keeps(key.tolist(), x.numel(), drop)
    s64 = g["res"] + torch.where(keep.view(B, T, D), g["x"] * factor, torch.zeros(()).double())
    rms = lambda t: t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    rows = (rms(s64) * g["w"] @ _host(proj)).unflatten(2, (-1, d))
    ang = _host(positions.double())[:, :, None, None] * _host(inv)

    def turned(t, weight):
        t = rms(t) * weight
        a, b = t[..., :rot // 2], t[..., rot // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1).transpose(1, 2)

    q64, k64 = turned(rows[:, :, :H], g["wq"]), turned(rows[:, :, H:H + Hk], g["wk"]).repeat_interleave(H // Hk, 1)
    v64 = rows[:, :, H + Hk:].transpose(1, 2).repeat_interleave(H // Hk, 1)
    mask = ref.seen(T, T, window, first.cpu())[:, None]
    o64 = torch.softmax((q64 @ k64.mT * d ** -0.5).masked_fill(~mask, -torch.inf), -1) @ v64
    out64 = (rms(o64) * g["wo"]).transpose(1, 2).flatten(2) @ _host(back)
    grads = torch.autograd.grad((out64 * _host(dout)).sum() + (s64 * _host(ds_in)).sum(), list(g.values()))
    # a chain of a dozen operators of some 2^-20 each (products of 256 terms, norms), forward and back
    for name, got, want in [("out", out, out64.detach())] + [(n, t, u) for n, t, u in zip(g, (dx, dres, dw, dwq, dwk, dwo), grads)]:
        off = ((_host(got) - want).norm() / want.norm()).item()
        print("[layer] %s %.2e" % (name, off), flush=True)
        assert off < 2e-5, name


def test_binding_refusals():
    torch, pdn = torch_mod(), _pdn()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32
    q, o, kp, vp = z(4, 4, 64), z(4, 4, 64), z(6, 16, 2, 64), z(6, 16, 2, 64)
    ok = dict(q=q, o=o, k_pages=kp, v_pages=vp, table=z(2, 3, dtype=i32), lens=z(2, dtype=i32))
    pdn.pdn_attn_paged(**ok)
    for bad in (dict(q=z(5, 4, 64), o=z(5, 4, 64)), dict(q=z(4, 4, 128), o=z(4, 4, 128)), dict(lens=z(3, dtype=i32)), dict(lens=z(2, dtype=torch.int64)),
                dict(table=z(2, 3, dtype=torch.int64)), dict(starts=z(2, dtype=i32)), dict(v_pages=z(6, 16, 2, 128)), dict(v_pages=vp.float()),
                dict(k_pages=z(6, 24, 2, 64), v_pages=z(6, 24, 2, 64)), dict(max_new=1), dict(max_new=-1), dict(scale=0.0), dict(q=q.float()),
                dict(o=z(4, 4, 64, dtype=torch.float16)), dict(lse=z(4, 4)), dict(q=z(4, 3, 64), o=z(4, 3, 64)), dict(lens=z(2, dtype=i32).cpu()),
                dict(table=z(0, 3, dtype=i32), lens=z(0, dtype=i32))):
        with pytest.raises((ValueError, pdn.PdnError)):
            pdn.pdn_attn_paged(**{**ok, **bad})
    ok = dict(k=z(4, 2, 64), v=z(4, 2, 64), k_pages=kp, v_pages=vp, table=z(2, 3, dtype=i32), lens=z(2, dtype=i32))
    pdn.pdn_cache_append(**ok)
    for bad in (dict(k=z(4, 1, 64)), dict(v=z(3, 2, 64)), dict(k=z(4, 2, 64).float()), dict(k=z(3, 2, 64), v=z(3, 2, 64)), dict(k=z(4, 128))):
        with pytest.raises((ValueError, pdn.PdnError)):
            pdn.pdn_cache_append(**{**ok, **bad})
