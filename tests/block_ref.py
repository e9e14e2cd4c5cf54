"""64-bit references (torch on the CPU) of the operators of include/pdn_block.h, each
with the elementwise bound that the kernels' arithmetic can be off by.

U = 2^-24 is half a step of fp32, HALF[type] that of an output's type (relative); the
bounds count roundings on the way to a result, and the tests add an output's own.

  seam       s: one product and one sum, exact in the order the formula gives but for
             their two roundings.  r = rsqrt(mean s^2 + eps): 32 fused terms in a lane
             at most, 10 sums over lanes and waves, the mean and eps, halved by the
             root, one step of the root: under 30 U.
  scores     d products, each added in fp32: (d + 2) U of sum |q k|, as matrix
             instructions may truncate where they add 2 U a step; times the scale this
             is what the exponent is off by, and so (relative) an exponential.
  sums       n terms: 2 (n + 8) U of the sum of magnitudes.
  P, dS      with bf16 operands each is rounded once: HALF["bf16"], relative.
"""
import torch

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24, "e4m3": 2.0 ** -4}
f64 = torch.float64


# -- the seam ----------------------------------------------------------------

def philox_keeps(seed, n, p):
    """Which of n elements dropout keeps, in Python's own integers: key seed[0],
    counter (n / 8, seed[1]), 16 bits an element."""
    limit = min(65535, round(p * 65536))
    m32, keep = 2 ** 32 - 1, []
    key, call = seed[0] % 2 ** 64, seed[1] % 2 ** 64
    for block in range((n + 7) // 8):
        c = [block & m32, block >> 32, call & m32, call >> 32]
        k = [key & m32, key >> 32]
        for _ in range(10):
            p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & m32, (p0 >> 32) ^ c[3] ^ k[1], p0 & m32]
            k = [(k[0] + 0x9E3779B9) & m32, (k[1] + 0xBB67AE85) & m32]
        keep += [((c[j // 2] >> (16 * (j % 2))) & 0xffff) >= limit for j in range(8)]
    return torch.tensor(keep[:n]), 65536 / (65536 - limit)


def held(x, dtype):
    """x (float64) to the nearest of a type, as float64."""
    return x.float().to(torch.bfloat16 if dtype == "bf16" else torch.float32).double()


def seam(x, res, w, eps, keep, factor):
    """(sum before it is held, y of a held sum, its bound) as functions of the sum."""
    d = x if keep is None else torch.where(keep, x * factor, torch.zeros_like(x))
    return d if res is None else res + d


def seam_norm(s, w, eps):
    r = ((s * s).mean(-1, keepdim=True) + eps).rsqrt()
    y = s * r * (1.0 if w is None else w)
    return y, y.abs() * 34 * U


def seam_bwd(s, dy, ds, w, eps, keep, factor):
    """dres, dx, dw and their bounds."""
    D = s.shape[-1]
    r = ((s * s).mean(-1, keepdim=True) + eps).rsqrt()
    g = dy if w is None else dy * w
    dot, size = (g * s).mean(-1, keepdim=True), (g * s).abs().mean(-1, keepdim=True)
    norm = r * (g - s * r * r * dot)
    dres = norm if ds is None else ds + norm
    # the sum of g s: 32 fused terms, 10 sums over lanes; r three times
    b = r * (g.abs() * 36 * U + (s * r * r).abs() * (dot.abs() * 110 * U + size * 2 * 44 * U)) + 4 * U * dres.abs()
    out = {"dres": (dres, b)}
    dx = dres if keep is None else torch.where(keep, dres * factor, torch.zeros_like(dres))
    bx = b if keep is None else torch.where(keep, b * factor + 2 * U * dx.abs(), torch.zeros_like(b))
    out["dx"] = (dx, bx)
    if w is not None:
        t = dy * s * r
        n = t[..., 0].numel()
        out["dw"] = (t.flatten(0, -2).sum(0), t.abs().flatten(0, -2).sum(0) * (34 + n) * U)
    return out


# -- attention ---------------------------------------------------------------

def seen(Tq, Tk, window, first):
    """[B or 1, Tq, Tk]: which keys each query sees."""
    p = torch.arange(Tq)[:, None] + Tk - Tq
    j = torch.arange(Tk)[None]
    m = j <= p
    if window:
        m = m & (j > p - window)
    m = m[None]
    return m if first is None else m & (j[None] >= first[:, :, None])


def attn(q, k, v, scale, mask, dtype):
    """o, lse and their bounds: q [B,H,Tq,d], k, v [B,Hk,Tk,d], mask [B or 1,Tq,Tk]."""
    rep, d = q.shape[1] // k.shape[1], q.shape[-1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    m = mask[:, None]
    some = m.any(-1)
    s = (q @ k.mT) * scale
    env = (q.abs() @ k.abs().mT) * scale
    x = s.masked_fill(~m, -torch.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.where(m, torch.exp(x - torch.where(some, lse, 0.0)[..., None]), torch.zeros_like(s))
    o = p @ v
    n = mask.shape[-1]
    # the exponent: the scores', the scale's and the maximum's roundings; the exponential's own
    e = torch.where(m, env * (d + 4) * 2 * U + s.abs() * 4 * U, torch.zeros_like(env)).amax(-1, keepdim=True) + 4 * U if n else torch.zeros(o.shape[:-1] + (1,), dtype=f64)
    size = p @ v.abs()
    half = HALF["bf16"] if dtype == "bf16" else 0.0
    bo = size * (half + 2 * e + 2 * (n + 8) * U) + o.abs() * (e + 2 * (n + 8) * U)
    bl = e[..., 0] + 2 * (n + 8) * U + torch.where(some, lse, 0.0).abs() * 4 * U
    return dict(o=o, bo=bo, lse=lse, bl=torch.where(some, bl, 0.0), p=p, e=e, s=s, k=k, v=v, some=some, mask=m, size=size)


def attn_bwd(q, k, v, o, do, scale, mask, dtype, rounded_do, odtype="fp32"):
    """dq, dk, dv and their bounds; o is what the backward is given.  rounded_do: dO is
    fp32 and rounded to bf16 for its products.  D_i is formed from o or from P: the two
    differ by o's own rounding, HALF[odtype] of sum |dO o|, and what o is off by
    otherwise: with bf16 P's rounding too, another HALF["bf16"] of sum |dO| (P |v|)."""
    Hk, rep, d = k.shape[1], q.shape[1] // k.shape[1], q.shape[-1]
    f = attn(q, k, v, scale, mask, dtype)
    p, kk, vv, m = f["p"], f["k"], f["v"], f["mask"]
    h = HALF["bf16"] if dtype == "bf16" else 0.0
    hd = HALF["bf16"] if rounded_do else 0.0
    do = torch.where(f["some"][..., None], do, torch.zeros_like(do))
    delta = (do * o).sum(-1, keepdim=True)
    size_d = (do * o).abs().sum(-1, keepdim=True)
    dp, size_p = do @ vv.mT, do.abs() @ vv.abs().mT
    off_d = HALF[odtype] * size_d + (h + 4 * f["e"] + 4 * (k.shape[2] + 8) * U) * (do.abs() * f["size"]).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    n, nq = k.shape[2], q.shape[2] * rep
    # an exponential against the forward's lse: the scores' error here, and there
    e = 2 * f["e"] + 2 * (n + 8) * U + 4 * U * torch.where(f["some"], f["lse"], 0.0).abs()[..., None]
    eds = p * (size_p * (hd + 2 * (d + 2) * U) + size_d * 2 * (d + 2) * U + off_d) + ds.abs() * (e + 4 * U)
    eds = eds * (1 + h) + ds.abs() * h
    ep = p * (e + 4 * U) * (1 + h) + p * h
    fold = lambda t: t.unflatten(1, (Hk, rep)).sum(2)  # noqa: E731  heads that share a key head
    acc, accq = 2 * (n + 8) * U, 2 * (nq + 8) * U
    out = {}
    out["dq"] = (scale * (ds @ kk), scale * (eds @ kk.abs() + acc * (ds.abs() @ kk.abs())))
    out["dk"] = (scale * fold(ds.mT @ q), scale * fold(eds.mT @ q.abs() + accq * (ds.abs().mT @ q.abs())))
    out["dv"] = (fold(p.mT @ do), fold(ep.mT @ do.abs() + (hd + accq) * (p.mT @ do.abs())))
    return out


# -- the paged cache ---------------------------------------------------------

def gathered(pages, table, length):
    """[length, Hk, d] of a sequence."""
    size = pages.shape[1]
    if length == 0:
        return pages[:0].flatten(0, 1)
    at = torch.arange(length)
    return pages[table[at // size].long(), at % size]
