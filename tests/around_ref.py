"""64-bit references (numpy) of the operators around the recurrence, each with
the elementwise bound that fp32 arithmetic can be off by.

U = 2^-24 is half a step of fp32 (the bound of one rounding, relative).  The
bounds count roundings on the way to a result; an output's own rounding
(HALF[type], relative to the value) is added by the tests.

  norm    r = rsqrt(c sum x^2 + eps): 8 fused terms in a lane and up to 5 adds
          across lanes, one for c and eps, halved by the root, and one step of
          the root itself: under 10 U
  rotate  cos and sin of an angle whose turn fraction is rounded once to fp32
          (2 pi 2^-25 absolute, 3.2 U) by a function good to 2 steps (4 U)
"""
import numpy as np

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}   # half a step, relative


def bf16(x):
    """The nearest bf16 (ties to even) of a float32 array, as float32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000
    return u.astype(np.uint32).view(np.float32)


# -- q/k norm and rotation ---------------------------------------------------

def rotation(positions, inv_freq, d, layout, rope_scale):
    """cos [B,T,1,d], sin with its element's sign, and each element's partner."""
    rot = 2 * len(inv_freq)
    c, s = np.full(positions.shape + (1, d), 1.0), np.zeros(positions.shape + (1, d))
    partner = np.arange(d)
    ang = positions[..., None, None].astype(np.float64) * inv_freq
    for p in range(rot // 2):
        i, j = (p, p + rot // 2) if layout == 0 else (2 * p, 2 * p + 1)
        c[..., i] = c[..., j] = np.cos(ang[..., p]) * rope_scale
        s[..., i] = -np.sin(ang[..., p]) * rope_scale
        s[..., j] = np.sin(ang[..., p]) * rope_scale
        partner[i], partner[j] = j, i
    return c, s, partner


def norm_factor(x, norm, eps):
    d = x.shape[-1]
    if norm == 0:
        return np.ones(x.shape[:-1] + (1,)), 0.0
    mean = 1.0 / d if norm == 1 else 1.0
    return 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) * mean + eps), mean


def qk_one(x, w, scale, H, norm, eps, rot):
    """[B,T,Hx,d] -> ([B,H,T,d], bound)."""
    r, _ = norm_factor(x, norm, eps)
    n = x * r * scale * (1.0 if w is None else w)
    if rot is None:
        y, env = n, np.abs(n)
    else:
        c, s, partner = rot
        y = n * c + n[..., partner] * s
        # the angle is off by up to 8 U whatever its cosine is
        top = max(1.0, np.abs(c).max())
        env = top * (np.abs(n) + np.abs(n[..., partner]))
    rep = H // x.shape[2]
    order = lambda t: np.repeat(t, rep, axis=2).transpose(0, 2, 1, 3)
    return order(y), order(env) * 24 * U


def qk_one_bwd(x, w, scale, g, norm, eps, rot):
    """(dx, bound, dw, bound) from g [B,H,T,d]."""
    B, T, Hx, d = x.shape
    rep = g.shape[1] // Hx
    gs = g.transpose(0, 2, 1, 3).reshape(B, T, Hx, rep, d)
    ga = np.abs(gs).sum(3)
    gs = gs.sum(3)
    if rot is not None:
        c, s, partner = rot
        gs = gs * c - gs[..., partner] * s
        ga = max(1.0, np.abs(c).max()) * (ga + ga[..., partner])
    r, mean = norm_factor(x, norm, eps)
    gs, ga = gs * scale, ga * abs(scale)
    wv = 1.0 if w is None else w
    if norm == 0:
        return gs, ga * (16 + rep) * U, None, None
    gw, gwa = gs * wv, ga * np.abs(wv)
    dot = (gw * x).sum(-1, keepdims=True)
    dota = (gwa * np.abs(x)).sum(-1, keepdims=True)
    dx = r * (gw - x * r * r * mean * dot)
    # 16 + rep for the gradient, 14 for the sum, 3 x 10 for r^3, 6 products
    bound = r * (gwa + np.abs(x) * r * r * mean * dota) * (66 + rep) * U
    dw = (gs * x * r).sum((0, 1, 2))
    terms = B * T * Hx
    # a lane's own sum, 32 slots, then the workgroups': at most terms roundings in a chain
    dwb = (ga * np.abs(x) * r).sum((0, 1, 2)) * (30 + rep + min(terms, 200 + terms // 16)) * U
    return dx, bound, dw, dwb


# -- gated output norm -------------------------------------------------------

def act(kind, z):
    """(factor, derivative); 64 bits."""
    with np.errstate(over="ignore"):
        f = 1.0 / (1.0 + np.exp(-z))
    return (z * f, f * (1 + z * (1 - f))) if kind == 1 else (f, f * (1 - f))


def out_fwd(o, w, z, kind, eps):
    """o [B,H,T,d], z [B,T,H,d] -> (y [B,T,H,d], bound).  The sigmoid's
    argument is rounded once (|z| U in its value), exp2, add and rcp take 6 U."""
    x = o.transpose(0, 2, 1, 3)
    y = x * norm_factor(x, 1, eps)[0] * (1.0 if w is None else w)
    u = 16.0
    if kind:
        y = y * act(kind, z)[0]
        u = 24.0 + np.abs(z)
    return y, np.abs(y) * u * U


def out_bwd(o, w, z, dy, kind, eps):
    """(do [B,H,T,d], bound), (dz, bound) or None, (dw, bound)."""
    x = o.transpose(0, 2, 1, 3)
    r, mean = norm_factor(x, 1, eps)
    wv = 1.0 if w is None else w
    g, ga, u, dz = dy, np.abs(dy), 2.0, None
    if kind:
        f, slope = act(kind, z)
        n1 = dy * x * r * wv
        # f is off by (|z| + 8) U at most, and so is 1 - f, whatever is left of it
        dz = (n1 * slope, np.abs(n1) * (1 + np.abs(z)) * (40 + 2 * np.abs(z)) * U)
        g, ga, u = dy * f, np.abs(dy * f), 10.0 + np.abs(z)
    gw, gwa = g * wv, ga * np.abs(wv)
    dot = (gw * x).sum(-1, keepdims=True)
    dota = (gwa * np.abs(x)).sum(-1, keepdims=True)
    um = np.max(u, axis=-1, keepdims=True) if np.ndim(u) else u
    do = r * (gw - x * r * r * mean * dot)
    dob = r * (gwa + np.abs(x) * r * r * mean * dota) * (52 + um) * U
    terms = x.shape[0] * x.shape[1] * x.shape[2]
    dw = (g * x * r).sum((0, 1, 2))
    dwb = (ga * np.abs(x) * r * (30 + u + min(terms, 200 + terms // 16))).sum((0, 1, 2)) * U
    t = lambda a: a.transpose(0, 2, 1, 3)
    return (t(do), t(dob)), dz, (dw, dwb)


# -- scan --------------------------------------------------------------------

def gain(kind, la, a):
    """(gain, derivative by la)."""
    if kind == 0:
        return np.ones_like(a), np.zeros_like(a)
    if kind == 1:
        return -np.expm1(la), -a
    g = np.sqrt(-np.expm1(2 * la))
    with np.errstate(divide="ignore"):
        return g, -a * a / g


def scan_fwd(x, la, h0, kind):
    """[B,T,D] -> (h, bound): a carries (|la| + 4) U; a zero decay drops the
    state.  The tile's products add a rounding a token, their joins 16 in all."""
    with np.errstate(invalid="ignore"):
        a = np.exp(la)
        g, _ = gain(kind, la, a)
        b = g * x
    h, bound = np.empty_like(x), np.empty_like(x)
    s = np.zeros_like(x[:, 0]) if h0 is None else h0.astype(np.float64)
    env, err = np.abs(s), np.zeros_like(s)
    with np.errstate(invalid="ignore"):
        for t in range(x.shape[1]):
            at, dropped = a[:, t], a[:, t] == 0
            lat = np.where(dropped, 0.0, np.abs(la[:, t]))
            err = np.where(dropped, 0.0, at * (err + (lat + 5) * U * env)) + np.abs(b[:, t]) * 10 * U
            env = np.where(dropped, 0.0, at * env) + np.abs(b[:, t])
            err = err + env * U
            s = np.where(dropped, 0.0, at * s) + b[:, t]
            h[:, t], bound[:, t] = s, err + 16 * U * env
    return h, bound


def scan_bwd(x, la, h0, dh, dhT, kind):
    """(dx, bound), (dlog_a, bound), (dh0, bound)."""
    h, hb = scan_fwd(x, la, h0, kind)
    zero = np.zeros_like(x[:, 0])
    before = np.concatenate([(zero if h0 is None else h0)[:, None], h[:, :-1]], 1)
    beforeb = np.concatenate([zero[:, None], hb[:, :-1]], 1)
    a = np.exp(la)
    g, slope = gain(kind, la, a)
    c = zero if dhT is None else dhT.astype(np.float64)
    env, err = np.abs(c), np.zeros_like(c)
    out = [np.empty_like(x) for _ in range(4)]
    with np.errstate(invalid="ignore"):
        for t in reversed(range(x.shape[1])):
            at, dropped = a[:, t], a[:, t] == 0
            lat = np.where(dropped, 0.0, np.abs(la[:, t]))
            G, E = dh[:, t] + c, np.abs(dh[:, t]) + env
            ge = err + 17 * U * E
            keep = lambda v: np.where(dropped, 0.0, at * v)
            out[0][:, t] = g[:, t] * G
            out[1][:, t] = np.abs(g[:, t]) * (ge + 10 * U * E)
            out[2][:, t] = keep(before[:, t]) * G + slope[:, t] * x[:, t] * G
            out[3][:, t] = (keep(np.abs(before[:, t])) * (ge + (lat + 8) * U * E) + keep(beforeb[:, t]) * E
                            + np.abs(slope[:, t] * x[:, t]) * (ge + 24 * U * E))
            c, err, env = keep(G), keep(err + (lat + 6) * U * E), keep(E)
    return (out[0], out[1]), (out[2], out[3]), (c, err + 17 * U * env)
