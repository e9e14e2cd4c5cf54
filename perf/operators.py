"""The operators around the delta rule, as cases to be timed and compared: the norm and rotation of
queries and keys into the recurrence's layout (``qk_norm``), the gated linear recurrence with a vector
state (``scan``) and the gated norm of the recurrence's output (``out_norm``), forward and backward.

Each case has a plain form in elementary torch operations (``own`` false), the library's calls (``own``
true) and the definition in 64 bits (``exact``)."""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}
_EPS = 1e-6


def listed():
    return [
        # one token for each of 32 sequences far into their contexts: a decode step's q and k
        dict(name="qk_decode", op="qk_norm", way="fwd", B=32, T=1, Hq=16, Hk=16, H=16, d=128, dtype="bf16",
             norm="l2", weight=False, rot=128, layout="half", stretch=1.0, pos0=60000),
        # the prefill workload (B4 H16 T8192 d128): L2 norm alone, as gated delta-rule layers use it
        dict(name="qk_prefill", op="qk_norm", way="fwd", B=4, T=8192, Hq=16, Hk=16, H=16, d=128, dtype="bf16",
             norm="l2", weight=False, rot=0, layout="half", stretch=1.0, pos0=0),
        # one long sequence, fewer key heads than value heads, RMS norm with weights, half of each head
        # rotated, frequencies stretched for positions past the trained length
        dict(name="qk_long_grouped", op="qk_norm", way="fwd", B=1, T=65536, Hq=16, Hk=4, H=16, d=128, dtype="bf16",
             norm="rms", weight=True, rot=64, layout="half", stretch=8.0, pos0=983040),
        # the backward of the two-sequence, 32-head workload: fp32 gradients as the recurrence's backward
        # leaves them, interleaved pairs
        dict(name="qk_backward", op="qk_norm", way="bwd", B=2, T=8192, Hq=32, Hk=32, H=32, d=128, dtype="bf16",
             norm="rms", weight=True, rot=128, layout="interleaved", stretch=1.0, pos0=0),
        # a ragged fp32 backward with shared heads of 64
        dict(name="qk_backward_fp32", op="qk_norm", way="bwd", B=3, T=1237, Hq=4, Hk=2, H=8, d=64, dtype="fp32",
             norm="l2", weight=True, rot=32, layout="half", stretch=4.0, pos0=17),
        # one token of the vector-state recurrence for 256 sequences
        dict(name="scan_step", op="scan", way="step", B=256, T=1, D=2048, dtype="bf16", ldtype="fp32",
             gain="norm", packed=False),
        # four prompts, decays in fp32 as the library's other decays are
        dict(name="scan_prefill", op="scan", way="fwd", B=4, T=8192, D=2048, dtype="bf16", ldtype="fp32",
             gain="norm", packed=False),
        # one long packed row of several sequences, decays in bf16
        dict(name="scan_long", op="scan", way="fwd", B=1, T=65536, D=2048, dtype="bf16", ldtype="bf16",
             gain="none", packed=True),
        # a training step's share: forward, then backward
        dict(name="scan_train", op="scan", way="train", B=2, T=8192, D=4096, dtype="bf16", ldtype="bf16",
             gain="norm", packed=True),
        # a ragged fp32 training step
        dict(name="scan_train_fp32", op="scan", way="train", B=3, T=1237, D=520, dtype="fp32", ldtype="fp32",
             gain="complement", packed=False),
        # the prefill workload's output through the gated norm, back to the model's layout
        dict(name="out_prefill", op="out_norm", way="fwd", B=4, T=8192, H=16, d=128, odtype="fp32", dtype="bf16",
             act="silu", weight=True),
        # and its backward for the 32-head workload
        dict(name="out_backward", op="out_norm", way="bwd", B=2, T=8192, H=32, d=128, odtype="fp32", dtype="bf16",
             act="silu", weight=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["qk_norm", "scan", "out_norm"])
    if op == "scan":
        D = 8 * _spread(rng, 8, 640)
        way = rng.choice(["fwd", "train", "train", "step"])
        if way == "step":
            B, T = _spread(rng, 1, 512), 1
        else:
            B = _spread(rng, 1, 16)
            T = min(_spread(rng, 1, 65536), max(1, (1 << (26 if way == "train" else 27)) // (B * D)))
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, way=way, B=B, T=T, D=D, dtype=dtype,
                    ldtype="fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"]),
                    gain=rng.choice(["none", "complement", "norm"]), packed=rng.random() < 0.5 and T > 1)
    B = _spread(rng, 1, 64)
    H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
    way = rng.choice(["fwd", "bwd"])
    if op == "out_norm":
        d = 16 * rng.randint(1, 16)
        T = min(_spread(rng, 1, 32768), max(1, (1 << 26) // (B * H * d)))
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, way=way, B=B, T=T, H=H, d=d,
                    odtype="fp32" if dtype == "fp32" or way == "bwd" else rng.choice(["fp32", "bf16"]), dtype=dtype,
                    act=rng.choice(["silu", "sigmoid", "none"]), weight=rng.random() < 0.7)
    d = rng.choice([64, 128])
    T = min(_spread(rng, 1, 65536), max(1, (1 << 26) // (B * H * d)))
    parts = [n for n in range(1, H + 1) if H % n == 0]
    rot = 16 * rng.randint(0, d // 16)
    return dict(op=op, way=way, B=B, T=T, Hq=rng.choice(parts), Hk=rng.choice(parts), H=H, d=d,
                dtype=rng.choice(["bf16", "bf16", "fp32"]), norm=rng.choice(["l2", "rms", "none"] if rot else ["l2", "rms"]),
                weight=rng.random() < 0.5, rot=rot, layout=rng.choice(["half", "interleaved"]),
                stretch=rng.choice([1.0, 1.0, 2.0, 8.0]), pos0=rng.choice([0, 0, _spread(rng, 1, 1 << 20)]))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    s = {"case": c}
    if c["op"] == "qk_norm":
        B, T, Hq, Hk, H, d = (c[n] for n in ("B", "T", "Hq", "Hk", "H", "d"))
        # one projection holds q, k and v side by side: q and k are views into its rows
        rows = normal(B, T, (Hq + Hk + H) * d, dtype=_DT[c["dtype"]])
        s["xq"] = rows[:, :, :Hq * d].unflatten(2, (Hq, d))
        s["xk"] = rows[:, :, Hq * d:(Hq + Hk) * d].unflatten(2, (Hk, d))
        s["wq"] = 1 + normal(d, scale=0.1) if c["weight"] and c["norm"] != "none" else None
        s["wk"] = 1 + normal(d, scale=0.1) if c["weight"] and c["norm"] != "none" else None
        # sequences of a batch stand at positions of their own
        s["positions"] = (c["pos0"] + 5 * torch.arange(B, device="cuda")[:, None] + torch.arange(T, device="cuda")[None, :]).contiguous() if c["rot"] else None
        i = torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = 10000.0 ** (-i / c["rot"]) / c["stretch"] if c["rot"] else None
        if c["way"] == "bwd":
            s["dq"], s["dk"] = normal(B, H, T, d), normal(B, H, T, d)
    elif c["op"] == "scan":
        B, T, D = c["B"], c["T"], c["D"]
        s["x"] = normal(B, T, D, dtype=_DT[c["dtype"]])
        # a per-channel rate that alone would leave 0.9 to 0.999 of the state, times a gate of the token
        rate = -torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda")) * 2
        la = normal(B, T, D).sigmoid_().mul_(rate).neg_()
        if c["packed"]:  # sequences packed into a row: the first token of each drops the state before it
            for b in range(B):
                at = torch.randint(0, T, (1 + T // 1500,), generator=gen, device="cuda")
                la[b, at] = -math.inf
        s["la"] = la.to(_DT[c["ldtype"]])
        s["h0"] = normal(B, D)
        if c["way"] == "train":
            s["dh"], s["dhT"] = normal(B, T, D, dtype=_DT[c["dtype"]]), normal(B, D)
    else:
        B, T, H, d = c["B"], c["T"], c["H"], c["d"]
        s["o"] = normal(B, H, T, d, dtype=_DT[c["odtype"]], scale=0.3)
        # the gate lies beside another part of the same projection's rows
        s["z"] = normal(B, T, 2 * H * d, dtype=_DT[c["dtype"]])[:, :, H * d:].unflatten(2, (H, d)) if c["act"] != "none" else None
        s["w"] = 1 + normal(d, scale=0.1) if c["weight"] else None
        if c["way"] == "bwd":
            s["dy"] = normal(B, T, H, d, dtype=_DT[c["dtype"]])
    return s


def work(case):
    c = case
    if c["op"] == "qk_norm":
        n = c["B"] * c["T"] * c["d"]
        e = _BYTES[c["dtype"]]
        side = n * (c["Hq"] + c["Hk"]) * e
        small = c["B"] * c["T"] * 8 * (c["rot"] > 0) + 4 * c["rot"]
        if c["way"] == "fwd":
            return {"bytes": side + n * 2 * c["H"] * e + small, "flops": n * (c["Hq"] + c["Hk"]) * 8}
        return {"bytes": 2 * side + n * 2 * c["H"] * 4 + small, "flops": n * (c["Hq"] + c["Hk"]) * 14}
    if c["op"] == "scan":
        n, e, l = c["B"] * c["T"] * c["D"], _BYTES[c["dtype"]], _BYTES[c["ldtype"]]
        state = 8 * c["B"] * c["D"]
        if c["way"] == "train":  # x, la, dh once; h, dx, dla once
            return {"bytes": n * (4 * e + 2 * l) + 2 * state, "flops": n * 14}
        return {"bytes": n * (2 * e + l) + state, "flops": n * 5}
    n, e, f = c["B"] * c["T"] * c["H"] * c["d"], _BYTES[c["dtype"]], _BYTES[c["odtype"]]
    gate = c["act"] != "none"
    if c["way"] == "fwd":
        return {"bytes": n * (f + e + gate * e), "flops": n * 10}
    return {"bytes": n * (2 * f + e + gate * 2 * e), "flops": n * 20}


def _scales(c):
    """(what the sum of squares is multiplied by, what q and k are): no norm leaves the rows as they are."""
    return {"l2": 1.0, "rms": 1.0 / c["d"], "none": None}[c["norm"]], c["d"] ** -0.5, 1.0


def _angles(s):
    t = s["positions"].double()[:, :, None, None] * s["inv_freq"]
    return t.cos().float(), t.sin().float()


def _halves(c, y):
    """The first and second elements of the rotated pairs."""
    r = y[..., :c["rot"]]
    if c["layout"] == "half":
        return r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
    return r[..., 0::2], r[..., 1::2]


def _joined(c, u, v, y):
    r = torch.cat([u, v], -1) if c["layout"] == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([r, y[..., c["rot"]:]], -1)


def _qk_fwd(s):
    c, out = s["case"], []
    m, *scales = _scales(c)
    cs = _angles(s) if c["rot"] else None
    for x, w, scale in ((s["xq"], s["wq"], scales[0]), (s["xk"], s["wk"], scales[1])):
        x = x.float()
        y = x * scale if m is None else x * ((x * x).sum(-1, keepdim=True) * m + _EPS).rsqrt() * scale
        if w is not None:
            y = y * w
        if cs is not None:
            u, v = _halves(c, y)
            y = _joined(c, u * cs[0] - v * cs[1], v * cs[0] + u * cs[1], y)
        y = y.repeat_interleave(c["H"] // y.shape[2], 2)
        out.append(y.permute(0, 2, 1, 3).to(_DT[c["dtype"]]).contiguous())
    return {"q": out[0], "k": out[1]}


def _qk_bwd(s):
    c, out = s["case"], {}
    m, *scales = _scales(c)
    cs = _angles(s) if c["rot"] else None
    for n, scale in (("q", scales[0]), ("k", scales[1])):
        x, w, g = s["x" + n].float(), s["w" + n], s["d" + n]
        g = g.permute(0, 2, 1, 3).unflatten(2, (x.shape[2], -1)).sum(3)
        if cs is not None:
            u, v = _halves(c, g)
            g = _joined(c, u * cs[0] + v * cs[1], v * cs[0] - u * cs[1], g)
        g = g * scale
        if m is not None:
            r = ((x * x).sum(-1, keepdim=True) * m + _EPS).rsqrt()
            if w is not None:
                out["dw" + n] = (g * x * r).sum((0, 1, 2))
                g = g * w
            g = r * (g - x * (r * r * m) * (g * x).sum(-1, keepdim=True))
        out["dx" + n] = g.to(_DT[c["dtype"]])
    return out


def _gain(c, la, a):
    """The gain of the input, and its derivative by the logarithm of the decay."""
    if c["gain"] == "none":
        return torch.ones_like(a), torch.zeros_like(a)
    if c["gain"] == "complement":
        return -torch.expm1(la), -a
    g = torch.sqrt(-torch.expm1(2 * la))
    return g, -a * a / g


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along the second axis, in steps that double what each element covers."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _scan_fwd(s):
    c = s["case"]
    la = s["la"].float()
    a = la.exp()
    b = _gain(c, la, a)[0] * s["x"].float()
    b[:, 0] += a[:, 0] * s["h0"]
    return _recur(a, b)


def _scan(s):
    c = s["case"]
    h = _scan_fwd(s)
    out = {"h": h.to(_DT[c["dtype"]]), "hT": h[:, -1].clone()}
    if c["way"] == "train":
        la, x = s["la"].float(), s["x"].float()
        a = la.exp()
        after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
        g = s["dh"].to(torch.float32, copy=True)  # the state's own gradient stays as it is
        g[:, -1] += s["dhT"]
        g = _recur(after.flip(1), g.flip(1)).flip(1)
        gain, slope = _gain(c, la, a)
        before = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
        out.update(dx=(gain * g).to(_DT[c["dtype"]]), dla=((a * before + slope * x) * g).to(_DT[c["ldtype"]]), dh0=a[:, 0] * g[:, 0])
    return out


def _act(c, z):
    """The gate's factor, and its derivative."""
    p = 1 / (1 + torch.exp(-z))
    return (z * p, p * (1 + z * (1 - p))) if c["act"] == "silu" else (p, p * (1 - p))


def _out_fwd(s):
    c = s["case"]
    o = s["o"].float().permute(0, 2, 1, 3)
    y = o * ((o * o).mean(-1, keepdim=True) + _EPS).rsqrt()
    if s["w"] is not None:
        y = y * s["w"]
    if s["z"] is not None:
        y = y * _act(c, s["z"].float())[0]
    return {"y": y.to(_DT[c["dtype"]]).contiguous()}


def _out_bwd(s):
    c, out = s["case"], {}
    o = s["o"].float().permute(0, 2, 1, 3)
    r = ((o * o).mean(-1, keepdim=True) + _EPS).rsqrt()
    g = s["dy"].float()
    n = o * r
    if s["z"] is not None:
        f, slope = _act(c, s["z"].float())
        out["dz"] = (g * (n if s["w"] is None else n * s["w"]) * slope).to(_DT[c["dtype"]])
        g = g * f
    if s["w"] is not None:
        out["dw"] = (g * n).sum((0, 1, 2))
        g = g * s["w"]
    g = r * (g - n * (g * n).mean(-1, keepdim=True))
    out["do"] = g.permute(0, 2, 1, 3).contiguous()
    return out


def run(state):
    c = state["case"]
    if own:
        return _own(state)
    if c["op"] == "qk_norm":
        return _qk_fwd(state) if c["way"] == "fwd" else _qk_bwd(state)
    if c["op"] == "scan":
        return _scan(state)
    return _out_fwd(state) if c["way"] == "fwd" else _out_bwd(state)


def _own(s):
    import gated_delta_rule_77_amd as pdn
    c = s["case"]
    if c["op"] == "qk_norm":
        B, T, Hq, Hk, H, d = (c[n] for n in ("B", "T", "Hq", "Hk", "H", "d"))
        norm = {"l2": pdn.PDN_NORM_L2, "rms": pdn.PDN_NORM_RMS, "none": pdn.PDN_NORM_NONE}[c["norm"]]
        same = dict(norm=norm, eps=_EPS, wq=s["wq"], wk=s["wk"], q_scale=d ** -0.5, inv_freq=s["inv_freq"], positions=s["positions"],
                    rope_layout=pdn.PDN_ROPE_HALF if c["layout"] == "half" else pdn.PDN_ROPE_INTERLEAVED)
        new = dict(dtype=_DT[c["dtype"]], device="cuda")
        if c["way"] == "fwd":
            q, k = torch.empty((B, H, T, d), **new), torch.empty((B, H, T, d), **new)
            pdn.pdn_qk_norm_fwd(s["xq"], s["xk"], q, k, **same)
            return {"q": q, "k": k}
        out = {"dxq": torch.empty((B, T, Hq, d), **new), "dxk": torch.empty((B, T, Hk, d), **new)}
        if s["wq"] is not None:
            out["dwq"], out["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
        pdn.pdn_qk_norm_bwd(s["xq"], s["xk"], s["dq"], s["dk"], out["dxq"], out["dxk"], dwq=out.get("dwq"), dwk=out.get("dwk"), **same)
        return out
    if c["op"] == "scan":
        gain = {"none": pdn.PDN_GAIN_NONE, "complement": pdn.PDN_GAIN_COMPLEMENT, "norm": pdn.PDN_GAIN_NORM}[c["gain"]]
        h, hT = torch.empty_like(s["x"]), torch.empty_like(s["h0"])
        if c["way"] == "step":
            pdn.pdn_scan_step(s["x"][:, 0], s["la"][:, 0], h[:, 0], s["h0"], hT, gain=gain)
            return {"h": h, "hT": hT}
        if c["way"] == "fwd":
            pdn.pdn_scan_fwd(s["x"], s["la"], h, h0=s["h0"], hT=hT, gain=gain)
            return {"h": h, "hT": hT}
        marks = torch.empty((c["B"], pdn.pdn_scan_marks(c["T"]), c["D"]), device="cuda")
        pdn.pdn_scan_fwd(s["x"], s["la"], h, h0=s["h0"], hT=hT, marks=marks, gain=gain)
        dx, dla, dh0 = torch.empty_like(s["x"]), torch.empty_like(s["la"]), torch.empty_like(s["h0"])
        pdn.pdn_scan_bwd(s["x"], s["la"], s["dh"], dx, dla, h0=s["h0"], dhT=s["dhT"], dh0=dh0, marks=marks, gain=gain)
        return {"h": h, "hT": hT, "dx": dx, "dla": dla, "dh0": dh0}
    act = {"none": pdn.PDN_ACT_NONE, "silu": pdn.PDN_ACT_SILU, "sigmoid": pdn.PDN_ACT_SIGMOID}[c["act"]]
    if c["way"] == "fwd":
        y = torch.empty((c["B"], c["T"], c["H"], c["d"]), dtype=_DT[c["dtype"]], device="cuda")
        pdn.pdn_out_norm_fwd(s["o"], y, z=s["z"], w=s["w"], act=act, eps=_EPS)
        return {"y": y}
    out = {"do": torch.empty_like(s["o"])}
    if s["z"] is not None:
        out["dz"] = torch.empty((c["B"], c["T"], c["H"], c["d"]), dtype=_DT[c["dtype"]], device="cuda")
    if s["w"] is not None:
        out["dw"] = torch.empty_like(s["w"])
    pdn.pdn_out_norm_bwd(s["o"], s["dy"], out["do"], z=s["z"], dz=out.get("dz"), w=s["w"], dw=out.get("dw"), act=act, eps=_EPS)
    return out


def exact(case, seed):
    s, c = prepare(case, seed), case
    wide = {n: t.double().detach() for n, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point()}
    if c["op"] == "scan":
        return _exact_scan(c, wide)
    if c["op"] == "qk_norm":
        return _exact_qk(c, wide, s["positions"])
    leaves = [wide[n].requires_grad_(c["way"] == "bwd") for n in ("o", "z", "w") if n in wide]
    o = wide["o"].transpose(1, 2)
    y = o / torch.sqrt(torch.linalg.vector_norm(o, dim=-1, keepdim=True) ** 2 / c["d"] + _EPS)
    if "w" in wide:
        y = y * wide["w"]
    if "z" in wide:
        y = y * (torch.sigmoid(wide["z"]) * wide["z"] if c["act"] == "silu" else torch.sigmoid(wide["z"]))
    if c["way"] == "fwd":
        return {"y": y}
    return dict(zip(("d" + n for n in ("o", "z", "w") if n in wide), torch.autograd.grad(y, leaves, wide["dy"])))


def _exact_qk(c, wide, positions):
    out = {}
    for n, scale in (("q", 1 / math.sqrt(c["d"])), ("k", 1.0)):
        x, w = wide["x" + n].clone().requires_grad_(c["way"] == "bwd"), wide.get("w" + n)
        w = None if w is None else w.requires_grad_(c["way"] == "bwd")
        size = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2
        y = x if c["norm"] == "none" else x / torch.sqrt((size if c["norm"] == "l2" else size / c["d"]) + _EPS)
        y = y * scale if w is None else y * (w * scale)
        if c["rot"]:  # each pair as one complex number, turned by its angle
            first, rest = y[..., :c["rot"]], y[..., c["rot"]:]
            half = c["layout"] == "half"
            pairs = torch.view_as_complex((first.unflatten(-1, (2, -1)).transpose(-1, -2) if half else first.unflatten(-1, (-1, 2))).contiguous())
            angle = torch.outer(positions.flatten().double(), wide["inv_freq"]).view(c["B"], c["T"], 1, -1)
            turned = torch.view_as_real(pairs * torch.polar(torch.ones_like(angle), angle))
            y = torch.cat([(turned.transpose(-1, -2) if half else turned).flatten(-2), rest], -1)
        heads = torch.arange(c["H"], device=y.device) // (c["H"] // y.shape[2])
        y = y[:, :, heads].transpose(1, 2)
        if c["way"] == "fwd":
            out[n] = y
        else:
            grads = torch.autograd.grad(y, [x] if w is None else [x, w], wide["d" + n])
            out.update(zip(("dx" + n, "dw" + n), grads))
    return out


def _exact_scan(c, wide):
    """Token by token, over time-major copies."""
    la, x = (wide[n].transpose(0, 1).contiguous() for n in ("la", "x"))
    a = torch.exp(la)
    if c["gain"] == "none":
        gain, slope = torch.ones_like(a), torch.zeros_like(a)
    elif c["gain"] == "complement":
        gain, slope = -torch.expm1(la), -a
    else:
        gain = (-torch.expm1(2 * la)).sqrt()
        slope = -a.square() / gain
    b, h = gain * x, torch.empty_like(x)
    last = wide["h0"]
    for t in range(c["T"]):
        last = torch.addcmul(b[t], a[t], last, out=h[t])
    out = {"h": h.transpose(0, 1), "hT": last}
    if c["way"] == "train":
        dh, carry = wide["dh"].transpose(0, 1).contiguous(), wide["dhT"]
        for t in reversed(range(c["T"])):
            dh[t] += carry
            carry = a[t] * dh[t]
        dla = slope * x * dh
        dla[0] += carry * wide["h0"]
        dla[1:] += a[1:] * dh[1:] * h[:-1]
        out.update(dx=(gain * dh).transpose(0, 1), dla=dla.transpose(0, 1), dh0=carry)
    return out
