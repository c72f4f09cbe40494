"""Cases of the operators around the MoE layer: residual addition with RMS norm
(forward and backward), the dense gated feed-forward block in bf16 (forward
and backward) and on MXFP8 operands.

`run` computes them in plain torch operations in 32 bits, or, where `own` is
true, through the package's entry points; `exact` computes them in 64 bits.
"""
import torch

own = False

EPS = 1e-6
B1, B2 = 4.0, 25.0        # SiTU caps of the framework's layers
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token entering a feed-forward layer: the latency of a small launch
        {"name": "norm t1 d7168", "op": "norm", "T": 1, "d": 7168, "res": "bf16", "fmt": "bf16"},
        # an odd batch at the latent width, fp32 residual stream, encoded for an MXFP8 product
        {"name": "norm mx t333 d3584", "op": "norm", "T": 333, "d": 3584, "res": "fp32", "fmt": "mxfp8"},
        # a prefill batch: pure memory traffic
        {"name": "norm t8192 d7168", "op": "norm", "T": 8192, "d": 7168, "res": "bf16", "fmt": "bf16"},
        # training: a micro-batch with the gradient that flows along the residual stream
        {"name": "norm bwd t4096 d7168", "op": "norm_bwd", "T": 4096, "d": 7168, "res": "bf16", "dh": True},
        # training of a narrow model, odd rows, first norm (no gradient along the stream)
        {"name": "norm bwd t509 d1152", "op": "norm_bwd", "T": 509, "d": 1152, "res": "bf16", "dh": False},
        # one decoded token through the shared MLP's width: streaming the weights
        {"name": "ffn t1 d7168 f6144", "op": "ffn", "T": 1, "d": 7168, "F": 6144, "act": "situ", "save": False},
        # a decode batch through the non-latent layer's shared MLP
        {"name": "ffn t64 d7168 f2048", "op": "ffn", "T": 64, "d": 7168, "F": 2048, "act": "swiglu", "save": False},
        # training forward, saving the pre-activations for the backward pass
        {"name": "ffn t4096 d7168 f6144", "op": "ffn", "T": 4096, "d": 7168, "F": 6144, "act": "situ", "save": True},
        # training backward: all four gradients
        {"name": "ffn bwd t4096 d7168 f6144", "op": "ffn_bwd", "T": 4096, "d": 7168, "F": 6144, "act": "situ"},
        # training backward of a mid-size layer on an odd number of tokens
        {"name": "ffn bwd t1003 d1152 f864", "op": "ffn_bwd", "T": 1003, "d": 1152, "F": 864, "act": "swiglu"},
        # serving in 8 bits: a small decode batch
        {"name": "ffn mx t16 d7168 f6144", "op": "ffn_mx", "T": 16, "d": 7168, "F": 6144, "act": "situ"},
        # serving in 8 bits: a prefill chunk
        {"name": "ffn mx t4096 d7168 f6144", "op": "ffn_mx", "T": 4096, "d": 7168, "F": 6144, "act": "situ"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    """Tokens 1..8192 (forward norm) or 1..4096, widths 256..7168 and 256..6144, every option."""
    op = rng.choice(["norm", "norm_bwd", "ffn", "ffn", "ffn_bwd", "ffn_mx"])
    act = rng.choice(["situ", "swiglu"])
    if op == "norm":
        return {"op": op, "T": _log_int(rng, 1, 8192), "d": _log_int(rng, 256, 7168, 32),
                "res": rng.choice(["none", "bf16", "fp32"]), "fmt": rng.choice(["bf16", "mxfp8"])}
    if op == "norm_bwd":
        return {"op": op, "T": _log_int(rng, 1, 4096), "d": _log_int(rng, 256, 7168, 8),
                "res": rng.choice(["bf16", "fp32"]), "dh": rng.random() < 0.5}
    if op == "ffn":
        return {"op": op, "T": _log_int(rng, 1, 4096), "d": _log_int(rng, 256, 7168, 8),
                "F": _log_int(rng, 256, 6144, 8), "act": act, "save": rng.random() < 0.5}
    if op == "ffn_bwd":
        return {"op": op, "T": _log_int(rng, 64, 4096), "d": _log_int(rng, 256, 7168, 8),
                "F": _log_int(rng, 256, 6144, 8), "act": act}
    return {"op": op, "T": _log_int(rng, 1, 4096), "d": _log_int(rng, 256, 7168, 32),
            "F": _log_int(rng, 256, 6144, 32), "act": act}


def work(case):
    T, d = case["T"], case["d"]
    if case["op"] == "norm":
        rb = {"none": 0, "bf16": 4, "fp32": 8}[case["res"]]            # residual read, sum written
        yb = 2 if case["fmt"] == "bf16" else 1 + 1 / 32
        return {"bytes": T * d * (2 + rb + yb) + 2 * d, "flops": 6 * T * d}
    if case["op"] == "norm_bwd":
        hb = 2 if case["res"] == "bf16" else 4
        return {"bytes": T * d * (2 + hb * (3 if case["dh"] else 2)) + 6 * d, "flops": 10 * T * d}
    F = case["F"]
    if case["op"] == "ffn":
        return {"bytes": 6 * d * F + 4 * T * d + (4 * T * F if case["save"] else 0), "flops": 6 * T * d * F}
    if case["op"] == "ffn_bwd":
        return {"bytes": 12 * d * F + 6 * T * d + 4 * T * F, "flops": 12 * T * d * F}
    return {"bytes": (3 * d * F + T * d) * 33 / 32 + 2 * T * d, "flops": 6 * T * d * F}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def _stream(g, T, d, dtype=torch.bfloat16):
    """Rows of a residual stream: their norms spread, a few channels far larger than the rest."""
    row = torch.exp(0.5 * torch.randn(T, 1, device="cuda", generator=g))
    ch = 1 + 15 * (torch.rand(1, d, device="cuda", generator=g) < 0.01)
    return (torch.randn(T, d, device="cuda", generator=g) * row * ch).to(dtype)


def _mx_encode(v):
    """MXFP8 of v (32 bits) along its last axis: E4M3 codes, and a power of two for each 32 values, the
    smallest that keeps them within 448."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    m, e = torch.frexp(b.abs().amax(-1))
    s = (e - 1 + 127 - 8 + (m > 0.875)).clamp(1, 253)
    q = (b * torch.exp2(127.0 - s)[..., None]).to(F8)
    return q.reshape(v.shape), s.to(torch.uint8)


def _mx_values(q, s):
    v = q.float().reshape(*q.shape[:-1], -1, 32) * torch.exp2(s.float() - 127)[..., None]
    return v.reshape(q.shape)


def _inputs(case, seed):
    g, T, d = _gen(seed), case["T"], case["d"]
    st = dict(case)
    if case["op"] == "norm":
        st["x"] = _stream(g, T, d)
        if case["res"] != "none":
            st["r"] = _stream(g, T, d, torch.bfloat16 if case["res"] == "bf16" else torch.float32)
        st["w"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16)
        return st
    if case["op"] == "norm_bwd":
        ht = torch.bfloat16 if case["res"] == "bf16" else torch.float32
        st["h"] = _stream(g, T, d, ht)
        st["dy"] = _normal(g, T, d, std=1e-3)
        st["dh"] = _normal(g, T, d, std=1e-3, dtype=ht) if case["dh"] else None
        st["w"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16)
        return st
    F = case["F"]
    x = _normal(g, T, d)
    if case["op"] == "ffn_mx":
        st["xq"], st["xs"] = _mx_encode(x.float())
        for n, o, i in (("gate", F, d), ("up", F, d), ("down", d, F)):
            st[n], st[n + "_s"] = _mx_encode(torch.randn(o, i, device="cuda", generator=g) * i ** -0.5)
        return st
    st["x"] = x
    st["gate"] = _normal(g, F, d, std=d ** -0.5)
    st["up"] = _normal(g, F, d, std=d ** -0.5)
    st["down"] = _normal(g, d, F, std=F ** -0.5)
    if case["op"] == "ffn_bwd":
        st["dy"] = _normal(g, T, d, std=1e-3)
        st["g"], st["u"] = x @ st["gate"].T, x @ st["up"].T          # saved by the forward pass, bf16
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own and "F" in case:
        from latent_mixture_experts_gb300 import GatedFFN
        names = ("gate", "up", "down", "gate_s", "up_s", "down_s")
        weights = {n: st[n].view(torch.uint8) if case["op"] == "ffn_mx" else st[n] for n in names if n in st}
        st["layer"] = GatedFFN(weights, max_tokens=case["T"], act=case["act"], situ_beta=B1, situ_linear_beta=B2,
                               training=case["op"] == "ffn_bwd")
        if case["op"] == "ffn_mx":
            st["xq"] = st["xq"].view(torch.uint8)
    return st


# --------------------------------------------------------------- operators
def _act(g, u, act):
    if act == "swiglu":
        return g * torch.sigmoid(g) * u
    return B1 * torch.tanh(g / B1) * torch.sigmoid(g) * (B2 * torch.tanh(u / B2))


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from latent_mixture_experts_gb300 import lmoe_add_rms_norm, lmoe_add_rms_norm_backward
    op = st["op"]
    if op == "norm":
        y, s, h = lmoe_add_rms_norm(st["x"], st["w"], EPS, residual=st.get("r"), out_format=st["fmt"])
        return [y, h] if s is None else [y.view(F8), s.view(E8), h]
    if op == "norm_bwd":
        return list(lmoe_add_rms_norm_backward(st["dy"], st["h"], st["w"], EPS, dh=st["dh"]))
    if op == "ffn":
        if st["save"]:
            return list(st["layer"].lmoe_ffn_forward(st["x"], save=True))
        return [st["layer"].lmoe_ffn_forward(st["x"])]
    if op == "ffn_bwd":
        return list(st["layer"].lmoe_ffn_backward(st["x"], st["g"], st["u"], st["dy"]))
    return [st["layer"].lmoe_ffn_forward_mx(st["xq"], st["xs"])]


def _run_plain(st):
    op, bf = st["op"], torch.bfloat16
    if op == "norm":
        x, r = st["x"], st.get("r")
        h = x if r is None else (x.float() + r.float()).to(r.dtype)
        hf = h.float()
        y = hf * torch.rsqrt((hf * hf).mean(-1, keepdim=True) + EPS) * st["w"].float()
        h = None if r is None else h
        if st["fmt"] == "bf16":
            return [y.to(bf), h]
        q, s = _mx_encode(y)
        return [q, s.view(E8), h]
    if op == "norm_bwd":
        dy, h, w = st["dy"].float(), st["h"].float(), st["w"].float()
        r1 = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        wdy = dy * w
        dx = r1 * (wdy - h * (r1 * r1 * (wdy * h).mean(-1, keepdim=True)))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return [dx.to(st["h"].dtype), (dy * h * r1).sum(0)]
    if op == "ffn_mx":
        x = _mx_values(st["xq"].view(F8), st["xs"])
        wg, wu, wd = (_mx_values(st[n].view(F8), st[n + "_s"]) for n in ("gate", "up", "down"))
        hid = _mx_values(*_mx_encode(_act(x @ wg.T, x @ wu.T, st["act"])))
        return [(hid @ wd.T).to(bf)]
    x, wg, wu, wd = (st[n].float() for n in ("x", "gate", "up", "down"))
    if op == "ffn":
        g, u = x @ wg.T, x @ wu.T
        y = (_act(g, u, st["act"]) @ wd.T).to(bf)
        return [y, g.to(bf), u.to(bf)] if st["save"] else [y]
    g, u, dy = st["g"].float(), st["u"].float(), st["dy"].float()
    dhid = dy @ wd
    sg = torch.sigmoid(g)
    if st["act"] == "swiglu":
        a, da, ub, dub = g * sg, sg * (1 + g * (1 - sg)), u, 1.0
    else:
        tg, tu = torch.tanh(g / B1), torch.tanh(u / B2)
        a, da = B1 * tg * sg, (1 - tg * tg) * sg + B1 * tg * sg * (1 - sg)
        ub, dub = B2 * tu, 1 - tu * tu
    dg, du = dhid * ub * da, dhid * a * dub
    return [t.to(bf) for t in (dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ (a * ub))]


# ------------------------------------------------------------------- exact
def _e4m3_64(v):
    """v rounded to the nearest E4M3 value, ties to even, in 64 bits."""
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _mx_64(v):
    """(codes, scales) of MXFP8, as the 64-bit values that they stand for."""
    b = v.reshape(v.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(-1) / 448)
    s = torch.exp2((e - (m == 0.5).int()).clamp(-126, 126).double())
    return _e4m3_64(b / s[..., None]).reshape(v.shape), s


def _spread_64(q, s):
    return q.double() * s.repeat_interleave(32, -1)


def exact(case, seed):
    if 12 * case["T"] * case["d"] * case.get("F", 1) > 4.5e12:      # 64-bit products of over some seconds
        return None
    st = _inputs(case, seed)
    D = torch.float64
    if case["op"] == "norm":
        x, r, w = st["x"].to(D), st.get("r"), st["w"].to(D)
        h = x if r is None else x + r.to(D)
        # the sum is stored in the stream's type and normalised as stored (a 64-bit sum of two bf16 values is exact)
        h = h if r is None else h.to(r.dtype)
        hd = h.to(D)
        y = w * hd / torch.sqrt((hd ** 2).sum(-1, keepdim=True) / case["d"] + EPS)
        h = None if r is None else hd
        if case["fmt"] == "bf16":
            return [y, h]
        q, s = _mx_64(y)
        return [q, s, h]
    if case["op"] == "norm_bwd":
        dy, h, w = st["dy"].to(D), st["h"].to(D), st["w"].to(D)
        n = torch.sqrt((h ** 2).sum(-1, keepdim=True) / case["d"] + EPS)
        dx = dy * w / n - h * (dy * w * h).sum(-1, keepdim=True) / (case["d"] * n ** 3)
        if st["dh"] is not None:
            dx = dx + st["dh"].to(D)
        return [dx, (dy * h / n).sum(0)]

    def glu(g, u):
        if case["act"] == "swiglu":
            return g / (1 + torch.exp(-g)) * u
        return B1 * torch.tanh(g / B1) / (1 + torch.exp(-g)) * B2 * torch.tanh(u / B2)

    if case["op"] == "ffn_mx":
        x, wg, wu, wd = (_spread_64(st[q].view(F8), torch.exp2(st[s].to(D) - 127)) for q, s in
                         (("xq", "xs"), ("gate", "gate_s"), ("up", "up_s"), ("down", "down_s")))
        hid = _spread_64(*_mx_64(glu(x @ wg.T, x @ wu.T)))
        return [hid @ wd.T]
    x, wg, wu, wd = (st[n].to(D) for n in ("x", "gate", "up", "down"))
    if case["op"] == "ffn":
        g, u = x @ wg.T, x @ wu.T
        y = glu(g, u) @ wd.T
        return [y, g, u] if case["save"] else [y]
    g, u, dy = (st[n].to(D) for n in ("g", "u", "dy"))
    sg, dhid = 1 / (1 + torch.exp(-g)), dy @ wd
    if case["act"] == "swiglu":
        dg, du = dhid * u * (sg + g * sg * (1 - sg)), dhid * g * sg
    else:
        lin = B1 * torch.tanh(g / B1)
        dg = dhid * B2 * torch.tanh(u / B2) * sg * (1 / torch.cosh(g / B1) ** 2 + lin * (1 - sg))
        du = dhid * lin * sg / torch.cosh(u / B2) ** 2
    return [dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ glu(g, u)]
