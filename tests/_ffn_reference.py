"""Plain 64-bit forms of the operators in include/lmoe_ffn.h (any device),
and the rounding counts that the tolerances are made of."""
import torch

D = torch.float64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # finfo.eps / 2: the most one rounding is off
# fp32 accumulation in the tensor cores: the sum of K products is taken to be
# off by at most 2^-16 of the sum of their magnitudes (K <= 16384 additions,
# each to 2^-24 or truncated to 2^-23, with room for alignment of partial sums).
ACC = 2.0 ** -16
FAST = 2.0 ** -18     # the epilogues' exp, tanh and division, relative


def act_parts(g, u, act, b1=4.0, b2=25.0):
    """a(g), v(u) and their derivatives."""
    s = torch.sigmoid(g)
    if act == "swiglu":
        return g * s, u, s * (1 + g * (1 - s)), torch.ones_like(u)
    tg, tu = torch.tanh(g / b1), torch.tanh(u / b2)
    return b1 * tg * s, b2 * tu, (1 - tg * tg) * s + b1 * tg * s * (1 - s), 1 - tu * tu


def forward(x, gate, up, down, act, b1=4.0, b2=25.0):
    x, gate, up, down = (t.to(D) for t in (x, gate, up, down))
    g, u = x @ gate.T, x @ up.T
    a, v, _, _ = act_parts(g, u, act, b1, b2)
    return (a * v) @ down.T, g, u


def forward_bound(x, gate, up, down, act, b1=4.0, b2=25.0):
    """Largest |y - exact| of the bf16 path: g and u to fp32 accumulation, hid
    rounded to bf16, fp32 accumulation, y rounded to bf16."""
    x, gate, up, down = (t.to(D) for t in (x, gate, up, down))
    g, u = x @ gate.T, x @ up.T
    dg, du = ACC * (x.abs() @ gate.abs().T), ACC * (x.abs() @ up.abs().T)
    a, v, da, dv = act_parts(g, u, act, b1, b2)
    hid = a * v
    # |a''|, |v''| stay below 1: second order in dg, du
    dh = (v.abs() * (da.abs() * dg + dg * dg) + a.abs() * (dv.abs() * du + du * du) + 2 * dg * du
          + (HALF[torch.bfloat16] + FAST) * hid.abs() + 1e-30)
    y = hid @ down.T
    e = dh @ down.abs().T + ACC * (hid.abs() @ down.abs().T)
    return e * (1 + HALF[torch.bfloat16]) + HALF[torch.bfloat16] * y.abs() + 1e-30


def backward(x, g, u, dy, gate, up, down, act, b1=4.0, b2=25.0):
    x, g, u, dy, gate, up, down = (t.to(D) for t in (x, g, u, dy, gate, up, down))
    a, v, da, dv = act_parts(g, u, act, b1, b2)
    dhid = dy @ down
    dg, du = dhid * v * da, dhid * a * dv
    return dg @ gate + du @ up, dg.T @ x, du.T @ x, dy.T @ (a * v)


def backward_bound(x, g, u, dy, gate, up, down, act, b1=4.0, b2=25.0):
    """Largest error of each gradient: dhid in fp32, dg, du and hid rounded to
    bf16, the products in fp32, the result rounded to bf16."""
    x, g, u, dy, gate, up, down = (t.to(D) for t in (x, g, u, dy, gate, up, down))
    h = HALF[torch.bfloat16]
    a, v, da, dv = act_parts(g, u, act, b1, b2)
    dhid, dacc = dy @ down, ACC * (dy.abs() @ down.abs())
    s = torch.sigmoid(g)
    # a' is a sum of two terms that may cancel: its fast functions are off relative to their sizes
    das = s + (a * (1 - s)).abs()
    dg, du, hid = dhid * v * da, dhid * a * dv, a * v
    edg = (dacc * (v * da).abs() + FAST * (dhid * v).abs() * das) * (1 + h) + h * dg.abs() + 1e-30
    edu = (dacc * (a * dv).abs() + FAST * (dhid * a).abs()) * (1 + h) + h * du.abs() + 1e-30
    eh = (h + FAST) * hid.abs() + 1e-30
    out = []
    for y, e, mag in (
            (dg @ gate + du @ up, edg @ gate.abs() + edu @ up.abs(), dg.abs() @ gate.abs() + du.abs() @ up.abs()),
            (dg.T @ x, edg.T @ x.abs(), dg.abs().T @ x.abs()),
            (du.T @ x, edu.T @ x.abs(), du.abs().T @ x.abs()),
            (dy.T @ hid, dy.abs().T @ eh, dy.abs().T @ hid.abs())):
        out.append((e + ACC * mag) * (1 + h) + h * y.abs() + 1e-30)
    return out


def norm(x, r, w, eps):
    """(y, h) with h stored in r's dtype."""
    h = x if r is None else (x.to(D) + r.to(D)).to(r.dtype)
    hd = h.to(D)
    return w.to(D) * hd / torch.sqrt((hd * hd).mean(-1, keepdim=True) + eps), h


def norm_backward(dy, h, w, eps, dh=None):
    dy, h, w = dy.to(D), h.to(D), w.to(D)
    rho = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    dx = rho * (w * dy - h * rho ** 2 * (w * dy * h).mean(-1, keepdim=True))
    return (dx if dh is None else dx + dh.to(D)), (dy * h * rho).sum(0)


def e4m3(v):
    """Nearest E4M3 value, ties to even."""
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp(min=-6).to(D) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def mx_scale(v):
    """E8M0 bytes of the 32-value blocks of v (64 bits)."""
    amax = v.reshape(*v.shape[:-1], -1, 32).abs().amax(-1)
    m, e = torch.frexp(amax / 448)
    s = (e - (m == 0.5).int() + 127).clamp(1, 253)
    return torch.where(amax > 0, s, torch.ones_like(s)).to(torch.int64)


def mx_encode(v):
    """The MXFP8 values nearest to v, and the scale bytes."""
    s = mx_scale(v)
    f = torch.exp2(s.to(D) - 127).repeat_interleave(32, -1)
    return e4m3(v / f) * f, s


def mx_decode(q, s):
    return q.view(torch.float8_e4m3fn).to(D) * torch.exp2(s.to(D) - 127).repeat_interleave(32, -1)


def mx_random(shape, std, gen, device):
    """Codes and scales of a random MXFP8 matrix."""
    v, s = mx_encode(torch.randn(*shape, generator=gen, device=device, dtype=D) * std)
    f = torch.exp2(s.to(D) - 127).repeat_interleave(32, -1)
    return (v / f).float().to(torch.float8_e4m3fn).view(torch.uint8), s.to(torch.uint8)


def rel_l2(a, b):
    return float((a.to(D) - b).norm() / b.norm())
