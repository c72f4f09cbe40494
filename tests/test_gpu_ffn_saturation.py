"""The activation gradient from one end of the gates to the other, element by
element.

With x (its first T rows) and down the identity, dw_gate is dg^T and dw_up is du^T: a
bf16 value times one, added to zeros.  What is off is one rounding to bf16, and the
fp32 arithmetic relative to the sizes of the terms of each derivative: FAST for
the functions and products, and for each exponential the roundings of its
argument, at most four of 2^-24 of |2 x| (tanh) or |g| (sigmoid)."""
import pytest
import torch

from tests import _ffn_reference as R
from tests._harness import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    return P


# b1 and b2 as in the framework's layers, small ones (the sigmoid's tail decides a'), large ones
@pytest.mark.parametrize("act,b1,b2", [("situ", 4.0, 25.0), ("situ", 0.5, 2.0), ("situ", 30.0, 100.0),
                                       ("swiglu", 4.0, 25.0)])
@pytest.mark.parametrize("T,N", [(64, 256), (256, 256), (2048, 2048)])
def test_gradient_over_the_gates_range(ops, act, b1, b2, T, N):
    gen = torch.Generator(device="cuda").manual_seed(11)
    # |x| of tanh up to 20, |g| up to 80: a' and v' stay normal numbers of fp32
    top_g, top_u = min(20 * b1, 80.0), 20 * b2
    g = ((2 * torch.rand(T, N, device="cuda", generator=gen) - 1) * top_g).bfloat16()
    u = ((2 * torch.rand(T, N, device="cuda", generator=gen) - 1) * top_u).bfloat16()
    g[:, ::3] = (g[:, ::3].float() / 16).bfloat16()
    u[:, 1::3] = (u[:, 1::3].float() / 16).bfloat16()
    dy = torch.randn(T, N, device="cuda", generator=gen).bfloat16()
    eye = torch.eye(N, device="cuda", dtype=torch.bfloat16)
    layer = ops.GatedFFN({"gate": eye, "up": eye.clone(), "down": eye.clone()}, max_tokens=N, act=act, situ_beta=b1,
                         situ_linear_beta=b2, training=True)
    _, dwg, dwu, _ = layer.lmoe_ffn_backward(eye[:T], g, u, dy)
    layer.lmoe_ffn_sync_status()
    G, U, dh = g.to(R.D), u.to(R.D), dy.to(R.D)
    s, rest = torch.sigmoid(G), torch.sigmoid(-G)
    half, arg = R.HALF[torch.bfloat16], 4 * 2.0 ** -24
    eg = arg * G.abs()
    if act == "swiglu":
        v, a, dv, terms, da = U, G * s, torch.ones_like(U), s + (G * s * rest).abs(), s + G * s * rest
        ea = eg
        ev = torch.zeros_like(eg)
    else:
        sech_g, sech_u = 1 / torch.cosh(G / b1) ** 2, 1 / torch.cosh(U / b2) ** 2
        v, a, dv = b2 * torch.tanh(U / b2), b1 * torch.tanh(G / b1) * s, sech_u
        da, terms = sech_g * s + a * rest, sech_g * s + (a * rest).abs()
        ea, ev = eg + arg * (2 * G / b1).abs(), arg * (2 * U / b2).abs()
    for got, ref, tol in ((dwg, dh * v * da, (R.FAST + ea + ev) * (dh * v).abs() * terms),
                          (dwu, dh * a * dv, (R.FAST + ea + ev) * (dh * a * dv).abs())):
        err = (got[:, :T].T.to(R.D) - ref).abs()
        bound = half * ref.abs() + (1 + half) * tol + 2.0 ** -126
        assert bool((err <= bound).all()), float((err / bound).max())
