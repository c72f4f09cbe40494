"""The feed-forward block on MXFP8 operands against the 64-bit form.

Elementwise: the hidden activation is off by its fp32 error and at most half
an E4M3 step (2^-4 relative, 2^-10 of the block's scale; the scale itself may
be the next one where the block's maximum is at the border), then fp32 and one
bf16 rounding.  Relative L2 against the reference that encodes the hidden
activation itself: an fp32 error of 2^-15 moves about 2^-11 of the values to
the neighbouring code, 2^-3.5 off, 2^-9 in all; with the output's rounding,
2^-8 / sqrt(3), below 2^-8."""
import pytest
import torch

from tests import _ffn_reference as R
from tests._harness import built_library

pytestmark = pytest.mark.gpu
REL = 2.0 ** -8


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    return P


def _make(T, d, F, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = {}
    for n, o, i in (("gate", F, d), ("up", F, d), ("down", d, F)):
        W[n], W[n + "_s"] = R.mx_random((o, i), i ** -0.5, g, "cuda")
    # scales that differ from row to row and block to block
    row = torch.exp(torch.randn(T, 1, device="cuda", generator=g, dtype=R.D))
    x, s = R.mx_encode(torch.randn(T, d, device="cuda", generator=g, dtype=R.D) * row)
    f = torch.exp2(s.to(R.D) - 127).repeat_interleave(32, -1)
    return (x / f).float().to(torch.float8_e4m3fn).view(torch.uint8), s.to(torch.uint8), W


def _check(y, q, s, W, act, b1=4.0, b2=25.0):
    x = R.mx_decode(q, s)
    wg, wu, wd = (R.mx_decode(W[n], W[n + "_s"]) for n in ("gate", "up", "down"))
    g, u = x @ wg.T, x @ wu.T
    a, v, da, dv = R.act_parts(g, u, act, b1, b2)
    h = a * v
    hq, hs = R.mx_encode(h)
    ref = hq @ wd.T
    dg, du = R.ACC * (x.abs() @ wg.abs().T), R.ACC * (x.abs() @ wu.abs().T)
    eh = v.abs() * (da.abs() * dg + dg * dg) + a.abs() * (dv.abs() * du + du * du) + 2 * dg * du + R.FAST * h.abs()
    f = torch.exp2(hs.to(R.D) - 127).repeat_interleave(32, -1)
    # from the exact h to the stored one: half a step of the GPU's own encoding (a scale one up doubles the least)
    eq = eh + torch.maximum(2.0 ** -4 * (h.abs() + eh), 2.0 ** -9 * f)
    bound = eq @ wd.abs().T + R.ACC * ((h.abs() + eq) @ wd.abs().T)
    exact = h @ wd.T
    err = (y.to(R.D) - exact).abs()
    assert bool((err <= bound + R.HALF[torch.bfloat16] * (exact.abs() + bound) + 1e-30).all())
    if ref.numel() >= 2048:
        assert R.rel_l2(y, ref) <= REL, R.rel_l2(y, ref)


SHAPES = [(1, 32, 32), (1, 128, 256), (3, 64, 96), (8, 160, 224), (16, 1152, 864), (17, 256, 192), (33, 640, 512),
          (64, 704, 608), (100, 1024, 992), (127, 512, 256), (128, 320, 384), (129, 320, 288), (200, 256, 1056),
          (256, 256, 256), (257, 448, 160), (513, 1152, 608), (1000, 544, 1024), (700, 960, 960)]


@pytest.mark.parametrize("act", ["situ", "swiglu"])
@pytest.mark.parametrize("T,d,F", SHAPES)
def test_forward(ops, T, d, F, act):
    q, s, W = _make(T, d, F, T + d + F)
    layer = ops.GatedFFN(W, max_tokens=T, act=act)
    y = layer.lmoe_ffn_forward_mx(q, s)
    _check(y, q, s, W, act)
    assert torch.equal(layer.lmoe_ffn_forward_mx(q, s), y)
    layer.lmoe_ffn_sync_status()
    layer.close()


@pytest.mark.parametrize("T,d,F", [(1, 7168, 2048), (16, 7168, 6144), (300, 2048, 6144), (2100, 1152, 864)])
def test_model_widths(ops, T, d, F):
    q, s, W = _make(T, d, F, 3)
    layer = ops.GatedFFN(W, max_tokens=T)
    _check(layer.lmoe_ffn_forward_mx(q, s), q, s, W, "situ")
    layer.lmoe_ffn_sync_status()


def test_every_scale_is_its_own(ops):
    """One nonzero value per row and block in turn, with a scale that no other block has: a scale read from another
    row, block or tile shows as a power of two."""
    T, d, F = 140, 256, 224
    q, s, W = _make(T, d, F, 9)
    s = (torch.arange(T * (d // 32), device="cuda") % 11 + 117).view(T, d // 32).to(torch.uint8)
    for n in ("gate_s", "up_s", "down_s"):
        t = W[n]
        W[n] = (t.to(torch.int64) + (torch.arange(t.numel(), device="cuda").view(t.shape) * 7) % 3).to(torch.uint8)
    layer = ops.GatedFFN(W, max_tokens=T, act="swiglu")
    _check(layer.lmoe_ffn_forward_mx(q, s), q, s, W, "swiglu")


@pytest.mark.parametrize("T", [5, 300])
def test_nan_blocks_stay_in_their_rows(ops, T):
    q, s, W = _make(T, 192, 160, 51)
    layer = ops.GatedFFN(W, max_tokens=T)
    want = layer.lmoe_ffn_forward_mx(q, s)
    s[1, 2] = 255                   # a NaN block
    q[3, 7] = 0x7F                  # a NaN code
    y = layer.lmoe_ffn_forward_mx(q, s)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[1, 3]] = False
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[3]).all()) and torch.equal(y[keep], want[keep])


def test_zero_rows_and_reuse(ops):
    q, s, W = _make(300, 256, 320, 61)
    layer = ops.GatedFFN(W, max_tokens=300)
    layer.lmoe_ffn_forward_mx(q, s)
    q[2] = 0
    for T in (7, 150, 300):         # after a larger batch
        y = layer.lmoe_ffn_forward_mx(q[:T], s[:T])
        assert bool((y[2] == 0).all())
        _check(y, q[:T], s[:T], W, "situ")
    assert layer.lmoe_ffn_forward_mx(q[:0], s[:0]).shape == (0, 256)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_after_the_norm_and_in_a_graph(ops, T):
    """The norm's MXFP8 output feeds the block; on a side stream and replayed from a graph."""
    d, F = 512, 384
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    r = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    _, _, W = _make(1, d, F, 71)
    layer = ops.GatedFFN(W, max_tokens=T)
    q, s, h = ops.lmoe_add_rms_norm(x, w, 1e-6, residual=r, out_format="mxfp8")
    y = layer.lmoe_ffn_forward_mx(q, s)
    _check(y, q, s, W, "situ")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ys = layer.lmoe_ffn_forward_mx(q, s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ys)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qc, sc, _ = ops.lmoe_add_rms_norm(x, w, 1e-6, residual=r, out_format="mxfp8")
        yc = layer.lmoe_ffn_forward_mx(qc, sc)
    x.copy_(torch.randn(T, d, device="cuda", generator=g).bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    _check(yc, qc, sc, W, "situ")
    layer.lmoe_ffn_sync_status()


def test_refusals(ops):
    q, s, W = _make(8, 64, 64, 91)
    with pytest.raises(ops.LmoeError):
        ops.GatedFFN(W, max_tokens=8, training=True)
    with pytest.raises(ValueError):
        ops.GatedFFN({**W, "gate_s": W["gate_s"][:, :1]}, max_tokens=8)
    layer = ops.GatedFFN(W, max_tokens=8)
    for f in (lambda: layer.lmoe_ffn_forward_mx(q, s[:, :1]), lambda: layer.lmoe_ffn_forward_mx(q.float(), s),
              lambda: layer.lmoe_ffn_forward_mx(q.cpu(), s.cpu())):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ops.LmoeError):
        layer.lmoe_ffn_forward(torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ops.LmoeError):
        layer.lmoe_ffn_forward_mx(torch.cat([q, q]), torch.cat([s, s]))
