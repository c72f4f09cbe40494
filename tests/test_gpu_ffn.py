"""The dense gated feed-forward block (bf16) against the 64-bit forms: every
element within the bound that counts the path's roundings, and the relative
L2 error below 2^-8 - two roundings in a row are off by at most 2^-8 / sqrt(3)
each in the root mean square, 0.82 * 2^-8 together."""
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


def _make(T, d, F, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).bfloat16()
    W = {"gate": rnd(F, d, std=scale * d ** -0.5), "up": rnd(F, d, std=scale * d ** -0.5),
         "down": rnd(d, F, std=F ** -0.5)}
    return rnd(T, d), W, rnd(T, d, std=1e-2)


def _check_forward(y, x, W, act):
    ref, g, u = R.forward(x, W["gate"], W["up"], W["down"], act)
    err = (y.to(R.D) - ref).abs()
    bound = R.forward_bound(x, W["gate"], W["up"], W["down"], act)
    assert bool((err <= bound).all()), float((err / bound).max())
    if ref.numel() >= 256:
        assert R.rel_l2(y, ref) <= REL, R.rel_l2(y, ref)
    return g, u


def _check_pre(got, ref, x, w):
    tol = R.HALF[torch.bfloat16] * ref.abs() + 2 * R.ACC * (x.to(R.D).abs() @ w.to(R.D).abs().T)
    assert bool(((got.to(R.D) - ref).abs() <= tol).all())


def _check_backward(grads, x, g, u, dy, W, act):
    ref = R.backward(x, g, u, dy, W["gate"], W["up"], W["down"], act)
    bound = R.backward_bound(x, g, u, dy, W["gate"], W["up"], W["down"], act)
    for name, got, r, b in zip(("dx", "dw_gate", "dw_up", "dw_down"), grads, ref, bound):
        assert got.shape == r.shape and got.dtype == torch.bfloat16
        err = (got.to(R.D) - r).abs()
        assert bool((err <= b).all()), (name, float((err / b).max()))
        if r.numel() >= 256:
            assert R.rel_l2(got, r) <= REL, (name, R.rel_l2(got, r))


# tokens on both sides of every tile edge; widths that end inside a 64-wide K block, a 128-feature and a 256-column tile
SHAPES = [(1, 8, 8), (1, 64, 128), (2, 72, 136), (7, 256, 40), (16, 1152, 864), (17, 264, 520), (33, 640, 512),
          (64, 704, 608), (100, 1024, 1000), (127, 512, 256), (128, 320, 384), (129, 320, 264), (200, 256, 1096),
          (255, 768, 128), (256, 256, 256), (257, 448, 136), (513, 1152, 608), (1000, 520, 1032)]


@pytest.mark.parametrize("act", ["situ", "swiglu"])
@pytest.mark.parametrize("T,d,F", SHAPES)
def test_forward_and_backward(ops, T, d, F, act):
    x, W, dy = _make(T, d, F, T + d + F)
    layer = ops.GatedFFN(W, max_tokens=T, act=act, training=True)
    y = layer.lmoe_ffn_forward(x)
    y2, g, u = layer.lmoe_ffn_forward(x, save=True)
    assert torch.equal(y, y2)
    gref, uref = _check_forward(y, x, W, act)
    _check_pre(g, gref, x, W["gate"])
    _check_pre(u, uref, x, W["up"])
    grads = layer.lmoe_ffn_backward(x, g, u, dy)
    _check_backward(grads, x, g, u, dy, W, act)
    again = layer.lmoe_ffn_backward(x, g, u, dy)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    layer.lmoe_ffn_sync_status()
    layer.close()


# the last: more 256-column tiles than the GPU has CTA pairs, with a few left over in every product
@pytest.mark.parametrize("T,d,F", [(1, 7168, 2048), (64, 7168, 2048), (96, 2048, 1040), (97, 2048, 1040),
                                   (300, 2048, 6144), (2100, 1152, 864), (2600, 1752, 2000)])
def test_model_widths(ops, T, d, F):
    x, W, dy = _make(T, d, F, 3)
    layer = ops.GatedFFN(W, max_tokens=T, training=True)
    y, g, u = layer.lmoe_ffn_forward(x, save=True)
    _check_forward(y, x, W, "situ")
    _check_backward(layer.lmoe_ffn_backward(x, g, u, dy), x, g, u, dy, W, "situ")
    layer.lmoe_ffn_sync_status()


# K split over two or four pairs of CTAs: every tail of tokens, K blocks, features and columns, one tile and many
@pytest.mark.parametrize("act", ["situ", "swiglu"])
@pytest.mark.parametrize("T,d,F", [(73, 256, 256), (128, 264, 520), (130, 1000, 712), (256, 2048, 2048),
                                   (257, 512, 1288), (300, 768, 768), (500, 4104, 1032), (513, 520, 8),
                                   (700, 72, 3080), (1003, 1152, 864), (256, 7168, 512)])
def test_split_products(ops, T, d, F, act):
    test_forward_and_backward(ops, T, d, F, act)


@pytest.mark.parametrize("T,d,F", [(100, 1024, 512), (200, 768, 768), (300, 2048, 2048), (1003, 1152, 864)])
def test_split_products_back_to_back(ops, T, d, F):
    """The workspace and the products that run beside one another: calls that follow at once, each form of the
    backward pass among them, give the bits of calls alone."""
    x, W, dy = _make(T, d, F, 31)
    x2, _, dy2 = _make(T, d, F, 32)
    layer = ops.GatedFFN(W, max_tokens=T, training=True)
    calls = []
    for a, b in ((x, dy), (x2, dy2)):
        _, g, u = layer.lmoe_ffn_forward(a, save=True)
        calls += [lambda a=a, g=g, u=u, b=b, kw=kw: layer.lmoe_ffn_backward(a, g, u, b, **kw)
                  for kw in ({}, {"need_dw": False}, {"need_dx": False})]
        calls.append(lambda a=a: (layer.lmoe_ffn_forward(a),))
    alone = []
    for call in calls:
        torch.cuda.synchronize()
        alone.append(call())
    torch.cuda.synchronize()
    got = [(call(), want) for _ in range(8) for call, want in zip(calls, alone)]
    layer.lmoe_ffn_sync_status()
    for have, want in got:
        for p, q in zip(have, want):
            assert (p is None) == (q is None) and (p is None or torch.equal(p, q))


def test_large_preactivations(ops):
    """Saturated gates: tanh and sigmoid at their ends, caps other than the default."""
    x, W, dy = _make(40, 256, 192, 21, scale=30.0)
    for act, b1, b2 in (("situ", 4.0, 25.0), ("situ", 0.5, 2.0), ("swiglu", 4.0, 25.0)):
        layer = ops.GatedFFN(W, max_tokens=64, act=act, situ_beta=b1, situ_linear_beta=b2, training=True)
        y, g, u = layer.lmoe_ffn_forward(x, save=True)
        ref = R.forward(x, W["gate"], W["up"], W["down"], act, b1, b2)[0]
        assert R.rel_l2(y, ref) <= REL
        grads = layer.lmoe_ffn_backward(x, g, u, dy)
        want = R.backward(x, g, u, dy, W["gate"], W["up"], W["down"], act, b1, b2)
        bound = R.backward_bound(x, g, u, dy, W["gate"], W["up"], W["down"], act, b1, b2)
        for a, r, b in zip(grads, want, bound):
            assert bool(((a.to(R.D) - r).abs() <= b).all())


def test_gradient_against_differences(ops):
    """The GPU's gradients as the slope of the exact forward along random directions; the saved g and u are rounded to
    bf16 (2^-8 relative) and so are the gradients, so the slope is compared to 2^-6 of the gradient's length."""
    T, d, F = 24, 128, 96
    x, W, dy = _make(T, d, F, 31)
    layer = ops.GatedFFN(W, max_tokens=T, training=True)
    _, g, u = layer.lmoe_ffn_forward(x, save=True)
    grads = dict(zip(("x", "gate", "up", "down"), layer.lmoe_ffn_backward(x, g, u, dy)))
    gen = torch.Generator(device="cuda").manual_seed(5)
    base = {"x": x, **W}
    for n in base:
        v = grads[n].to(R.D) + grads[n].to(R.D).norm() * torch.randn(base[n].shape, device="cuda", generator=gen,
                                                                     dtype=R.D) / base[n].numel() ** 0.5
        v /= v.norm()
        f = []
        for s in (1e-5, -1e-5):
            P = {k: t.to(R.D) for k, t in base.items()}
            P[n] = P[n] + s * v
            f.append(float((R.forward(P["x"], P["gate"], P["up"], P["down"], "situ")[0] * dy.to(R.D)).sum()))
        slope = (f[0] - f[1]) / 2e-5
        got = float((grads[n].to(R.D) * v).sum())
        assert abs(slope - got) <= 2.0 ** -6 * float(grads[n].to(R.D).norm()), (n, slope, got)


def test_strided_rows(ops):
    T, d, F = 70, 256, 320
    x, W, dy = _make(T, d, F, 41)
    wide = torch.full((T, 2 * d), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[:, 64:64 + d] = x
    xs = wide[:, 64:64 + d]
    wdy = torch.full((T, d + 8), float("nan"), device="cuda", dtype=torch.bfloat16)
    wdy[:, :d] = dy
    layer = ops.GatedFFN(W, max_tokens=128, training=True)
    y, g, u = layer.lmoe_ffn_forward(x, save=True)
    ys, gs, us = layer.lmoe_ffn_forward(xs, save=True)
    assert torch.equal(y, ys) and torch.equal(g, gs) and torch.equal(u, us)
    for a, b in zip(layer.lmoe_ffn_backward(x, g, u, dy), layer.lmoe_ffn_backward(xs, g, u, wdy[:, :d])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [3, 300])
def test_nan_rows_stay_in_their_rows(ops, T):
    x, W, dy = _make(T, 192, 136, 51)
    layer = ops.GatedFFN(W, max_tokens=T)
    want = layer.lmoe_ffn_forward(x)
    x[1, 7] = float("nan")
    x[2, 100] = float("inf")
    y = layer.lmoe_ffn_forward(x)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    assert bool(torch.isnan(y[1]).all()) and torch.equal(y[keep], want[keep])


def test_partial_gradients_and_empty(ops):
    x, W, dy = _make(50, 128, 72, 61)
    layer = ops.GatedFFN(W, max_tokens=64, training=True)
    _, g, u = layer.lmoe_ffn_forward(x, save=True)
    full = layer.lmoe_ffn_backward(x, g, u, dy)
    only_dx = layer.lmoe_ffn_backward(x, g, u, dy, need_dw=False)
    only_dw = layer.lmoe_ffn_backward(x, g, u, dy, need_dx=False)
    assert torch.equal(only_dx[0], full[0]) and only_dx[1:] == (None, None, None)
    assert only_dw[0] is None and all(torch.equal(a, b) for a, b in zip(only_dw[1:], full[1:]))
    y = layer.lmoe_ffn_forward(x[:0])
    assert y.shape == (0, 128)
    e = layer.lmoe_ffn_backward(x[:0], g[:0], u[:0], dy[:0])
    assert e[0].shape == (0, 128) and all(bool((t == 0).all()) for t in e[1:])
    # a block that is reused for fewer tokens after more
    y5 = layer.lmoe_ffn_forward(x[:5])
    _check_forward(y5, x[:5], W, "situ")


def test_weight_updates_are_seen(ops):
    x, W, _ = _make(20, 128, 128, 71)
    layer = ops.GatedFFN(W, max_tokens=32)
    layer.lmoe_ffn_forward(x)
    W["down"].mul_(-0.5)
    W["gate"].mul_(2.0)
    _check_forward(layer.lmoe_ffn_forward(x), x, W, "situ")


@pytest.mark.parametrize("T", [1, 40, 300])
def test_streams_and_graph(ops, T):
    x, W, dy = _make(T, 256, 384, 81)
    layer = ops.GatedFFN(W, max_tokens=T, training=True)
    y, g, u = layer.lmoe_ffn_forward(x, save=True)
    grads = layer.lmoe_ffn_backward(x, g, u, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ys = layer.lmoe_ffn_forward(x, stream=side)
    gs = layer.lmoe_ffn_backward(x, g, u, dy, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ys) and all(torch.equal(a, b) for a, b in zip(grads, gs))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yc, gc, uc = layer.lmoe_ffn_forward(x, save=True)
        out = layer.lmoe_ffn_backward(x, gc, uc, dy)
    x2, _, dy2 = _make(T, 256, 384, 82)
    x.copy_(x2)
    dy.copy_(dy2)
    graph.replay()
    torch.cuda.synchronize()
    _check_forward(yc, x, W, "situ")
    _check_backward(out, x, gc, uc, dy, W, "situ")
    layer.lmoe_ffn_sync_status()


def test_workspace_that_does_not_fit(ops):
    """An allocation that fails is refused, and leaves no error behind for the caller's next launch."""
    x, W, _ = _make(8, 64, 512, 90)
    with pytest.raises(ops.LmoeError) as e:
        ops.GatedFFN(W, max_tokens=2 ** 31 - 1, training=True)      # 6.6 TB
    assert e.value.status == ops.LMOE_ERR_OOM
    assert bool((x + 0 == x).all())
    layer = ops.GatedFFN(W, max_tokens=8)
    _check_forward(layer.lmoe_ffn_forward(x), x, W, "situ")


def test_binding_refusals(ops):
    x, W, dy = _make(8, 64, 64, 91)
    with pytest.raises(ValueError):
        ops.GatedFFN({**W, "up": W["up"].float()}, max_tokens=8)
    with pytest.raises(ValueError):
        ops.GatedFFN({**W, "down": W["down"].t()[:32]}, max_tokens=8)
    with pytest.raises(ValueError):
        ops.GatedFFN(W, max_tokens=8, act="relu")
    with pytest.raises(ops.LmoeError):
        ops.GatedFFN(W, max_tokens=0)
    layer = ops.GatedFFN(W, max_tokens=8)
    _, g, u = layer.lmoe_ffn_forward(x, save=True)
    with pytest.raises(ops.LmoeError):
        layer.lmoe_ffn_backward(x, g, u, dy)            # not created for training
    for f in (lambda: layer.lmoe_ffn_forward(x.float()), lambda: layer.lmoe_ffn_forward(x[:, :32]),
              lambda: layer.lmoe_ffn_forward(x.cpu()), lambda: layer.lmoe_ffn_backward(x, g[:4], u, dy),
              lambda: layer.lmoe_ffn_forward(x, out=torch.empty(8, 64, device="cuda"))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ops.LmoeError):
        layer.lmoe_ffn_forward(torch.cat([x, x]))       # more than max_tokens
    with pytest.raises(ops.LmoeError):
        layer.lmoe_ffn_forward_mx(torch.zeros(8, 64, device="cuda", dtype=torch.uint8),
                                  torch.zeros(8, 2, device="cuda", dtype=torch.uint8))
