"""Where the weights lie and how wide they are: gate and up as slices of one
buffer in either order, one tensor as both, hidden layers far wider than the
model, and MXFP8 batches of more tile rows than one raster group."""
import pytest
import torch

from tests import _ffn_reference as R
from tests import test_gpu_ffn as bf16
from tests import test_gpu_ffn_mx as mx
from tests._harness import built_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    return P


def _lay_out(W, order):
    """W with gate and up in one buffer, rows apart; or one tensor as both."""
    if order == "same":
        return {**W, "up": W["gate"]}
    F, d = W["gate"].shape
    buf = torch.empty(2 * F + 3, d, device="cuda", dtype=W["gate"].dtype)
    gate, up = (buf[:F], buf[F + 3:]) if order == "gate first" else (buf[F + 3:], buf[:F])
    gate.copy_(W["gate"])
    up.copy_(W["up"])
    return {**W, "gate": gate, "up": up}


# up to 72 tokens stream gate and up through one map where they lie in one address range; K a multiple of 64 and not
@pytest.mark.parametrize("order", ["gate first", "up first", "same"])
@pytest.mark.parametrize("T,d,F", [(1, 512, 256), (3, 264, 136), (16, 1024, 40), (40, 1096, 520), (72, 256, 256),
                                   (200, 264, 136), (600, 512, 1288)])
def test_order_of_gate_and_up(ops, T, d, F, order):
    x, W, dy = bf16._make(T, d, F, T + d + F)
    W = _lay_out(W, order)
    layer = ops.GatedFFN(W, max_tokens=T, training=True)
    y, g, u = layer.lmoe_ffn_forward(x, save=True)
    gref, uref = bf16._check_forward(y, x, W, "situ")
    bf16._check_pre(g, gref, x, W["gate"])
    bf16._check_pre(u, uref, x, W["up"])
    bf16._check_backward(layer.lmoe_ffn_backward(x, g, u, dy), x, g, u, dy, W, "situ")
    assert torch.equal(layer.lmoe_ffn_forward(x), y)
    layer.lmoe_ffn_sync_status()


@pytest.mark.parametrize("order", ["gate first", "up first", "same"])
@pytest.mark.parametrize("T", [5, 300])
def test_order_of_gate_and_up_mxfp8(ops, T, order):
    q, s, W = mx._make(T, 288, 160, 7)
    V = _lay_out(W, order)
    if order == "same":
        V["up_s"] = V["gate_s"]
    layer = ops.GatedFFN(V, max_tokens=T)
    mx._check(layer.lmoe_ffn_forward_mx(q, s), q, s, V, "situ")
    layer.lmoe_ffn_sync_status()


@pytest.mark.parametrize("act", ["situ", "swiglu"])
@pytest.mark.parametrize("T,d,F", [(1, 512, 18432), (3, 264, 16392), (64, 256, 18432), (72, 16384, 256),
                                   (300, 256, 18432), (700, 264, 12296)])
def test_wide_hidden_layers(ops, T, d, F, act):
    x, W, dy = bf16._make(T, d, F, 17)
    layer = ops.GatedFFN(W, max_tokens=T, act=act, training=True)
    y, g, u = layer.lmoe_ffn_forward(x, save=True)
    bf16._check_forward(y, x, W, act)
    bf16._check_backward(layer.lmoe_ffn_backward(x, g, u, dy), x, g, u, dy, W, act)
    layer.lmoe_ffn_sync_status()


@pytest.mark.parametrize("act", ["situ", "swiglu"])
@pytest.mark.parametrize("T,d,F", [(1, 512, 18432), (5, 288, 16416), (48, 256, 18432), (48, 16384, 256),
                                   (300, 256, 18432), (700, 288, 12320), (4400, 256, 320), (8200, 416, 224)])
def test_wide_hidden_layers_and_many_tokens_mxfp8(ops, T, d, F, act):
    q, s, W = mx._make(T, d, F, 19)
    layer = ops.GatedFFN(W, max_tokens=T, act=act)
    y = layer.lmoe_ffn_forward_mx(q, s)
    mx._check(y, q, s, W, act)
    assert torch.equal(layer.lmoe_ffn_forward_mx(q, s), y)
    layer.lmoe_ffn_sync_status()


@pytest.mark.parametrize("T", [4400, 9000])
def test_many_tokens(ops, T):
    """More tile rows than a raster group of the bf16 pair tiles, several times over."""
    x, W, dy = bf16._make(T, 264, 520, 23)
    layer = ops.GatedFFN(W, max_tokens=T, training=True)
    y, g, u = layer.lmoe_ffn_forward(x, save=True)
    bf16._check_forward(y, x, W, "situ")
    bf16._check_backward(layer.lmoe_ffn_backward(x, g, u, dy), x, g, u, dy, W, "situ")
    assert R.rel_l2(y, R.forward(x, W["gate"], W["up"], W["down"], "situ")[0]) <= bf16.REL
    layer.lmoe_ffn_sync_status()


@pytest.mark.parametrize("T,d,F", [(3, 8, 128), (8, 8, 128), (1, 24, 304), (40, 64, 16), (72, 264, 136)])
def test_matrices_gigabytes_apart(ops, T, d, F):
    """Small weights with other allocations between them, as layers loaded one after the other leave them."""
    x, W, dy = bf16._make(T, d, F, T + d)
    far, between = {}, []
    for n in ("gate", "up", "down"):
        far[n] = W[n].clone()
        between.append(torch.empty(1 << 31, device="cuda", dtype=torch.uint8))
        # the caching allocator's small blocks come 2 MB at a time: the next matrix lies in another such block
        between += [torch.empty(1 << 20, device="cuda", dtype=torch.uint8) for _ in range(4)]
    layer = ops.GatedFFN(far, max_tokens=T, training=True)
    y, g, u = layer.lmoe_ffn_forward(x, save=True)
    gref, uref = bf16._check_forward(y, x, W, "situ")
    bf16._check_pre(g, gref, x, W["gate"])
    bf16._check_pre(u, uref, x, W["up"])
    bf16._check_backward(layer.lmoe_ffn_backward(x, g, u, dy), x, g, u, dy, W, "situ")
    layer.lmoe_ffn_sync_status()
