"""What the C calls promise beyond the binding: outputs in place of inputs, each
set of gradients, and rows of a few values."""
import itertools

import pytest
import torch

from tests import _ffn_reference as R
from tests import test_gpu_ffn as ffn
from tests import test_gpu_norm as norm
from tests._harness import built_library

pytestmark = pytest.mark.gpu
EPS = norm.EPS


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    return P


def _stream():
    return torch.cuda.current_stream().cuda_stream


# few rows, a ring of rows, wide ones
@pytest.mark.parametrize("T,d", [(5, 256), (700, 7168), (2000, 1152), (1023, 8200)])
def test_norm_in_place(ops, T, d):
    lib = ops.load_library()
    x, r, w = norm._make(T, d, 3, torch.bfloat16)
    want, _, hwant = ops.lmoe_add_rms_norm(x, w, EPS, residual=r)
    y, h = x.clone(), r.clone()
    assert lib.lmoe_add_rms_norm(y.data_ptr(), d, h.data_ptr(), d, 0, T, d, w.data_ptr(), EPS, h.data_ptr(),
                                 y.data_ptr(), 0, None, _stream()) == ops.LMOE_OK
    assert torch.equal(y, want) and torch.equal(h, hwant)


@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(5, 256), (700, 7168), (2000, 1152), (457, 16384)])
def test_norm_backward_in_place(ops, T, d, rt):
    lib = ops.load_library()
    dy, h, w, e = norm._bwd_inputs(T, d, 5, rt, True)
    want, dwant = ops.lmoe_add_rms_norm_backward(dy, h, w, EPS, dh=e)
    dw, ws = torch.empty(d, device="cuda"), torch.empty(4 * 152 * d, device="cuda", dtype=torch.uint8)
    assert lib.lmoe_add_rms_norm_backward(dy.data_ptr(), d, h.data_ptr(), d, e.data_ptr(), d, int(rt == torch.float32),
                                          T, d, w.data_ptr(), EPS, e.data_ptr(), dw.data_ptr(), ws.data_ptr(),
                                          ws.numel(), _stream()) == ops.LMOE_OK
    assert torch.equal(e, want) and torch.equal(dw, dwant)


@pytest.mark.parametrize("T", [50, 300, 1003])
def test_each_set_of_gradients(ops, T):
    lib = ops.load_library()
    d, F = 264, 520
    x, W, dy = ffn._make(T, d, F, 7)
    layer = ops.GatedFFN(W, max_tokens=T, training=True)
    _, g, u = layer.lmoe_ffn_forward(x, save=True)
    ref = R.backward(x, g, u, dy, W["gate"], W["up"], W["down"], "situ")
    bound = R.backward_bound(x, g, u, dy, W["gate"], W["up"], W["down"], "situ")
    for asked in itertools.product((False, True), repeat=4):
        out = [torch.full(r.shape, 7.0, device="cuda", dtype=torch.bfloat16) for r in ref]
        ptr = [o.data_ptr() if a else None for o, a in zip(out, asked)]
        assert lib.lmoe_ffn_backward(layer._h, x.data_ptr(), d, g.data_ptr(), u.data_ptr(), dy.data_ptr(), d, T, *ptr,
                                     _stream()) == ops.LMOE_OK
        for o, a, r, b in zip(out, asked, ref, bound):
            if a:
                assert bool(((o.to(R.D) - r).abs() <= b).all()), asked
            else:
                assert bool((o == 7).all()), asked
    layer.lmoe_ffn_sync_status()


@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(300001, 8), (100003, 32), (65537, 40), (30011, 264)])
def test_many_rows_of_few_values(ops, T, d, rt):
    norm.test_forward_many_rows(ops, T, d, rt)
    norm.test_backward(ops, T, d, rt, True)
