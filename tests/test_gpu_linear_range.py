"""The backward pass of Linear at the ends of its range: many rows for each thread of the
bias gradient's sums, and pre-activations that are NaN."""
import pytest
import torch

from tests import _block_reference as R
from tests._harness import built_library

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    return P


def _bias_gradient(ops, dy):
    T, N = dy.shape
    x = torch.zeros(T, 8, device="cuda", dtype=BF)
    layer = ops.Linear(torch.zeros(N, 8, device="cuda", dtype=BF), torch.zeros(N, device="cuda", dtype=BF),
                       max_tokens=T, training=True)
    return layer.lmoe_linear_backward(x, dy, need_dx=False)[2]


@pytest.mark.parametrize("T,N", [(1 << 20, 512), (1 << 14, 80000), (1 << 17, 6144)])
def test_bias_gradient_of_many_rows(ops, T, N):
    """Values whose last bits a running sum of a thousand of them loses, always to the same side: the sum stays within
    2^-16 of the terms, as few rows' sums do."""
    v = 1 + 0.99 * 2.0 ** -14
    dy = torch.full((T, N), v, device="cuda")
    want = T * float(dy[0, 0])
    got = _bias_gradient(ops, dy).to(R.D)
    assert bool(((got - want).abs() <= 2.0 ** -16 * want).all()), float((got - want).abs().max()) / want


@pytest.mark.parametrize("T,N,dt", [(65536, 6144, F32), (65536, 264, BF), (4099, 80008, BF), (20000, 8, F32)])
def test_bias_gradient_of_random_rows(ops, T, N, dt):
    g = torch.Generator(device="cuda").manual_seed(T + N)
    dy = torch.randn(T, N, device="cuda", generator=g).to(dt)
    got = _bias_gradient(ops, dy).to(R.D)
    for c in range(0, N, 4096):
        d = dy[:, c:c + 4096].to(R.D)
        assert bool(((got[c:c + 4096] - d.sum(0)).abs() <= 2.0 ** -16 * d.abs().sum(0) + R.TINY).all())


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "fp32"])
def test_slope_of_nan_is_nan(ops, act, dt):
    """Where the forward pass gave NaN, so does the backward pass: a saved z of NaN is no zero slope."""
    T, N = 40, 64
    layer = ops.Linear(torch.eye(N, device="cuda").to(BF), torch.zeros(N, device="cuda", dtype=BF), act, max_tokens=T,
                       training=True)
    x = torch.randn(T, N, device="cuda").to(BF)
    x[3, 5] = float("nan")
    y, z = layer.lmoe_linear_forward(x, save=True)
    assert bool(y[3].isnan().all()) and bool(y[4:].isfinite().all())
    z[4:] = x[4:]
    dx, dw, db = layer.lmoe_linear_backward(x.nan_to_num(0.0), torch.ones(T, N, device="cuda", dtype=dt), z)
    keep = torch.arange(T, device="cuda") != 3
    assert bool(dx[3].isnan().all()) and bool(dx[keep].isfinite().all())
    assert bool(dw.isnan().all()) and bool(db.isnan().all())
