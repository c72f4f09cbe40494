"""AdamW at the ends of its ranges: blocks whose values lie far apart, decays far below a
weight's last bit, values numbered from 2^32 on."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from tests import _block_reference as R
from tests._harness import built_library
from tests.test_gpu_adamw import BETAS, DECAY, EPS, LR, _check_step, _make, _optimizer, _snapshot

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    return P


@pytest.mark.parametrize("size", [1.0, 1e-6, 1e8])
@pytest.mark.parametrize("apart", [8, 20, 29, 31, 36, 38, 40, 50])
def test_roots_far_below_their_block(ops, apart, size):
    """Some gradients of each block are 2^apart below the others: their roots are not stored as zero, also in blocks
    with values over 28672, which are scaled in two steps."""
    params, grads = _make(21, shapes=[(2048,), (33, 65), (31,), (16384,)], pt=F32, gt=F32)
    opt, decay = _optimizer(ops, params, "mxfp8")
    for t, g in enumerate(grads[:2], 1):
        g = [x * size for x in g]
        for x in g:
            x.view(-1)[5::32] *= 2.0 ** -apart
            x.view(-1)[6::32] *= 2.0 ** -(apart + 1)
        before = [_snapshot(opt, i) for i in range(len(params))]
        opt.step(g)
        for i, x in enumerate(g):
            small = x.reshape(-1).to(R.D) ** 2 * (1 - BETAS[1]) >= 2.0 ** -125
            assert bool((opt.state(i)["v"] != 0)[small].all()), i
        _check_step(opt, before, g, decay, t)
