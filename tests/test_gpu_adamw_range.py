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


@pytest.mark.parametrize("rate", [1e-5, 1e-6, 1e-7, 4e-8])
@pytest.mark.parametrize("pt,masters", [(F32, True), (BF, True)], ids=["fp32", "master"])
def test_decay_far_below_a_weight(ops, pt, masters, rate):
    """Without a gradient a weight loses lr weight_decay of itself, rounded once: off by half a step of fp32 at the
    weight's size, and by the rounding of the product lr weight_decay w (three of 2^-24)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    p = (1 + torch.rand(1 << 16, device="cuda", generator=g)).to(pt)
    lr = 1e-3
    opt = ops.AdamW([p], lr=lr, weight_decay=rate / lr, masters=masters)
    if pt is BF:
        opt.master.copy_(1 + torch.rand(1 << 16, device="cuda", generator=g))
    w = (opt.master if pt is BF else p).to(R.D).clone()
    opt.step([torch.zeros_like(p)])
    got = (opt.master if pt is BF else p).to(R.D)
    want = w * (1 - rate)
    assert bool(((got - want).abs() <= 2.0 ** -24 + 3 * 2.0 ** -24 * rate * w).all()), float((got - want).abs().max())


def test_steps_and_decay_are_added_before_the_weight(ops):
    """A step and a decay that each are less than half of a weight's last bit, and together more, arrive."""
    n = 1 << 12
    p = torch.full((n,), 1.5, device="cuda")
    rate = 0.4 * 2.0 ** -23 / 1.5
    opt = ops.AdamW([p], lr=0.4 * 2.0 ** -23, betas=(0.0, 0.0), eps=0.0, weight_decay=rate / (0.4 * 2.0 ** -23))
    opt.step([torch.ones(n, device="cuda")])
    assert bool((p == 1.5 - 2.0 ** -23).all())


@pytest.mark.parametrize("first", [(1 << 32) - 2048 - 32, (1 << 32) - 32, 1 << 32, 5 << 32, (1 << 40) + 96])
def test_numbers_beyond_32_bits(ops, first):
    """A tensor whose values are numbered from `first` on, through the C call: the words of the numbers, of whole
    vectors and of the last values, also where they pass 2^32."""
    from latent_mixture_experts_gb300 import binding as b
    lib, n = b.load_library(), 4096 + 77
    params, grads = _make(22, shapes=[(n,)])
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    t = b.LmoeAdamwTensor(param=params[0].data_ptr(), n=n, first=first, weight_decay=DECAY, m=m.data_ptr(),
                          v=v.data_ptr(), m_scale=ms.data_ptr(), v_scale=vs.data_ptr())
    c = b.LmoeAdamwConfig(beta1=BETAS[0], beta2=BETAS[1], eps=EPS, states=1, seed=7, step=count.data_ptr())
    h = ctypes.c_void_p()
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.lmoe_adamw_create(ctypes.byref(c), ctypes.byref(t), 1, stream, ctypes.byref(h)) == b.LMOE_OK
    opt = SimpleNamespace(params=params, offsets=[first], seed=7, states="mxfp8",
                          state=lambda i: {"m": m, "v": v, "m_scales": ms, "v_scales": vs})
    for k, g in enumerate(grads, 1):
        before = [_snapshot(opt, 0)]
        assert lib.lmoe_adamw_step(h, (ctypes.c_void_p * 1)(g[0].data_ptr()), None, LR, None, None,
                                   stream) == b.LMOE_OK
        _check_step(opt, before, g, [DECAY], k)
    assert int(count) == 3 and lib.lmoe_adamw_destroy(h) == b.LMOE_OK
