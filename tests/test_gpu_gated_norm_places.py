"""lmoe_gated_add_norm where its outputs take its inputs' places, and at the widths where
the number of vectors per thread changes."""
import pytest
import torch

from tests.test_gpu_gated_norm import (A, B, BF, EPS, F32, GATES, TYPES, _check_forward, _make, ops,  # noqa: F401
                                       pytestmark)  # noqa: F401


@pytest.mark.parametrize("T,d", [(1, 64), (37, 520), (400, 1152), (1500, 7168)])
@GATES
def test_c_call_in_place_of_the_block_output(ops, T, d, gate):
    """The C call's promise: o in place of y, h in place of the stream, and both."""
    import ctypes
    from latent_mixture_experts_gb300 import binding as b
    from latent_mixture_experts_gb300.block import _gated_args
    for rt in (BF, F32):
        c = _make(T, d, rt, gate)
        o, _, h = _check_forward(ops, c)
        for o_in, h_in in ((True, False), (False, True), (True, True)):
            y, s = c["y"].clone(), c["s"].clone()
            a, _ = _gated_args(y, s, "residual", c["w1"], c["w2"], EPS, c["gate"], A, B)
            o2, h2 = y if o_in else torch.empty_like(y), s if h_in else torch.empty_like(s)
            st = b.load_library().lmoe_gated_add_norm(ctypes.byref(a), h2.data_ptr(), o2.data_ptr(), 0, None,
                                                      torch.cuda.current_stream().cuda_stream)
            assert st == b.LMOE_OK
            assert torch.equal(o2, o) and torch.equal(h2, h)


@GATES
@TYPES
@pytest.mark.parametrize("T,d", [(1024, 3584), (1030, 3616), (1025, 4096), (1100, 4608), (1027, 4640), (1024, 5120),
                                 (1029, 5152), (1026, 6144), (1025, 6176), (1024, 7168), (1031, 7200), (1023, 7200),
                                 (333, 8192), (1024, 8192), (4095, 4096), (4096, 4088), (4099, 4104), (4096, 6144)])
def test_forward_on_both_sides_of_each_border(ops, T, d, rt, gate):
    c = _make(T, d, rt, gate)
    _check_forward(ops, c)
    if d % 32 == 0:
        _check_forward(ops, c, "mxfp8")
