"""Sizes near 2^31, which the C calls' ints still hold: taken or refused, on the stand-in
for the CUDA runtime.  Rows of the products are counted in ints, tiles of 256 at a time, so
that they refuse sizes over 2^30; the norms take every T."""
import ctypes

import pytest

from tests import _fake_block, _fake_cuda
from tests._harness import built_library

A = 0x10000      # an aligned address that nothing reads
MOST, LAST = 1 << 30, (1 << 31) - 1


@pytest.fixture(scope="module")
def b():
    built_library()
    from latent_mixture_experts_gb300 import binding
    return binding


@pytest.mark.parametrize("training", [0, 1])
@pytest.mark.parametrize("size", [dict(d_in=MOST + 8), dict(d_in=LAST - 7), dict(d_out=MOST + 8),
                                  dict(d_out=LAST - 7)])
def test_products_wider_than_2_30_are_refused(tmp_path_factory, b, size, training):
    lib = _fake_block.load(tmp_path_factory)
    c = b.LmoeLinearConfig(**(dict(d_in=8, d_out=8, act=0, max_tokens=1, training=training) | size))
    h = ctypes.c_void_p()
    assert lib.lmoe_linear_create(ctypes.byref(c), A, None, None, ctypes.byref(h)) == b.LMOE_ERR_UNSUPPORTED
    assert not h.value


@pytest.mark.parametrize("T", [MOST + 1, LAST])
def test_products_of_more_than_2_30_rows_are_refused(tmp_path_factory, b, T):
    lib = _fake_block.load(tmp_path_factory)
    c, h = b.LmoeLinearConfig(d_in=8, d_out=8, act=0, max_tokens=T, training=0), ctypes.c_void_p()
    assert lib.lmoe_linear_create(ctypes.byref(c), A, None, None, ctypes.byref(h)) == b.LMOE_OK
    n = lib.fake_launches()
    assert lib.lmoe_linear_forward(h, A, 8, T, None, 8, 0, A, A, None) == b.LMOE_ERR_UNSUPPORTED
    assert lib.lmoe_linear_selftest_timeout(h, A, T, A, None) == b.LMOE_ERR_UNSUPPORTED
    assert lib.fake_launches() == n and lib.lmoe_linear_destroy(h) == b.LMOE_OK


@pytest.mark.parametrize("size", [dict(max_tokens=MOST), dict(d_in=MOST), dict(d_out=MOST)])
def test_products_of_2_30_run(tmp_path_factory, b, size):
    lib = _fake_block.load(tmp_path_factory)
    kw = dict(d_in=8, d_out=8, act=1, max_tokens=1, training=0) | size
    c, h = b.LmoeLinearConfig(**kw), ctypes.c_void_p()
    assert lib.lmoe_linear_create(ctypes.byref(c), A, None, None, ctypes.byref(h)) == b.LMOE_OK
    assert lib.lmoe_linear_forward(h, A, kw["d_in"], kw["max_tokens"], A, kw["d_out"], 0, A, A, None) == b.LMOE_OK
    assert lib.lmoe_linear_destroy(h) == b.LMOE_OK


@pytest.mark.parametrize("mx", [0, 1])
@pytest.mark.parametrize("size", [dict(d_model=MOST + 32), dict(d_ff=LAST - 31)])
def test_blocks_wider_than_2_30_are_refused(tmp_path_factory, b, size, mx):
    lib = _fake_cuda.load(tmp_path_factory)
    c = b.LmoeFfnConfig(**(dict(d_model=32, d_ff=32, act=0, situ_beta=4.0, situ_linear_beta=25.0, wfmt=mx,
                                max_tokens=1, training=0) | size))
    w, h = b.LmoeFfnWeights(**{n: A for n in b._FFN_WEIGHT_FIELDS}), ctypes.c_void_p()
    assert lib.lmoe_ffn_create(ctypes.byref(c), ctypes.byref(w), None, ctypes.byref(h)) == b.LMOE_ERR_UNSUPPORTED
    assert not h.value


@pytest.mark.parametrize("T", [MOST, LAST])
def test_norms_of_any_number_of_rows(tmp_path_factory, b, T):
    lib = _fake_block.load(tmp_path_factory)
    for gate in (0, 1, 2):
        a = b.LmoeGatedNormArgs(T=T, d=8, y=A, ldy=8, stream=A, lds=8, stream_type=1, gate_type=gate, gate=A, ldgate=8,
                                w_post=A, w_next=A, stream_scale=1.0, branch_scale=1.0, eps=1e-6)
        assert lib.lmoe_gated_add_norm(ctypes.byref(a), A, A, 0, None, None) == b.LMOE_OK
        assert lib.lmoe_gated_add_norm_backward(ctypes.byref(a), A, 8, A, 8, A, A, A, A, A, A, 1 << 30,
                                                None) == b.LMOE_OK
    lib = _fake_cuda.load(tmp_path_factory)
    assert lib.lmoe_add_rms_norm(A, 8, A, 8, 0, T, 8, A, 1e-6, A, A, 0, A, None) == b.LMOE_OK
    assert lib.lmoe_add_rms_norm_backward(A, 8, A, 8, A, 8, 0, T, 8, A, 1e-6, A, A, A, 1 << 30, None) == b.LMOE_OK
