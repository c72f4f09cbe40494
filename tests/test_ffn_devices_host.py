"""Calls of include/lmoe_ffn.h with two devices, with a failing runtime call and
with tensors anywhere in memory, on a stand-in for the CUDA runtime."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from tests import _fake_cuda
from tests._harness import built_library

A = 0x10000      # an aligned address that nothing reads


@pytest.fixture
def lib(tmp_path_factory):
    lib = _fake_cuda.load(tmp_path_factory)
    yield lib
    lib.fake_set_device(0)


@pytest.fixture(scope="module")
def b():
    from latent_mixture_experts_gb300 import binding
    return binding


def _block(lib, b, mx=False, d=512, F=768, max_tokens=4096, training=1):
    h = ctypes.c_void_p()
    cfg = b.LmoeFfnConfig(d_model=d, d_ff=F, act=0, situ_beta=4.0, situ_linear_beta=25.0, wfmt=int(mx),
                          max_tokens=max_tokens, training=0 if mx else training)
    w = b.LmoeFfnWeights(**{n: A + (i << 20) for i, n in enumerate(b._FFN_WEIGHT_FIELDS)})
    assert lib.lmoe_ffn_create(ctypes.byref(cfg), ctypes.byref(w), None, ctypes.byref(h)) == b.LMOE_OK
    return h


def _calls(lib, h, mx, T, d=512):
    if mx:
        return [lambda: lib.lmoe_ffn_forward_mx(h, A, A, T, A, None)]
    return [lambda: lib.lmoe_ffn_forward(h, A, d, T, A, None, None, None),
            lambda: lib.lmoe_ffn_backward(h, A, d, A, A, A, d, T, A, A, A, A, None)]


# a token and small, middle and large batches: each form of the products
@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_block_on_each_of_two_devices(lib, b, mx):
    """A process may keep blocks on both of its devices: the second one's launches are as good as the first one's."""
    for dev in (0, 1):
        lib.fake_set_device(dev)
        h = _block(lib, b, mx)
        for T in (1, 40, 100, 300, 4096):
            for call in _calls(lib, h, mx, T):
                assert call() == b.LMOE_OK, (dev, T)
                assert lib.fake_last_device() == dev
        assert lib.lmoe_ffn_destroy(h) == b.LMOE_OK


@pytest.mark.parametrize("T,d", [(1, 256), (4000, 7168), (2000, 1152), (1023, 16384)])
def test_norm_on_each_of_two_devices(lib, b, T, d):
    for dev in (0, 1):
        lib.fake_set_device(dev)
        for st in (0, 1):
            for r in (None, A):
                for fmt in (0, 1):
                    assert lib.lmoe_add_rms_norm(A, d, r, d, st, T, d, A, 1e-6, A, A, fmt, A, None) == b.LMOE_OK
            for dh in (None, A):
                assert lib.lmoe_add_rms_norm_backward(A, d, A, d, dh, d, st, T, d, A, 1e-6, A, A, A, 1 << 30,
                                                      None) == b.LMOE_OK
        assert lib.fake_last_device() == dev


def test_a_failed_call_is_not_kept(lib, b):
    """A limit that could not be raised once is asked for again by the next call; then not any more."""
    def norm():
        return lib.lmoe_add_rms_norm_backward(A, 1152, A, 1152, None, 1152, 0, 2000, 1152, A, 1e-6, A, A, A, 1 << 30,
                                              None)
    lib.fake_fail_attributes(1)
    assert norm() == b.LMOE_ERR_OOM
    assert norm() == b.LMOE_OK
    n = lib.fake_attribute_calls()
    assert norm() == b.LMOE_OK and lib.fake_attribute_calls() == n
    h = _block(lib, b)
    for T in (1, 100, 4096):
        for call in _calls(lib, h, False, T):
            lib.fake_fail_attributes(1)      # of a kernel that no call before has launched, if there is one
            assert call() in (b.LMOE_ERR_OOM, b.LMOE_OK)
            lib.fake_fail_attributes(0)
            assert call() == b.LMOE_OK
    assert lib.lmoe_ffn_destroy(h) == b.LMOE_OK


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_a_block_is_refused_while_another_device_is_current(lib, b, mx):
    """Its memory lies on the other one, and a NULL stream would be this one's: nothing is launched."""
    h = _block(lib, b, mx)
    calls = _calls(lib, h, mx, 4) + _calls(lib, h, mx, 300) + [lambda: lib.lmoe_ffn_sync_status(h, None)]
    lib.fake_set_device(1)
    n = lib.fake_launches()
    for call in calls:
        assert call() == b.LMOE_ERR_INVALID_ARG
    assert lib.fake_launches() == n
    lib.fake_set_device(0)
    assert all(call() == b.LMOE_OK for call in calls)
    lib.fake_set_device(1)
    assert lib.lmoe_ffn_destroy(h) == b.LMOE_OK


def test_binding_refuses_a_block_while_another_device_is_current(monkeypatch):
    built_library()
    from latent_mixture_experts_gb300 import GatedFFN, feed_forward

    class Lib:                       # reached by none of the calls
        def __getattr__(self, name):
            raise AssertionError(name)
    block = GatedFFN.__new__(GatedFFN)
    block._lib, block._h, block._dev, block._device = Lib(), None, 1, torch.device("cuda:1")
    block.d_model, block.d_ff, block.max_tokens = 64, 128, 8
    with FakeTensorMode():           # tensors of a device that this machine need not have
        x, g = (torch.empty(4, n, device="cuda:1", dtype=torch.bfloat16) for n in (64, 128))
        q, s = (torch.empty(4, n, device="cuda:1", dtype=torch.uint8) for n in (64, 2))
    monkeypatch.setattr(feed_forward, "_raw_device", lambda: 0)
    for call in (lambda: block.lmoe_ffn_forward(x), lambda: block.lmoe_ffn_forward(x, save=True),
                 lambda: block.lmoe_ffn_backward(x, g, g, x), lambda: block.lmoe_ffn_forward_mx(q, s),
                 lambda: block.lmoe_ffn_sync_status()):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_self_test_arguments(lib, b, mx):
    h = _block(lib, b, mx)
    for T in (1, 16, 40, 300, 4096):
        assert lib.lmoe_ffn_selftest_timeout(h, A, A, T, A, None) == b.LMOE_OK
    for x, s, T, out in ((None, A, 4, A), (A, A, 0, A), (A, A, -1, A), (A, A, 4097, A), (A, A, 4, None),
                         (A + 8, A, 4, A), (A, None if mx else A, 4, A if mx else A + 2)):
        assert lib.lmoe_ffn_selftest_timeout(h, x, s, T, out, None) == b.LMOE_ERR_INVALID_ARG
    lib.fake_set_device(1)
    assert lib.lmoe_ffn_selftest_timeout(h, A, A, 4, A, None) == b.LMOE_ERR_INVALID_ARG
    lib.fake_set_device(0)
    assert lib.lmoe_ffn_destroy(h) == b.LMOE_OK


def test_binding_refuses_sizes_beyond_32_bits(monkeypatch):
    """They would reach the library cut to 32 bits: 2^32 + 4 rows as four."""
    built_library()
    from latent_mixture_experts_gb300 import GatedFFN, feed_forward, lmoe_add_rms_norm, lmoe_add_rms_norm_backward

    class Lib:                       # reached by none of the calls
        def __getattr__(self, name):
            raise AssertionError(name)
    monkeypatch.setattr(feed_forward.B, "load_library", lambda: Lib())
    monkeypatch.setattr(feed_forward, "_raw_device", lambda: 0)
    monkeypatch.setattr(feed_forward, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(feed_forward, "_norm_backward_workspace", lambda T, d: 32)
    block = GatedFFN.__new__(GatedFFN)
    block._lib, block._h, block._dev, block._device = Lib(), None, 0, torch.device("cuda:0")
    block.d_model, block.d_ff, block.max_tokens = 64, 64, 8
    n = 2 ** 32 + 4
    with FakeTensorMode():           # no memory behind them
        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, device="cuda:0", dtype=dtype)
        x8, w8, x1, w1 = empty(n, 8), empty(8), empty(1, n - 4 + 8), empty(n - 4 + 8)
        x, q, s = empty(n, 64), empty(n, 64, dtype=torch.uint8), empty(n, 2, dtype=torch.uint8)
        W = {"gate": empty(n + 4, 8), "up": empty(n + 4, 8), "down": empty(8, n + 4)}
        W8 = {k: empty(8, 8) for k in W}
        for call in (lambda: lmoe_add_rms_norm(x8, w8, 1e-6), lambda: lmoe_add_rms_norm(x8, w8, 1e-6, residual=x8),
                     lambda: lmoe_add_rms_norm(x1, w1, 1e-6), lambda: lmoe_add_rms_norm_backward(x8, x8, w8, 1e-6),
                     lambda: lmoe_add_rms_norm_backward(x1, x1, w1, 1e-6), lambda: block.lmoe_ffn_forward(x),
                     lambda: block.lmoe_ffn_backward(x, x, x, x), lambda: block.lmoe_ffn_forward_mx(q, s)):
            with pytest.raises(ValueError, match="32 bits"):
                call()
        monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
        for weights, tokens in ((W, 8), (W8, n)):
            with pytest.raises(ValueError, match="32 bits"):
                GatedFFN(weights, max_tokens=tokens)


@pytest.mark.parametrize("up_first", [False, True])
@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_every_tensor_map_lies_within_one_tensor(lib, b, mx, up_first):
    """The weights, the tokens and the workspace are allocations of their own, gigabytes apart or side by side: what a
    copy may touch between them, or past their ends, need not be memory."""
    lib.fake_tensor.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
    at = [1 << 40]

    def tensor(nbytes, gap=0):
        p = at[0]
        at[0] += (nbytes + 511) // 512 * 512 + gap
        lib.fake_tensor(p, nbytes)
        return p
    size = 1 if mx else 2
    sizes = ((32, 96), (288, 160), (2048, 6144)) if mx else ((8, 128), (64, 16), (264, 136), (512, 768), (2048, 6144))
    for d, F in sizes:
        for gap in (0, 512, 1 << 21, 5 << 29):
            for T in (1, 3, 8, 40, 72, 100, 300, 2100):
                lib.fake_forget_tensors()
                one, two, down = (tensor(size * d * F, gap) for _ in range(3))
                scales = tensor(d * F // 32, gap)
                gate, up = (two, one) if up_first else (one, two)
                w = b.LmoeFfnWeights(gate=gate, up=up, down=down, gate_s=scales, up_s=scales, down_s=scales)
                cfg = b.LmoeFfnConfig(d_model=d, d_ff=F, act=0, situ_beta=4.0, situ_linear_beta=25.0, wfmt=int(mx),
                                      max_tokens=T, training=int(not mx))
                h = ctypes.c_void_p()
                assert lib.lmoe_ffn_create(ctypes.byref(cfg), ctypes.byref(w), None, ctypes.byref(h)) == b.LMOE_OK
                n = lib.fake_maps()
                if mx:
                    x, s, y = tensor(T * d, gap), tensor(T * d // 32, gap), tensor(2 * T * d, gap)
                    assert lib.lmoe_ffn_forward_mx(h, x, s, T, y, None) == b.LMOE_OK
                else:
                    ld = d + 24
                    x, dy = (tensor(2 * ((T - 1) * ld + d), gap) for _ in range(2))
                    y, dx = (tensor(2 * T * d, gap) for _ in range(2))
                    g, u = (tensor(2 * T * F, gap) for _ in range(2))
                    dw = [tensor(2 * d * F, gap) for _ in range(3)]
                    assert lib.lmoe_ffn_forward(h, x, ld, T, y, g, u, None) == b.LMOE_OK
                    assert lib.lmoe_ffn_backward(h, x, ld, g, u, dy, ld, T, dx, *dw, None) == b.LMOE_OK
                assert lib.fake_maps() > n and lib.fake_maps_outside() == 0, (d, F, gap, T)
                assert lib.lmoe_ffn_destroy(h) == b.LMOE_OK
