"""Host side of include/lmoe_ffn.h without a GPU: refusals of every entry
point (nothing is launched: the pointers are never dereferenced), and the
64-bit reference's gradients against differences."""
import ctypes

import pytest
import torch

from tests import _ffn_reference as R
from tests._harness import built_library

A = 0x10000      # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    built_library()
    from latent_mixture_experts_gb300 import binding
    return binding.load_library()


@pytest.fixture(scope="module")
def b():
    from latent_mixture_experts_gb300 import binding
    return binding


def _norm(lib, x=A, ldx=64, r=None, ldr=64, st=0, T=4, d=64, w=A, eps=1e-6, h=None, y=A, fmt=0, s=None):
    return lib.lmoe_add_rms_norm(x, ldx, r, ldr, st, T, d, w, eps, h, y, fmt, s, None)


def test_norm_refusals(lib, b):
    inv, uns = b.LMOE_ERR_INVALID_ARG, b.LMOE_ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=A + 2), dict(w=A + 8), dict(y=A + 4), dict(T=-1),
               dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=56), dict(r=A),
               dict(r=A, h=A + 2), dict(r=A, h=A, ldr=56), dict(fmt=1), dict(fmt=2), dict(st=2), dict(d=0)):
        assert _norm(lib, **kw) == inv, kw
    for kw in (dict(d=60), dict(d=40, ldx=40, fmt=1, s=A), dict(d=16392, ldx=16392), dict(ldx=66),
               dict(r=A, h=A, ldr=68)):
        assert _norm(lib, **kw) == uns, kw
    assert _norm(lib, T=0, x=None, y=None) == b.LMOE_OK


def _norm_bwd(lib, dy=A, lddy=64, h=A, ldh=64, dh=None, lddh=64, st=0, T=4, d=64, w=A, eps=1e-6, dx=A, dw=A, ws=A,
              n=1 << 30):
    return lib.lmoe_add_rms_norm_backward(dy, lddy, h, ldh, dh, lddh, st, T, d, w, eps, dx, dw, ws, n, None)


def test_norm_backward_refusals(lib, b):
    inv, uns = b.LMOE_ERR_INVALID_ARG, b.LMOE_ERR_UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.lmoe_add_rms_norm_backward_workspace(4, 64, ctypes.byref(n)) == b.LMOE_OK and n.value >= 256
    for kw in (dict(dy=None), dict(h=None), dict(dx=None), dict(dw=None), dict(ws=None), dict(n=n.value - 1),
               dict(ws=A + 8), dict(T=-1), dict(ldh=32), dict(dh=A, lddh=8), dict(dh=A + 2), dict(st=3),
               dict(eps=-1.0)):
        assert _norm_bwd(lib, **kw) == inv, kw
    for kw in (dict(d=12), dict(d=16392), dict(lddy=68)):
        assert _norm_bwd(lib, **kw) == uns, kw
    assert lib.lmoe_add_rms_norm_backward_workspace(4, 64, None) == inv
    assert lib.lmoe_add_rms_norm_backward_workspace(-1, 64, ctypes.byref(n)) == inv
    assert lib.lmoe_add_rms_norm_backward_workspace(4, 63, ctypes.byref(n)) == uns
    assert lib.lmoe_add_rms_norm_backward_workspace(0, 64, ctypes.byref(n)) == b.LMOE_OK and n.value == 0


def _create(lib, b, weights=None, null=(), **kw):
    c = dict(d_model=64, d_ff=128, act=0, situ_beta=4.0, situ_linear_beta=25.0, wfmt=0, max_tokens=16, training=0)
    c.update(kw)
    vals = {n: A for n in b._FFN_WEIGHT_FIELDS}
    vals.update(weights or {})
    h = ctypes.c_void_p()
    cfg, w = b.LmoeFfnConfig(**c), b.LmoeFfnWeights(**vals)
    st = lib.lmoe_ffn_create(None if "cfg" in null else ctypes.byref(cfg), None if "w" in null else ctypes.byref(w),
                             None, None if "out" in null else ctypes.byref(h))
    assert not h.value or st == b.LMOE_OK
    return st, h


def test_ffn_create_refusals(lib, b):
    inv, uns = b.LMOE_ERR_INVALID_ARG, b.LMOE_ERR_UNSUPPORTED
    for null in ("cfg", "w", "out"):
        assert _create(lib, b, null=(null,))[0] == inv
    for kw in (dict(d_model=0), dict(d_ff=-8), dict(max_tokens=0), dict(act=2), dict(wfmt=2), dict(training=2),
               dict(situ_beta=0.0), dict(situ_linear_beta=float("nan")), dict(situ_beta=float("inf"))):
        assert _create(lib, b, **kw)[0] == inv, kw
    for w in (dict(gate=0), dict(up=0), dict(down=0), dict(gate=A + 8)):
        assert _create(lib, b, weights=w)[0] == inv, w
    for w in (dict(gate_s=0), dict(down_s=A + 4)):
        assert _create(lib, b, weights=w, wfmt=1)[0] == inv, w
    for kw in (dict(d_model=60), dict(d_ff=100), dict(wfmt=1, d_model=72), dict(wfmt=1, training=1)):
        assert _create(lib, b, **kw)[0] == uns, kw


def test_ffn_create_without_gpu_reports_cuda(lib, b):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _create(lib, b)[0] == b.LMOE_ERR_CUDA


def test_ffn_null_handle(lib, b):
    inv = b.LMOE_ERR_INVALID_ARG
    assert lib.lmoe_ffn_forward(None, A, 64, 1, A, None, None, None) == inv
    assert lib.lmoe_ffn_backward(None, A, 64, A, A, A, 64, 1, A, A, A, A, None) == inv
    assert lib.lmoe_ffn_forward_mx(None, A, A, 1, A, None) == inv
    assert lib.lmoe_ffn_sync_status(None, None) == inv
    assert lib.lmoe_ffn_selftest_timeout(None, A, A, 1, A, None) == inv
    assert lib.lmoe_ffn_last_launch_count(None) == 0
    assert lib.lmoe_ffn_destroy(None) == b.LMOE_OK


def test_binding_refuses_host_tensors():
    built_library()
    from latent_mixture_experts_gb300 import lmoe_add_rms_norm, lmoe_add_rms_norm_backward
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lmoe_add_rms_norm(x, w, 1e-6)
    with pytest.raises(ValueError):
        lmoe_add_rms_norm(x, w, 1e-6, out_format="fp4")
    with pytest.raises(ValueError):
        lmoe_add_rms_norm_backward(x, x, w, 1e-6)


@pytest.mark.parametrize("act", ["situ", "swiglu"])
def test_reference_gradients_against_differences(act):
    """backward() is the derivative of forward(): central differences in 64 bits."""
    g = torch.Generator().manual_seed(3)
    T, d, F = 5, 8, 12
    P = {n: torch.randn(*s, generator=g, dtype=R.D) for n, s in
         (("x", (T, d)), ("gate", (F, d)), ("up", (F, d)), ("down", (d, F)))}
    dy = torch.randn(T, d, generator=g, dtype=R.D)
    _, gg, uu = R.forward(P["x"], P["gate"], P["up"], P["down"], act, 1.5, 2.5)
    grads = dict(zip(("x", "gate", "up", "down"),
                     R.backward(P["x"], gg, uu, dy, P["gate"], P["up"], P["down"], act, 1.5, 2.5)))
    eps = 1e-5
    for n in P:
        v = torch.randn(P[n].shape, generator=g, dtype=R.D)
        f = []
        for sgn in (1, -1):
            Q = dict(P)
            Q[n] = P[n] + sgn * eps * v
            f.append((R.forward(Q["x"], Q["gate"], Q["up"], Q["down"], act, 1.5, 2.5)[0] * dy).sum())
        num = float(f[0] - f[1]) / (2 * eps)
        assert abs(num - float((grads[n] * v).sum())) <= 1e-7 * (1 + abs(num)), n


def test_reference_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(4)
    T, d = 3, 16
    h, w, dy = (torch.randn(*s, generator=g, dtype=R.D) for s in ((T, d), (d,), (T, d)))
    dx, dw = R.norm_backward(dy, h, w, 1e-3)
    eps = 1e-6
    for base, grad, which in ((h, dx, 0), (w, dw, 1)):
        v = torch.randn(base.shape, generator=g, dtype=R.D)
        f = [(R.norm(base + s * eps * v, None, w, 1e-3)[0] if which == 0 else
              R.norm(h, None, base + s * eps * v, 1e-3)[0]).mul(dy).sum() for s in (1, -1)]
        num = float(f[0] - f[1]) / (2 * eps)
        assert abs(num - float((grad * v).sum())) <= 1e-7 * (1 + abs(num))


def test_norm_self_test_refusals(lib, b):
    def call(backward=0, x=A, T=2048, d=4096, w=A, y=A, dw=A, ws=A, n=1 << 30):
        return lib.lmoe_add_rms_norm_selftest_timeout(backward, x, T, d, w, y, dw, ws, n, None)
    inv, uns = b.LMOE_ERR_INVALID_ARG, b.LMOE_ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(T=0), dict(T=-1), dict(x=A + 2), dict(backward=1, dw=None),
               dict(backward=1, ws=None), dict(backward=1, n=16)):
        assert call(**kw) == inv, kw
    for kw in (dict(d=4100), dict(d=16392), dict(T=2047)):
        assert call(**kw) == uns, kw
