"""lmoe_add_rms_norm and its backward pass against the 64-bit forms.

Tolerances: one rounding of the output type (bf16 2^-8, fp32 2^-24 relative;
E4M3 2^-4 relative or half a subnormal step, 2^-10 of the scale) on top of
the fp32 arithmetic: sums of d values to 2^-20 relative."""
import pytest
import torch

from tests import _ffn_reference as R
from tests._harness import built_library

pytestmark = pytest.mark.gpu
EPS = 1e-6
F32 = 2.0 ** -19      # fp32 sums, rsqrt and products, relative to the terms


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    return P


def _make(T, d, seed, rt=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(T, d, device="cuda", generator=g) * torch.exp(torch.randn(T, 1, device="cuda", generator=g)))
    w = (1 + 0.3 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    r = None if rt is None else (2 * torch.randn(T, d, device="cuda", generator=g)).to(rt)
    return x.bfloat16(), r, w


def _check_y(y, ref):
    err = (y.to(R.D) - ref).abs()
    assert bool((err <= (R.HALF[y.dtype] + F32) * ref.abs() + 1e-30).all()), float(err.max())


def _check_mx(q, s, ref):
    """Scales: the encoding's own, or the neighbour where the block's maximum is within F32 of the border.
    Codes: the decoded value within half a step of the exact one."""
    s64 = s.to(torch.int64)
    want = R.mx_scale(ref)
    lo, hi = R.mx_scale(ref * (1 - F32)), R.mx_scale(ref * (1 + F32))
    assert bool(((s64 == want) | (s64 == lo) | (s64 == hi)).all())
    dec = R.mx_decode(q, s)
    f = torch.exp2(s64.to(R.D) - 127).repeat_interleave(32, -1)
    tol = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * f) + F32 * ref.abs()
    assert bool(((dec - ref).abs() <= tol).all())
    own, _ = R.mx_encode(ref)
    assert float((dec != own).double().mean()) <= 1e-3     # boundary cases only


SHAPES = [(1, 8), (1, 7168), (2, 32), (3, 264), (5, 1152), (17, 256), (7, 2056), (33, 4096), (300, 3584), (4, 8192),
          (3, 12000), (2, 16384)]


@pytest.mark.parametrize("rt", [None, torch.bfloat16, torch.float32], ids=["none", "bf16", "fp32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(ops, T, d, rt):
    x, r, w = _make(T, d, T + d, rt)
    y, s, h = ops.lmoe_add_rms_norm(x, w, EPS, residual=r)
    ref, href = R.norm(x, r, w, EPS)
    assert s is None and (h is None) == (r is None)
    if r is not None:
        assert torch.equal(h, href)
    _check_y(y, ref)
    if d % 32 == 0:
        q, s, h = ops.lmoe_add_rms_norm(x, w, EPS, residual=r, out_format="mxfp8")
        assert r is None or torch.equal(h, href)
        _check_mx(q, s, ref)


@pytest.mark.parametrize("rt", [None, torch.bfloat16, torch.float32], ids=["none", "bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(4000, 7168), (8200, 256), (3001, 1152), (1000, 2600), (300, 8192), (301, 8184)])
def test_forward_many_rows(ops, T, d, rt):
    x, r, w = _make(T, d, 5, rt)
    y, _, h = ops.lmoe_add_rms_norm(x, w, EPS, residual=r)
    ref, href = R.norm(x, r, w, EPS)
    assert r is None or torch.equal(h, href)
    _check_y(y, ref)
    if d % 32 == 0:
        q, s, h = ops.lmoe_add_rms_norm(x, w, EPS, residual=r, out_format="mxfp8")
        assert r is None or torch.equal(h, href)
        _check_mx(q, s, ref)
    if r is not None:                # strided rows, the sum in place
        wide = torch.empty(T, d + 64, device="cuda", dtype=torch.bfloat16)
        wide[:, 32:32 + d] = x
        y2, _, h2 = ops.lmoe_add_rms_norm(wide[:, 32:32 + d], w, EPS, residual=r, h_out=r)
        assert torch.equal(h2, href) and torch.equal(y2, y)


@pytest.mark.parametrize("rt", [None, torch.bfloat16, torch.float32], ids=["none", "bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(1023, 8200), (911, 9216), (601, 16384)])
def test_forward_many_wide_rows(ops, T, d, rt):
    test_forward_many_rows(ops, T, d, rt)


def test_strided_rows_in_place_and_none(ops):
    T, d = 37, 512
    wide_x, _, w = _make(T, 3 * d, 6)
    wide_r = torch.randn(T, 2 * d, device="cuda")
    x, r = wide_x[:, d:2 * d], wide_r[:, :d]
    ref, href = R.norm(x, r, w[:d].contiguous(), EPS)
    y, _, h = ops.lmoe_add_rms_norm(x, w[:d].contiguous(), EPS, residual=r)
    assert torch.equal(h, href)
    _check_y(y, ref)
    r2 = r.contiguous()
    y2, _, h2 = ops.lmoe_add_rms_norm(x, w[:d].contiguous(), EPS, residual=r2, h_out=r2)
    assert h2.data_ptr() == r2.data_ptr() and torch.equal(h2, href) and torch.equal(y2, y)
    y0, s0, h0 = ops.lmoe_add_rms_norm(x[:0], w[:d].contiguous(), EPS, out_format="mxfp8")
    assert y0.shape == (0, d) and s0.shape == (0, d // 32) and h0 is None


def test_zero_infinite_and_nan_rows(ops):
    T, d = 6, 256
    x, _, w = _make(T, d, 7)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 9] = float("nan")
    x[4] = 3e38                      # the mean square overflows fp32: y = 0 as in 32-bit arithmetic
    ref, _ = R.norm(x, None, w, EPS)
    y, _, _ = ops.lmoe_add_rms_norm(x, w, EPS)
    for t in (0, 1, 5):
        _check_y(y[t:t + 1], ref[t:t + 1])
    assert torch.isnan(y[2, 5]) and bool((y[2, torch.arange(d, device="cuda") != 5] == 0).all())
    assert bool(torch.isnan(y[3]).all()) and bool((y[4] == 0).all())
    q, s, _ = ops.lmoe_add_rms_norm(x, w, EPS, out_format="mxfp8")
    _check_mx(q[:2], s[:2], ref[:2])
    assert bool((s[1] == 1).all()) and bool((q[1] == 0).all())
    assert int(s[2, 0]) == 255 and bool((s[2, 1:] == 1).all()) and bool((s[3] == 255).all())


def _bwd_inputs(T, d, seed, rt, dh):
    x, r, w = _make(T, d, seed, rt)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    dy = (torch.randn(T, d, device="cuda", generator=g) * 1e-2).bfloat16()
    return dy, r, w, (torch.randn(T, d, device="cuda", generator=g) * 1e-2).to(rt) if dh else None


def _check_bwd(dx, dw, dy, h, w, dh):
    rdx, rdw = R.norm_backward(dy, h, w, EPS, dh)
    hd, wd, dyd = h.to(R.D), w.to(R.D), dy.to(R.D)
    rho = 1 / torch.sqrt((hd * hd).mean(-1, keepdim=True) + EPS)
    terms = rho * ((wd * dyd).abs() + hd.abs() * rho ** 2 * (wd * dyd * hd).abs().mean(-1, keepdim=True))
    err = (dx.to(R.D) - rdx).abs()
    assert bool((err <= R.HALF[dx.dtype] * rdx.abs() + F32 * (terms + rdx.abs())).all())
    assert bool(((dw.to(R.D) - rdw).abs() <= F32 * (dyd * hd * rho).abs().sum(0) + 1e-30).all())


@pytest.mark.parametrize("dh", [False, True], ids=["alone", "with_stream"])
@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,d", SHAPES + [(509, 1152), (2500, 640)])
def test_backward(ops, T, d, rt, dh):
    dy, h, w, e = _bwd_inputs(T, d, T + d, rt, dh)
    dx, dw = ops.lmoe_add_rms_norm_backward(dy, h, w, EPS, dh=e)
    assert dx.dtype == rt and dw.dtype == torch.float32
    _check_bwd(dx, dw, dy, h, w, e)
    again = ops.lmoe_add_rms_norm_backward(dy, h, w, EPS, dh=e)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dh", [False, True], ids=["alone", "with_stream"])
@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(2000, 2560), (1500, 2568), (1201, 7168), (911, 8192), (903, 8200), (601, 12288),
                                 (457, 16384)])
def test_backward_many_wide_rows(ops, T, d, rt, dh):
    test_backward(ops, T, d, rt, dh)


def test_backward_strided_and_empty(ops):
    dy, h, w, e = _bwd_inputs(40, 1024, 9, torch.bfloat16, True)
    sl = slice(256, 768)
    dx, dw = ops.lmoe_add_rms_norm_backward(dy[:, sl], h[:, sl], w[sl].contiguous(), EPS, dh=e[:, sl])
    _check_bwd(dx, dw, dy[:, sl], h[:, sl], w[sl], e[:, sl])
    dx, dw = ops.lmoe_add_rms_norm_backward(dy[:0], h[:0], w, EPS)
    assert dx.shape == (0, 1024) and bool((dw == 0).all())


def test_streams_and_graph(ops):
    """On another stream than the current one, and captured into a graph."""
    x, r, w = _make(64, 1024, 11, torch.bfloat16)
    want = ops.lmoe_add_rms_norm(x, w, EPS, residual=r)
    dwant = ops.lmoe_add_rms_norm_backward(x, r, w, EPS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.lmoe_add_rms_norm(x, w, EPS, residual=r, stream=side)
    dgot = ops.lmoe_add_rms_norm_backward(x, r, w, EPS, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert torch.equal(dgot[0], dwant[0]) and torch.equal(dgot[1], dwant[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _, h = ops.lmoe_add_rms_norm(x, w, EPS, residual=r)
        dx, dw = ops.lmoe_add_rms_norm_backward(x, h, w, EPS)
    x2, r2, _ = _make(64, 1024, 12, torch.bfloat16)
    x.copy_(x2)
    r.copy_(r2)
    graph.replay()
    torch.cuda.synchronize()
    ref, href = R.norm(x2, r2, w, EPS)
    assert torch.equal(h, href)
    _check_y(y, ref)
    _check_bwd(dx, dw, x2, href, w, None)


def test_binding_refusals(ops):
    x, r, w = _make(4, 64, 13, torch.bfloat16)
    bad = [lambda: ops.lmoe_add_rms_norm(x.float(), w, EPS), lambda: ops.lmoe_add_rms_norm(x, w.float(), EPS),
           lambda: ops.lmoe_add_rms_norm(x, w[:32], EPS), lambda: ops.lmoe_add_rms_norm(x, w, EPS, residual=r[:3]),
           lambda: ops.lmoe_add_rms_norm(x.t().contiguous().t(), w, EPS),
           lambda: ops.lmoe_add_rms_norm(x, w, EPS, h_out=r),
           lambda: ops.lmoe_add_rms_norm(x, w, EPS, residual=r.half()),
           lambda: ops.lmoe_add_rms_norm_backward(x, r, w, EPS, dh=r.float()),
           lambda: ops.lmoe_add_rms_norm_backward(x[:2], r, w, EPS)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ops.LmoeError):
        ops.lmoe_add_rms_norm(x, w, -1.0)
    odd = torch.zeros(4, 72, device="cuda", dtype=torch.bfloat16)[:, 4:68]     # rows start 8 bytes off
    with pytest.raises(ops.LmoeError):
        ops.lmoe_add_rms_norm(odd, w, EPS)
