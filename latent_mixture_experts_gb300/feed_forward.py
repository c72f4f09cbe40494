"""Binding of include/lmoe_ffn.h: the residual addition with RMS norm and the
dense gated feed-forward block around the MoE layer, with their backward
passes.  Argument checks and marshalling only; every step runs in the
library's CUDA kernels and there is no CPU path.

Tensors are CUDA tensors of the current device; the last dimension is
contiguous, rows may be strided.  Outputs are allocated on the stream the
call runs on."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import binding as B

_OUT_FORMATS = {"bf16": 0, "mxfp8": 1}
_STREAM_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_BF16, _U8, _F32 = torch.bfloat16, torch.uint8, torch.float32
_PACKED = torch.contiguous_format


def _rows(name: str, t: torch.Tensor, dtypes, shape) -> int:
    """Row stride of a 2-D tensor, after checking what the kernels rely on."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.shape == shape:
        if t.is_contiguous() or t.shape[0] <= 1 and t.stride(1) == 1:
            return t.shape[1]
        if t.stride(1) == 1 or t.shape[1] <= 1:
            return t.stride(0)
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _counts(what: str, *n: int):
    """Row counts and widths cross the C ABI as ints of 32 bits, which ctypes would cut without a word."""
    for v in n:
        if v > 0x7FFFFFFF:
            raise ValueError(f"{what} {v} does not fit 32 bits")


def _packed(name: str, t: torch.Tensor, dtype, shape):
    if _rows(name, t, (dtype,), shape) != shape[1]:
        raise ValueError(f"{name} must be contiguous")


def _on_device(dev: int, *tensors):
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, not on CUDA device {dev}")


# The current device and stream without building their objects: a call on one
# token takes a few microseconds.
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _device_of(t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev != _raw_device():
        raise ValueError("tensors must be on the current CUDA device")
    return dev


def _norm_weight(w: torch.Tensor, shape):
    if w.dtype is not _BF16 or w.shape != shape or not w.is_contiguous():
        raise ValueError(f"norm_w must be a contiguous CUDA bfloat16 tensor of shape {tuple(shape)}")


def lmoe_add_rms_norm(x: torch.Tensor, norm_w: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
                      out_format: str = "bf16", h_out: torch.Tensor | None = None, stream=None):
    """h = residual + x (in residual's dtype, bf16 or fp32; h = x without a
    residual), y = norm_w * h / sqrt(mean(h^2) + eps).

    Returns (y, scales, h): y bf16 [T][d] and scales None, or with
    out_format="mxfp8" E4M3 codes uint8 [T][d] and E8M0 scales uint8
    [T][d/32]; h None without a residual.  h_out may be the residual itself."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return lmoe_add_rms_norm(x, norm_w, eps, residual, out_format, h_out)
    fmt = _OUT_FORMATS.get(out_format)
    if fmt is None:
        raise ValueError(f"out_format must be one of {sorted(_OUT_FORMATS)}")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [T][d]")
    T, d = shape
    _counts("a size of x,", T, d)
    ldx = _rows("x", x, (_BF16,), shape)
    dev = _device_of(x)
    _norm_weight(norm_w, shape[1:])
    s = sp = rp = hp = h = None
    ldr, st = d, 0
    if residual is not None:
        ldr = _rows("residual", residual, (_BF16, _F32), shape)
        _on_device(dev, norm_w, residual)
        st = _STREAM_TYPES[residual.dtype]
        if h_out is None:
            h = torch.empty_like(residual, memory_format=_PACKED)
        else:
            h = h_out
            _packed("h_out", h, residual.dtype, shape)
            _on_device(dev, h)
        rp, hp = residual.data_ptr(), h.data_ptr()
    else:
        _on_device(dev, norm_w)
        if h_out is not None:
            raise ValueError("h_out needs a residual")
    if fmt:
        y = torch.empty_like(x, dtype=_U8, memory_format=_PACKED)
        s = torch.empty(T, d // 32, dtype=_U8, device=x.device)
        sp = s.data_ptr()
    else:
        y = torch.empty_like(x, memory_format=_PACKED)
    status = B.load_library().lmoe_add_rms_norm(x.data_ptr(), ldx, rp, ldr, st, T, d, norm_w.data_ptr(), eps, hp,
                                                y.data_ptr(), fmt, sp, _raw_stream(dev))
    if status:
        raise B.LmoeError("lmoe_add_rms_norm", status)
    return y, s, h


@functools.lru_cache(maxsize=1024)
def _norm_backward_workspace(T: int, d: int) -> int:
    n = ctypes.c_size_t()
    B._check("lmoe_add_rms_norm_backward_workspace",
             B.load_library().lmoe_add_rms_norm_backward_workspace(T, d, ctypes.byref(n)))
    return n.value


def lmoe_add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, norm_w: torch.Tensor, eps: float,
                               dh: torch.Tensor | None = None, stream=None):
    """Gradients of lmoe_add_rms_norm from dy bf16 [T][d] and its h (bf16 or
    fp32); dh (h's dtype): the gradient along the residual stream.  Returns
    (dx in h's dtype, the gradient of x and of the residual alike; d norm_w
    fp32 [d])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return lmoe_add_rms_norm_backward(dy, h, norm_w, eps, dh)
    shape = h.shape
    if len(shape) != 2:
        raise ValueError("h must be [T][d]")
    T, d = shape
    _counts("a size of h,", T, d)
    ldh = _rows("h", h, (_BF16, _F32), shape)
    lddy = _rows("dy", dy, (_BF16,), shape)
    dev = _device_of(h)
    _norm_weight(norm_w, shape[1:])
    _on_device(dev, dy, norm_w)
    lddh, ep = d, None
    if dh is not None:
        lddh = _rows("dh", dh, (h.dtype,), shape)
        _on_device(dev, dh)
        ep = dh.data_ptr()
    n = _norm_backward_workspace(T, d)
    dx = torch.empty_like(h, memory_format=_PACKED)
    dw = torch.empty(d, dtype=_F32, device=h.device)
    ws = torch.empty(n, dtype=_U8, device=h.device)
    status = B.load_library().lmoe_add_rms_norm_backward(
        dy.data_ptr(), lddy, h.data_ptr(), ldh, ep, lddh, _STREAM_TYPES[h.dtype], T, d, norm_w.data_ptr(), eps,
        dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), n, _raw_stream(dev))
    if status:
        raise B.LmoeError("lmoe_add_rms_norm_backward", status)
    return dx, dw


def lmoe_add_rms_norm_selftest_timeout(x: torch.Tensor, norm_w: torch.Tensor, backward: bool = False):
    """A norm whose rows never are complete, so that its waits run out: (y,
    None), or with backward=True (dx, dw), all NaN."""
    T, d = x.shape
    _packed("x", x, _BF16, x.shape)
    _on_device(_device_of(x), norm_w)
    _norm_weight(norm_w, x.shape[1:])
    y = torch.empty_like(x)
    n = _norm_backward_workspace(T, d)
    dw = torch.empty(d, dtype=_F32, device=x.device) if backward else None
    ws = torch.empty(n, dtype=_U8, device=x.device)
    B._check("lmoe_add_rms_norm_selftest_timeout", B.load_library().lmoe_add_rms_norm_selftest_timeout(
        int(backward), x.data_ptr(), T, d, norm_w.data_ptr(), y.data_ptr(), dw.data_ptr() if backward else None,
        ws.data_ptr(), n, B._stream(None)))
    return y, dw


class GatedFFN:
    """One dense gated feed-forward block on the current CUDA device:
    y = (a(x gate^T) * v(x up^T)) down^T with SiTU-GLU or SwiGLU.

    weights: dict of contiguous CUDA tensors gate, up [d_ff][d_model] and down
    [d_model][d_ff]: bf16, or uint8 E4M3 codes with gate_s, up_s, down_s
    uint8 E8M0 scales (one per 32 input values).  Borrowed: in-place updates
    of bf16 weights between calls are seen; MXFP8 weights must not change.
    training=True allocates what the backward pass needs (bf16 weights).  One
    stream at a time."""

    def __init__(self, weights: dict, max_tokens: int, act: str = "situ", situ_beta: float = 4.0,
                 situ_linear_beta: float = 25.0, training: bool = False, stream=None):
        lib = B.load_library()
        if not torch.cuda.is_available():
            raise RuntimeError("lmoe needs a CUDA GPU; no CPU implementation exists")
        if act not in ("situ", "swiglu"):
            raise ValueError("act must be 'situ' or 'swiglu'")
        gate = weights["gate"]
        if gate.dim() != 2 or gate.dtype not in (torch.bfloat16, torch.uint8):
            raise ValueError("gate must be [d_ff][d_model], bfloat16 or uint8")
        F, d = gate.shape
        _counts("a size of gate or max_tokens,", F, d, int(max_tokens))
        self.mx = gate.dtype == torch.uint8
        shapes = {"gate": (F, d), "up": (F, d), "down": (d, F)}
        if self.mx:
            if d % 32 or F % 32:
                raise ValueError("MXFP8 weights need widths that are multiples of 32")
            shapes |= {"gate_s": (F, d // 32), "up_s": (F, d // 32), "down_s": (d, F // 32)}
        self._weights = {}
        for n, shape in shapes.items():
            t = weights[n]
            _packed(n, t, gate.dtype, shape)
            _on_device(_device_of(gate), t)
            self._weights[n] = t
        self.d_model, self.d_ff, self.max_tokens, self.act = d, F, int(max_tokens), act
        self.training = bool(training)
        c = B.LmoeFfnConfig(d_model=d, d_ff=F, act=B.LMOE_ACT_SITU if act == "situ" else B.LMOE_ACT_SWIGLU,
                            situ_beta=situ_beta, situ_linear_beta=situ_linear_beta, wfmt=int(self.mx),
                            max_tokens=int(max_tokens), training=int(self.training))
        w = B.LmoeFfnWeights(**{n: t.data_ptr() for n, t in self._weights.items()})
        self._device, self._dev = gate.device, gate.get_device()
        h = ctypes.c_void_p()
        B._check("lmoe_ffn_create", lib.lmoe_ffn_create(ctypes.byref(c), ctypes.byref(w), B._stream(stream),
                                                        ctypes.byref(h)))
        self._h, self._lib = h, lib

    def _current(self):
        if _raw_device() != self._dev:
            raise ValueError(f"the block is on {self._device}, which is not the current CUDA device")

    def _tokens(self, t: torch.Tensor, name: str, T: int) -> int:
        ld = _rows(name, t, (_BF16,), (T, self.d_model))
        if t.get_device() != self._dev:
            raise ValueError(f"{name} is on {t.device}, the block on {self._device}")
        return ld

    def _out(self, T: int, out):
        if out is None:
            return torch.empty(T, self.d_model, dtype=_BF16, device=self._device)
        _packed("out", out, _BF16, (T, self.d_model))
        _on_device(self._dev, out)
        return out

    def lmoe_ffn_forward(self, x: torch.Tensor, save: bool = False, out: torch.Tensor | None = None, stream=None):
        """x bf16 [T][d_model] -> y bf16; with save=True (y, g, u): the
        pre-activations bf16 [T][d_ff] that lmoe_ffn_backward takes."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.lmoe_ffn_forward(x, save, out)
        self._current()
        T = x.shape[0]
        _counts("the number of tokens,", T)
        ldx = self._tokens(x, "x", T)
        y = torch.empty_like(x, memory_format=_PACKED) if out is None else self._out(T, out)
        if not save:
            status = self._lib.lmoe_ffn_forward(self._h, x.data_ptr(), ldx, T, y.data_ptr(), None, None,
                                                _raw_stream(self._dev))
            if status:
                raise B.LmoeError("lmoe_ffn_forward", status)
            return y
        g = torch.empty(T, self.d_ff, dtype=_BF16, device=self._device)
        u = torch.empty_like(g)
        status = self._lib.lmoe_ffn_forward(self._h, x.data_ptr(), ldx, T, y.data_ptr(), g.data_ptr(), u.data_ptr(),
                                            _raw_stream(self._dev))
        if status:
            raise B.LmoeError("lmoe_ffn_forward", status)
        return y, g, u

    def lmoe_ffn_backward(self, x: torch.Tensor, g: torch.Tensor, u: torch.Tensor, dy: torch.Tensor,
                          need_dx: bool = True, need_dw: bool = True, stream=None):
        """-> (dx, dw_gate, dw_up, dw_down), bf16; None for those not asked for."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.lmoe_ffn_backward(x, g, u, dy, need_dx, need_dw)
        self._current()
        T, shape = x.shape[0], (x.shape[0], self.d_ff)
        _counts("the number of tokens,", T)
        ldx = self._tokens(x, "x", T)
        lddy = self._tokens(dy, "dy", T)
        _packed("g", g, _BF16, shape)
        _packed("u", u, _BF16, shape)
        _on_device(self._dev, g, u)
        dx = dwg = dwu = dwd = xp = gp = up = dp = None
        if need_dx:
            dx = torch.empty_like(x, memory_format=_PACKED)
            xp = dx.data_ptr()
        if need_dw:
            w = self._weights
            dwg, dwu, dwd = torch.empty_like(w["gate"]), torch.empty_like(w["up"]), torch.empty_like(w["down"])
            gp, up, dp = dwg.data_ptr(), dwu.data_ptr(), dwd.data_ptr()
        status = self._lib.lmoe_ffn_backward(self._h, x.data_ptr(), ldx, g.data_ptr(), u.data_ptr(), dy.data_ptr(),
                                             lddy, T, xp, gp, up, dp, _raw_stream(self._dev))
        if status:
            raise B.LmoeError("lmoe_ffn_backward", status)
        return dx, dwg, dwu, dwd

    def lmoe_ffn_forward_mx(self, x_codes: torch.Tensor, x_scales: torch.Tensor, out: torch.Tensor | None = None,
                            stream=None):
        """MXFP8 x (codes uint8 [T][d_model], scales uint8 [T][d_model/32],
        as lmoe_add_rms_norm(out_format="mxfp8") returns them) -> y bf16."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.lmoe_ffn_forward_mx(x_codes, x_scales, out)
        self._current()
        T = x_codes.shape[0]
        _counts("the number of tokens,", T)
        _packed("x_codes", x_codes, _U8, (T, self.d_model))
        _packed("x_scales", x_scales, _U8, (T, self.d_model // 32))
        _on_device(self._dev, x_codes, x_scales)
        y = self._out(T, out)
        status = self._lib.lmoe_ffn_forward_mx(self._h, x_codes.data_ptr(), x_scales.data_ptr(), T, y.data_ptr(),
                                               _raw_stream(self._dev))
        if status:
            raise B.LmoeError("lmoe_ffn_forward_mx", status)
        return y

    def lmoe_ffn_sync_status(self, stream=None):
        self._current()
        B._check("lmoe_ffn_sync_status", self._lib.lmoe_ffn_sync_status(self._h, B._stream(stream)))

    def lmoe_ffn_selftest_timeout(self, x: torch.Tensor, x_scales: torch.Tensor | None = None, stream=None):
        """A forward pass whose first product waits for rows that never come:
        the next lmoe_ffn_sync_status reports a timeout.  Returns its output."""
        self._current()
        _packed("x", x, _U8 if self.mx else _BF16, (x.shape[0], self.d_model))
        if self.mx:
            _packed("x_scales", x_scales, _U8, (x.shape[0], self.d_model // 32))
        y = torch.empty(x.shape[0], self.d_model, dtype=_BF16, device=self._device)
        B._check("lmoe_ffn_selftest_timeout", self._lib.lmoe_ffn_selftest_timeout(
            self._h, x.data_ptr(), x_scales.data_ptr() if self.mx else None, x.shape[0], y.data_ptr(),
            B._stream(stream)))
        return y

    def lmoe_ffn_last_launch_count(self) -> int:
        return int(self._lib.lmoe_ffn_last_launch_count(self._h))

    def lmoe_ffn_destroy(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            B._check("lmoe_ffn_destroy", self._lib.lmoe_ffn_destroy(self._h))
        self._h = None

    forward = lmoe_ffn_forward
    backward = lmoe_ffn_backward
    close = lmoe_ffn_destroy

    def __del__(self):
        try:
            self.lmoe_ffn_destroy()
        except Exception:
            pass
