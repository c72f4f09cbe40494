"""Binding of include/lmoe_ffn.h: the residual addition with RMS norm and the
dense gated feed-forward block around the MoE layer, with their backward
passes.  Argument checks and marshalling only; every step runs in the
library's CUDA kernels and there is no CPU path.

Tensors are CUDA tensors of the current device; the last dimension is
contiguous, rows may be strided.  Outputs are allocated on the stream the
call runs on."""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding as B

_OUT_FORMATS = {"bf16": 0, "mxfp8": 1}
_STREAM_TYPES = {torch.bfloat16: 0, torch.float32: 1}


def _rows(name: str, t: torch.Tensor, dtypes, shape) -> int:
    """Row stride of a 2-D tensor, after checking what the kernels rely on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if t.shape[0] <= 1:
        return t.shape[1]
    return t.stride(0)


def _packed(name: str, t: torch.Tensor, dtype, shape):
    if _rows(name, t, (dtype,), shape) != shape[1]:
        raise ValueError(f"{name} must be contiguous")


def _same_device(ref: torch.Tensor, **others):
    if ref.device.index != torch.cuda.current_device():
        raise ValueError("tensors must be on the current CUDA device")
    for name, t in others.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} is on {t.device}, not {ref.device}")


def _on(stream):
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _norm_weight(w: torch.Tensor, d: int):
    if not w.is_cuda or w.dtype != torch.bfloat16 or tuple(w.shape) != (d,) or not w.is_contiguous():
        raise ValueError(f"norm_w must be a contiguous CUDA bfloat16 tensor of shape ({d},)")


def lmoe_add_rms_norm(x: torch.Tensor, norm_w: torch.Tensor, eps: float, residual: torch.Tensor | None = None,
                      out_format: str = "bf16", h_out: torch.Tensor | None = None, stream=None):
    """h = residual + x (in residual's dtype, bf16 or fp32; h = x without a
    residual), y = norm_w * h / sqrt(mean(h^2) + eps).

    Returns (y, scales, h): y bf16 [T][d] and scales None, or with
    out_format="mxfp8" E4M3 codes uint8 [T][d] and E8M0 scales uint8
    [T][d/32]; h None without a residual.  h_out may be the residual itself."""
    if out_format not in _OUT_FORMATS:
        raise ValueError(f"out_format must be one of {sorted(_OUT_FORMATS)}")
    if x.dim() != 2:
        raise ValueError("x must be [T][d]")
    T, d = x.shape
    ldx = _rows("x", x, (torch.bfloat16,), (T, d))
    _norm_weight(norm_w, d)
    ldr, st, h = d, 0, None
    _same_device(x, norm_w=norm_w, residual=residual, h_out=h_out)
    if residual is not None:
        ldr = _rows("residual", residual, tuple(_STREAM_TYPES), (T, d))
        st = _STREAM_TYPES[residual.dtype]
        if h_out is not None:
            _packed("h_out", h_out, residual.dtype, (T, d))
    elif h_out is not None:
        raise ValueError("h_out needs a residual")
    mx = out_format == "mxfp8"
    with _on(stream):
        y = torch.empty(T, d, dtype=torch.uint8 if mx else torch.bfloat16, device=x.device)
        s = torch.empty(T, d // 32, dtype=torch.uint8, device=x.device) if mx else None
        if residual is not None:
            h = h_out if h_out is not None else torch.empty(T, d, dtype=residual.dtype, device=x.device)
    B._check("lmoe_add_rms_norm", B.load_library().lmoe_add_rms_norm(
        B._ptr(x), ldx, B._ptr(residual), ldr, st, T, d, B._ptr(norm_w), float(eps), B._ptr(h), B._ptr(y),
        _OUT_FORMATS[out_format], B._ptr(s), B._stream(stream)))
    return y, s, h


def lmoe_add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, norm_w: torch.Tensor, eps: float,
                               dh: torch.Tensor | None = None, stream=None):
    """Gradients of lmoe_add_rms_norm from dy bf16 [T][d] and its h (bf16 or
    fp32); dh (h's dtype): the gradient along the residual stream.  Returns
    (dx in h's dtype, the gradient of x and of the residual alike; d norm_w
    fp32 [d])."""
    if h.dim() != 2:
        raise ValueError("h must be [T][d]")
    T, d = h.shape
    ldh = _rows("h", h, tuple(_STREAM_TYPES), (T, d))
    lddy = _rows("dy", dy, (torch.bfloat16,), (T, d))
    lddh = d if dh is None else _rows("dh", dh, (h.dtype,), (T, d))
    _norm_weight(norm_w, d)
    _same_device(h, dy=dy, norm_w=norm_w, dh=dh)
    lib = B.load_library()
    n = ctypes.c_size_t()
    B._check("lmoe_add_rms_norm_backward_workspace",
             lib.lmoe_add_rms_norm_backward_workspace(T, d, ctypes.byref(n)))
    with _on(stream):
        dx = torch.empty(T, d, dtype=h.dtype, device=h.device)
        dw = torch.empty(d, dtype=torch.float32, device=h.device)
        ws = torch.empty(n.value, dtype=torch.uint8, device=h.device)
    B._check("lmoe_add_rms_norm_backward", lib.lmoe_add_rms_norm_backward(
        B._ptr(dy), lddy, B._ptr(h), ldh, B._ptr(dh), lddh, _STREAM_TYPES[h.dtype], T, d, B._ptr(norm_w), float(eps),
        B._ptr(dx), B._ptr(dw), B._ptr(ws), n.value, B._stream(stream)))
    return dx, dw


class GatedFFN:
    """One dense gated feed-forward block on the current CUDA device:
    y = (a(x gate^T) * v(x up^T)) down^T with SiTU-GLU or SwiGLU.

    weights: dict of contiguous CUDA tensors gate, up [d_ff][d_model] and down
    [d_model][d_ff]: bf16, or uint8 E4M3 codes with gate_s, up_s, down_s
    uint8 E8M0 scales (one per 32 input values).  Borrowed: in-place updates
    between calls are seen.  training=True allocates what the backward pass
    needs (bf16 weights).  One stream at a time."""

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
            _same_device(t)
            self._weights[n] = t
        self.d_model, self.d_ff, self.max_tokens, self.act = d, F, int(max_tokens), act
        self.training = bool(training)
        c = B.LmoeFfnConfig(d_model=d, d_ff=F, act=B.LMOE_ACT_SITU if act == "situ" else B.LMOE_ACT_SWIGLU,
                            situ_beta=situ_beta, situ_linear_beta=situ_linear_beta, wfmt=int(self.mx),
                            max_tokens=int(max_tokens), training=int(self.training))
        w = B.LmoeFfnWeights(**{n: t.data_ptr() for n, t in self._weights.items()})
        self._device = gate.device
        h = ctypes.c_void_p()
        B._check("lmoe_ffn_create", lib.lmoe_ffn_create(ctypes.byref(c), ctypes.byref(w), B._stream(stream),
                                                        ctypes.byref(h)))
        self._h, self._lib = h, lib

    def _tokens(self, t: torch.Tensor, name: str, dtype=torch.bfloat16):
        ld = _rows(name, t, (dtype,), (t.shape[0], self.d_model))
        if t.device != self._device:
            raise ValueError(f"{name} is on {t.device}, the block on {self._device}")
        return ld

    def lmoe_ffn_forward(self, x: torch.Tensor, save: bool = False, out: torch.Tensor | None = None, stream=None):
        """x bf16 [T][d_model] -> y bf16; with save=True (y, g, u): the
        pre-activations bf16 [T][d_ff] that lmoe_ffn_backward takes."""
        ldx, T = self._tokens(x, "x"), x.shape[0]
        g = u = None
        with _on(stream):
            if out is None:
                out = torch.empty(T, self.d_model, dtype=torch.bfloat16, device=x.device)
            else:
                _packed("out", out, torch.bfloat16, (T, self.d_model))
            if save:
                g = torch.empty(T, self.d_ff, dtype=torch.bfloat16, device=x.device)
                u = torch.empty_like(g)
        B._check("lmoe_ffn_forward", self._lib.lmoe_ffn_forward(
            self._h, B._ptr(x), ldx, T, B._ptr(out), B._ptr(g), B._ptr(u), B._stream(stream)))
        return (out, g, u) if save else out

    def lmoe_ffn_backward(self, x: torch.Tensor, g: torch.Tensor, u: torch.Tensor, dy: torch.Tensor,
                          need_dx: bool = True, need_dw: bool = True, stream=None):
        """-> (dx, dw_gate, dw_up, dw_down), bf16; None for those not asked for."""
        ldx, T = self._tokens(x, "x"), x.shape[0]
        lddy = self._tokens(dy, "dy")
        if dy.shape[0] != T:
            raise ValueError("x and dy must have the same number of rows")
        _packed("g", g, torch.bfloat16, (T, self.d_ff))
        _packed("u", u, torch.bfloat16, (T, self.d_ff))
        _same_device(x, g=g, u=u, dy=dy)
        dx = dwg = dwu = dwd = None
        with _on(stream):
            if need_dx:
                dx = torch.empty(T, self.d_model, dtype=torch.bfloat16, device=x.device)
            if need_dw:
                dwg = torch.empty(self.d_ff, self.d_model, dtype=torch.bfloat16, device=x.device)
                dwu = torch.empty_like(dwg)
                dwd = torch.empty(self.d_model, self.d_ff, dtype=torch.bfloat16, device=x.device)
        B._check("lmoe_ffn_backward", self._lib.lmoe_ffn_backward(
            self._h, B._ptr(x), ldx, B._ptr(g), B._ptr(u), B._ptr(dy), lddy, T, B._ptr(dx), B._ptr(dwg), B._ptr(dwu),
            B._ptr(dwd), B._stream(stream)))
        return dx, dwg, dwu, dwd

    def lmoe_ffn_forward_mx(self, x_codes: torch.Tensor, x_scales: torch.Tensor, out: torch.Tensor | None = None,
                            stream=None):
        """MXFP8 x (codes uint8 [T][d_model], scales uint8 [T][d_model/32],
        as lmoe_add_rms_norm(out_format="mxfp8") returns them) -> y bf16."""
        T = x_codes.shape[0]
        _packed("x_codes", x_codes, torch.uint8, (T, self.d_model))
        _packed("x_scales", x_scales, torch.uint8, (T, self.d_model // 32))
        self._tokens(x_codes, "x_codes", torch.uint8)
        _same_device(x_codes, x_scales=x_scales)
        with _on(stream):
            if out is None:
                out = torch.empty(T, self.d_model, dtype=torch.bfloat16, device=x_codes.device)
            else:
                _packed("out", out, torch.bfloat16, (T, self.d_model))
        B._check("lmoe_ffn_forward_mx", self._lib.lmoe_ffn_forward_mx(
            self._h, B._ptr(x_codes), B._ptr(x_scales), T, B._ptr(out), B._stream(stream)))
        return out

    def lmoe_ffn_sync_status(self, stream=None):
        B._check("lmoe_ffn_sync_status", self._lib.lmoe_ffn_sync_status(self._h, B._stream(stream)))

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
