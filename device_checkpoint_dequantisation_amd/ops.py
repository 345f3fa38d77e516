"""Operators that compute on quantised weights: the matrix product (st_linear), the 8-bit encoding of its input
(st_encode) and the norm ahead of it (st_rms_norm).  Like the rest of the package this only checks and
marshals arguments; the kernels are in the library and there is no fallback.

    q = ckpt.quantized()                                         # weights as stored
    a, h = rms_norm(x, norm_w, residual=h, quantize="MXFP8")     # 8-bit activations and the new residual stream
    u = linear(a, q["up.weight"])                                # bf16
    g = linear(a, q["gate.weight"])
    h = linear(quantize_activation(u, "MXFP8", gate=g), q["down.weight"], residual=h)

or, with the activations left in bf16, ``linear(x, q["up.weight"], activation="silu")``.

They run on the current stream (or ``stream``), allocate their outputs with torch, synchronise nothing and can be
captured into a HIP graph.  They have no backward pass: with grad mode on, inputs that require grad are refused, and
so are inputs with a forward-mode tangent."""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch
import torch.autograd.forward_ad as _fwd

from . import _lib
from ._lib import EncodeArgs, LinearArgs, OUT_DTYPES, RmsNormArgs, check, lib

ACTIVATIONS = (None, "relu", "silu", "gelu", "gelu_tanh")      # st_activation codes 0..4
# st_x_type codes 2..4, and the weight kinds each goes with
ACTIVATION_KINDS = ("FP8_ROW", "FP8_GROUP128", "MXFP8")
PAIRS = {"FP8_ROW": ("FP8_TENSOR",), "FP8_GROUP128": ("FP8_BLOCK128",), "MXFP8": ("MXFP8", "MXFP4")}

_TYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}            # st_out_dtype (and st_x_type 0, 1)
_TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ACT = {a: i for i, a in enumerate(ACTIVATIONS)}
_KIND = {k: i for i, k in enumerate(_lib.KINDS)}
_XKIND = {k: i + 2 for i, k in enumerate(ACTIVATION_KINDS)}
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# the current stream's handle without the Python object around it (0.1 instead of 2 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


@dataclass
class QuantizedActivation:
    """Rows in 8 bits with scales; a value is code * scale.
      FP8_ROW       data float8_e4m3fn [..., K], scale fp32 [...]
      FP8_GROUP128  data float8_e4m3fn [..., K], scale fp32 [..., ceil(K/128)]
      MXFP8         data float8_e4m3fn [..., K], scale float8_e8m0fnu [..., K/32]"""
    kind: str
    shape: tuple        # logical shape [..., K]
    data: object
    scale: object


def _scale_shape(kind: str, shape) -> tuple:
    if kind == "FP8_ROW":
        return tuple(shape[:-1])
    return (*shape[:-1], -(-shape[-1] // 128) if kind == "FP8_GROUP128" else shape[-1] // 32)


def _on_device(device, tensors, who: str):
    if device.type != "cuda":
        raise ValueError(f"{who}: needs GPU tensors, got one on {device}")
    grad = torch.is_grad_enabled()
    forward = getattr(_fwd, "_current_level", 0) >= 0      # inside a forward-mode level: a dual tensor does not require grad
    for t in tensors:
        if t is None:
            continue
        if t.device != device:
            raise ValueError(f"{who}: tensors on {device} and {t.device}")
        if grad and t.requires_grad:
            raise RuntimeError(f"{who}: has no backward pass; call it under torch.no_grad() or detach its inputs")
        if forward and _fwd.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{who}: has no derivative; an input carries a forward-mode tangent, which would be lost")


def adjacent_rows(t):
    """t [M, K], or a copy of it where its rows' elements are not adjacent or its rows overlap (one row for all is neither)."""
    ok = (t.shape[1] <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) == 0 or t.stride(0) >= t.shape[1])
    return t if ok else t.contiguous()


def _rows(t, cols: int, name: str, who: str):
    """t as [rows, cols] with adjacent columns: (tensor, pitch in elements).  A matrix is taken as it is, other shapes are copied
    where they are no such rows (whether reshape itself copies depends on the batch)."""
    if t.dim() != 2:
        t = adjacent_rows(t.reshape(-1, cols)) if t.numel() else t.new_empty((_count(t.shape[:-1]), cols))
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{who}: the last dimension of {name} must be contiguous (stride 1, got {t.stride(1)})")
    return t, t.stride(0)


def _count(shape) -> int:
    n = 1
    for s in shape:
        n *= s
    return n


def _launch(fn, args, device, stream, tensors, who):
    """Enqueue fn(args, stream) on ``stream``, ordered after the current stream's work, with ``device`` current."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _launch(fn, args, device, stream, tensors, who)
    if stream is None:
        raw = _raw_stream(device.index)
    else:
        if stream.device != device:
            raise ValueError(f"{who}: stream of {stream.device}, tensors on {device}")
        cur = torch.cuda.current_stream(device)
        if stream != cur:
            stream.wait_stream(cur)
            for t in tensors:       # allocated on the current stream, used on this one
                if t is not None:
                    t.record_stream(stream)
        raw = stream.cuda_stream
    check(fn(C.byref(args), raw), who)


def _check_weight(w, who: str):
    shape = tuple(w.shape)
    kind = w.kind
    if not (kind in _KIND and _KIND[kind] >= 3):
        raise ValueError(f"{who}: weight kind {kind!r} is not a quantised kind")
    if not (len(shape) == 2):
        raise ValueError(f"{who}: weight of shape {shape}; a matrix [N, K] is needed")
    n, k = shape
    d, s = w.data, w.scale
    fp4 = kind == "NVFP4" or kind == "MXFP4"
    if not (d.dtype == (torch.uint8 if fp4 else _E4M3) and tuple(d.shape) == (n, k // 2 if fp4 else k) and d.is_contiguous()):
        raise ValueError(f"{who}: {kind} weight [{n}, {k}] holds {d.dtype} {tuple(d.shape)}, strides {d.stride()}")
    if kind == "FP8_TENSOR":
        want, dt = 1, torch.float32
        if not (s.numel() == 1):
            raise ValueError(f"{who}: FP8_TENSOR scale has {s.numel()} elements")
        want = tuple(s.shape)
    elif kind == "FP8_BLOCK128":
        want, dt = (-(-n // 128), -(-k // 128)), torch.float32
    elif kind == "NVFP4":
        if not (k % 16 == 0):
            raise ValueError(f"{who}: NVFP4 K {k} is not a multiple of 16")
        want, dt = (n, k // 16), _E4M3
        g = w.scale2
        if not (g is not None and g.numel() == 1 and g.dtype == torch.float32):
            raise ValueError(f"{who}: NVFP4 needs one fp32 global scale")
    else:
        if not (k % 32 == 0):
            raise ValueError(f"{who}: {kind} K {k} is not a multiple of 32")
        want, dt = (n, k // 32), _E8M0
    if not (s.dtype == dt and tuple(s.shape) == want and s.is_contiguous()):
        raise ValueError(f"{who}: {kind} weight [{n}, {k}] has scales {s.dtype} {tuple(s.shape)}, strides {s.stride()}")
    return n, k


def _span(t):
    """First byte and the byte after the last of a tensor with elements."""
    p = t.data_ptr()
    last = t.numel() - 1 if t.is_contiguous() else sum((s - 1) * st for s, st in zip(t.shape, t.stride()))
    return p, p + (last + 1) * t.element_size()


def _overlaps(out, t) -> bool:
    if t is None or t.numel() == 0 or out.numel() == 0:
        return False
    (a, b), (c, d) = _span(out), _span(t)
    if not (a < d and c < b):
        return False
    if out.dim() in (2, 3) and t.dim() in (2, 3) and out.shape[0] > 1 and t.shape[0] > 1:
        # columns of one buffer: the same pitch p, and rows (of a head's elements, or of all heads') that start `by` bytes apart modulo p
        p = out.stride(0) * out.element_size()
        wide, other = _row_bytes(out), _row_bytes(t)
        if p == t.stride(0) * t.element_size() and 0 < wide <= p and 0 < other <= p:
            by = (c - a) % p
            return by < wide or by + other > p
    return True


def _row_bytes(t) -> int:
    """Bytes from the first to behind the last of t[i], a row or one row for each head; 0 for rows whose elements are not adjacent."""
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        return 0
    heads = 0 if t.dim() == 2 else (t.shape[1] - 1) * t.stride(1)
    return (heads + t.shape[-1]) * t.element_size()


def linear(x, weight, bias=None, residual=None, activation: str | None = None, out_dtype: str | None = None, out=None,
           stream=None):
    """act(x @ weight.T + bias) + residual for a :class:`QuantizedWeight` ``weight`` [N, K].

    ``x`` [..., K]: bf16 or fp16 (any weight kind), or a :class:`QuantizedActivation` whose kind goes with the weight's
    (FP8_ROW with FP8_TENSOR, FP8_GROUP128 with FP8_BLOCK128, MXFP8 with MXFP8 and MXFP4).  ``bias`` [N] and ``residual``
    [..., N] are bf16, fp16 or fp32; ``activation`` is None, "relu", "silu", "gelu" (erf) or "gelu_tanh".  The result
    has ``out_dtype`` (bf16, f16 or f32; default x's type, bf16 for 8-bit x), or goes to ``out``, which may be
    ``residual`` itself.  The rows of a matrix (and of ``residual``) are read where they are, at any pitch, and have to have
    adjacent elements; inputs of other shapes are copied where they have not.  The weight's exact values enter (code
    times scale, not rounded to bf16 first), sums are fp32 and the result is rounded once.  The exception: bf16 results of more than 64 8-bit rows come from the scaled matrix
    instructions, whose sums carry some 16 bits (off by 2e-5 of the results' root mean square on average, a fiftieth of bf16's
    rounding); ``out_dtype`` "f16" or "f32" has fp32 sums."""
    who = "linear"
    n, k = _check_weight(weight, who)
    if isinstance(x, QuantizedActivation):
        if x.kind not in PAIRS or weight.kind not in PAIRS[x.kind]:
            raise ValueError(f"{who}: {x.kind} activations do not go with {weight.kind} weights")
        xd, xs, x_type = x.data, x.scale, _XKIND[x.kind]
        if not (xd.dtype == _E4M3 and xd.is_contiguous() and tuple(xd.shape) == tuple(x.shape)):
            raise ValueError(f"{who}: {x.kind} activations hold {xd.dtype} {tuple(xd.shape)}, strides {xd.stride()}")
        if not (xs.dtype == (_E8M0 if x.kind == "MXFP8" else torch.float32) and xs.is_contiguous() and tuple(xs.shape) == _scale_shape(x.kind, x.shape)):
            raise ValueError(f"{who}: {x.kind} activations {tuple(x.shape)} have scales {xs.dtype} {tuple(xs.shape)}, strides {xs.stride()}")
        default = torch.bfloat16
    else:
        xd, xs, default = x, None, x.dtype
        x_type = _TYPE.get(default, 2)
        if not (x_type < 2):
            raise ValueError(f"{who}: x is {default}; bf16, fp16 or a QuantizedActivation is needed")
    lead = xd.shape[:-1]
    if not (xd.dim() >= 1 and xd.shape[-1] == k):
        raise ValueError(f"{who}: x {tuple(xd.shape)} against a weight of K {k}")
    device = xd.device
    _on_device(device, (xd, xs, weight.data, weight.scale, weight.scale2, bias, residual, out), who)
    if activation not in _ACT:
        raise ValueError(f"{who}: unknown activation {activation!r}; one of {ACTIVATIONS}")
    x2, x_pitch = _rows(xd, k, "x", who)
    m = x2.shape[0]
    if bias is not None:
        if not (bias.dtype in _TYPE and tuple(bias.shape) == (n,) and (n <= 1 or bias.stride(0) == 1)):
            raise ValueError(f"{who}: bias {bias.dtype} {tuple(bias.shape)}, strides {bias.stride()}; [{n}] is needed")
    shape = (*lead, n)
    r2, r_pitch = None, 0
    if residual is not None:
        if not (residual.dtype in _TYPE and tuple(residual.shape) == shape):
            raise ValueError(f"{who}: residual {residual.dtype} {tuple(residual.shape)}; {shape} is needed")
        r2, r_pitch = _rows(residual, n, "residual", who)
    if out is None:
        if out_dtype is not None and out_dtype not in _TORCH:
            raise ValueError(f"{who}: unknown out_dtype {out_dtype!r}; one of {OUT_DTYPES}")
        out = xd.new_empty(shape, dtype=_TORCH[out_dtype] if out_dtype else default)
        o2 = out if out.dim() == 2 else out.view(m, n)
    else:
        if not (out.dtype in _TYPE and tuple(out.shape) == shape):
            raise ValueError(f"{who}: out {out.dtype} {tuple(out.shape)}; {shape} is needed")
        if not (out_dtype is None or _TORCH.get(out_dtype) == out.dtype):
            raise ValueError(f"{who}: out is {out.dtype}, out_dtype {out_dtype!r}")
        try:
            o2 = out if out.dim() == 2 else out.view(m, n)
        except RuntimeError:
            raise ValueError(f"{who}: out {shape} with strides {out.stride()} is not a matrix of rows") from None
        if not ((n <= 1 or o2.stride(1) == 1) and (m <= 1 or o2.stride(0) >= n)):
            raise ValueError(f"{who}: out has strides {out.stride()}")
        same = r2 is not None and r2.data_ptr() == o2.data_ptr() and r2.dtype == o2.dtype and r2.stride() == o2.stride()
        for t in (x2, xs, weight.data, weight.scale, weight.scale2, bias, None if same else r2):
            if _overlaps(o2, t):
                raise ValueError(f"{who}: out overlaps an input")
    if m == 0 or n == 0:
        return out
    s2 = weight.scale2
    args = LinearArgs(x2.data_ptr(), None if xs is None else xs.data_ptr(), weight.data.data_ptr(), weight.scale.data_ptr(),
                      None if s2 is None else s2.data_ptr(), None if bias is None else bias.data_ptr(),
                      None if r2 is None else r2.data_ptr(), o2.data_ptr(), None, 0, m, n, k, x_pitch, r_pitch, o2.stride(0),
                      x_type, _KIND[weight.kind], _ACT[activation], 0 if bias is None else _TYPE[bias.dtype],
                      0 if r2 is None else _TYPE[r2.dtype], _TYPE[o2.dtype])
    need = C.c_uint64()
    check(lib().st_linear_workspace_bytes(C.byref(args), C.byref(need)), who)
    work = None
    if need.value:
        work = xd.new_empty(need.value, dtype=torch.uint8)
        args.workspace, args.workspace_bytes = work.data_ptr(), need.value
    _launch(lib().st_linear, args, device, stream, (x2, xs, weight.data, weight.scale, s2, bias, r2, o2, work), who)
    return out


def _new_activation(kind: str, x):
    """An empty activation of x's shape."""
    shape = tuple(x.shape)
    return QuantizedActivation(kind, shape, torch.empty_like(x, dtype=_E4M3, memory_format=torch.contiguous_format),
                               x.new_empty(_scale_shape(kind, shape), dtype=_E8M0 if kind == "MXFP8" else torch.float32))


def _check_kind(kind, cols: int, who: str):
    if kind not in ACTIVATION_KINDS:
        raise ValueError(f"{who}: unknown encoding {kind!r}; one of {ACTIVATION_KINDS}")
    if not (kind != "MXFP8" or cols % 32 == 0):
        raise ValueError(f"{who}: MXFP8 needs a multiple of 32 columns, got {cols}")


def quantize_activation(x, kind: str, gate=None, stream=None) -> QuantizedActivation:
    """x [..., K] (bf16, fp16 or fp32), or silu(gate) * x with ``gate`` of x's shape and type, in e4m3 with scales:
    ``kind`` "FP8_ROW" (fp32 amax / 448 per row), "FP8_GROUP128" (the same per 128 columns) or "MXFP8" (the power of two at
    or above it per 32 columns).  A value that is not finite becomes the NaN code and does not enter amax."""
    who = "quantize_activation"
    if not (x.dtype in _TYPE and x.dim() >= 1):
        raise ValueError(f"{who}: x is {x.dtype} {tuple(x.shape)}; bf16, fp16 or fp32 rows are needed")
    k = x.shape[-1]
    _check_kind(kind, k, who)
    _on_device(x.device, (x, gate), who)
    x2, x_pitch = _rows(x, k, "x", who)
    g2, g_pitch = None, 0
    if gate is not None:
        if not (gate.dtype == x.dtype and gate.shape == x.shape):
            raise ValueError(f"{who}: gate {gate.dtype} {tuple(gate.shape)}, x {x.dtype} {tuple(x.shape)}")
        g2, g_pitch = _rows(gate, k, "gate", who)
    q = _new_activation(kind, x)
    m = x2.shape[0]
    if m == 0:
        return q
    args = EncodeArgs(x2.data_ptr(), None if g2 is None else g2.data_ptr(), q.data.data_ptr(), q.scale.data_ptr(), m, k, x_pitch,
                      g_pitch, _TYPE[x.dtype], _XKIND[kind])
    _launch(lib().st_encode, args, x.device, stream, (x2, g2, q.data, q.scale), who)
    return q


def rms_norm(x, weight=None, eps: float = 1e-6, residual=None, quantize: str | None = None, out_dtype: str | None = None,
             stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight over the last dimension, with h = x + residual.

    Returns y, or (y, h) with a ``residual`` (of x's shape and type; h rounded to that type, y from the unrounded h).  y has
    ``out_dtype`` (default x's type) or, with ``quantize`` (an encoding of :func:`quantize_activation`), is the
    :class:`QuantizedActivation` of the unrounded y.  ``weight`` [K] may be bf16, fp16 or fp32."""
    who = "rms_norm"
    if not (x.dtype in _TYPE and x.dim() >= 1):
        raise ValueError(f"{who}: x is {x.dtype} {tuple(x.shape)}; bf16, fp16 or fp32 rows are needed")
    k = x.shape[-1]
    _on_device(x.device, (x, weight, residual), who)
    if not (eps >= 0.0):
        raise ValueError(f"{who}: eps {eps} is negative")
    x2, x_pitch = _rows(x, k, "x", who)
    m = x2.shape[0]
    if weight is not None:
        if not (weight.dtype in _TYPE and tuple(weight.shape) == (k,) and (k <= 1 or weight.stride(0) == 1)):
            raise ValueError(f"{who}: weight {weight.dtype} {tuple(weight.shape)}, strides {weight.stride()}; [{k}] is needed")
    r2, r_pitch, h = None, 0, None
    if residual is not None:
        if not (residual.dtype == x.dtype and residual.shape == x.shape):
            raise ValueError(f"{who}: residual {residual.dtype} {tuple(residual.shape)}, x {x.dtype} {tuple(x.shape)}")
        r2, r_pitch = _rows(residual, k, "residual", who)
        h = torch.empty_like(x, memory_format=torch.contiguous_format)
    if quantize is not None:
        if not (out_dtype is None):
            raise ValueError(f"{who}: out_dtype and quantize exclude each other")
        _check_kind(quantize, k, who)
        y = _new_activation(quantize, x)
        yd, ys, kind, out_type = y.data, y.scale, _XKIND[quantize], 0
    else:
        if out_dtype is not None and out_dtype not in _TORCH:
            raise ValueError(f"{who}: unknown out_dtype {out_dtype!r}; one of {OUT_DTYPES}")
        y = yd = torch.empty_like(x, dtype=_TORCH[out_dtype] if out_dtype else x.dtype, memory_format=torch.contiguous_format)
        ys, kind, out_type = None, 0, _TYPE[y.dtype]
    if m:
        args = RmsNormArgs(x2.data_ptr(), None if r2 is None else r2.data_ptr(), None if weight is None else weight.data_ptr(),
                           None if h is None else h.data_ptr(), yd.data_ptr(), None if ys is None else ys.data_ptr(), m, k, x_pitch,
                           r_pitch, eps, _TYPE[x.dtype], 0 if weight is None else _TYPE[weight.dtype], out_type, kind)
        _launch(lib().st_rms_norm, args, x.device, stream, (x2, r2, weight, h, yd, ys), who)
    return y if residual is None else (y, h)
