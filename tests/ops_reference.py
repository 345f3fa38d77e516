"""Plain 64-bit forms of the operators on quantised weights, on the CPU, and random operands for their tests.
Codes are read from their bit fields here; nothing of the package is used but its QuantizedWeight container."""
import math

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], dtype=torch.float64)


def e4m3(d):
    c = d.contiguous().view(torch.uint8).to(torch.int64)
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.pow(2.0, (e - 10).double()))
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(c >= 128, -v, v)


def e8m0(s):
    c = s.contiguous().view(torch.uint8).double()
    return torch.where(c == 255, torch.full_like(c, math.nan), torch.pow(2.0, c - 127))


def nibbles(d):
    return E2M1[torch.stack((d & 15, d >> 4), -1).flatten(-2).long()]


def weight_value(w):
    """fp64 [N, K] of a QuantizedWeight on the CPU."""
    n, k = w.shape
    if w.kind == "FP8_TENSOR":
        return e4m3(w.data) * w.scale.double()
    if w.kind == "FP8_BLOCK128":
        return e4m3(w.data) * w.scale.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    if w.kind == "NVFP4":
        return nibbles(w.data) * e4m3(w.scale).repeat_interleave(16, 1) * w.scale2.double()
    return (e4m3(w.data) if w.kind == "MXFP8" else nibbles(w.data)) * e8m0(w.scale).repeat_interleave(32, 1)


def rows_value(kind, data, scale):
    """fp64 [M, K] of 8-bit rows on the CPU."""
    k = data.shape[-1]
    if kind == "FP8_ROW":
        return e4m3(data) * scale.double().unsqueeze(-1)
    if kind == "FP8_GROUP128":
        return e4m3(data) * scale.double().repeat_interleave(128, -1)[..., :k]
    return e4m3(data) * e8m0(scale).repeat_interleave(32, -1)


def activate(act, v):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v)) if not v.isnan().any() else torch.relu(v)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def random_codes(g, *shape):
    """e4m3 codes of every finite value, evenly over the codes of modest size."""
    c = torch.randint(0, 127, shape, generator=g, dtype=torch.uint8)
    c = torch.where(c > 0x60, c - 0x30, c)          # keep most magnitudes below 2^5: the sums stay comparable
    return (c | (torch.randint(0, 2, shape, generator=g, dtype=torch.uint8) << 7)).view(torch.float8_e4m3fn)


def random_weight(st, kind, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    u = lambda lo, hi, *s: torch.rand(*s, generator=g) * (hi - lo) + lo   # noqa: E731
    if kind in ("NVFP4", "MXFP4"):
        d = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    else:
        d = random_codes(g, n, k)
    s2 = None
    if kind == "FP8_TENSOR":
        s = u(0.001, 0.01, 1)[0]
    elif kind == "FP8_BLOCK128":
        s = 10.0 ** u(-4, -2, -(-n // 128), -(-k // 128))
    elif kind == "NVFP4":
        s, s2 = (2.0 ** u(-6, 6, n, k // 16)).to(torch.float8_e4m3fn), u(1e-3, 1e-1, 1)[0]
    else:
        s = torch.randint(117, 132, (n, k // 32), generator=g, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    return st.QuantizedWeight("w", kind, (n, k), d, s, s2)


def random_rows(st, kind, m, k, seed):
    """A dense tensor, or a QuantizedActivation, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    if kind in DT:
        return torch.randn(m, k, generator=g).to(DT[kind])
    d = random_codes(g, m, k)
    if kind == "MXFP8":
        s = torch.randint(117, 132, (m, k // 32), generator=g, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    else:
        s = torch.rand(*((m,) if kind == "FP8_ROW" else (m, -(-k // 128))), generator=g) * 0.1 + 0.001
    return st.QuantizedActivation(kind, (m, k), d, s)


def to(obj, device):
    """A copy of a QuantizedWeight / QuantizedActivation / tensor on `device`."""
    if obj is None or torch.is_tensor(obj):
        return None if obj is None else obj.to(device)
    new = type(obj)(**{f: getattr(obj, f) for f in obj.__dataclass_fields__})
    for f in ("data", "scale", "scale2"):
        if getattr(new, f, None) is not None:
            setattr(new, f, getattr(new, f).to(device))
    return new


def linear(x, w, bias=None, residual=None, activation=None):
    """(y, s) in fp64: the result, and the sum of magnitudes that its rounding errors are measured by."""
    a = x.double() if torch.is_tensor(x) else rows_value(x.kind, x.data, x.scale)
    b = weight_value(w)
    y, s = a @ b.t(), a.abs() @ b.abs().t()
    if bias is not None:
        y, s = y + bias.double(), s + bias.double().abs()
    y = activate(activation, y)
    if residual is not None:
        y, s = y + residual.double(), s + residual.double().abs()
    return y, s


def linear_tolerance(y, s, k, dtype):
    """Largest error of a result summed in fp32 in any order and rounded once to `dtype`.
    Summing k exact products: at most (k + 2) steps, each off by 2^-23 of the magnitudes' sum s (2^-24 for rounding to
    nearest; a matrix instruction may cut instead); scales, bias, activation (slope at most 1.13, itself evaluated to
    a few 2^-24) and residual: 16 more such steps.  Rounding to dtype: half a step relative, and half the smallest
    subnormal."""
    fp32 = 1.13 * (k + 18) * 2.0 ** -23 * s
    return fp32 + (y.abs() + fp32) * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def f8_tolerance(x, w):
    """What the f8f6f4 matrix instructions may cut: of 16 neighbouring products, what lies below 2^-13 of the largest
    one; at most 15 times 2^-13 times max|x| max|w| over the 16."""
    a, b = rows_value(x.kind, x.data, x.scale).abs(), weight_value(w).abs()
    pad = -a.shape[1] % 16
    big = lambda t: torch.nn.functional.pad(t, (0, pad)).unflatten(1, (-1, 16)).amax(2)   # noqa: E731
    return 1.13 * 15 * 2.0 ** -13 * (big(a) @ big(b).t())


def scale_of(kind, v):
    """(scale as fp32 or E8M0 codes, its fp64 value spread over v's columns) by the definition, for finite or other v."""
    m, d = v.shape
    w = {"FP8_ROW": max(d, 1), "FP8_GROUP128": 128, "MXFP8": 32}[kind]
    a = torch.where(v.isfinite(), v.abs(), torch.zeros_like(v))
    groups = -(-d // w) if d else (1 if kind == "FP8_ROW" else 0)
    p = torch.zeros(m, groups * w, dtype=torch.float64)
    p[:, :d] = a
    amax = p.view(m, groups, w).amax(2) if groups else p.new_zeros(m, 0)
    if kind == "MXFP8":
        e = torch.ceil(torch.log2((amax / 448).clamp_min(2.0 ** -200)))
        # log2 may be off by an ulp at a power of two
        e = torch.where(torch.pow(2.0, e - 1) >= amax / 448, e - 1, e)
        e = torch.where(torch.pow(2.0, e) < amax / 448, e + 1, e).clamp(-127, 127)
        e = torch.where(amax == 0, torch.zeros_like(e), e)
        s, value = (e + 127).to(torch.uint8), torch.pow(2.0, e)
    else:
        s = (amax / 448).float().clamp_min(2.0 ** -126)
        s = torch.where(amax == 0, torch.ones_like(s), s)
        value = s.double()
    spread = value.repeat_interleave(w, 1)[:, :d]
    return (s[:, 0] if kind == "FP8_ROW" else s), spread


def e4m3_codes(t):
    """Codes of fp64 values rounded to nearest even, saturated; NaN codes for what is not finite."""
    a = t.abs().clamp_max(448.0)
    a = torch.where(t.isfinite(), a, torch.zeros_like(a))
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -6)))
    q = torch.round(a / torch.pow(2.0, e - 3))          # 0..16 steps of the binade
    e = torch.where(q == 16, e + 1, e)
    q = torch.where(q == 16, torch.full_like(q, 8.0), q)
    code = torch.where(q < 8, q, q - 8 + 8 * (e + 7)).to(torch.uint8)
    code = torch.where(t.isfinite(), code, torch.full_like(code, 127))
    return code


def rms_norm(x, weight, eps, residual):
    h = x.double() if residual is None else x.double() + residual.double()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return (y if weight is None else y * weight.double()), h
