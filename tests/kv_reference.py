"""Plain 64-bit forms of the operators on the 8-bit cache, on the CPU: appending as its definition has it, one page and head at a
time, and attention with the bound that its arithmetic keeps to."""
import math

import torch

from tests import ops_reference as ref

DT = ref.DT


def random_cache(st, pages, heads, dim, block, seed, spread=2):
    """Codes of every finite value and scales of a few binades."""
    g = torch.Generator().manual_seed(seed)
    e = lambda: (torch.randint(0, 2 * spread + 1, (pages, heads), generator=g) + 120 - spread).to(torch.uint8).view(torch.float8_e8m0fnu)   # noqa: E731
    return st.QuantizedKvCache(ref.random_codes(g, pages, heads, block, dim), ref.random_codes(g, pages, heads, dim, block), e(), e())


def to(cache, dev):
    return type(cache)(*(t.to(dev) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))


def cpu(cache):
    return to(cache, "cpu")


def raw(t):
    return t.cpu().contiguous().view(torch.uint8)


def spans(tokens, lengths, starts, max_new):
    """(first row, rows, position of the first) of each sequence."""
    out, n = [], len(lengths)
    for s in range(n):
        a, b = (starts[s], starts[s + 1]) if starts is not None else (s * (tokens // n), (s + 1) * (tokens // n))
        out.append((a, min(b - a, max_new if max_new is not None else b - a), lengths[s] - (b - a)))
    return out


def least_power(amax):
    """The exponent of the smallest power of two at or above amax / 448, -127 at least."""
    if amax == 0:
        return -127
    m, e = math.frexp(amax)           # amax = m * 2^e, m in [1/2, 1): 448 = 0.875 * 2^9
    return max(-127, e - 9 + (1 if m > 0.875 else 0))


def nearest(v):
    """e4m3 values nearest to v (|v| <= 448), halves to even; NaN where v is not finite."""
    m, e = torch.frexp(v)
    step = torch.pow(2.0, (e.clamp_min(-5) - 4).double())
    q = torch.round(v / step) * step
    return torch.where(v.isfinite(), q, torch.full_like(q, math.nan))


def codes(v):
    """Codes of e4m3 values."""
    return v.float().to(torch.float8_e4m3fn)


def append(cache, k, v, table, lengths, starts=None, max_new=None):
    """The cache after the append, with codes as values."""
    pages, heads, block, dim = cache.k.shape
    kv, vv = ref.e4m3(cache.k), ref.e4m3(cache.v)
    ks, vs = (raw(t).to(torch.int64) - 127 for t in (cache.k_scale, cache.v_scale))
    ks, vs = ks.clone(), vs.clone()
    for s, (first, rows, pos) in enumerate(spans(k.shape[0], lengths, starts, max_new)):
        t = max(0, -pos)
        while t < rows:
            p = pos + t
            b, lo = p // block, p % block
            n = min(block - lo, rows - t)
            page = int(table[s][b]) if b < len(table[s]) else -1
            if 0 <= page < pages:
                for x, c, e in ((k, kv, ks), (v, vv.transpose(2, 3), vs)):
                    for h in range(heads):
                        new = x[first + t:first + t + n, h].double()
                        fin = new[new.isfinite()]
                        was = int(e[page, h]) if lo else -127
                        now = max(was, least_power(fin.abs().max().item() if fin.numel() else 0.0))
                        c[page, h, :lo] = nearest(c[page, h, :lo] * 2.0 ** (was - now))
                        c[page, h, lo:lo + n] = nearest(new * 2.0 ** -now)
                        e[page, h] = now
            t += n
    return kv, vv, ks, vs


def attention(q, cache, table, lengths, starts=None, max_new=None, scale=None, causal=True, window=None):
    """(result, bound on its error before the last rounding); rows of no sequence are 0."""
    pages, heads, block, dim = cache.k.shape
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    group = q.shape[1] // heads
    kv = ref.e4m3(cache.k) * ref.e8m0(cache.k_scale)[:, :, None, None]
    vv = (ref.e4m3(cache.v) * ref.e8m0(cache.v_scale)[:, :, None, None]).transpose(2, 3)
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for s, (first, rows, pos) in enumerate(spans(q.shape[0], lengths, starts, max_new)):
        n = min(max(lengths[s], 0), block * len(table[s]))
        ids = torch.tensor([int(x) for x in table[s][:-(-n // block)]], dtype=torch.int64)
        there = ((ids >= 0) & (ids < pages)).repeat_interleave(block)[:n]
        ids = ids.clamp(0, pages - 1)
        K = kv[ids].permute(1, 0, 2, 3).reshape(heads, -1, dim)[:, :n]
        V = vv[ids].permute(1, 0, 2, 3).reshape(heads, -1, dim)[:, :n]
        at = torch.arange(n)
        for t in range(rows):
            see = there.clone()
            if causal:
                see &= at <= pos + t
                if window:
                    see &= at > pos + t - window
            if not see.any():
                continue
            for h in range(q.shape[1]):
                x = q[first + t, h].double()
                k, v = K[h // group][see], V[h // group][see]
                z = (k @ x) * scale
                p = torch.exp(z - z.max())
                y = (p @ v) / p.sum()
                # a score: dim products summed in fp32, then a few roundings of its own; numerators: fp16's half step, the hardware's
                # exponential and a smallest step 30 binades below the largest; sums of n terms in fp32, numerator and denominator
                ds = ((k.abs() @ x.abs()) * scale).max() * (dim + 4) * 2.0 ** -24 + z.abs().max() * 2.0 ** -21
                m = len(z)
                size = (p @ v.abs()) / p.sum()
                rel = 2.0 ** -11 + 2 * ds + 2.0 ** -22 + 2 * (m + 64) * 2.0 ** -24
                out[first + t, h] = y
                tol[first + t, h] = size * rel * 1.01 + v.abs().max(0).values * (m * 2.0 ** -30 / p.sum() + 2.0 ** -32)
    return out, tol


def check(got, want, tol):
    """|got - want| within tol and the rounding to got's type (half a step, or half its smallest number)."""
    got = got.cpu()
    f = torch.finfo(got.dtype)
    allowed = tol + (want.abs() + tol) * f.eps / 2 + f.smallest_normal * f.eps / 2
    err = (got.double() - want).abs()
    bad = ~((err <= allowed) | (want.isnan() & got.isnan()))
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} results are off, worst {(err / allowed)[bad].max().item():.3g} of what is "
                           f"allowed; first at {bad.nonzero()[0].tolist()}: {got[bad][0].item()} for {want[bad][0].item()}")
