"""Plain 64-bit forms of the router and the experts, on the CPU, with the bounds that their arithmetic keeps to."""
import math

import torch

from tests import ops_reference as ref

DT = ref.DT


def random_experts(st, kind, down_kind, experts, i, k, n, seed):
    make = lambda kind, rows, cols, s: [ref.random_weight(st, kind, rows, cols, seed + 100 * s + e) for e in range(experts)]   # noqa: E731
    return make(kind, i, k, 0), make(kind, i, k, 1), make(down_kind, n, i, 2)


def route(x, router, top_k, score="softmax", bias=None, renormalize=True, scaling=1.0):
    z = x.double() @ router.double().t()
    s = torch.softmax(z, -1) if score == "softmax" else torch.sigmoid(z)
    key = z if bias is None else s + bias.double()
    key = torch.where(key.isnan(), torch.full_like(key, -torch.inf), key)
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :top_k]
    w = s.gather(-1, ids)
    if renormalize:
        w = w / w.sum(-1, keepdim=True)
    return w * scaling, ids.to(torch.int32)


def moe(x, lists, ids, weights, activation="silu", residual=None):
    """(result, bound on its error before the last rounding) for rows x [m, K]."""
    gate, up, down = lists
    x64 = x.double()
    n, i = down[0].shape
    k = x.shape[1]
    y, tol = torch.zeros(x.shape[0], n, dtype=torch.float64), torch.zeros(x.shape[0], n, dtype=torch.float64)
    step = 2.0 ** -23          # a matrix instruction may cut instead of round
    for e in range(len(gate)):
        t, j = torch.where(ids == e)
        if not len(t):
            continue
        g, u, d = (ref.weight_value(w[e]) for w in lists)
        a, b = x64[t] @ g.t(), x64[t] @ u.t()
        # K products each, then the scale's
        da, db = ((k + 4) * step * (x64[t].abs() @ w.abs().t()) for w in (g, u))
        act = ref.activate(activation, a)
        h = act * b
        # the activation's slope is at most 1.13 and it is evaluated to a few steps; h in two bf16 terms keeps 16 bits
        dh = 1.13 * da * (b.abs() + db) + act.abs() * db + h.abs() * (2.0 ** -17 + 8 * step)
        w = weights[t, j].double()[:, None]
        y.index_add_(0, t, w * (h @ d.t()))
        size = h.abs() @ d.abs().t()
        tol.index_add_(0, t, w.abs() * (dh @ d.abs().t() + (2 * i + ids.shape[1] + 8) * step * size))
    if residual is not None:
        y = y + residual.double()
        tol = tol + y.abs() * step
    return y, tol * 1.01


def check(got, want, tol):
    got = got.cpu()
    f = torch.finfo(got.dtype)
    allowed = tol + (want.abs() + tol) * f.eps / 2 + f.smallest_normal * f.eps / 2
    err = (got.double() - want).abs()
    # rounding to nearest turns what lies half a step or more above the largest number into an infinity
    edge = f.max + 2.0 ** math.floor(math.log2(f.max)) * f.eps / 2
    over = got.isinf() & (got.sign() == want.sign()) & (want.abs() + tol >= edge)
    bad = ~((err <= allowed) | (want.isnan() & got.isnan()) | over)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} results are off, worst {(err / allowed)[bad].max().item():.3g} of what is allowed, first at {bad.nonzero()[0].tolist()}"
