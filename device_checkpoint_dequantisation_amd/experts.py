"""Mixtures of experts whose weights stay as the checkpoint stores them: the router (st_moe_route) and the experts (st_moe).

    q = sd.load_quantized(names, copy=True)                     # each expert's gate, up and down
    experts = MoeExperts([q[f"experts.{e}.gate.weight"] for e in range(128)],
                         [q[f"experts.{e}.up.weight"] for e in range(128)],
                         [q[f"experts.{e}.down.weight"] for e in range(128)])
    weights, ids = moe_route(x, router, top_k=8)                # x [tokens, K], router [128, K]
    h = moe(x, experts, ids, weights, residual=h)

They run on the current stream (or ``stream``), allocate with torch, synchronise nothing and can be captured into a HIP
graph.  They have no backward pass."""
from __future__ import annotations

import bisect
import ctypes as C

import torch

from ._lib import MoeArgs, MoeRouteArgs, OUT_DTYPES, check, lib
from .ops import _ACT, _KIND, _TORCH, _TYPE, ACTIVATIONS, _check_weight, _launch, _on_device, _overlaps, _rows, _span

SCORES = ("softmax", "sigmoid")     # st_route_score codes 0, 1
MAX_TOP_K = 32                      # of moe
MAX_EXPERTS = 1024                  # of moe_route


class MoeExperts:
    """The experts of one layer: lists of :class:`QuantizedWeight` ``gate`` [I, K], ``up`` [I, K] and ``down`` [N, I], one of each
    for an expert, all on one GPU.  Gates and ups have one kind, downs one (another, if so).  The weights are used where they are: the object
    holds them and a table of their addresses (72 bytes an expert).  Its construction copies that table to the GPU and waits for it."""

    def __init__(self, gate, up, down):
        who = "MoeExperts"
        gate, up, down = list(gate), list(up), list(down)
        if not (gate and len(gate) == len(up) == len(down)):
            raise ValueError(f"{who}: {len(gate)} gates, {len(up)} ups and {len(down)} downs; one of each is needed for every expert")
        if len(gate) > 16384:
            raise ValueError(f"{who}: {len(gate)} experts; at most 16384 are possible")
        self.shape = _check_weight(gate[0], who)
        self.width, self.kind, self.down_kind = _check_weight(down[0], who)[0], gate[0].kind, down[0].kind
        i, k = self.shape
        for e, three in enumerate(zip(gate, up, down)):
            for w, shape, kind, name in zip(three, ((i, k), (i, k), (self.width, i)), (self.kind, self.kind, self.down_kind), ("gate", "up", "down")):
                if _check_weight(w, who) != shape or w.kind != kind:
                    raise ValueError(f"{who}: expert {e}'s {name} is {w.kind} {tuple(w.shape)}; {kind} {shape} is needed")
        if not (i and k):
            raise ValueError(f"{who}: experts of [{i}, {k}]")
        self.device = gate[0].data.device
        self.weights = tuple(zip(gate, up, down))
        table = []
        for three in self.weights:
            for w in three:
                _on_device(self.device, (w.data, w.scale, w.scale2), who)
                for t, n in ((w.scale, 4 if w.kind.startswith("FP8") else 1), (w.scale2, 4)):
                    if t is not None and t.data_ptr() % n:
                        raise ValueError(f"{who}: an fp32 scale is not 4-byte aligned")
                table.append([w.data.data_ptr(), w.scale.data_ptr(), 0 if w.scale2 is None else w.scale2.data_ptr()])
        self.table = torch.tensor(table, dtype=torch.int64).to(self.device)
        # what they take: disjoint ranges of bytes in rising order, and a tensor of each allocation
        held = [t for three in self.weights for w in three for t in (w.data, w.scale, w.scale2) if t is not None and t.numel()]
        self._spans = []
        for a, b in sorted(map(_span, held)):
            if self._spans and a <= self._spans[-1][1]:
                self._spans[-1] = (self._spans[-1][0], max(b, self._spans[-1][1]))
            else:
                self._spans.append((a, b))
        self._held = list({t.untyped_storage().data_ptr(): t for t in held}.values())

    def _overlaps(self, t) -> bool:
        a, b = _span(t)
        i = bisect.bisect_left(self._spans, (b,)) - 1        # the last range that begins before t's end
        return t.numel() > 0 and i >= 0 and self._spans[i][1] > a

    def __len__(self) -> int:
        return len(self.weights)


def moe_route(x, router, top_k: int, score: str = "softmax", bias=None, renormalize: bool = True, scaling: float = 1.0, stream=None):
    """The ``top_k`` experts of each row of ``x`` [..., K] and their weights: (weights fp32 [..., top_k], ids int32 [..., top_k]).  A call
    takes fewer than 2**17 rows.

    Scores are softmax(x @ router.T) over the experts of ``router`` [experts, K], or its elements' logistic function ("sigmoid"); x and
    the router are bf16, fp16 or fp32, sums are 64-bit.  The experts with the largest scores are chosen, with a ``bias`` (fp32
    [experts]) those with the largest score + bias; they come in falling order, equal ones by their number, NaN last.  A weight is the
    expert's score without the bias, divided by the sum of the chosen ones' if ``renormalize``, times ``scaling``."""
    who = "moe_route"
    if not (x.dtype in _TYPE and x.dim() >= 1):
        raise ValueError(f"{who}: x is {x.dtype} {tuple(x.shape)}; bf16, fp16 or fp32 rows are needed")
    k = x.shape[-1]
    if not (router.dtype in _TYPE and router.dim() == 2 and router.shape[1] == k and (k <= 1 or router.stride(1) == 1)
            and (router.shape[0] <= 1 or router.stride(0) >= k)):
        raise ValueError(f"{who}: router {router.dtype} {tuple(router.shape)}, strides {router.stride()}, against x {tuple(x.shape)}")
    experts = router.shape[0]
    if not (isinstance(top_k, int) and 1 <= top_k <= experts <= MAX_EXPERTS):
        raise ValueError(f"{who}: {top_k!r} of {experts} experts; 1 to all of at most {MAX_EXPERTS} are needed")
    if score not in SCORES:
        raise ValueError(f"{who}: unknown score {score!r}; one of {SCORES}")
    if bias is not None and not (bias.dtype == torch.float32 and tuple(bias.shape) == (experts,) and (experts <= 1 or bias.stride(0) == 1)):
        raise ValueError(f"{who}: bias {bias.dtype} {tuple(bias.shape)}, strides {bias.stride()}; fp32 [{experts}] is needed")
    _on_device(x.device, (x, router, bias), who)
    x2, pitch = _rows(x, k, "x", who)
    m = x2.shape[0]
    weights = x.new_empty((*x.shape[:-1], top_k), dtype=torch.float32)
    ids = x.new_empty((*x.shape[:-1], top_k), dtype=torch.int32)
    if m == 0:
        return weights, ids
    work = x.new_empty(m * experts, dtype=torch.float64)
    args = MoeRouteArgs(x2.data_ptr(), router.data_ptr(), None if bias is None else bias.data_ptr(), weights.data_ptr(), ids.data_ptr(),
                        work.data_ptr(), m * experts * 8, m, k, pitch, router.stride(0), float(scaling), experts, top_k,
                        SCORES.index(score), int(bool(renormalize)), _TYPE[x.dtype], _TYPE[router.dtype])
    _launch(lib().st_moe_route, args, x.device, stream, (x2, router, bias, weights, ids, work), who)
    return weights, ids


def moe(x, experts: MoeExperts, ids, weights, activation: str | None = "silu", residual=None, out_dtype: str | None = None, out=None,
        stream=None):
    """sum_j weights[..., j] * down(act(gate(x)) * up(x)) of expert ids[..., j], + residual, for few rows ``x`` [..., K] in bf16 or fp16.

    ``ids`` int32 and ``weights`` fp32 [..., top_k], as :func:`moe_route` gives them; an id that is no expert (of another GPU, say)
    adds nothing, one that a row has twice counts twice.  ``activation`` is one of :func:`linear`'s, ``residual`` [..., N] bf16,
    fp16 or fp32; the result has ``out_dtype`` (default x's type) or goes to ``out``, which may be ``residual`` itself.

    Each chosen expert's weights are read once for up to 16 of its rows, or 64 where experts have many on average, and again, from cache or memory, for as
    many more: a batch most of whose rows share one expert meets its weights many times.  From some 300 to 500 rows an expert on,
    :func:`linear` on each expert's rows is the faster way.  The weights' exact values enter, sums are fp32; act(gate) * up enters the down product with 16
    significant bits."""
    who = "moe"
    if not isinstance(experts, MoeExperts):
        raise ValueError(f"{who}: experts is a {type(experts).__name__}; MoeExperts are needed")
    i, k = experts.shape
    n = experts.width
    if not (x.dtype in (torch.bfloat16, torch.float16) and x.dim() >= 1 and x.shape[-1] == k):
        raise ValueError(f"{who}: x is {x.dtype} {tuple(x.shape)}; bf16 or fp16 rows of {k} are needed")
    lead = x.shape[:-1]
    if not (ids.dtype == torch.int32 and ids.dim() == x.dim() and ids.shape[:-1] == lead and ids.is_contiguous()):
        raise ValueError(f"{who}: ids {ids.dtype} {tuple(ids.shape)}, strides {ids.stride()}; contiguous int32 {(*lead, 'top_k')} are needed")
    top = ids.shape[-1]
    if not 1 <= top <= MAX_TOP_K:
        raise ValueError(f"{who}: {top} experts a row; 1 to {MAX_TOP_K} are needed")
    if not (weights.dtype == torch.float32 and weights.shape == ids.shape and weights.is_contiguous()):
        raise ValueError(f"{who}: weights {weights.dtype} {tuple(weights.shape)}, strides {weights.stride()}; contiguous fp32 {tuple(ids.shape)} are needed")
    if activation not in _ACT:
        raise ValueError(f"{who}: unknown activation {activation!r}; one of {ACTIVATIONS}")
    device = x.device
    _on_device(device, (x, ids, weights, experts.table, residual, out), who)
    x2, x_pitch = _rows(x, k, "x", who)
    m = x2.shape[0]
    shape = (*lead, n)
    r2, r_pitch = None, 0
    if residual is not None:
        if not (residual.dtype in _TYPE and tuple(residual.shape) == shape):
            raise ValueError(f"{who}: residual {residual.dtype} {tuple(residual.shape)}; {shape} is needed")
        r2, r_pitch = _rows(residual, n, "residual", who)
    if out is None:
        if out_dtype is not None and out_dtype not in _TORCH:
            raise ValueError(f"{who}: unknown out_dtype {out_dtype!r}; one of {OUT_DTYPES}")
        out = x.new_empty(shape, dtype=_TORCH[out_dtype] if out_dtype else x.dtype)
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
        if experts._overlaps(o2) or any(_overlaps(o2, t) for t in (x2, ids, weights, experts.table, None if same else r2)):
            raise ValueError(f"{who}: out overlaps an input")
    if m == 0 or n == 0:
        return out
    args = MoeArgs(x2.data_ptr(), ids.data_ptr(), weights.data_ptr(), experts.table.data_ptr(), None if r2 is None else r2.data_ptr(),
                   o2.data_ptr(), None, 0, m, k, i, n, x_pitch, r_pitch, o2.stride(0), len(experts.weights), top, _TYPE[x.dtype],
                   _KIND[experts.kind], _KIND[experts.down_kind], _ACT[activation], 0 if r2 is None else _TYPE[r2.dtype], _TYPE[o2.dtype])
    need = C.c_uint64()
    check(lib().st_moe_workspace_bytes(C.byref(args), C.byref(need)), who)
    work = x.new_empty(need.value, dtype=torch.uint8)
    args.workspace, args.workspace_bytes = work.data_ptr(), need.value
    # (on another stream the experts' weights are in use there as well)
    held = () if stream is None else experts._held
    _launch(lib().st_moe, args, device, stream, (x2, ids, weights, experts.table, r2, o2, work, *held), who)
    return out
