"""Cases of the operators of a decoding step on a quantised checkpoint: ``moe_route`` (the router's scores and the
choice of experts), ``moe`` (the experts of a mixture on their stored weights), ``kv_append`` (new keys and values into a cache
of 8 bits with a scale for each block of tokens and head) and ``kv_attention`` (attention over that cache).  ``own`` chooses
between the framework's kernels and the plain form written here.

Hidden sizes are those of the synthetic checkpoints in synth/configs.py (block FP8: 4096, packed fp4: 5120, narrow ones 320 and
1280); numbers of experts, heads and tokens are generic.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
KINDS = ("FP8_TENSOR", "FP8_BLOCK128", "NVFP4", "MXFP8", "MXFP4")


def _route(name, t, k, e, top, score, bias, x, router):
    return {"name": name, "op": "route", "t": t, "k": k, "e": e, "top": top, "score": score, "bias": bias, "x": x, "router": router}


def _moe(name, t, k, i, e, top, weight, x, residual):
    return {"name": name, "op": "moe", "t": t, "k": k, "i": i, "e": e, "top": top, "weight": weight, "x": x, "residual": residual}


def _attn(name, b, new, least, most, heads, group, d, block, x, window):
    """b sequences of least..most tokens, the last ``new`` (or up to as many, where it is negative) of them queries."""
    return {"name": name, "op": "attention", "b": b, "new": new, "least": least, "most": most, "heads": heads, "group": group, "d": d,
            "block": block, "x": x, "window": window}


def _append(name, b, new, least, most, heads, d, block, x):
    return {"name": name, "op": "append", "b": b, "new": new, "least": least, "most": most, "heads": heads, "d": d, "block": block, "x": x}


def listed():
    return [
        # one token's choice of 8 experts of 128: latency
        _route("route one token", 1, 4096, 128, 8, "softmax", False, "bf16", "bf16"),
        # a ragged prefill chunk, sigmoid scores with a correction of the choice, the router kept in fp32
        _route("route ragged 777", 777, 5120, 256, 6, "sigmoid", True, "bf16", "f32"),
        # single-token decoding through packed-fp4 experts, added to the residual stream: the chosen experts' bytes
        _moe("experts nvfp4 one token", 1, 5120, 1280, 64, 8, "NVFP4", "bf16", True),
        # a decoding batch of 8 through block-FP8 experts, few of which meet twice
        _moe("experts block fp8 batch of 8", 8, 4096, 1280, 128, 8, "FP8_BLOCK128", "bf16", False),
        # a decoding batch of 40 in fp16, MXFP4 experts that all have some tokens
        _moe("experts mxfp4 batch of 40", 40, 5120, 1280, 32, 4, "MXFP4", "f16", True),
        # a large batch: every expert has about 20 tokens, unevenly
        _moe("experts block fp8 batch of 320", 320, 4096, 1280, 128, 8, "FP8_BLOCK128", "bf16", False),
        # four draft tokens of three short sequences are checked, small heads, small pages, a sliding window: latency
        _attn("attention 3 x 4 drafts, window", 3, 4, 700, 1000, 8, 4, 64, 16, "f16", 512),
        # a decoding batch of ragged lengths
        _attn("attention batch of 48, ragged", 48, 1, 100, 8192, 8, 4, 128, 64, "bf16", 0),
        # two long contexts, five query heads to one of the cache: split over the cache's length
        _attn("attention 2 x 131071", 2, 1, 131071, 131071, 8, 5, 128, 128, "bf16", 0),
        # chunks of prompts of which a part is in the cache already: bound by the matrix instructions
        _attn("attention prefill chunks", 4, -2048, 2100, 6200, 8, 4, 128, 64, "bf16", 0),
        # one new token for each of 48 sequences: latency
        _append("append batch of 48", 48, 1, 100, 2000, 8, 128, 64, "bf16"),
        # prompts' chunks, one after the other in one packed batch
        _append("append prefill chunks", 6, -2048, 2100, 2500, 8, 128, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "attention", "attention", "append"])
    if op == "route":
        e = _log(rng, 4, 512)
        c = _route("", _log(rng, 1, 777), _log(rng, 64, 5120), e, rng.randint(1, min(8, e)), rng.choice(["softmax", "sigmoid"]),
                   rng.random() < 0.5, rng.choice(["bf16", "f16"]), rng.choice(["bf16", "f32"]))
        while c["t"] * c["e"] * c["k"] > 1e9:
            c["t"] //= 2
    elif op == "moe":
        weight = rng.choice(KINDS)
        step = {"NVFP4": 16, "MXFP8": 32, "MXFP4": 32}.get(weight) or rng.choice([1, 16])
        k = max(1, _log(rng, 128, 5120) // step) * step
        i = max(1, _log(rng, 64, 2048) // step) * step
        e = _log(rng, 4, 128)
        while e * k * i > 7e8:
            e //= 2
        c = _moe("", _log(rng, 1, 320), k, i, e, rng.randint(1, min(8, e)), weight, rng.choice(["bf16", "f16"]), rng.random() < 0.5)
    else:
        b, d = _log(rng, 1, 64), rng.choice([64, 128, 128, 256])
        block, x, heads = rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "f16"]), _log(rng, 1, 16)
        new = rng.choice([1, 1, rng.randint(2, 8), -_log(rng, 16, 2048)])
        most = max(abs(new), _log(rng, 1, 131072 if op == "attention" else 4096))
        while b > 1 and b * most * heads * d > 2.6e8:
            b //= 2
        while most * heads * d > 2.6e8:
            heads = max(1, heads // 2)
        least = max(abs(new), _log(rng, 1, most))
        if op == "append":
            while b > 1 and b * abs(new) > 8192:
                b //= 2
            c = _append("", b, new, least, most, heads, d, block, x)
        else:
            group = rng.choice([1, 2, 4, 5, 7, 8, 16])
            while b > 1 and b * abs(new) * most * heads * group * d * 4 > 4e11:
                b //= 2
            while new < -16 and abs(new) * most * heads * group * d * 4 > 4e11:
                new //= 2
            c = _attn("", b, new, least, most, heads, group, d, block, x, rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ inputs

def _pow2(e):
    """2^e for whole e, from the fields of a 64-bit number (the GPU's exp2 and ldexp are off by a last bit)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _e8m0(e):
    return (e + 127).clamp(0, 254).to(torch.uint8).view(torch.float8_e8m0fnu)


def _least_power(a):
    """Exponents of the smallest powers of two at or above a (a > 0)."""
    f, e = torch.frexp(a)
    return e - (f == 0.5).to(e.dtype)


def _fp4(v):
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    c = torch.bucketize(v.abs(), mid).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _weight(kind, n, k, g):
    """A weight of N(0, 0.02) values quantised as such checkpoints are: (data, scale, global scale)."""
    w = torch.randn(n, k, generator=g, device=DEV) * 0.02
    if kind == "FP8_TENSOR":
        s = w.abs().amax() / E4M3_MAX
        return (w / s).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s, None
    if kind == "FP8_BLOCK128":
        gn, gk = -(-n // 128), -(-k // 128)
        p = torch.nn.functional.pad(w, (0, gk * 128 - k, 0, gn * 128 - n)).view(gn, 128, gk, 128)
        s = (p.abs().amax((1, 3)) / E4M3_MAX).clamp_min(1e-12)
        p = (p / s[:, None, :, None]).view(gn * 128, gk * 128)[:n, :k].clamp(-E4M3_MAX, E4M3_MAX)
        return p.to(torch.float8_e4m3fn).contiguous(), s, None
    if kind == "NVFP4":
        b = w.view(n, k // 16, 16)
        s2 = w.abs().amax() / (6.0 * E4M3_MAX)
        s = (b.abs().amax(2) / (6.0 * s2)).clamp(2.0 ** -6, E4M3_MAX).to(torch.float8_e4m3fn)
        return _fp4((b / (s.float() * s2)[:, :, None]).view(n, k)), s, s2
    b = w.view(n, k // 32, 32)
    e = _least_power(b.abs().amax(2).clamp_min(1e-20) / (6.0 if kind == "MXFP4" else E4M3_MAX))
    v = (b / _pow2(e).float()[:, :, None]).view(n, k)
    return (_fp4(v) if kind == "MXFP4" else v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)), _e8m0(e), None


def _stream(rows, k, g):
    """Normalised rows of a residual stream: a few channels are large."""
    return torch.randn(rows, k, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(k, generator=g, device=DEV))


def _cache(c, lengths, g):
    """A cache of pages in random order that holds the sequences' tokens: keys with large channels, values without."""
    h, d, block = c["heads"], c["d"], c["block"]
    per = -(-max(lengths) // block)
    need = [-(-n // block) for n in lengths]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table, at = torch.zeros(len(lengths), per, dtype=torch.int32, device=DEV), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    ch = torch.exp(0.5 * torch.randn(h, 1, d, generator=g, device=DEV))
    out = []
    for which in "kv":
        x = torch.randn(pages, h, block, d, generator=g, device=DEV)
        if which == "k":
            x *= ch
        e = _least_power(x.abs().amax((2, 3)) / E4M3_MAX)
        x = (x * _pow2(-e).float()[:, :, None, None]).to(torch.float8_e4m3fn)
        out += [x if which == "k" else x.transpose(2, 3).contiguous(), _e8m0(e)]
    return out, table


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    dt = DT[case["x"]]
    if case["op"] == "route":
        t, k, e = case["t"], case["k"], case["e"]
        s["xd"] = _stream(t, k, g).to(dt)
        s["w"] = (torch.randn(e, k, generator=g, device=DEV) / math.sqrt(k)).to(DT[case["router"]])
        s["b"] = torch.randn(e, generator=g, device=DEV) * 0.1 if case["bias"] else None
        return s
    if case["op"] == "moe":
        t, k, i, e, top = case["t"], case["k"], case["i"], case["e"], case["top"]
        s["xd"] = _stream(t, k, g).to(dt)
        # some experts are liked better than others
        z = torch.randn(t, e, generator=g, device=DEV) + 0.7 * torch.randn(e, generator=g, device=DEV)
        p, ids = torch.softmax(z, 1).topk(top, 1)
        s["p"], s["ids"] = (p / p.sum(1, keepdim=True)).contiguous(), ids.to(torch.int32).contiguous()
        s["r"] = torch.randn(t, k, generator=g, device=DEV).to(dt) if case["residual"] else None
        s["experts"] = [[_weight(case["weight"], *nk, g) for _ in range(e)] for nk in ((i, k), (i, k), (k, i))]
        if own:
            import device_checkpoint_dequantisation_amd as st
            lists = [[st.QuantizedWeight(f"{j}", case["weight"], nk, *w) for j, w in enumerate(ws)]
                     for ws, nk in zip(s["experts"], ((i, k), (i, k), (k, i)))]
            s["handle"] = st.MoeExperts(*lists)
        return s
    # lengths and numbers of new tokens spread over their ranges, in an order of the seed's
    b, new = case["b"], case["new"]
    steps = [j / max(1, b - 1) if b > 1 else 1.0 for j in range(b)]
    mix = torch.rand(2, b, generator=g, device=DEV).argsort(1).tolist()
    lengths = [case["least"] + int(steps[j] * (case["most"] - case["least"])) for j in mix[0]]
    count = [new if new > 0 else max(1, int(steps[j] * -new)) for j in mix[1]]
    s["len_list"], s["new_list"] = lengths, count
    (s["kc"], s["ks"], s["vc"], s["vs"]), s["table"] = _cache(case, lengths, g)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    n = sum(count)
    ends = [0]
    for a in count:
        ends.append(ends[-1] + a)
    s["starts"] = torch.tensor(ends, dtype=torch.int32, device=DEV) if new < 0 else None
    h, d = case["heads"], case["d"]
    if case["op"] == "append":
        s["knew"] = (torch.randn(n, h, d, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(h, d, generator=g, device=DEV))).to(dt)
        s["vnew"] = torch.randn(n, h, d, generator=g, device=DEV).to(dt)
    else:
        s["q"] = (1.5 * torch.randn(n, h * case["group"], d, generator=g, device=DEV)).to(dt)
    if own:
        import device_checkpoint_dequantisation_amd as st
        s["handle"] = st.QuantizedKvCache(s["kc"], s["vc"], s["ks"], s["vs"])
    return s


# ------------------------------------------------------------------------------------------------ plain form

def _scale_e8m0(s):
    c = s.view(torch.uint8).to(torch.int32)
    return torch.where(c == 0, torch.full_like(c, 0x00400000), c << 23).view(torch.float32)


def _nibbles(d):
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=d.device)
    return t[torch.stack((d & 15, d >> 4), 2).flatten(1).to(torch.int32)]


def _plain_weight(kind, w, n, k):
    d, s, s2 = w
    if kind == "FP8_TENSOR":
        return d.float() * s
    if kind == "FP8_BLOCK128":
        return d.float() * s.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    if kind == "NVFP4":
        return _nibbles(d) * s.float().repeat_interleave(16, 1) * s2
    return (d.float() if kind == "MXFP8" else _nibbles(d)) * _scale_e8m0(s).repeat_interleave(32, 1)


def _plain_route(c):
    z = c["xd"].double() @ c["w"].double().t()      # 64 bits: choices between near scores
    s = torch.softmax(z, 1) if c["score"] == "softmax" else 1 / (1 + torch.exp(-z))
    key = z if c["b"] is None else s + c["b"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["top"]]
    w = s.gather(1, ids)
    return (w / w.sum(1, keepdim=True) * 2.5).float(), ids.to(torch.int32)


def _plain_moe(c):
    t, k, i, e, top, kind = c["t"], c["k"], c["i"], c["e"], c["top"], c["weight"]
    x = c["xd"].float()
    y = torch.zeros(t, k, device=DEV) if c["r"] is None else c["r"].float()
    for j in range(e):
        rows, slot = torch.where(c["ids"] == j)
        if rows.numel() == 0:
            continue
        v = x[rows]
        a = v @ _plain_weight(kind, c["experts"][0][j], i, k).t()
        h = a / (1 + torch.exp(-a)) * (v @ _plain_weight(kind, c["experts"][1][j], i, k).t())
        y.index_add_(0, rows, h @ _plain_weight(kind, c["experts"][2][j], k, i).t() * c["p"][rows, slot][:, None])
    return y.to(DT[c["x"]])


def _plain_attention(c):
    h, g, d, block = c["heads"], c["group"], c["d"], c["block"]
    out, at = torch.empty_like(c["q"]), 0
    for b, (n, new) in enumerate(zip(c["len_list"], c["new_list"])):
        pages = c["table"][b, :-(-n // block)].long()
        k = (c["kc"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * _scale_e8m0(c["ks"])[pages][:, :, None, None])
        v = (c["vc"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * _scale_e8m0(c["vs"])[pages][:, :, None, None])
        k = k.permute(1, 0, 2, 3).reshape(h, -1, d)[:, :n]
        v = v.permute(1, 0, 3, 2).reshape(h, -1, d)[:, :n]
        q = c["q"][at:at + new].float().view(new, h, g, d).permute(1, 2, 0, 3).reshape(h, g * new, d)
        s = torch.bmm(q, k.transpose(1, 2).contiguous()).view(h, g, new, n) / math.sqrt(d)
        pos = torch.arange(n - new, n, device=DEV)[:, None] - torch.arange(n, device=DEV)[None, :]
        gone = pos < 0 if not c["window"] else (pos < 0) | (pos >= c["window"])
        s.masked_fill_(gone, -math.inf)
        p = torch.exp(s - s.amax(3, keepdim=True))
        p /= p.sum(3, keepdim=True)
        o = torch.bmm(p.view(h, g * new, n), v).view(h, g, new, d)
        out[at:at + new] = o.permute(2, 0, 1, 3).reshape(new, h * g, d).to(out.dtype)
        at += new
    return out


def _plain_append(c):
    h, d, block = c["heads"], c["d"], c["block"]
    at = 0
    for b, (n, new) in enumerate(zip(c["len_list"], c["new_list"])):
        first, last = (n - new) // block, (n - 1) // block
        pages = c["table"][b, first:last + 1].long()
        pos = torch.arange(first * block, (last + 1) * block, device=DEV)
        fresh = ((pos >= n - new) & (pos < n)).view(-1, 1, block, 1)
        old = (pos < n - new).view(-1, 1, block, 1)
        for x, codes, scale, flip in ((c["knew"], c["kc"], c["ks"], False), (c["vnew"], c["vc"], c["vs"], True)):
            was = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
            if flip:
                was = was.transpose(2, 3)
            v = torch.zeros(pos.numel(), h, d, device=DEV)
            v[n - new - first * block:n - first * block] = x[at:at + new].float()
            v = v.view(-1, block, h, d).transpose(1, 2)
            a = v.abs().amax((2, 3))
            e = torch.where(a == 0, torch.full_like(a, -127).int(), _least_power(a / E4M3_MAX).clamp(-127, 127).int())
            had = scale.view(torch.uint8)[pages].int() - 127
            had[1:] = -127
            if (n - new) % block == 0:
                had[:1] = -127
            e = torch.maximum(e, had)
            up = _pow2(-e).float()[:, :, None, None]
            keep = _pow2(had - e).float()[:, :, None, None]
            new_codes = torch.where(fresh, v * up, torch.where(old, was * keep, was)).to(torch.float8_e4m3fn)
            codes.view(torch.uint8)[pages] = (new_codes.transpose(2, 3) if flip else new_codes).contiguous().view(torch.uint8)
            scale.view(torch.uint8)[pages] = (e + 127).to(torch.uint8)
        at += new
    return c["kc"], c["vc"], c["ks"], c["vs"]


_PLAIN = {"route": _plain_route, "moe": _plain_moe, "attention": _plain_attention, "append": _plain_append}


# ------------------------------------------------------------------------------------------------ the framework's calls

def _calls(c):
    import device_checkpoint_dequantisation_amd as st
    if c["op"] == "route":
        return st.moe_route(c["xd"], c["w"], c["top"], score=c["score"], bias=c["b"], scaling=2.5)
    if c["op"] == "moe":
        return st.moe(c["xd"], c["handle"], c["ids"], c["p"], residual=c["r"])
    most = max(c["new_list"]) if c["new"] < 0 else None
    if c["op"] == "attention":
        return st.kv_attention(c["q"], c["handle"], c["table"], c["lengths"], starts=c["starts"], max_new=most,
                               window=c["window"] or None)
    st.kv_append(c["handle"], c["knew"], c["vnew"], c["table"], c["lengths"], starts=c["starts"], max_new=most)
    return c["kc"], c["vc"], c["ks"], c["vs"]


def run(state):
    return _calls(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------------------ what it cannot do without

def _weight_bytes(kind, n, k):
    if kind in ("FP8_TENSOR", "FP8_BLOCK128"):
        return n * k + (4 if kind == "FP8_TENSOR" else 4 * -(-n // 128) * -(-k // 128))
    if kind == "NVFP4":
        return n * k // 2 + n * (k // 16) + 4
    return n * k // (1 if kind == "MXFP8" else 2) + n * (k // 32)


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "route":
        t, k, e, top = case["t"], case["k"], case["e"], case["top"]
        return {"bytes": t * k * 2 + e * k * size[case["router"]] + 8 * t * top + (4 * e if case["bias"] else 0), "flops": 2 * t * e * k}
    if case["op"] == "moe":
        t, k, i, e, top = case["t"], case["k"], case["i"], case["e"], case["top"]
        # experts that have a token, if all were liked alike
        met = max(min(e, top), e * (1 - (1 - top / e) ** t))
        w = 2 * _weight_bytes(case["weight"], i, k) + _weight_bytes(case["weight"], k, i)
        return {"bytes": int(met * w) + t * k * 2 * (3 if case["residual"] else 2) + 8 * t * top, "flops": 6 * t * top * k * i}
    b, new, h, d = case["b"], case["new"], case["heads"], case["d"]
    count = b * new if new > 0 else b * (1 - new) // 2
    if case["op"] == "append":
        return {"bytes": count * h * d * 2 * 3, "flops": 4 * count * h * d}
    mean = (case["least"] + case["most"]) / 2
    seen = min(mean, case["window"] + count / b) if case["window"] else mean
    pairs = min(mean - count / b / 2, case["window"] or mean)
    return {"bytes": int(b * seen * h * d * 2) + count * h * case["group"] * d * 4, "flops": int(4 * count * pairs * h * case["group"] * d)}


# ------------------------------------------------------------------------------------------------ 64-bit values

def _bits8(d):
    """e4m3 codes to their values from the fields: (-1)^s 2^(e-7) (1 + f/8), or 2^-6 f/8 where e is 0."""
    c = d.view(torch.uint8).to(torch.int64)
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * _pow2(e - 10))
    return torch.where(c >= 128, -v, v)


def _bits4(d):
    c = d.to(torch.int64)
    c = torch.stack((c % 16, c // 16), -1).reshape(d.shape[0], -1)
    e, f = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, f / 2, (2 + f) * _pow2(e - 2))
    return torch.where(c >= 8, -v, v)


def _spread(s, like, per_row, per_col):
    i = torch.arange(like.shape[0], device=like.device) // per_row
    j = torch.arange(like.shape[1], device=like.device) // per_col
    return s[i][:, j]


def _exponents(s):
    return s.view(torch.uint8).to(torch.int64) - 127


def _value(kind, w):
    d, s, s2 = w
    v = _bits4(d) if kind in ("NVFP4", "MXFP4") else _bits8(d)
    if kind == "FP8_TENSOR":
        return v.mul_(s.double())
    if kind == "FP8_BLOCK128":
        return v.mul_(_spread(s.double(), v, 128, 128))
    if kind == "NVFP4":
        return v.mul_(_spread(_bits8(s), v, 1, 16)).mul_(s2.double())
    return v.mul_(_spread(_pow2(_exponents(s)), v, 1, 32))


def _exact_route(c):
    x, w = c["xd"].double(), c["w"].double()
    z = torch.stack([(row * w).sum(1) for row in x])
    p = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.exp(torch.log_softmax(z, 1))
    left = z.clone() if c["b"] is None else p + c["b"].double()
    ids, got = [], []
    for _ in range(c["top"]):
        best = left.max(1, keepdim=True).values
        j = torch.argmax((left == best).to(torch.int8), 1, keepdim=True)      # the first of equals
        ids.append(j)
        got.append(p.gather(1, j))
        left = left.scatter(1, j, -math.inf)
    got = torch.cat(got, 1)
    return got * (2.5 / got.sum(1, keepdim=True)), torch.cat(ids, 1).to(torch.int32)


def _exact_moe(c):
    x, kind = c["xd"].double(), c["weight"]
    y = torch.zeros(c["t"], c["k"], dtype=torch.float64, device=DEV)
    for e in torch.unique(c["ids"]).tolist():
        share = torch.where(c["ids"] == e, c["p"].double(), torch.zeros((), dtype=torch.float64, device=DEV)).sum(1)
        rows = share.nonzero().squeeze(1)
        gate = torch.mm(_value(kind, c["experts"][0][e]), x[rows].t().contiguous())
        gate = gate * torch.sigmoid(gate) * torch.mm(_value(kind, c["experts"][1][e]), x[rows].t().contiguous())
        y[rows] += torch.mm(_value(kind, c["experts"][2][e]), gate).t() * share[rows].unsqueeze(1)
    return y if c["r"] is None else y + c["r"].double()


def _token(c, codes, scale, b, head, n, flip):
    """Rows 0..n-1 of one sequence and head, from the cache."""
    block = c["block"]
    i = torch.arange(n, device=DEV)
    page, at = c["table"][b][i // block].long(), i % block
    raw = codes.view(torch.uint8)
    raw = raw[page, head, :, at] if flip else raw[page, head, at]
    return _bits8(raw.contiguous()) * _pow2(_exponents(scale)[page, head]).unsqueeze(1)


def _exact_attention(c):
    g, d, w = c["group"], c["d"], c["window"]
    out, at = torch.empty(c["q"].shape, dtype=torch.float64, device=DEV), 0
    for b, (n, new) in enumerate(zip(c["len_list"], c["new_list"])):
        for head in range(c["heads"]):
            k, v = _token(c, c["kc"], c["ks"], b, head, n, False), _token(c, c["vc"], c["vs"], b, head, n, True)
            kt = k.t().contiguous()
            for j in range(head * g, head * g + g):
                z = torch.mm(c["q"][at:at + new, j].double(), kt) * d ** -0.5
                p = torch.tril(torch.ones(new, n, dtype=torch.bool, device=DEV), n - new)
                if w:
                    p = torch.triu(p, n - new - w + 1)
                z = torch.where(p, z, torch.full_like(z, -math.inf))
                out[at:at + new, j] = torch.mm(torch.exp(z - torch.logsumexp(z, 1, keepdim=True)), v)
        at += new
    return out


def _nearest8(v):
    """The multiple of the e4m3 step nearest to v, halves to even."""
    step = _pow2(torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent - 4)
    return torch.round(v / step) * step


def _exact_append(c):
    block, at = c["block"], 0
    kc, vc, ks, vs = _bits8(c["kc"]), _bits8(c["vc"]), _exponents(c["ks"]).clone(), _exponents(c["vs"]).clone()
    for b, (n, new) in enumerate(zip(c["len_list"], c["new_list"])):
        p = n - new
        while p < n:
            page, lo = int(c["table"][b, p // block]), p % block
            hi = min(block, lo + n - p)
            for x, codes, scale in ((c["knew"], kc, ks), (c["vnew"], vc.transpose(2, 3), vs)):
                rows = x[at:at + hi - lo].double().transpose(0, 1)
                a = rows.abs().amax((1, 2))
                f, e = torch.frexp(a / E4M3_MAX)
                e = torch.where(a == 0, -127, torch.where(f > 0.5, e, e - 1).clamp(-127, 127)).long()
                if lo:
                    e = torch.maximum(e, scale[page])
                    codes[page][:, :lo] = _nearest8(codes[page][:, :lo] * _pow2(scale[page] - e)[:, None, None])
                codes[page][:, lo:hi] = _nearest8(rows / _pow2(e)[:, None, None])
                scale[page] = e
            at, p = at + hi - lo, p + hi - lo
    return kc, vc, _pow2(ks), _pow2(vs)


def exact(case, seed):
    c = prepare(case, seed)
    return {"route": _exact_route, "moe": _exact_moe, "attention": _exact_attention, "append": _exact_append}[c["op"]](c)
