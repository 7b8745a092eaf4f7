"""Performance cases of the block's operators: routing to experts by scores, MXFP4 quantization, the
MXFP4 product and the pass of tokens through MXFP4 experts.

Every case runs in two forms on the same inputs: plain torch operations (``own`` false) and the
library's entry points (``own`` true).  MXFP4 is the OCP microscaled format: blocks of 32 values of a row share
one power-of-two scale (a byte: exponent + 127), each value is 4 bits (e2m1: 0, .5, 1, 1.5, 2, 3, 4, 6
with a sign), two to a byte, the even element in the low half.
"""
import math

import torch

own = False

_MEMBERS = 32   # values of one block


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's few tokens: pure latency
        {"name": "route_few_tokens", "op": "route", "tokens": 16, "experts": 64, "top_k": 6, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_score": "max", "renormalize": True},
        # one calibration batch of a 64-expert block, softmax over all experts
        {"name": "route_batch", "op": "route", "tokens": 65536, "experts": 64, "top_k": 6, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_score": "max", "renormalize": True},
        # many experts in groups, sigmoid scores with a balancing bias; a ragged token count
        {"name": "route_groups", "op": "route", "tokens": 32749, "experts": 256, "top_k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_score": "top2", "renormalize": True},
        # one expert's gate and up weights, from the fp32 master copy
        {"name": "quantize_weights", "op": "quantize", "rows": 2816, "cols": 2048, "dtype": "f32"},
        # a batch of activations
        {"name": "quantize_activations", "op": "quantize", "rows": 65536, "cols": 2048, "dtype": "bf16"},
        # one token through one matrix: the weights are read once
        {"name": "matmul_token", "op": "matmul", "m": 1, "n": 2816, "k": 2048, "out": "bf16"},
        # a ragged batch: no size a multiple of a tile, fp32 out
        {"name": "matmul_ragged", "op": "matmul", "m": 77, "n": 4001, "k": 1440, "out": "f32"},
        # a prompt batch: bound by the matrix cores
        {"name": "matmul_batch", "op": "matmul", "m": 65536, "n": 2816, "k": 2048, "out": "bf16"},
        # decode: one token, its 6 routed and 2 shared experts
        {"name": "experts_token", "op": "experts", "tokens": 1, "d": 2048, "f": 1408, "experts": 64, "top_k": 6,
         "shared": 2, "out": "bf16"},
        # decode of a batch: most experts have a few tokens, all weights are read
        {"name": "experts_decode_batch", "op": "experts", "tokens": 48, "d": 2048, "f": 1408, "experts": 64,
         "top_k": 6, "shared": 2, "out": "bf16"},
        # a prompt batch: experts with some hundreds of tokens each, the shared ones with all
        {"name": "experts_prompt", "op": "experts", "tokens": 8192, "d": 2048, "f": 1408, "experts": 64, "top_k": 6,
         "shared": 2, "out": "bf16"},
        # another block's sizes, ragged tokens, fp32 out
        {"name": "experts_ragged", "op": "experts", "tokens": 333, "d": 1280, "f": 896, "experts": 20, "top_k": 3,
         "shared": 1, "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _one(rng):
    op = rng.choice(("route", "quantize", "matmul", "experts"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * max(1, _log(rng, 4, 256) // groups)
        per = experts // groups
        top_groups = rng.randint(1, groups)
        return {"op": op, "tokens": _log(rng, 1, 65536), "experts": experts,
                "top_k": rng.randint(1, min(16, per * top_groups)), "score": rng.choice(("softmax", "sigmoid")),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups,
                "group_score": rng.choice(("max", "top2")), "renormalize": rng.random() < 0.7}
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 65536), "cols": 32 * _log(rng, 1, 256),
                "dtype": rng.choice(("bf16", "f32"))}
    if op == "matmul":
        return {"op": op, "m": _log(rng, 1, 65536), "n": _log(rng, 16, 8192), "k": 32 * _log(rng, 4, 256),
                "out": rng.choice(("bf16", "f32"))}
    experts = _log(rng, 4, 96)
    return {"op": op, "tokens": _log(rng, 1, 8192), "d": 128 * _log(rng, 2, 32), "f": 128 * _log(rng, 2, 16),
            "experts": experts, "top_k": rng.randint(1, min(8, experts)), "shared": rng.randint(0, 2),
            "out": rng.choice(("bf16", "f32"))}


def draw(rng):
    """A case no dearer than the largest listed one of its operator."""
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = [max(a, b) for a, b in zip(most.get(c["op"], (0, 0)), (w["bytes"], w["flops"]))]
    while True:
        c = _one(rng)
        w = work(c)
        if w["bytes"] <= most[c["op"]][0] and w["flops"] <= most[c["op"]][1]:
            return c


def work(case):
    c = case
    mx = 0.5 + 1.0 / _MEMBERS   # bytes of one MXFP4 value with its share of the scale
    if c["op"] == "route":
        n, e, k = c["tokens"], c["experts"], c["top_k"]
        return {"bytes": 4 * n * e + 8 * n * k + (4 * e if c["bias"] else 0), "flops": 4 * n * e}
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]   # in, codes and scales out and back in, bf16 values out
        return {"bytes": n * ((2 if c["dtype"] == "bf16" else 4) + 2 * mx + 2), "flops": 4 * n}
    if c["op"] == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m + n) * k * mx + m * n * (2 if c["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    n, d, f, ko = c["tokens"], c["d"], c["f"], c["top_k"] + c["shared"]
    slots = min(c["experts"], n * c["top_k"]) + c["shared"]   # experts that can have a token
    return {"bytes": slots * 3 * d * f * mx + n * d * (2 + (2 if c["out"] == "bf16" else 4)) + 8 * n * c["top_k"],
            "flops": 6 * n * ko * d * f}


# ------------------------------------------------------------------ inputs

def _pack(x):
    """fp32 [..., cols] -> (codes uint8 [..., cols/2], scales uint8 [..., cols/32]): plain MXFP4 quantization."""
    b = x.unflatten(-1, (-1, _MEMBERS))
    e = torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 3      # floor(log2 amax) - 2
    e = torch.where(b.abs().amax(-1, keepdim=True) > 0, e, -127).clamp(-127, 127)
    a = torch.ldexp(b.abs(), -e)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = ((a / step).round() * step).clamp(max=6.0)
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + 8 * (b < 0).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (e + 127).squeeze(-1).to(torch.uint8)


def _values(codes, scales):
    """The fp32 values that codes and scales stand for."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    m = c & 7
    low = (m & 1).float() * 0.5
    a = torch.where(m < 2, low, torch.ldexp(1.0 + low, (m >> 1).int() - 1))
    a = torch.where(c > 7, -a, a).unflatten(-1, (-1, _MEMBERS))
    return torch.ldexp(a, scales.int().unsqueeze(-1) - 127).flatten(-2)


def _normal(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda") * scale


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "route":
        n, e = c["tokens"], c["experts"]
        # logits with per-expert offsets: a router's load is never even
        s["logits"] = _normal(g, (n, e), 1.5) + _normal(g, (e,), 0.7)
        s["bias"] = _normal(g, (e,), 0.05) if c["bias"] else None
    elif c["op"] == "quantize":
        # heavy-tailed rows, as activations and weights have, each with a magnitude of its own
        x = _normal(g, (c["rows"], c["cols"])) * torch.exp2(_normal(g, (c["rows"], 1), 2.0))
        s["x"] = x.bfloat16() if c["dtype"] == "bf16" else x
    elif c["op"] == "matmul":
        s["a"], s["a_scales"] = _pack(_normal(g, (c["m"], c["k"])))
        s["w"], s["w_scales"] = _pack(_normal(g, (c["n"], c["k"]), 0.02))
    else:
        n, d, f, e, slots = c["tokens"], c["d"], c["f"], c["experts"], c["experts"] + c["shared"]
        s["x"] = _normal(g, (n, d)).bfloat16()
        s["wgu"], s["wgu_scales"] = _pack(_normal(g, (slots, 2 * f, d), d ** -0.5))
        s["wd"], s["wd_scales"] = _pack(_normal(g, (slots, d, f), f ** -0.5))
        scores = torch.softmax(_normal(g, (n, e), 1.5) + _normal(g, (e,), 0.7), -1)
        w, topk = torch.topk(scores, c["top_k"], dim=-1)
        s["topk"], s["weights"] = topk.int(), w / w.sum(-1, keepdim=True)
    if own:
        import gptq_calibration_moe_amd as clha
        if c["op"] == "route":
            s["ctx"] = clha.Context(256, c["experts"], c["top_k"], 0, c["tokens"])
        elif c["op"] == "experts":
            s["ctx"] = clha.Context(c["d"], c["experts"], c["top_k"], c["shared"], c["tokens"])
        else:
            s["ctx"] = clha.Context(256, 8, 2, 0, 1)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    return {"route": _route, "quantize": _quantize, "matmul": _matmul, "experts": _experts}[c["op"]](state, c)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _route(s, c):
    if own:
        topk, weights = s["ctx"].route(s["logits"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                       top_groups=c["top_groups"], group_score=c["group_score"],
                                       renormalize=c["renormalize"])
        return {"topk": topk, "weights": weights}
    # 64 bits: which of two close choices is larger decides whole numbers
    l = s["logits"].double()
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    choice = l if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        per = choice.unflatten(-1, (c["groups"], -1))
        if c["group_score"] == "max":
            mark = per.amax(-1)
        else:
            two = (p if s["bias"] is None else choice).unflatten(-1, (c["groups"], -1))
            mark = two.sort(dim=-1, descending=True)[0][..., :2].sum(-1)
        order = mark.sort(dim=-1, descending=True, stable=True)[1][..., :c["top_groups"]]
        keep = torch.zeros_like(mark, dtype=torch.bool).scatter(-1, order, True)
        choice = torch.where(keep.unsqueeze(-1), per, -math.inf).flatten(-2)
    topk = choice.sort(dim=-1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = p.gather(-1, topk)
    if c["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return {"topk": topk.int(), "weights": w.float()}


def _quantize(s, c):
    if own:
        codes, scales = s["ctx"].mx_quantize(s["x"])
        return s["ctx"].mx_dequantize(codes, scales)
    return _values(*_pack(s["x"].float())).bfloat16()   # 4-bit values times powers of two are exact in bf16


def _matmul(s, c):
    if own:
        return s["ctx"].mx_matmul(s["a"], s["a_scales"], s["w"], s["w_scales"], dtype=_type(c["out"]))
    return (_values(s["a"], s["a_scales"]) @ _values(s["w"], s["w_scales"]).T).to(_type(c["out"]))


def _experts(s, c):
    if own:
        return s["ctx"].mx_experts(s["x"], s["topk"], s["weights"], s["wgu"], s["wgu_scales"], s["wd"],
                                   s["wd_scales"], dtype=_type(c["out"]))
    n, f, e, shared = c["tokens"], c["f"], c["experts"], c["shared"]
    slots, ko = e + shared, c["top_k"] + shared
    dev = s["x"].device
    x = _values(*_pack(s["x"].float()))
    # every (token, expert) pair, sorted by expert and laid into tiles of `rows` pairs of one expert
    extra = torch.arange(e, slots, device=dev, dtype=torch.int32).expand(n, shared)
    slot = torch.cat((s["topk"], extra), 1).flatten().long()
    weight = torch.cat((s["weights"], torch.ones(n, shared, device=dev)), 1)
    pairs = n * ko
    rows = min(256, 1 << max(0, (pairs // slots).bit_length() - 1)) if pairs > slots else 1
    tiles = pairs if rows == 1 else pairs // rows + slots
    by, at = slot.sort(stable=True)
    count = torch.zeros(slots, dtype=torch.long, device=dev).scatter_add_(0, slot, torch.ones_like(slot))
    need = (count + rows - 1) // rows
    first_tile = need.cumsum(0) - need
    rank = torch.arange(pairs, device=dev) - (count.cumsum(0) - count)[by]
    place = torch.empty_like(slot)
    place[at] = first_tile[by] * rows + rank
    owner = torch.searchsorted(need.cumsum(0), torch.arange(tiles, device=dev), right=True).clamp(max=slots - 1)
    xt = x.new_zeros(tiles * rows, x.shape[1])
    xt[place] = x.repeat_interleave(ko, 0)
    gu = torch.bmm(xt.view(tiles, rows, -1), _values(s["wgu"][owner], s["wgu_scales"][owner]).mT.contiguous())
    gate, up = gu[..., :f], gu[..., f:]
    h = _values(*_pack(gate / (1.0 + torch.exp(-gate)) * up))
    y = torch.bmm(h, _values(s["wd"][owner], s["wd_scales"][owner]).mT.contiguous()).flatten(0, 1)
    return (y[place].view(n, ko, -1) * weight.unsqueeze(-1)).sum(1).to(_type(c["out"]))


# ------------------------------------------------------------------ 64 bits

_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest64(x):
    """MXFP4's values of fp64 x, from the definition: the nearest of the eight levels, a tie to the even one."""
    b = x.unflatten(-1, (-1, _MEMBERS))
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2((torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2).clamp(-127, 127))
    # log2 may round up to a whole number just below a power of two: amax / scale lies in [4, 8)
    scale = torch.where(top / scale < 4, scale / 2, torch.where(top / scale >= 8, scale * 2, scale))
    a = b.abs() / scale
    q = torch.zeros_like(a)
    for i in range(7):
        mid = (_LEVELS[i] + _LEVELS[i + 1]) / 2
        up = a >= mid if i % 2 else a > mid
        q = torch.where(up, _LEVELS[i + 1], q)
    return (torch.sign(b) * q * scale).flatten(-2)


def _stored64(codes, scales):
    level = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), dtype=torch.float64, device=codes.device)
    v = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    v[..., 0::2], v[..., 1::2] = level[(codes % 16).int()], level[(codes // 16).int()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(_MEMBERS, -1)


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "route":
        l = s["logits"].double()
        p = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
        score = l if s["bias"] is None else p + s["bias"].double()
        n, g = c["tokens"], c["groups"]
        if g > 1:
            by = (p if s["bias"] is None and c["group_score"] == "top2" else score).view(n, g, -1)
            mark = by.max(-1).values if c["group_score"] == "max" else by.topk(min(2, by.shape[-1]), -1).values.sum(-1)
            worst = mark.topk(c["top_groups"], -1).values[:, -1:]
            score = score.masked_fill((mark < worst).repeat_interleave(c["experts"] // g, -1), -math.inf)
        best = score.topk(c["top_k"], -1).indices
        w = p.gather(1, best)
        return {"topk": None, "weights": w / w.sum(1, keepdim=True) if c["renormalize"] else w}
    if c["op"] == "quantize":
        return _nearest64(s["x"].double())
    if c["op"] == "matmul":
        return _stored64(s["a"], s["a_scales"]) @ _stored64(s["w"], s["w_scales"]).T
    x, f, e = _nearest64(s["x"].double()), c["f"], c["experts"]
    y = torch.zeros_like(x)
    for slot in range(e + c["shared"]):
        w = (s["weights"].double() * (s["topk"] == slot)).sum(1)
        t = torch.nonzero((s["topk"] == slot).any(1)).flatten()
        if slot >= e:
            w, t = torch.ones_like(w), torch.arange(c["tokens"], device=x.device)
        if t.numel():
            gu = x[t] @ _stored64(s["wgu"][slot], s["wgu_scales"][slot]).T
            h = _nearest64(gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:])
            y[t] += w[t, None] * (h @ _stored64(s["wd"][slot], s["wd_scales"][slot]).T)
    return y
