"""The operators of libgemm whose rows choose their own matrices, as they are measured: cases, inputs, plain forms and calls.

  route       a router's choice of experts from its logits: softmax or sigmoid scores, a bias that only the choice
              sees, groups of experts, the top_k, their weights (renormalised or not) and how often each is chosen
  route_step  the same in a training step: the choice and the gradient of the logits from that of the weights
  experts     a router's choice and the mixture-of-experts layer on it, for a few tokens, with microscaled weights
  lora        low-rank adapters beside a shared projection: Y = C + s_a (X A_a^T) B_a^T, a being each row's own adapter
  lora_step   the same in a training step: Y, and from dY the gradients dX, dA and dB

Microscaled operands (OCP Microscaling, MXFP4) are those of perf/operators.py: every 32 consecutive values of a row are
e2m1 numbers under one e8m0 scale, a row padded to a multiple of 128 values.
"""
import functools
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32          # microscaled values that share a scale
ALIGN = 128         # a microscaled row is padded to a multiple of this
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WORKSPACE = 256 << 20   # bytes that a program keeps for what lies between an operator's kernels


def padded(k):
    return -(-k // ALIGN) * ALIGN


# ----------------------------------------------------------------------------------------------------------------
# Cases.

def _route(op, tokens, experts, top_k, kind, score, bias, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0, **more):
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "type": kind, "score": score, "bias": bias,
            "groups": groups, "top_groups": top_groups, "group_top": group_top, "renormalize": renormalize, "scale": scale, **more}


def _lora(op, rows, n, k, rank, adapters, kind, mixed):
    return {"op": op, "rows": rows, "n": n, "k": k, "rank": rank, "adapters": adapters, "type": kind, "mixed": mixed}


def listed():
    return [
        # one decoding token's choice: the latency of a call
        {"name": "route_1_of_128x8_softmax_f32", **_route("route", 1, 128, 8, "f32", "softmax", False)},
        # a prompt through a router with many experts in groups, balanced by a bias
        {"name": "route_4096_of_256x8_sigmoid_groups_bf16",
         **_route("route", 4096, 256, 8, "bf16", "sigmoid", True, 8, 4, 2, True, 2.5)},
        # a ragged training batch, the plain probabilities as weights, the best groups by their best expert
        {"name": "route_step_1001_of_96x6_softmax_groups_f16",
         **_route("route_step", 1001, 96, 6, "f16", "softmax", False, 6, 3, 1, False, 1.0)},
        # a large training batch on few experts, balanced by a bias
        {"name": "route_step_65536_of_64x4_sigmoid_f32", **_route("route_step", 65536, 64, 4, "f32", "sigmoid", True)},
        # one token through a routed mixture of experts: the latency of decoding
        {"name": "experts_1_of_64x4_4096x2048_bf16",
         **_route("experts", 1, 64, 4, "bf16", "softmax", False, renormalize=False, hidden=4096, inter=2048)},
        # a decoding batch that reaches most of the experts
        {"name": "experts_32_of_128x8_4096x1024_bf16",
         **_route("experts", 32, 128, 8, "bf16", "sigmoid", True, 8, 4, 2, True, 2.5, hidden=4096, inter=1024)},
        # one decoding request with an adapter
        {"name": "lora_1x4096x4096_r16_bf16", **_lora("lora", 1, 4096, 4096, 16, 8, "bf16", True)},
        # a decoding batch of requests with adapters of different ranks, some rows without one
        {"name": "lora_48x8192x4096_r64_bf16", **_lora("lora", 48, 8192, 4096, 64, 32, "bf16", True)},
        # the ragged standing shape of the FP32 product
        {"name": "lora_1001x777x513_r24_f32", **_lora("lora", 1001, 777, 513, 24, 5, "f32", False)},
        # prompts of several requests packed one behind the other
        {"name": "lora_8192x4096x4096_r16_bf16", **_lora("lora", 8192, 4096, 4096, 16, 8, "bf16", False)},
        # a small ragged training step
        {"name": "lora_step_513x1001x777_r9_f16", **_lora("lora_step", 513, 1001, 777, 9, 3, "f16", False)},
        # a training step of several adapters on one batch: the largest
        {"name": "lora_step_8192x4096x4096_r32_bf16", **_lora("lora_step", 8192, 4096, 4096, 32, 4, "bf16", False)},
    ]


def _between(rng, low, high, multiple=1):
    """A size in [low, high], spread over its logarithm, mostly a multiple of `multiple`."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if multiple > 1 and rng.random() < 0.6:
        n = -(-n // multiple) * multiple
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(("route", "route_step", "experts", "lora", "lora", "lora_step"))
    kind = rng.choice(("f32", "bf16", "f16"))
    while op in ("route", "route_step", "experts"):
        few = op == "experts"
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = _between(rng, 4 if few else 8, 128 if few else 512, 8) if groups == 1 else \
            groups * _between(rng, 2, (128 if few else 512) // groups, 4)
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, 8)
        tokens = _between(rng, 1, 64 if few else 65536)
        c = _route(op, tokens, experts, top_k, kind, rng.choice(("softmax", "sigmoid")), rng.random() < 0.6, groups, top_groups,
                   rng.choice((1, 2)), rng.random() < 0.6, rng.choice((1.0, 2.5)))
        if few:
            c["hidden"], c["inter"] = _between(rng, 256, 5120, 64), _between(rng, 128, 2560, 64)
        if top_k <= experts // groups * top_groups and (not few or experts * c["hidden"] * c["inter"] <= 1 << 29) and \
                tokens * experts <= 1 << 22:
            return c
    while True:
        rows, n, k = _between(rng, 1, 8192, 16), _between(rng, 64, 8192, 64), _between(rng, 64, 8192, 64)
        rank, adapters = _between(rng, 1, 128, 8), _between(rng, 1, 64)
        size = 2 if kind == "f32" else 1
        if size * rows * (n + k) <= 1 << 26 and rows * (n + k) * rank <= 1 << 31 and adapters * rank * (n + k) <= 1 << 25 and \
                max(rows, 64) * adapters * rank * (n + k) <= 1 << 33:
            return _lora(op, rows, n, k, rank, adapters, kind, rows <= 256 and rng.random() < 0.7)


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}[case["type"]]
    if case["op"].startswith("lora"):
        rows, n, k, r, a = (case[x] for x in ("rows", "n", "k", "rank", "adapters"))
        used = a * (1.0 - (1.0 - 1.0 / a) ** rows) if case["mixed"] else min(a, rows)   # adapters that some row has
        weights = used * r * (n + k) * size
        if case["op"] == "lora":
            return {"bytes": rows * (k + 2 * n) * size + weights, "flops": 2 * rows * r * (n + k)}
        # X, C and Y, dY, the projection's own dX and dX, the weights, and dA and dB in 32 bits
        return {"bytes": rows * (3 * k + 3 * n) * size + weights + 4 * a * r * (n + k), "flops": 6 * rows * r * (n + k)}
    t, e, c = case["tokens"], case["experts"], case["top_k"]
    route = {"bytes": t * e * size + 8 * t * c + 4 * e, "flops": t * e * 8}
    if case["op"] == "route":
        return route
    if case["op"] == "route_step":
        return {"bytes": route["bytes"] + t * e * size + 4 * t * c, "flops": t * e * 16}
    h, i = case["hidden"], case["inter"]
    reached = e * (1.0 - (1.0 - c / e) ** t)   # experts that some token chooses, when all are as likely
    return {"bytes": reached * 3 * i * h * (0.5 + 1.0 / BLOCK) + 2 * t * h * size + 4 * t * e, "flops": 6 * t * c * h * i}


# ----------------------------------------------------------------------------------------------------------------
# The plain form.

def plain_scores(l, score):
    if score == "softmax":
        p = torch.exp(l - l.amax(dim=1, keepdim=True))
        return p / p.sum(dim=1, keepdim=True)
    return 1 / (1 + torch.exp(-l))


def plain_route(s):
    """Experts, weights and how often each expert is chosen. In 64 bits: scores lie next to each other."""
    c = s["case"]
    t, e, groups = c["tokens"], c["experts"], c["groups"]
    score = plain_scores(s["logits"].double(), c["score"])
    value = score + s["bias"].double() if c["bias"] else score
    if groups > 1:
        best = torch.sort(value.view(t, groups, -1), dim=2, descending=True)[0][:, :, :c["group_top"]].sum(dim=2)
        stay = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]   # ties: lowest index
        out = torch.ones(t, groups, dtype=torch.bool, device=value.device).scatter_(1, stay, False)
        value = torch.where(out[:, :, None], -torch.inf, value.view(t, groups, -1)).view(t, e)
    chosen = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    weight = torch.gather(score, 1, chosen)
    if c["renormalize"]:
        weight = weight / weight.sum(dim=1, keepdim=True)
    counts = torch.zeros(e, dtype=torch.int32, device=value.device)
    counts.index_add_(0, chosen.reshape(-1), torch.ones(t * c["top_k"], dtype=torch.int32, device=value.device))
    return chosen.to(torch.int32), (c["scale"] * weight).float(), counts


def plain_route_backward(s, chosen):
    c = s["case"]
    chosen, dw = chosen.long(), c["scale"] * s["dweights"]
    score = plain_scores(s["logits"].float(), c["score"])
    at = torch.gather(score, 1, chosen)
    slope = at * (1 - at) if c["score"] == "sigmoid" else at     # of a sigmoid; for softmax the own part alone
    if c["renormalize"]:
        q = at / at.sum(dim=1, keepdim=True)
        d = q * (dw - (q * dw).sum(dim=1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1 - at)
        return torch.zeros_like(score).scatter_(1, chosen, d).to(s["logits"].dtype)
    dl = torch.zeros_like(score).scatter_(1, chosen, slope * dw)
    if c["score"] == "softmax":
        dl = dl - score * (at * dw).sum(dim=1, keepdim=True)
    return dl.to(s["logits"].dtype)


def power(e):
    """2^e in float32 for whole numbers e in [-127, 127], put together from bits."""
    return torch.where(e > -127, (e.int() + 127) << 23, 1 << 22).view(torch.float32)


@functools.lru_cache(maxsize=None)
def e2m1(device):
    return torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=device)


def plain_decode(codes, scales):
    """Stored codes [..., KP / 2] and scales [..., KP / 32] -> float32 values [..., KP]."""
    table = e2m1(codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), dim=-1)
    v = v.view(*scales.shape, BLOCK)
    return (v * power(scales.int() - 127)[..., None]).view(*codes.shape[:-1], -1)


def plain_experts(s):
    c = s["case"]
    t, e, h, i = c["tokens"], c["experts"], c["hidden"], c["inter"]
    chosen, weight, counts = plain_route(s)
    chosen = chosen.long()
    x = s["x"].float()
    w1c, w1s = s["w1_codes"].view(e, 2 * i, -1), s["w1_scales"].view(e, 2 * i, -1)
    w2c, w2s = s["w2_codes"].view(e, h, -1), s["w2_scales"].view(e, h, -1)
    if chosen.numel() < e:   # the chosen experts, pair by pair
        pairs = chosen.reshape(-1)
        rows = x.repeat_interleave(c["top_k"], dim=0)
        g = torch.matmul(plain_decode(w1c[pairs], w1s[pairs])[:, :, :h], rows[:, :, None])[:, :, 0]
        a = g[:, :i] / (1 + torch.exp(-g[:, :i])) * g[:, i:]
        y = torch.matmul(plain_decode(w2c[pairs], w2s[pairs])[:, :, :i], a[:, :, None])[:, :, 0]
        y = (y.view(t, -1, h) * weight[:, :, None]).sum(dim=1)
    else:                    # every expert for every token, those not chosen with weight zero
        share = torch.zeros(t, e, dtype=torch.float32, device=x.device).scatter_(1, chosen, weight)
        g = torch.matmul(plain_decode(w1c, w1s)[:, :, :h].reshape(e * 2 * i, h), x.t().contiguous()).view(e, 2 * i, t)
        a = g[:, :i] / (1 + torch.exp(-g[:, :i])) * g[:, i:] * share.t()[:, None, :]
        y = torch.bmm(plain_decode(w2c, w2s)[:, :, :i].contiguous(), a.contiguous()).sum(dim=0).t()
    return {"chosen": chosen.to(torch.int32), "weights": weight, "counts": counts, "y": y.to(s["x"].dtype).contiguous()}


def plain_lora_all(s):
    """Adapters side by side as one matrix of adapters * rank rows, what is not a row's own set to zero:
    (A, B as matrices, whether [row, adapter * rank] is the row's own, each row's scale)."""
    c = s["case"]
    n, k, r, a = c["n"], c["k"], c["rank"], c["adapters"]
    ids = s["ids"].long()
    own_part = (ids[:, None] == torch.arange(a, device=ids.device))[:, :, None]
    own_part = (own_part & (torch.arange(r, device=ids.device) < s["ranks"][:, None])).view(-1, a * r)
    scale = s["scales"][ids.clamp(min=0)][:, None]
    return (s["a"].float().view(a * r, k), s["b"].float().transpose(0, 1).reshape(n, a * r), own_part, scale)


def plain_lora(s):
    c = s["case"]
    if c["rows"] > c["adapters"]:
        wa, wb, own_part, scale = plain_lora_all(s)
        hidden = torch.where(own_part, torch.matmul(s["x"].float(), wa.t()), 0.0)
        delta = torch.matmul(hidden * scale, wb.t())
    else:   # each row's own matrices
        ids = s["ids"].long()
        at = ids.clamp(min=0)
        hidden = torch.matmul(s["a"][at].float(), s["x"].float()[:, :, None])
        live = (ids >= 0)[:, None] & (torch.arange(c["rank"], device=ids.device) < s["ranks"][at][:, None])
        hidden = torch.where(live, hidden[:, :, 0], 0.0) * s["scales"][at][:, None]
        delta = torch.matmul(s["b"][at].float(), hidden[:, :, None])[:, :, 0]
    return (s["c"].float() + delta).to(s["x"].dtype)


def plain_lora_backward(s):
    c = s["case"]
    n, k, r, a = c["n"], c["k"], c["rank"], c["adapters"]
    wa, wb, own_part, scale = plain_lora_all(s)
    x, dy = s["x"].float(), s["dy"].float()
    hidden = torch.where(own_part, torch.matmul(x, wa.t()), 0.0) * scale
    dhidden = torch.where(own_part, torch.matmul(dy, wb), 0.0) * scale
    dx = (s["dc"].float() + torch.matmul(dhidden, wa)).to(s["x"].dtype)
    da = torch.matmul(dhidden.t(), x).view(a, r, k)
    db = torch.matmul(dy.t(), hidden).view(n, a, r).transpose(0, 1).contiguous()
    return dx, da, db


def plain_run(s):
    op = s["case"]["op"]
    if op == "experts":
        return plain_experts(s)
    if op == "lora":
        return {"y": plain_lora(s)}
    if op == "lora_step":
        dx, da, db = plain_lora_backward(s)
        return {"y": plain_lora(s), "dx": dx, "da": da, "db": db}
    chosen, weights, counts = plain_route(s)
    out = {"chosen": chosen, "weights": weights, "counts": counts}
    if op == "route_step":
        out["dlogits"] = plain_route_backward(s, chosen)
    return out


# ----------------------------------------------------------------------------------------------------------------
# Inputs.

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _operand(g, rows, k, spread):
    """A microscaled operand as a program keeps it: any codes, the scales of normal values. Made in pieces: a layer's
    experts are many."""
    codes = torch.empty(rows, padded(k) // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, padded(k) // BLOCK, dtype=torch.uint8, device=DEV)
    many = max(1, (1 << 27) // padded(k))
    for r in range(0, rows, many):
        n = min(many, rows - r)
        v = torch.zeros(n, padded(k), device=DEV)
        v[:, :k] = _normal(g, n, k) * spread
        v = v.view(n, -1, BLOCK)
        most = v.abs().amax(dim=2, keepdim=True)
        e = torch.where(most > 0, (torch.frexp(most)[1] - 3).clamp(min=-127), -127)   # the largest e2m1 number is 1.5 * 2^2
        q = v / power(e)
        z = q.abs()
        step = torch.where(z < 2, 0.5, torch.where(z < 4, 1.0, 2.0))
        z = (torch.round(z / step) * step).clamp(max=6.0)
        code = torch.round(torch.where(z < 2, 2 * z, torch.where(z < 4, z + 2, z / 2 + 4))).to(torch.uint8)
        code = (code | (torch.signbit(q).to(torch.uint8) << 3)).view(n, -1, 2)
        codes[r:r + n] = code[:, :, 0] | (code[:, :, 1] << 4)
        scales[r:r + n] = (e[:, :, 0] + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    kind = TYPES[case["type"]]
    s = {"case": dict(case), "workspace": torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV)}
    if case["op"].startswith("lora"):
        rows, n, k, r, a = (case[x] for x in ("rows", "n", "k", "rank", "adapters"))
        s["x"], s["c"] = _normal(g, rows, k).to(kind), _normal(g, rows, n).to(kind)
        s["a"] = (_normal(g, a, r, k) / math.sqrt(k)).to(kind)
        s["b"] = (_normal(g, a, n, r) / math.sqrt(r)).to(kind)
        # adapters' own ranks: the stored one, its half or its quarter; what is stored behind them has no meaning
        s["ranks"] = (r // (1 << torch.randint(0, 3, (a,), generator=g, device=DEV))).clamp(min=1).to(torch.int32)
        s["scales"] = torch.exp(0.3 * _normal(g, a))
        who = torch.randint(0, a, (rows,), generator=g, device=DEV)
        if case["mixed"]:   # a row each request; about one in eight has no adapter
            who = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.125, -1, who) if rows > 1 else who
        else:               # prompts of different lengths, the requests in order, the last rows those of one without an adapter
            who = torch.sort(who)[0]
            who[rows - rows // 16:] = -1
        s["ids"] = who.to(torch.int32)
        s["y"] = torch.empty_like(s["c"])
        if case["op"] == "lora_step":
            s["dy"], s["dc"] = _normal(g, rows, n).to(kind), _normal(g, rows, k).to(kind)
            s["dx"] = torch.empty_like(s["x"])
            s["da"], s["db"] = torch.empty(a, r, k, device=DEV), torch.empty(a, n, r, device=DEV)
        return s
    t, e, top_k = case["tokens"], case["experts"], case["top_k"]
    # logits as a trained router gives them: some experts liked more than others by every token
    s["logits"] = (_normal(g, t, e) + 0.5 * _normal(g, 1, e)).to(torch.float32 if case["op"] == "experts" else kind)
    s["bias"] = 0.05 * _normal(g, e) if case["bias"] else None
    s["chosen"] = torch.empty(t, top_k, dtype=torch.int32, device=DEV)
    s["weights"] = torch.empty(t, top_k, device=DEV)
    s["counts"] = torch.empty(e, dtype=torch.int32, device=DEV)
    if case["op"] == "route_step":
        s["dweights"], s["dlogits"] = _normal(g, t, top_k), torch.empty_like(s["logits"])
    if case["op"] == "experts":
        h, i = case["hidden"], case["inter"]
        s["x"] = _normal(g, t, h).to(kind)
        s["w1_codes"], s["w1_scales"] = _operand(g, e * 2 * i, h, 1.0 / math.sqrt(h))
        s["w2_codes"], s["w2_scales"] = _operand(g, e * h, i, 1.0 / math.sqrt(i))
        s["y"] = torch.empty(t, h, dtype=kind, device=DEV)
    return s


# ----------------------------------------------------------------------------------------------------------------
# One pass.

def own_run(s):
    from fp32_gemm_07_amd import binding as lib
    c = s["case"]
    kinds = {"f32": lib.GEMM_TYPE_F32, "bf16": lib.GEMM_TYPE_BF16, "f16": lib.GEMM_TYPE_F16}
    kind = kinds[c["type"]]
    stream = torch.cuda.current_stream().cuda_stream
    ws = s["workspace"]
    if c["op"].startswith("lora"):
        n, k = c["n"], c["k"]
        adapters = lib.gemm_lora_t(kind, n, k, c["rank"], c["adapters"], s["a"], s["b"], s["ranks"], s["scales"])
        lib.gemm_lora(c["rows"], adapters, s["ids"], s["x"], k, s["c"], n, s["y"], n, ws, WORKSPACE, stream)
        if c["op"] == "lora":
            return {"y": s["y"]}
        lib.gemm_lora_backward(c["rows"], adapters, s["ids"], s["x"], k, s["dy"], n, s["dc"], k, s["dx"], k, s["da"], s["db"],
                               ws, WORKSPACE, stream)
        return {"y": s["y"], "dx": s["dx"], "da": s["da"], "db": s["db"]}
    t, e, top_k = c["tokens"], c["experts"], c["top_k"]
    router = lib.gemm_route_t(e, top_k, lib.GEMM_ROUTE_SIGMOID if c["score"] == "sigmoid" else lib.GEMM_ROUTE_SOFTMAX, c["groups"],
                              c["top_groups"], c["group_top"], c["renormalize"], c["scale"])
    logits_kind = lib.GEMM_TYPE_F32 if c["op"] == "experts" else kind
    lib.gemm_route(t, router, s["logits"], logits_kind, e, s["bias"], s["chosen"], s["weights"], s["counts"], stream)
    out = {"chosen": s["chosen"], "weights": s["weights"], "counts": s["counts"]}
    if c["op"] == "route_step":
        lib.gemm_route_backward(t, router, s["logits"], kind, e, s["chosen"], s["dweights"], s["dlogits"], e, stream)
        out["dlogits"] = s["dlogits"]
    if c["op"] == "experts":
        h, i = c["hidden"], c["inter"]
        lib.gemm_mx_moe_routed(t, h, i, e, top_k, s["chosen"], s["weights"], s["x"], kind, h, s["w1_codes"], s["w1_scales"],
                               s["w2_codes"], s["w2_scales"], s["y"], h, ws, WORKSPACE, stream)
        out["y"] = s["y"]
    return out


def run(state):
    return own_run(state) if own else plain_run(state)


# ----------------------------------------------------------------------------------------------------------------
# The definition in 64 bits.

def _two_to(n):
    """2^n in float64 for whole numbers n in [-1022, 1022], its exponent put together from bits."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_decode(codes, scales, k):
    lo, hi = codes.long() % 16, codes.long() // 16
    n = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int64, device=codes.device)
    n[:, 0::2], n[:, 1::2] = lo, hi
    exponent, mantissa = (n % 8) // 2, (n % 2).double()
    v = torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * _two_to(exponent - 1))
    v = v * (1 - 2 * (n // 8)).double()
    return (v * _two_to(scales.long() - 127).repeat_interleave(BLOCK, dim=1))[:, :k]


def _exact_route(s):
    """The rounds of a top-k one by one. Returns (chosen, weights in float64, counts, scores, all weights [tokens, experts])."""
    c = s["case"]
    t, e, size = c["tokens"], c["experts"], c["experts"] // c["groups"]
    l = s["logits"].double()
    score = torch.softmax(l, dim=1) if c["score"] == "softmax" else torch.sigmoid(l)
    value = score + s["bias"].double()[None, :] if c["bias"] else score.clone()
    row = torch.arange(t, device=l.device)

    def first_largest(v):   # of equal ones the first
        return (v == v.amax(dim=1, keepdim=True)).to(torch.int8).argmax(dim=1)

    if c["groups"] > 1:
        best = torch.zeros(t, c["groups"], dtype=torch.float64, device=l.device)
        for n in range(c["groups"]):
            best[:, n] = torch.topk(value[:, n * size:(n + 1) * size], min(c["group_top"], size), dim=1)[0].sum(dim=1)
        stays = torch.zeros(t, c["groups"], dtype=torch.bool, device=l.device)
        for _ in range(c["top_groups"]):
            at = first_largest(best)
            stays[row, at] = True
            best[row, at] = -math.inf
        value = value.masked_fill(~stays.repeat_interleave(size, dim=1), -math.inf)
    chosen = torch.zeros(t, c["top_k"], dtype=torch.int64, device=l.device)
    for n in range(c["top_k"]):
        chosen[:, n] = first_largest(value)
        value[row, chosen[:, n]] = -math.inf
    weights = score[row[:, None], chosen]
    if c["renormalize"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    weights = c["scale"] * weights
    share = torch.zeros(t, e, dtype=torch.float64, device=l.device)
    share[row[:, None], chosen] = weights
    return chosen.to(torch.int32), weights, (share > 0).sum(dim=0).to(torch.int32), score, share


def _exact_dlogits(s, chosen, score):
    """The chain rule through the scores' and the weights' whole derivatives, a stretch of tokens at a time."""
    c = s["case"]
    parts = []
    for t0 in range(0, c["tokens"], 4096):
        at, sc, dw = chosen[t0:t0 + 4096].long(), score[t0:t0 + 4096], c["scale"] * s["dweights"][t0:t0 + 4096].double()
        own_score = torch.gather(sc, 1, at)
        if c["renormalize"]:   # w_i = s_i / z: dw_i / ds_j = ([i = j] - w_i) / z
            z = own_score.sum(dim=1, keepdim=True)
            dw = (dw - (dw * own_score / z).sum(dim=1, keepdim=True)) / z
        ds = torch.zeros_like(sc).scatter_add_(1, at, dw)
        if c["score"] == "softmax":
            parts.append(sc * (ds - (ds * sc).sum(dim=1, keepdim=True)))
        else:
            parts.append(ds * sc * (1 - sc))
    return torch.cat(parts)


def _exact_lora(s, what):
    c = s["case"]
    x, y = s["x"].double(), s["c"].double()
    if what == "step":
        dy, dx = s["dy"].double(), s["dc"].double()
        da, db = torch.zeros(s["a"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["b"].shape, dtype=torch.float64, device=DEV)
    ranks, scales = s["ranks"].tolist(), s["scales"].double().tolist()
    for n in range(c["adapters"]):
        who = torch.nonzero(s["ids"] == n)[:, 0]
        if not len(who):
            continue
        r, scale = ranks[n], scales[n]
        wa, wb = s["a"][n, :r].double(), s["b"][n, :, :r].double()
        h = x[who] @ wa.t()
        y[who] += scale * (h @ wb.t())
        if what == "step":
            dh = scale * (dy[who] @ wb)
            dx[who] += dh @ wa
            da[n, :r] = dh.t() @ x[who]
            db[n, :, :r] = scale * (dy[who].t() @ h)
    return {"y": y, "dx": dx, "da": da, "db": db} if what == "step" else {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("lora"):
        return _exact_lora(s, "step" if case["op"] == "lora_step" else "forward")
    chosen, weights, counts, score, share = _exact_route(s)
    out = {"chosen": chosen, "weights": weights, "counts": counts}
    if case["op"] == "route_step":
        out["dlogits"] = _exact_dlogits(s, chosen, score)
    if case["op"] == "experts":
        e, h, i = case["experts"], case["hidden"], case["inter"]
        x = s["x"].double()
        y = torch.zeros_like(x)
        for n in range(e):
            who = torch.nonzero(share[:, n])[:, 0]
            if not len(who):
                continue
            up = _exact_decode(s["w1_codes"][n * 2 * i:(n + 1) * 2 * i], s["w1_scales"][n * 2 * i:(n + 1) * 2 * i], h) @ x[who].t()
            a = up[:i] * torch.sigmoid(up[:i]) * up[i:]
            y[who] += share[who, n][:, None] * (_exact_decode(s["w2_codes"][n * h:(n + 1) * h], s["w2_scales"][n * h:(n + 1) * h], i) @ a).t()
        out["y"] = y
    return out
