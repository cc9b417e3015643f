"""Measured cases of products whose rows choose their weights: routing to
experts, the experts' MXFP4 products, the sum of what they give, and low-rank
adapters of many requests beside a shared projection.

A case is one pass of one operator, or of the chain of them that a layer of
experts runs.  ``run`` has two forms: the framework's calls (``own``), and
plain elementary torch operations in float32 (choices of experts in float64,
where a near tie must not depend on rounding).

Definitions.  An entry is a (token, choice) pair, number token * k + choice.
Entries are sorted by the expert they chose, those of one expert in ascending
order, those of none at the end: ``rows`` holds their numbers, ``offsets``
where each expert's begin.  MXFP4: blocks of 32 elements share an exponent E
(byte E + 127), elements are E2M1 codes, element 2i in the low nibble of byte
i.  An adapter adds scale (x A^T) B^T to the rows that carry it.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------- cases ----
def _route(name, tokens, experts, k, score, bias, n_groups, top_groups, renorm, scale, masked, dtype):
    c = dict(kind="route", tokens=tokens, experts=experts, k=k, score=score, bias=bias, n_groups=n_groups,
             top_groups=top_groups, renorm=renorm, scale=scale, masked=masked, dtype=dtype)
    return dict(c, name=name) if name else c


def _product(name, tokens, experts, k, kdim, n, up, padded, dtype):
    """up: from the tokens' activations, gate and up halves joined, to the grouped order; else: from the grouped
    order back to the entries'."""
    c = dict(kind="product", tokens=tokens, experts=experts, k=k, kdim=kdim, n=n, up=up, padded=padded, dtype=dtype)
    return dict(c, name=name) if name else c


def _combine(name, tokens, k, n, add, padded, dtype):
    c = dict(kind="combine", tokens=tokens, k=k, n=n, add=add, padded=padded, dtype=dtype)
    return dict(c, name=name) if name else c


def _lora(name, tokens, adapters, rank, kdim, n, spans, plain_share, dtype):
    """spans: tokens of a request lie together; plain_share: share of the requests without an adapter."""
    c = dict(kind="lora", tokens=tokens, adapters=adapters, rank=rank, kdim=kdim, n=n, spans=spans,
             plain_share=plain_share, dtype=dtype)
    return dict(c, name=name) if name else c


def _layer(name, tokens, experts, k, hidden, inner):
    c = dict(kind="layer", tokens=tokens, experts=experts, k=k, hidden=hidden, inner=inner)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one conversation: the smallest call, where latency counts
        _route("route, one token", 1, 128, 8, "softmax", False, 1, 1, True, 1.0, False, "bfloat16"),
        # a long prompt; sigmoid scores with a bias for balance, four of eight groups, scaled weights
        _route("route, prompt, groups", 8192, 256, 8, "sigmoid", True, 8, 4, True, 2.5, False, "float32"),
        # odd sizes, some experts off, padding tokens, weights left as the softmax gives them
        _route("route, odd, masked", 1021, 60, 4, "softmax", False, 1, 1, False, 1.0, True, "bfloat16"),
        # a decoding batch through many small experts: about one row an expert, bound by the weights
        _product("product, 16 tokens, gate-up", 16, 128, 8, 4096, 1536, True, False, "bfloat16"),
        # the same layer over a prompt: about 256 rows an expert, bound by the matrix cores
        _product("product, prompt, gate-up", 4096, 128, 8, 4096, 1536, True, False, "bfloat16"),
        # few large experts (the 8B layer's down projection for each), back to the entries' order
        _product("product, 8 experts, down", 2048, 8, 2, 14336, 4096, False, False, "bfloat16"),
        # odd sizes with padding tokens, float32 results for the sum that follows
        _product("product, odd, down", 333, 60, 4, 704, 2040, False, True, "float32"),
        # the weighted sum of a prompt's eight results a token
        _combine("combine, prompt", 8192, 8, 4096, False, False, "bfloat16"),
        # of a decoding batch, float32, added to another projection's result, padding tokens
        _combine("combine, 17 tokens", 17, 4, 4096, True, True, "float32"),
        # a decoding batch of 64 requests on 32 adapters, some on none, beside a float32 product
        _lora("adapters, 64 requests", 64, 32, 16, 4096, 4096, False, 0.2, "float32"),
        # prompts of several requests on five adapters beside the 8B layer's gate projection
        _lora("adapters, prompts", 8191, 5, 64, 4096, 14336, True, 0.2, "bfloat16"),
        # a layer of experts for a small decoding batch: quantize, route, products, sum
        _layer("layer, 7 tokens", 7, 64, 6, 4096, 1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(["route", "route", "product", "product", "product", "combine", "lora", "lora", "layer"])
    experts = rng.choice([8, 16, 60, 64, 128, 160, 256])
    k = min(rng.choice([1, 2, 4, 6, 8]), experts // 4)
    if kind == "route":
        experts = rng.choice([experts, 72, 384, 512])
        n_groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0 and experts // g >= 2])
        top_groups = rng.randint(1, n_groups)
        while top_groups * (experts // n_groups) < k:
            top_groups += 1
        score = rng.choice(["softmax", "sigmoid"])
        return _route("", _log(rng, 1, 8192 * 256 // experts), experts, k, score, rng.random() < 0.5, n_groups,
                      top_groups, rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.random() < 0.3,
                      rng.choice(["bfloat16", "float32"]))
    if kind == "combine":
        n = rng.choice([96, 1024, 2040, 4096, 5120, 8192])
        dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
        most = 8192 * 8 * 4096 // (k * n * (2 if dtype == "float32" else 1))
        return _combine("", _log(rng, 1, most), k, n, rng.random() < 0.5, rng.random() < 0.3, dtype)
    if kind == "lora":
        kdim, n = rng.choice([1024, 2040, 4096, 8192]), rng.choice([1000, 1024, 4096, 8192, 14336])
        rank = rng.choice([8, 16, 16, 32, 64, 128])
        dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
        spans = rng.random() < 0.5
        most = 8191 * 18432 // ((kdim + n) * (2 if dtype == "float32" else 1)) if spans else 256
        return _lora("", _log(rng, 1, min(8191, most)), rng.choice([1, 3, 8, 32, 100]), rank, kdim, n, spans,
                     rng.choice([0.0, 0.2, 0.5]), dtype)
    if kind == "layer":
        return _layer("", _log(rng, 1, 64), rng.choice([8, 16, 60, 64]), rng.choice([1, 2]), rng.choice([1024, 2048]),
                      rng.choice([512, 768, 1024]))
    up = rng.random() < 0.5
    kdim, n = rng.choice([512, 704, 1024, 1792, 2048, 4096]), rng.choice([1024, 1536, 2040, 2048, 3584, 4096])
    while experts * kdim * n > 128 * 4096 * 1536:
        experts //= 2
    k = min(k, experts // 4)
    tokens = _log(rng, 1, max(1, 4096 * 8 * 4096 * 1536 // (k * kdim * n * 2)))
    return _product("", min(tokens, 16384), experts, k, kdim, n, up, rng.random() < 0.3,
                    rng.choice(["bfloat16", "bfloat16", "float32"]))


# ------------------------------------------------------------- inputs ----
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7907 + 29)
    return g


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _logits(g, tokens, experts):
    """A router's logits: some experts are chosen more often than others."""
    return 1.5 * _normal(g, tokens, experts) + 0.5 * _normal(g, experts)


def _activations(g, rows, cols, dtype=torch.float32):
    """Rows with a few channels several times larger than the rest."""
    gain = 1.0 + 4.0 * (torch.rand((cols,), generator=g, device=DEV) < 0.02).float()
    return (_normal(g, rows, cols) * gain).to(dtype)


def _held(g, rows, cols, scale):
    """MXFP4 codes and exponent bytes of normal rows of that scale, a part at a time."""
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=DEV)
    part = max(1, (1 << 27) // cols)
    for a in range(0, rows, part):
        z = min(rows, a + part)
        codes[a:z], scales[a:z] = _quantized(_normal(g, z - a, cols) * scale)
    return codes, scales


def _sorted_entries(ids, groups):
    """rows and offsets of a vector of group numbers (negative: none)."""
    key = torch.where(ids >= 0, ids.long(), groups)
    rows = torch.sort(key, stable=True)[1].to(torch.int32)
    counts = torch.bincount(key, minlength=groups + 1)[:groups]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)]).to(torch.int32)
    return offsets, rows


def prepare(case, seed):
    g = _generator(seed)
    rng = random.Random(seed)
    kind = case["kind"]
    s = dict(case=dict(case))
    dtype = getattr(torch, case.get("dtype", "bfloat16"))
    t, k, e = case["tokens"], case.get("k", 1), case.get("experts", 0)
    if kind == "route":
        x = _logits(g, t, e)
        if case["masked"]:  # experts that are off for some tokens, and tokens that are padding
            x = x.masked_fill(torch.rand((t, e), generator=g, device=DEV) < 0.3, -math.inf)
            x[torch.rand((t,), generator=g, device=DEV) < 0.1] = -math.inf
        s["logits"] = x.to(dtype)
        s["bias"] = 0.1 * _normal(g, e) if case["bias"] else None
        return s
    if kind in ("product", "combine"):
        ids = torch.topk(_logits(g, t, max(e, 4 * k)), k, dim=1)[1].to(torch.int32)
        if case["padded"]:
            ids[torch.rand((t,), generator=g, device=DEV) < 0.15] = -1
        s["experts"] = ids
    if kind == "product":
        s["offsets"], s["rows"] = _sorted_entries(ids.flatten(), e)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        kd, n = case["kdim"], case["n"]
        s["a"] = _quantized(_activations(g, t if case["up"] else t * k, kd))
        codes, scales = _held(g, e * n, kd, kd ** -0.5)
        s["b"] = codes.view(e, n, kd // 2), scales.view(e, n, kd // 32)
        s["out"] = torch.zeros((t * k, n // 2 if case["up"] else n), dtype=dtype, device=DEV)
        return s
    if kind == "combine":
        s["y"] = _normal(g, t, k, case["n"], dtype=dtype)
        s["weights"] = torch.softmax(_normal(g, t, k), dim=1).contiguous()
        s["add"] = _normal(g, t, case["n"], dtype=dtype) if case["add"] else None
        return s
    if kind == "lora":
        m, r = case["adapters"], case["rank"]
        if case["spans"]:  # requests of several lengths, one after the other
            cuts = sorted(rng.randrange(t + 1) for _ in range(2 * m - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [t])]
            mine = [-1 if rng.random() < case["plain_share"] else rng.randrange(m) for _ in lens]
            ids = torch.repeat_interleave(torch.tensor(mine), torch.tensor(lens))
        else:
            ids = torch.tensor([-1 if rng.random() < case["plain_share"] else rng.randrange(m) for _ in range(t)])
        ids = ids.to(device=DEV, dtype=torch.int32)
        s["offsets"], s["rows"] = _sorted_entries(ids, m)
        s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
        s["x"] = _activations(g, t, case["kdim"], torch.bfloat16)
        s["y"] = _normal(g, t, case["n"], dtype=dtype)
        s["a"] = (_normal(g, m, r, case["kdim"]) * case["kdim"] ** -0.5).to(torch.bfloat16)
        s["b"] = (_normal(g, m, case["n"], r) * r ** -0.5).to(torch.bfloat16)
        s["scales"] = 0.25 + torch.rand((m,), generator=g, device=DEV)
        return s
    h, i = case["hidden"], case["inner"]
    s["x"] = _activations(g, t, h, torch.bfloat16)
    s["logits"] = _logits(g, t, e)
    codes, scales = _held(g, e * 2 * i, h, h ** -0.5)
    s["up"] = codes.view(e, 2 * i, h // 2), scales.view(e, 2 * i, h // 32)
    codes, scales = _held(g, e * h, i, i ** -0.5)
    s["down"] = codes.view(e, h, i // 2), scales.view(e, h, i // 32)
    return s


# --------------------------------------------------------- plain forms ----
def _quantized(x):
    """MXFP4 codes and exponent bytes of float32 rows [rows, cols]: least exponent with 6 * 2^E >= max."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, torch.where(m <= 0.75, e - 3, e - 2), torch.full_like(e, -127)).clamp(-127, 127)
    y = torch.ldexp(b.abs(), -e)
    i = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = (i.to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e[..., 0] + 127).to(torch.uint8)


def _decoded(codes, scales):
    """float32 values of MXFP4 rows."""
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    q = e2m1[torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()]
    two = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    return (q.view(*scales.shape, 32) * two[..., None]).view(q.shape)


def _routed(x, bias, c):
    """Weights, choices (-1: none), offsets and rows."""
    e, k, ng = c["experts"], c["k"], c["n_groups"]
    x = x.double()
    off = x == -math.inf
    top = x.amax(1, keepdim=True)
    if c["score"] == "softmax":
        ex = (x - torch.where(top > -math.inf, top, torch.zeros_like(top))).exp()
        total = ex.sum(1, keepdim=True)
        score = ex / torch.where(total > 0, total, torch.ones_like(total))
    else:
        score = 1.0 / (1.0 + (-x).exp())
    # without a bias the logits themselves order the experts, and the scores the groups
    pick = (score if bias is None else score + bias.double()).masked_fill(off, -math.inf)
    if ng > 1:
        best = torch.sort(pick.view(-1, ng, e // ng), dim=2, descending=True)[0]
        first, second = best[..., 0], best[..., 1]
        value = first if bias is None else torch.where(second > -math.inf, first + second, first)
        order = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros((len(x), ng), dtype=torch.bool, device=x.device).scatter_(1, order, True)
        off = off | ~keep.repeat_interleave(e // ng, dim=1)
    pick = (x if bias is None else pick).masked_fill(off, -math.inf)
    value, chosen = torch.sort(pick, dim=1, descending=True, stable=True)
    none = value[:, :k] == -math.inf
    chosen = chosen[:, :k]
    w = score.gather(1, chosen).masked_fill(none, 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    ids = chosen.masked_fill(none, -1).to(torch.int32)
    return [(w * c["scale"]).float(), ids, *_sorted_entries(ids.flatten(), e)]


def _by_group(x, offsets, most):
    """Rows in grouped order as [groups, most, ...], and which of them are there."""
    at = offsets[:-1, None].long() + torch.arange(most, device=DEV)
    there = at < offsets[1:, None]
    return x[torch.where(there, at, torch.zeros_like(at))], there


def _products(a, b, offsets, most):
    """Rows in grouped order times their groups' matrices [groups, n, k], in grouped order."""
    rows, there = _by_group(a, offsets, most)
    return torch.matmul(rows, b.transpose(1, 2))[there]


def _gated(y):
    gate, up = y.chunk(2, dim=1)
    return gate / (1.0 + (-gate).exp()) * up


def _summed(y, weights, ids, add):
    y = torch.where((ids >= 0)[..., None], y.float() * weights[..., None], torch.zeros((), device=DEV)).sum(1)
    return y if add is None else y + add.float()


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "route":
        return _routed(s["logits"], s["bias"], c)
    if kind == "product":
        rows = s["rows"].long()
        live = int(s["offsets"][-1])
        a = _decoded(*s["a"])
        y = _products(a[rows // c["k"]] if c["up"] else a, _decoded(*s["b"]), s["offsets"], s["most"])
        out = torch.zeros_like(s["out"])
        if c["up"]:
            out[:live] = _gated(y).to(out.dtype)
        else:
            out[rows[:live]] = y.to(out.dtype)
        return [out]
    if kind == "combine":
        return [_summed(s["y"], s["weights"], s["experts"], s["add"]).to(s["y"].dtype)]
    if kind == "lora":
        rows = s["rows"].long()
        live = int(s["offsets"][-1])
        x, there = _by_group(s["x"][rows].float(), s["offsets"], s["most"])
        u = torch.matmul(x, s["a"].float().transpose(1, 2)) * s["scales"][:, None, None]
        out = s["y"].to(torch.float32, copy=True)
        out[rows[:live]] += torch.matmul(u, s["b"].float().transpose(1, 2))[there]
        return [out.to(s["y"].dtype)]
    k = c["k"]
    x = _decoded(*_quantized(s["x"].float()))
    weights, ids, offsets, rows = _routed(s["logits"], None, dict(c, score="softmax", n_groups=1, renorm=True, scale=1.0))
    rows = rows.long()
    z = _gated(_products(x[rows // k], _decoded(*s["up"]), offsets, c["tokens"])).to(torch.bfloat16)
    y = torch.empty((c["tokens"] * k, c["hidden"]), device=DEV)
    y[rows] = _products(_decoded(*_quantized(z.float())), _decoded(*s["down"]), offsets, c["tokens"])
    return [weights, ids, _summed(y.view(-1, k, c["hidden"]), weights, ids, None).to(torch.bfloat16)]


# ------------------------------------------------- the framework's calls ----
def _framework(s):
    import fp4_post_quantization_amd as fq

    c = s["case"]
    kind = c["kind"]
    if kind == "route":
        r = fq.route_experts(s["logits"], c["k"], score=c["score"], bias=s["bias"], n_groups=c["n_groups"],
                             top_groups=c["top_groups"], group_best=1 if s["bias"] is None else 2,
                             renormalize=c["renorm"], scale=c["scale"])
        return [r.weights, r.experts, r.groups.offsets, r.groups.rows]
    if kind == "product":
        groups = fq.RowGroups(s["offsets"], s["rows"])
        if c["up"]:
            return [fq.gemm_mxfp4_grouped(s["a"], s["b"], groups, gather=c["k"], gated=True, out=s["out"])]
        return [fq.gemm_mxfp4_grouped(s["a"], s["b"], groups, scatter=True, out=s["out"])]
    if kind == "combine":
        return [fq.combine_experts(s["y"], s["weights"], s["experts"], add=s["add"])]
    if kind == "lora":
        return [fq.lora_add(s["y"], s["x"], s["a"], s["b"], fq.RowGroups(s["offsets"], s["rows"]),
                            scales=s["scales"])]
    k = c["k"]
    x = fq.quantize_mxfp4(s["x"], window=(0, 0), with_loss=False, with_offsets=False)
    r = fq.route_experts(s["logits"], k)
    z = fq.gemm_mxfp4_grouped(x, s["up"], r.groups, gather=k, gated=True, out_dtype=torch.bfloat16)
    z = fq.quantize_mxfp4(z, window=(0, 0), with_loss=False, with_offsets=False)
    y = fq.gemm_mxfp4_grouped(z, s["down"], r.groups, scatter=True, out_dtype=torch.float32)
    out = fq.combine_experts(y.view(c["tokens"], k, -1), r.weights, r.experts, out_dtype=torch.bfloat16)
    return [r.weights, r.experts, out]


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------ the work ----
def _hit(groups, tokens, k):
    """Groups that tokens of k different choices each use, on average."""
    return groups * (1.0 - (1.0 - k / groups) ** tokens)


def work(case):
    kind, t, k, e = case["kind"], case["tokens"], case.get("k", 1), case.get("experts", 0)
    size = 4 if case.get("dtype") == "float32" else 2
    if kind == "route":
        return {"bytes": t * (e * size + 12 * k) + 4 * (e + 1) + (4 * e if case["bias"] else 0), "flops": 4 * t * e}
    if kind == "product":
        kd, n = case["kdim"], case["n"]
        b = _hit(e, t, k) * n * kd * 17 / 32 + (t if case["up"] else t * k) * kd * 17 / 32
        return {"bytes": int(b + t * k * ((n // 2 if case["up"] else n) * size + 4)), "flops": 2 * t * k * n * kd}
    if kind == "combine":
        n = case["n"]
        return {"bytes": t * n * size * (k + 1 + case["add"]) + 8 * t * k, "flops": 2 * t * k * n}
    if kind == "lora":
        live = t * (1 - case["plain_share"])
        used = min(case["adapters"], _hit(case["adapters"], live, 1)) if not case["spans"] else case["adapters"]
        kd, n, r = case["kdim"], case["n"], case["rank"]
        return {"bytes": int(2 * live * kd + 2 * t * n * size + used * r * (kd + n) * 2),
                "flops": int(2 * live * r * (kd + n))}
    h, i = case["hidden"], case["inner"]
    b = _hit(e, t, k) * 3 * h * i * 17 / 32 + t * (4 * h + 4 * e)
    return {"bytes": int(b), "flops": 6 * t * k * h * i}


# ----------------------------------------------- from the definition, 64 bits ----
def _exact_held(codes, scales):
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=codes.device) / 2
    c = codes.int()
    low, high = [torch.where(n >= 8, -mag[n & 7], mag[n & 7]) for n in (c % 16, c // 16)]
    return torch.stack([low, high], -1).flatten(-2) * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_mxfp4(x):
    """The values that MXFP4 holds for x (float64): nearest of the E2M1 values at the block's exponent."""
    b = x.reshape(-1, 32)
    top = b.abs().amax(1, keepdim=True)
    step = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 6.0)))
    step = torch.where(6.0 * step < top, step * 2, torch.where(3.0 * step >= top, step / 2, step))
    y = b / step
    a = y.abs()
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return (torch.copysign(a, y) * step).view(x.shape)


def _exact_route(x, bias, c):
    """Token by token on the host."""
    e, k, ng = c["experts"], c["k"], c["n_groups"]
    per = e // ng
    weights, ids = [], []
    bs = [0.0] * e if bias is None else bias.double().tolist()
    for row in x.double().tolist():
        on = [i for i in range(e) if row[i] > -math.inf]
        if c["score"] == "softmax":
            top = max((row[i] for i in on), default=0.0)
            ex = {i: math.exp(row[i] - top) for i in on}
            total = math.fsum(ex.values())
            score = {i: v / total for i, v in ex.items()}
        else:
            score = {i: 1.0 / (1.0 + math.exp(-row[i])) for i in on}
        if ng > 1:
            value = []
            for j in range(ng):
                best = sorted((score[i] + bs[i] for i in on if i // per == j), reverse=True)[:1 if bias is None else 2]
                value.append(sum(best) if best else -math.inf)
            kept = set(sorted(range(ng), key=lambda j: (-value[j], j))[:c["top_groups"]])
            on = [i for i in on if i // per in kept]
        mine = sorted(on, key=lambda i: (-(row[i] if bias is None else score[i] + bs[i]), i))[:k]
        w = [score[i] for i in mine]
        if c["renorm"] and mine:
            total = math.fsum(w)
            w = [v / total for v in w]
        weights.append([v * c["scale"] for v in w] + [0.0] * (k - len(mine)))
        ids.append(mine + [-1] * (k - len(mine)))
    flat = [i for row in ids for i in row]
    rows = sorted(range(len(flat)), key=lambda p: (flat[p] if flat[p] >= 0 else e, p))
    offsets = [sum(1 for i in flat if 0 <= i < j) for j in range(e + 1)] if len(flat) < 4096 else None
    if offsets is None:
        counts = [0] * (e + 1)
        for i in flat:
            if i >= 0:
                counts[i + 1] += 1
        offsets = [sum(counts[:j + 1]) for j in range(e + 1)]
    ints = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (ids, offsets, rows)]
    return [torch.tensor(weights, dtype=torch.float64, device=DEV), *ints]


def _exact_products(rows_of, b, offsets, put):
    for g in range(len(offsets) - 1):
        if offsets[g + 1] > offsets[g]:
            put(offsets[g], offsets[g + 1], rows_of(offsets[g], offsets[g + 1]) @ _exact_held(b[0][g], b[1][g]).T)


def _exact_gated(y):
    n = y.shape[1] // 2
    return y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:]


def exact(case, seed):
    s = prepare(case, seed)
    c, kind = s["case"], case["kind"]
    if kind == "route":
        return _exact_route(s["logits"], s["bias"], c)
    if kind == "product":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        a, rows = _exact_held(*s["a"]), s["rows"].long()

        def put(i, j, y):
            if c["up"]:
                out[i:j] = _exact_gated(y)
            else:
                out[rows[i:j]] = y

        _exact_products(lambda i, j: a[rows[i:j] // c["k"]] if c["up"] else a[i:j], s["b"], s["offsets"].tolist(), put)
        return [out]
    if kind == "combine":
        out = torch.zeros((c["tokens"], c["n"]), dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            on = s["experts"][:, j] >= 0
            out[on] += s["y"][on, j].double() * s["weights"][on, j, None].double()
        return [out if s["add"] is None else out + s["add"].double()]
    if kind == "lora":
        out, rows, cut = s["y"].double(), s["rows"].long(), s["offsets"].tolist()
        for g in range(c["adapters"]):
            mine = rows[cut[g]:cut[g + 1]]
            u = s["x"][mine].double() @ s["a"][g].double().T
            out[mine] += (u @ s["b"][g].double().T) * float(s["scales"][g])
        return [out]
    k = c["k"]
    weights, ids, offsets, rows = _exact_route(
        s["logits"], None, dict(c, score="softmax", n_groups=1, renorm=True, scale=1.0))
    x, cut, rows = _exact_mxfp4(s["x"].double()), offsets.tolist(), rows.long()
    z = torch.zeros((c["tokens"] * k, c["inner"]), dtype=torch.float64, device=DEV)
    y = torch.zeros((c["tokens"] * k, c["hidden"]), dtype=torch.float64, device=DEV)

    def put_z(i, j, v):
        z[i:j] = _exact_gated(v)

    def put_y(i, j, v):
        y[rows[i:j]] = v

    _exact_products(lambda i, j: x[rows[i:j] // k], s["up"], cut, put_z)
    # the second product's activations are those that MXFP4 holds of the bfloat16 rows handed on
    z = _exact_mxfp4(z.to(torch.bfloat16).double())
    _exact_products(lambda i, j: z[i:j], s["down"], cut, put_y)
    return [weights, ids, (y.view(-1, k, c["hidden"]) * weights[..., None]).sum(1)]
