"""Measured cases of the serving operators around the MXFP4 key/value cache.

A case is one pass of one operator, or of the chain of them that a decoding
step runs.  ``run`` has two forms: the framework's calls (``own``), and plain
elementary torch operations in float32 (the sum of squares of a norm in
float64), which follow the operators' definitions step by step.

Definitions.  Keys and queries [T, H, D] are optionally normed per head
(r = fp32(1 / sqrt(mean x^2 + eps)), y = fp32(fp32(x r) w)), rotated by their
position on the first ``rot`` elements (cosines and sines from a table), and
optionally put through the orthonormal block Hadamard transform.  Keys and
values are held as MXFP4: blocks of 32 elements of a head share the least
exponent E with 6 * 2^E >= max, elements are the nearest E2M1 value to
x / 2^E, ties to even.  Pages hold [heads, page, D/2] code bytes (element 2i
in the low nibble of byte i) and [heads, page, D/32] exponent bytes (E + 127).
"""

import math
import random

import torch

own = False

EPS = 1e-6
BASE = 500000.0
DEV = "cuda"


# ------------------------------------------------------------- cases ----
def _rotate(name, tokens, heads, dim, rot, interleaved, norm, hadamard, dtype):
    c = dict(kind="rotate", tokens=tokens, heads=heads, dim=dim, rot=rot, interleaved=interleaved, norm=norm,
             hadamard=hadamard, dtype=dtype)
    return dict(c, name=name) if name else c


def _append(name, tokens, heads, dim, page, rot, interleaved, norm, hadamard, dtype):
    c = dict(kind="append", tokens=tokens, heads=heads, dim=dim, page=page, rot=rot, interleaved=interleaved,
             norm=norm, hadamard=hadamard, dtype=dtype)
    return dict(c, name=name) if name else c


def _attend(name, batch, new, context, ragged, heads, kv_heads, dim, page, causal, window, lse):
    c = dict(kind="attend", batch=batch, new=new, context=context, ragged=ragged, heads=heads, kv_heads=kv_heads,
             dim=dim, page=page, causal=causal, window=window, lse=lse)
    return dict(c, name=name) if name else c


def _step(name, batch, context, heads, kv_heads, dim, page, rot, interleaved, norm, hadamard):
    c = dict(kind="step", batch=batch, new=1, context=context, ragged=True, heads=heads, kv_heads=kv_heads, dim=dim,
             page=page, causal=True, window=0, lse=False, rot=rot, interleaved=interleaved, norm=norm,
             hadamard=hadamard, dtype="bfloat16")
    return dict(c, name=name) if name else c


def listed():
    return [
        # queries of one token of the 8B-shaped layer (32 heads of 128): the smallest call, where latency counts
        _rotate("rotate, one token", 1, 32, 128, 128, False, True, 0, "bfloat16"),
        # queries of a long prompt, half of each head rotated in adjacent pairs, then the 32-point micro-rotation
        _rotate("rotate, prompt, float32", 8192, 32, 128, 64, True, False, 32, "float32"),
        # one new token for each of 64 sequences, keys normed; the values written are read back
        _append("append, 64 sequences", 64, 8, 128, 16, 128, False, True, 0, "bfloat16"),
        # a whole prompt's keys and values, keys with the 128-point micro-rotation; read back
        _append("append, prompt", 8192, 8, 128, 64, 128, False, False, 128, "bfloat16"),
        # an odd number of tokens of a small model, a quarter of the head rotated, float32 projections; read back
        _append("append, odd, float32", 1021, 4, 64, 32, 16, True, True, 0, "float32"),
        # one token of one short conversation: the smallest attention
        _attend("attend, one token", 1, 1, 1024, False, 32, 8, 128, 16, True, 0, False),
        # a full decoding batch of the 70B-shaped layer (64 heads on 8), lengths from 0 to 8192
        _attend("attend, 64 sequences", 64, 1, 8192, True, 64, 8, 128, 64, True, 0, False),
        # one token of one very long context, the log-sum-exp kept for merging
        _attend("attend, long context", 1, 1, 131072, False, 64, 8, 128, 64, True, 0, True),
        # four drafted tokens per sequence verified at once, heads of 256
        _attend("attend, drafted tokens", 16, 4, 4001, True, 16, 2, 256, 32, True, 0, False),
        # prompts of a small model of several lengths behind a sliding window
        _attend("attend, window", 5, 317, 2777, True, 12, 4, 64, 32, True, 1000, True),
        # a chunk of a long prompt against all that came before it, matrix-core bound
        _attend("attend, prompt chunk", 1, 4096, 8192, False, 32, 8, 128, 64, True, 0, False),
        # a decoding step's chain: queries rotated, keys and values appended, attention
        _step("step, 17 sequences", 17, 4099, 32, 8, 128, 16, 128, False, True, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotate", "append", "attend", "attend", "attend", "step"])
    dim = rng.choice([64, 128, 128, 256])
    rot = rng.choice([dim, dim, dim // 2, dim // 4])
    inter, norm = rng.random() < 0.5, rng.random() < 0.5
    had = rng.choice([n for n in (0, 0, 16, 32, 64, 128) if n <= dim])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "rotate":
        heads = rng.choice([1, 2, 5, 8, 12, 32])
        return _rotate("", _log(rng, 1, 8192 * 32 * 128 // (heads * dim)), heads, dim, rot, inter, norm, had, dtype)
    if kind == "append":
        heads = rng.choice([1, 2, 4, 7, 8])
        return _append("", _log(rng, 1, 8192 * 8 * 128 // (heads * dim * (2 if dtype == "float32" else 1))), heads,
                       dim, page, rot, inter, norm, had, dtype)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    if kind == "step":
        batch = _log(rng, 1, 64)
        return _step("", batch, _log(rng, 1, min(32768, 64 * 4096 * 128 // (batch * dim))), heads, kv_heads, dim,
                     page, rot, inter, norm, had)
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    causal = rng.random() < 0.8
    if rng.random() < 0.6:  # few new tokens on a long context
        batch, new = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
        context = _log(rng, new, min(131072, 64 * 4096 * 128 // (batch * dim)))
    else:  # prompts, or chunks of them
        batch = _log(rng, 1, 8)
        new = _log(rng, 9, min(4096, 4096 * 32 * 128 * 3 // (4 * heads * dim)) // batch)
        context = new + _log(rng, 1, 4096)
    return _attend("", batch, new, context, rng.random() < 0.7, heads, kv_heads, dim, page, causal, window,
                   rng.random() < 0.3)


def _lengths(case):
    """Cached lengths and new tokens of the sequences, in an order that the seed shuffles: evenly spread when
    ragged, one sequence empty where there are more than two."""
    b, ctx, new = case["batch"], case["context"], case["new"]
    if not case["ragged"]:
        return [ctx] * b, [new] * b
    lens = [max(1, ctx * (i + 1) // b) for i in range(b)]
    news = [max(1, new * ((5 * i) % b + 1) // b) for i in range(b)]
    if b > 2 and case["kind"] == "attend":
        lens[0] = 0
    return lens, [min(n, max(1, le)) for n, le in zip(news, lens)]


# ------------------------------------------------------------- inputs ----
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _keys(g, *shape, dtype=torch.float32):
    """Keys and queries as projections give them: some channels of a head several times larger than the rest."""
    gain = 1.0 + 4.0 * (torch.rand(shape[-2:], generator=g, device=DEV) < 0.05).float()
    return (torch.randn(shape, generator=g, device=DEV) * gain).to(dtype)


def _table(positions, rot):
    """Cosines, then sines, of every position: angles in float64, rounded once."""
    inv = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _empty_cache(pages, heads, page, dim):
    codes = [torch.zeros((pages, heads, page, dim // 2), dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.full((pages, heads, page, dim // 32), 127, dtype=torch.uint8, device=DEV) for _ in range(2)]
    return [codes[0], scales[0], codes[1], scales[1]]


def prepare(case, seed):
    g = _generator(seed)
    rng = random.Random(seed)
    s = dict(case=dict(case))
    dim, kind = case["dim"], case["kind"]
    dtype = getattr(torch, case.get("dtype", "bfloat16"))
    if "rot" in case:
        n = case["context"] + 1 if kind == "step" else 32768
        s["table"] = _table(n, case["rot"])
        s["norm_q"] = s["norm_k"] = None
        if case["norm"]:
            s["norm_q"] = 1.0 + 0.1 * _normal(g, dim)
            s["norm_k"] = 1.0 + 0.1 * _normal(g, dim)
    if kind == "rotate":
        t = case["tokens"]
        s["x"] = _keys(g, t, case["heads"], dim, dtype=dtype)
        s["positions"] = torch.randint(0, 32768, (t,), generator=g, device=DEV)
        return s
    if kind == "append":
        t, page = case["tokens"], case["page"]
        pages = -(-t // page) + 3
        s["cache"] = _empty_cache(pages, case["heads"], page, dim)
        s["k"] = _keys(g, t, case["heads"], dim, dtype=dtype)
        s["v"] = _normal(g, t, case["heads"], dim, dtype=dtype)
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(t, device=DEV)
        s["slots"] = order[at // page] * page + at % page
        s["positions"] = at + int(rng.randrange(32768 - t + 1))
        return s
    lens, news = _lengths(case)
    order = list(range(len(lens)))
    rng.shuffle(order)
    lens, news = [lens[i] for i in order], [news[i] for i in order]
    page, hk = case["page"], case["kv_heads"]
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + 2, max(1, max(need))
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32)
    mine, at = perm.cpu(), 0
    for b, n in enumerate(need):
        table[b, :n] = mine[at:at + n]
        at += n
    s["cache"] = _empty_cache(pages, hk, page, dim)
    flat = [c.view(pages * hk * page, -1) for c in s["cache"]]
    part = max(1, (1 << 25) // dim)
    for a in range(0, pages * hk * page, part):
        n = min(part, pages * hk * page - a)
        for j in (0, 2):
            rows = _keys(g, n, 1, dim)[:, 0] if j == 0 else _normal(g, n, dim)
            flat[j][a:a + n], flat[j + 1][a:a + n] = _quantized(rows)
    s["block_table"] = table.to(DEV)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["max_len"], s["max_new"] = max(lens), max(news)
    total = sum(news)
    if kind == "step":
        s["qkv"] = _keys(g, total, case["heads"] + 2 * hk, dim, dtype=dtype)
        s["positions"] = s["seq_lens"].long() - 1
        last = torch.clamp(s["positions"], min=0)
        s["slots"] = s["block_table"].long().gather(1, (last // page)[:, None])[:, 0] * page + last % page
        s["cu_q"] = None
        return s
    s["q"] = _keys(g, total, case["heads"], dim, dtype=dtype)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    s["cu_q"] = None if total == len(lens) and max(news) == 1 else torch.tensor(cu, dtype=torch.int32, device=DEV)
    return s


# --------------------------------------------------------- plain forms ----
def _hadamard(y, n):
    z = y.reshape(-1, n)
    h = 1
    while h < n:
        v = z.view(-1, n // (2 * h), 2, h)
        z = torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], dim=2).view(-1, n)
        h *= 2
    return (z * torch.tensor(1.0 / math.sqrt(n), dtype=torch.float32, device=z.device)).view(y.shape)


def _rotated(x, positions, table, case, norm):
    """Norm, rotation and Hadamard of [T, H, D] in float32, each step rounded once."""
    y = x.float()
    if norm is not None:
        r = (1.0 / (y.double().square().mean(-1, keepdim=True) + EPS).sqrt()).float()
        y = y * r * norm
    rot = case["rot"]
    cs = table[positions][:, None, :]
    c, s = cs[..., : rot // 2], cs[..., rot // 2:]
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        z = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    y = torch.cat([z, y[..., rot:]], dim=-1)
    return _hadamard(y, case["hadamard"]) if case["hadamard"] else y


def _quantized(x):
    """MXFP4 codes and exponent bytes of float32 rows [..., D]."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1): 6 * 2^E >= top from E = e - 3 where m <= 0.75, else e - 2
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


def _put(cache, rows, slots, j):
    page = cache[j].shape[2]
    codes, scales = _quantized(rows)
    cache[j][slots // page, :, slots % page] = codes
    cache[j + 1][slots // page, :, slots % page] = scales


def _taken(cache, slots, j):
    page = cache[j].shape[2]
    return _decoded(cache[j][slots // page, :, slots % page], cache[j + 1][slots // page, :, slots % page])


def _attention(q, s):
    """Attention of [T, H, D] queries, all sequences padded to the longest; outputs bfloat16, log-sum-exp float32."""
    c = s["case"]
    b, hk, dim = len(s["seq_lens"]), c["kv_heads"], c["dim"]
    groups, page = c["heads"] // hk, c["page"]
    lens = s["seq_lens"].long()
    starts = torch.arange(b + 1, device=DEV) if s["cu_q"] is None else s["cu_q"].long()
    news, most = starts[1:] - starts[:-1], max(1, s["max_new"])
    pages = s["block_table"][:, : max(1, -(-s["max_len"] // page))].long()
    k, v = [_decoded(s["cache"][j][pages], s["cache"][j + 1][pages]).transpose(1, 2).flatten(2, 3) for j in (0, 2)]
    i = torch.arange(most, device=DEV)
    rows = (starts[:-1, None] + i).clamp(max=len(q) - 1)
    qp = q.float()[rows].view(b, most, hk, groups, dim).permute(0, 2, 1, 3, 4).reshape(b, hk, most * groups, dim)
    x = torch.matmul(qp, k.transpose(2, 3)) * (1.0 / math.sqrt(dim))
    j = torch.arange(k.shape[2], device=DEV)
    own_pos = (lens - news)[:, None] + i
    see = (j < lens[:, None])[:, None, :].expand(b, most, -1)
    if c["causal"]:
        see = see & (j <= own_pos[..., None])
    if c["window"]:
        see = see & (j > own_pos[..., None] - c["window"])
    see = see.repeat_interleave(groups, dim=1)[:, None]
    x = x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
    valid = i < news[:, None]
    o = o.view(b, hk, most, groups, dim).permute(0, 2, 1, 3, 4).reshape(b, most, hk * groups, dim)[valid]
    if not c["lse"]:
        return [o.to(torch.bfloat16)]
    lse = (top + total.log()).view(b, hk, most, groups).permute(0, 2, 1, 3).reshape(b, most, hk * groups)[valid]
    return [o.to(torch.bfloat16), lse]


def _plain(s):
    c = s["case"]
    if c["kind"] == "rotate":
        return [_rotated(s["x"], s["positions"], s["table"], c, s["norm_q"]).to(s["x"].dtype)]
    if c["kind"] == "append":
        _put(s["cache"], _rotated(s["k"], s["positions"], s["table"], c, s["norm_k"]), s["slots"], 0)
        _put(s["cache"], s["v"].float(), s["slots"], 2)
        return [_taken(s["cache"], s["slots"], j).to(torch.bfloat16) for j in (0, 2)]
    if c["kind"] == "attend":
        return _attention(s["q"], s)
    h, hk = c["heads"], c["kv_heads"]
    q = _rotated(s["qkv"][:, :h], s["positions"], s["table"], c, s["norm_q"]).to(torch.bfloat16)
    _put(s["cache"], _rotated(s["qkv"][:, h:h + hk], s["positions"], s["table"], c, s["norm_k"]), s["slots"], 0)
    _put(s["cache"], s["qkv"][:, h + hk:].float(), s["slots"], 2)
    return [q] + _attention(q, s) + [_taken(s["cache"], s["slots"], j).to(torch.bfloat16) for j in (0, 2)]


# ------------------------------------------------- the framework's calls ----
def _framework(s):
    import fp4_post_quantization_amd as fq

    c = s["case"]
    if c["kind"] == "rotate":
        return [fq.rotate_heads(s["x"], s["positions"], s["table"], interleaved=c["interleaved"],
                                norm_weight=s["norm_q"], eps=EPS, hadamard_n=c["hadamard"])]
    cache = fq.KVCacheMXFP4(*s["cache"])
    if c["kind"] == "append":
        fq.kv_append_mxfp4(cache, s["k"], s["v"], s["slots"], s["positions"], s["table"],
                           interleaved=c["interleaved"], norm_weight=s["norm_k"], eps=EPS, hadamard_n=c["hadamard"],
                           window=(0, 0))
        return list(fq.kv_read_mxfp4(cache, s["slots"]))
    if c["kind"] == "attend":
        r = fq.attention_mxfp4(s["q"], cache, s["block_table"], s["seq_lens"], s["cu_q"], max_new=s["max_new"],
                               max_len=s["max_len"], causal=c["causal"], window=c["window"], return_lse=c["lse"])
        return list(r) if c["lse"] else [r]
    h, hk = c["heads"], c["kv_heads"]
    q = fq.rotate_heads(s["qkv"][:, :h], s["positions"], s["table"], interleaved=c["interleaved"],
                        norm_weight=s["norm_q"], eps=EPS, hadamard_n=c["hadamard"])
    fq.kv_append_mxfp4(cache, s["qkv"][:, h:h + hk], s["qkv"][:, h + hk:], s["slots"], s["positions"], s["table"],
                       interleaved=c["interleaved"], norm_weight=s["norm_k"], eps=EPS, hadamard_n=c["hadamard"],
                       window=(0, 0))
    o = fq.attention_mxfp4(q, cache, s["block_table"], s["seq_lens"], max_len=s["max_len"])
    return [q, o] + list(fq.kv_read_mxfp4(cache, s["slots"]))


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------ the work ----
def work(case):
    dim, kind = case["dim"], case["kind"]
    size = 4 if case.get("dtype") == "float32" else 2
    if kind == "rotate":
        n = case["tokens"] * case["heads"] * dim
        return {"bytes": 2 * size * n + case["tokens"] * (8 + 4 * case["rot"]), "flops": 10 * n}
    if kind == "append":
        n = 2 * case["tokens"] * case["heads"] * dim
        # read, held in 17/32 bytes an element (written and read back), and the values read back in two
        return {"bytes": int(n * (size + 17 / 32 + 2)) + case["tokens"] * (16 + 4 * case["rot"]), "flops": 12 * n}
    lens, news = _lengths(case)
    keys, pairs = 0, 0
    for n, new in zip(lens, news):
        low = n
        for i in range(new):
            p = n - new + i
            hi = min(n, p + 1) if case["causal"] else n
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            pairs += max(0, hi - lo)
            low = min(low, lo)
        keys += n - low
    total = sum(news)
    b = keys * case["kv_heads"] * dim * 17 // 16 + 4 * total * case["heads"] * dim
    f = 4 * pairs * case["heads"] * dim
    if kind == "step":
        n = total * (case["heads"] + 2 * case["kv_heads"]) * dim
        b += 2 * n + int(total * 2 * case["kv_heads"] * dim * (2 + 17 / 32)) + total * (24 + 4 * case["rot"])
        f += 12 * n
    return {"bytes": b, "flops": f}


# ----------------------------------------------- from the definition, 64 bits ----
def _exact_rotation(x, positions, table, case, weight):
    z = x.double()
    if weight is not None:
        z = z * torch.rsqrt(torch.mean(z * z, dim=-1, keepdim=True) + EPS) * weight.double()
    half = case["rot"] // 2
    turn = torch.complex(table[positions][:, :half].double(), table[positions][:, half:].double())[:, None]
    first = torch.arange(half, device=z.device) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    w = torch.complex(z[..., first], z[..., second]) * turn
    z = z.clone()
    z[..., first], z[..., second] = w.real, w.imag
    n = case["hadamard"]
    if n:
        i = torch.arange(n, device=z.device)
        ones = sum(((i[:, None] & i[None, :]) >> k) & 1 for k in range(7))
        z = ((z.reshape(-1, n) @ (1.0 - 2.0 * (ones % 2).double())) / math.sqrt(n)).view(z.shape)
    return z


def _exact_mxfp4(x):
    """The values that MXFP4 holds for x (float64): nearest of the E2M1 values at the block's exponent."""
    b = x.reshape(-1, 32)
    top = b.abs().amax(1, keepdim=True)
    step = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 6.0)))
    step = torch.where(6.0 * step < top, step * 2, torch.where(3.0 * step >= top, step / 2, step))
    y = b / step
    a = y.abs()
    # spacing 1/2 below 2, 1 below 4, 2 above; round() takes ties to even multiples, which are the even codes
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return (torch.copysign(a, y) * step).view(x.shape)


def _exact_cached(cache, j, pages):
    codes, scales = cache[j][pages].int(), cache[j + 1][pages]
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=codes.device) / 2
    low, high = [torch.where(n >= 8, -mag[n & 7], mag[n & 7]) for n in (codes % 16, codes // 16)]
    x = torch.stack([low, high], -1).flatten(-2)
    return x * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_attention(q, s, fresh=None):
    c = s["case"]
    g, dim, page = c["heads"] // c["kv_heads"], c["dim"], c["page"]
    outs, lses, at = [], [], 0
    lens = s["seq_lens"].tolist()
    ends = list(range(1, len(lens) + 1)) if s["cu_q"] is None else s["cu_q"].tolist()[1:]
    for b, n in enumerate(lens):
        new, first = ends[b] - at, at
        at = ends[b]
        o = torch.zeros((new, c["heads"], dim), dtype=torch.float64, device=DEV)
        lse = torch.full((new, c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
        pages = s["block_table"][b, : -(-n // page)].long()
        keys, values = [_exact_cached(s["cache"], j, pages).transpose(0, 1).flatten(1, 2)[:, :n] for j in (0, 2)]
        if fresh is not None:  # the last position's keys and values, appended in this pass
            keys[:, -1], values[:, -1] = fresh[0][b], fresh[1][b]
        rows = max(1, (1 << 28) // max(1, n))
        for h in range(c["heads"] if n else 0):
            for a in range(0, new, rows):
                z = min(new, a + rows)
                x = (q[first + a:first + z, h].double() @ keys[h // g].T) / math.sqrt(dim)
                pos = torch.arange(n - new + a, n - new + z, device=DEV)[:, None]
                key = torch.arange(n, device=DEV)[None]
                hide = torch.zeros_like(x, dtype=torch.bool)
                if c["causal"]:
                    hide |= key > pos
                if c["window"]:
                    hide |= key <= pos - c["window"]
                x[hide] = -math.inf
                lse[a:z, h] = torch.logsumexp(x, 1)
                o[a:z, h] = torch.nan_to_num(torch.softmax(x, 1)) @ values[h // g]
        outs.append(o)
        lses.append(lse)
    return [torch.cat(outs)] + ([torch.cat(lses)] if c["lse"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["kind"] == "rotate":
        return [_exact_rotation(s["x"], s["positions"], s["table"], c, s["norm_q"])]
    if c["kind"] == "append":
        return [_exact_mxfp4(_exact_rotation(s["k"], s["positions"], s["table"], c, s["norm_k"])),
                _exact_mxfp4(s["v"].double())]
    if c["kind"] == "attend":
        return _exact_attention(s["q"], s)
    h, hk = c["heads"], c["kv_heads"]
    q = _exact_rotation(s["qkv"][:, :h], s["positions"], s["table"], c, s["norm_q"])
    fresh = [_exact_mxfp4(_exact_rotation(s["qkv"][:, h:h + hk], s["positions"], s["table"], c, s["norm_k"])),
             _exact_mxfp4(s["qkv"][:, h + hk:].double())]
    # the attention's queries are the bfloat16 ones that the rotation hands on
    return [q] + _exact_attention(q.to(torch.bfloat16), s, fresh) + fresh
