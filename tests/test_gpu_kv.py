"""Rotation of heads, the MXFP4 key/value cache and attention over it against
the CPU oracle (oracle/kv.py, oracle/quant.py).

Rotation and quantization are defined step by step in float32, so they are
compared bit for bit.  Attention is compared with float64 on the decoded
cache, with tolerances from the arithmetic the header states:
  * the result is rounded to bfloat16: half a step, 2^-8 of its value;
  * every probability is rounded to bfloat16 before the second product:
    2^-8 of sum p |v|;
  * a score is off by at most 2^-20 of the largest sum of |q_d k_d| (float32
    sums of at most 256 exact products), and its exponential by that much
    relative, as is the sum, plus 2^-18 for the exponential's own error and
    its float32 sums.
"""

import numpy as np
import pytest
import torch

from oracle import kv as KV
from oracle import quant as Q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _fq():
    import fp4_post_quantization_amd as fq
    return fq


def _bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def _heads(rng, t, h, d, dtype, outliers=True):
    x = rng.standard_normal((t, h, d)).astype(np.float32)
    if outliers:
        x *= 1 + 6 * (rng.random((h, d)) < 0.05)
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


# ------------------------------------------------------ heads and rows ----
MAPS = [  # rot, interleaved, norm, hadamard
    (0, False, False, 0), (0, False, True, 0), (64, False, False, 0), (64, True, False, 0), (32, False, True, 16),
    (16, True, True, 32), (48, False, False, 64), (64, False, True, 64), (16, False, False, 0), (0, False, False, 32),
]


def _map_args(rng, t, d, rot, norm, n_pos=4096):
    table = torch.from_numpy(KV.rotary_table(n_pos, rot)) if rot else None
    pos = torch.from_numpy(rng.integers(0, n_pos, t)) if rot else None
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)) if norm else None
    return pos, table, w


def _oracle_map(x, pos, table, inter, w, had):
    return KV.map_heads(x.float().numpy(), None if pos is None else pos.numpy(),
                        None if table is None else table.numpy(), inter, None if w is None else w.numpy(), 1e-6, had)


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rot,inter,norm,had", MAPS)
def test_rotate_heads_bit_exact(dtype, dim, rot, inter, norm, had):
    fq = _fq()
    rng = np.random.default_rng(dim + rot)
    rot = rot * dim // 64
    for t, h in ((1, 1), (3, 5), (67, 2)):
        x = _heads(rng, t, h, dim, dtype)
        pos, table, w = _map_args(rng, t, dim, rot, norm)
        ref = torch.from_numpy(_oracle_map(x, pos, table, inter, w, had))
        p, tb, wd = _dev(pos, table, w)
        for out_dtype in (torch.float32, torch.bfloat16):
            got = fq.rotate_heads(x.to(DEV), p, tb, interleaved=inter, norm_weight=wd, eps=1e-6, hadamard_n=had,
                                  out_dtype=out_dtype, check=True).cpu()
            assert torch.equal(_bits(got), _bits(ref.to(out_dtype))), (t, h, out_dtype)


def test_rotate_heads_strided_in_place_and_empty():
    fq = _fq()
    rng = np.random.default_rng(5)
    big = _heads(rng, 9, 12, 128, torch.bfloat16).to(DEV)
    pos, table, w = _map_args(rng, 9, 128, 128, True)
    p, tb, wd = _dev(pos, table, w)
    part = big[:, 3:8]
    want = fq.rotate_heads(part.contiguous(), p, tb, norm_weight=wd)
    keep = big.clone()
    assert torch.equal(fq.rotate_heads(part, p, tb, norm_weight=wd), want)
    assert torch.equal(big, keep)
    x = part.contiguous()
    fq.rotate_heads(x, p, tb, norm_weight=wd, out=x)
    assert torch.equal(x, want)
    one = big[:1].expand(9, 12, 128)  # a broadcast input: every token the same heads
    assert torch.equal(fq.rotate_heads(one, p, tb), fq.rotate_heads(one.contiguous(), p, tb))
    assert fq.rotate_heads(big[:0], p[:0], tb, check=True).shape == (0, 12, 128)


def test_rotate_heads_passes_non_finite_on_and_reports_positions():
    fq = _fq()
    x = torch.ones(2, 1, 64, device=DEV)
    x[0, 0, 3], x[1, 0, 5] = float("inf"), float("nan")
    y = fq.rotate_heads(x, check=True)
    assert torch.equal(_bits(y), _bits(x))
    table = torch.from_numpy(KV.rotary_table(8, 64)).to(DEV)
    for bad in (-1, 8, 2 ** 62, -2 ** 62):
        with pytest.raises(fq.FP4QError, match="position"):
            fq.rotate_heads(x, torch.tensor([0, bad], device=DEV), table, check=True)
    fq.rotate_heads(x, torch.tensor([0, 7], device=DEV), table, check=True)


def _oracle_rows(x, window):
    """Codes and scales of [tokens, heads, dim] float32 rows."""
    t, h, d = x.shape
    r = Q.quantize_mxfp4(x.reshape(t * h, d), window=window)
    return r.codes.reshape(t, h, d // 2), r.scales.reshape(t, h, d // 32)


def _garbage_cache(fq, pages, heads, page, dim, order="phtd"):
    shapes = [(pages, heads, page, dim // 2), (pages, heads, page, dim // 32)] * 2
    if order == "pthd":
        return fq.KVCacheMXFP4(*(torch.full((s[0], s[2], s[1], s[3]), 255, dtype=torch.uint8, device=DEV).transpose(1, 2)
                                 for s in shapes))
    if order == "hptd":
        return fq.KVCacheMXFP4(*(torch.full((s[1], s[0], s[2], s[3]), 255, dtype=torch.uint8, device=DEV).transpose(0, 1)
                                 for s in shapes))
    return fq.KVCacheMXFP4(*(torch.full(s, 255, dtype=torch.uint8, device=DEV) for s in shapes))


@pytest.mark.parametrize("window", [(0, 0), (-1, 0), (-3, 2)])
@pytest.mark.parametrize("dim,page,order,dtype", [(64, 16, "phtd", torch.bfloat16), (128, 64, "pthd", torch.float32),
                                                  (256, 32, "hptd", torch.bfloat16), (128, 1024, "phtd", torch.bfloat16)])
def test_append_writes_the_quantizers_rows_and_nothing_else(window, dim, page, order, dtype):
    fq = _fq()
    rng = np.random.default_rng(dim + page)
    t, h, pages = 37, 3, 5
    k, v = _heads(rng, t, h, dim, dtype), _heads(rng, t, h, dim, dtype, outliers=False)
    pos, table, w = _map_args(rng, t, dim, dim // 2, True)
    slots = torch.from_numpy(rng.permutation(pages * page)[:t].astype(np.int64))
    slots[4] = -1
    slots[9] = -2 ** 60
    cache = _garbage_cache(fq, pages, h, page, dim, order)
    p, tb, wd, sl = _dev(pos, table, w, slots)
    fq.kv_append_mxfp4(cache, k.to(DEV), v.to(DEV), sl, p, tb, interleaved=True, norm_weight=wd, hadamard_n=64,
                       window=window, check=True)
    want = [torch.full(tuple(c.shape), 255, dtype=torch.uint8) for c in cache]
    rows = (*_oracle_rows(_oracle_map(k, pos, table, True, w, 64), window), *_oracle_rows(v.float().numpy(), window))
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            for c, r in zip(want, rows):
                c[s // page, :, s % page] = torch.from_numpy(r[i])
    for name, c, r in zip(cache._fields, cache, want):
        assert torch.equal(c.cpu(), r), name


def test_append_equals_rotate_then_quantize_on_edges():
    """Zeros, subnormals, the largest float32 and exact ties of the window."""
    fq = _fq()
    x = torch.zeros(6, 1, 64)
    x[1] = 1e-45
    x[2, 0, 7] = -1.17549435e-38
    x[3] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0] * 8)
    x[4, 0, 40] = 3.0e38
    x[5] = -torch.arange(64) / 8
    cache = _garbage_cache(fq, 1, 1, 16, 64)
    slots = torch.arange(6, device=DEV)
    for window in ((0, 0), (-1, 0), (-16, 0)):
        q = fq.quantize_mxfp4(x.view(6, 64).to(DEV), window=window)
        fq.kv_append_mxfp4(cache, x.to(DEV), x.to(DEV), slots, window=window, check=True)
        for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
            assert torch.equal(c[0, 0, :6], q.codes) and torch.equal(s[0, 0, :6], q.scales), window


def test_append_data_errors():
    fq = _fq()
    cache = _garbage_cache(fq, 2, 2, 16, 64)
    x = torch.ones(3, 2, 64, device=DEV)
    before = [c.clone() for c in cache]
    for bad in (32, 2 ** 62):
        with pytest.raises(fq.FP4QError, match="slot"):
            fq.kv_append_mxfp4(cache, x, x, torch.full((3,), bad, device=DEV, dtype=torch.int64), check=True)
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    y = x.clone()
    y[1, 1, 63] = float("nan")
    sl = torch.tensor([0, -1, 31], device=DEV)
    fq.kv_append_mxfp4(cache, y, x, sl, check=True)          # the token with the NaN is skipped
    with pytest.raises(fq.FP4QError, match="non-finite"):
        fq.kv_append_mxfp4(cache, x, y, sl + 1, check=True)  # 1, 0, 32: also past the end
    fq.kv_append_mxfp4(cache, x[:0], x[:0], sl[:0], check=True)


@pytest.mark.parametrize("dim,order", [(64, "phtd"), (128, "pthd"), (256, "hptd")])
def test_read_decodes_rows(dim, order):
    fq = _fq()
    rng = np.random.default_rng(dim)
    cache = _garbage_cache(fq, 4, 3, 32, dim, order)
    for c in cache:
        c.copy_(torch.from_numpy(rng.integers(0, 255, tuple(c.shape)).astype(np.uint8)))
    for c in (cache.k_scales, cache.v_scales):
        c.copy_(torch.from_numpy(rng.integers(100, 150, tuple(c.shape)).astype(np.uint8)))
    slots = torch.tensor([0, 127, 31, -1, 32, 64, 64, 5])
    for out_dtype in (torch.float32, torch.bfloat16):
        got = fq.kv_read_mxfp4(cache, slots.to(DEV), out_dtype=out_dtype, check=True)
        for g, codes, scales in zip(got, (cache.k_codes, cache.v_codes), (cache.k_scales, cache.v_scales)):
            for i, s in enumerate(slots.tolist()):
                want = torch.zeros(3, dim)
                if s >= 0:
                    want = torch.from_numpy(Q.dequantize_mxfp4(codes[s // 32, :, s % 32].cpu().numpy(),
                                                               scales[s // 32, :, s % 32].cpu().numpy()))
                assert torch.equal(g[i].cpu().float(), want.float()), (i, out_dtype)
    with pytest.raises(fq.FP4QError, match="slot"):
        fq.kv_read_mxfp4(cache, torch.tensor([128], device=DEV), check=True)
    assert fq.kv_read_mxfp4(cache, slots[:0].to(DEV))[0].shape == (0, 3, dim)


# -------------------------------------------------------------- attention ----
def _filled(fq, rng, pages, heads, page, dim, order="phtd", spread=6):
    """A cache with every row written: random codes, scales around 2^0."""
    cache = _garbage_cache(fq, pages, heads, page, dim, order)
    for c in (cache.k_codes, cache.v_codes):
        c.copy_(torch.from_numpy(rng.integers(0, 256, tuple(c.shape)).astype(np.uint8)))
    for c in (cache.k_scales, cache.v_scales):
        c.copy_(torch.from_numpy((125 - rng.integers(0, spread, tuple(c.shape))).astype(np.uint8)))
    return cache


def _rows_of(cache, table, b, length):
    """Decoded keys and values [length, heads, dim] of a sequence, float64."""
    page = cache.k_codes.shape[2]
    out = []
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        ids = table[b, : -(-length // page)].tolist()
        if length == 0:
            out.append(np.zeros((0, codes.shape[1], 2 * codes.shape[3])))
            continue
        c, r = (t.cpu().numpy()[ids].transpose(0, 2, 1, 3).reshape(len(ids) * page * t.shape[1], t.shape[3])
                for t in (codes, scales))
        d = Q.dequantize_mxfp4(np.ascontiguousarray(c), np.ascontiguousarray(r)).astype(np.float64)
        out.append(d.reshape(len(ids) * page, codes.shape[1], -1)[:length])
    return out


def _check(o, lse, q, cache, table, lens, starts, scale, causal, window, rows=None):
    o, lse, qn = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy(), q.float().cpu().numpy()
    for b, n in enumerate(lens):
        a, z = starts[b], starts[b + 1]
        if z == a:
            continue
        k, v = _rows_of(cache, table, b, n)
        pick = np.arange(z - a) if rows is None else np.unique(np.clip(rows, 0, z - a - 1))
        for i in pick:  # a row alone: its position is len - (z - a) + i, so later keys are cut off for causal
            p = n - (z - a) + i
            kk, vv = (k[: max(0, p + 1)], v[: max(0, p + 1)]) if causal else (k, v)
            if not causal and window:
                kk, vv = k[max(0, p - window + 1):], v[max(0, p - window + 1):]
                ref = KV.attention(qn[a + i][None].astype(np.float64), kk, vv, scale, False, 0)
            else:
                ref = KV.attention(qn[a + i][None].astype(np.float64), kk, vv, scale, causal, window)
            out, ls, mag, top = (x[0] for x in ref)
            d = top[:, None] * 2.0 ** -20 + 2.0 ** -18
            tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * d) * mag
            assert (np.abs(o[a + i] - out) <= tol).all(), (b, i, np.abs(o[a + i] - out).max())
            seen = np.isfinite(ls)
            assert np.array_equal(np.isneginf(lse[a + i]), ~seen), (b, i)
            assert (np.abs(lse[a + i][seen] - ls[seen]) <= (2 * d[:, 0] + 2.0 ** -22 * np.abs(ls))[seen]).all(), (b, i)


def _run(fq, rng, lens, news, heads, kv_heads, dim, page, causal=True, window=0, order="phtd", scale=None, cu=None,
         rows=None, cache=None, q_gain=1.0, **kw):
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    cache = cache or _filled(fq, rng, pages, kv_heads, page, dim, order)
    perm = rng.permutation(pages)
    table = np.full((len(lens), max(1, max(need))), -7, dtype=np.int32)  # entries past a sequence's end: never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    starts = np.concatenate([[0], np.cumsum(news)])
    q = torch.from_numpy((q_gain * rng.standard_normal((int(starts[-1]), heads, dim))).astype(np.float32))
    q = q.to(torch.bfloat16)
    cu = (set(news) != {1}) if cu is None else cu
    cu_t = torch.from_numpy(starts.astype(np.int32)).to(DEV) if cu else None
    scale = dim ** -0.5 if scale is None else scale
    o, lse = fq.attention_mxfp4(q.to(DEV), cache, torch.from_numpy(table).to(DEV),
                                torch.tensor(lens, dtype=torch.int32, device=DEV), cu_t, causal=causal, window=window,
                                scale=scale, return_lse=True, check=True, **kw)
    _check(o, lse, q, cache, table, lens, starts, scale, causal, window, rows)
    return o, lse


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 2), (7, 1), (16, 1), (20, 1), (6, 6), (66, 2)])
def test_attention_single_tokens(dim, heads, kv_heads):
    rng = np.random.default_rng(dim + heads)
    _run(_fq(), rng, [1, 0, 15, 16, 17, 63, 64, 65, 130, 700], [1] * 10, heads, kv_heads, dim, 16)


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("order", ["phtd", "pthd", "hptd"])
def test_attention_pages_and_orders(page, order):
    rng = np.random.default_rng(page)
    _run(_fq(), rng, [5, 1023, 1024, 1025, 2048, 33], [1] * 6, 8, 2, 128, page, order=order)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 37), (False, 50), (True, 4000)])
def test_attention_several_new_tokens(dim, causal, window):
    rng = np.random.default_rng(dim + window)
    _run(_fq(), rng, [0, 3, 40, 77, 300, 129, 2], [1, 3, 5, 0, 2, 40, 6], 6, 2, dim, 32, causal=causal, window=window)


@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 8, 2), (64, 12, 4), (256, 4, 1)])
@pytest.mark.parametrize("window", [0, 300])
def test_attention_prompts(dim, heads, kv_heads, window):
    rng = np.random.default_rng(dim)
    rows = np.array([0, 1, 15, 16, 17, 31, 63, 64, 100, 127, 128, 129, 255, 256, 299, 400, 10 ** 6])
    _run(_fq(), rng, [301, 700, 129, 1], [301, 256, 1, 1], heads, kv_heads, dim, 64, window=window, rows=rows)
    _run(_fq(), rng, [513, 450], [17, 450], heads, kv_heads, dim, 16, causal=False, window=window, rows=rows)


@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 8, 1), (64, 4, 2), (256, 2, 2)])
def test_attention_long_contexts_split(dim, heads, kv_heads):
    rng = np.random.default_rng(dim)
    _run(_fq(), rng, [20011], [1], heads, kv_heads, dim, 64)
    _run(_fq(), rng, [9000, 1, 12345, 0, 64], [1, 1, 1, 1, 1], heads, kv_heads, dim, 128)
    _run(_fq(), rng, [9000, 1, 5345], [3, 1, 2], heads, kv_heads, dim, 64, window=5000)


def test_attention_many_sequences():
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 1500, 131).tolist()
    _run(_fq(), rng, lens, [1] * 131, 4, 2, 64, 16, rows=None)


@pytest.mark.parametrize("cu", [False, True])
def test_attention_many_short_sequences_of_two_row_tiles(cu):
    """More sequences than a wave has lanes, 20 query heads on one, a workgroup for each unit."""
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 60, 150).tolist()
    _run(_fq(), rng, lens, [1] * 150, 40, 2, 64, 16, cu=cu)


def test_attention_large_and_small_scores():
    """Scores far apart (one key takes everything), and a scale of zero and a negative one."""
    fq = _fq()
    for gain, scale in ((60.0, None), (1e-3, None), (1.0, 0.0), (1.0, -0.2)):
        rng = np.random.default_rng(7)
        _run(fq, rng, [500, 33, 2000], [1, 1, 1], 8, 2, 128, 32, q_gain=gain, scale=scale)


@pytest.mark.parametrize("gain,scale", [(1e33, 1e-34), (1e36, -1e-37), (1e30, 0.0), (1.0, 1e-40), (1e-36, 1e35)])
@pytest.mark.parametrize("dim,new", [(64, 300), (128, 300), (256, 300), (128, 1)])
def test_attention_scales_far_from_one(dim, new, gain, scale):
    """Scores near one from huge queries and a tiny scale or the reverse, and a scale of zero: in one-row tiles and
    in a prompt's (300 rows a head of 8 query heads: 152 row tiles of 128)."""
    rng = np.random.default_rng(dim + new)
    rows = np.array([0, 1, 31, 32, 150, 299])
    _run(_fq(), rng, [max(new, 40)], [new], 64, 8, dim, 16, cu=True, q_gain=gain, scale=scale, rows=rows)


def test_attention_ignores_what_no_row_sees():
    """NaN scales and every byte value behind the last key, before the window and in other pages."""
    fq = _fq()
    rng = np.random.default_rng(3)
    lens, page, dim = [50, 130, 1], 64, 128
    clean = _filled(fq, rng, 5, 2, page, dim)
    table = np.array([[0, -1, -1], [1, 2, 3], [4, 9, 9]], dtype=np.int32)
    dirty = fq.KVCacheMXFP4(*(c.clone() for c in clean))
    for b, n in enumerate(lens):
        for j in range(3):
            for r in range(page):
                tok = j * page + r
                if table[b, j] in range(5) and (tok >= n or tok <= n - 1 - 20):
                    for c in dirty:
                        c[table[b, j], :, r] = 255
    q = torch.from_numpy(rng.standard_normal((3, 4, dim)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    args = (torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    a = fq.attention_mxfp4(q, clean, *args, window=20, check=True, return_lse=True)
    b = fq.attention_mxfp4(q, dirty, *args, window=20, check=True, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_data_errors_are_reported_and_harmless():
    fq = _fq()
    rng = np.random.default_rng(9)
    cache = _filled(fq, rng, 6, 2, 32, 64)
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32)
    lens = torch.tensor([40, 64, 10], dtype=torch.int32)
    good = fq.attention_mxfp4(q, cache, table.to(DEV), lens.to(DEV), check=True)
    cases = []
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 1] = bad
        cases.append((t, lens))
    for bad in (-5, 65, 2 ** 31 - 1):
        le = lens.clone()
        le[1] = bad
        cases.append((table, le))
    for t, le in cases:
        with pytest.raises(fq.FP4QError, match="page number"):
            fq.attention_mxfp4(q, cache, t.to(DEV), le.to(DEV), check=True)
        o = fq.attention_mxfp4(q, cache, t.to(DEV), le.to(DEV))
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])   # other sequences are not touched
    for cu in ([0, 2, 1, 3], [0, 1, 2, 9], [-4, 1, 2, 3]):
        with pytest.raises(fq.FP4QError, match="row offset"):
            fq.attention_mxfp4(q, cache, table.to(DEV), lens.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV),
                               check=True)


def test_attention_leaves_other_rows_alone():
    fq = _fq()
    rng = np.random.default_rng(4)
    cache = _filled(fq, rng, 4, 1, 32, 64)
    q = torch.ones(9, 2, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([40, 64], dtype=torch.int32, device=DEV)
    out = torch.full((9, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([2, 4, 7], dtype=torch.int32, device=DEV)
    fq.attention_mxfp4(q, cache, table, lens, cu, out=out, check=True)
    assert bool((out[:2] == 7).all()) and bool((out[7:] == 7).all()) and bool((out[2:7] != 7).all())
    empty = fq.attention_mxfp4(q[:0], cache, table[:0], lens[:0], check=True)
    assert empty.shape == (0, 2, 64)
    none = torch.zeros(3, dtype=torch.int32, device=DEV)
    fq.attention_mxfp4(q, cache, table, lens, none, out=out.fill_(3), check=True)
    assert bool((out == 3).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kw", [{}, dict(max_new=200)])
@pytest.mark.parametrize("window", [0, 130])
def test_attention_chunk_beside_decoding_sequences(dim, kw, window):
    """Rows of prompts and single tokens in one call, which the two kernels share between them: with and without a
    bound on a sequence's rows, sequences at the border between them (96 and 97 rows of a head), empty ones."""
    rows = np.array([0, 1, 15, 23, 24, 63, 99, 127, 128, 199])
    lens = [40, 5000, 700, 1, 320, 16, 17, 999, 90, 200, 210, 2300]
    news = [1, 1, 100, 1, 0, 1, 1, 1, 2, 24, 25, 200]
    _run(_fq(), np.random.default_rng(dim), lens, news, 8, 2, dim, 64, rows=rows, window=window, **kw)
    _run(_fq(), np.random.default_rng(dim), lens[:3], [1, 1, 199], 36, 4, dim, 64, rows=rows, window=window, **kw)
    _run(_fq(), np.random.default_rng(dim), [0] * 40 + [300], [0] * 40 + [200], 64, 16, dim, 16, rows=rows,
         window=window)  # a padded batch


def test_attention_errors_of_both_kernels_are_kept():
    """A call that both kernels share reports what either finds, and leaves the other sequences as they would be; a
    call without errors on the same workspace clears them; captured and replayed it gives the same bits."""
    fq = _fq()
    rng = np.random.default_rng(17)
    lens, news, page, heads, kv, dim = [5000, 40, 70, 600], [200, 1, 1, 150], 64, 8, 2, 128
    width = -(-max(lens) // page)
    cache = _filled(fq, rng, 4 * width, kv, page, dim)
    ids = torch.from_numpy(rng.permutation(4 * width).reshape(4, width).astype(np.int32)).to(DEV)
    starts = np.concatenate([[0], np.cumsum(news)]).tolist()
    cu = torch.tensor(starts, dtype=torch.int32, device=DEV)
    le = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.from_numpy(rng.standard_normal((starts[-1], heads, dim)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    need = fq._lib.load().fp4q_attention_mxfp4_workspace_bytes(starts[-1], 4, heads, kv, dim, starts[-1],
                                                               width * page, 0)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
    good = fq.attention_mxfp4(q, cache, ids, le, cu, ws=ws, check=True)
    for b in range(4):
        bad_ids, bad_len = ids.clone(), le.clone()
        bad_ids[b, 0] = 4 * width
        bad_len[b] = width * page + 1
        for t, n in ((bad_ids, le), (ids, bad_len)):
            with pytest.raises(fq.FP4QError, match="page number"):
                fq.attention_mxfp4(q, cache, t, n, cu, ws=ws, check=True)
            got = fq.attention_mxfp4(q, cache, t, n, cu, ws=ws)
            # another length moves the cuts of the work, so the others are as near as two results of one call may be:
            # twice 2^-8 of the value and of sum p |v|, which are at most 1.5, and 2^-10 for the scores
            near = 0.0 if n is le else 2 * 1.5 * (2.0 ** -7 + 2.0 ** -10)
            assert bool(((got - good).float().abs()[:starts[b]] <= near).all())
            assert bool(((got - good).float().abs()[starts[b + 1]:] <= near).all())
        assert torch.equal(fq.attention_mxfp4(q, cache, ids, le, cu, ws=ws, check=True), good)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.attention_mxfp4(q, cache, ids, le, cu, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fq.attention_mxfp4(q, cache, ids, le, cu, out=out, ws=ws)
    for k in range(4):
        ids[2, 0] = ids[2, 0] if k % 2 == 0 else -1
        want = fq.attention_mxfp4(q, cache, ids, le, cu)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and fq.read_status(ws) == (0 if k == 0 else fq._lib.DATA_BAD_TABLE)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,news", [([700, 90], [1, 1]), ([9000], [1]), ([300, 5], [3, 2])])
def test_attention_many_query_heads_on_one(dim, lens, news):
    """128 query heads on one cache head: many rows for few tokens."""
    _run(_fq(), np.random.default_rng(dim), lens, news, 128, 1, dim, 64)


@pytest.mark.parametrize("dim,order", [(64, "pthd"), (64, "hptd"), (256, "pthd")])
def test_attention_prompts_in_other_orders(dim, order):
    rng = np.random.default_rng(dim)
    rows = np.array([0, 1, 63, 64, 127, 128, 200, 299])
    _run(_fq(), rng, [300, 211, 1100], [300, 200, 120], 6, 3, dim, 16, order=order, rows=rows)


def test_attention_long_prompts_split_and_whole():
    """Chunks of prompts on long contexts, whose keys several workgroups share, and prompts with enough rows to fill
    the chip, 128 and 256 rows a workgroup."""
    rows = np.array([0, 31, 32, 63, 64, 127, 128, 255, 256, 511, 700, 1023])
    _run(_fq(), np.random.default_rng(1), [9000, 5000], [130, 40], 8, 2, 128, 64, rows=rows)
    _run(_fq(), np.random.default_rng(2), [6000], [200], 4, 1, 256, 128, rows=rows)
    _run(_fq(), np.random.default_rng(3), [7000, 300], [150, 300], 6, 2, 64, 32, window=4500, rows=rows)
    _run(_fq(), np.random.default_rng(4), [3000], [2900], 24, 2, 64, 64, rows=np.array([0, 1000, 2047, 2048, 2899]))
    _run(_fq(), np.random.default_rng(5), [2300], [2200], 128, 8, 128, 64, rows=np.array([0, 1111, 2199]))


def test_attention_rows_with_nan_keep_to_themselves():
    fq = _fq()
    rng = np.random.default_rng(21)
    for new in (1, 3, 150):
        cache = _filled(fq, rng, 12, 2, 16, 128)
        lens = torch.tensor([180], dtype=torch.int32, device=DEV)
        ids = torch.from_numpy(rng.permutation(12).astype(np.int32))[None].to(DEV)
        cu = torch.tensor([0, new], dtype=torch.int32, device=DEV)
        q = torch.from_numpy(rng.standard_normal((new, 8, 128)).astype(np.float32)).to(torch.bfloat16).to(DEV)
        want = fq.attention_mxfp4(q, cache, ids, lens, cu, check=True)
        bad = q.clone()
        bad[new // 2, 3, 7], bad[0, 6, 0] = float("nan"), float("inf")
        got = fq.attention_mxfp4(bad, cache, ids, lens, cu, check=True)
        hit = torch.zeros(new, 8, dtype=torch.bool, device=DEV)
        hit[new // 2, 3] = hit[0, 6] = True
        assert torch.equal(got[~hit], want[~hit]), new
        assert bool(torch.isnan(got[new // 2, 3]).all())


def test_attention_without_keys_or_table():
    fq = _fq()
    cache = fq.kv_cache_mxfp4(1, 2, 16, 64, DEV)
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    for width in (0, 1):
        o, lse = fq.attention_mxfp4(q, cache, torch.zeros((3, width), dtype=torch.int32, device=DEV), lens,
                                    return_lse=True, check=True)
        assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    with pytest.raises(fq.FP4QError, match="page number"):
        fq.attention_mxfp4(q, cache, torch.zeros((3, 1), dtype=torch.int32, device=DEV), lens + 9, max_len=0,
                           check=True)
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    with pytest.raises(fq.FP4QError, match="row offset"):
        fq.attention_mxfp4(q, cache, torch.zeros((3, 1), dtype=torch.int32, device=DEV), lens, cu, max_new=0,
                           check=True)


def test_attention_without_new_tokens_on_a_long_cache():
    """max_new 0 with a table long enough to be split: no row belongs to a sequence, out is left as it is, and an
    offset that gives one a row is reported."""
    fq = _fq()
    cache = fq.kv_cache_mxfp4(64, 2, 64, 64, DEV)
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.arange(64, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([4096], dtype=torch.int32, device=DEV)
    out = torch.full((3, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    none = torch.zeros(2, dtype=torch.int32, device=DEV)
    fq.attention_mxfp4(q, cache, table, lens, none, max_new=0, out=out, check=True)
    assert bool((out == 5).all())
    with pytest.raises(fq.FP4QError, match="row offset"):
        fq.attention_mxfp4(q, cache, table, lens, none + torch.tensor([0, 2], dtype=torch.int32, device=DEV),
                           max_new=0, out=out, check=True)
    assert bool((out == 5).all())


def test_attention_bad_pages_in_every_kernel():
    """A page number out of range masks its tokens and is reported, whichever kernel the sizes choose; sequences
    beside it are as they would be."""
    fq = _fq()
    rng = np.random.default_rng(31)
    for lens, new in (([600, 600], 1), ([5000, 5000], 1), ([600, 600], 300), ([5000, 5000], 40)):
        width = -(-max(lens) // 64)
        cache = _filled(fq, rng, 2 * width, 2, 64, 64)
        ids = torch.from_numpy(rng.permutation(2 * width).reshape(2, width).astype(np.int32))
        cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device=DEV)
        q = torch.from_numpy(rng.standard_normal((2 * new, 8, 64)).astype(np.float32)).to(torch.bfloat16).to(DEV)
        le = torch.tensor(lens, dtype=torch.int32, device=DEV)
        good = fq.attention_mxfp4(q, cache, ids.to(DEV), le, cu, check=True)
        bad = ids.clone()
        bad[0, width // 2] = 2 * width
        bad[0, 0] = -3
        with pytest.raises(fq.FP4QError, match="page number"):
            fq.attention_mxfp4(q, cache, bad.to(DEV), le, cu, check=True)
        got = fq.attention_mxfp4(q, cache, bad.to(DEV), le, cu)
        assert torch.equal(got[new:], good[new:]) and bool(torch.isfinite(got).all())


def test_attention_strided_queries_and_padded_table():
    fq = _fq()
    rng = np.random.default_rng(6)
    cache = _filled(fq, rng, 8, 2, 16, 128)
    big = torch.from_numpy(rng.standard_normal((3, 12, 128)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    wide = torch.from_numpy(rng.permutation(8)[:6].reshape(2, 3).astype(np.int32)).to(DEV)
    table = torch.empty((2, 7), dtype=torch.int32, device=DEV)
    table[:, :3] = wide
    lens = torch.tensor([33, 48], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)
    a = fq.attention_mxfp4(big[:, 2:10], cache, table[:, :3], lens, cu, check=True)
    b = fq.attention_mxfp4(big[:, 2:10].contiguous(), cache, wide, lens, cu, max_new=2, max_len=48, check=True)
    assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """A cache whose pages lie 3 GiB apart: appended, read and attended."""
    fq = _fq()
    far = 3 << 30
    codes = [torch.zeros(2 * far + 4096, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros(2 * far // 16 + 4096, dtype=torch.uint8, device=DEV) for _ in range(2)]
    c4 = [t.as_strided((3, 1, 16, 64), (far, 1024, 64, 1)) for t in codes]
    s4 = [t.as_strided((3, 1, 16, 4), (far // 16, 64, 4, 1)) for t in scales]
    cache = fq.KVCacheMXFP4(c4[0], s4[0], c4[1], s4[1])
    rng = np.random.default_rng(8)
    k, v = _heads(rng, 48, 1, 128, torch.bfloat16).to(DEV), _heads(rng, 48, 1, 128, torch.bfloat16).to(DEV)
    slots = torch.arange(48, device=DEV)
    fq.kv_append_mxfp4(cache, k, v, slots, check=True)
    near = fq.kv_cache_mxfp4(3, 1, 16, 128, DEV)
    fq.kv_append_mxfp4(near, k, v, slots, check=True)
    for a, b in zip(fq.kv_read_mxfp4(cache, slots), fq.kv_read_mxfp4(near, slots)):
        assert torch.equal(a, b)
    q = _heads(rng, 1, 4, 128, torch.bfloat16).to(DEV)
    args = (torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV), torch.tensor([47], dtype=torch.int32, device=DEV))
    assert torch.equal(fq.attention_mxfp4(q, cache, *args, check=True), fq.attention_mxfp4(q, near, *args, check=True))


# ------------------------------------------------------------ used together ----
def _layer_step(fq, qkv, cache, slots, pos, table, w, block_table, lens, heads, kv_heads, ws=None, out=None, st=None):
    q = fq.rotate_heads(qkv[:, :heads], pos, table, norm_weight=w, hadamard_n=64, ws=st)
    fq.kv_append_mxfp4(cache, qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], slots, pos, table,
                       norm_weight=w, hadamard_n=64, ws=st)
    return fq.attention_mxfp4(q, cache, block_table, lens, ws=ws, out=out)


def test_prompt_then_decoding_matches_attention_on_the_whole():
    """A prompt appended in one call and attended, then tokens one at a time: each step's row equals the row of one
    causal pass over the finished cache, within the tolerance of two such results."""
    fq = _fq()
    rng = np.random.default_rng(12)
    heads, kv, dim, page, prompt, steps = 8, 2, 128, 16, 45, 8
    total = prompt + steps
    cache = _garbage_cache(fq, 6, kv, page, dim)
    table = torch.from_numpy(KV.rotary_table(total, dim)).to(DEV)
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(dim)).astype(np.float32)).to(DEV)
    qkv = _heads(rng, total, heads + 2 * kv, dim, torch.bfloat16).to(DEV)
    ids = torch.from_numpy(rng.permutation(6).astype(np.int32))[None].to(DEV)
    at = torch.arange(total, device=DEV)
    slots = ids[0].long()[at // page] * page + at % page
    q = fq.rotate_heads(qkv[:, :heads], at, table, norm_weight=w, hadamard_n=64, check=True)
    fq.kv_append_mxfp4(cache, qkv[:prompt, heads:heads + kv], qkv[:prompt, heads + kv:], slots[:prompt], at[:prompt],
                       table, norm_weight=w, hadamard_n=64, check=True)
    cu = torch.tensor([0, prompt], dtype=torch.int32, device=DEV)
    rows = [fq.attention_mxfp4(q[:prompt], cache, ids, torch.tensor([prompt], dtype=torch.int32, device=DEV), cu)]
    for t in range(prompt, total):
        rows.append(_layer_step(fq, qkv[t:t + 1], cache, slots[t:t + 1], at[t:t + 1], table, w, ids,
                                torch.tensor([t + 1], dtype=torch.int32, device=DEV), heads, kv))
    got = torch.cat(rows)
    cu = torch.tensor([0, total], dtype=torch.int32, device=DEV)
    one, lse = fq.attention_mxfp4(q, cache, ids, torch.tensor([total], dtype=torch.int32, device=DEV), cu,
                                  return_lse=True, check=True)
    _check(got, lse, q, cache, ids.cpu().numpy(), [total], [0, total], dim ** -0.5, True, 0)
    _check(one, lse, q, cache, ids.cpu().numpy(), [total], [0, total], dim ** -0.5, True, 0)


def test_step_in_a_captured_graph_and_on_two_streams():
    """A decoding step captured and replayed with eager work between the replays, and the same step on two streams at
    once on caches of their own: every result equals the eager one."""
    fq = _fq()
    rng = np.random.default_rng(13)
    heads, kv, dim, page, batch = 8, 2, 128, 32, 5
    lens = torch.tensor([1500, 1, 64, 333, 1200], dtype=torch.int32, device=DEV)
    width = 47
    caches = [_filled(fq, rng, batch * width, kv, page, dim) for _ in range(2)]
    ids = torch.from_numpy(rng.permutation(batch * width).reshape(batch, width).astype(np.int32)).to(DEV)
    last = lens.long() - 1
    slots = ids.long().gather(1, (last // page)[:, None])[:, 0] * page + last % page
    table = torch.from_numpy(KV.rotary_table(1500, dim)).to(DEV)
    w = torch.ones(dim, device=DEV)
    qkv = _heads(rng, batch, heads + 2 * kv, dim, torch.bfloat16).to(DEV)
    out = torch.empty(batch, heads, dim, dtype=torch.bfloat16, device=DEV)
    need = fq._lib.load().fp4q_attention_mxfp4_workspace_bytes(batch, batch, heads, kv, dim, 1, width * page, 0)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    st = torch.empty(8192, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _layer_step(fq, qkv, caches[0], slots, last, table, w, ids, lens, heads, kv, ws, out, st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _layer_step(fq, qkv, caches[0], slots, last, table, w, ids, lens, heads, kv, ws, out, st)
    for k in range(4):
        qkv.copy_(_heads(np.random.default_rng(100 + k), batch, heads + 2 * kv, dim, torch.bfloat16))
        eager = _layer_step(fq, qkv, caches[1], slots, last, table, w, ids, lens, heads, kv)
        caches[0].k_codes.copy_(caches[1].k_codes)
        torch.cuda.synchronize()
        for c in zip(*caches):
            c[0].copy_(c[1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), k
        assert fq.read_status(ws) == 0 and fq.read_status(st) == 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(3):
        got = []
        for s, c in zip(streams, caches):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(_layer_step(fq, qkv, c, slots, last, table, w, ids, lens, heads, kv))
        torch.cuda.synchronize()
        assert torch.equal(got[0], eager) and torch.equal(got[1], eager)


def test_refusals_of_the_binding_on_device_tensors():
    fq = _fq()
    cache = fq.kv_cache_mxfp4(4, 2, 16, 64, DEV)
    x = torch.ones(2, 2, 64, device=DEV)
    sl = torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        fq.kv_append_mxfp4(cache, x, x[:1], sl)
    with pytest.raises(ValueError):
        fq.kv_append_mxfp4(cache, x[:, :1], x[:, :1], sl)
    with pytest.raises(ValueError):
        fq.kv_append_mxfp4(cache, x, x, sl.int())
    with pytest.raises(TypeError):
        fq.kv_append_mxfp4(cache, x.half(), x.half(), sl)
    with pytest.raises(ValueError):
        fq.kv_append_mxfp4(cache._replace(v_codes=cache.v_codes[:3]), x, x, sl)
    with pytest.raises(ValueError):
        fq.kv_append_mxfp4(cache._replace(k_scales=cache.v_scales.transpose(1, 2).contiguous().transpose(1, 2)), x, x,
                           sl)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    t, le = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        fq.attention_mxfp4(q.float(), cache, t, le)
    with pytest.raises(ValueError):
        fq.attention_mxfp4(q[:, :3], cache, t, le)
    with pytest.raises(ValueError):
        fq.attention_mxfp4(q, cache, t.long(), le)
    with pytest.raises(ValueError):
        fq.attention_mxfp4(q, cache, t, le.long())
    with pytest.raises(ValueError):
        fq.attention_mxfp4(q[:1], cache, t, le)
    with pytest.raises(fq.FP4QError):
        fq.attention_mxfp4(q, cache, t, le, window=-1)
    with pytest.raises(fq.FP4QError):
        fq.attention_mxfp4(q, cache, t, le, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
