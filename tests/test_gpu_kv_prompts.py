"""Attention's kernel for prompts (attn_prompt_kernel) with tiles of 128 and of 256 rows, whole and split: masks,
windows, cache orders, scales, moving maxima, NaN rows, bad pages and rows that see nothing, against float64.  SHAPES
names the sizes that lead there; tests/test_kv_plan.py asserts on the host that they do.

Tolerances are those that tests/test_gpu_kv.py derives, and 2^-100 for what float32 cannot hold: an exponential below
2^-126 is zero, and so is what a factor below that rescales.  The sum that divides it is at least 1, at most 2^14 keys
of values below 2 and exponentials up to 2^8 are dropped: less than 2^-126 2^14 2 2^8 = 2^-103.  Rows with scores
hundreds apart have elements that small, where the leading keys' values are zero.
"""

import numpy as np
import pytest
import torch

from oracle import kv as KV
from test_gpu_kv import DEV, _filled, _fq, _rows_of

pytestmark = pytest.mark.gpu

# name: rows of a tile, split, and lengths, new tokens, query heads, cache heads, page
SHAPES = {
    "128 whole": (128, False, [301, 700, 129, 1], [301, 256, 1, 1], 64, 8, 64),
    "128 whole, small pages": (128, False, [433], [300], 48, 16, 16),
    "128 split": (128, True, [5000, 4500], [150, 41], 12, 4, 64),
    "128 split, large pages": (128, True, [9000], [130], 8, 2, 1024),
    "256 whole": (256, False, [950], [900], 128, 64, 32),
    "256 whole, two": (256, False, [650, 1200], [650, 620], 96, 96, 16),
}
DIMS = {128: (64, 128, 256), 256: (64, 128)}
CASES = [(name, dim) for name, s in SHAPES.items() for dim in DIMS[s[0]]]

# rows of a sequence that are compared: at the edges of waves and tiles, and far in
ROWS = np.array([0, 1, 7, 8, 31, 32, 63, 64, 100, 127, 128, 149, 255, 256, 299, 511, 600, 10 ** 6])


def _check(o, lse, q, cache, table, lens, starts, scale, causal=True, window=0, rows=ROWS):
    o, q = (t.float().cpu().numpy().astype(np.float64) for t in (o, q))
    lse = lse.cpu().numpy()
    for b, n in enumerate(lens):
        a, new = int(starts[b]), int(starts[b + 1] - starts[b])
        if new == 0:
            continue
        k, v = _rows_of(cache, table, b, n)
        for i in np.unique(np.clip(rows, 0, new - 1)):
            p = n - new + i  # the row's position; the keys it sees are cut out, so that it is a row alone
            lo = max(0, p - window + 1) if window else 0
            hi = max(0, p + 1) if causal else n
            out, ls, mag, top = (x[0] for x in KV.attention(q[a + i][None], k[lo:hi], v[lo:hi], scale, False, 0))
            d = top[:, None] * 2.0 ** -20 + 2.0 ** -18
            tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * d) * mag + 2.0 ** -100
            err = np.abs(o[a + i] - out)
            assert (err <= tol).all(), (b, i, (err / tol).max())
            seen = np.isfinite(ls)
            assert np.array_equal(np.isneginf(lse[a + i]), ~seen), (b, i)
            assert (np.abs(lse[a + i][seen] - ls[seen]) <= (2 * d[:, 0] + 2.0 ** -22 * np.abs(ls))[seen]).all(), (b, i)


def _inputs(rng, name, dim, order="phtd", gain=1.0):
    """Queries, a filled cache, page numbers [batch, pages] (-7 past a sequence's end), lengths and offsets of a
    shape."""
    _, _, lens, news, heads, kv_heads, page = SHAPES[name]
    need = [-(-n // page) for n in lens]
    pages, at = sum(need) + 2, 0
    cache = _filled(_fq(), rng, pages, kv_heads, page, dim, order)
    perm, ids = rng.permutation(pages), np.full((len(lens), max(need)), -7, dtype=np.int32)
    for b, n in enumerate(need):
        ids[b, :n] = perm[at:at + n]
        at += n
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = torch.from_numpy((gain * rng.standard_normal((int(starts[-1]), heads, dim))).astype(np.float32))
    return q.to(torch.bfloat16), cache, ids, lens, starts


def _dev(*arrays):
    return [torch.as_tensor(np.asarray(a), dtype=torch.int32, device=DEV) for a in arrays]


def _go(name, dim, seed=0, order="phtd", q_gain=1.0, scale=None, causal=True, window=0):
    fq = _fq()
    q, cache, ids, lens, starts = _inputs(np.random.default_rng(seed + dim), name, dim, order, q_gain)
    scale = dim ** -0.5 if scale is None else scale
    o, lse = fq.attention_mxfp4(q.to(DEV), cache, *_dev(ids, lens, starts), causal=causal, window=window, scale=scale,
                                return_lse=True, check=True)
    _check(o, lse, q, cache, ids, lens, starts, scale, causal, window)


@pytest.mark.parametrize("name,dim", CASES)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 300), (True, 1), (False, 77)])
def test_prompts_masks(name, dim, causal, window):
    _go(name, dim, causal=causal, window=window)


@pytest.mark.parametrize("name,dim", CASES)
@pytest.mark.parametrize("order", ["pthd", "hptd"])
def test_prompts_cache_orders(name, dim, order):
    _go(name, dim, seed=1, order=order)


@pytest.mark.parametrize("name,dim", CASES)
@pytest.mark.parametrize("gain,scale", [(1.0, 0.0), (1.0, -0.3), (60.0, None), (60.0, -0.1), (1e-3, None)])
def test_prompts_scales_and_large_scores(name, dim, gain, scale):
    _go(name, dim, seed=2, q_gain=gain, scale=scale)


def _rising(fq, rng, pages, kv_heads, page, dim, ids, falling):
    """A cache whose keys grow (or shrink) by a factor of two every so many tokens of the sequence on pages ids, from
    2^-5 to 2^3 of the usual ones, so that a row's maximum moves again and again."""
    cache = _filled(fq, rng, pages, kv_heads, page, dim, spread=1)
    tokens = len(ids) * page
    step = np.arange(tokens) * 9 // tokens - 5
    step = step[::-1] if falling else step
    by_page = torch.from_numpy((122 + step).reshape(len(ids), page).astype(np.uint8)).to(DEV)
    cache.k_scales[torch.from_numpy(ids.astype(np.int64)).to(DEV)] = by_page[:, None, :, None].expand(
        len(ids), kv_heads, page, dim // 32).contiguous()
    return cache


@pytest.mark.parametrize("name,dim", [c for c in CASES if len(SHAPES[c[0]][2]) == 1] + [("rows", d) for d in DIMS[128]])
@pytest.mark.parametrize("falling", [False, True])
@pytest.mark.parametrize("window", [0, 400])
def test_moving_maxima(name, dim, falling, window):
    """Scores that grow (fall) along the keys far beyond the step at which a running maximum is taken again.  "rows"
    is the kernel for few rows, on 3000 keys."""
    fq = _fq()
    rng = np.random.default_rng(dim + falling)
    lens, news, heads, kv_heads, page = SHAPES[name][2:] if name in SHAPES else ([3000], [3], 8, 2, 64)
    n = -(-lens[0] // page)
    ids = rng.permutation(n + 1)[:n]
    cache = _rising(fq, rng, n + 1, kv_heads, page, dim, ids, falling)
    q = torch.from_numpy((8 * rng.standard_normal((news[0], heads, dim))).astype(np.float32)).to(torch.bfloat16)
    o, lse = fq.attention_mxfp4(q.to(DEV), cache, *_dev(ids[None], lens, [0, news[0]]), window=window, return_lse=True,
                                check=True)
    _check(o, lse, q, cache, ids[None], lens, [0, news[0]], dim ** -0.5, True, window)


@pytest.mark.parametrize("name,dim", CASES)
def test_prompts_with_fewer_keys_than_rows(name, dim):
    """Rows before the first key see nothing: zeros and minus infinity, in whole row tiles and within one."""
    fq, news = _fq(), SHAPES[name][3]
    q, cache, ids, _, starts = _inputs(np.random.default_rng(dim), name, dim)
    lens = [max(0, n - 170) for n in news]
    o, lse = fq.attention_mxfp4(q.to(DEV), cache, *_dev(ids, lens, starts), return_lse=True, check=True)
    _check(o, lse, q, cache, ids, lens, starts, dim ** -0.5, rows=np.concatenate([ROWS, [168, 169, 170, 171]]))
    for a, n in zip(starts, news):
        assert bool((o[a:a + min(n, 170)] == 0).all()) and bool(torch.isneginf(lse[a:a + min(n, 170)]).all())


@pytest.mark.parametrize("name,dim", CASES)
def test_prompt_rows_with_nan_keep_to_themselves(name, dim):
    """The caches' scores lie within the step at which a maximum moves, so the other rows keep their bits."""
    fq, new = _fq(), SHAPES[name][3][0]
    q, cache, *rest = _inputs(np.random.default_rng(21 + dim), name, dim)
    q, args = q.to(DEV), _dev(*rest)
    want = fq.attention_mxfp4(q, cache, *args, check=True)
    bad, hit = q.clone(), torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    for row, head, value in ((new // 2, 3, float("nan")), (0, -1, float("inf")), (new - 1, 0, -float("inf"))):
        bad[row, head, 7] = value
        hit[row, head] = True
    got = fq.attention_mxfp4(bad, cache, *args, check=True)
    assert torch.equal(got[~hit], want[~hit])
    assert bool(torch.isnan(got[new // 2, 3]).all())


@pytest.mark.parametrize("name,dim", CASES)
def test_prompt_pages_out_of_range_are_masked_and_reported(name, dim):
    """The last row of a sequence with two such pages sees the other keys alone; other sequences are as they would
    be."""
    fq = _fq()
    _, _, lens, news, _, _, page = SHAPES[name]
    q, cache, ids, _, starts = _inputs(np.random.default_rng(31 + dim), name, dim)
    args = _dev(lens, starts)
    good = fq.attention_mxfp4(q.to(DEV), cache, *_dev(ids), *args, check=True)
    bad, middle = ids.copy(), -(-lens[0] // page) // 2
    bad[0, middle], bad[0, 0] = len(cache.k_codes), -3
    with pytest.raises(fq.FP4QError, match="page number"):
        fq.attention_mxfp4(q.to(DEV), cache, *_dev(bad), *args, check=True)
    got, lse = fq.attention_mxfp4(q.to(DEV), cache, *_dev(bad), *args, return_lse=True)
    assert torch.equal(got[news[0]:], good[news[0]:]) and bool(torch.isfinite(got).all())
    k, v = _rows_of(cache, ids, 0, lens[0])
    keep = ~np.isin(np.arange(lens[0]) // page, (0, middle))
    row = q[news[0] - 1].float().numpy()[None].astype(np.float64)
    out, ls, mag, top = (x[0] for x in KV.attention(row, k[keep], v[keep], dim ** -0.5, False, 0))
    d = top[:, None] * 2.0 ** -20 + 2.0 ** -18
    err = np.abs(got[news[0] - 1].float().cpu().numpy() - out)
    assert (err <= 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * d) * mag + 2.0 ** -100).all()
    assert (np.abs(lse[news[0] - 1].cpu().numpy() - ls) <= 2 * d[:, 0] + 2.0 ** -22 * np.abs(ls)).all()


@pytest.mark.parametrize("name,dim", CASES)
def test_prompts_ignore_what_no_row_sees(name, dim):
    """NaN patterns behind the last key, before the window and in other pages change nothing."""
    fq, window = _fq(), 90
    page = SHAPES[name][6]
    q, clean, ids, lens, starts = _inputs(np.random.default_rng(41 + dim), name, dim)
    seen = np.zeros((len(clean.k_codes), page), dtype=bool)
    for b, (n, new) in enumerate(zip(lens, np.diff(starts))):
        t = np.arange(max(0, n - new - window + 1), n)
        seen[ids[b, t // page], t % page] = True
    hide = torch.from_numpy(~seen).to(DEV)[:, None, :, None]
    dirty = fq.KVCacheMXFP4(*(torch.where(hide, torch.full_like(c, 255), c) for c in clean))
    a, b = (fq.attention_mxfp4(q.to(DEV), c, *_dev(ids, lens, starts), window=window, check=True, return_lse=True)
            for c in (clean, dirty))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("name,dim", CASES)
def test_prompts_repeat_and_replay(name, dim):
    """The same call twice, and captured and replayed on other queries, gives the same bits."""
    fq, rng = _fq(), np.random.default_rng(51 + dim)
    q, cache, *rest = _inputs(rng, name, dim)
    q, args = q.to(DEV), _dev(*rest)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.attention_mxfp4(q, cache, *args, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fq.attention_mxfp4(q, cache, *args, out=out)
    for _ in range(3):
        q.copy_(torch.from_numpy(rng.standard_normal(tuple(q.shape)).astype(np.float32)))
        first = fq.attention_mxfp4(q, cache, *args, check=True)
        again = fq.attention_mxfp4(q, cache, *args, check=True)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, again) and torch.equal(first, out)
