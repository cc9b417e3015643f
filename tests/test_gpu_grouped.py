"""Routing to experts, grouped MXFP4 products, the sum of the experts' results
and adapters against the CPU oracle (oracle/grouped.py, oracle/gemm.py).

Choices, offsets and rows are whole numbers and have to be equal.  Tolerances
come from the arithmetic the header states, u = 2^-24 being float32's half
step, and h a half step of the result's type (bfloat16 2^-8, float32 2^-24):
  * weights: float64, rounded once (u), and one more u for float64's own
    steps; a softmax that is not renormalised and has no bias divides by a
    float32 sum of float32 exponentials, each off by at most (2 d + 3) u for a
    logit d below the largest (subtraction, product, exponential), which
    weighs exp(-d), and d exp(-d) < 0.4; at most 16 of them are added in a
    lane: 20 u.
  * products: (2 ceil(K / 64) + 2) u sum |a| |b| as for the plain product;
    silu(g) adds, for g off by d, 1.1 d, and its own exponential, sum and
    quotient (|g| + 8) u of it; the product with the up half one u.
  * combine: k + 1 steps, u each, of the sum of magnitudes.
  * adapters: x A^T sums K products in float32, in steps of 32 and over at
    most 32 shares, then scale, then rank products three times over, then y:
    (K / 32 + 32 + 1 + 3 rank / 32 + 2) u of s (|x| |A|^T) |B|^T, u |y|.
"""

import math

import numpy as np
import pytest
import torch

from oracle import gemm as GM
from oracle import grouped as GR

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _fq():
    import fp4_post_quantization_amd as fq
    return fq


def _np(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _within(got, ref, tol, dtype=torch.float32):
    # half a step of the result: relative, and below float32's (and bfloat16's) normal range, where float32's are 2^-149
    # apart and bfloat16's 2^-133, absolute
    tol = tol + HALF[dtype] * np.abs(ref) + (2.0 ** -150 if dtype == torch.float32 else 2.0 ** -134)
    err = np.abs(_np(got) - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), bad.size, float(np.nanmax(err / np.maximum(tol, 1e-300))))


# ------------------------------------------------------------- routing ----
def _check_route(x, k, **kw):
    fq = _fq()
    bias = kw.get("bias")
    r = fq.route_experts(x, k, check=True, **kw)
    w, ids, bad = GR.route(_np(x), k, **dict(kw, bias=None if bias is None else _np(bias)))
    assert not bad.any()
    np.testing.assert_array_equal(_np(r.experts), ids)
    loose = kw.get("score", "softmax") == "softmax" and not kw.get("renormalize", True) and bias is None
    _within(r.weights, w, (20 if loose else 2) * U * np.abs(w))
    off, rows = GR.group_rows(ids, x.shape[1])
    np.testing.assert_array_equal(_np(r.groups.offsets), off)
    np.testing.assert_array_equal(_np(r.groups.rows), rows)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("experts,k", [(1, 1), (7, 2), (60, 4), (64, 64), (65, 3), (128, 8), (200, 6), (256, 8),
                                       (512, 10), (1000, 5), (1024, 32)])
def test_route_experts(dtype, experts, k):
    g = torch.Generator().manual_seed(experts)
    bias = (0.1 * torch.randn(experts, generator=g)).to(DEV)
    for tokens in (1, 3, 64, 65, 301):
        x = (1.5 * torch.randn(tokens, experts, generator=g)).to(dtype).to(DEV)
        for score in ("softmax", "sigmoid"):
            _check_route(x, k, score=score)
            _check_route(x, k, score=score, renormalize=False, scale=2.5)
            _check_route(x, k, score=score, bias=bias)


@pytest.mark.parametrize("experts,n_groups,top_groups,k", [(64, 8, 3, 6), (60, 5, 2, 4), (72, 8, 1, 9), (256, 8, 4, 8),
                                                           (256, 64, 7, 8), (512, 2, 1, 8), (1024, 16, 16, 2)])
def test_route_within_groups(experts, n_groups, top_groups, k):
    g = torch.Generator().manual_seed(n_groups)
    bias = (0.1 * torch.randn(experts, generator=g)).to(DEV)
    for tokens in (1, 70, 515):
        x = (1.5 * torch.randn(tokens, experts, generator=g)).to(DEV)
        for best in (1, 2):
            kw = dict(n_groups=n_groups, top_groups=top_groups, group_best=best)
            _check_route(x, k, score="sigmoid", bias=bias, **kw)
            _check_route(x, k, bias=bias, renormalize=False, **kw)
            _check_route(x, k, score="sigmoid", **kw)
            _check_route(x, k, **kw)


@pytest.mark.parametrize("experts", [60, 64, 65, 256, 300])
def test_route_where_one_workgroup_ends(experts):
    """Tokens around the numbers up to which one workgroup routes and sorts."""
    g = torch.Generator().manual_seed(experts)
    bias = (0.1 * torch.randn(experts, generator=g)).to(DEV)
    for tokens in (8, 16, 17, 24, 25):
        x = (1.5 * torch.randn(tokens, experts, generator=g)).to(DEV)
        for k in (6, 50):
            _check_route(x, k)
            _check_route(x, k, score="sigmoid", bias=bias)


def test_route_ties_take_the_lowest_index():
    """Equal logits (both zeros among them), equal scores with a bias, equal groups."""
    g = torch.Generator().manual_seed(3)
    for tokens in (5, 200):
        x = torch.randint(-2, 3, (tokens, 192), generator=g).float()
        x = torch.where((x == 0) & (torch.rand(x.shape, generator=g) < 0.5), -0.0, x).to(DEV)
        zero = torch.zeros(192, device=DEV)
        for score in ("softmax", "sigmoid"):
            _check_route(x, 8, score=score)
            _check_route(x, 8, score=score, bias=zero)
            _check_route(x, 8, score=score, bias=zero, n_groups=6, top_groups=2, group_best=2)
            _check_route(x, 8, score=score, n_groups=6, top_groups=2)


def test_route_settles_near_ties_in_float64():
    """Scores with a bias that float32 rounds to the same value."""
    x = torch.full((70, 100), 0.5)
    x[:, 1::3] += 2.0 ** -24
    x[:, 2::7] += 2.0 ** -23
    bias = torch.full((100,), 7.0)
    _check_route(x.to(DEV), 20, score="sigmoid", bias=bias.to(DEV))
    _check_route(x.to(DEV), 20, score="softmax", bias=bias.to(DEV))
    _check_route(x.to(DEV), 20, score="sigmoid", bias=bias.to(DEV), n_groups=4, top_groups=2, group_best=2)


def test_route_masked_and_far_logits():
    g = torch.Generator().manual_seed(4)
    for tokens in (6, 130):
        x = 3.0 * torch.randn(tokens, 96, generator=g)
        x[torch.rand(x.shape, generator=g) < 0.4] = -math.inf
        x[0] = -math.inf                  # nothing on
        x[1, 3:] = -math.inf              # fewer than k on
        x[2], x[3], x[4, :50] = -300.0, 300.0, -3e38
        bias = torch.zeros(96)
        bias[7] = -math.inf
        for b in (None, bias.to(DEV)):
            for score in ("softmax", "sigmoid"):
                _check_route(x.to(DEV), 8, score=score, bias=b)
                _check_route(x.to(DEV), 8, score=score, bias=b, n_groups=4, top_groups=2, renormalize=False)
        low = torch.full((3, 96), -2000.0)  # sigmoids of 0 in float64: no sum to divide by
        _check_route(low.to(DEV), 8, score="sigmoid")


@pytest.mark.parametrize("tokens", [4, 100])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_route_reports_bad_tokens(tokens, bad):
    fq = _fq()
    x = torch.randn(tokens, 40)
    x[2, 39] = bad
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    for kw in ({}, dict(score="sigmoid"), dict(bias=torch.zeros(40, device=DEV)), dict(n_groups=4, top_groups=2)):
        with pytest.raises(fq.FP4QError, match="non-finite"):
            fq.route_experts(x.to(DEV), 3, check=True, **kw)
        r = fq.route_experts(x.to(DEV), 3, ws=ws, **kw)
        assert (r.experts[2] == -1).all() and (r.weights[2] == 0).all()
        assert int(r.groups.offsets[-1]) == 3 * (tokens - 1)
        good = torch.cat([x[:2], x[3:]]).to(DEV)
        again = fq.route_experts(good, 3, ws=ws, check=True, **kw)  # a call without errors clears the status
        assert torch.equal(again.experts, torch.cat([r.experts[:2], r.experts[3:]]))
    with pytest.raises(fq.FP4QError, match="non-finite"):
        fq.route_experts(torch.zeros(tokens, 40, device=DEV), 3, bias=torch.full((40,), bad, device=DEV), check=True)


def test_route_strided_large_and_empty():
    fq = _fq()
    wide = torch.randn(300, 200, device=DEV)
    for k in (1, 5):
        _check_route(wide[:, 37:165], k)
        _check_route(wide.bfloat16()[:, 1:161], k, score="sigmoid")
    _check_route(torch.randn(20000, 64, device=DEV).bfloat16(), 6)
    r = fq.route_experts(wide[:0], 4, check=True)
    assert r.weights.shape == (0, 4) and r.groups.rows.numel() == 0 and (r.groups.offsets == 0).all()
    assert fq.route_experts(wide, 4, group=False).groups is None


@pytest.mark.parametrize("groups", [1, 2, 60, 300, 2048])
@pytest.mark.parametrize("entries", [0, 1, 63, 1024, 1025, 2048, 2049, 5000, 100001])
def test_group_rows(entries, groups):
    fq = _fq()
    rng = np.random.default_rng(entries + groups)
    ids = rng.integers(-1, groups, entries).astype(np.int32)
    if entries > 60:
        ids[rng.random(entries) < 0.3] = groups - 1  # one long group
        ids[-30:] = -5
    r = fq.group_rows(torch.from_numpy(ids).to(DEV), groups, check=True)
    off, rows = GR.group_rows(ids, groups)
    np.testing.assert_array_equal(_np(r.offsets), off)
    np.testing.assert_array_equal(_np(r.rows), rows)


@pytest.mark.parametrize("entries", [100, 4000])
def test_group_rows_reports_numbers_past_the_last(entries):
    fq = _fq()
    ids = torch.arange(entries, dtype=torch.int32) % 9
    ids[5] = 9
    ids[7] = 2 ** 31 - 1
    with pytest.raises(fq.FP4QError, match="group"):
        fq.group_rows(ids.to(DEV), 9, check=True)
    r = fq.group_rows(ids.to(DEV), 9)
    off, rows = GR.group_rows(ids.numpy(), 9)
    np.testing.assert_array_equal(_np(r.offsets), off)
    np.testing.assert_array_equal(_np(r.rows), rows)


# ------------------------------------------------------ grouped products ----
def _held(rng, rows, k, scale=1.0):
    """MXFP4 operands made directly: every code, exponents over six steps."""
    codes = rng.integers(0, 256, (rows, k // 2)).astype(np.uint8)
    scales = rng.integers(122, 129, (rows, k // 32)).astype(np.uint8)
    return codes, scales


def _case(rng, tokens, groups, top_k, k, n, none=0.0):
    ids = np.stack([rng.permutation(groups)[:top_k] for _ in range(tokens)]).astype(np.int32)
    ids[rng.random(tokens) < none] = -1
    off, rows = GR.group_rows(ids, groups)
    bc, bs = _held(rng, groups * n, k)
    bh = GM.decode_mxfp4_64(bc, bs).reshape(groups, n, k)
    return ids, off, rows, (bc.reshape(groups, n, k // 2), bs.reshape(groups, n, k // 32)), bh


def _dev(*ts):
    return tuple(torch.from_numpy(np.ascontiguousarray(t)).to(DEV) for t in ts)


def _product_tol(ref, mag, k, gated):
    tol = (2 * math.ceil(k / 64) + 2) * U * mag
    if not gated:
        return ref, tol
    half = ref.shape[1] // 2
    g, u, tg, tu = ref[:, :half], ref[:, half:], tol[:, :half], tol[:, half:]
    with np.errstate(over="ignore"):
        s = GR.silu(g)
    tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(s) * tu + (np.abs(g) + 9) * U * np.abs(s * u)
    return s * u, tol + 2.0 ** -126 * (1 + np.abs(u))  # exponentials past float32's range: silu below its normals


PRODUCTS = [  # tokens, groups, top_k, k, n
    (1, 8, 2, 512, 256), (3, 60, 4, 704, 40), (16, 128, 8, 1024, 96), (17, 4, 1, 4096, 200), (64, 8, 2, 2048, 512),
    (100, 3, 2, 256, 130), (130, 16, 4, 1056, 66), (257, 5, 2, 128, 260), (300, 2, 1, 1536, 384), (700, 2, 2, 768, 320),
    (40, 200, 3, 32, 34), (9, 1, 1, 8192, 64), (1500, 6, 2, 640, 256), (33, 2, 2, 14336, 48),
    (100, 16, 4, 1024, 520), (64, 16, 4, 4096, 520), (90, 40, 6, 4608, 258), (500, 4, 1, 2048, 640),
    (4096, 6, 2, 512, 4000), (2900, 20, 3, 768, 4096), (3000, 3, 3, 1280, 3602),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,groups,top_k,k,n", PRODUCTS)
def test_grouped_product(tokens, groups, top_k, k, n, dtype):
    """Gathered and gated into the groups' order; from there scattered back; both with entries of no group."""
    fq = _fq()
    rng = np.random.default_rng(k + n)
    ids, off, rows, b, bh = _case(rng, tokens, groups, top_k, k, n, none=0.2 if tokens > 2 else 0.0)
    live, entries = int(off[-1]), tokens * top_k
    gr = fq.RowGroups(*_dev(off, rows))
    bd = _dev(*b)
    a = _held(rng, tokens, k)
    ref, mag = GR.products(GM.decode_mxfp4_64(*a), bh, off, rows, gather=top_k)
    for gated in (False, True):
        out = torch.full((entries, n // 2 if gated else n), 7.0, dtype=dtype, device=DEV)
        got = fq.gemm_mxfp4_grouped(_dev(*a), bd, gr, gather=top_k, gated=gated, alpha=0.0625, out=out, check=True)
        assert got is out and (out[live:] == 7.0).all()
        r, tol = _product_tol(0.0625 * ref, 0.0625 * mag, k, gated)
        _within(out[:live], r[:live], tol[:live], dtype)
    a = _held(rng, entries, k)
    ref, mag = GR.products(GM.decode_mxfp4_64(*a), bh, off, rows)
    out = torch.full((entries, n + 8), 7.0, dtype=dtype, device=DEV)
    fq.gemm_mxfp4_grouped(_dev(*a), bd, gr, scatter=True, out=out[:, :n], check=True)
    assert (out[:, n:] == 7.0).all() and (out[torch.from_numpy(rows[live:]).long().to(DEV)] == 7.0).all()
    r, tol = _product_tol(ref, mag, k, False)
    _within(out[torch.from_numpy(rows[:live]).long().to(DEV), :n], r[:live], tol[:live], dtype)


def test_grouped_product_matches_the_plain_one():
    """One group: gemm_mxfp4's product."""
    fq = _fq()
    a = fq.quantize_mxfp4(torch.randn(200, 1024, device=DEV))
    w = fq.quantize_mxfp4(torch.randn(300, 1024, device=DEV))
    gr = fq.RowGroups(torch.tensor([0, 200], dtype=torch.int32, device=DEV),
                      torch.arange(200, dtype=torch.int32, device=DEV))
    got = fq.gemm_mxfp4_grouped(a, (w.codes[None], w.scales[None]), gr, check=True)
    ref, mag = GR.products(GM.decode_mxfp4_64(*map(_np, a[:2])), GM.decode_mxfp4_64(*map(_np, w[:2]))[None], [0, 200],
                           np.arange(200))
    _within(got, ref, _product_tol(ref, mag, 1024, False)[1])
    assert torch.allclose(got, fq.gemm_mxfp4(a, w), rtol=1e-5, atol=1e-3)


@pytest.mark.parametrize("tokens,k,n", [(12, 1024, 128), (400, 512, 256), (90, 96, 64), (90, 4096, 2000),
                                        (4096, 512, 4096)])
def test_grouped_product_keeps_nan_to_its_row_and_column(tokens, k, n):
    fq = _fq()
    rng = np.random.default_rng(8)
    ids, off, rows, b, bh = _case(rng, tokens, 4, 2, k, n)
    a = _held(rng, tokens * 2, k)
    ref = fq.gemm_mxfp4_grouped(_dev(*a), _dev(*b), fq.RowGroups(*_dev(off, rows)))
    p, g = int(off[1]), 2
    a[1][p, 1] = 255
    b[1][g, 5, 0] = 255
    got = fq.gemm_mxfp4_grouped(_dev(*a), _dev(*b), fq.RowGroups(*_dev(off, rows)), check=True)
    nan = np.zeros(got.shape, bool)
    nan[p] = True
    nan[off[g]:off[g + 1], 5] = True
    assert np.array_equal(np.isnan(_np(got)), nan)
    assert np.array_equal(_np(got)[~nan], _np(ref)[~nan])


@pytest.mark.parametrize("tokens,k,n", [(20, 1024, 96), (500, 512, 256), (90, 96, 64), (90, 4096, 2000),
                                        (5000, 512, 4096)])
def test_grouped_product_with_bad_groups_stays_inside(tokens, k, n):
    """Offsets and rows out of range are reported and not followed; guards around C stay."""
    fq = _fq()
    rng = np.random.default_rng(9)
    ids, off, rows, b, bh = _case(rng, tokens, 6, 2, k, n)
    entries = tokens * 2
    a, bd = _dev(*_held(rng, tokens, k)), _dev(*b)
    for what in range(7):
        o, r = off.copy(), rows.copy()
        if what == 0:
            o[3] = 2 ** 31 - 1
        elif what == 1:
            o[2] = -2 ** 31
        elif what == 2:
            o[0] = 1
        elif what == 3:
            o[6] = entries + 1
        elif what == 4:
            r[3] = -1
        elif what == 5:
            r[4] = entries
        else:
            o[:], r[:] = rng.integers(-2 ** 31, 2 ** 31, 7), rng.integers(-2 ** 31, 2 ** 31, entries)
        for scatter in (False, True):
            big = torch.full((entries + 128, n), 3.0, device=DEV)
            with pytest.raises(fq.FP4QError, match="group"):
                fq.gemm_mxfp4_grouped(a, bd, fq.RowGroups(*_dev(o, r)), gather=2, scatter=scatter,
                                      out=big[64:64 + entries], check=True)
            assert (big[:64] == 3.0).all() and (big[64 + entries:] == 3.0).all()


@pytest.mark.parametrize("rows,groups,k,n", [(2 ** 21 + 77, 2, 4096, 32), (300, 3, 4096, 2 ** 20 - 24)])
def test_grouped_product_past_4_gib(rows, groups, k, n):
    """Rows of A, and matrices of B, that begin more than 2^32 bytes from the first."""
    fq = _fq()
    g = torch.Generator(device=DEV).manual_seed(3)
    held = lambda r: (torch.randint(0, 256, (r, k // 2), generator=g, dtype=torch.uint8, device=DEV),
                      torch.randint(122, 129, (r, k // 32), generator=g, dtype=torch.uint8, device=DEV))
    a, b = held(rows), held(groups * n)
    ids = (torch.arange(rows, device=DEV) % groups).int()
    gr = fq.group_rows(ids, groups)
    out = fq.gemm_mxfp4_grouped(a, (b[0].view(groups, n, -1), b[1].view(groups, n, -1)), gr, gather=1, scatter=True,
                                out_dtype=torch.bfloat16, check=True)
    pick = sorted({0, 1, 2, 150, rows // 2, rows - 2, rows - 1})
    cols = sorted({0, 1, 17, n // 2, n - 2, n - 1})
    hat = lambda t, i: GM.decode_mxfp4_64(_np(t[0][i]), _np(t[1][i]))
    ah = hat(a, pick)
    for i, e in enumerate(pick):
        bh = hat(b, [int(ids[e]) * n + c for c in cols])
        ref, mag = bh @ ah[i], np.abs(bh) @ np.abs(ah[i])
        _within(out[e, cols], ref, _product_tol(ref[None], mag[None], k, False)[1][0], torch.bfloat16)


def test_grouped_product_empty():
    fq = _fq()
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    b = (torch.zeros(3, 8, 16, dtype=torch.uint8, device=DEV), torch.zeros(3, 8, 1, dtype=torch.uint8, device=DEV))
    a = (torch.zeros(0, 16, dtype=torch.uint8, device=DEV), torch.zeros(0, 1, dtype=torch.uint8, device=DEV))
    assert fq.gemm_mxfp4_grouped(a, b, fq.RowGroups(off, z), check=True).shape == (0, 8)
    # entries, all of no group
    a = (torch.zeros(5, 16, dtype=torch.uint8, device=DEV), torch.zeros(5, 1, dtype=torch.uint8, device=DEV))
    out = torch.full((5, 8), 2.0, device=DEV)
    fq.gemm_mxfp4_grouped(a, b, fq.RowGroups(off, torch.arange(5, dtype=torch.int32, device=DEV)), out=out, check=True)
    assert (out == 2.0).all()


# --------------------------------------------------------- weighted sum ----
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,k,n", [(1, 1, 8), (3, 8, 4096), (33, 4, 2040), (5, 64, 100), (300, 6, 33), (2, 2, 1)])
def test_combine_experts(tokens, k, n, dtype, out_dtype):
    fq = _fq()
    g = torch.Generator().manual_seed(n)
    y = torch.randn(tokens, k, n, generator=g).to(dtype).to(DEV)
    w = torch.rand(tokens, k, generator=g).to(DEV)
    ids = torch.randint(-1, 5, (tokens, k), generator=g, dtype=torch.int32).to(DEV)
    add = torch.randn(tokens, n, generator=g).to(out_dtype).to(DEV)
    y[ids < 0] = float("nan")  # what a product leaves there
    for a in (None, add):
        got = fq.combine_experts(y, w, ids, add=a, out_dtype=out_dtype)
        ref, mag = GR.combine(_np(y), _np(w), _np(ids), None if a is None else _np(a))
        _within(got, ref, (k + 1) * U * mag, out_dtype)
    big = torch.zeros(tokens, n + 3, dtype=out_dtype, device=DEV)
    big[:, :n] = add
    fq.combine_experts(y, w, ids, add=big[:, :n], out=big[:, :n])  # into what is added
    assert torch.equal(big[:, :n], got) and (big[:, n:] == 0).all()
    y = torch.nan_to_num(y)
    ref, mag = GR.combine(_np(y), _np(w))
    _within(fq.combine_experts(y, w, out_dtype=out_dtype), ref, (k + 1) * U * mag, out_dtype)


# -------------------------------------------------------------- adapters ----
LORA = [  # rows, adapters, rank, k, n, none
    (1, 1, 16, 512, 256, 0.0), (1, 3, 8, 40, 7, 1.0), (5, 3, 8, 1000, 100, 0.4), (64, 32, 16, 4096, 512, 0.2),
    (64, 1, 64, 1024, 300, 0.0), (200, 3, 24, 2040, 130, 0.3), (300, 2, 128, 256, 640, 0.1), (1000, 5, 40, 768, 264, 0.2),
    (700, 1, 256, 512, 72, 0.0), (2000, 7, 16, 128, 1000, 0.5), (90, 100, 200, 64, 64, 0.2),
    # K shared by several workgroups whose rows the second kernel takes many at a time
    (700, 1, 64, 2048, 200, 0.1), (300, 1, 128, 4088, 96, 0.0), (400, 1, 208, 2040, 70, 0.3), (500, 2, 8, 1600, 516, 0.2),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,adapters,rank,k,n,none", LORA)
def test_lora_add(rows, adapters, rank, k, n, none, dtype):
    fq = _fq()
    g = torch.Generator().manual_seed(rows + k)
    ids = torch.randint(0, adapters, (rows,), generator=g, dtype=torch.int32)
    ids[torch.rand(rows, generator=g) < none] = -1
    x = torch.randn(rows, k, generator=g).bfloat16()
    y = torch.randn(rows, n, generator=g).to(dtype)
    a = (torch.randn(adapters, rank, k, generator=g) * k ** -0.5).bfloat16()
    b = torch.randn(adapters, n, rank, generator=g).bfloat16()
    sc = torch.rand(adapters, generator=g) + 0.5
    gr = fq.group_rows(ids.to(DEV), adapters, check=True)
    off, order = GR.group_rows(ids.numpy(), adapters)
    yd, xd, ad, bd = (t.to(DEV) for t in (y, x, a, b))
    for scales in (None, sc):
        got = fq.lora_add(yd, xd, ad, bd, gr, scales=None if scales is None else scales.to(DEV), check=True)
        ref, mag = GR.lora(_np(y), _np(x), _np(a), _np(b), off, order, None if scales is None else _np(scales))
        steps = k / 32 + 35 + 3 * rank / 32
        _within(got, ref, steps * U * mag + U * np.abs(_np(y)), dtype)
        assert torch.equal(got[ids < 0].cpu(), y[ids < 0])
    # in place, in a wider tensor whose rows are not aligned
    big = torch.full((rows, n + 3), 5.0, dtype=dtype, device=DEV)
    view = big[:, 1:n + 1]
    view.copy_(yd)
    same = fq.lora_add(view, xd, ad, bd, gr, scales=sc.to(DEV), out=view, check=True)
    assert same is view and torch.equal(view, got) and (big[:, 0] == 5.0).all() and (big[:, n + 1:] == 5.0).all()


def test_strided_broadcast_and_unaligned_operands():
    """Views that the calls read in place or copy: the result of dense ones."""
    fq = _fq()
    g = torch.Generator().manual_seed(12)
    w, ids = torch.rand(9, 3, generator=g).to(DEV), torch.randint(-1, 4, (9, 3), generator=g, dtype=torch.int32).to(DEV)
    big = torch.randn(9, 3, 80, generator=g).to(DEV)
    for y in (big[:, :, 3:43], big[:, :, 8:72], big.transpose(0, 1).contiguous().transpose(0, 1), big[:, :1].expand(9, 3, 80),
              big[..., ::2]):
        assert torch.equal(fq.combine_experts(y, w, ids), fq.combine_experts(y.contiguous(), w, ids))
    assert torch.equal(fq.combine_experts(big[:, :1, :40], w[:, :1].contiguous()),
                       fq.combine_experts(big[:, :1, :40].contiguous(), w[:, :1].contiguous()))
    x = torch.randn(300, 201, generator=g).bfloat16().to(DEV)
    a, b = torch.randn(2, 16, 128, generator=g).bfloat16().to(DEV), torch.randn(2, 96, 16, generator=g).bfloat16().to(DEV)
    gr = fq.group_rows((torch.arange(300, device=DEV) % 3 - 1).int(), 2)
    y = torch.randn(96, generator=g).to(DEV)
    for v in (x[:, 1:129], x[:, 8:136], x[:1, :128].expand(300, 128), x[:, :128].t().contiguous().t()):
        got = fq.lora_add(y.expand(300, 96), v, a, b, gr, check=True)
        assert torch.equal(got, fq.lora_add(y.repeat(300, 1), v.contiguous(), a, b, gr))
    codes = torch.randint(0, 256, (40, 96), generator=g, dtype=torch.uint8).to(DEV)
    scales = torch.randint(122, 129, (40, 8), generator=g, dtype=torch.uint8).to(DEV)
    m = (torch.randint(0, 256, (2, 24, 64), generator=g, dtype=torch.uint8).to(DEV),
         torch.randint(122, 129, (2, 24, 4), generator=g, dtype=torch.uint8).to(DEV))
    gr = fq.group_rows((torch.arange(40, device=DEV) % 2).int(), 2)
    got = fq.gemm_mxfp4_grouped((codes[:, 16:80], scales[:, 2:6]), m, gr, check=True)
    assert torch.equal(got, fq.gemm_mxfp4_grouped((codes[:, 16:80].contiguous(), scales[:, 2:6].contiguous()), m, gr))


def test_lora_add_keeps_non_finite_rows_to_themselves():
    fq = _fq()
    for rows in (20, 600):
        x, y = torch.randn(rows, 256, device=DEV).bfloat16(), torch.randn(rows, 128, device=DEV)
        a, b = torch.randn(2, 16, 256, device=DEV).bfloat16(), torch.randn(2, 128, 16, device=DEV).bfloat16()
        gr = fq.group_rows((torch.arange(rows, device=DEV) % 2).int(), 2)
        want = fq.lora_add(y, x, a, b, gr)
        x[3, 7], x[4, 9] = float("inf"), float("nan")
        y[9, 3] = float("inf")
        got = fq.lora_add(y, x, a, b, gr, check=True)
        rest = [i for i in range(rows) if i not in (3, 4, 9)]
        assert torch.equal(got[rest], want[rest])
        assert not torch.isfinite(got[3]).any() and torch.isnan(got[4]).all()
        assert got[9, 3] == float("inf") and torch.equal(got[9, 4:], want[9, 4:])


def test_lora_add_with_bad_groups_stays_inside():
    fq = _fq()
    rng = np.random.default_rng(2)
    for rows in (40, 900):
        x = torch.randn(rows, 128, device=DEV).bfloat16()
        a, b = torch.randn(3, 16, 128, device=DEV).bfloat16(), torch.randn(3, 72, 16, device=DEV).bfloat16()
        off, order = GR.group_rows(rng.integers(-1, 3, rows), 3)
        for what in range(5):
            o, r = off.copy(), order.copy()
            if what == 0:
                o[1] = 2 ** 31 - 1
            elif what == 1:
                o[2] = -7
            elif what == 2:
                r[0] = rows
            elif what == 3:
                r[1] = -2 ** 31
            else:
                o[:], r[:] = rng.integers(-2 ** 31, 2 ** 31, 4), rng.integers(-2 ** 31, 2 ** 31, rows)
            big = torch.full((rows + 128, 72), 3.0, device=DEV)
            with pytest.raises(fq.FP4QError, match="group"):
                fq.lora_add(torch.zeros(rows, 72, device=DEV), x, a, b, fq.RowGroups(*_dev(o, r)),
                            out=big[64:64 + rows], check=True)
            assert (big[:64] == 3.0).all() and (big[64 + rows:] == 3.0).all()


def test_lora_add_beside_a_product():
    """What a W4A4 projection with adapters runs: quantize, product, adapters in place."""
    fq = _fq()
    g = torch.Generator().manual_seed(6)
    x = torch.randn(70, 512, generator=g).bfloat16().to(DEV)
    w = fq.quantize_mxfp4(torch.randn(384, 512, generator=g).to(DEV))
    a = torch.randn(4, 16, 512, generator=g).bfloat16().to(DEV)
    b = torch.randn(4, 384, 16, generator=g).bfloat16().to(DEV)
    gr = fq.group_rows(torch.randint(-1, 4, (70,), generator=g, dtype=torch.int32).to(DEV), 4)
    y = fq.gemm_mxfp4(fq.quantize_mxfp4(x), w)
    base = _np(y)
    fq.lora_add(y, x, a, b, gr, out=y, check=True)
    ref, mag = GR.lora(base, _np(x), _np(a), _np(b), _np(gr.offsets), _np(gr.rows))
    _within(y, ref, (512 / 32 + 35 + 3) * U * mag + U * np.abs(base))
    empty = fq.lora_add(y[:0], x[:0], a, b, fq.group_rows(torch.zeros(0, dtype=torch.int32, device=DEV), 4), check=True)
    assert empty.shape == (0, 384)


# --------------------------------------------------- a layer of experts ----
def _layer(fq, x, logits, up, down, k, ws=None):
    """Route, gate and up products, activation, down products, sum; every step's result."""
    r = fq.route_experts(logits, k, score="sigmoid", bias=None, renormalize=True)
    z = fq.gemm_mxfp4_grouped(fq.quantize_mxfp4(x), up, r.groups, gather=k, gated=True, out_dtype=torch.bfloat16)
    y = fq.gemm_mxfp4_grouped(fq.quantize_mxfp4(z), down, r.groups, scatter=True, out_dtype=torch.bfloat16)
    return r, z, y, fq.combine_experts(y.view(len(x), k, -1), r.weights, r.experts, add=x)


def _layer_inputs(fq, tokens, experts, hidden, inner, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g).bfloat16().to(DEV)
    logits = torch.randn(tokens, experts, generator=g).to(DEV)
    up = fq.quantize_mxfp4((torch.randn(experts * 2 * inner, hidden, generator=g) * hidden ** -0.5).to(DEV))
    down = fq.quantize_mxfp4((torch.randn(experts * hidden, inner, generator=g) * inner ** -0.5).to(DEV))
    return (x, logits, (up.codes.view(experts, 2 * inner, -1), up.scales.view(experts, 2 * inner, -1)),
            (down.codes.view(experts, hidden, -1), down.scales.view(experts, hidden, -1)))


@pytest.mark.parametrize("tokens", [1, 7, 150])
def test_layer_of_experts(tokens):
    """Each step against 64 bits, from the operands that the step before handed on."""
    fq = _fq()
    experts, k, hidden, inner = 12, 3, 256, 192
    x, logits, up, down = _layer_inputs(fq, tokens, experts, hidden, inner, tokens)
    r, z, y, out = _layer(fq, x, logits, up, down, k)
    w, ids, _ = GR.route(_np(logits), k, score="sigmoid")
    np.testing.assert_array_equal(_np(r.experts), ids)
    off, rows = GR.group_rows(ids, experts)
    xq, zq = (fq.quantize_mxfp4(t) for t in (x, z))
    hat = lambda c, s: GM.decode_mxfp4_64(_np(c), _np(s))
    dec = lambda p: np.stack([hat(c, s) for c, s in zip(*p)])
    ref, mag = GR.products(hat(xq.codes, xq.scales), dec(up), off, rows, gather=k)
    ref, tol = _product_tol(ref, mag, hidden, True)
    _within(z, ref, tol, torch.bfloat16)
    ref, mag = GR.products(hat(zq.codes, zq.scales), dec(down), off, rows)
    _within(y[torch.from_numpy(rows).long().to(DEV)], ref, _product_tol(ref, mag, inner, False)[1], torch.bfloat16)
    ref, mag = GR.combine(_np(y).reshape(tokens, k, hidden), _np(r.weights), ids, _np(x))
    _within(out, ref, (k + 1) * U * mag, torch.bfloat16)


def test_layer_in_a_captured_graph_and_on_two_streams():
    """A layer and adapters captured and replayed with eager work between the replays; two graphs replayed at once;
    the same on two streams: every result equals the eager one."""
    fq = _fq()
    tokens, experts, k, hidden, inner = 300, 8, 2, 256, 128
    x, logits, up, down = _layer_inputs(fq, tokens, experts, hidden, inner, 5)
    a = torch.randn(3, 16, hidden, device=DEV).bfloat16()
    b = torch.randn(3, hidden, 16, device=DEV).bfloat16()
    ids = (torch.arange(tokens, device=DEV) % 4 - 1).int()

    def step(x, logits):
        out = _layer(fq, x, logits, up, down, k)[3]
        return fq.lora_add(out, x, a, b, fq.group_rows(ids, 3))

    xs = [x, x.clone()]
    ls = [logits, logits.clone()]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(xs[0], ls[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(xs[i], ls[i]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(4):
        want = []
        for j in range(2):
            ls[j].copy_(torch.randn(tokens, experts, generator=torch.Generator().manual_seed(10 * i + j)))
            xs[j].copy_(torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(20 * i + j)))
            want.append(step(xs[j], ls[j]).clone())
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for j in range(2):
            assert torch.equal(outs[j], want[j]), (i, j)
        got = []
        for j, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(step(xs[j], ls[j]))
        torch.cuda.synchronize()
        for j in range(2):
            assert torch.equal(got[j], want[j]), (i, j)


def test_refusals_of_the_binding_on_device_tensors():
    fq = _fq()
    x = torch.zeros(6, 64, device=DEV)
    gr = fq.RowGroups(torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV),
                      torch.arange(6, dtype=torch.int32, device=DEV))
    for bad in (dict(top_k=0), dict(top_k=65), dict(top_k=2, score="relu"), dict(top_k=2, bias=torch.zeros(3, device=DEV)),
                dict(top_k=2, bias=[0.0] * 64)):
        with pytest.raises(ValueError):
            fq.route_experts(x, **bad)
    with pytest.raises(ValueError):
        fq.route_experts(x.half(), 2)
    for bad in (dict(n_groups=3), dict(group_best=3), dict(scale=float("nan")), dict(n_groups=4, top_groups=5)):
        with pytest.raises(fq.FP4QError):
            fq.route_experts(x, 2, **bad)
    with pytest.raises(ValueError):
        fq.group_rows(torch.zeros(4, device=DEV), 2)
    with pytest.raises(fq.FP4QError):
        fq.group_rows(gr.rows, 3000)
    a = fq.quantize_mxfp4(x)
    b = (torch.zeros(2, 32, 32, dtype=torch.uint8, device=DEV), torch.zeros(2, 32, 2, dtype=torch.uint8, device=DEV))
    fq.gemm_mxfp4_grouped(a, b, gr, check=True)
    for bad in (None, gr.rows, (gr.offsets.long(), gr.rows), (gr.offsets, gr.rows.cpu()), (gr.offsets, gr.rows[::2])):
        with pytest.raises(ValueError):
            fq.gemm_mxfp4_grouped(a, b, bad)
    for bad in ((b[0][:1], b[1][:1]), (b[0], b[1][:1]), (b[0][:, :, :16].contiguous(), b[1]), (b[0].int(), b[1])):
        with pytest.raises(ValueError):
            fq.gemm_mxfp4_grouped(a, bad, gr)
    with pytest.raises(ValueError):
        fq.gemm_mxfp4_grouped(a, b, gr, out=torch.zeros(6, 31, device=DEV))
    with pytest.raises(ValueError):
        fq.gemm_mxfp4_grouped(a, b, gr, out=torch.zeros(32, 6, device=DEV).t())
    with pytest.raises(fq.FP4QError):
        fq.gemm_mxfp4_grouped((a.codes[:2], a.scales[:2]), b, gr, gather=2)
    with pytest.raises(fq.FP4QError):
        fq.gemm_mxfp4_grouped(a, b, gr, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    y3 = torch.zeros(3, 2, 8, device=DEV)
    for bad in (torch.zeros(3, 3, device=DEV), torch.zeros(3, 2, device=DEV).double()):
        with pytest.raises(ValueError):
            fq.combine_experts(y3, bad)
    with pytest.raises(ValueError):
        fq.combine_experts(y3, torch.zeros(3, 2, device=DEV), add=torch.zeros(3, 8, device=DEV).bfloat16())
    la, lb = torch.zeros(2, 8, 64, device=DEV).bfloat16(), torch.zeros(2, 16, 8, device=DEV).bfloat16()
    y, xb = torch.zeros(6, 16, device=DEV), x.bfloat16()
    fq.lora_add(y, xb, la, lb, gr, check=True)
    for bad in ((y, x, la, lb), (y, xb, la[:1], lb), (y, xb, la.float(), lb), (y[:5], xb, la, lb), (y, xb, la, lb[:, :8])):
        with pytest.raises(ValueError):
            fq.lora_add(*bad, gr)
    with pytest.raises(ValueError):
        fq.lora_add(y, xb, la, lb, gr, scales=torch.zeros(3, device=DEV))
    with pytest.raises(ValueError):
        fq.lora_add(y, xb, la, lb, gr, out=torch.zeros(6, 16, device=DEV).bfloat16())
