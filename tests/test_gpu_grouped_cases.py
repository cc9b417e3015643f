"""Cases of the grouped calls where a result depends on the last bits, on rows
of no group, or on a group far down the list, against the CPU oracle
(oracle/grouped.py).  u = 2^-24 is float32's half step, h a half step of the
result's type.
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
    # half a step of the result: relative, and below the normal range absolute
    tol = tol + HALF[dtype] * np.abs(ref) + (2.0 ** -150 if dtype == torch.float32 else 2.0 ** -134)
    err = np.abs(_np(got) - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), bad.size, float(np.nanmax(err / np.maximum(tol, 1e-300))))


def _dev(*ts):
    return tuple(torch.from_numpy(np.ascontiguousarray(t)).to(DEV) for t in ts)


# -------------------------------------------------------------- adapters ----
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,adapters,rank,k,n", [
    (20, 3, 8, 40, 36), (20, 2, 64, 4096, 36), (700, 2, 64, 40, 300), (700, 1, 128, 40, 72), (600, 2, 200, 40, 68),
    (300, 1, 128, 2048, 40), (9000, 2, 16, 40, 36),
])
def test_adapters_that_cancel_the_projection(rows, adapters, rank, k, n, dtype):
    """y is close to -s (x A^T) B^T, so that what is left shows every bit of x A^T: its sum in float32, the scale, then
    products of its 24 bits.  One rank carries all of it, x and A are positive: the steps' bound is
    (k / 32 + 35 + 3 rank / 32) u of s (x A^T) |B|^T."""
    fq = _fq()
    g = torch.Generator().manual_seed(rows + rank)
    ids = torch.randint(0, adapters, (rows,), generator=g, dtype=torch.int32)
    x = (0.1 + torch.rand(rows, k, generator=g)).bfloat16()
    a = (0.1 + torch.rand(adapters, rank, k, generator=g)).bfloat16()
    b = torch.zeros(adapters, n, rank)
    b[:, :, rank - 3] = torch.randn(adapters, n, generator=g)
    b = b.bfloat16()
    sc = torch.rand(adapters, generator=g) + 0.5
    off, order = GR.group_rows(ids.numpy(), adapters)
    away, _ = GR.lora(np.zeros((rows, n)), _np(x), _np(a), _np(b), off, order, _np(sc))
    y = torch.from_numpy(-away).to(dtype)
    ref, mag = GR.lora(_np(y), _np(x), _np(a), _np(b), off, order, _np(sc))
    yd, xd, ad, bd, sd = (t.to(DEV) for t in (y, x, a, b, sc))
    got = fq.lora_add(yd, xd, ad, bd, fq.group_rows(ids.to(DEV), adapters), scales=sd, check=True)
    _within(got, ref, (k / 32 + 35 + 3 * rank / 32) * U * mag + U * np.abs(_np(y)), dtype)


# --------------------------------------------------------------- routing ----
@pytest.mark.parametrize("experts,k", [(60, 4), (128, 8), (256, 8), (500, 6), (1024, 16)])
@pytest.mark.parametrize("tokens", [1, 20, 301])
def test_softmax_weights_are_rounded_once(experts, k, tokens):
    """A softmax that is not renormalised: float64 (its own steps below one u), rounded once; and the same bits with a
    bias of zeros, which changes no choice."""
    fq = _fq()
    g = torch.Generator().manual_seed(experts + tokens)
    for spread in (0.02, 1.5, 6.0):
        x = spread * torch.randn(tokens, experts, generator=g)
        x[torch.rand(x.shape, generator=g) < 0.1] = -math.inf
        for t in (x, x.bfloat16()):
            d = t.to(DEV)
            r = fq.route_experts(d, k, renormalize=False, scale=2.5, check=True)
            w, ids, _ = GR.route(_np(t), k, renormalize=False, scale=2.5)
            np.testing.assert_array_equal(_np(r.experts), ids)
            _within(r.weights, w, U * np.abs(w))
            if t.dtype == torch.float32:  # without equal logits, whose order a bias leaves to float64 scores
                z = fq.route_experts(d, k, renormalize=False, scale=2.5, bias=torch.zeros(experts, device=DEV))
                same = (z.experts == r.experts).all(1)
                assert same.float().mean() > 0.9 and torch.equal(z.weights[same], r.weights[same])


# ------------------------------------------------------ grouped products ----
_E2M1 = [0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _single(values, k):
    """MXFP4 rows of k whose first element is the value (an E2M1 number times a power of two), the rest zero."""
    codes, scales = np.zeros((len(values), k // 2), np.uint8), np.full((len(values), k // 32), 127, np.uint8)
    for i, v in enumerate(values):
        e = next(e for e in range(-8, 12) if abs(v) / 2.0 ** e in _E2M1)
        codes[i, 0] = _E2M1.index(abs(v) / 2.0 ** e) + 1 | (8 if v < 0 else 0)
        scales[i, 0] = 127 + e
    return codes, scales


@pytest.mark.parametrize("rows,k", [(7, 32), (7, 512), (700, 320), (700, 512)])
@pytest.mark.parametrize("alpha", [1.0, 0.9371, 0.0371, -1.3])
def test_gates_to_float32(rows, k, alpha):
    """silu(z) * up for z = alpha a b exactly known: z spans -125 .. 125, where exp(-z) leaves float32's range and
    silu(z), down to -92, does not.  silu: exp(-|z|) off by 2.4 u (its instruction by one unit), which z < 0 takes in
    full, then a product, a sum, a reciprocal and a product, one u each: 6.4 u; the product with up is the result's
    half step.  Below float32's normal range its steps count."""
    fq = _fq()
    gates = [s * v * 2.0 ** e for e in range(-5, 5) for v in _E2M1 for s in (1, -1)]
    n = len(gates)
    bc, bs = _single(gates + [1.0] * n, k)
    av = [(1.0, 1.5, 0.5, 1.0)[i % 4] for i in range(rows)]
    ac, as_ = _single(av, k)
    off, order = _dev(np.array([0, rows], np.int32), np.arange(rows, dtype=np.int32))
    got = fq.gemm_mxfp4_grouped(_dev(ac, as_), _dev(bc[None], bs[None]), fq.RowGroups(off, order), gated=True, alpha=alpha,
                                check=True)
    al = np.float32(alpha)
    z = (al * np.outer(av, gates).astype(np.float32)).astype(np.float64)
    up = (al * np.array(av, np.float32)[:, None]).astype(np.float64)
    e = np.exp(-np.abs(z))
    ref = np.where(z < 0, z * e, z) / (1.0 + e) * up
    _within(got, ref, 6.4 * U * np.abs(ref) + 2.0 ** -140)


def _poisoned(monkeypatch):
    """Fresh floating tensors hold NaN."""
    empty = torch.empty

    def fresh(*a, **kw):
        t = empty(*a, **kw)
        return t.fill_(math.nan) if t.is_floating_point() else t

    monkeypatch.setattr(torch, "empty", fresh)


SHAPES = [  # tokens, groups, top_k, k, n
    (9, 3, 2, 64, 40), (9, 3, 2, 512, 66), (100, 16, 4, 704, 130), (100, 16, 4, 1024, 520), (90, 40, 6, 4608, 258),
    (1500, 6, 2, 640, 256), (700, 2, 2, 768, 320), (4096, 6, 2, 512, 4000),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,groups,top_k,k,n", SHAPES)
def test_fresh_rows_of_no_group_are_zeros(tokens, groups, top_k, k, n, dtype, monkeypatch):
    """Half of the entries, and all of them, of no group: their rows of a result that the call makes are zeros, in the
    groups' order and scattered; the others are what a given result gets."""
    fq = _fq()
    rng = np.random.default_rng(k)
    ids = np.stack([rng.permutation(groups)[:top_k] for _ in range(tokens)]).astype(np.int32)
    ids[rng.random(ids.shape) < 0.5] = -1
    a = (rng.integers(0, 256, (tokens, k // 2)).astype(np.uint8), rng.integers(122, 129, (tokens, k // 32)).astype(np.uint8))
    b = (rng.integers(0, 256, (groups, n, k // 2)).astype(np.uint8),
         rng.integers(122, 129, (groups, n, k // 32)).astype(np.uint8))
    a, b = _dev(*a), _dev(*b)
    for which in (ids, np.full_like(ids, -1)):
        off, order = GR.group_rows(which, groups)
        live, gr = int(off[-1]), fq.RowGroups(*_dev(off, order))
        rows = torch.from_numpy(order).long().to(DEV)
        for gated in (False, True):
            for scatter in (False, True):
                given = torch.full((tokens * top_k, n // 2 if gated else n), 7.0, dtype=dtype, device=DEV)
                kw = dict(gather=top_k, gated=gated, scatter=scatter, alpha=0.0625, check=True)
                fq.gemm_mxfp4_grouped(a, b, gr, out=given, **kw)
                with monkeypatch.context() as m:
                    _poisoned(m)
                    got = fq.gemm_mxfp4_grouped(a, b, gr, out_dtype=dtype, **kw)
                if scatter:
                    got, given = got[rows], given[rows]
                assert (given[live:] == 7.0).all()
                assert (got[live:] == 0.0).all() and torch.equal(got[:live], given[:live])


@pytest.mark.parametrize("tokens", [5, 40, 200])
def test_layer_of_experts_with_padding(tokens, monkeypatch):
    """Tokens that are padding (every expert off), tokens with fewer experts than choices, and an expert that nobody may
    use, through every step of a layer, whose data errors are all looked at."""
    fq = _fq()
    experts, k, hidden, inner = 12, 3, 256, 192
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, hidden, generator=g).bfloat16().to(DEV)
    logits = torch.randn(tokens, experts, generator=g)
    logits[torch.rand(tokens, generator=g) < 0.3] = -math.inf
    logits[0], logits[1, 2:], logits[:, 7] = -math.inf, -math.inf, -math.inf
    logits = logits.to(DEV)
    up = fq.quantize_mxfp4((torch.randn(experts * 2 * inner, hidden, generator=g) * hidden ** -0.5).to(DEV))
    down = fq.quantize_mxfp4((torch.randn(experts * hidden, inner, generator=g) * inner ** -0.5).to(DEV))
    up = (up.codes.view(experts, 2 * inner, -1), up.scales.view(experts, 2 * inner, -1))
    down = (down.codes.view(experts, hidden, -1), down.scales.view(experts, hidden, -1))
    with monkeypatch.context() as m:
        _poisoned(m)
        r = fq.route_experts(logits, k, score="sigmoid", check=True)
        xq = fq.quantize_mxfp4(x, check=True)
        z = fq.gemm_mxfp4_grouped(xq, up, r.groups, gather=k, gated=True, out_dtype=torch.bfloat16, check=True)
        zq = fq.quantize_mxfp4(z, check=True)
        y = fq.gemm_mxfp4_grouped(zq, down, r.groups, scatter=True, out_dtype=torch.bfloat16, check=True)
        out = fq.combine_experts(y.view(tokens, k, hidden), r.weights, r.experts, add=x)
        bare = fq.combine_experts(y.view(tokens, k, hidden), r.weights, add=x)
    w, ids, _ = GR.route(_np(logits), k, score="sigmoid")
    np.testing.assert_array_equal(_np(r.experts), ids)
    assert (ids == -1).any() and torch.equal(out, bare)
    off, rows = GR.group_rows(ids, experts)
    live = int(off[-1])
    hat = lambda c, s: GM.decode_mxfp4_64(_np(c), _np(s))
    dec = lambda p: np.stack([hat(c, s) for c, s in zip(*p)])
    ref, mag = GR.products(hat(zq.codes, zq.scales), dec(down), off, rows)
    want, size = np.zeros((tokens * k, hidden)), np.zeros((tokens * k, hidden))
    want[rows[:live]], size[rows[:live]] = ref[:live], mag[:live]
    _within(y, want, (2 * math.ceil(inner / 64) + 2) * U * size, torch.bfloat16)
    ref, mag = GR.combine(_np(y).reshape(tokens, k, hidden), _np(r.weights), ids, _np(x))
    _within(out, ref, (k + 1) * U * mag, torch.bfloat16)
    assert torch.equal(out[0], x[0])


FAR = [  # groups, rows a group, k, n: more groups than one step of the search takes
    (65, 30, 512, 300), (70, 28, 704, 260), (200, 10, 512, 130), (200, 10, 704, 130), (80, 12, 4096, 300),
    (70, 80, 768, 64), (70, 80, 640, 64), (65, 200, 512, 498), (130, 200, 512, 758), (512, 200, 512, 256),
    (513, 200, 512, 256), (2048, 3, 512, 40), (2048, 3, 96, 40),
]


@pytest.mark.parametrize("empty", [False, True])
@pytest.mark.parametrize("groups,rows,k,n", FAR)
def test_groups_past_the_first_64(groups, rows, k, n, empty):
    """Groups of different lengths, and runs of empty ones across every step of 64: around those places, at both ends and
    at random ones, results against 64 bits; rows past the last group stay."""
    fq = _fq()
    rng = np.random.default_rng(groups + k)
    share = rng.uniform(0.5, 1.5, groups)
    if empty:
        for g in range(60, groups, 64):
            share[g:g + 8] = 0
        share[0] = share[-1] = 0
    counts = rng.multinomial(groups * rows - 3, share / share.sum())
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    live = int(off[-1])
    entries, tokens = live + 3, 64
    gather = -(-entries // tokens)
    order = rng.permutation(entries).astype(np.int32)
    a = (rng.integers(0, 256, (tokens, k // 2)).astype(np.uint8), rng.integers(122, 129, (tokens, k // 32)).astype(np.uint8))
    b = (rng.integers(0, 256, (groups, n, k // 2)).astype(np.uint8),
         rng.integers(122, 129, (groups, n, k // 32)).astype(np.uint8))
    ah = GM.decode_mxfp4_64(*a)
    out = torch.full((entries, n), math.nan, device=DEV)
    fq.gemm_mxfp4_grouped(_dev(*a), _dev(*b), fq.RowGroups(*_dev(off, order)), gather=gather, out=out, check=True)
    assert out[live:].isnan().all() and not out[:live].isnan().any()
    near = {g + d for g in list(range(0, groups, 64)) + [groups] for d in (-3, -2, -1, 0, 1, 4, 5)}
    look = sorted({g for g in near if 0 <= g < groups} | set(rng.integers(0, groups, 12).tolist()))
    got = _np(out)
    for g in look:
        p = slice(int(off[g]), int(off[g + 1]))
        x, w = ah[order[p] // gather], GM.decode_mxfp4_64(b[0][g], b[1][g])
        ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
        err = np.abs(got[p] - ref)
        assert (err <= (2 * math.ceil(k / 64) + 3) * U * mag).all(), g
