"""Host-only checks of the key/value cache calls (no GPU): the header's
functions are exported, bad arguments are refused before anything is
enqueued, and the index arithmetic that the kernels share with the host
(csrc/fp4q_kv_host.h) stays inside the given tensors whatever the sequence
lengths, row offsets and sizes say, and hands out every key tile once."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp4_post_quantization_amd", "csrc")


def _lib():
    from fp4_post_quantization_amd import _lib as L
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("libfp4q.so not built (run __graft_entry__.build())")
    return L, L.load()


def test_header_and_exports_agree():
    L, lib = _lib()
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp4q_kv.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fp4q_[a-z0-9_]+)\s*\(", text))
    assert names == set(L.KV_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


# fake, aligned device addresses: validation must reject before any use
X, OUT, WS, IDX = 0x10000, 0x20000, 0x40000, 0x60000


def _cache(L, **kw):
    a = dict(kc=X, ks=X, vc=X, vs=X, pages=4, page=64, heads=2, dim=128, ps=64 * 2 * 64, hs=64 * 64, ts=64)
    a.update(kw)
    return L.KVCacheStruct(*a.values())


def _map(L, **kw):
    a = dict(w=None, eps=1e-6, pos=IDX, table=X, n=100, rot=128, inter=0, had=0)
    a.update(kw)
    return L.HeadMapStruct(*a.values())


def _rotate(L, lib, m=None, **kw):
    a = dict(x=X, dtype=L.BF16, tokens=3, heads=2, dim=128, st=256, sh=128)
    o = dict(odtype=L.BF16, out=OUT, ws=WS, wsb=lib.fp4q_workspace_bytes())
    for k, v in kw.items():
        (a if k in a else o)[k] = v
    return lib.fp4q_rotate_heads(*a.values(), ctypes.byref(_map(L, **(m or {}))), *o.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), "ERR_NULL"), (dict(out=None), "ERR_NULL"), (dict(ws=None), "ERR_WORKSPACE"),
    (dict(wsb=16), "ERR_WORKSPACE"), (dict(ws=WS + 4), "ERR_WORKSPACE"), (dict(dtype=9), "ERR_ARG"),
    (dict(odtype=-1), "ERR_ARG"), (dict(dim=96), "ERR_SHAPE"), (dict(tokens=-1), "ERR_SHAPE"),
    (dict(heads=70000), "ERR_SHAPE"), (dict(tokens=1 << 30), "ERR_SHAPE"), (dict(st=-256), "ERR_SHAPE"),
    (dict(st=100), "ERR_ALIGN"), (dict(x=X + 8), "ERR_ALIGN"), (dict(out=OUT + 8), "ERR_ALIGN"),
])
def test_rotate_refusals(kw, want):
    L, lib = _lib()
    assert _rotate(L, lib, **kw) == getattr(L, want)


@pytest.mark.parametrize("m,want", [
    (dict(rot=8), "ERR_SHAPE"), (dict(rot=144), "ERR_SHAPE"), (dict(table=None), "ERR_NULL"),
    (dict(pos=None), "ERR_NULL"), (dict(rot=0), "ERR_SHAPE"), (dict(n=0), "ERR_SHAPE"), (dict(inter=2), "ERR_ARG"),
    (dict(had=48), "ERR_ARG"), (dict(w=X, eps=-1.0), "ERR_ARG"), (dict(w=X, eps=float("nan")), "ERR_ARG"),
    (dict(w=X + 4), "ERR_ALIGN"), (dict(table=X + 8), "ERR_ALIGN"), (dict(pos=IDX + 4), "ERR_ALIGN"),
])
def test_map_refusals(m, want):
    L, lib = _lib()
    assert _rotate(L, lib, m=m) == getattr(L, want)


@pytest.mark.parametrize("dim,most", [(64, 1 << 21), (128, 1 << 20), (256, 1 << 19)])
def test_sizes_that_a_launch_could_not_cover_are_refused(dim, most):
    """2^33 elements and more, among them counts whose product passes 64 bits."""
    L, lib = _lib()
    c = _cache(L, heads=64, dim=dim, ps=dim // 2 * 64 * 64, hs=dim // 2 * 64, ts=dim // 2)
    wsb, st = lib.fp4q_workspace_bytes(), 64 * dim
    for tokens in (most, 1 << 30, 1 << 40, (1 << 58) + 1, (1 << 62) + 1):
        assert _rotate(L, lib, tokens=tokens, heads=64, dim=dim, st=st, sh=dim) == L.ERR_SHAPE
        assert lib.fp4q_kv_append_mxfp4(ctypes.byref(c), X, st, dim, X, st, dim, L.BF16, tokens, IDX,
                                        ctypes.byref(_map(L, rot=64)), -1, 0, WS, wsb, None) == L.ERR_SHAPE
        assert lib.fp4q_kv_read_mxfp4(ctypes.byref(c), IDX, tokens, L.BF16, OUT, OUT, WS, wsb, None) == L.ERR_SHAPE
        assert lib.fp4q_attention_mxfp4_workspace_bytes(tokens, 1, 64, 64, dim, 1, 64, 0) == 0
    assert lib.fp4q_attention_mxfp4_workspace_bytes(most - 1, 1, 64, 64, dim, 1, 64, 0) > 0


def test_more_units_than_a_launch_has_workgroups_are_split():
    """2^21 sequences of one token and 32 heads: a workgroup a unit would be 2^26 of them."""
    L, lib = _lib()
    f = lib.fp4q_attention_mxfp4_workspace_bytes
    one = f(1 << 17, 1 << 17, 32, 32, 64, 1, 64, 0)
    many = f(1 << 21, 1 << 21, 32, 32, 64, 1, 64, 0)
    assert one == 256 < many < 1 << 23
    # sequences without tokens have no units
    assert f(4, 1 << 23, 8, 8, 64, 1, 64, 0) == 256


def test_workspace_of_windows_that_a_call_refuses_is_zero():
    """From 2^31 on, where a window and the new tokens behind it could pass 63 bits as well."""
    L, lib = _lib()
    f = lib.fp4q_attention_mxfp4_workspace_bytes
    assert f(8, 8, 8, 2, 128, 1, 4096, (1 << 31) - 1) == f(8, 8, 8, 2, 128, 1, 4096, 0) > 0
    for window in (1 << 31, (1 << 63) - 1):
        assert f(8, 8, 8, 2, 128, 1, 4096, window) == 0
        assert _attend(L, lib, window=window) == L.ERR_ARG


def test_calls_without_new_tokens_are_not_split():
    """max_new 0 on a long cache has no units, so no partial results and no second kernel, which would have a grid
    without workgroups."""
    L, lib = _lib()
    for dim in (64, 128, 256):
        assert lib.fp4q_attention_mxfp4_workspace_bytes(5, 3, 32, 8, dim, 0, 100000, 0) == 256


@pytest.mark.parametrize("tokens,heads,st,sh", [
    (1 << 26, 1, 1 << 40, 64), (1 << 26, 1, 1 << 36, 64), (2, 1, 1 << 61, 64), (1, 1 << 16, 64, 1 << 46),
    (1 << 13, 1 << 13, 1 << 47, 1 << 47), (3, 2, (1 << 63) - 16, 64),
])
def test_strides_whose_offsets_pass_63_bits_are_refused(tokens, heads, st, sh):
    """The last element's byte offset is checked as a whole, not stride by stride."""
    L, lib = _lib()
    for dtype in (L.BF16, L.F32):
        assert _rotate(L, lib, m=dict(rot=64), tokens=tokens, heads=heads, dim=64, st=st, sh=sh,
                       dtype=dtype) == L.ERR_SHAPE
    assert _attend(L, lib, tst=1 << 61) == L.ERR_SHAPE
    assert _attend(L, lib, tokens=1 << 20, batch=1 << 20, tst=1 << 41) == L.ERR_SHAPE


def test_map_hadamard_wider_than_the_head():
    L, lib = _lib()
    assert _rotate(L, lib, m=dict(rot=64, had=128), dim=64, st=128, sh=64) == L.ERR_SHAPE


CACHE_FAULTS = [
    (dict(kc=None), "ERR_NULL"), (dict(vs=None), "ERR_NULL"), (dict(dim=32), "ERR_SHAPE"), (dict(heads=0), "ERR_SHAPE"),
    (dict(page=48), "ERR_SHAPE"), (dict(page=8), "ERR_SHAPE"), (dict(page=2048), "ERR_SHAPE"),
    (dict(pages=0), "ERR_SHAPE"), (dict(pages=1 << 32), "ERR_SHAPE"), (dict(ts=-64), "ERR_SHAPE"),
    (dict(ts=48), "ERR_SHAPE"),                       # rows overlap
    (dict(hs=64 * 32), "ERR_SHAPE"),                  # heads overlap
    (dict(ps=64 * 64), "ERR_SHAPE"),                  # pages overlap
    (dict(ts=72, hs=72 * 64, ps=72 * 128), "ERR_ALIGN"), (dict(kc=X + 4), "ERR_ALIGN"),
]


@pytest.mark.parametrize("c,want", CACHE_FAULTS)
def test_cache_refusals(c, want):
    L, lib = _lib()
    c = _cache(L, **c)
    wsb = lib.fp4q_workspace_bytes()
    assert lib.fp4q_kv_append_mxfp4(ctypes.byref(c), X, 256, 128, X, 256, 128, L.BF16, 3, IDX,
                                    ctypes.byref(_map(L)), -1, 0, WS, wsb, None) == getattr(L, want)
    assert lib.fp4q_kv_read_mxfp4(ctypes.byref(c), IDX, 3, L.BF16, OUT, OUT, WS, wsb, None) == getattr(L, want)
    assert _attend(L, lib, c) == getattr(L, want)


def test_append_and_read_refusals():
    L, lib = _lib()
    c = _cache(L)
    wsb = lib.fp4q_workspace_bytes()

    def app(k=X, st=256, sh=128, dtype=L.BF16, tokens=3, slots=IDX, lo=-1, hi=0, ws=WS, v=X):
        return lib.fp4q_kv_append_mxfp4(ctypes.byref(c), k, st, sh, v, 256, 128, dtype, tokens, slots,
                                        ctypes.byref(_map(L)), lo, hi, ws, wsb, None)
    assert app(k=None) == L.ERR_NULL and app(v=None) == L.ERR_NULL and app(slots=None) == L.ERR_NULL
    assert app(lo=1) == L.ERR_ARG and app(hi=-1) == L.ERR_ARG and app(lo=-17) == L.ERR_ARG and app(hi=17) == L.ERR_ARG
    assert app(st=4) == L.ERR_ALIGN and app(slots=IDX + 4) == L.ERR_ALIGN and app(v=X + 2) == L.ERR_ALIGN
    assert app(ws=None) == L.ERR_WORKSPACE and app(dtype=5) == L.ERR_ARG and app(tokens=-1) == L.ERR_SHAPE

    def read(slots=IDX, tokens=3, odt=L.BF16, k=OUT, v=OUT, ws=WS):
        return lib.fp4q_kv_read_mxfp4(ctypes.byref(c), slots, tokens, odt, k, v, ws, wsb, None)
    assert read(slots=None) == L.ERR_NULL and read(k=None, v=None) == L.ERR_NULL and read(odt=3) == L.ERR_ARG
    assert read(tokens=-2) == L.ERR_SHAPE and read(k=OUT + 8) == L.ERR_ALIGN and read(ws=None) == L.ERR_WORKSPACE


def _attend(L, lib, c=None, **kw):
    c = c or _cache(L)
    a = dict(q=X, qst=512, qsh=128, tokens=3, heads=4, table=IDX, tst=4, width=4, batch=3, lens=IDX, cu=None, new=1,
             len=256, scale=0.1, causal=1, window=0, out=OUT, lse=None, ws=WS, wsb=1 << 40)
    a.update(kw)
    return lib.fp4q_attention_mxfp4(ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), "ERR_NULL"), (dict(table=None), "ERR_NULL"), (dict(lens=None), "ERR_NULL"),
    (dict(out=None), "ERR_NULL"), (dict(heads=3), "ERR_SHAPE"), (dict(heads=1), "ERR_SHAPE"),
    (dict(tokens=-1), "ERR_SHAPE"), (dict(tokens=4), "ERR_SHAPE"), (dict(batch=-1), "ERR_SHAPE"),
    (dict(new=4), "ERR_SHAPE"), (dict(new=0), "ERR_SHAPE"), (dict(new=-1), "ERR_SHAPE"),
    (dict(len=257), "ERR_SHAPE"), (dict(len=-1), "ERR_SHAPE"), (dict(width=-1), "ERR_SHAPE"),
    (dict(tst=3), "ERR_SHAPE"), (dict(causal=2), "ERR_ARG"), (dict(window=-1), "ERR_ARG"),
    (dict(scale=float("inf")), "ERR_ARG"), (dict(scale=float("nan")), "ERR_ARG"), (dict(qst=500), "ERR_ALIGN"),
    (dict(q=X + 2), "ERR_ALIGN"), (dict(out=OUT + 4), "ERR_ALIGN"), (dict(table=IDX + 2), "ERR_ALIGN"),
    (dict(lse=OUT + 2), "ERR_ALIGN"), (dict(ws=None), "ERR_WORKSPACE"), (dict(wsb=64), "ERR_WORKSPACE"),
    (dict(ws=WS + 8), "ERR_WORKSPACE"), (dict(cu=IDX + 1), "ERR_ALIGN"),
])
def test_attention_refusals(kw, want):
    L, lib = _lib()
    assert _attend(L, lib, **kw) == getattr(L, want)


@pytest.mark.parametrize("scale", [1.8e38, -1.8e38, 2.5e38, 3e38])
def test_scales_that_overflow_in_units_of_log_2_are_refused(scale):
    """scale * log2(e) has to be a finite float32: 2^127 and less in magnitude are."""
    L, lib = _lib()
    assert _attend(L, lib, scale=scale) == L.ERR_ARG


def test_attention_workspace_of_invalid_sizes_is_zero():
    L, lib = _lib()
    f = lib.fp4q_attention_mxfp4_workspace_bytes
    assert f(8, 8, 8, 2, 128, 1, 4096, 0) >= 256
    for bad in ((-1, 8, 8, 2, 128, 1, 64, 0), (8, 8, 7, 2, 128, 1, 64, 0), (8, 8, 8, 2, 80, 1, 64, 0),
                (8, 8, 8, 0, 128, 1, 64, 0), (8, 8, 8, 2, 128, 9, 64, 0), (8, 8, 8, 2, 128, 1, 1 << 31, 0),
                (8, 8, 8, 2, 128, 1, 64, -1)):
        assert f(*bad) == 0


# ------------------------------------------------- the binding's checks ----
def test_packed_structs_are_the_ctypes_ones():
    L, _ = _lib()
    args = (1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11)
    assert L.KV_CACHE_PACK(*args) == bytes(L.KVCacheStruct(*args))
    args = (1, 0.5, 3, 4, 5, 6, 1, 8)
    assert L.HEAD_MAP_PACK(*args) == bytes(L.HeadMapStruct(*args))


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import fp4_post_quantization_amd as fq
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):
        fq.rotate_heads(x)
    cache = fq.kv_cache_mxfp4(2, 1, 16, 64, device="cpu")
    assert cache.k_codes.shape == (2, 1, 16, 32) and cache.v_scales.shape == (2, 1, 16, 2)
    with pytest.raises(ValueError, match="device"):
        fq.kv_read_mxfp4(cache, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="together"):
        fq._head_map(2, 64, torch.device("cpu"), torch.zeros(2, dtype=torch.int64), None, False, None, 0.0, 0)
    with pytest.raises(ValueError, match="table"):
        fq._head_map(2, 64, torch.device("cpu"), torch.zeros(2, dtype=torch.int64), torch.zeros(4, 64).double(), False,
                     None, 0.0, 0)
    with pytest.raises(ValueError, match="positions"):
        fq._head_map(2, 64, torch.device("cpu"), torch.zeros(3, dtype=torch.int64), torch.zeros(4, 64), False, None,
                     0.0, 0)


# ------------------------------------------------ index arithmetic, on the host ----
_PROGRAM = r"""
#include "fp4q_kv_host.h"
using namespace fp4q;
extern "C" void seq(const int64_t *s, int64_t len, int64_t begin, int64_t end, int64_t rows, int64_t tile, int64_t *o) {
  AttnShape a{s[0], (int)s[1], (int)s[2], (int)s[3], (int)s[4], (int)s[5], (int)s[6], (int)s[7]};
  AttnSeq q = attn_seq(a, (int)len, begin, end);
  AttnWork w = attn_work(a, q, (int)rows, (int)tile);
  o[0] = q.first; o[1] = q.fresh; o[2] = q.len; o[3] = q.bad; o[4] = w.row_tiles; o[5] = w.lo; o[6] = w.n;
}
extern "C" void keys(const int64_t *s, int64_t len, int64_t begin, int64_t end, int64_t i, int64_t *o) {
  AttnShape a{s[0], (int)s[1], (int)s[2], (int)s[3], (int)s[4], (int)s[5], (int)s[6], (int)s[7]};
  AttnSeq q = attn_seq(a, (int)len, begin, end);
  o[0] = attn_lo(a, q, (int)i); o[1] = attn_hi(a, q, (int)i);
}
extern "C" int64_t cut(int64_t total, int64_t spans, int64_t i) { return attn_cut(total, spans, i); }
extern "C" void part(int64_t from, int64_t to, int64_t n, int64_t *o) {
  AttnPart p = attn_part(from, to, (int)n); o[0] = p.t0; o[1] = p.t1;
}
extern "C" int64_t div_by(int64_t n, int64_t d) { return divide((uint32_t)n, make_divider((uint32_t)d)); }
extern "C" int64_t unit_cost() { return kUnitCost; }
extern "C" int64_t worth(int64_t total, int64_t spans) { return attn_spans(total, (int)spans); }
extern "C" int64_t span_of(int64_t total, int64_t spans, int64_t p) { return attn_span_of(total, spans, p); }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("kvhost")
    src, so = d / "host.cpp", d / "host.so"
    src.write_text(_PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-shared", "-fPIC", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(so)],
                   check=True)
    lib = ctypes.CDLL(str(so))
    P, I = ctypes.c_void_p, ctypes.c_int64
    lib.seq.argtypes, lib.keys.argtypes = [P, I, I, I, I, I, P], [P, I, I, I, I, P]
    lib.part.argtypes, lib.unit_cost.restype = [I, I, I, P], I
    lib.div_by.argtypes, lib.div_by.restype = [I, I], I
    lib.worth.argtypes, lib.worth.restype = [I, I], I
    for f in (lib.cut, lib.span_of):
        f.argtypes, f.restype = [I, I, I], I
    return lib


def _shape(tokens, batch, groups, heads, max_new, max_len, causal, window):
    return np.array([tokens, batch, groups, heads, max_new, max_len, causal, window], dtype=np.int64)


def _seq(host, s, length, begin, end, rows=16, tile=64):
    o = np.zeros(7, dtype=np.int64)
    host.seq(s.ctypes.data, length, begin, end, rows, tile, o.ctypes.data)
    return dict(zip(("first", "fresh", "len", "bad", "row_tiles", "lo", "n"), o.tolist()))


I32 = 2 ** 31 - 1


@pytest.mark.parametrize("causal,window", [(1, 0), (0, 0), (1, 1), (1, 100), (0, 7), (1, I32)])
def test_bad_lengths_and_offsets_stay_inside(host, causal, window):
    """Whatever a device tensor holds, rows stay in q and keys below max_len."""
    rng = np.random.default_rng(3)
    s = _shape(40, 3, 4, 2, 9, 500, causal, window)
    edge = [-(2 ** 31), -1, 0, 1, 8, 9, 39, 40, 41, 499, 500, 501, I32]
    for _ in range(3000):
        length, begin, end = (int(rng.choice(edge)) if rng.random() < 0.7 else int(rng.integers(0, 500))
                              for _ in range(3))
        r = _seq(host, s, length, begin, end)
        assert 0 <= r["len"] <= 500 and 0 <= r["fresh"] <= 9
        assert 0 <= r["first"] and r["first"] + r["fresh"] <= 40
        good = 0 <= length <= 500 and 0 <= begin <= end <= 40 and end - begin <= 9
        assert r["bad"] == (not good)
        if good:
            assert (r["len"], r["first"], r["fresh"]) == (length, begin, end - begin)
        assert r["row_tiles"] == -(-r["fresh"] * 4 // 16)
        assert r["n"] >= 1 and r["lo"] >= 0
        o = np.zeros(2, dtype=np.int64)
        for i in range(r["fresh"]):
            host.keys(s.ctypes.data, length, begin, end, i, o.ctypes.data)
            p = r["len"] - r["fresh"] + i
            want = [j for j in range(r["len"]) if (not causal or j <= p) and (not window or j > p - window)]
            assert list(range(max(0, o[0]), o[1])) == want
            assert 0 <= o[0] <= r["len"] and 0 <= o[1] <= r["len"]
            if want:  # the tiles of the sequence cover every visible key
                assert r["lo"] * 64 <= want[0] and want[-1] < (r["lo"] + r["n"]) * 64


def test_spans_cover_the_work_once(host):
    for total in (0, 1, 5, 511, 512, 513, 100003, 2 ** 40 + 7):
        for spans in (1, 3, 512):
            cuts = [host.cut(total, spans, i) for i in range(spans + 1)]
            assert cuts[0] == 0 and cuts[-1] == total
            sizes = {b - a for a, b in zip(cuts, cuts[1:])}
            assert min(sizes) >= 0 and max(sizes) - min(sizes) <= 1
            assert sorted(cuts) == cuts
            for i, (a, b) in enumerate(zip(cuts, cuts[1:])):
                for p in {a, b - 1} if b > a else ():
                    assert host.span_of(total, spans, p) == i


def test_units_of_spans_cover_every_tile_once_and_join(host):
    """The walk of the attention kernel over its work: every key tile of every unit is taken by one span; the parts of
    a unit that several spans share lie in the slots that the joining kernel reads, from the span that has its first
    tile to the span that its work ends in."""
    rng = np.random.default_rng(5)
    cost, o = host.unit_cost(), np.zeros(2, dtype=np.int64)
    for trial in range(60):
        tiles = rng.integers(1, [2, 5, 40, 700][trial % 4] + 1, rng.integers(1, 60)).tolist()
        spans = int(rng.choice([1, 2, 7, 64, 256]))
        starts = np.concatenate([[0], np.cumsum([n + cost for n in tiles])])
        total = int(starts[-1])
        spans = host.worth(total, spans)
        seen = [np.zeros(n, dtype=int) for n in tiles]
        parts = {}   # slot -> unit, tiles
        joins = {}
        for s in range(spans):
            pos, end = host.cut(total, spans, s), host.cut(total, spans, s + 1)
            while pos < end:
                u = int(np.searchsorted(starts, pos, side="right")) - 1
                size, frm = tiles[u] + cost, pos - int(starts[u])
                here = min(end - pos, size - frm)
                host.part(frm, frm + here, tiles[u], o.ctypes.data)
                t0, t1 = int(o[0]), int(o[1])
                pos += here
                if t0 == t1:
                    continue
                seen[u][t0:t1] += 1
                if (t0, t1) != (0, tiles[u]):
                    slot = 2 * s + (1 if t0 == 0 else 0)
                    assert slot not in parts
                    parts[slot] = (u, t1 - t0)
                    if t0 == 0:
                        assert s not in joins
                        joins[s] = (u, host.span_of(total, spans, pos - here - frm + size - 1))
        assert all((x == 1).all() for x in seen)
        used = set()
        for s, (u, last) in joins.items():
            slots = [2 * s + 1] + [2 * k for k in range(s + 1, last + 1)]
            assert sum(parts[k][1] for k in slots) == tiles[u] and all(parts[k][0] == u for k in slots)
            used |= set(slots)
        assert used == set(parts)


def test_divider_is_exact(host):
    rng = np.random.default_rng(2)
    for d in list(range(1, 300)) + [1 << k for k in range(17)] + [65535, 65521] + rng.integers(1, 65537, 200).tolist():
        top = (2 ** 31 - 1) // d
        ns = {0, 1, d - 1, d, d + 1, top * d - 1, top * d, 2 ** 31 - 1} | {int(q) * d + e for q in
                                                                          rng.integers(1, top + 1, 5) for e in (-1, 0)}
        for n in ns:
            if 0 <= n < 2 ** 31:
                assert host.div_by(n, d) == n // d, (n, d)
