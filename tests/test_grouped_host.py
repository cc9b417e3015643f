"""Host-only checks of the grouped calls (no GPU): the header's functions are
exported, bad arguments are refused before anything is enqueued, and the
arithmetic that the kernels share with the host (csrc/fp4q_grouped_host.h)
covers every entry once and stays inside the given tensors."""

import ctypes
import os
import re
import subprocess
import sys

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
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp4q_grouped.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fp4q_[a-z0-9_]+)\s*\(", text))
    assert names == set(L.GROUPED_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_packed_structs_are_the_structs():
    L, _ = _lib()
    assert bytes(L.RowGroupsStruct(1, 2, 3, 4)) == L.ROW_GROUPS_PACK(1, 2, 3, 4)
    assert bytes(L.RouterStruct(1, 2, 3, 4, 5, 6, 7, 2.5)) == L.ROUTER_PACK(1, 2, 3, 4, 5, 6, 7, 2.5)


# fake, aligned device addresses: validation must reject before any use
X, Y, OUT, WS, IDX = 0x10000, 0x18000, 0x20000, 0x40000, 0x60000


def _group(L, lib, **kw):
    a = dict(ids=IDX, entries=5000, groups=10, offsets=IDX, rows=IDX, ws=WS, wsb=1 << 20)
    a.update(kw)
    return lib.fp4q_group_rows(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(entries=-1), "ERR_SHAPE"), (dict(entries=(1 << 30) + 1), "ERR_SHAPE"), (dict(groups=0), "ERR_SHAPE"),
    (dict(groups=2049), "ERR_SHAPE"), (dict(ids=None), "ERR_NULL"), (dict(offsets=None), "ERR_NULL"),
    (dict(rows=None), "ERR_NULL"), (dict(ws=None), "ERR_WORKSPACE"), (dict(wsb=64), "ERR_WORKSPACE"),
    (dict(ws=WS + 8), "ERR_WORKSPACE"), (dict(ids=IDX + 2), "ERR_ALIGN"), (dict(rows=IDX + 1), "ERR_ALIGN"),
])
def test_group_rows_refusals(kw, want):
    L, lib = _lib()
    assert _group(L, lib, **kw) == getattr(L, want)


def _route(L, lib, r=None, **kw):
    a = dict(x=X, dtype=L.F32, tokens=300, experts=64, ld=64)
    q = dict(score=L.SOFTMAX, bias=None, k=8, ng=1, tg=1, gb=1, re=1, scale=1.0)
    o = dict(w=OUT, ch=OUT, off=IDX, rows=IDX, ws=WS, wsb=1 << 22)
    q.update(r or {})
    for k, v in kw.items():
        (a if k in a else o)[k] = v
    return lib.fp4q_route_experts(*a.values(), ctypes.byref(L.RouterStruct(*q.values())), *o.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), "ERR_NULL"), (dict(w=None), "ERR_NULL"), (dict(ch=None), "ERR_NULL"), (dict(off=None), "ERR_NULL"),
    (dict(rows=None), "ERR_NULL"), (dict(dtype=3), "ERR_ARG"), (dict(tokens=-1), "ERR_SHAPE"),
    (dict(tokens=1 << 28), "ERR_SHAPE"), (dict(experts=0, ld=0), "ERR_SHAPE"), (dict(experts=1025, ld=1025), "ERR_SHAPE"),
    (dict(ld=63), "ERR_SHAPE"), (dict(ws=None), "ERR_WORKSPACE"), (dict(wsb=300), "ERR_WORKSPACE"),
    (dict(x=X + 2), "ERR_ALIGN"), (dict(w=OUT + 2), "ERR_ALIGN"), (dict(ld=1 << 62), "ERR_SHAPE"),
])
def test_route_refusals(kw, want):
    L, lib = _lib()
    assert _route(L, lib, **kw) == getattr(L, want)


@pytest.mark.parametrize("r,want", [
    (dict(score=2), "ERR_ARG"), (dict(k=0), "ERR_SHAPE"), (dict(k=65), "ERR_SHAPE"), (dict(ng=0), "ERR_SHAPE"),
    (dict(ng=3), "ERR_SHAPE"), (dict(ng=8, tg=9), "ERR_SHAPE"), (dict(ng=8, tg=0), "ERR_SHAPE"),
    (dict(gb=3), "ERR_ARG"), (dict(gb=0), "ERR_ARG"), (dict(re=2), "ERR_ARG"), (dict(scale=float("nan")), "ERR_ARG"),
    (dict(scale=float("inf")), "ERR_ARG"), (dict(bias=X + 2), "ERR_ALIGN"),
])
def test_router_refusals(r, want):
    L, lib = _lib()
    assert _route(L, lib, r=r) == getattr(L, want)


def test_more_choices_than_experts_are_refused():
    L, lib = _lib()
    assert _route(L, lib, r=dict(k=9), experts=8, ld=8) == L.ERR_SHAPE
    assert _route(L, lib, r=dict(ng=128, tg=1), experts=256, ld=256) == L.ERR_SHAPE


def _product(L, lib, g=None, **kw):
    a = dict(ac=X, as_=X, rows=100, bc=X, bs=X)
    gr = dict(off=IDX, rows=IDX, groups=4, entries=100)
    o = dict(n=256, k=512, gather=0, scatter=0, gated=0, alpha=1.0, dtype=L.BF16, c=OUT, ldc=256, ws=WS, wsb=8192)
    gr.update(g or {})
    for k, v in kw.items():
        (a if k in a else o)[k] = v
    return lib.fp4q_gemm_mxfp4_grouped(*a.values(), ctypes.byref(L.RowGroupsStruct(*gr.values())), *o.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(ac=None), "ERR_NULL"), (dict(as_=None), "ERR_NULL"), (dict(bc=None), "ERR_NULL"), (dict(bs=None), "ERR_NULL"),
    (dict(c=None), "ERR_NULL"), (dict(ws=None), "ERR_WORKSPACE"), (dict(wsb=256), "ERR_WORKSPACE"),
    (dict(dtype=5), "ERR_ARG"), (dict(scatter=2), "ERR_ARG"), (dict(gated=-1), "ERR_ARG"),
    (dict(gated=1, n=255, ldc=255), "ERR_SHAPE"), (dict(k=48), "ERR_SHAPE"), (dict(k=0), "ERR_SHAPE"),
    (dict(n=-1), "ERR_SHAPE"), (dict(ldc=255), "ERR_SHAPE"), (dict(rows=99), "ERR_SHAPE"),
    (dict(gather=8, rows=12), "ERR_SHAPE"), (dict(gather=-1), "ERR_SHAPE"), (dict(ac=X + 8), "ERR_ALIGN"),
    (dict(bc=X + 4), "ERR_ALIGN"), (dict(as_=X + 1), "ERR_ALIGN"), (dict(c=OUT + 1), "ERR_ALIGN"),
    (dict(n=1 << 31, ldc=1 << 31), "ERR_SHAPE"), (dict(n=(1 << 31) - 2, ldc=1 << 31), "ERR_SHAPE"),
])
def test_product_refusals(kw, want):
    L, lib = _lib()
    assert _product(L, lib, **kw) == getattr(L, want)


@pytest.mark.parametrize("g,want", [
    (dict(off=None), "ERR_NULL"), (dict(rows=None), "ERR_NULL"), (dict(groups=0), "ERR_SHAPE"),
    (dict(groups=2049), "ERR_SHAPE"), (dict(entries=-1), "ERR_SHAPE"), (dict(entries=101), "ERR_SHAPE"),
    (dict(off=IDX + 2), "ERR_ALIGN"), (dict(rows=IDX + 2), "ERR_ALIGN"),
])
def test_row_groups_refusals(g, want):
    L, lib = _lib()
    assert _product(L, lib, g=g) == getattr(L, want)


def _combine(L, lib, **kw):
    a = dict(y=X, dtype=L.BF16, tokens=10, k=4, n=256, ldy=256, w=Y, ch=IDX, add=None, ldadd=256, odt=L.BF16, out=OUT,
             ldo=256)
    a.update(kw)
    return lib.fp4q_combine_experts(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(y=None), "ERR_NULL"), (dict(w=None), "ERR_NULL"), (dict(out=None), "ERR_NULL"), (dict(dtype=2), "ERR_ARG"),
    (dict(odt=2), "ERR_ARG"), (dict(k=0), "ERR_SHAPE"), (dict(k=65), "ERR_SHAPE"), (dict(tokens=-1), "ERR_SHAPE"),
    (dict(ldy=255), "ERR_SHAPE"), (dict(ldo=255), "ERR_SHAPE"), (dict(add=X, ldadd=255), "ERR_SHAPE"),
    (dict(y=X + 1), "ERR_ALIGN"), (dict(out=OUT + 1), "ERR_ALIGN"), (dict(w=Y + 2), "ERR_ALIGN"),
    (dict(ch=IDX + 1), "ERR_ALIGN"), (dict(tokens=1 << 25, n=8192, ldy=8192, ldo=8192), "ERR_SHAPE"),
    (dict(tokens=0), "OK"), (dict(n=0, ldy=0, ldo=0), "OK"),
])
def test_combine_refusals(kw, want):
    L, lib = _lib()
    assert _combine(L, lib, **kw) == getattr(L, want)


def _lora(L, lib, g=None, **kw):
    a = dict(y=X, dtype=L.BF16, ldy=256, x=X, ldx=512, a=X, b=X, sc=None)
    gr = dict(off=IDX, rows=IDX, groups=4, entries=100)
    o = dict(n=256, k=512, rank=16, out=OUT, ldo=256, ws=WS, wsb=1 << 20)
    gr.update(g or {})
    for k, v in kw.items():
        (a if k in a else o)[k] = v
    return lib.fp4q_lora_add(*a.values(), ctypes.byref(L.RowGroupsStruct(*gr.values())), *o.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(y=None), "ERR_NULL"), (dict(x=None), "ERR_NULL"), (dict(a=None), "ERR_NULL"), (dict(b=None), "ERR_NULL"),
    (dict(out=None), "ERR_NULL"), (dict(dtype=2), "ERR_ARG"), (dict(rank=4), "ERR_SHAPE"), (dict(rank=12), "ERR_SHAPE"),
    (dict(rank=264), "ERR_SHAPE"), (dict(k=510), "ERR_SHAPE"), (dict(k=0), "ERR_SHAPE"), (dict(n=-1), "ERR_SHAPE"),
    (dict(ldy=255), "ERR_SHAPE"), (dict(ldo=255), "ERR_SHAPE"), (dict(ldx=511), "ERR_SHAPE"),
    (dict(ldx=516), "ERR_ALIGN"), (dict(x=X + 8), "ERR_ALIGN"), (dict(a=X + 2), "ERR_ALIGN"), (dict(b=X + 2), "ERR_ALIGN"),
    (dict(sc=X + 2), "ERR_ALIGN"), (dict(y=X + 1), "ERR_ALIGN"), (dict(wsb=1000), "ERR_WORKSPACE"),
    (dict(ws=WS + 4), "ERR_WORKSPACE"), (dict(out=X, ldo=300), "ERR_ARG"),
])
def test_lora_refusals(kw, want):
    L, lib = _lib()
    assert _lora(L, lib, **kw) == getattr(L, want)


def test_workspace_sizes_of_refused_calls_are_zero():
    L, lib = _lib()
    assert lib.fp4q_group_rows_workspace_bytes(-1, 4) == lib.fp4q_group_rows_workspace_bytes(8, 0) == 0
    assert lib.fp4q_route_experts_workspace_bytes(1 << 28, 64, 8) == 0
    assert lib.fp4q_route_experts_workspace_bytes(8, 1025, 8) == 0
    assert lib.fp4q_lora_add_workspace_bytes(8, 4, 256, 512, 12) == 0
    assert lib.fp4q_lora_add_workspace_bytes(8, 4, 256, 512, 16) > 256


def test_binding_refuses_host_and_wrong_tensors():
    import fp4_post_quantization_amd as fq
    cpu = torch.device("cpu")
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="ids"):
        fq.group_rows(i, 2)
    with pytest.raises(ValueError, match="logits"):
        fq.route_experts(torch.zeros(2, 4), 2)
    with pytest.raises(ValueError, match="y must"):
        fq.combine_experts(torch.zeros(2, 2, 4), torch.zeros(2, 2))
    with pytest.raises(ValueError, match="y is on"):
        fq.lora_add(torch.zeros(2, 8), torch.zeros(2, 8).bfloat16(), torch.zeros(1, 8, 8).bfloat16(),
                    torch.zeros(1, 8, 8).bfloat16(), fq.RowGroups(i[:2], i[:2]))
    for bad in (i.long(), i[::2], i.view(2, 2)):
        with pytest.raises(ValueError, match="offsets"):
            fq._groups_struct(fq.RowGroups(bad, i), cpu)
        with pytest.raises(ValueError, match="rows"):
            fq._groups_struct(fq.RowGroups(i, bad), cpu)
    with pytest.raises(ValueError, match="one entry more"):
        fq._groups_struct(fq.RowGroups(i[:1], i), cpu)
    assert fq._groups_struct(fq.RowGroups(i, i[:3]), cpu)[1:] == (3, 3)


# ------------------------------------------------ index arithmetic, on the host ----
_PROGRAM = r"""
#include "fp4q_grouped_host.h"
using namespace fp4q;
extern "C" void span(int64_t o0, int64_t o1, int64_t entries, int64_t rows, int64_t *o) {
  GroupSpan s = group_span((int)o0, (int)o1, (int)entries);
  o[0] = s.lo; o[1] = s.hi; o[2] = s.bad; o[3] = span_tiles(s.lo, s.hi, (int)rows);
}
extern "C" int64_t most(int64_t entries, int64_t groups, int64_t rows) { return most_tiles(entries, groups, rows); }
extern "C" void plan(int64_t units, int64_t per_unit, int64_t least, int64_t *o) {
  SortPlan p = sort_plan(units, per_unit, least);
  o[0] = p.per; o[1] = p.blocks; o[2] = p.join; o[3] = p.places;
}
extern "C" void product(int64_t entries, int64_t groups, int64_t n, int64_t k, int64_t *o) {
  ProductTiles t = product_tiles(entries, groups, n, k, entries);
  o[0] = t.kind; o[1] = t.rows; o[2] = t.cols; o[3] = t.run; o[4] = t.workgroups;
}
extern "C" int64_t splits(int64_t entries, int64_t groups, int64_t k) { return lora_plan(entries, groups, k).splits; }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("groupedhost")
    src, so = d / "host.cpp", d / "host.so"
    src.write_text(_PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-shared", "-fPIC", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(so)],
                   check=True)
    lib = ctypes.CDLL(str(so))
    P, I = ctypes.c_void_p, ctypes.c_int64
    lib.span.argtypes, lib.plan.argtypes, lib.product.argtypes = [I, I, I, I, P], [I, I, I, P], [I, I, I, I, P]
    for f in (lib.most, lib.splits):
        f.argtypes, f.restype = [I, I, I], I
    return lib


def test_bad_offsets_stay_inside(host):
    rng = np.random.default_rng(1)
    o = np.zeros(4, np.int64)
    edge = [-2 ** 31, -1, 0, 1, 63, 64, 65, 99, 100, 101, 2 ** 31 - 1]
    for _ in range(2000):
        a, b = (int(rng.choice(edge)) if rng.random() < 0.8 else int(rng.integers(0, 100)) for _ in range(2))
        host.span(a, b, 100, 64, o.ctypes.data)
        lo, hi, bad, tiles = o.tolist()
        assert 0 <= lo <= hi <= 100 and bad == (not 0 <= a <= b <= 100) and tiles == -(-(hi - lo) // 64)
        if not bad:
            assert (lo, hi) == (a, b)


def test_a_launch_has_a_workgroup_for_every_row_tile(host):
    rng = np.random.default_rng(2)
    for _ in range(500):
        groups = int(rng.integers(1, 50))
        counts = rng.integers(0, rng.choice([2, 20, 300]), groups) * (rng.random(groups) < 0.7)
        entries = int(counts.sum() + rng.integers(0, 5))
        for rows in (16, 32, 64, 128, 256):
            assert sum(-(-c // rows) for c in counts.tolist()) <= host.most(entries, groups, rows)


def test_sorting_covers_every_entry_once(host):
    o = np.zeros(4, np.int64)
    for units, per_unit, least in [(1, 1, 1024), (65, 8, 4), (1021, 4, 4), (8192, 8, 4), (8193, 64, 4), (5000, 1, 1024),
                                   (10 ** 6, 8, 4), (2 ** 30, 1, 1024), (2 ** 24, 64, 4), (70, 1, 4)]:
        host.plan(units, per_unit, least, o.ctypes.data)
        per, blocks, join, places = o.tolist()
        assert per * per_unit <= 65535 and (blocks <= 512 or per == 65535 // per_unit)  # counts are 16 bits
        assert (blocks - 1) * per < units <= blocks * per
        assert (places - 1) * join < blocks <= places * join
        assert join == 1 or join * per * per_unit <= 1024


def test_adapter_splits_keep_whole_steps(host):
    for entries in (1, 17, 64, 500, 8191):
        for groups in (1, 5, 100):
            for k in (8, 64, 1024, 4096, 14336):
                assert 1 <= host.splits(entries, groups, k) <= 8


def _tiles(host, *sizes):
    o = np.zeros(5, np.int64)
    host.product(*sizes, o.ctypes.data)
    return dict(zip(("kind", "rows", "cols", "run", "workgroups"), o.tolist()))


ANY, FEW, RING, DEEP, PERSIST = range(5)


def test_product_tiles_cover_the_rows(host):
    """Every launch but the persistent one has a workgroup for each tile there can be, in whole runs for every XCD."""
    rng = np.random.default_rng(4)
    for _ in range(2000):
        groups = int(rng.integers(1, 300))
        entries = int(np.exp(rng.uniform(0, 12)))
        n, k = int(rng.integers(1, 9000)), 32 * int(rng.integers(1, 500))
        t = _tiles(host, entries, groups, n, k)
        most = host.most(entries, groups, t["rows"]) * -(-n // t["cols"])
        assert t["workgroups"] % (8 * t["run"] if t["kind"] in (FEW, RING, DEEP) else 1) == 0
        assert t["workgroups"] >= (min(most, 256) if t["kind"] == PERSIST else most)
        assert k >= 256 or t["kind"] == ANY
        assert t["kind"] not in (DEEP, PERSIST) or k % 256 == 0
        assert t["kind"] != PERSIST or (k >= 512 and groups <= 512 and t["workgroups"] % 8 == 0)
        assert t["kind"] != FEW or k % 128 == 0


def test_products_past_32_bit_offsets_and_launches(host):
    """Operands of 4 GiB and more go to the kernel with 64-bit addresses; more tiles than a launch has are counted."""
    assert _tiles(host, 1 << 20, 4, 4096, 8192)["kind"] == ANY       # 2^20 rows of 4096 bytes
    assert _tiles(host, 1 << 19, 4, 4096, 8192)["kind"] == PERSIST
    assert _tiles(host, 4096, 4, 1 << 21, 4096)["kind"] == ANY       # a matrix of 2^32 bytes
    assert _tiles(host, 1 << 22, 2, 1 << 20, 512)["workgroups"] > 1 << 22


def test_product_sizes_of_the_gpu_tests_reach_every_kernel(host):
    sys.path.insert(0, os.path.join(ROOT, "tests"))
    from test_gpu_grouped import PRODUCTS
    seen = set()
    for tokens, groups, top_k, k, n in PRODUCTS:
        t = _tiles(host, tokens * top_k, groups, n, k)
        tail = t["kind"] == RING and k % 256 != 0
        several = t["kind"] == PERSIST and (tokens * top_k // 256) * (n // 256) > 256  # tiles, at least
        seen.add((t["kind"], t["rows"], tail, several))
    assert seen >= {(ANY, 64, False, False), (FEW, 16, False, False), (RING, 64, False, False), (RING, 64, True, False),
                    (RING, 128, False, False), (RING, 128, True, False), (DEEP, 64, False, False),
                    (PERSIST, 256, False, True)}
