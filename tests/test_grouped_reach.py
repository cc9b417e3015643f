"""Host-only: which kernels the GPU cases of grouped products reach (the choice is the one the library makes), and the
refusals of the call for fresh results."""

import ctypes
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from test_grouped_host import ANY, DEEP, FEW, PERSIST, RING, _lib, _tiles, host  # noqa: E402,F401
from test_gpu_grouped_cases import FAR, SHAPES  # noqa: E402


def _reached(t, k):
    return t["kind"], t["rows"], t["kind"] == RING and k % 256 != 0


EVERY = {(ANY, 64, False), (FEW, 16, False), (RING, 64, False), (RING, 64, True), (RING, 128, False), (RING, 128, True),
         (DEEP, 64, False), (PERSIST, 256, False)}


def test_cases_with_rows_of_no_group_reach_every_kernel(host):  # noqa: F811
    assert {_reached(_tiles(host, t * top, g, n, k), k) for t, g, top, k, n in SHAPES} >= EVERY


def test_cases_past_64_groups_reach_every_kernel(host):  # noqa: F811
    far = {g: _reached(_tiles(host, g * rows, g, n, k), k) for g, rows, k, n in FAR if rows == 200}
    assert far[65] == far[130] == far[512] == (PERSIST, 256, False) and far[513] == (RING, 128, False)
    assert {_reached(_tiles(host, g * rows, g, n, k), k) for g, rows, k, n in FAR} >= EVERY - {(FEW, 16, False)}


def test_few_rows_take_small_tiles_up_to_one_a_cu(host):  # noqa: F811
    kind = lambda *s: _tiles(host, *s)["kind"]
    assert kind(2, 8, 4096, 4096) == kind(2, 8, 4096, 14336) == kind(4, 16, 2048, 1408) == FEW  # 256 tiles of 16 x 32
    assert kind(8, 256, 2048, 2048) == kind(8, 60, 1408, 2048) == kind(2, 8, 4128, 2048) == RING
    assert kind(8, 128, 1536, 4096) == kind(4, 4, 2080, 4096) == DEEP


@pytest.mark.parametrize("at,value,want", [
    (0, None, "ERR_NULL"), (3, None, "ERR_NULL"), (13, None, "ERR_NULL"), (15, None, "ERR_WORKSPACE"), (16, 256, "ERR_WORKSPACE"),
    (12, 5, "ERR_ARG"), (9, 2, "ERR_ARG"), (10, -1, "ERR_ARG"), (7, 48, "ERR_SHAPE"), (6, -1, "ERR_SHAPE"),
    (14, 255, "ERR_SHAPE"), (2, 99, "ERR_SHAPE"), (0, 0x10008, "ERR_ALIGN"), (13, 0x20001, "ERR_ALIGN"),
])
def test_refusals_of_the_call_for_fresh_results(at, value, want):
    """Fake addresses: every call is refused before any is used."""
    L, lib = _lib()
    gr = L.RowGroupsStruct(0x60000, 0x60000, 4, 100)
    a = [0x10000, 0x10000, 100, 0x10000, 0x10000, ctypes.byref(gr), 256, 512, 0, 0, 0, 1.0, L.BF16, 0x20000, 256, 0x40000, 8192,
         None]
    a[at] = value
    assert lib.fp4q_gemm_mxfp4_grouped_zeroed(*a) == getattr(L, want)
