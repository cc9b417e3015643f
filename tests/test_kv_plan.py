"""The choice of attention's kernels (csrc/fp4q_kv_host.h, make_plan), on the host: which row tile and how many
spans a call gets from its sizes, and that the shapes of the GPU tests reach the kernels that they are there for."""

import ctypes
import os
import subprocess
from collections import namedtuple

import pytest

import test_gpu_kv_prompts as prompts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_PROGRAM = r"""
#include "fp4q_kv_host.h"
extern "C" void plan(const int64_t *s, int64_t *o) {
  const fp4q::Plan p = fp4q::make_plan(s[0], s[1], s[2], s[3], s[4], s[5], s[6], s[7]);
  o[0] = p.rows; o[1] = p.waves; o[2] = p.units; o[3] = p.spans; o[4] = p.part_floats;
}
"""

Plan = namedtuple("Plan", "rows waves units spans part_floats")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("kvplan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(_PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-shared", "-fPIC", "-I", os.path.join(ROOT, "fp4_post_quantization_amd", "csrc"), "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def call(lens, news, heads, kv_heads, dim, page, window=0, max_new=None):
        """The plan of the binding's call: max_new by default the rows of q, max_len what the table holds."""
        tokens, width = sum(news), max(1, max(-(-n // page) for n in lens))
        s = (ctypes.c_int64 * 8)(tokens, len(lens), heads, kv_heads, dim, tokens if max_new is None else max_new,
                                 width * page, window)
        o = (ctypes.c_int64 * 5)()
        lib.plan(s, o)
        return Plan(*o)
    return call


def test_decoding_gets_tiles_of_16_rows_whatever_bounds_the_new_tokens(plan):
    """64 sequences of one row each, their number of rows bounded by 1 or only by the rows of q."""
    lens = [8192] * 64
    for dim in (64, 128, 256):
        for bound in (1, None):
            assert plan(lens, [1] * 64, 64, 8, dim, 64, max_new=bound).rows == 16


@pytest.mark.parametrize("lens,news,rows", [
    ([8192] * 64, [1] * 63 + [512], 16),           # one chunk beside 63 decoding sequences: 36 rows a sequence and head
    ([2048] * 128, [1] * 127 + [128], 16),
    ([4096] * 64, [1] * 56 + [256] * 8, 128),      # 131
    ([4096] * 32, [1] * 31 + [2048], 128),         # 260: tiles of 256 would be filled for one sequence in 32
    ([4096] * 64, [32] * 64, 128),                 # 128 each
    ([2048] * 64, [128] * 64, 256),                # 512 each
    ([8192], [4096], 256), ([1500] * 4, [512] * 4, 128), ([600], [150], 16),
])
def test_the_average_sequence_fills_the_row_tile(plan, lens, news, rows):
    assert plan(lens, news, 32, 8, 128, 64, max_new=max(news)).rows == rows


def test_plans_stay_inside_what_a_launch_and_a_workspace_may_have(plan):
    for lens, news, heads, kv in (([8192] * 64, [1] * 64, 64, 8), ([131072], [1], 64, 8), ([9000], [130], 8, 2),
                                  ([100000] * 3, [0] * 3, 8, 8)):
        for dim in (64, 128, 256):
            p = plan(lens, news, heads, kv, dim, 64)
            assert 0 <= p.units <= 1 << 22 and 0 <= p.spans < 512
            assert p.part_floats == (2 * p.spans * p.rows * (dim + 2) if p.spans else 0)
            assert p.spans == 0 or p.units > 0


def test_tiles_of_256_rows_are_never_split(plan):
    """Over sizes up to the largest that a call may have."""
    found = 0
    for dim in (64, 128):
        for kv_heads in (1, 8, 64, 65536 // dim):
            for groups in (1, 4, 64):
                for log_batch in (0, 3, 9, 16):
                    for new in (1, 7, 512, 100000, (1 << 33) // (kv_heads * groups * dim) >> log_batch):
                        batch = 1 << log_batch
                        if not 0 < batch * new * kv_heads * groups * dim < 1 << 33 or kv_heads * groups > 65536:
                            continue
                        for length in (new, 1 << 20):
                            p = plan([length] * batch, [new] * batch, kv_heads * groups, kv_heads, dim, 1024,
                                     max_new=new)
                            if p.rows == 256:
                                found += 1
                                assert p.spans == 0 and p.units < 1 << 20
    assert found > 50


@pytest.mark.parametrize("name,dim", prompts.CASES)
def test_shapes_of_the_prompt_tests_reach_their_kernels(plan, name, dim):
    rows, split, lens, news, heads, kv_heads, page = prompts.SHAPES[name]
    windows = (0,) if split else (0, 1, 77, 90, 300, 400)  # a window bounds the keys that are worth a split
    for window in windows:
        p = plan(lens, news, heads, kv_heads, dim, page, window)
        assert (p.rows, p.spans > 0) == (rows, split), window
