"""The choice of attention's kernels (csrc/fp4q_kv_host.h, make_plan), on the host: which row tile and how many
spans a call gets from its sizes, and that the shapes of the GPU tests reach the kernels that they are there for."""

import ctypes
import os
import subprocess
from collections import namedtuple

import numpy as np
import pytest

import test_gpu_kv_prompts as prompts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_PROGRAM = r"""
#include "fp4q_kv_host.h"
extern "C" void plan(const int64_t *s, int64_t *o) {
  const fp4q::Plan p = fp4q::make_plan(s[0], s[1], s[2], s[3], s[4], s[5], s[6], s[7]);
  *o++ = p.passes;
  for (int i = 0; i < p.passes; ++i) {
    const fp4q::Pass &x = p.pass[i];
    *o++ = x.rows; *o++ = x.waves; *o++ = x.units; *o++ = x.spans; *o++ = x.part_floats; *o++ = x.min_rows;
    *o++ = x.max_rows;
  }
}
"""

Pass = namedtuple("Pass", "rows waves units spans part_floats min_rows max_rows")


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
        """The passes of the binding's call: max_new by default the rows of q, max_len what the table holds."""
        tokens, width = sum(news), max(1, max(-(-n // page) for n in lens))
        s = (ctypes.c_int64 * 8)(tokens, len(lens), heads, kv_heads, dim, tokens if max_new is None else max_new,
                                 width * page, window)
        o = (ctypes.c_int64 * 15)()
        lib.plan(s, o)
        return [Pass(*o[1 + 7 * i: 8 + 7 * i]) for i in range(o[0])]
    return call


def _tile(passes, rows):
    """The row tile that serves a sequence of so many rows: one pass does, whatever their number."""
    tiles = [p.rows for p in passes if p.min_rows <= rows <= p.max_rows]
    assert len(tiles) == 1
    return tiles[0]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bound", [1, 8, None])
@pytest.mark.parametrize("batch,heads,kv_heads", [(1, 32, 8), (64, 64, 8), (64, 32, 32), (4096, 32, 8), (64, 96, 1)])
def test_decoding_gets_tiles_of_16_rows_whatever_bounds_the_new_tokens(plan, dim, bound, batch, heads, kv_heads):
    """One row for each sequence, their number bounded by 1, by more or only by the rows of q."""
    p = plan([8192] * batch, [1] * batch, heads, kv_heads, dim, 64, max_new=bound and min(bound, batch))
    assert _tile(p, heads // kv_heads) == 16


@pytest.mark.parametrize("lens,news,rows", [
    ([8192] * 64, [1] * 63 + [512], [16, 128]),          # one chunk beside 63 decoding sequences
    ([8192] * 64, [0] * 63 + [512], [16, 128]),          # alone in a padded batch
    ([2048] * 128, [1] * 127 + [128], [16, 128]),
    ([4096] * 64, [1] * 56 + [256] * 8, [16, 128]),
    ([4096] * 32, [1] * 31 + [2048], [16, 128]),
    ([2048] * 4, [1, 1, 1, 1000], [128]),                # 280 units, which run at once
    ([2048] * 8, [0] * 7 + [2000], [16, 128]),
    ([8192] * 16, [1] * 15 + [60], [16, 128]),           # few units, but most of them of 4 rows
    ([600, 600], [5, 100], [16]),                        # too few rows for the prompt kernel, and few keys
    ([4096] * 64, [32] * 64, [128]),                     # 128 rows each: tiles of 256 would be half empty
    ([2048] * 64, [128] * 64, [256]),                    # 512 each
    ([4096] * 32, [i + 1 for i in range(32)], [128]),    # 4 to 128
    ([8192], [4096], [256]), ([1500] * 4, [512] * 4, [128]), ([600], [150], [16]),
])
def test_each_sequence_gets_a_row_tile_that_it_fills(plan, lens, news, rows):
    p = plan(lens, news, 32, 8, 128, 64, max_new=max(news))
    assert sorted(x.rows for x in p) == rows
    if len(rows) == 2:
        assert _tile(p, 4) == _tile(p, 96) == 16 and _tile(p, 97) == _tile(p, 4 * max(news)) == 128
    assert _tile(p, 0) and _tile(p, 2 ** 27)


def test_units_of_a_pass_are_bounded(plan):
    """Whatever the lengths, no pass has more units than its bound, which sizes the launch."""
    rng = np.random.default_rng(1)
    two = 0
    for _ in range(400):
        batch, groups = int(rng.integers(1, 70)), int(rng.choice([1, 3, 4, 8, 100]))
        kv_heads = int(rng.choice([1, 2, 8]))
        news = rng.integers(0, int(rng.choice([2, 9, 40, 700])), batch)
        news[rng.integers(0, batch)] += int(rng.choice([0, 1, 130, 2000]))
        if news.sum() == 0:
            continue
        passes = plan([6000] * batch, news.tolist(), groups * kv_heads, kv_heads, int(rng.choice([64, 256])), 64,
                      max_new=None if rng.random() < 0.5 else int(news.max()))
        two += len(passes) == 2
        served = np.zeros(batch, dtype=int)
        for p in passes:
            mine = (news * groups >= p.min_rows) & (news * groups <= p.max_rows)
            served += mine
            assert (-(-news[mine] * groups // p.rows)).sum() * kv_heads <= p.units
        assert (served == 1).all()
    assert two > 50


def test_plans_stay_inside_what_a_launch_and_a_workspace_may_have(plan):
    for lens, news, heads, kv in (([8192] * 64, [1] * 64, 64, 8), ([131072], [1], 64, 8), ([9000], [130], 8, 2),
                                  ([100000] * 3, [0] * 3, 8, 8)):
        for dim in (64, 128, 256):
            for p in plan(lens, news, heads, kv, dim, 64):
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
                            for p in plan([length] * batch, [new] * batch, kv_heads * groups, kv_heads, dim, 1024,
                                          max_new=new):
                                if p.rows == 256:
                                    found += 1
                                    assert p.spans == 0 and p.units < 1 << 20
    assert found > 50


@pytest.mark.parametrize("name,dim", prompts.CASES)
def test_shapes_of_the_prompt_tests_reach_their_kernels(plan, name, dim):
    rows, split, lens, news, heads, kv_heads, page = prompts.SHAPES[name]
    windows = (0,) if split else (0, 1, 77, 90, 300, 400)  # a window bounds the keys that are worth a split
    for window in windows:
        passes = plan(lens, news, heads, kv_heads, dim, page, window)
        assert (passes[0].rows, passes[0].spans > 0) == (rows, split), window
        assert _tile(passes, news[0] * heads // kv_heads) == rows
