"""bf16_linear's choice of kernel, tile and K split (host code, built with g++)."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "csrc")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

DRIVER = r"""
#include <cstdio>
#include "gemm_bf16_plan.h"
int main() {
  long long M, N, K;
  int act, ws;
  while (std::scanf("%lld %lld %lld %d %d", &M, &N, &K, &act, &ws) == 5) {
    const w4a4::GemmPlan p = w4a4::plan_gemm(M, N, K, act, ws != 0);
    std::printf("%d %d %d %d %d %d\n", (int)p.rows, p.tile, p.tiles_m, p.tiles_n, p.splits, p.pn);
  }
}
"""
TILES = [(256, 320, 512), (256, 256, 512), (128, 256, 512), (128, 128, 512), (64, 128, 512), (32, 128, 256)]
NONE, SWIGLU = 0, 5


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "driver.cpp").write_text(DRIVER)
    exe = str(d / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + CSRC, str(d / "driver.cpp"), "-o", exe], capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]

    def run(shapes):
        text = "".join(f"{M} {N} {K} {act} {int(ws)}\n" for M, N, K, act, ws in shapes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60).stdout.splitlines()
        assert len(out) == len(shapes)
        return [dict(zip(("rows", "tile", "tiles_m", "tiles_n", "splits", "pn"), map(int, line.split()))) for line in out]
    return run


def test_the_gpu_tests_meet_every_tile(plans):
    pytest.importorskip("torch")
    from test_linear_tiles_gpu import SHAPES
    for (tile, gated, split), (M, N, K, ws) in SHAPES.items():
        p, = plans([(M, N, K, SWIGLU if gated else NONE, ws)])
        got = ("rows", gated, False) if p["rows"] else (p["tile"], gated, p["splits"] > 1)
        assert got == (tile, gated, split), ((M, N, K, ws), p)
    # every tile, whole and split; 256 columns of SwiGLU need an even number of fragments, which 320 lack
    want = {(t, g, s) for t in range(6) for g in (False, True) for s in (False, True) if t or not g}
    assert set(SHAPES) == want | {("rows", False, False), ("rows", True, False)}


def test_few_rows_over_many_columns_take_the_tiles(plans):
    """Where the tiles need no split, a workspace changes nothing; more than
    four rows, or at most 1024 of K, are the tiles' there."""
    for ws in (0, 1):
        for M, N, K, act in [(16, 32768, 8192, NONE), (16, 65536, 5120, NONE), (8, 24576, 8192, NONE), (16, 20480, 4096, NONE),
                             (1, 32768, 1024, NONE), (16, 16384, 5120, SWIGLU), (12, 131072, 2048, NONE)]:
            p, = plans([(M, N, K, act, ws)])
            assert not p["rows"] and p["splits"] == 1, (M, N, K, act, ws, p)
        for M, N, K, act in [(1, 32768, 8192, NONE), (4, 32768, 4096, NONE), (1, 65536, 2048, SWIGLU)]:
            assert plans([(M, N, K, act, ws)])[0]["rows"], (M, N, K, act, ws)


def test_few_rows_and_columns(plans):
    for M, N, K in [(1, 2048, 2048), (16, 4096, 4096), (16, 2048, 1024), (3, 77, 264), (1, 1, 8)]:
        for ws in (0, 1):
            assert plans([(M, N, K, NONE, ws)])[0]["rows"]
    for M, N, K in [(1, 64, 8192), (16, 4096, 8192), (16, 8192, 5120)]:
        split, alone = plans([(M, N, K, NONE, 1), (M, N, K, NONE, 0)])
        assert not split["rows"] and split["splits"] > 1      # K over workgroups, where they may be joined
        assert alone["rows"]
    assert not plans([(17, 2048, 2048, NONE, 1)])[0]["rows"]


def test_every_accepted_size_has_a_launch(plans):
    """A grid holds fewer than 2^32 threads, and its tiles cover the output."""
    r = random.Random(1)
    shapes = [(1, 1 << 22, 8, NONE, 1), (16, 1 << 22, 8, SWIGLU, 0), (16, 1 << 22, 1 << 21, NONE, 0), (1 << 30, 1, 8, NONE, 1),
              (1 << 30, 8, 8, NONE, 1), (1 << 30, 128, 8, NONE, 0), (1 << 30, 128, 8, SWIGLU, 0),
              (1 << 15, 1 << 22, 8, SWIGLU, 1)]
    for _ in range(3000):
        M = int(2 ** r.uniform(0, 30))
        act = r.choice([NONE, SWIGLU])
        N = int(2 ** r.uniform(0, min(22, 37 - M.bit_length() + 0.9)))
        if M * N <= 1 << 37:
            shapes.append((M, N, 8 * int(2 ** r.uniform(0, 18)), act, r.randint(0, 1)))
    for (M, N, K, act, ws), p in zip(shapes, plans(shapes)):
        where = (M, N, K, act, ws, p)
        if p["rows"]:
            assert M <= 16 and (N + 15) // 16 * 512 < 1 << 32, where
            continue
        bm, bn, threads = TILES[p["tile"]]
        bn = bn // 2 if act == SWIGLU else bn
        assert p["tiles_m"] * bm >= M and p["tiles_n"] * bn >= N, where
        assert 0 < p["tiles_m"] * p["tiles_n"] * p["splits"] * threads < 1 << 32, where
        assert p["splits"] == 1 or (ws and p["tiles_m"] * p["tiles_n"] * p["splits"] <= 512), where
        if p["splits"] > 1:                                     # the join: a thread takes 8 columns
            assert (M * ((N + 7) // 8) + 63) // 64 * 64 < 1 << 32, where
