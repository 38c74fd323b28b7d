"""cache_attention's choice of tile and parts (host code, built with g++), and
that the GPU tests' shapes meet every one of them."""
import os
import random
import shutil
import subprocess

import pytest

pytest.importorskip("torch")

from test_cache_attention_tiles_gpu import SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "csrc")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

DRIVER = r"""
#include <cstdio>
#include "cache_attention_plan.h"
int main() {
  long long B, T, Hq, Hkv, D, L;
  int ws;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %d", &B, &T, &Hq, &Hkv, &D, &L, &ws) == 7) {
    const w4a4::CacheAttnPlan p = w4a4::plan_cache_attention(B, T, Hq, Hkv, D, L, ws != 0);
    std::printf("%d %d %d %d\n", p.rows, p.waves, p.tiles, p.parts);
  }
}
"""
TILES = {64: [(16, 4), (16, 8), (32, 8), (256, 8)], 128: [(16, 4), (16, 8), (32, 8), (256, 8)],
         256: [(16, 4), (16, 8), (128, 4)]}


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "driver.cpp").write_text(DRIVER)
    exe = str(d / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + CSRC, str(d / "driver.cpp"), "-o", exe], capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]

    def run(shapes):
        text = "".join(" ".join(str(int(v)) for v in s) + "\n" for s in shapes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60).stdout.splitlines()
        assert len(out) == len(shapes)
        return [dict(zip(("rows", "waves", "tiles", "parts"), map(int, line.split()))) for line in out]
    return run


def test_the_gpu_tests_meet_every_tile(plans):
    for (D, rows, waves, parts, several), (B, T, Hq, Hkv, L, ws) in SHAPES.items():
        p, = plans([(B, T, Hq, Hkv, D, L, ws)])
        assert (p["rows"], p["waves"], p["parts"] > 1) == (rows, waves, parts), ((D, rows, waves, parts), p)
        assert several is None or (p["tiles"] > 1) == several, ((D, rows, waves, parts), p)
    # the kernels for few rows read keys in two ways, by whether a sequence has one row tile
    for D, tiles in TILES.items():
        for rows, waves in tiles:
            for several in (False, True) if rows <= 32 else (None,):
                assert any(k[:3] == (D, rows, waves) and k[4] == several for k in SHAPES)
            assert {k[3] for k in SHAPES if k[:3] == (D, rows, waves)} == {False, True}


def test_plans_cover_the_rows_and_fit_a_launch(plans):
    r = random.Random(3)
    shapes = [(1 << 22, 1, 1, 1, 64, 1 << 30, True), (64, 1 << 16, 16, 16, 128, 1 << 20, True),
              (1, 1 << 20, 64, 64, 256, 1 << 30, False), (1, 1, 65536, 1, 64, 0, True), (1 << 16, 16, 64, 64, 128, 5, True)]
    while len(shapes) < 4000:
        Hkv, D = r.choice([1, 2, 5, 8, 64]), r.choice([64, 128, 256])
        B, T = int(2 ** r.uniform(0, 22)), int(2 ** r.uniform(0, 20))
        Hq = Hkv * r.choice([1, 3, 7, 8])
        if B * T * Hq <= 1 << 30 and B * Hkv * -(-T * (Hq // Hkv) // 16) <= 1 << 22:     # what the entry point takes
            shapes.append((B, T, Hq, Hkv, D, int(2 ** r.uniform(0, 30)) - 1, r.random() < 0.5))
    for s, p in zip(shapes, plans(shapes)):
        B, T, Hq, Hkv, D, L, ws = s
        assert (p["rows"], p["waves"]) in TILES[D], (s, p)
        assert p["tiles"] * p["rows"] >= T * (Hq // Hkv) > (p["tiles"] - 1) * p["rows"], (s, p)
        assert 1 <= p["parts"] <= 64 and (ws or p["parts"] == 1), (s, p)
        assert B * Hkv * p["tiles"] * p["parts"] * 64 * p["waves"] < 1 << 32, (s, p)   # threads of the launch
        if p["parts"] > 1:
            assert B * Hq * T * (D // 4) < 1 << 32                                     # and of the join
