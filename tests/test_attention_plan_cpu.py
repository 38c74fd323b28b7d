"""prefix_attention's choice of tile and parts (host code, built with g++), and
that the GPU tests' shapes meet every one of them."""
import os
import random
import shutil
import subprocess

import pytest

pytest.importorskip("torch")

from test_attention_places_gpu import RING, RING_SHAPE, SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "csrc")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

DRIVER = r"""
#include <cstdio>
#include "attention_plan.h"
int main() {
  long long B, T, Hq, Hkv, D, P, S;
  int ws;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %d", &B, &T, &Hq, &Hkv, &D, &P, &S, &ws) == 8) {
    const w4a4::AttnPlan p = w4a4::plan_attention(B, T, Hq, Hkv, D, P, S, ws != 0);
    std::printf("%d %d %d %d %d %d %d\n", p.cfg, p.rpt, p.tiles, p.parts, p.np, p.ns, p.per);
  }
}
"""
TILES = {64: [(1, 8, 64), (2, 4, 64), (4, 2, 64), (8, 1, 64)], 128: [(1, 8, 32), (2, 4, 32), (4, 2, 64), (8, 1, 64)],
         256: [(2, 2, 32), (4, 1, 32)]}                               # row waves, key groups, keys of a block


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
        return [dict(zip(("cfg", "rpt", "tiles", "parts", "np", "ns", "per"), map(int, line.split()))) for line in out]
    return run


def test_the_gpu_tests_meet_every_tile(plans):
    for (D, cfg, parts), (B, T, Hq, Hkv, P, S, ws) in SHAPES.items():
        p, = plans([(B, T, Hq, Hkv, D, P, S, ws)])
        assert (p["cfg"], p["parts"] > 1) == (cfg, parts), ((D, cfg, parts), p)
    assert set(SHAPES) == {(D, c, p) for D, t in TILES.items() for c in range(len(t)) for p in (False, True)}
    for D, (B, T, Hq, Hkv, S) in RING_SHAPE.items():
        for p in plans([(B, T, Hq, Hkv, D, P, S, False) for P in RING]):
            assert p["cfg"] == 3 and p["parts"] == 1


def test_plans_cover_rows_and_keys(plans):
    r = random.Random(2)
    shapes = [(1 << 13, 2, 1 << 16, 1 << 16, 64, 0, 0, True), (1 << 22, 1, 64, 64, 256, 0, 1, False),
              (1, 1 << 23, 64, 1, 128, 5, 5, True), (1 << 13, 1, 1 << 16, 1 << 16, 128, 1, 0, False)]
    while len(shapes) < 4000:
        Hkv, D = r.choice([1, 2, 5, 8, 64]), r.choice([64, 128, 256])
        B, T = int(2 ** r.uniform(0, 10)), int(2 ** r.uniform(0, 12))
        Hq = Hkv * r.choice([1, 3, 7, 8])
        if B * T * Hq * D <= 1 << 36:                                  # q alone is 137 GB there
            shapes.append((B, T, Hq, Hkv, D, int(2 ** r.uniform(0, 30)) - 1, int(2 ** r.uniform(0, 24)) - 1, r.random() < 0.5))
    for s, p in zip(shapes, plans(shapes)):
        B, T, Hq, Hkv, D, P, S, ws = s
        wq, wk, bn = TILES[D][p["cfg"]]
        tg = T * (Hq // Hkv)
        assert 0 < p["rpt"] <= 32 * wq and p["tiles"] * p["rpt"] >= B * tg, (s, p)
        assert p["np"] * bn >= P and p["ns"] * bn >= S, (s, p)
        seqs = max((min(B * tg, (i + 1) * p["rpt"]) - 1) // tg - i * p["rpt"] // tg + 1 for i in {0, p["tiles"] // 2, p["tiles"] - 1})
        assert p["parts"] * p["per"] >= p["np"] + seqs * p["ns"], (s, p)
        assert p["parts"] == 1 or (ws and p["parts"] <= 256), (s, p)
        assert Hkv * p["tiles"] * p["parts"] * 64 * wq * wk < 1 << 32, (s, p)   # threads of the launch
