"""A workspace of cache_attention made for the longest history that a program meets
serves every shorter one (host code; no GPU needed)."""
import os
import random
import shutil

import pytest

pytest.importorskip("torch")

from test_cache_attention_plan_cpu import ROOT, plans  # noqa: F401  (the plan, built with g++)

pytestmark = [pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++"),
              pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "libw4a4.so")),
                                 reason="libw4a4.so not built")]

SIZES = [  # B, T, Hq, Hkv, D
    (1, 1, 8, 1, 64), (2, 13, 8, 1, 256), (8, 50, 16, 4, 128), (64, 1, 32, 8, 128), (1, 200, 8, 1, 128),
    (4, 1, 32, 8, 128), (2, 1560, 16, 16, 128), (16, 16, 32, 4, 256), (3, 700, 4, 2, 64), (1, 1, 1, 1, 128),
]


def _lengths():
    r = random.Random(11)
    return sorted({0, 1, 63, 64, 65, 65536, 65537, 1 << 30} | set(range(64, 9000, 64)) | {int(2 ** r.uniform(0, 30)) for _ in range(300)})


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_the_longest_history_s_workspace_covers_the_shorter_ones(plans, size):  # noqa: F811
    from w4a4_post_quantized_channel_amd import ops
    B, T, Hq, Hkv, D = size
    lengths = _lengths()
    most = 0
    for L, p in zip(lengths, plans([(*size, L, True) for L in lengths])):
        if p["parts"] > 1:                             # sums, maximum and output of every part of a row, fp32
            most = max(most, p["parts"] * B * T * Hq * (D + 2) * 4)
        assert ops.cache_attention_workspace_size(*size, L) >= most, L


def test_it_is_no_larger_than_some_shorter_history_needs(plans):  # noqa: F811
    from w4a4_post_quantized_channel_amd import ops
    for size in SIZES:
        B, T, Hq, Hkv, D = size
        needs = {p["parts"] * B * T * Hq * (D + 2) * 4 if p["parts"] > 1 else 0
                 for p in plans([(*size, 64 * n, True) for n in range(1, 513)])}
        assert ops.cache_attention_workspace_size(*size, 64 * 512) == max(needs)


def test_the_range_tests_meet_the_kernels_they_name(plans):  # noqa: F811
    from test_cache_attention_range_gpu import KEYS, PEAKS, SHIFTED, VALUES
    shapes = [((1, T, Hq, 1, D, L, split), rows) for T, Hq, D, L, split, rows in SHIFTED]
    shapes += [((1, T, Hq, 1, D, 2 ** 17, split), rows) for T, Hq, D, split, rows in PEAKS]
    shapes += [((1, T, Hq, 1, D, L, split), rows) for T, Hq, D, L, split, rows in VALUES]
    shapes += [((1, T, 4, 2, 128, 480, False), rows) for T, rows in KEYS]
    for (s, rows), p in zip(shapes, plans([s for s, _ in shapes])):
        assert p["rows"] == rows and (p["parts"] > 1) == s[-1], (s, p)
