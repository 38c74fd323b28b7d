"""Attention over the 4-bit cache at the ends of what its arguments may be: scales
near the ends of fp32's range, small probabilities in every kernel, one workspace
for histories of every length.  References in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_cache_ops_gpu as R  # noqa: E402  (values of a cache, tolerance)
from test_cache_attention_tiles_gpu import _reference  # noqa: E402

DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


@pytest.mark.parametrize("B,T,Hq,Hkv,D", [(1, 1, 8, 1, 64), (2, 13, 8, 1, 256), (1, 200, 8, 1, 128), (3, 700, 4, 2, 64)])
def test_one_workspace_serves_shorter_histories(ops, B, T, Hq, Hkv, D):
    page, longest = 64, 4096
    c = R._cache(ops, 3, B * longest // page, page, Hkv, D, 2.0 ** -9, 2.0 ** -9)
    table = torch.arange(c.n_pages, dtype=torch.int32, device=DEV).view(B, -1)
    q = R._rand(4, B, T, Hq, D).to(BF).to(DEV)
    ws = ops.make_cache_attention_workspace(B, T, Hq, Hkv, D, longest, device=DEV)
    for L in (1, 65, 700, 1280, 2100, 2240, 3000, 4096):
        lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
        out = ops.cache_attention(q, c, table, lens, max_len=L, workspace=ws)
        R._assert_attention(out, _reference(q, c, table, lens, False, D ** -0.5, L), L, 6 * 2.0 ** 6 * c.v_scale)
        own = ops.make_cache_attention_workspace(B, T, Hq, Hkv, D, L, device=DEV)
        assert torch.equal(out, ops.cache_attention(q, c, table, lens, max_len=L, workspace=own))


PEAKS = [  # T, Hq, D, split, rows of a workgroup
    (1, 2, 128, True, 16), (1300, 4, 128, True, 256), (4000, 8, 64, False, 256), (700, 4, 256, True, 128),
    (3000, 8, 256, False, 128),
]


@pytest.mark.parametrize("T,Hq,D,split,rows", PEAKS)
def test_small_weights_beside_a_peak(ops, T, Hq, D, split, rows):
    """One key ahead of 2^17 - 1 of 2^-20.7 of its weight, which together make 7 percent: subnormal fp16 numbers in
    the product and in the sum of the kernels for many rows."""
    L, page = 2 ** 17, 256
    c = R._cache(ops, 7, L // page, page, 1, D, 1.0, 1.0)
    for t, byte in ((c.k_codes, 0), (c.k_scales, 0x38), (c.v_codes, 0x22), (c.v_scales, 0x38)):
        t.fill_(byte)
    c.k_codes[0, 0, 0], c.v_codes[0, 0, 0] = 0x22, 0   # key 0: ones, its value zeros; the others: the reverse
    table = torch.arange(L // page, dtype=torch.int32, device=DEV).view(1, -1)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    q = torch.ones(1, T, Hq, D, dtype=BF, device=DEV)
    scale = 20.7 * math.log(2.0) / D
    ref = [r.expand(1, T, Hq, -1) for r in _reference(q[:, :1, :1], c, table, lens, False, scale, L)]
    ws = ops.make_cache_attention_workspace(1, T, Hq, 1, D, L, device=DEV) if split else None
    R._assert_attention(ops.cache_attention(q, c, table, lens, scale=scale, workspace=ws), ref, L, 1.0)
VALUES = [  # T, Hq, D, keys, split, rows of a workgroup
    (1, 2, 128, 2 ** 15, True, 16), (1, 2, 64, 2 ** 15, False, 16), (4096, 8, 128, 2 ** 12, False, 256),
    (404, 8, 128, 2 ** 14, True, 256),
]


@pytest.mark.parametrize("T,Hq,D,L,split,rows", VALUES)
@pytest.mark.parametrize("v_scale", [2.0 ** -122, 2.0 ** 110])
def test_value_scales_near_the_ends(ops, T, Hq, D, L, split, rows, v_scale):
    """The outputs are the same numbers, scaled: sums of 2^12 weights and more, 2^5 or 2^7 each, do not cost them bits."""
    page = 128
    c = R._cache(ops, 5, L // page, page, 1, D, 2.0 ** -12, v_scale)
    plain = ops.KVCache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.k_scale, 1.0)
    table = torch.arange(L // page, dtype=torch.int32, device=DEV).view(1, -1)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    q = R._rand(6, 1, T, Hq, D).to(BF).to(DEV)
    ws = ops.make_cache_attention_workspace(1, T, Hq, 1, D, L, device=DEV) if split else None
    out, want = (ops.cache_attention(q, x, table, lens, workspace=ws).double() for x in (c, plain))
    want = want * v_scale                              # exact
    # below bf16's normal numbers: half of their step, and of what ``want`` had beyond it
    err, tol = (out - want).abs(), (2.0 ** -134 + 2.0 ** -135) * 1.01 * (want.abs() <= 2.0 ** -126)
    assert bool((err <= tol).all()), float((err / want.abs().clamp(min=2.0 ** -126)).max())


KEYS = [(5, 16), (6000, 256)]   # T, rows of a workgroup


@pytest.mark.parametrize("T,rows", KEYS)
@pytest.mark.parametrize("gain", [2.0 ** 112, 2.0 ** 125])
def test_keys_of_the_smallest_scales(ops, T, rows, gain):
    """Queries near bf16's largest over keys whose scale is a subnormal number: the scores are the same."""
    q, c, table, lens = R._attention_case(ops, 51, 1, T, 4, 2, 128, 16, 30, [470])
    q = q.clamp(-7, 7)
    small = ops.KVCache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.k_scale / gain, c.v_scale)
    out = ops.cache_attention((q.float() * gain).to(BF), small, table, lens, max_len=480)
    assert torch.equal(out, ops.cache_attention(q, c, table, lens, max_len=480))


@pytest.mark.parametrize("T,rows", KEYS)
def test_scores_of_nothing_under_the_largest_scales(ops, T, rows):
    """Queries of zero make scores of zero, however large scale * k_scale: the mean of the values."""
    q, c, table, lens = R._attention_case(ops, 53, 1, T, 4, 2, 128, 16, 30, [470])
    big = ops.KVCache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, 2.0 ** 127, c.v_scale)
    zero = torch.zeros_like(q)
    assert torch.equal(ops.cache_attention(zero, big, table, lens, scale=1e30, max_len=480),
                       ops.cache_attention(zero, c, table, lens, max_len=480))


@pytest.mark.parametrize("T,rows", KEYS)
def test_large_scores_under_a_small_scale(ops, T, rows):
    """Scores of 2^40 and more are still numbers: the largest takes all the weight, under either scale of the keys."""
    q, c, table, lens = R._attention_case(ops, 54, 1, T, 4, 2, 128, 16, 30, [470])
    q = q.clamp(-7, 7)
    gain = 2.0 ** 124
    big = ops.KVCache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, 2.0 ** 30, c.v_scale)
    small = ops.KVCache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, 2.0 ** 30 / gain, c.v_scale)
    out = ops.cache_attention((q.float() * gain).to(BF), small, table, lens, max_len=480)
    assert torch.equal(out, ops.cache_attention(q, big, table, lens, max_len=480))
    assert bool(torch.isfinite(out.float()).all())
