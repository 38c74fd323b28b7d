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


@pytest.mark.parametrize("T,rows", KEYS)
@pytest.mark.parametrize("log2", [8, 11, 13, 14, 15, 16, 17, 18, 19, 20, 22, 26, 40, 70, 100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_of_any_size(ops, T, rows, log2, sign):
    """A key ahead of the others takes all the weight, also where a step of the scores is more than the whole range
    of the weights.  A score is off by (D / 2 2^-24 + 2^-22) smax (see _assert_attention): rows with a second key
    within twice that and 40 are not compared."""
    q, c, table, lens = R._attention_case(ops, 55, 1, T, 4, 2, 128, 16, 30, [470])
    big = ops.KVCache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, 2.0 ** log2, c.v_scale)
    out = ops.cache_attention(q, big, table, lens, scale=sign * 128 ** -0.5, max_len=480)
    assert bool(torch.isfinite(out.float()).all())
    kv, _ = R._values(c.k_codes, c.k_scales, 1.0)
    vv, _ = R._values(c.v_codes, c.v_scales, 1.0)
    at = table[0].cpu().long()
    clear = 0
    for h in range(4):
        k = kv[at, h // 2].reshape(480, 128)[:470].to(DEV) * 2.0 ** log2 * sign * 128 ** -0.5
        v = vv[at, h // 2].reshape(480, 128)[:470].to(DEV) * c.v_scale
        x = q[0, :, h].double()
        s = x @ k.t().contiguous()
        smax = (x.abs() @ k.abs().t().contiguous()).amax(-1)
        top = s.topk(2, dim=-1)
        gap = top.values[:, 0] - top.values[:, 1]
        far = gap > 2.02 * (64 * 2.0 ** -24 + 2.0 ** -22) * smax + 40
        clear += int(far.sum())
        want = v[top.indices[:, 0]]
        err = (out[0, :, h].double() - want).abs()[far]
        assert bool((err <= 2.0 ** -8 * want.abs()[far] + 2.0 ** -30).all()), float(err.max())
    assert clear > 3 * T


SHIFTED = [  # T, Hq, D, keys, split, rows of a workgroup
    (5, 8, 128, 480, False, 16), (5, 8, 64, 1920, True, 16), (5, 8, 256, 480, False, 16), (3000, 8, 64, 480, False, 256),
    (3000, 8, 128, 480, False, 256), (3000, 8, 256, 480, False, 128), (404, 8, 128, 2 ** 14, True, 256),
]


@pytest.mark.parametrize("T,Hq,D,L,split,rows", SHIFTED)
@pytest.mark.parametrize("gain", [2.0 ** 9, 2.0 ** 10, 2.0 ** 12])
@pytest.mark.parametrize("shift", ["up", "down", "up then none", "down then none then up", "none then up", "by keys", "by blocks"])
def test_scores_beside_each_other_far_from_zero(ops, T, Hq, D, L, split, rows, gain, shift):
    """Scores of a few units on top of plus or minus 2^19, 2^20 or 2^22 in one channel.  They are multiples of 1 / 8
    (quarters times halves): beside 2^20 exact in fp32, whose last place there is 1 / 8.  Beside 2^22 it is 1 / 2: each
    score is off by half of that, d = 1 / 4, a weight by a factor of e^d at most and its sum too, the output by
    (e^(2 d) - 1) A < 0.65 A."""
    page = 16
    c = R._cache(ops, 61, L // page, page, 1, D, 1.0, 2.0 ** -9)
    g = torch.Generator().manual_seed(62)
    codes = torch.zeros(L, D, dtype=torch.uint8)
    codes[:, 16] = torch.randint(0, 16, (L,), generator=g)               # -6 to 6
    n, j = L // 3, torch.arange(L)
    up = {"up": j >= 0, "down": j < 0, "up then none": j < n, "down then none then up": j >= 2 * n, "none then up": j >= n,
          "by keys": j % 2 == 0, "by blocks": j // 64 % 3 == 1}[shift]
    down = {"down": j >= 0, "down then none then up": j < n, "by blocks": j // 64 % 3 == 0}.get(shift, j < 0)
    codes[up, 0], codes[down, 0] = 6, 14                                 # 4 and -4 times a scale of 256
    c.k_codes.copy_((codes[:, 0::2] | codes[:, 1::2] << 4).view(L // page, 1, page, D // 2))
    c.k_scales.fill_(0x38)
    c.k_scales[..., 0] = 0x78
    table = torch.arange(L // page, dtype=torch.int32, device=DEV).view(1, -1)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    q = torch.zeros(1, T, Hq, D, dtype=BF, device=DEV)
    q[..., 0] = gain
    q[..., 16] = (torch.randint(-4, 5, (1, T, Hq), generator=g) / 4).to(BF).to(DEV)
    ws = ops.make_cache_attention_workspace(1, T, Hq, 1, D, L, device=DEV) if split else None
    out = ops.cache_attention(q, c, table, lens, scale=1.0, max_len=L, workspace=ws)
    ref, A, smax = _reference(q, c, table, lens, False, 1.0, L)
    # (where scores are exact, so are their differences: an error like that of scores of a few units)
    smax.fill_(16.0 if gain < 2.0 ** 11 else 0.325 / (D / 2 * 2.0 ** -24 + 2.0 ** -22))
    R._assert_attention(out, (ref, A, smax), L, 6 * 2.0 ** 6 * c.v_scale)
