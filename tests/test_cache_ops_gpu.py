"""The operators around the 4-bit cache on the GPU, against their definitions
in 64 bits (codes, scales and values read back: exactly)."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from oracle import w4a4_oracle as O  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


def _rand(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g)


def _cache(ops, seed, n_pages, page, Hkv, D, k_scale=2.0 ** -8, v_scale=2.0 ** -9, sane=True):
    """A cache of random bytes; sane: scale codes of values around one, else any byte."""
    g = torch.Generator().manual_seed(seed)
    c = ops.make_kv_cache(n_pages, page, Hkv, D, k_scale, v_scale, device=DEV)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.randint(88 if sane else 0, 113 if sane else 256, t.shape, generator=g, dtype=torch.uint8))
    return c


def _values(codes, scales, g):
    """float64 [..., D] of packed codes and scales, scales read without sign and 0x7F as 480."""
    c = O.unpack_nibbles(codes.cpu().numpy())
    e = scales.cpu().numpy() & 0x7F
    s = np.where(e == 0x7F, 480.0, O.e4m3_value(np.minimum(e, 0x7E)))
    v = O.e2m1_value(c).reshape(*s.shape, 16) * s[..., None]
    return torch.from_numpy(v.reshape(c.shape)), float(np.float32(g))


# ----------------------------------------------------------------------------
# Writing and reading back
# ----------------------------------------------------------------------------
APPEND = [  # M, Hkv, D, page, dtype, k_scale, v_scale
    (1, 1, 64, 16, BF, 2.0 ** -8, 2.0 ** -9),
    (5, 2, 128, 16, BF, 2.0 ** -8, 2.0 ** -9),
    (77, 3, 256, 32, BF, 0.0031, 0.0017),
    (200, 8, 128, 64, F32, 0.0031, 0.0017),
    (130, 5, 64, 128, F32, 2.0 ** -8, 1.0),
    (300, 1, 128, 256, BF, 1e-30, 1e30),
]


@pytest.mark.parametrize("M,H,D,page,dtype,gk,gv", APPEND)
def test_append_writes_the_quantizers_codes(ops, M, H, D, page, dtype, gk, gv):
    n_pages = M // page + 3
    c = _cache(ops, 1, n_pages, page, H, D, gk, gv)
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    big = _rand(2, M, 2 * H + 1, D) * torch.exp(_rand(3, 1, 2 * H + 1, D))
    big[M // 2] = 0                                    # an all-zero token
    big[0, :, :16] *= 1e-6                             # scales that round to zero or below the normal ones
    big[-1, :, 16:32] *= 3e3                           # and that saturate
    kv = big.to(dtype).to(DEV)
    k, v = kv[:, :H], kv[:, H:2 * H]                   # views of one projection's output
    slots = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(4))[:M].int()
    if M > 3:
        slots[1], slots[2], slots[3] = -1, n_pages * page, 2 ** 31 - 1    # outside: skipped
    ops.cache_append(c, k, v, slots.to(DEV))
    torch.cuda.synchronize()
    for x, g, codes, scales, old_c, old_s in ((k, gk, c.k_codes, c.k_scales, before[0], before[1]),
                                              (v, gv, c.v_codes, c.v_scales, before[2], before[3])):
        want_c, want_s = old_c.cpu().numpy(), old_s.cpu().numpy()
        rows = x.float().cpu().numpy().reshape(M * H, D)
        nib, e, _, _ = O.quantize_nvfp4(rows, np.float32(g))
        nib, e = O.pack_nibbles(nib).reshape(M, H, D // 2), e.reshape(M, H, D // 16)
        for m, s in enumerate(slots.tolist()):
            if 0 <= s < n_pages * page:
                want_c[s // page, :, s % page], want_s[s // page, :, s % page] = nib[m], e[m]
        assert np.array_equal(scales.cpu().numpy(), want_s)      # the rest of the cache as it was
        assert np.array_equal(codes.cpu().numpy(), want_c)


def test_append_is_quantize_act_without_its_transform(ops):
    M, H, D = 64, 4, 128
    x = (_rand(5, M, H, D) * 3).to(BF).to(DEV)
    c = ops.make_kv_cache(4, 16, H, D, 0.005, 0.005, device=DEV)
    ops.cache_append(c, x, x, torch.arange(M, dtype=torch.int32, device=DEV))
    codes, scales = ops.quantize_act(x.view(M * H, D), None, "nvfp4", fwht_block=0, tensor_scale=0.005)
    assert torch.equal(c.k_codes.transpose(1, 2).reshape(M * H, D // 2), codes)
    assert torch.equal(c.v_scales.transpose(1, 2).reshape(M * H, D // 16), scales)


@pytest.mark.parametrize("D,page,H", [(64, 16, 3), (128, 64, 2), (256, 256, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("g", [2.0 ** -7, 0.0043])
def test_read_gives_every_byte_its_value(ops, D, page, H, dtype, g):
    c = _cache(ops, 6, 3, page, H, D, g, 1.0, sane=False)      # every code, every scale byte
    c.k_scales.view(-1)[:256] = torch.arange(256, dtype=torch.uint8, device=DEV)
    slots = torch.randint(0, 3 * page, (130,), generator=torch.Generator().manual_seed(7)).int()
    slots[5], slots[6], slots[7], slots[8] = -1, 3 * page, slots[9], -2 ** 31
    big = torch.full((130, 2 * H, D + 8), 7.0, dtype=dtype, device=DEV)
    k, v = ops.cache_read(c, slots.to(DEV), k=big[:, :H, :D], v=big[:, H:, :D])
    for got, codes, scales, gg in ((k, c.k_codes, c.k_scales, g), (v, c.v_codes, c.v_scales, 1.0)):
        vals, gg = _values(codes, scales, gg)
        want = torch.zeros(130, H, D, dtype=torch.float64)
        for m, s in enumerate(slots.tolist()):
            if 0 <= s < 3 * page:
                want[m] = vals[s // page, :, s % page]
        want = (want.float() * torch.tensor(gg, dtype=F32)).to(dtype)    # one fp32 product, then the dtype
        assert torch.equal(got.cpu(), want)
    assert bool((big[:, :, D:] == 7).all())


def test_round_trip_in_a_layer_pool_and_a_graph(ops):
    """Pages of two layers side by side; the append and the read captured, replayed with other tokens."""
    M, H, D, page, n = 40, 2, 128, 32, 4
    codes = torch.zeros(n, 2, 2, H, page, D // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(n, 2, 2, H, page, D // 16, dtype=torch.uint8, device=DEV)
    c = [ops.KVCache(codes[:, i, 0], scales[:, i, 0], codes[:, i, 1], scales[:, i, 1], 0.01, 0.01) for i in range(2)]
    k, v = (torch.zeros(M, H, D, dtype=BF, device=DEV) for _ in range(2))
    slots = torch.zeros(M, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.cache_append(c[1], k, v, slots)
        ops.cache_read(c[1], slots)
    torch.cuda.current_stream().wait_stream(side)
    codes.zero_(), scales.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.cache_append(c[1], k, v, slots)
        k2, v2 = ops.cache_read(c[1], slots)
    for seed in range(3):
        k.copy_((_rand(10 + seed, M, H, D) * 2).to(BF))
        v.copy_(_rand(20 + seed, M, H, D).to(BF))
        slots.copy_(torch.randperm(n * page, generator=torch.Generator().manual_seed(seed))[:M].int())
        graph.replay()
        torch.cuda.synchronize()
        for x, got in ((k, k2), (v, v2)):
            nib, e, _, _ = O.quantize_nvfp4(x.float().cpu().numpy().reshape(M * H, D), np.float32(0.01))
            want = torch.from_numpy(O.e2m1_value(nib).reshape(M * H, -1, 16) * O.e4m3_value(e)[..., None]).float()
            want = (want * torch.tensor(0.01, dtype=F32)).to(BF).view(M, H, D)
            assert torch.equal(got.cpu(), want)
        assert not codes[:, 0].any() and not scales[:, 0].any()     # the other layer's pages


def test_last_page_of_a_cache_past_4_gib(ops):
    """Offsets in a page pool pass 32 bits."""
    page, H, D = 256, 1, 256
    n = (1 << 32) // (page * D // 2) + 2
    c = ops.make_kv_cache(n, page, H, D, 2.0 ** -8, 2.0 ** -8, device=DEV)
    slots = torch.tensor([0, n * page - 1], dtype=torch.int32, device=DEV)
    k, v = (_rand(s, 2, H, D).to(BF).to(DEV) for s in (30, 31))
    ops.cache_append(c, k, v, slots)
    k2, v2 = ops.cache_read(c, slots)
    table = torch.tensor([[0], [n - 1]], dtype=torch.int32, device=DEV)
    far, near = c.k_codes[n - 1, 0, page - 1].cpu(), c.k_codes[0, 0, 0].cpu()
    for x, got in ((k, k2), (v, v2)):
        nib, e, _, _ = O.quantize_nvfp4(x.float().cpu().numpy().reshape(2, D), np.float32(2.0 ** -8))
        want = O.e2m1_value(nib).reshape(2, -1, 16) * O.e4m3_value(e)[..., None] * 2.0 ** -8
        assert torch.equal(got.cpu().double().view(2, D), torch.from_numpy(want.reshape(2, D)))
    nib = O.pack_nibbles(O.quantize_nvfp4(k.float().cpu().numpy().reshape(2, D), np.float32(2.0 ** -8))[0])
    assert np.array_equal(near.numpy(), nib[0]) and np.array_equal(far.numpy(), nib[1])
    # one visible key: the output is its value, which bf16 holds exactly
    one = ops.make_kv_cache(1, 16, 1, D, 2.0 ** -8, 2.0 ** -8, device=DEV)
    del one
    c.k_scales[n - 1].zero_(), c.v_scales[n - 1, :, :page - 1].zero_()
    q = torch.zeros(2, 1, 1, D, dtype=BF, device=DEV)
    out = ops.cache_attention(q, c, table, torch.tensor([1, page], dtype=torch.int32, device=DEV))
    assert torch.equal(out[0, 0, 0].cpu(), v2[0, 0].cpu())
    # 256 keys of weight 1 / 256, all values but the last zero; 2^-8 |v| is the output's rounding
    want = v2[1, 0].cpu().double() / page
    assert bool(((out[1, 0, 0].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs()).all())


# ----------------------------------------------------------------------------
# Attention over the cache
# ----------------------------------------------------------------------------
def _attention_reference(q, c, table, lens, causal, scale, max_len=None):
    """(out, A, smax) in float64: A[...] = sum p |v| / sum p, smax: the largest sum |q k| scale of a row."""
    B, T, Hq, D = q.shape
    G, page = Hq // c.Hkv, c.page
    kv, gk = _values(c.k_codes, c.k_scales, c.k_scale)
    vv, gv = _values(c.v_codes, c.v_scales, c.v_scale)
    q = q.double().cpu()
    table, lens = table.cpu(), lens.cpu()
    reach = table.shape[1] * page
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64)
    A, smax = torch.zeros_like(out), torch.zeros(B, T, Hq, 1, dtype=torch.float64)
    for b in range(B):
        n = max(0, int(lens[b]))
        j = torch.arange(min(n, reach if max_len is None else min(reach, max_len)))
        pg = table[b, j // page] if len(j) else torch.zeros(0, dtype=torch.int32)
        held = (pg >= 0) & (pg < c.n_pages)
        j, pg = j[held], pg[held].long()
        k, v = kv[pg, :, j % page] * gk, vv[pg, :, j % page] * gv          # [n, Hkv, D]
        for t in range(T):
            see = j < (n - T + t + 1 if causal else n)
            if not bool(see.any()):
                continue
            for h in range(Hq):
                ks, vs = k[see, h // G], v[see, h // G]
                s = ks @ q[b, t, h] * scale
                p = torch.softmax(s, 0)
                out[b, t, h], A[b, t, h] = p @ vs, p @ vs.abs()
                smax[b, t, h] = (ks.abs() @ q[b, t, h].abs()).max() * abs(scale)
    return out, A, smax


def _assert_attention(got, ref, n, vmax):
    """The output's rounding to bf16 is 2^-8 of it.  A probability enters the second product as fp16, off by
    2^-11 of it (below 2^-14, by 2^-25, against a sum of at least 2^5); a score is a sum of D products in 24 bits, D / 2 * 2^-24 of sum |q k| at most in any order of
    pairs of partial sums, plus exp2's argument and result (2^-22 of smax, 2^-22).  An error d of a score moves
    the output by 2 d A.  Sums of n probabilities and products in 24 bits: n 2^-24 A, twice."""
    out, A, smax = ref
    D = out.shape[-1]
    d = (D / 2 * 2.0 ** -24 + 2.0 ** -22) * smax + 2.0 ** -22
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2 * d + n * 2.0 ** -23) * A * 1.01 + n * 2.0 ** -30 * vmax
    err = (got.double().cpu() - out).abs()
    worst = (err - tol).max()
    assert bool((err <= tol).all()), f"over by {float(worst):.3g} at {int((err - tol).argmax())}"
    empty = A.sum(-1) == 0
    assert bool((got.cpu()[empty] == 0).all())


ATTN = [  # B, T, Hq, Hkv, D, page, pages, lens, causal
    (1, 1, 1, 1, 64, 16, 1, [1], True),
    (1, 1, 8, 1, 64, 16, 20, [317], True),
    (3, 1, 8, 2, 128, 16, 9, [0, 1, 144], False),
    (3, 1, 32, 8, 128, 64, 5, [63, 64, 65], True),
    (2, 1, 4, 4, 256, 32, 11, [352, 33], False),
    (2, 3, 10, 2, 128, 128, 3, [2, 384], True),         # a sequence shorter than its queries
    (2, 16, 4, 4, 128, 16, 25, [400, 16], True),
    (2, 17, 2, 2, 64, 32, 12, [300, 17], True),
    (1, 13, 8, 1, 256, 32, 17, [531], True),
    (2, 7, 21, 3, 128, 16, 30, [475, 222], False),
    (2, 50, 16, 4, 128, 16, 20, [310, 111], False),
    (1, 50, 6, 2, 64, 64, 6, [380], True),
    (2, 40, 8, 2, 256, 64, 5, [300, 40], True),
    (1, 33, 4, 4, 128, 256, 2, [511], True),
    (2, 130, 4, 2, 128, 16, 18, [288, 130], True),
    (1, 300, 2, 2, 128, 64, 9, [555], True),
    (1, 300, 3, 3, 64, 32, 20, [640], False),
    (1, 257, 1, 1, 256, 128, 4, [400], True),
    (2, 2, 2, 1, 128, 16, 300, [4790, 2000], True),
]


def _attention_case(ops, i, B, T, Hq, Hkv, D, page, pages, lens, absent=False, sane=True):
    n_pages = B * pages + 2
    c = _cache(ops, 100 + i, n_pages, page, Hkv, D, 2.0 ** -9 if D > 64 else 2.0 ** -8, 2.0 ** -9, sane=sane)
    g = torch.Generator().manual_seed(200 + i)
    table = torch.randperm(n_pages, generator=g)[:B * pages].view(B, pages).int()
    if absent:
        for b in range(B):
            for n, bad in enumerate((-1, n_pages, 2 ** 31 - 1, -2 ** 31)):
                table[b, (5 * n + b + 1) % pages] = bad
    wide = torch.full((B, pages + 3), 12345678, dtype=torch.int32)
    wide[:, :pages] = table
    big = (_rand(300 + i, B, T, Hq + 3, D + 8) * 1.2).to(BF).to(DEV)
    q = big[:, :, 1:Hq + 1, :D]                        # a view with strides of its own
    return q, c, wide.to(DEV)[:, :pages], torch.tensor(lens, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("i", range(len(ATTN)))
@pytest.mark.parametrize("split", [True, False])
def test_attention(ops, i, split):
    B, T, Hq, Hkv, D, page, pages, lens, causal = ATTN[i]
    q, c, table, lens = _attention_case(ops, i, B, T, Hq, Hkv, D, page, pages, lens, absent=i % 2 == 1 and pages > 8)
    ws = ops.make_cache_attention_workspace(B, T, Hq, Hkv, D, pages * page, device=DEV) if split else None
    big = torch.full((B, T, Hq + 1, D + 8), 3.0, dtype=BF, device=DEV)
    out = ops.cache_attention(q, c, table, lens, causal=causal, out=big[:, :, :Hq, :D], workspace=ws)
    ref = _attention_reference(q, c, table, lens, causal, D ** -0.5)
    _assert_attention(out, ref, pages * page, 6 * 2.0 ** 6 * c.v_scale)
    assert bool((big[:, :, Hq:] == 3).all()) and bool((big[..., D:] == 3).all())
    again = ops.cache_attention(q, c, table, lens, causal=causal, workspace=ws)
    assert torch.equal(out, again)                     # bit for bit


@pytest.mark.parametrize("scale", [0.0, -0.09, 1e-3, 0.5])
def test_attention_scales(ops, scale):
    q, c, table, lens = _attention_case(ops, 50, 2, 3, 4, 2, 128, 16, 20, [300, 77])
    out = ops.cache_attention(q, c, table, lens, scale=scale)
    _assert_attention(out, _attention_reference(q, c, table, lens, False, scale), 320, 6 * 2.0 ** 6 * c.v_scale)


@pytest.mark.parametrize("gain", [2.0 ** -100, 2.0 ** -30, 2.0 ** 40, 2.0 ** 100])
def test_attention_takes_queries_of_any_size(ops, gain):
    """Queries far outside fp16's range, with the cache's scale the other way."""
    q, c, table, lens = _attention_case(ops, 51, 1, 5, 4, 2, 128, 16, 12, [180])
    c2 = ops.KVCache(c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.k_scale / gain, c.v_scale)
    q2 = (q.float() * gain).to(BF)                     # exact
    out = ops.cache_attention(q2, c2, table, lens, causal=True)
    assert torch.equal(out, ops.cache_attention(q, c, table, lens, causal=True))
    _assert_attention(out, _attention_reference(q, c, table, lens, True, 128 ** -0.5), 192, 6 * 2.0 ** 6 * c.v_scale)


@pytest.mark.parametrize("T", [1, 60, 200])
def test_attention_never_sees_what_is_excluded(ops, T):
    """Bytes of other pages, of keys past a sequence's end and behind max_len do not change the result."""
    B, Hq, Hkv, D, page, pages = 2, 4, 2, 128, 32, 10
    q, c, table, lens = _attention_case(ops, 52, B, T, Hq, Hkv, D, page, pages, [250, 1000])
    ws = ops.make_cache_attention_workspace(B, T, Hq, Hkv, D, 280, device=DEV)
    one = ops.cache_attention(q, c, table, lens, causal=True, max_len=280, workspace=ws)
    seen = torch.zeros(c.n_pages, page, dtype=torch.bool)
    for b, n in enumerate((250, 280)):
        for j in range(n):
            seen[int(table[b, j // page]), j % page] = True
    hidden = ~seen.to(DEV)[:, None, :].expand(-1, Hkv, -1)
    for t, byte in ((c.k_codes, 0x77), (c.v_codes, 0xFF), (c.k_scales, 0x7F), (c.v_scales, 0xFF)):
        t[hidden] = byte
    two = ops.cache_attention(q, c, table, lens, causal=True, max_len=280, workspace=ws)
    assert torch.equal(one, two)
    ref = _attention_reference(q, c, table, lens, True, D ** -0.5, max_len=280)
    _assert_attention(two, ref, 288, 6 * 2.0 ** 6 * c.v_scale)


def test_attention_of_any_bytes_is_finite(ops):
    q, c, table, lens = _attention_case(ops, 53, 2, 5, 4, 2, 128, 16, 12, [180, 192], sane=False)
    assert bool(torch.isfinite(ops.cache_attention(q * 0.01, c, table, lens, causal=True).float()).all())


@pytest.mark.parametrize("B,T,Hq,Hkv,D", [(2, 1, 8, 2, 128), (1, 40, 4, 1, 128), (1, 150, 4, 4, 64), (1, 3, 8, 1, 256)])
def test_a_bad_query_row_stays_alone(ops, B, T, Hq, Hkv, D):
    q, c, table, lens = _attention_case(ops, 54, B, T, Hq, Hkv, D, 32, 10, [300] * B)
    q = q.clone()
    good = ops.cache_attention(q, c, table, lens)
    q[0, T // 2, 1, 5], q[0, T - 1, 0, 0] = float("nan"), float("inf")
    out = ops.cache_attention(q, c, table, lens)
    same = torch.ones(B, T, Hq, dtype=torch.bool, device=DEV)
    same[0, T // 2, 1] = same[0, T - 1, 0] = False
    assert torch.equal(out[same], good[same])
    assert bool(torch.isnan(out[0, T // 2, 1].float()).all())


def test_every_key_counts_once(ops):
    """Equal weights and one-hot values: each sequence's output counts its visible keys by channel."""
    B, T, H, D, page, pages = 3, 2, 1, 128, 16, 24
    c = ops.make_kv_cache(B * pages, page, H, D, 1.0, 1.0, device=DEV)
    for t in (c.k_codes, c.k_scales, c.v_codes):
        t.zero_()
    c.v_scales.fill_(0x38)                             # 1.0
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(9)).view(B, pages).int()
    lens = [384, 129, 7]
    count = torch.zeros(B, T, D, dtype=torch.float64)
    codes = torch.zeros(B * pages, H, page, D, dtype=torch.uint8)
    for b, n in enumerate(lens):
        for j in range(n):
            d = (j * 7 + j // 128) % D
            codes[int(table[b, j // page]), 0, j % page, d] = 2          # E2M1 1.0
            for t in range(T):
                count[b, t, d] += j < n - T + t + 1
    c.v_codes.copy_((codes[..., 0::2] | (codes[..., 1::2] << 4)).to(DEV))
    q = torch.zeros(B, T, H, D, dtype=BF, device=DEV)
    out = ops.cache_attention(q, c, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), causal=True,
                              workspace=ops.make_cache_attention_workspace(B, T, H, H, D, pages * page, device=DEV))
    for b, n in enumerate(lens):
        for t in range(T):
            # weights are exactly 1, sums of them exact: one division and one rounding
            want = count[b, t] / (n - T + t + 1)
            err = (out[b, t, 0].cpu().double() - want).abs()
            assert bool((err <= (2.0 ** -8 + 2.0 ** -21) * want).all())


@pytest.mark.parametrize("B,T,Hq,Hkv,D,pages", [(4, 1, 8, 2, 128, 40), (1, 50, 8, 2, 128, 40), (1, 300, 2, 2, 128, 40)])
def test_attention_in_graphs_and_on_streams(ops, B, T, Hq, Hkv, D, pages):
    q, c, table, lens = _attention_case(ops, 55, B, T, Hq, Hkv, D, 16, pages, [pages * 16] * B)
    q, lens = q.clone(), lens.clone()
    ws = [ops.make_cache_attention_workspace(B, T, Hq, Hkv, D, pages * 16, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.cache_attention(q, c, table, lens, causal=True, workspace=ws[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.cache_attention(q, c, table, lens, causal=True, workspace=ws[0])
    for n in range(3):
        q.copy_((_rand(60 + n, *q.shape)).to(BF))
        lens.copy_(torch.tensor([max(1, pages * 16 - 37 * (n + b)) for b in range(B)], dtype=torch.int32))
        eager = ops.cache_attention(q, c, table, lens, causal=True, workspace=ws[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    a = torch.cuda.Stream()
    torch.cuda.synchronize()
    one = ops.cache_attention(q, c, table, lens, causal=True, workspace=ws[0], stream=a)
    two = ops.cache_attention(q, c, table, lens, causal=True, workspace=ws[1])
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(two, eager)


def test_attention_of_nothing(ops):
    c = _cache(ops, 1, 2, 16, 2, 64)
    table = torch.zeros(2, 0, dtype=torch.int32, device=DEV)
    lens = torch.tensor([5, 9], dtype=torch.int32, device=DEV)
    out = ops.cache_attention(torch.ones(2, 3, 4, 64, dtype=BF, device=DEV), c, table, lens)
    assert out.shape == (2, 3, 4, 64) and not bool(out.any())
    one = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    neg = torch.tensor([-5, -2 ** 31], dtype=torch.int32, device=DEV)
    assert not bool(ops.cache_attention(torch.ones(2, 3, 4, 64, dtype=BF, device=DEV), c, one, neg, causal=True).any())
    assert not bool(ops.cache_attention(torch.ones(2, 3, 4, 64, dtype=BF, device=DEV), c, one, lens, max_len=0).any())
    assert ops.cache_attention(torch.ones(0, 3, 4, 64, dtype=BF, device=DEV), c, one[:0], lens[:0]).shape[0] == 0
    assert ops.cache_attention(torch.ones(2, 0, 4, 64, dtype=BF, device=DEV), c, one, lens).shape[1] == 0
    empty = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert ops.cache_read(c, empty)[0].shape == (0, 2, 64)
    ops.cache_append(c, torch.ones(0, 2, 64, device=DEV), torch.ones(0, 2, 64, device=DEV), empty)


def test_norms_and_positions_of_nothing(ops):
    x = torch.ones(0, 40, dtype=BF, device=DEV)
    mod = torch.ones(0, 40, device=DEV)                # a modulation a row
    for m in (mod, torch.ones(3, 40, device=DEV), None):
        xo, y = ops.gated_norm(x, x, gate=m, scale=m, shift=m)
        assert xo.shape == y.shape == (0, 40)
    q = torch.ones(0, 2, 64, dtype=BF, device=DEV)
    out = ops.rotary_axes(q, q, torch.ones(0, 1, dtype=torch.int32, device=DEV), ops.make_rotary_table([32], device=DEV))
    assert out[0].shape == out[1].shape == (0, 2, 64)
    q = torch.ones(3, 2, 64, dtype=BF, device=DEV)
    none = torch.ones(3, 0, 64, dtype=BF, device=DEV)  # no key heads
    pos = torch.ones(3, 1, dtype=torch.int32, device=DEV)
    assert torch.equal(ops.rotary_axes(q, none, pos, ops.make_rotary_table([32], device=DEV))[0],
                       ops.rotary_axes(q, None, pos, ops.make_rotary_table([32], device=DEV))[0])


# ----------------------------------------------------------------------------
# Rotary positions
# ----------------------------------------------------------------------------
ROTARY = [  # M, Hq, Hk, D, sections, interleaved, dtype, far
    (1, 1, 1, 2, [1], True, F32, 0),
    (3, 2, 0, 64, [32], True, BF, 0),
    (50, 16, 4, 128, [64], False, BF, 0),
    (400, 16, 4, 128, [64], False, BF, 1000000),
    (37, 5, 2, 128, [22, 21, 21], True, BF, 100000),
    (37, 5, 2, 128, [22, 21, 21], False, F32, 16000000),
    (70, 3, 3, 128, [16, 24, 24], False, BF, -3000),
    (9, 2, 1, 72, [12, 12, 12], True, F32, 0),
    (9, 2, 1, 72, [12, 12, 8], True, BF, 50),        # some channels behind the pairs
    (9, 7, 1, 80, [8, 0, 24], False, BF, 50),
    (33, 4, 4, 50, [10, 5, 3, 7], False, BF, 7),
    (33, 4, 4, 50, [5, 5, 3, 7], True, F32, 7),
    (2, 40, 24, 256, [64], False, BF, 3),
    (1500, 2, 2, 256, [44, 42, 42], True, BF, 0),
    (5, 1, 1, 1024, [512], True, BF, 0),
    (1, 32, 8, 128, [64], True, BF, 12345),
    (31, 3, 1, 128, [64], False, F32, 2 ** 25 + 1),
    (31, 3, 1, 128, [20, 20, 24], True, F32, -2 ** 26),
    (31, 3, 1, 50, [25], True, F32, 2 ** 26 - 61),
    (200, 9, 2, 64, [8, 8, 8], False, BF, 0),
    (200, 9, 2, 64, [12, 9, 9], True, F32, 0),
]


def _rotary_reference(x, pos, sections, interleaved):
    """(y, |u| + |w| of each value's pair) in float64."""
    x, pos = x.double().cpu(), pos.double().cpu()
    y, size = x.clone(), torch.zeros_like(x)
    P = sum(sections)
    i = 0
    for a, s in enumerate(sections):
        for j in range(s):
            ang = (pos[:, a] * 10000.0 ** (-j / s)).unsqueeze(1)
            c0, c1 = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
            u, w = x[:, :, c0], x[:, :, c1]
            y[:, :, c0], y[:, :, c1] = u * ang.cos() - w * ang.sin(), u * ang.sin() + w * ang.cos()
            size[:, :, c0] = size[:, :, c1] = u.abs() + w.abs()
            i += 1
    return y, size


def _assert_rotary(got, x, pos, sections, interleaved):
    """The angle is off by 2^-25 of a turn at most (2^-22.3), sine and cosine by 2^-23, three roundings in 24 bits:
    under 2^-21 of |u| + |w|; then the output's own rounding.  Channels behind the pairs are copied.
    int32 positions from 2^24 to 2^26: the table's 2^-52 of a turn times 2^26, and roundings of angles up to 1 and
    up to 1.5 turns, 2^-25 and 2^-24, are 7 2^-26 of a turn, with the rest under 2^-20."""
    want, size = _rotary_reference(x, pos, sections, interleaved)
    far = pos.numel() and pos.double().abs().max() > 2 ** 24
    tol = torch.finfo(x.dtype).eps / 2 * want.abs() + (2.0 ** -20 if far else 2.0 ** -21) * size
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    assert torch.equal(got[..., 2 * sum(sections):], x[..., 2 * sum(sections):])


@pytest.mark.parametrize("i", range(len(ROTARY)))
@pytest.mark.parametrize("how", ["new", "views", "in place"])
def test_rotary(ops, i, how):
    M, Hq, Hk, D, sections, inter, dtype, far = ROTARY[i]
    g = torch.Generator().manual_seed(i)
    pos = torch.randint(0, 60, (M, len(sections)), generator=g) + far
    pos = pos.int() if i % 2 == 0 or abs(far) > 2 ** 24 else pos.float() + 0.25 * (abs(far) < 1000)
    odd = 8 if how != "views" else 3                   # views: strides that are no multiple of anything
    big = _rand(400 + i, M, Hq + Hk + 1, D + odd).to(dtype).to(DEV)
    q, k = big[:, :Hq, :D], big[:, Hq:Hq + Hk, :D]
    if how == "new":
        q, k = q.contiguous(), k.contiguous()
    wide = torch.zeros(M, len(sections) + 2, dtype=pos.dtype)
    wide[:, :len(sections)] = pos
    table = ops.make_rotary_table(sections, device=DEV)
    before, q0, k0 = big.clone(), q.clone(), k.clone()
    kw = dict(q_out=q, k_out=k if Hk else None) if how == "in place" else {}
    qo, ko = ops.rotary_axes(q, k if Hk else None, wide.to(DEV)[:, :len(sections)], table, interleaved=inter, **kw)
    for x, got in ((q0, qo), (k0, ko)):
        if x.shape[1]:
            _assert_rotary(got, x, pos, sections, inter)
    if how == "in place":
        assert torch.equal(big[:, Hq + Hk:], before[:, Hq + Hk:]) and torch.equal(big[..., D:], before[..., D:])


def test_rotary_infinities_stay_in_their_pair(ops):
    M, H, D = 4, 3, 128
    x = _rand(1, M, H, D).to(BF).to(DEV)
    pos = torch.ones(M, 1, dtype=torch.int32, device=DEV)
    for inter, sections in ((True, [30]), (False, [32])):
        P = sum(sections)
        table = ops.make_rotary_table(sections, device=DEV)
        good, _ = ops.rotary_axes(x, None, pos, table, interleaved=inter)
        y = x.clone()
        y[1, 2, 5], y[2, 0, D - 1], y[0, 0, 2 * P] = float("inf"), float("nan"), float("inf")
        out, _ = ops.rotary_axes(y, None, pos, table, interleaved=inter)
        pair = [4, 5] if inter else [5, 5 + P]
        same = torch.ones(M, H, D, dtype=torch.bool, device=DEV)
        same[1, 2, pair] = False
        same[2, 0, D - 1] = same[0, 0, 2 * P] = False
        assert torch.equal(out[same], good[same])
        assert not bool(torch.isfinite(out[1, 2, pair].float()).any())
        assert bool(torch.isnan(out[2, 0, D - 1])) and float(out[0, 0, 2 * P]) == float("inf")
    assert ops.rotary_axes(x[:0], x[:0], pos[:0], table)[0].shape == (0, H, D)


# ----------------------------------------------------------------------------
# Gated residual and norms
# ----------------------------------------------------------------------------
GATED = [  # M, C, R, kind, h, post, gate, mod, affine, x, h dtype, y
    (1, 1, 1, "rms", True, False, True, True, False, F32, F32, F32),
    (1, 2048, 1, "layer", True, True, True, True, True, BF, BF, BF),
    (64, 2048, 1, "rms", True, True, True, True, True, BF, BF, BF),
    (7, 64, 7, "layer", True, False, True, True, False, F32, BF, BF),
    (12, 520, 4, "layer", True, True, False, True, True, F32, BF, F32),
    (777, 1155, 3, "layer", True, False, True, True, False, F32, F32, F32),
    (30, 3, 2, "layer", True, False, True, True, True, BF, BF, F32),
    (6, 5120, 2, "rms", True, True, True, True, True, F32, BF, BF),
    (5, 8192, 1, "layer", True, True, True, False, True, BF, F32, BF),
    (4, 16384, 2, "layer", True, True, True, True, True, F32, F32, F32),
    (4, 16383, 2, "rms", True, True, True, True, True, BF, F32, BF),
    (9, 1024, 3, "layer", False, False, False, True, False, BF, BF, BF),
    (9, 1001, 1, "rms", False, False, False, False, True, F32, BF, F32),
    (9, 4104, 1, "layer", True, False, False, False, False, BF, BF, BF),
    (300, 127, 300, "rms", True, True, True, True, False, F32, BF, BF),
    (2100, 256, 3, "layer", True, False, True, True, False, BF, BF, BF),
    # a row's last channels alone: at a wave's and a workgroup's end
    (13, 505, 13, "layer", True, True, True, True, True, BF, F32, BF),
    (13, 511, 1, "rms", True, True, True, True, True, F32, BF, F32),
    (3000, 513, 5, "layer", True, True, True, True, True, BF, BF, BF),
    (2, 8191, 1, "layer", True, True, True, True, True, BF, BF, BF),
    (3, 8185, 3, "rms", True, False, True, True, True, F32, BF, BF),
    (2, 16377, 2, "layer", True, True, True, True, True, BF, BF, BF),
]


def _gated_reference(x, h, gate, alpha, post, kind, weight, bias, scale, shift, eps):
    d = lambda t: None if t is None else t.double().cpu()  # noqa: E731
    x, h, gate, post, weight, bias, scale, shift = (d(t) for t in (x, h, gate, post, weight, bias, scale, shift))
    M, C = x.shape

    def rows(t):
        return t.repeat_interleave(M // t.shape[0], dim=0)

    u = torch.zeros_like(x) if h is None else h
    if post is not None:
        u = u / (u.square().mean(-1, keepdim=True) + eps).sqrt() * post
    if gate is not None:
        u = u * rows(gate)
    xn = alpha * x + u
    size = (alpha * x).abs() + u.abs()                 # what the sum is rounded from
    mean = xn.mean(-1, keepdim=True) if kind == "layer" else 0.0
    rs = 1.0 / ((xn - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    n = (xn - mean) * rs
    y, f = n, torch.ones_like(n)
    if weight is not None:
        y, f = y * weight, f * weight.abs()
    extra = torch.zeros_like(n)
    if bias is not None:
        y, extra = y + bias, extra + bias.abs()
    if scale is not None:
        y, f, extra = y * (1 + rows(scale)), f * (1 + rows(scale)).abs(), extra * (1 + rows(scale)).abs()
    if shift is not None:
        y, extra = y + rows(shift), extra + rows(shift).abs()
    return xn, size, n, rs, y, f, extra


def _assert_gated(xo, y, ref, post):
    """Sums of C values in 24 bits over at most 64 steps a thread and ten joins: 74 2^-24 of the sum of sizes at
    most, and half of that again for divisions and roots: 2^-17.  x' carries 2^-17 of h's part for the inner norm
    and four roundings; y the same of |n| (a value's own error through rs, and rs itself), of the mean's size, and
    of what is added.  Then each output's own rounding."""
    xn, size, n, rs, want, f, extra = ref
    e = 2.0 ** -17 if post else 2.0 ** -22
    tx = e * size
    if xo is not None:
        tol = torch.finfo(xo.dtype).eps / 2 * xn.abs() + tx + 1e-30
        err = (xo.double().cpu() - xn).abs()
        assert bool((err <= tol).all()), float((err - tol).max())
    if y is not None:
        mean_err = (2.0 ** -17 + e) * size.mean(-1, keepdim=True)
        ty = f * (rs * (tx + mean_err) + n.abs() * (2.0 ** -17 + e) + n.abs() * rs * size.mean(-1, keepdim=True) * e * 2)
        ty = ty + 2.0 ** -21 * (f * n.abs() + extra)
        err = (y.double().cpu() - want).abs()
        tol = torch.finfo(y.dtype).eps / 2 * want.abs() + ty * 1.01
        assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("i", range(len(GATED)))
@pytest.mark.parametrize("how", ["new", "views", "in place"])
def test_gated_norm(ops, i, how):
    M, C, R, kind, has_h, post, gate, mod, affine, xd, hd, yd = GATED[i]
    pad = {"new": 0, "views": 3, "in place": 8}[how]
    base = _rand(500 + i, M, C + pad) * 1.5 + 0.7
    bx = base.to(xd).to(DEV)
    bh = (_rand(600 + i, M, C + pad) * torch.exp(_rand(601 + i, 1, C + pad))).to(hd).to(DEV)
    x, h = bx[:, :C], bh[:, :C] if has_h else None
    mods = (_rand(700 + i, R, 3, C) * 0.3).to(DEV)
    if how == "in place":                              # modulations one after the other, not side by side
        mods = mods.transpose(0, 1).contiguous().transpose(0, 1)
    vec = [(1 + 0.2 * _rand(800 + i + n, C)).to(DEV) for n in range(3)]
    kw = dict(gate=mods[:, 2] if gate else None, scale=mods[:, 1] if mod else None, shift=mods[:, 0] if mod else None,
              post_weight=vec[0] if post else None, weight=vec[1] if affine else None, bias=vec[2] if affine else None,
              alpha=1.0 if i % 3 else 0.75, kind=kind, eps=1e-6)
    ref = _gated_reference(x, h, kw["gate"], kw["alpha"], kw["post_weight"], kind, kw["weight"], kw["bias"],
                           kw["scale"], kw["shift"], 1e-6)
    before = bx.clone()
    xo, y = ops.gated_norm(x, h, **kw, y_dtype=yd, x_out=x if how == "in place" else None)
    torch.cuda.synchronize()
    assert (xo is None) == (not has_h and how != "in place")
    _assert_gated(xo, y, ref, post)
    if how == "in place" and xo is not None:
        assert xo.data_ptr() == x.data_ptr() and torch.equal(bx[:, C:], before[:, C:])
    else:
        assert torch.equal(bx, before)
    only, none = ops.gated_norm(x, h, **{**kw, "scale": None, "shift": None}, norm=False,
                                x_out=torch.empty_like(x))
    assert none is None
    if how != "in place" and xo is not None:
        assert torch.equal(only, xo)


def test_gated_norm_far_from_zero_and_constant_rows(ops):
    """A mean of 1000 times the spread, and rows without spread."""
    M, C = 8, 2048
    x = (1000 + _rand(1, M, C)).to(DEV)
    x[3] = 5.0
    _, y = ops.gated_norm(x, y_dtype=F32, eps=1e-6)
    d = x.double().cpu()
    want = (d - d.mean(-1, keepdim=True)) / (d.var(-1, unbiased=False, keepdim=True) + 1e-6).sqrt()
    # the mean of values near 1000 is off by 2^-24 of it and little more: 2^-12 of the spread
    assert float((y.double().cpu() - want).abs().max()) <= 2.0 ** -11
    assert bool((y[3].abs() <= 1e-2).all())
    rows = torch.randn(3, 64, device=DEV)
    rows[1, 7] = float("nan")
    _, y = ops.gated_norm(rows, y_dtype=F32)
    assert bool(torch.isfinite(y[0]).all()) and bool(torch.isnan(y[1]).all()) and bool(torch.isfinite(y[2]).all())
    assert ops.gated_norm(rows[:0], rows[:0])[1].shape == (0, 64)


def test_gated_norm_and_rotary_in_a_graph(ops):
    M, C, H, D = 20, 512, 4, 128
    x, h = _rand(1, M, C).to(DEV), _rand(2, M, C).to(BF).to(DEV)
    gate = _rand(3, 1, C).to(DEV)
    pos = torch.arange(M, dtype=torch.int32, device=DEV).view(M, 1)
    table = ops.make_rotary_table([64], device=DEV)

    def step():
        _, y = ops.gated_norm(x, h, gate=gate, x_out=x)
        return ops.rotary_axes(y.view(M, H, D), None, pos, table)[0]

    x0 = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(x0)
    want = [step().clone() for _ in range(3)]
    x.copy_(x0)
    for n in range(3):
        pos_before = pos.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[n]) and torch.equal(pos, pos_before)


def test_copies_of_a_cache(ops):
    import copy
    import io
    c = _cache(ops, 40, 4, 16, 2, 64)
    slots = torch.arange(40, dtype=torch.int32, device=DEV)
    want = [t.clone() for t in ops.cache_read(c, slots)]
    buf = io.BytesIO()
    torch.save(c, buf)
    buf.seek(0)
    same, own, loaded = copy.copy(c), copy.deepcopy(c), torch.load(buf, weights_only=False)   # (written two lines above)
    c.k_codes.zero_()
    for d, shared in ((same, True), (own, False), (loaded, False)):
        k, v = ops.cache_read(d, slots)
        assert torch.equal(v, want[1]) and torch.equal(k, torch.zeros_like(k) if shared else want[0])
        assert (d.k_codes.data_ptr() == c.k_codes.data_ptr()) == shared
