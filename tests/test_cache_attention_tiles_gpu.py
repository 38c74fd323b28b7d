"""Every tile of the attention over the 4-bit cache, with and without parts, at
the ends of what it covers: ragged histories, absent pages, rows that see
nothing, strides.  References in 64 bits on the GPU."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_cache_ops_gpu as R  # noqa: E402  (values of a cache, tolerance)

DEV = "cuda"

# (D, rows of a workgroup, its waves, in parts, several row tiles of a sequence (None: any)):
# B, T, Hq, Hkv, max_len, with workspace
SHAPES = {
    (128, 16, 4, False, False): (257, 1, 1, 1, 33, True),
    (128, 16, 4, False, True): (1, 523, 8, 1, 66, True),
    (128, 16, 4, True, False): (13, 1, 10, 5, 1557, True),
    (128, 16, 4, True, True): (11, 17, 3, 3, 1767, True),
    (128, 16, 8, False, False): (1, 4, 4, 1, 700, False),
    (128, 16, 8, False, True): (1, 8, 3, 1, 257, False),
    (128, 16, 8, True, False): (1, 1, 9, 1, 1562, True),
    (128, 16, 8, True, True): (1, 18, 1, 1, 1639, True),
    (128, 256, 8, False, None): (6, 400, 4, 2, 300, False),
    (128, 256, 8, True, None): (5, 404, 4, 4, 577, True),
    (128, 32, 8, False, False): (44, 6, 12, 3, 257, True),
    (128, 32, 8, False, True): (1, 1447, 3, 3, 264, False),
    (128, 32, 8, True, False): (13, 4, 5, 1, 4642, True),
    (128, 32, 8, True, True): (1, 181, 4, 1, 2603, True),
    (256, 128, 4, False, None): (1, 347, 25, 5, 32, False),
    (256, 128, 4, True, None): (4, 724, 3, 1, 580, True),
    (256, 16, 4, False, False): (129, 1, 6, 2, 32, False),
    (256, 16, 4, False, True): (10, 162, 5, 1, 141, True),
    (256, 16, 4, True, False): (22, 1, 4, 4, 1026, True),
    (256, 16, 4, True, True): (1, 116, 6, 3, 2652, True),
    (256, 16, 8, False, False): (1, 1, 2, 1, 257, False),
    (256, 16, 8, False, True): (1, 10, 2, 1, 266, False),
    (256, 16, 8, True, False): (1, 1, 2, 1, 10569, True),
    (256, 16, 8, True, True): (1, 3, 8, 1, 10055, True),
    (64, 16, 4, False, False): (129, 1, 2, 2, 32, True),
    (64, 16, 4, False, True): (33, 6, 12, 4, 32, True),
    (64, 16, 4, True, False): (22, 1, 2, 2, 2683, True),
    (64, 16, 4, True, True): (1, 5, 5, 1, 1068, True),
    (64, 16, 8, False, False): (1, 1, 1, 1, 258, True),
    (64, 16, 8, False, True): (1, 9, 2, 1, 272, False),
    (64, 16, 8, True, False): (1, 1, 1, 1, 5009, True),
    (64, 16, 8, True, True): (1, 17, 1, 1, 4919, True),
    (64, 256, 8, False, None): (4, 600, 4, 2, 330, False),
    (64, 256, 8, True, None): (1, 1365, 6, 3, 654, True),
    (64, 32, 8, False, False): (44, 7, 9, 3, 269, False),
    (64, 32, 8, False, True): (1, 1029, 4, 1, 269, True),
    (64, 32, 8, True, False): (4, 4, 15, 3, 5122, True),
    (64, 32, 8, True, True): (1, 228, 2, 1, 4160, True),
}


def _reference(q, c, table, lens, causal, scale, max_len):
    """_attention_reference by products of a sequence and KV head."""
    B, T, Hq, D = q.shape
    G, page = Hq // c.Hkv, c.page
    kv, gk = R._values(c.k_codes, c.k_scales, c.k_scale)
    vv, gv = R._values(c.v_codes, c.v_scales, c.v_scale)
    kv, vv = kv.to(DEV) * gk, vv.to(DEV) * gv
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=DEV)
    A, smax = torch.zeros_like(out), torch.zeros(B, T, Hq, 1, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = max(0, int(lens[b]))
        j = torch.arange(min(n, table.shape[1] * page, max_len), device=DEV)
        pg = table[b, j // page] if len(j) else j.int()
        held = (pg >= 0) & (pg < c.n_pages)
        j, pg = j[held], pg[held].long()
        if not len(j):
            continue
        end = n - T + torch.arange(T, device=DEV) + 1 if causal else torch.full((T,), n, device=DEV)
        see = (j < end.unsqueeze(1)).repeat_interleave(G, 0)             # [T G, n]
        for h in range(c.Hkv):
            k, v = kv[pg, h, j % page], vv[pg, h, j % page]
            x = q[b, :, h * G:(h + 1) * G].double().reshape(T * G, D)
            s = (x @ k.t().contiguous() * scale).masked_fill(~see, -torch.inf)
            p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
            size = (x.abs() @ k.abs().t().contiguous()).masked_fill(~see, 0).amax(-1) * abs(scale)
            at = (b, slice(None), slice(h * G, (h + 1) * G))
            out[at], A[at] = (p @ v).view(T, G, D), (p @ v.abs()).view(T, G, D)
            smax[at] = size.view(T, G, 1)
    return out.cpu(), A.cpu(), smax.cpu()


def _case(key, page, seed):
    D = key[0]
    B, T, Hq, Hkv, L, ws = SHAPES[key]
    from w4a4_post_quantized_channel_amd import ops
    pages = -(-L // page)
    c = R._cache(ops, seed, B * pages + 1, page, Hkv, D, 2.0 ** -9, 2.0 ** -9)
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(B * pages + 1, generator=g)[:B * pages].view(B, pages).int()
    lens = torch.randint(0, L + 1, (B,), generator=g).int()
    lens[0] = L
    if B > 2:
        lens[1], lens[2] = 0, 1
    for b in range(B):                                                   # a few pages that nobody holds
        for bad in (-1, B * pages + 1, -2 ** 31):
            if pages > 6:
                table[b, int(torch.randint(0, pages, (1,), generator=g))] = bad
    if B > 3:
        table[3] = -1                                                    # a sequence whose history is gone
    q = (R._rand(seed + 1, B, T, Hq, D) * 1.3).to(torch.bfloat16).to(DEV)
    work = ops.make_cache_attention_workspace(B, T, Hq, Hkv, D, L, device=DEV) if ws else None
    return ops, q, c, table.to(DEV), lens.to(DEV), L, work


@pytest.mark.parametrize("key", list(SHAPES), ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("causal,page", [(False, 16), (True, 64), (True, 256)])
def test_tile(key, causal, page):
    ops, q, c, table, lens, L, ws = _case(key, page, 1000 + 7 * list(SHAPES).index(key) + page)
    assert (ws is not None) == SHAPES[key][5] or not key[3]
    out = ops.cache_attention(q, c, table, lens, causal=causal, max_len=L, workspace=ws)
    ref = _reference(q, c, table, lens, causal, key[0] ** -0.5, L)
    R._assert_attention(out, ref, L + page, 6 * 2.0 ** 6 * c.v_scale)
    assert torch.equal(out, ops.cache_attention(q, c, table, lens, causal=causal, max_len=L, workspace=ws))


@pytest.mark.parametrize("key", [(128, 16, 4, True, False), (128, 16, 8, True, True), (128, 32, 8, True, True), (128, 256, 8, True, None),
                                 (256, 128, 4, True, None)],
                         ids=lambda k: "-".join(map(str, k)))
def test_a_later_maximum(key):
    """Scores that climb by far more than the running maximum may lag, key after key, and fall again."""
    ops, q, c, table, lens, L, ws = _case(key, 16, 77)
    n = c.n_pages * 16
    table.copy_(torch.arange(table.numel(), dtype=torch.int32).view(table.shape))
    ramp = torch.arange(n, device=DEV)
    ramp = torch.minimum(ramp % 600, 600 - ramp % 600) // 12             # scale codes 64 .. 89: factors of 1 to 9
    c.k_scales.copy_((64 + ramp).view(c.n_pages, 1, 16, 1).expand_as(c.k_scales).to(torch.uint8))
    out = ops.cache_attention(q * 3, c, table, lens, max_len=L, workspace=ws)
    ref = _reference(q * 3, c, table, lens, False, key[0] ** -0.5, L)
    R._assert_attention(out, ref, L + 16, 6 * 2.0 ** 6 * c.v_scale)


@pytest.mark.parametrize("L,T", [(16383, 1), (16384, 33), (9001, 700)])
def test_long_histories(L, T):
    """Thousands of keys of nearly equal weight: what small probabilities add up to."""
    from w4a4_post_quantized_channel_amd import ops
    Hq, Hkv, D, page = 2, 1, 128, 128
    pages = -(-L // page)
    c = R._cache(ops, 5, pages, page, Hkv, D, 2.0 ** -12, 2.0 ** -9)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, pages)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    q = R._rand(6, 1, T, Hq, D).to(torch.bfloat16).to(DEV)
    ws = ops.make_cache_attention_workspace(1, T, Hq, Hkv, D, L, device=DEV)
    for w in (ws, None):
        out = ops.cache_attention(q, c, table, lens, causal=True, max_len=L, workspace=w)
        R._assert_attention(out, _reference(q, c, table, lens, True, D ** -0.5, L), L, 6 * 2.0 ** 6 * c.v_scale)


@pytest.mark.parametrize("T", [1, 17, 150])
def test_a_peak_leaves_the_rest_its_weight(T):
    """One key ahead of 2^19 - 1 of 2^-22.7 of its weight, which together make 8 percent: two and a half of fp16's
    smallest steps each, were the peak's probability 1."""
    from w4a4_post_quantized_channel_amd import ops
    L, D, page = 2 ** 19, 128, 256
    c = R._cache(ops, 7, L // page, page, 1, D, 1.0, 1.0)
    for t, byte in ((c.k_codes, 0), (c.k_scales, 0x38), (c.v_codes, 0x22), (c.v_scales, 0x38)):
        t.fill_(byte)
    c.k_codes[0, 0, 0], c.v_codes[0, 0, 0] = 0x22, 0                     # key 0: ones, its value zeros; the others: the reverse
    table = torch.arange(L // page, dtype=torch.int32, device=DEV).view(1, -1)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    q = torch.ones(1, T, 2, D, dtype=torch.bfloat16, device=DEV)
    scale = (24.0 - math.log2(2.5)) * math.log(2.0) / D
    ref = _reference(q, c, table, lens, False, scale, L)
    for w in (ops.make_cache_attention_workspace(1, T, 2, 1, D, L, device=DEV), None):
        R._assert_attention(ops.cache_attention(q, c, table, lens, scale=scale, workspace=w), ref, L, 1.0)


@pytest.mark.parametrize("T,D", [(4, 128), (40, 128), (300, 128), (150, 256)])
def test_sequences_longer_than_their_cache(T, D):
    """lens beyond max_len or the table: causal rows keep their positions, keys that do not exist are not seen."""
    from w4a4_post_quantized_channel_amd import ops
    c = R._cache(ops, 8, 60, 16, 2, D, 2.0 ** -9, 2.0 ** -9)
    table = torch.randperm(60, generator=torch.Generator().manual_seed(1)).view(3, 20).int().to(DEV)
    lens = torch.tensor([320 + T // 2, 2 ** 31 - 1, 301 + T // 3], dtype=torch.int32, device=DEV)
    q = R._rand(9, 3, T, 4, D).to(torch.bfloat16).to(DEV)
    for L in (320, 300, 4000):
        out = ops.cache_attention(q, c, table, lens, causal=True, max_len=L)
        R._assert_attention(out, _reference(q, c, table, lens, True, D ** -0.5, L), 320, 6 * 2.0 ** 6 * c.v_scale)


@pytest.mark.parametrize("seed", range(60))
def test_shapes_drawn_at_random(seed):
    import random
    from w4a4_post_quantized_channel_amd import ops
    r = random.Random(900 + seed)
    D, page, Hkv = r.choice([64, 128, 256]), r.choice([16, 32, 64, 128, 256]), r.choice([1, 1, 2, 3, 5])
    Hq, B = Hkv * r.choice([1, 2, 3, 5, 8]), r.choice([1, 2, 3, 7, 20])
    T, L = r.choice([1, 2, int(2 ** r.uniform(0, 9))]), int(2 ** r.uniform(0, 12.5))
    if B * T * Hq * L > 2 ** 26:
        B, T = 1, max(1, min(T, 2 ** 26 // (Hq * L)))
    causal, split, scale = r.random() < 0.5, r.random() < 0.7, r.choice([D ** -0.5, D ** -0.5, 0.3, -0.1])
    pages = -(-L // page) + r.choice([0, 0, 1])
    c = R._cache(ops, seed, B * pages + 2, page, Hkv, D, 2.0 ** -9 * r.choice([1.0, 1.3]), 0.0021)
    g = torch.Generator().manual_seed(seed)
    table = torch.randint(0, B * pages + 2, (B, pages), generator=g).int()   # pages that several hold
    table[torch.rand(B, pages, generator=g) < r.choice([0.0, 0.0, 0.3])] = -1
    lens = torch.randint(0, L + 1, (B,), generator=g).int()
    lens[r.randrange(B)] = L
    q = R._rand(seed + 5, B, T, Hq + 1, D).to(torch.bfloat16).to(DEV)[:, :, :Hq]
    out = torch.full((B, Hq, T + 1, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    into = out.transpose(1, 2)[:, :T]                                    # [B, Hq, T, D] in memory
    ws = ops.make_cache_attention_workspace(B, T, Hq, Hkv, D, L, device=DEV) if split else None
    table, lens = table.to(DEV), lens.to(DEV)
    ops.cache_attention(q, c, table, lens, causal=causal, scale=scale, max_len=L, out=into, workspace=ws)
    R._assert_attention(into, _reference(q, c, table, lens, causal, scale, L), L + page, 6 * 2.0 ** 6 * c.v_scale)
    assert bool(torch.isnan(out[:, :, T].float()).all())
