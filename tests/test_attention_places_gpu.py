"""Prefix attention on every tile, with and without parts: each key counted
once, excluded places that hold NaN and Inf, bad values that rows see, packed
strides and negative scales.  References in 64 bits on the GPU."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_dense_ops_gpu import BF16, F32

# (head width, tile of the plan, cut into parts): B, T, Hq, Hkv, P, S, workspace
SHAPES = {
    (64, 0, False): (1, 5, 12, 3, 797, 22, False),
    (64, 0, True): (2, 12, 1, 1, 915, 121, True),
    (64, 1, False): (1, 9, 3, 1, 162, 27, True),
    (64, 1, True): (59, 3, 12, 3, 2398, 19, True),
    (64, 2, False): (30, 87, 12, 4, 270, 112, False),
    (64, 2, True): (38, 6, 21, 3, 5700, 16, True),
    (64, 3, False): (61, 112, 8, 1, 463, 91, True),
    (64, 3, True): (43, 31, 14, 2, 2064, 9, True),
    (128, 0, False): (1, 3, 4, 1, 319, 69, False),
    (128, 0, True): (1, 2, 16, 4, 3062, 11, True),
    (128, 1, False): (27, 30, 12, 3, 219, 11, True),
    (128, 1, True): (2, 1, 4, 1, 749, 65, True),
    (128, 2, False): (72, 6, 28, 4, 487, 29, False),
    (128, 2, True): (17, 10, 32, 4, 1036, 225, True),
    (128, 3, False): (33, 84, 12, 3, 831, 84, False),
    (128, 3, True): (36, 35, 8, 4, 1376, 57, True),
    (256, 0, False): (16, 1, 6, 3, 219, 9, False),
    (256, 0, True): (2, 5, 3, 3, 893, 143, True),
    (256, 1, False): (47, 31, 12, 4, 364, 112, False),
    (256, 1, True): (39, 12, 12, 4, 1380, 55, True),
}
IDS = ["D%d-%d%s" % (d, c, "-parts" if p else "") for d, c, p in SHAPES]
# the tile for many rows keeps four buffers of 64 prefix keys: every remainder, whole and partial last blocks
RING = [0, 1, 63, 64, 65, 128, 129, 191, 192, 250, 256, 257, 320, 383, 449, 512, 577]
RING_SHAPE = {64: (61, 112, 8, 1, 70), 128: (64, 64, 32, 8, 64)}   # B, T, Hq, Hkv, S without a workspace


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


class _Case:
    """Masks of a call and, per sequence, which of its keys each row sees."""

    def __init__(self, g, B, T, P, S, causal, keep):
        self.B, self.T, self.P, self.S, self.causal = B, T, P, S, causal
        self.lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        self.lens[0] = S
        self.keep = None
        if keep:                                     # runs of keys, block edges among them, and single ones
            k = torch.rand(P, generator=g, device="cuda") < 0.85
            k[P // 3:P // 2] = False
            k[62:66] = torch.tensor([True, False, True, False], device="cuda")[:max(0, min(4, P - 62))]
            k[max(0, P - P // 40):] = False
            self.keep = k
        t = torch.arange(T, device="cuda")
        n = self.lens.view(B, 1).expand(B, T).long()
        self.lim = (n - T + 1 + t).clamp(min=0).minimum(n) if causal else n       # own keys of a row

    def kept(self):
        return torch.ones(self.P, dtype=torch.bool, device="cuda") if self.keep is None else self.keep

    def poison(self, kp, vp, ko, vo):
        """NaN and Inf wherever no row looks."""
        if self.keep is not None:
            kp[~self.keep], vp[~self.keep] = math.nan, math.inf
        gone = torch.arange(self.S, device="cuda") >= self.lens.view(-1, 1)
        ko[gone], vo[gone] = math.nan, -math.inf


def _layouts(B, T, Hq, Hkv, D, P, S, packed):
    """q, k_prefix, v_prefix, k_own, v_own, out: contiguous, or as slices of
    packed buffers (padded rows, K and V interleaved, heads outermost)."""
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    if not packed:
        return z(B, T, Hq, D), z(P, Hkv, D), z(P, Hkv, D), z(B, S, Hkv, D), z(B, S, Hkv, D), z(B, T, Hq, D)
    cache, own = z(P, 2, Hkv, D + 8), z(Hkv, B, S, 2, D)
    return (z(B, T, Hq + 3, D)[:, :, 2:Hq + 2], cache[:, 0, :, :D], cache[:, 1, :, :D], own[:, :, :, 0].permute(1, 2, 0, 3),
            own[:, :, :, 1].permute(1, 2, 0, 3), z(T, B, Hq, 2 * D)[..., D:].permute(1, 0, 2, 3))


def _call(ops, c, tensors, scale, workspace):
    q, kp, vp, ko, vo, out = tensors
    B, T, Hq, D = q.shape
    P, Hkv, S = kp.shape[0], kp.shape[1], ko.shape[1]
    print(f"[attn] {(B, T, Hq, Hkv, D, P, S)} causal={c.causal} keep={c.keep is not None} scale={scale} ws={workspace}",
          flush=True)
    ws = ops.make_prefix_attention_workspace(B, T, Hq, Hkv, D, P, S) if workspace else None
    ops.prefix_attention(q, kp, vp, ko, vo, own_len=c.lens, prefix_keep=c.keep, causal=c.causal, scale=scale, out=out,
                         workspace=ws)
    torch.cuda.synchronize()


def _reference(c, q, kp, vp, ko, vo, scale, b):
    """Sequence b in 64 bits and its error bound; excluded places hold finite numbers here."""
    T, Hq, D = q.shape[1:]
    P, Hkv = kp.shape[:2]
    G = Hq // Hkv
    k = torch.cat([kp, ko[b]]).double().repeat_interleave(G, 1).permute(1, 2, 0).contiguous()
    v = torch.cat([vp, vo[b]]).double().repeat_interleave(G, 1).permute(1, 0, 2).contiguous()
    qb = q[b].double().permute(1, 0, 2).contiguous()
    s = torch.matmul(qb, k) * scale
    hide = torch.cat([(~c.kept()).expand(T, P), torch.arange(c.S, device="cuda") >= c.lim[b].view(T, 1)], 1)
    p = torch.nan_to_num(torch.softmax(s.masked_fill(hide, -math.inf), -1))
    o, mag = torch.matmul(p, v).permute(1, 0, 2), torch.matmul(p, v.abs()).permute(1, 0, 2)
    sc = (torch.matmul(qb.abs(), k.abs()).amax(-1) * abs(scale)).t().unsqueeze(-1)
    # probabilities rounded to bf16, scores off by a few fp32 roundings of their terms, output rounded
    return o, BF16 * o.abs() + (1.01 * BF16 + 2 * D * F32 * sc + 1e-5) * mag + 1e-30


def _random(g, tensors):
    q, kp, vp, ko, vo, _ = tensors
    for t in (kp, vp, ko, vo):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    q.copy_(torch.randn(q.shape, generator=g, device="cuda") * 1.5)
    return [t.clone() for t in (q, kp, vp, ko, vo)]


def _sequences(B):
    return sorted(set(range(min(B, 4))) | {B // 2, B - 1})


def _poisoned(ops, D, B, T, Hq, Hkv, P, S, workspace, causal, packed, scale, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = _Case(g, B, T, P, S, causal, True)
    tensors = _layouts(B, T, Hq, Hkv, D, P, S, packed)
    clean = _random(g, tensors)
    c.poison(*tensors[1:5])
    _call(ops, c, tensors, scale, workspace)
    out = tensors[5]
    assert bool(torch.isfinite(out.float()).all())
    for b in _sequences(B):
        want, tol = _reference(c, *clean, scale, b)
        err = (out[b].double() - want).abs()
        assert bool((err <= tol).all()), (b, float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("key", SHAPES, ids=IDS)
@pytest.mark.parametrize("causal,packed", [(True, False), (False, True)])
def test_excluded_places_hold_anything(ops, key, causal, packed):
    B, T, Hq, Hkv, P, S, ws = SHAPES[key]
    scale = (-1 if packed else 1) * key[0] ** -0.5
    _poisoned(ops, key[0], B, T, Hq, Hkv, P, S, ws, causal, packed, scale, seed=P + S)


def _once(ops, D, B, T, Hq, Hkv, P, S, workspace, causal, packed, keep, classes):
    """Zero queries weigh all keys alike.  A key's value is one in the column of
    its class and zero elsewhere, so a row's output is the share of its keys in
    each class: a key dropped, doubled or wrongly let in moves a column by more
    than its rounding (all sums are whole numbers, exact in 32 bits)."""
    g = torch.Generator(device="cuda").manual_seed(P)
    c = _Case(g, B, T, P, S, causal, keep)
    tensors = _layouts(B, T, Hq, Hkv, D, P, S, packed)
    _, kp, vp, ko, vo, out = tensors
    j = torch.arange(P + S, device="cuda")
    hot = torch.nn.functional.one_hot(classes(j, D) % D, D)
    kp.fill_(1.0), ko.fill_(1.0)
    vp.copy_(hot[:P].unsqueeze(1).expand(P, Hkv, D))
    vo.copy_(hot[P:].view(1, S, 1, D).expand(B, S, Hkv, D))
    c.poison(kp, vp, ko, vo)
    _call(ops, c, tensors, None, workspace)
    prefix = (hot[:P] * c.kept().unsqueeze(1)).sum(0)
    own = torch.cat([torch.zeros(1, D, dtype=torch.long, device="cuda"), hot[P:].cumsum(0)])
    count = prefix + own[c.lim]                                       # B, T, D
    n = count.sum(-1, keepdim=True)
    want = (count.double() / n.clamp(min=1)).unsqueeze(2)
    assert int(count.max()) < 120                                     # one key is more than two roundings
    err = (out.double() - want).abs()
    tol = (BF16 + 4 * F32) * want
    assert bool((err <= tol).all()), (float((err - tol).max()), [int(i) for i in torch.nonzero(err > tol)[0]])


@pytest.mark.parametrize("key", SHAPES, ids=IDS)
@pytest.mark.parametrize("causal,packed,keep", [(True, False, True), (False, True, False), (False, False, True)])
def test_every_key_once(ops, key, causal, packed, keep):
    B, T, Hq, Hkv, P, S, ws = SHAPES[key]
    _once(ops, key[0], B, T, Hq, Hkv, P, S, ws, causal, packed, keep, lambda j, D: j)
    _once(ops, key[0], B, T, Hq, Hkv, P, S, ws, causal, packed, keep, lambda j, D: 5 * j + j // D)


@pytest.mark.parametrize("P", RING)
@pytest.mark.parametrize("D", [64, 128])
def test_ring_of_prefix_blocks(ops, D, P):
    B, T, Hq, Hkv, S = RING_SHAPE[D]
    for keep in (False, True):
        _once(ops, D, B, T, Hq, Hkv, P, S, False, True, keep, keep, lambda j, D: j)
    _poisoned(ops, D, B, T, Hq, Hkv, P, S, False, True, False, -0.11, seed=P)


@pytest.mark.parametrize("key", SHAPES, ids=IDS)
@pytest.mark.parametrize("causal", [True, False])
def test_bad_values_stay_with_their_rows(ops, key, causal):
    """NaN or Inf among a sequence's own values reaches the rows that see it, and no other row."""
    D = key[0]
    B, T, Hq, Hkv, P, S, ws = SHAPES[key]
    g = torch.Generator(device="cuda").manual_seed(S)
    c = _Case(g, B, T, P, S, causal, True)
    tensors = _layouts(B, T, Hq, Hkv, D, P, S, False)
    clean = _random(g, tensors)
    G = Hq // Hkv
    hit = torch.zeros(B, T, Hq, dtype=torch.bool, device="cuda")
    marks = [(0, 0, 0, 3, math.nan), (0, S - 1, Hkv - 1, D - 1, math.inf), (B // 2, S // 2, 0, 8, -math.inf),
             (B - 1, S // 3, Hkv // 2, D // 2 + 1, math.nan), (B - 1, S - 1, 0, 0, math.inf)]
    for b, j, h, d, bad in marks:
        tensors[4][b, j, h, d] = bad
        hit[b, :, h * G:(h + 1) * G] |= (j < c.lim[b]).view(T, 1)
    _call(ops, c, tensors, None, ws)
    out = tensors[5]
    assert bool(hit.any()) and not bool(torch.isfinite(out[hit].float()).all(-1).any())
    for b in _sequences(B):
        want, tol = _reference(c, *clean, D ** -0.5, b)
        ok = ~hit[b]
        err = (out[b].double() - want).abs()[ok]
        assert bool((err <= tol[ok]).all()), b
