"""The 16-bit operators (prefix attention, bf16 linear, group norm) against
plain 64-bit implementations on the CPU, through the public entry points.

Tolerances come from the arithmetic: the unit roundoff of the output type
(2^-8 for bf16's 8-bit significand, 2^-24 for fp32's 24-bit one) and of the
bf16 probabilities, and the worst-case growth of fp32 sums.
"""
import math
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _check(got, want, tol):
    torch.cuda.synchronize()
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err - tol).max()), float(err.max()))


# ----------------------------------------------------------------------------
# Prefix attention
# ----------------------------------------------------------------------------
def _attn_reference(q, kp, vp, ko, vo, lens, keep, causal, scale):
    """Output and its error bound, row by row in 64 bits; excluded keys are not touched."""
    B, T, Hq, D = q.shape
    P, Hkv = kp.shape[:2]
    G = Hq // Hkv
    out, tol = torch.zeros(B, T, Hq, D, dtype=torch.float64), torch.zeros(B, T, Hq, D, dtype=torch.float64)
    kept = torch.arange(P) if keep is None else torch.nonzero(keep.cpu().bool()).flatten()
    for b in range(B):
        n = ko.shape[1] if lens is None else min(max(int(lens[b]), 0), ko.shape[1])
        for t in range(T):
            m = max(0, min(n, n - T + 1 + t)) if causal else n
            for h in range(Hkv):
                k = torch.cat([kp[kept, h], ko[b, :m, h]]).double()
                v = torch.cat([vp[kept, h], vo[b, :m, h]]).double()
                if k.shape[0] == 0:
                    continue
                s = q[b, t, h * G:(h + 1) * G].double() @ k.t() * scale
                p = torch.softmax(s, -1)
                o, mag = p @ v, p @ v.abs()
                # probabilities rounded to bf16, scores off by a few fp32 roundings of their terms, output rounded
                sc = (q[b, t, h * G:(h + 1) * G].double().abs() @ k.abs().t()).amax(-1, keepdim=True) * abs(scale)
                rows = slice(h * G, (h + 1) * G)
                out[b, t, rows] = o
                tol[b, t, rows] = BF16 * o.abs() + (1.01 * BF16 + 2 * D * F32 * sc + 1e-5) * mag + 1e-30
    return out, tol


def _attn_case(ops, B, T, Hq, Hkv, D, P, S, causal, lens=None, keep=None, seed=0, scale=None, workspace=True, kv_gain=1.0,
               poison=False):
    g = _gen(seed)
    q = (torch.randn(B, T, Hq, D, generator=g) * 1.5).bfloat16()
    kp, vp = ((torch.randn(P, Hkv, D, generator=g) * kv_gain).bfloat16() for _ in range(2))
    ko, vo = ((torch.randn(B, S, Hkv, D, generator=g) * kv_gain).bfloat16() for _ in range(2))
    if keep is not None:
        keep = torch.rand(P, generator=g) < keep
    ref, tol = _attn_reference(q, kp, vp, ko, vo, lens, keep, causal, D ** -0.5 if scale is None else scale)
    if poison:                                   # whatever lies in excluded places must not matter
        if keep is not None:
            kp[~keep], vp[~keep] = math.nan, math.inf
        for b in range(B):
            n = S if lens is None else min(max(lens[b], 0), S)
            ko[b, n:], vo[b, n:] = math.nan, -math.inf
    dev = [t.cuda() for t in (q, kp, vp, ko, vo)]
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    kd = None if keep is None else keep.cuda()
    ws = ops.make_prefix_attention_workspace(B, T, Hq, Hkv, D, P, S) if workspace else None
    print(f"[attn] B={B} T={T} Hq={Hq} Hkv={Hkv} D={D} P={P} S={S} causal={causal} ws={ws is not None}", flush=True)
    out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.prefix_attention(*dev, own_len=ln, prefix_keep=kd, causal=causal, scale=scale, out=out, workspace=ws)
    _check(out, ref, tol)


ATTN = [
    # B, T, Hq, Hkv, D, P, S, causal, lens, keep
    (1, 1, 1, 1, 64, 1, 1, False, None, None),
    (1, 1, 8, 1, 64, 300, 17, True, None, None),
    (3, 1, 6, 2, 128, 129, 40, True, [0, 40, 23], None),
    (2, 5, 14, 2, 64, 0, 33, True, [33, 3], None),             # no prefix; early queries see nothing
    (2, 3, 4, 4, 128, 65, 0, False, None, None),               # no keys of its own
    (2, 2, 4, 2, 128, 0, 0, True, None, None),                 # no key at all: zeros
    (2, 2, 4, 2, 64, 70, 8, False, [0, 8], 0.0),               # prefix masked out entirely
    (4, 50, 8, 4, 128, 200, 50, False, None, 0.6),
    (2, 13, 8, 1, 256, 321, 130, True, [130, 70], 0.8),
    (5, 7, 3, 1, 128, 1000, 9, True, [9, 7, 3, 1, 0], None),
    (1, 33, 16, 2, 64, 640, 33, True, None, None),
    (70, 1, 4, 2, 128, 513, 20, True, [(i * 7) % 21 for i in range(70)], 0.9),
    (2, 129, 4, 1, 64, 257, 140, True, [140, 100], None),
    (1, 300, 2, 2, 128, 128, 64, False, None, None),
    (9, 4, 10, 5, 256, 66, 5, True, [5, 4, 3, 2, 1, 0, 5, 9, -3], None),   # lengths out of range are clamped
]


@pytest.mark.parametrize("case", ATTN, ids=[f"B{c[0]}T{c[1]}H{c[2]}-{c[3]}D{c[4]}P{c[5]}S{c[6]}" for c in ATTN])
@pytest.mark.parametrize("workspace", [True, False])
def test_attention(ops, case, workspace):
    B, T, Hq, Hkv, D, P, S, causal, lens, keep = case
    _attn_case(ops, B, T, Hq, Hkv, D, P, S, causal, lens, keep, seed=B + T + P, workspace=workspace, poison=True)


@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,S", [(64, 1, 32, 8, 128, 700, 30), (6, 64, 16, 2, 128, 320, 100),
                                              (2, 1, 8, 8, 64, 9000, 70)])
def test_attention_plans(ops, B, T, Hq, Hkv, D, P, S):
    """Shapes of the serving plans: a decoding batch, long chunks, a long prefix split over the card."""
    _attn_case(ops, B, T, Hq, Hkv, D, P, S, True, [max(1, S - 3 * i) for i in range(B)], None, seed=5)


@pytest.mark.parametrize("workspace", [True, False])
def test_attention_large_scores(ops, workspace):
    """Scores in the hundreds: the running maximum moves and nothing overflows."""
    _attn_case(ops, 2, 9, 4, 2, 128, 500, 40, True, None, None, seed=3, scale=1.0, workspace=workspace, kv_gain=3.0)
    _attn_case(ops, 2, 9, 4, 2, 128, 500, 40, True, None, None, seed=4, scale=-0.7, workspace=workspace, kv_gain=3.0)


def test_attention_strides_and_streams(ops):
    """Operands as slices of packed buffers, output in a strided buffer, on a side stream."""
    g = _gen(11)
    B, T, Hq, Hkv, D, P, S = 3, 4, 6, 2, 64, 150, 21
    qkv = torch.randn(B, T, 16, D, generator=g).bfloat16()                 # q heads sit beside other heads
    cache = torch.randn(P, 2, Hkv, D + 8, generator=g).bfloat16()          # padded rows, K and V interleaved
    own = torch.randn(Hkv, B, S, 2, D, generator=g).bfloat16()             # heads outermost
    ref, tol = _attn_reference(qkv[:, :, 5:11], cache[:, 0, :, :D], cache[:, 1, :, :D],
                               own[:, :, :, 0].permute(1, 2, 0, 3), own[:, :, :, 1].permute(1, 2, 0, 3), None, None,
                               False, D ** -0.5)
    s = torch.cuda.Stream()
    buf = torch.zeros(T, B, Hq, 2 * D, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        qd, cd, od = qkv.cuda(), cache.cuda(), own.cuda()
        out = buf[..., D:].permute(1, 0, 2, 3)
        ops.prefix_attention(qd[:, :, 5:11], cd[:, 0, :, :D], cd[:, 1, :, :D], od[:, :, :, 0].permute(1, 2, 0, 3),
                             od[:, :, :, 1].permute(1, 2, 0, 3), out=out,
                             workspace=ops.make_prefix_attention_workspace(B, T, Hq, Hkv, D, P, S))
    s.synchronize()
    _check(out, ref, tol)
    assert not buf[..., :D].any()


def test_attention_bad_values_stay_with_their_rows(ops):
    """A NaN or Inf among one sequence's values reaches the rows that see it, as NaN, and no other."""
    g = _gen(12)
    B, T, Hq, Hkv, D, P, S = 4, 6, 4, 2, 128, 90, 6
    q, kp, vp, ko, vo = ((torch.randn(*s, generator=g)).bfloat16() for s in
                         [(B, T, Hq, D), (P, Hkv, D), (P, Hkv, D), (B, S, Hkv, D), (B, S, Hkv, D)])
    ref, tol = _attn_reference(q, kp, vp, ko, vo, None, None, True, D ** -0.5)
    vo[1, 3, 1, 5], vo[2, 0, 0, 77] = math.nan, math.inf
    for ws in (None, ops.make_prefix_attention_workspace(B, T, Hq, Hkv, D, P, S)):
        out = ops.prefix_attention(q.cuda(), kp.cuda(), vp.cuda(), ko.cuda(), vo.cuda(), causal=True,
                                   workspace=ws).cpu()
        hit = torch.zeros(B, T, Hq, dtype=torch.bool)
        hit[1, 3:, 2:], hit[2, :, :2] = True, True
        _check(out[~hit], ref[~hit], tol[~hit])
        assert not torch.isfinite(out[hit]).all(-1).any()


def test_attention_repeats_bit_for_bit_and_in_a_graph(ops):
    """Same inputs, same bits; and replays of a captured call agree with the eager one."""
    g = _gen(13)
    B, T, Hq, Hkv, D, P, S = 8, 1, 16, 2, 128, 3000, 40
    mk = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    q, kp, vp, ko, vo = mk(B, T, Hq, D), mk(P, Hkv, D), mk(P, Hkv, D), mk(B, S, Hkv, D), mk(B, S, Hkv, D)
    ws = ops.make_prefix_attention_workspace(B, T, Hq, Hkv, D, P, S)
    want = ops.prefix_attention(q, kp, vp, ko, vo, workspace=ws)
    again = ops.prefix_attention(q, kp, vp, ko, vo, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(want.view(torch.int16), again.view(torch.int16))
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.prefix_attention(q, kp, vp, ko, vo, out=out, workspace=ws)
    for i in range(4):
        q.copy_(mk(B, T, Hq, D))
        graph.replay()
        eager = ops.prefix_attention(q, kp, vp, ko, vo, workspace=ops.make_prefix_attention_workspace(B, T, Hq, Hkv, D, P, S))
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), i


# ----------------------------------------------------------------------------
# bf16 linear
# ----------------------------------------------------------------------------
def _act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _linear_reference(x, w, bias, act, residual, y_half):
    x, w = x.double(), w.double()
    z = x @ w.t()
    dz = 2 * x.shape[1] * F32 * (x.abs() @ w.abs().t())     # fp32 products and sums, any order
    if bias is not None:
        z = z + bias.double()
        dz = dz + F32 * z.abs()
    if act == "swiglu":
        n = w.shape[0] // 2
        s, u = _act64(z[:, :n], "silu"), z[:, n:]
        ds, du = 1.2 * dz[:, :n] + 16 * F32 * s.abs(), dz[:, n:]
        y, dy = s * u, ds * u.abs() + s.abs() * du + ds * du
    else:
        y = _act64(z, act)
        # the activations' slopes are at most 1.2; their own evaluation is good to a few ulp
        dy = 1.2 * dz + (0 if act in ("none", "relu") else 16 * F32 * (y.abs() + z.abs() * (y.abs() > 1e-30)))
    if residual is not None:
        y = y + residual.double()
    return y, dy + (F32 + y_half) * y.abs() + 1e-30


LINEAR = [
    # M, N, K, act, bias, residual, y_dtype
    (1, 1, 8, "none", None, False, torch.float32),
    (1, 2048, 512, "none", torch.float32, True, torch.float32),
    (1, 131, 4104, "gelu", torch.bfloat16, True, torch.bfloat16),
    (3, 77, 264, "swiglu", torch.float32, True, torch.bfloat16),
    (17, 300, 1000, "silu", torch.bfloat16, False, torch.bfloat16),
    (33, 64, 2056, "relu", torch.float32, True, torch.float32),
    (64, 256, 4096, "none", torch.bfloat16, True, torch.bfloat16),
    (64, 200, 72, "swiglu", None, False, torch.float32),
    (65, 129, 136, "gelu_tanh", torch.float32, True, torch.bfloat16),
    (127, 513, 520, "swiglu", torch.bfloat16, True, torch.bfloat16),
    (200, 96, 64, "gelu", None, False, torch.float32),
    (300, 700, 328, "none", None, True, torch.float32),
    (513, 1030, 200, "silu", torch.float32, True, torch.bfloat16),
    (1100, 1290, 264, "gelu_tanh", torch.bfloat16, False, torch.bfloat16),
    (1025, 520, 136, "swiglu", torch.float32, True, torch.float32),
    (2100, 1800, 72, "relu", torch.float32, True, torch.bfloat16),
]


def _linear_inputs(M, N, K, act, bias, residual, y_dtype, seed):
    g = _gen(seed)
    nw = 2 * N if act == "swiglu" else N
    x, w = torch.randn(M, K, generator=g).bfloat16(), (torch.randn(nw, K, generator=g) / math.sqrt(K) * 2).bfloat16()
    b = None if bias is None else (torch.randn(nw, generator=g) * 0.5).to(bias)
    r = torch.randn(M, N, generator=g).to(y_dtype) if residual else None
    return x, w, b, r


@pytest.mark.parametrize("case", LINEAR, ids=[f"{c[0]}x{c[1]}x{c[2]}-{c[3]}" for c in LINEAR])
@pytest.mark.parametrize("workspace", [True, False])
def test_linear(ops, case, workspace):
    M, N, K, act, bias, residual, y_dtype = case
    x, w, b, r = _linear_inputs(M, N, K, act, bias, residual, y_dtype, seed=M + N + K)
    want, tol = _linear_reference(x, w, b, act, r, BF16 if y_dtype == torch.bfloat16 else F32)
    dev = lambda t: None if t is None else t.cuda()
    ws = ops.make_bf16_linear_workspace(M, N, K, act) if workspace else None
    print(f"[linear] {M}x{N}x{K} {act} ws={ws is not None}", flush=True)
    y = torch.full((M, N), 7.0, dtype=y_dtype, device="cuda")
    ops.bf16_linear(dev(x), dev(w), bias=dev(b), act=act, residual=dev(r), y=y, workspace=ws)
    _check(y, want, tol)


@pytest.mark.parametrize("M", [5, 130, 700])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_strides_and_in_place_residual(ops, M, act):
    """Padded rows whose padding holds NaN, output inside a wider buffer that is also the residual."""
    N, K = 150, 344
    x, w, b, r = _linear_inputs(M, N, K, act, torch.float32, True, torch.bfloat16, seed=M)
    want, tol = _linear_reference(x, w, b, act, r, BF16)
    xp = torch.full((M, K + 24), math.nan, dtype=torch.bfloat16, device="cuda")
    wp = torch.full((w.shape[0], K + 40), math.inf, dtype=torch.bfloat16, device="cuda")
    yp = torch.full((M + 2, N + 13), 3.0, dtype=torch.bfloat16, device="cuda")
    xp[:, :K], wp[:, :K], yp[1:-1, 4:N + 4] = x.cuda(), w.cuda(), r.cuda()
    y = yp[1:-1, 4:N + 4]
    ops.bf16_linear(xp[:, :K], wp[:, :K], bias=b.cuda(), act=act, residual=y, y=y,
                    workspace=ops.make_bf16_linear_workspace(M, N, K, act))
    _check(y, want, tol)
    rest = yp.clone()
    rest[1:-1, 4:N + 4] = 3.0
    assert (rest == 3.0).all()


def test_linear_activation_tails(ops):
    """Arguments far out on both sides of each activation."""
    z = torch.cat([torch.linspace(-60, 60, 97), torch.tensor([-1e4, 1e4, -300.0, 300.0, 0.0, -0.0])]).bfloat16()
    x = torch.zeros(z.numel(), 8, dtype=torch.bfloat16)
    x[:, 0] = z
    w = torch.zeros(16, 8, dtype=torch.bfloat16)
    w[:, 0] = 1.0
    for act in ["none", "relu", "gelu", "gelu_tanh", "silu"]:
        want, tol = _linear_reference(x, w, None, act, None, F32)
        y = ops.bf16_linear(x.cuda(), w.cuda(), act=act, y_dtype=torch.float32)
        # exp and erfc far out: relative accuracy is lost below the smallest normal only
        _check(y, want, tol + 1e-36)


# ----------------------------------------------------------------------------
# Group norm
# ----------------------------------------------------------------------------
def _norm_reference(x, groups, weight, bias, eps, act, half):
    N, S, C = x.shape
    v = x.double().view(N, S, groups, C // groups)
    mean = v.mean(dim=(1, 3), keepdim=True)
    var = ((v - mean) ** 2).mean(dim=(1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    hat = ((v - mean) * rstd).reshape(N, S, C)
    w = torch.ones(C).double() if weight is None else weight.double()
    b = torch.zeros(C).double() if bias is None else bias.double()
    # the mean is good to an ulp or two of the group's largest value, the variance to a few parts in 10^6
    top = v.abs().amax(dim=(1, 3), keepdim=True)
    dhat = (4 * F32 * top * rstd).expand_as(v).reshape(N, S, C) + 4e-6 * hat.abs()
    z = hat * w + b
    dz = dhat * w.abs() + 4 * F32 * (hat.abs() * w.abs() + b.abs())
    y = _act64(z, act)
    dy = 1.2 * dz + (0 if act in ("none", "relu") else 16 * F32 * (y.abs() + z.abs()))
    return y, dy + (F32 + half) * y.abs() + 1e-30


NORM = [
    # N, S, C, groups, dtype, act, affine, offset
    (1, 1, 8, 8, torch.float32, "none", True, 0.0),            # one value a group: the variance is zero
    (1, 1, 64, 4, torch.bfloat16, "silu", True, 0.0),
    (2, 77, 40, 8, torch.float32, "none", True, 3.0),
    (3, 130, 96, 32, torch.bfloat16, "silu", True, 0.0),
    (1, 1000, 6, 2, torch.bfloat16, "silu", True, 0.0),        # narrow rows, odd channel counts
    (2, 333, 7, 7, torch.float32, "gelu", False, 0.0),
    (1, 5000, 384, 32, torch.bfloat16, "silu", True, 1.0),
    (1, 40000, 96, 32, torch.bfloat16, "silu", True, 0.0),
    (4, 9000, 20, 4, torch.bfloat16, "relu", False, 0.0),
    (1, 60000, 24, 1, torch.float32, "gelu_tanh", True, 0.0),
    (2, 17, 1280, 32, torch.bfloat16, "silu", True, 0.0),
    (1, 3, 4100, 4, torch.float32, "silu", True, 0.0),
    (2, 2000, 64, 16, torch.float32, "none", True, 3000.0),    # a mean far above the deviation
]


@pytest.mark.parametrize("case", NORM, ids=[f"{c[0]}x{c[1]}x{c[2]}g{c[3]}-{c[5]}" for c in NORM])
@pytest.mark.parametrize("workspace", [True, False])
def test_group_norm(ops, case, workspace):
    N, S, C, groups, dtype, act, affine, offset = case
    g = _gen(N + S + C)
    x = (torch.randn(N, S, C, generator=g) * torch.exp(0.3 * torch.randn(C, generator=g)) + offset).to(dtype)
    w, b = (torch.randn(C, generator=g) for _ in range(2)) if affine else (None, None)
    want, tol = _norm_reference(x, groups, w, b, 1e-5, act, BF16 if dtype == torch.bfloat16 else F32)
    dev = lambda t: None if t is None else t.cuda()
    ws = ops.make_group_norm_workspace(N, S, C, groups) if workspace else None
    print(f"[norm] {N}x{S}x{C} groups={groups} {act} ws={ws is not None}", flush=True)
    _check(ops.group_norm_act(dev(x), groups, dev(w), dev(b), act=act, workspace=ws), want, tol)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_group_norm_strided_and_in_place(ops, dtype):
    g = _gen(21)
    N, S, C, groups = 2, 300, 48, 4
    buf = torch.randn(N, S + 3, C + 9, generator=g).to(dtype)
    want, tol = _norm_reference(buf[:, 2:-1, 5:C + 5].contiguous(), groups, None, None, 1e-5, "silu",
                                BF16 if dtype == torch.bfloat16 else F32)
    d = buf.cuda()
    x = d[:, 2:-1, 5:C + 5]
    out = ops.group_norm_act(x, groups, workspace=ops.make_group_norm_workspace(N, S, C, groups))
    _check(out, want, tol)
    ops.group_norm_act(x, groups, out=x, workspace=ops.make_group_norm_workspace(N, S, C, groups))
    _check(x, want, tol)
    rest = d.clone()
    rest[:, 2:-1, 5:C + 5] = buf[:, 2:-1, 5:C + 5].cuda()
    assert torch.equal(rest.cpu(), buf)


def test_group_norm_constant_and_side_stream(ops):
    """A constant group has variance zero: the output is the bias exactly, eps or not far from it."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = torch.full((2, 500, 32), 1234.5, device="cuda")
        b = torch.arange(32, dtype=torch.float32, device="cuda")
        y = ops.group_norm_act(x, 8, None, b, act="none", workspace=ops.make_group_norm_workspace(2, 500, 32, 8))
    s.synchronize()
    assert torch.equal(y.cpu(), b.cpu().expand(2, 500, 32))


def test_linear_and_norm_repeat_bit_for_bit(ops):
    x, w, b, r = _linear_inputs(48, 320, 6000, "gelu", torch.float32, True, torch.float32, 9)
    ws = ops.make_bf16_linear_workspace(48, 320, 6000, "gelu")
    a = [ops.bf16_linear(x.cuda(), w.cuda(), bias=b.cuda(), act="gelu", residual=r.cuda(), y_dtype=torch.float32,
                         workspace=ws).cpu() for _ in range(3)]
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])
    f = torch.randn(1, 20000, 96, generator=_gen(3)).bfloat16().cuda()
    ws = ops.make_group_norm_workspace(1, 20000, 96, 32)
    a = [ops.group_norm_act(f, 32, workspace=ws).view(torch.int16).cpu() for _ in range(3)]
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])


# ----------------------------------------------------------------------------
# Shapes large enough for the large tiles, against 64 bits on the GPU
# ----------------------------------------------------------------------------
LARGE_ATTN = [
    # B, T, Hq, Hkv, D, P, S, causal, keep, workspace
    (16, 64, 32, 8, 128, 4003, 70, True, 0.7, True),
    (16, 64, 32, 8, 64, 4003, 70, False, None, True),
    (33, 64, 32, 8, 128, 300, 64, True, None, False),
    (64, 64, 32, 8, 128, 100, 64, False, 0.5, False),
    (64, 64, 32, 8, 64, 30, 10, True, None, False),
    (20, 50, 40, 5, 128, 1000, 50, False, 0.9, True),
    (8, 64, 16, 4, 256, 700, 64, True, 0.9, True),
]


def _attention_on_gpu(ops, B, T, Hq, Hkv, D, P, S, causal, keep, workspace, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    q, kp, vp, ko, vo = mk(B, T, Hq, D), mk(P, Hkv, D), mk(P, Hkv, D), mk(B, S, Hkv, D), mk(B, S, Hkv, D)
    lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    mask = None if keep is None else torch.rand(P, generator=g, device="cuda") < keep
    ws = ops.make_prefix_attention_workspace(B, T, Hq, Hkv, D, P, S) if workspace else None
    print(f"[attn] {(B, T, Hq, Hkv, D, P, S, causal, keep, workspace, seed)}", flush=True)
    out = ops.prefix_attention(q, kp, vp, ko, vo, own_len=lens, prefix_keep=mask, causal=causal, workspace=ws)
    G, pos, t = Hq // Hkv, torch.arange(S, device="cuda"), torch.arange(T, device="cuda")
    for b in range(B):
        k = torch.cat([kp, ko[b]]).double().repeat_interleave(G, 1).permute(1, 2, 0).contiguous()   # Hq, D, keys
        v = torch.cat([vp, vo[b]]).double().repeat_interleave(G, 1).permute(1, 0, 2).contiguous()
        qb = q[b].double().permute(1, 0, 2).contiguous()
        s = torch.matmul(qb, k) / math.sqrt(D)
        end = lens[b] - T + 1 + t if causal else lens[b].expand(T)
        hide = torch.zeros(T, P + S, dtype=torch.bool, device="cuda")
        if mask is not None:
            hide[:, :P] = ~mask
        hide[:, P:] = pos >= end.unsqueeze(1)
        p = torch.nan_to_num(torch.softmax(s.masked_fill(hide, -math.inf), -1))
        o, mag = torch.matmul(p, v).permute(1, 0, 2), torch.matmul(p, v.abs()).permute(1, 0, 2)
        sc = (torch.matmul(qb.abs(), k.abs()).amax(-1) / math.sqrt(D)).t().unsqueeze(-1)
        tol = BF16 * o.abs() + (1.01 * BF16 + 2 * D * F32 * sc + 1e-5) * mag + 1e-30
        err = (out[b].double() - o).abs()
        assert bool((err <= tol).all()), (b, float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("case", LARGE_ATTN, ids=[f"B{c[0]}T{c[1]}H{c[2]}-{c[3]}D{c[4]}P{c[5]}S{c[6]}" for c in LARGE_ATTN])
def test_attention_large_tiles(ops, case):
    _attention_on_gpu(ops, *case, seed=case[0] + case[5])


@pytest.mark.parametrize("seed", range(10))
def test_attention_random_shapes(ops, seed):
    """Sizes over the whole range, so that every tile, with and without parts, is met."""
    r = random.Random(seed)
    n = 0
    while n < 12:
        Hkv = r.choice([1, 2, 4, 5, 8])
        B, T = int(2 ** r.uniform(0, 6)), r.choice([1, int(2 ** r.uniform(0, 6.2))])
        Hq, D, P, S = Hkv * r.choice([1, 2, 3, 4, 7, 8]), r.choice([64, 128, 256]), int(2 ** r.uniform(0, 13)), int(2 ** r.uniform(0, 8.3))
        if B * T * Hq * (P + S) > 4e7:
            continue
        _attention_on_gpu(ops, B, T, Hq, Hkv, D, P, S, r.random() < 0.5, r.choice([None, 0.0, 0.5, 0.95]), r.random() < 0.7,
                          seed=100 * seed + n)
        n += 1


LARGE_LINEAR = [
    # M, N, K, act, bias, residual, y_dtype
    (4090, 5117, 520, "gelu_tanh", torch.float32, True, torch.bfloat16),
    (4096, 5120, 328, "gelu", torch.bfloat16, True, torch.float32),
    (2040, 4090, 520, "swiglu", torch.float32, True, torch.bfloat16),
    (2048, 4096, 520, "relu", None, False, torch.float32),
    (1000, 4090, 2056, "swiglu", torch.bfloat16, True, torch.float32),
    (1000, 8200, 2056, "none", torch.float32, True, torch.bfloat16),
]


@pytest.mark.parametrize("case", LARGE_LINEAR, ids=[f"{c[0]}x{c[1]}x{c[2]}-{c[3]}" for c in LARGE_LINEAR])
def test_linear_large_tiles(ops, case):
    M, N, K, act, bias, residual, y_dtype = case
    x, w, b, r = _linear_inputs(M, N, K, act, bias, residual, y_dtype, seed=M)
    dev = [None if t is None else t.cuda() for t in (x, w, b, r)]
    want, tol = _linear_reference(dev[0], dev[1], dev[2], act, dev[3], BF16 if y_dtype == torch.bfloat16 else F32)
    print(f"[linear large] {case}", flush=True)
    y = ops.bf16_linear(dev[0], dev[1], bias=dev[2], act=act, residual=dev[3], y_dtype=y_dtype,
                        workspace=ops.make_bf16_linear_workspace(M, N, K, act))
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("seed", range(8))
def test_linear_random_shapes(ops, seed):
    r = random.Random(seed)
    for n in range(10):
        M, N, K = int(2 ** r.uniform(0, 11)), int(2 ** r.uniform(0, 12)), 8 * int(2 ** r.uniform(0, 8.5))
        act = r.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
        y_dtype = r.choice([torch.bfloat16, torch.float32])
        x, w, b, res = _linear_inputs(M, N, K, act, r.choice([None, torch.float32, torch.bfloat16]), r.random() < 0.5, y_dtype,
                                      100 * seed + n)
        dev = [None if t is None else t.cuda() for t in (x, w, b, res)]
        want, tol = _linear_reference(dev[0], dev[1], dev[2], act, dev[3], BF16 if y_dtype == torch.bfloat16 else F32)
        ws = ops.make_bf16_linear_workspace(M, N, K, act) if r.random() < 0.7 else None
        print(f"[linear] {M}x{N}x{K} {act} {y_dtype} ws={ws is not None}", flush=True)
        y = ops.bf16_linear(dev[0], dev[1], bias=dev[2], act=act, residual=dev[3], y_dtype=y_dtype, workspace=ws)
        err = (y.double() - want).abs()
        assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("seed", range(8))
def test_group_norm_random_shapes(ops, seed):
    r = random.Random(seed)
    for n in range(8):
        groups = r.choice([1, 2, 3, 8, 32])
        N, S, C = r.randint(1, 4), int(2 ** r.uniform(0, 14)), groups * r.choice([1, 2, 3, 5, 8, 12, 16, 40])
        dtype, act = r.choice([torch.bfloat16, torch.float32]), r.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        g = _gen(100 * seed + n)
        x = (torch.randn(N, S, C, generator=g) + 2 * torch.randn(C, generator=g)).to(dtype)
        w, b = torch.randn(C, generator=g), torch.randn(C, generator=g)
        ws = ops.make_group_norm_workspace(N, S, C, groups) if r.random() < 0.7 else None
        print(f"[norm] {N}x{S}x{C} groups={groups} {act} {dtype} ws={ws is not None}", flush=True)
        want, tol = _norm_reference(x, groups, w, b, 1e-5, act, BF16 if dtype == torch.bfloat16 else F32)
        _check(ops.group_norm_act(x.cuda(), groups, w.cuda(), b.cuda(), act=act, workspace=ws), want, tol)
