"""bf16 linear on every tile, with K whole and split over workgroups: products
of small whole numbers, which are exact in 32 bits in any order, and random
ones with every part of the epilogue, against 64 bits on the GPU."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_dense_ops_gpu import BF16, F32, _linear_inputs, _linear_reference

# (tile, SwiGLU, K split): M, N, K, workspace
SHAPES = {
    (0, False, False): (3819, 4971, 296, True),
    (0, False, True): (1330, 3067, 8144, True),
    (1, False, False): (2042, 6107, 280, True),
    (1, False, True): (4197, 140, 21936, True),
    (1, True, True): (2073, 67, 48120, True),
    (1, True, False): (778, 7950, 368, True),
    (2, False, False): (848, 5680, 376, False),
    (2, False, True): (2247, 398, 6656, True),
    (2, True, False): (399, 4341, 688, True),
    (2, True, True): (1276, 417, 7424, True),
    (3, False, False): (3089, 676, 416, True),
    (3, False, True): (1572, 323, 5560, True),
    (3, True, False): (537, 2277, 336, True),
    (3, True, True): (212, 1726, 3824, True),
    (4, False, False): (542, 2581, 288, True),
    (4, False, True): (518, 190, 6944, True),
    (4, True, False): (2236, 435, 200, True),
    (4, True, True): (34, 1349, 4008, True),
    (5, False, False): (25, 515, 696, False),
    (5, False, True): (10, 253, 6072, True),
    (5, True, False): (27, 169, 80, False),
    (5, True, True): (26, 70, 6552, True),
    ("rows", False, False): (4, 2840, 4088, True),
    ("rows", True, False): (16, 301, 776, True),
}
IDS = ["%s%s%s" % (t, "-swiglu" if g else "", "-split" if s else "") for t, g, s in SHAPES]


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


def _call(ops, x, w, act, workspace, **kw):
    M, K = x.shape
    N = w.shape[0] // (2 if act == "swiglu" else 1)
    print(f"[linear] {M}x{N}x{K} {act} ws={workspace}", flush=True)
    ws = ops.make_bf16_linear_workspace(M, N, K, act) if workspace else None
    return ops.bf16_linear(x, w, act=act, workspace=ws, **kw)


@pytest.mark.parametrize("key", SHAPES, ids=IDS)
def test_whole_numbers_are_exact(ops, key):
    M, N, K, ws = SHAPES[key]
    g = torch.Generator(device="cuda").manual_seed(M)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").bfloat16()
    # rows padded with NaN: what lies past K must not enter
    x = torch.full((M, K + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:, :K] = whole(M, K)
    w = whole(N, K)
    if key[1]:                                     # a gate of 32 passes the second factor on exactly
        x[:, K // 2] = 1.0
        gate = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
        gate[:, K // 2] = 32.0
        got = _call(ops, x[:, :K], torch.cat([gate, w]), "swiglu", ws, y_dtype=torch.float32)
        want = 32.0 * (x[:, :K].double() @ w.double().t().contiguous())
    else:
        got = _call(ops, x[:, :K], w, "none", ws, y_dtype=torch.float32)
        want = x[:, :K].double() @ w.double().t().contiguous()
    assert torch.equal(got.double(), want)


EPILOGUES = [(k, act) for k in SHAPES for act in (["swiglu"] if k[1] else ["gelu", "relu"])]


@pytest.mark.parametrize("key,act", EPILOGUES, ids=[IDS[list(SHAPES).index(k)] + "-" + act for k, act in EPILOGUES])
def test_epilogues(ops, key, act):
    M, N, K, ws = SHAPES[key]
    half = act != "relu"
    y_dtype = torch.bfloat16 if half else torch.float32
    x, w, b, r = [t.cuda() for t in _linear_inputs(M, N, K, act, torch.float32 if half else torch.bfloat16, True, y_dtype, M)]
    want, tol = _linear_reference(x, w, b, act, r, BF16 if half else F32)
    err = (_call(ops, x, w, act, ws, bias=b, residual=r, y_dtype=y_dtype).double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))
