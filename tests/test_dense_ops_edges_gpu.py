"""Sizes and places at the edges of the 16-bit operators' kernels, against 64
bits on the GPU."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_dense_ops_gpu import BF16, F32, _linear_inputs, _linear_reference


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ----------------------------------------------------------------------------
# bf16 linear
# ----------------------------------------------------------------------------
def _linear(ops, M, N, K, act, bias, residual, y_dtype, workspace, seed):
    x, w, b, r = [None if t is None else t.cuda() for t in _linear_inputs(M, N, K, act, bias, residual, y_dtype, seed)]
    want, tol = _linear_reference(x, w, b, act, r, BF16 if y_dtype == torch.bfloat16 else F32)
    print(f"[linear] {M}x{N}x{K} {act} {y_dtype} ws={workspace}", flush=True)
    y = ops.bf16_linear(x, w, bias=b, act=act, residual=r, y_dtype=y_dtype,
                        workspace=ops.make_bf16_linear_workspace(M, N, K, act) if workspace else None)
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("M,N,K,act", [(16, 32773, 4200, "gelu"), (5, 20011, 2056, "none"), (1, 32768, 4104, "silu"),
                                       (4, 33000, 1032, "none"), (4, 33000, 520, "gelu_tanh"), (9, 16500, 4168, "swiglu"),
                                       (2, 16500, 1544, "swiglu")])
def test_few_rows_over_many_columns(ops, M, N, K, act, workspace):
    """Both kernels for at most 16 rows where the columns alone fill the card."""
    _linear(ops, M, N, K, act, torch.float32, True, torch.float32 if M % 2 else torch.bfloat16, workspace, seed=M)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("M", [1, 40])
def test_activations_of_any_finite_argument(ops, act, M):
    """Both ends of the range: an activation is its argument or zero there, not
    a large argument times the smallest sigmoid."""
    mag = torch.tensor([80.0, 86.5, 87.5, 88.0, 88.5, 89.0, 100.0, 104.0, 1e3, 1e6, 1e10, 1e20, 1e30, 1e38, 3e38])
    z = torch.cat([-mag, mag]).bfloat16().cuda()
    x = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    w = torch.zeros(z.numel(), 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = z
    if act == "swiglu":
        w = torch.cat([w, torch.zeros_like(w)])
        w[z.numel():, 0] = 0.5                                     # the second factor
    want, tol = _linear_reference(x, w, None, act, None, F32)
    y = ops.bf16_linear(x, w, act=act, y_dtype=torch.float32).double()
    # relative accuracy is lost below the smallest normal number
    err = (y - want).abs()
    assert bool((err <= tol + 1e-36).all()), (float((err - tol).max()), y[0].tolist())


# ----------------------------------------------------------------------------
# Group norm
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("N,S,C,groups,dtype", [(70001, 1, 64, 1, torch.bfloat16), (131072, 1, 40, 4, torch.float32),
                                                (65536, 2, 7, 1, torch.float32), (65600, 1, 4100, 1, torch.bfloat16)])
def test_norm_of_more_samples_than_a_grid_dimension(ops, N, S, C, groups, dtype):
    x = (torch.randn(N, S, C, generator=_gen(N + C), device="cuda") + 1.0).to(dtype)
    print(f"[norm] {N}x{S}x{C} groups={groups} {dtype}", flush=True)
    y = ops.group_norm_act(x, groups, act="none", workspace=ops.make_group_norm_workspace(N, S, C, groups))
    half = BF16 if dtype == torch.bfloat16 else F32
    for n in range(0, N, 8192):
        v = x[n:n + 8192].double().view(-1, S, groups, C // groups)
        mean = v.mean(dim=(1, 3), keepdim=True)
        rstd = 1 / torch.sqrt(((v - mean) ** 2).mean(dim=(1, 3), keepdim=True) + 1e-5)
        want = (v - mean) * rstd
        # the mean to four ulp of the group's largest value, the variance to 4e-6, one rounding
        tol = 4 * F32 * v.abs().amax(dim=(1, 3), keepdim=True) * rstd + (4e-6 + 5 * F32 + half) * want.abs() + 1e-30
        err = (y[n:n + 8192].double().view(want.shape) - want).abs()
        assert bool((err <= tol).all()), (n, float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_activations_far_out(ops, act, dtype):
    """Biases that carry the activation's argument to both ends of the range."""
    mag = torch.tensor([60.0, 87.5, 88.5, 104.0, 1e4, 1e10, 1e30, 3e38], device="cuda")
    b = torch.cat([-mag, mag])
    x = torch.randn(2, 33, 16, generator=_gen(1), device="cuda").to(dtype)
    y = ops.group_norm_act(x, 4, torch.zeros(16, device="cuda"), b, act=act).double()
    z = b.double()
    slope = {"gelu": lambda: 0.5 * torch.special.erfc(-z / math.sqrt(2)),
             "gelu_tanh": lambda: torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)),
             "silu": lambda: torch.sigmoid(z)}[act]()
    want = (z * slope).expand_as(y)
    half = BF16 if dtype == torch.bfloat16 else F32
    err = (y - want).abs()
    assert bool((err <= (half + 32 * F32) * want.abs() + 1e-36).all()), (float(err.max()), y[0, 0].tolist())
