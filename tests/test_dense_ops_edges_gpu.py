"""Sizes and places at the edges of the 16-bit operators' kernels, against 64
bits on the GPU."""
import math

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
    return torch.Generator(device="cuda").manual_seed(seed)


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
