"""Group norm statistics over many positions a thread: groups wider than a
workgroup's threads and calls without a workspace run one workgroup a group.

Tolerance: the mean is good to four ulp of the group's largest value and the
variance to 4e-6, as for short inputs; fp32 sums over a whole walk are not
(added one by one, equal terms are rounded the same way every time)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = 2.0 ** -8, 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


def _compare(ops, x, groups, weight, bias, workspace):
    N, S, C = x.shape
    print(f"[norm long] {N}x{S}x{C} groups={groups} {x.dtype} ws={workspace}", flush=True)
    ws = ops.make_group_norm_workspace(N, S, C, groups) if workspace else None
    y = ops.group_norm_act(x, groups, weight, bias, eps=EPS, act="none", workspace=ws)
    half = BF16 if x.dtype == torch.bfloat16 else F32
    w = C // groups
    for n in range(N):
        for k in range(groups):
            ch = slice(k * w, (k + 1) * w)
            v = x[n, :, ch].double()
            var, mean = torch.var_mean(v, unbiased=False)
            rstd = 1 / torch.sqrt(var + EPS)
            hat = (v - mean) * rstd
            wt, b = weight[ch].double(), bias[ch].double()
            want = hat * wt + b
            dhat = 4 * F32 * v.abs().max() * rstd + 4e-6 * hat.abs()
            tol = dhat * wt.abs() + 4 * F32 * (hat.abs() * wt.abs() + b.abs()) + (F32 + half) * want.abs() + 1e-30
            err = (y[n, :, ch].double() - want).abs()
            assert bool((err <= tol).all()), (n, k, float((err - tol).max()), float(err.max()))


def _affine(C, g):
    return 1 + 0.2 * torch.randn(C, generator=g, device="cuda"), 0.2 * torch.randn(C, generator=g, device="cuda")


@pytest.mark.parametrize("C,groups", [(257, 1), (512, 1), (2100, 1), (600, 2)])
@pytest.mark.parametrize("workspace", [True, False])
def test_wide_groups(ops, C, groups, workspace):
    g = torch.Generator(device="cuda").manual_seed(C)
    x = torch.randn(1, 100003, C, generator=g, device="cuda") + 5.0
    _compare(ops, x, groups, *_affine(C, g), workspace)


@pytest.mark.parametrize("N,S,C,groups,dtype", [
    (1, 20003, 2048, 1, torch.bfloat16), (1, 9001, 2056, 1, torch.bfloat16), (2, 3001, 1024, 1, torch.float32),
    (1, 3001, 1028, 1, torch.float32), (3, 777, 1536, 3, torch.bfloat16), (1, 700, 4096, 2, torch.bfloat16),
    (1, 5003, 514, 2, torch.bfloat16), (1, 5003, 257, 1, torch.bfloat16), (1, 40, 1000, 1, torch.float32)])
@pytest.mark.parametrize("workspace", [True, False])
def test_groups_around_a_workgroups_channels(ops, N, S, C, groups, dtype, workspace):
    g = torch.Generator(device="cuda").manual_seed(S)
    x = (torch.randn(N, S, C, generator=g, device="cuda") + 2 * torch.randn(C, generator=g, device="cuda")).to(dtype)
    _compare(ops, x, groups, *_affine(C, g), workspace)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("C,groups", [(512, 1), (8, 1), (96, 32)])
@pytest.mark.parametrize("workspace", [True, False])
def test_equal_terms(ops, C, groups, dtype, workspace):
    """Features that take two values (a mask, say): every term of a sum of
    squares is the same, just under half an ulp of a sum in the ten thousands."""
    g = torch.Generator(device="cuda").manual_seed(C)
    S = 200001
    v = 1.00097 if dtype == torch.float32 else 1.0078125
    # a pattern that no workgroup's stride of positions divides: each walk meets both values
    up = (torch.arange(S, device="cuda") % 11 < 5).view(1, S, 1)
    x = torch.where(up, v, -v).expand(1, S, C).contiguous()
    _compare(ops, x.to(dtype), groups, *_affine(C, g), workspace)


@pytest.mark.parametrize("workspace", [True, False])
def test_a_first_value_far_from_the_rest(ops, workspace):
    """Rows of padding in front: the differences are taken to a value that is
    far from nearly all of the walk."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, 300000, 24, generator=g, device="cuda") + 300.0
    x[:, :600] = 0
    _compare(ops, x, 3, *_affine(24, g), workspace)
