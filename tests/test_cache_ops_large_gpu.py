"""The operators around the 4-bit cache where element offsets and work items pass
31 and 32 bits: parts of a large call equal the same rows called by themselves."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_cache_ops_gpu as R  # noqa: E402

DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from w4a4_post_quantized_channel_amd import ops
    yield ops
    torch.cuda.empty_cache()


def _fill(x, seed):
    """Every 2^20 elements the same random ones, shifted by a few (quick to make, different in neighbouring rows)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = torch.randn(2 ** 20 + 3, generator=g, device=DEV).to(x.dtype)
    flat = x.view(-1)
    for i in range(0, flat.numel(), r.numel()):
        n = min(r.numel(), flat.numel() - i)
        flat[i:i + n] = r[:n]
    return x


@pytest.mark.parametrize("M,D,sections,interleaved", [(2 ** 21 + 5, 1024, [512], True),        # more vectors than threads
                                                      (2 ** 21 + 8192, 1022, [1], False),      # and single pairs, past 2^31
                                                      (2 ** 21 + 8192, 1022, [1], True)])
def test_rotary_of_many_tokens(ops, M, D, sections, interleaved):
    x = _fill(torch.empty(M, 1, D, dtype=BF, device=DEV), 1)
    pos = torch.arange(M, dtype=torch.int32, device=DEV).view(M, 1) % 5000
    table = ops.make_rotary_table(sections, device=DEV)
    out, _ = ops.rotary_axes(x, None, pos, table, interleaved=interleaved)
    for i in (0, M // 2 - 300, M - 700):
        want, _ = ops.rotary_axes(x[i:i + 700], None, pos[i:i + 700], table, interleaved=interleaved)
        assert torch.equal(out[i:i + 700], want)


@pytest.mark.parametrize("C", [5120, 5121])
def test_gated_norm_of_many_rows(ops, C):
    M, R_ = 2 ** 19 + 4, 4
    x = _fill(torch.empty(M, C, dtype=BF, device=DEV), 2)
    mod = 0.3 * torch.randn(3, R_, C, device=DEV)
    xo, y = ops.gated_norm(x, x, gate=mod[0], scale=mod[1], shift=mod[2])
    per = M // R_
    for i in (0, M // 2 + 7, M - 900):
        r = i // per
        wx, wy = ops.gated_norm(x[i:i + 900], x[i:i + 900], gate=mod[0, r:r + 1], scale=mod[1, r:r + 1], shift=mod[2, r:r + 1])
        assert torch.equal(xo[i:i + 900], wx) and torch.equal(y[i:i + 900], wy)


@pytest.mark.parametrize("T", [1, 9, 300])
def test_attention_of_batches_far_apart(ops, T):
    B, Hq, Hkv, D, page, far = 2, 4, 2, 128, 32, 2 ** 32
    c = R._cache(ops, 3, 41, page, Hkv, D)
    table = torch.arange(40, dtype=torch.int32, device=DEV).view(2, 20)
    lens = torch.tensor([640, 601], dtype=torch.int32, device=DEV)
    span = far + T * Hq * D
    q = torch.empty(span, dtype=BF, device=DEV).as_strided((B, T, Hq, D), (far, Hq * D, D, 1))
    out = torch.empty(span, dtype=BF, device=DEV).as_strided((B, T, Hq, D), (far, Hq * D, D, 1))
    q.copy_(R._rand(4, B, T, Hq, D).to(BF))
    ws = ops.make_cache_attention_workspace(B, T, Hq, Hkv, D, 640, device=DEV)
    ops.cache_attention(q, c, table, lens, causal=True, out=out, workspace=ws)
    assert torch.equal(out, ops.cache_attention(q.contiguous(), c, table, lens, causal=True, workspace=ws))


def test_cache_rows_far_apart(ops):
    M, H, D, page, far = 5, 2, 128, 16, 2 ** 30
    c = R._cache(ops, 5, 3, page, H, D)
    k, v = R._rand(6, M, H, D).to(BF).to(DEV), R._rand(7, M, H, D).to(BF).to(DEV)
    buf = torch.empty(4 * far + H * D, dtype=BF, device=DEV)
    apart = buf.as_strided((M, H, D), (far, D, 1))
    apart.copy_(k)
    slots = torch.tensor([3, 47, 0, 20, 31], dtype=torch.int32, device=DEV)
    ops.cache_append(c, apart, v, slots)
    k1, v1 = ops.cache_read(c, slots)
    ops.cache_append(c, k, v, slots)
    k2, v2 = ops.cache_read(c, slots)
    assert torch.equal(k1, k2) and torch.equal(v1, v2)
    ops.cache_read(c, slots, k=apart, v=v1)
    assert torch.equal(apart, k2)
