"""Attention over the 4-bit cache at the ends of what its arguments may be: scales
near the ends of fp32's range, small probabilities in every kernel, one workspace
for histories of every length.  References in 64 bits."""
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
