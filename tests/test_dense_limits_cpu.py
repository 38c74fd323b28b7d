"""Sizes that the 16-bit operators accept and refuse, through the binding on
host tensors: an accepted size goes on to the check of pointers, which finds
no device memory (status -1); a refused one is status -2.  Nothing launches."""
import os

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "libw4a4.so")),
                                reason="libw4a4.so not built")


class _NoStream:
    cuda_stream = 0


def _status(call, *a, **kw):
    from w4a4_post_quantized_channel_amd import ops
    with pytest.raises(ops.W4A4Error) as e:
        getattr(ops, call)(*a, stream=_NoStream(), **kw)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("N", [65535, 65536, 70001, 1 << 20])
def test_norm_takes_more_samples_than_a_grid_dimension(N):
    """A layer norm of tokens has a sample per token."""
    status, msg = _status("group_norm_act", torch.zeros(N, 1, 8), 1, out=torch.zeros(N, 1, 8))
    assert status == -1 and "NULL" in msg


def test_norm_refuses_more_groups_than_it_counts():
    x = torch.zeros(1, 1, 8).expand(1 << 29, 1, 8)
    assert _status("group_norm_act", x, 4, out=x)[0] == -2
    assert _status("group_norm_act", x, 2, out=x)[0] == -1


def test_linear_sizes():
    from w4a4_post_quantized_channel_amd import ops

    def call(M, N, act=0):                                      # NULL operands: status -1 once the sizes are accepted
        return ops.LIB.bf16_linear(None, 64, None, 64, M, N, 64, ops._EPILOGUE.pack(act, 0, 0, 0, 0), None, ops.DT_BF16, N,
                                   None, 0, None)

    assert [call(1 << 30, 128), call(1 << 15, 1 << 22), call(1, 1 << 22, 5)] == [-1, -1, -1]
    # outputs that no memory holds, rows past the stride that y may have
    assert [call(1 << 30, 129), call((1 << 15) + 1, 1 << 22), call(1, (1 << 22) + 1, 5), call(1 << 31, 1)] == [-2] * 4


@pytest.mark.parametrize("C", [256, 257, 512, 1024, 2048])
def test_wide_groups_are_cut_over_positions(C):
    from w4a4_post_quantized_channel_amd import ops
    assert ops.LIB.w4a4_group_norm_workspace(1, 60000, C, 1) > 0
