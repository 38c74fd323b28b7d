"""Where the outputs lie that a cache operator makes for a call on another stream."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_cache_ops_gpu as R  # noqa: E402

DEV = "cuda"
BF = torch.bfloat16


class _Handle:
    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


def _stream_of(t):
    """The stream whose memory a tensor lies in, as the allocator has it."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_lie_in_the_memory_of_their_stream(handle):
    from w4a4_post_quantized_channel_amd import ops
    c = R._cache(ops, 1, 9, 16, 2, 64)
    table = torch.arange(9, dtype=torch.int32, device=DEV).view(1, 9)
    lens = torch.tensor([140], dtype=torch.int32, device=DEV)
    slots = torch.arange(70, dtype=torch.int32, device=DEV)
    q, k = R._rand(2, 70, 4, 64).to(BF).to(DEV), R._rand(3, 70, 2, 64).to(BF).to(DEV)
    pos, rot = torch.arange(70, dtype=torch.int32, device=DEV).view(70, 1), ops.make_rotary_table([32], device=DEV)
    x = R._rand(4, 70, 256).to(DEV)
    side = torch.cuda.Stream()
    calls = (lambda **kw: ops.cache_read(c, slots, **kw), lambda **kw: (ops.cache_attention(q.view(1, 70, 4, 64), c, table, lens, **kw),),
             lambda **kw: ops.rotary_axes(q, k, pos, rot, **kw), lambda **kw: ops.gated_norm(x, x, **kw))
    for call in calls:
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        got = call(stream=_Handle(side) if handle else side)
        torch.cuda.synchronize()
        for t, w in zip(got, want):
            assert torch.equal(t, w) and _stream_of(t) == side.cuda_stream
