"""Outputs that a cache operator makes for a call on another stream come from that
stream's memory: what the current stream freed may still be read or written by work
that it has queued.  (No GPU needed: host operands are refused, but only after the
outputs were made.)"""
import contextlib
import os

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "libw4a4.so")),
                                reason="libw4a4.so not built")


class _Side:
    cuda_stream = 0


@pytest.fixture
def ops(monkeypatch):
    from w4a4_post_quantized_channel_amd import ops as _ops
    inside, made = [], []

    @contextlib.contextmanager
    def stream(s):
        inside.append(s)
        yield
        inside.pop()

    empty = torch.empty

    def recorded(*args, **kw):
        made.append(inside[-1] if inside else None)
        return empty(*args, **kw)

    monkeypatch.setattr(torch.cuda, "Stream", _Side)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", recorded)
    _ops.made = made
    yield _ops
    del _ops.made


def _calls(ops):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    c = ops.KVCache(u8(4, 2, 16, 32), u8(4, 2, 16, 4), u8(4, 2, 16, 32), u8(4, 2, 16, 4), 0.5, 0.25)
    table = ops.make_rotary_table([12, 10, 10], device="cpu")
    return {"cache_read": (2, dict(cache=c, slots=i32(5))),
            "cache_attention": (1, dict(q=bf(2, 3, 4, 64), cache=c, table=i32(2, 4), lens=i32(2))),
            "rotary_axes": (2, dict(q=bf(5, 4, 64), k=bf(5, 2, 64), pos=i32(5, 3), table=table)),
            "gated_norm": (2, dict(x=torch.zeros(6, 40), h=bf(6, 40)))}


@pytest.mark.parametrize("fn", ["cache_read", "cache_attention", "rotary_axes", "gated_norm"])
def test_outputs_are_made_on_the_stream_of_the_call(ops, fn):
    n, kw = _calls(ops)[fn]
    side = _Side()
    ops.made.clear()
    with pytest.raises(ops.W4A4Error, match="NULL"):
        getattr(ops, fn)(**kw, stream=side)
    assert len(ops.made) == n and all(s is side for s in ops.made)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    from w4a4_post_quantized_channel_amd import ops

    class There:
        device = torch.device("cuda", 1)

        def get_device(self):
            return 1

    class On(_Side):
        def __init__(self, index):
            self.device_index = index

    monkeypatch.setattr(ops, "_current_device", lambda: 1)
    assert ops._stream_for(There(), On(1)) == 0
    with pytest.raises(ValueError, match="stream"):
        ops._stream_for(There(), On(0))
