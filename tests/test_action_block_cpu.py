"""Streams and memory of the action block, with the library's calls replaced by
stand-ins on the CPU: every call and every allocation of a step is on the
step's stream, and steps in flight share no scratch memory."""
import contextlib
import gc
import os
import weakref

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "libw4a4.so")),
                                reason="libw4a4.so not built")

DIM, HQ, HKV, D, F, C = 64, 2, 1, 64, 32, 16


class _Recorder:
    """Stand-ins for the library's calls.  ``calls``: (name, stream of the call,
    torch's current stream, tensors given and returned)."""

    def __init__(self):
        self.calls, self.current = [], None

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, self.current if s is None else s
        try:
            yield
        finally:
            self.current = before

    def _note(self, name, stream, given, out):
        self.calls.append((name, stream, self.current, [t for t in given if isinstance(t, torch.Tensor)], out))
        return out

    def group_norm_act(self, x, groups, weight=None, bias=None, *, eps=1e-5, act="silu", out=None, workspace=None,
                       stream=None):
        return self._note("norm", stream, [workspace, out], torch.zeros_like(x))

    def bf16_linear(self, x, w, *, bias=None, act="none", residual=None, y=None, y_dtype=torch.bfloat16,
                    workspace=None, stream=None):
        return self._note("linear", stream, [workspace, y],
                          torch.zeros(x.shape[0], w.shape[0] // (2 if act == "swiglu" else 1), dtype=y_dtype))

    def prefix_attention(self, q, k_prefix, v_prefix, k_own, v_own, *, own_len=None, prefix_keep=None, causal=False,
                         scale=None, out=None, workspace=None, stream=None):
        return self._note("attention", stream, [workspace, out], torch.zeros(q.shape, dtype=torch.bfloat16))

    def quantize_act(self, x, inv_smooth, fmt="int4", *, codes=None, scales=None, stream=None, **kw):
        self._note("quantize", stream, [codes, scales], None)

    def w4a4_linear(self, a_codes, a_scales, w_codes, w_scales, K, fmt="int4", *, y=None, workspace=None, stream=None,
                    **kw):
        return self._note("quantized linear", stream, [workspace, y], y)

    def workspace(self, *a, device=None, **kw):
        ws = torch.zeros(64, dtype=torch.uint8)
        self._note("workspace", self.current, [], ws)
        return ws


@pytest.fixture
def rec(monkeypatch):
    from w4a4_post_quantized_channel_amd import action_block, ops
    r = _Recorder()
    if hasattr(action_block, "_scratch_bytes"):
        action_block._scratch_bytes.cache_clear()
    for name in ("bf16_linear_workspace_size", "prefix_attention_workspace_size"):
        monkeypatch.setattr(ops, name, lambda *a: 64, raising=False)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: r._note("allocation", r.current, [], empty(*a, **kw)))
    for name in ("group_norm_act", "bf16_linear", "prefix_attention", "quantize_act", "w4a4_linear"):
        monkeypatch.setattr(ops, name, getattr(r, name))
    for name in ("make_bf16_linear_workspace", "make_prefix_attention_workspace", "make_group_norm_workspace",
                 "make_workspace"):
        monkeypatch.setattr(ops, name, r.workspace)
    monkeypatch.setattr(torch.cuda, "stream", r.stream)
    yield r
    if hasattr(action_block, "_scratch_bytes"):
        action_block._scratch_bytes.cache_clear()


def _block(fmt):
    from w4a4_post_quantized_channel_amd.action_block import ActionBlock
    from w4a4_post_quantized_channel_amd.pipeline import QuantizedLinear
    w = lambda n, k: torch.zeros(n, k, dtype=torch.bfloat16)
    nq = (HQ + 2 * HKV) * D
    b = ActionBlock(HQ, HKV, D, w(nq, DIM), w(2 * HKV * D, DIM), w(DIM, HQ * D), torch.zeros(DIM), w(2 * F, DIM),
                    w(DIM, F), None)
    if fmt:
        q = QuantizedLinear.__new__(QuantizedLinear)
        q.__dict__.update(fmt=fmt, a_fmt=fmt, fwht_block=64, order="smooth_then_rotate", use_workspace=True, N=nq, K=DIM,
                          inv_s=None, y_dtype=torch.bfloat16, branch=None, g_w=1.0, g_a=1.0, w_codes=None,
                          w_scales=None, _bufs={}, fuse_lowrank=False, launch_lowrank=True)
        b.qkv = q
    return b


def _tokens():
    from w4a4_post_quantized_channel_amd.action_block import FeatureTokens
    return FeatureTokens(4, torch.ones(C), torch.zeros(C), torch.zeros(DIM, C, dtype=torch.bfloat16), torch.zeros(DIM))


def _x(B=2, T=3):
    return torch.zeros(B, T, DIM, dtype=torch.bfloat16)


def _kv(P=5):
    return torch.zeros(P, HKV, D, dtype=torch.bfloat16), torch.zeros(P, HKV, D, dtype=torch.bfloat16)


@pytest.mark.parametrize("fmt", [None, "int4"])
def test_calls_and_allocations_are_on_the_given_stream(rec, fmt):
    """Memory that is allocated on another stream than the one that uses it can
    be handed out again while kernels still read it."""
    s = object()
    _tokens()(torch.zeros(7, C, dtype=torch.bfloat16), stream=s)
    block = _block(fmt)
    block.observe(torch.zeros(7, DIM, dtype=torch.bfloat16), stream=s)
    block.step(_x(), *_kv(), stream=s)
    assert len(rec.calls) > 10
    for name, stream, current, _, _ in rec.calls:
        assert current is s, name
        assert stream is s or (stream is None and current is s), name
    rec.calls.clear()
    block.step(_x(), *_kv())                     # without a stream: the caller's current one
    assert all(c[1] is None and c[2] is None for c in rec.calls)


@pytest.mark.parametrize("fmt", [None, "int4"])
def test_steps_in_flight_share_no_scratch(rec, fmt):
    """Partial sums, codes and results of a step may be in use until its stream
    reaches its end: another step (another stream, thread or captured graph)
    must not be given the same memory."""
    block = _block(fmt)
    used = []
    for s in (object(), object()):
        rec.calls.clear()
        block.step(_x(), *_kv(), stream=s)
        used.append([t for _, _, _, given, _ in rec.calls for t in given])   # held: the memory stays in use
    assert used[0] and used[1]
    first = {t.untyped_storage().data_ptr() for t in used[0]}
    assert first.isdisjoint(t.untyped_storage().data_ptr() for t in used[1])


def test_scratch_does_not_pile_up(rec):
    """Observations of ever new lengths leave nothing behind."""
    block, refs = _block("int4"), []
    for P in range(1, 40):
        rec.calls.clear()
        block.step(_x(T=1 + P % 5), *_kv(P))
        refs += [weakref.ref(t) for _, _, _, given, _ in rec.calls for t in given]
        rec.calls.clear()
    gc.collect()
    assert sum(r() is not None for r in refs) == 0
