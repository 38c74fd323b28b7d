"""The 16-bit operators' binding takes no operand that lies elsewhere than the
first one, and no operand in host memory: its address would fault the kernel
that reads it.  (CPU and meta tensors stand for two devices; no GPU needed.)"""
import os

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "libw4a4.so")),
                                reason="libw4a4.so not built")


class _NoStream:
    cuda_stream = 0


class _NoLaunch:
    """The library with its operators replaced: reaching one is a failure."""

    def __init__(self, lib):
        self._lib = lib

    def __getattr__(self, name):
        if name in ("w4a4_prefix_attention", "bf16_linear", "w4a4_group_norm_act"):
            return lambda *a: pytest.fail(f"{name} was called")
        return getattr(self._lib, name)


@pytest.fixture
def ops():
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


def _bf(*shape, **kw):
    return torch.zeros(*shape, dtype=torch.bfloat16, **kw)


def _attn():
    return dict(q=_bf(2, 3, 4, 64), k_prefix=_bf(9, 2, 64), v_prefix=_bf(9, 2, 64), k_own=_bf(2, 5, 2, 64),
                v_own=_bf(2, 5, 2, 64), own_len=torch.zeros(2, dtype=torch.int32), prefix_keep=torch.zeros(9, dtype=torch.bool),
                out=_bf(2, 3, 4, 64), workspace=torch.zeros(64, dtype=torch.uint8))


def _linear():
    return dict(x=_bf(3, 16), w=_bf(8, 16), bias=torch.zeros(8), residual=_bf(3, 8), y=_bf(3, 8),
                workspace=torch.zeros(64, dtype=torch.uint8))


def _norm():
    return dict(x=torch.zeros(2, 4, 12), weight=torch.zeros(12), bias=torch.zeros(12), out=torch.zeros(2, 4, 12),
                workspace=torch.zeros(64, dtype=torch.uint8))


CASES = [(fn, name) for fn, kw in (("prefix_attention", _attn()), ("bf16_linear", _linear()), ("group_norm_act", _norm()))
         for name in list(kw)[1:]]


def _call(ops, fn, kw):
    if fn == "group_norm_act":
        return ops.group_norm_act(groups=3, stream=_NoStream(), **kw)
    return getattr(ops, fn)(stream=_NoStream(), **kw)


@pytest.mark.parametrize("fn,name", CASES)
def test_an_operand_elsewhere_is_refused(ops, monkeypatch, fn, name):
    monkeypatch.setattr(ops, "LIB", _NoLaunch(ops.LIB))
    kw = {"prefix_attention": _attn, "bf16_linear": _linear, "group_norm_act": _norm}[fn]()
    kw[name] = kw[name].to("meta")
    with pytest.raises(ValueError, match=name):
        _call(ops, fn, kw)


@pytest.mark.parametrize("fn", ["prefix_attention", "bf16_linear", "group_norm_act"])
def test_host_memory_is_refused_before_any_launch(ops, fn):
    kw = {"prefix_attention": _attn, "bf16_linear": _linear, "group_norm_act": _norm}[fn]()
    with pytest.raises(ops.W4A4Error) as e:
        _call(ops, fn, kw)
    assert e.value.status == -1 and "NULL" in str(e.value)
