"""Refusals of the operators around the 4-bit cache: the C entry points' checks
built for the host under AddressSanitizer and UndefinedBehaviorSanitizer, and
the Python binding's own checks (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "csrc")
SAN = os.path.join(ROOT, "tests", "sanitize")
ROCM_INC = "/opt/rocm/include"
BUILT = os.path.exists(os.path.join(ROOT, "w4a4_post_quantized_channel_amd", "libw4a4.so"))
needs_library = pytest.mark.skipif(not BUILT, reason="libw4a4.so not built")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INC), reason="needs g++ and the HIP headers")
def test_checks_under_asan_and_ubsan(tmp_path):
    exe = str(tmp_path / "cache_sanitize")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I" + ROCM_INC, os.path.join(CSRC, "abi.cpp"),
           os.path.join(CSRC, "abi_cache.cpp"), os.path.join(SAN, "stubs.cpp"), os.path.join(SAN, "cache_driver.cpp"),
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and "ok: 0 failures" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


class _NoStream:
    cuda_stream = 0


@pytest.fixture(scope="module")
def ops():
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@needs_library
def test_cache_refuses(ops):
    good = dict(k_codes=_u8(3, 2, 16, 32), k_scales=_u8(3, 2, 16, 4), v_codes=_u8(3, 2, 16, 32), v_scales=_u8(3, 2, 16, 4))
    ops.KVCache(**good)
    for exc, change in [(ValueError, dict(k_codes=_u8(3, 2, 16))), (ValueError, dict(k_scales=_u8(3, 2, 16, 5))),
                        (TypeError, dict(v_codes=_bf(3, 2, 16, 32))), (ValueError, dict(v_scales=_u8(2, 2, 16, 4))),
                        (ValueError, dict(v_codes=_u8(3, 16, 2, 32).transpose(1, 2))),
                        (ValueError, dict(v_codes=_u8(3, 2, 16, 32).to("meta")))]:
        with pytest.raises(exc):
            ops.KVCache(**{**good, **change})
    pool = _u8(3, 5, 2, 16, 32)      # pages of several layers side by side
    c = ops.KVCache(pool[:, 1], good["k_scales"], pool[:, 2], good["v_scales"])
    assert c.D == 64 and c.page == 16 and c.Hkv == 2


def _calls(ops):
    c = ops.make_kv_cache(4, 16, 2, 64, 0.5, 0.25, device="cpu")
    kv = dict(k=_bf(5, 2, 64), v=_bf(5, 2, 64), slots=_i32(5), cache=c)
    table = ops.make_rotary_table([12, 10, 10], device="cpu")
    return {
        "cache_append": kv, "cache_read": dict(kv),
        "cache_attention": dict(q=_bf(2, 3, 4, 64), cache=c, table=_i32(2, 4), lens=_i32(2), out=_bf(2, 3, 4, 64),
                                workspace=_u8(64)),
        "rotary_axes": dict(q=_bf(5, 4, 64), k=_bf(5, 2, 64), pos=_i32(5, 3), table=table, q_out=_bf(5, 4, 64),
                            k_out=_bf(5, 2, 64)),
        "gated_norm": dict(x=torch.zeros(6, 40), h=_bf(6, 40), gate=torch.zeros(2, 40), scale=torch.zeros(2, 40),
                           shift=torch.zeros(2, 40), post_weight=torch.zeros(40), weight=torch.zeros(40),
                           bias=torch.zeros(40), x_out=torch.zeros(6, 40), y=_bf(6, 40)),
    }


BAD = [
    ("cache_append", TypeError, lambda: dict(slots=torch.zeros(5, dtype=torch.int64))),
    ("cache_append", TypeError, lambda: dict(slots=_i32(10)[::2])),
    ("cache_append", ValueError, lambda: dict(slots=_i32(4))),
    ("cache_append", ValueError, lambda: dict(v=_bf(5, 2, 128))),
    ("cache_append", TypeError, lambda: dict(v=torch.zeros(5, 2, 64))),
    ("cache_append", ValueError, lambda: dict(k=_bf(5, 2, 128)[..., ::2])),
    ("cache_append", TypeError, lambda: dict(k=torch.zeros(5, 2, 64, dtype=torch.float16), v=torch.zeros(5, 2, 64, dtype=torch.float16))),
    ("cache_read", ValueError, lambda: dict(k=_bf(4, 2, 64))),
    ("cache_read", TypeError, lambda: dict(v=torch.zeros(5, 2, 64))),
    ("cache_attention", ValueError, lambda: dict(q=_bf(2, 3, 4, 128))),
    ("cache_attention", TypeError, lambda: dict(q=torch.zeros(2, 3, 4, 64))),
    ("cache_attention", ValueError, lambda: dict(out=_bf(2, 3, 4, 32))),
    ("cache_attention", TypeError, lambda: dict(table=torch.zeros(2, 4, dtype=torch.int64))),
    ("cache_attention", TypeError, lambda: dict(table=_i32(3, 4))),
    ("cache_attention", TypeError, lambda: dict(table=_i32(4, 2).t())),
    ("cache_attention", TypeError, lambda: dict(lens=_i32(3))),
    ("cache_attention", TypeError, lambda: dict(lens=torch.zeros(2, dtype=torch.int64))),
    ("rotary_axes", TypeError, lambda: dict(pos=_i32(5, 2))),
    ("rotary_axes", TypeError, lambda: dict(pos=torch.zeros(5, 3, dtype=torch.int64))),
    ("rotary_axes", TypeError, lambda: dict(k=torch.zeros(5, 2, 64))),
    ("rotary_axes", ValueError, lambda: dict(k=_bf(4, 2, 64))),
    ("rotary_axes", ValueError, lambda: dict(q_out=_bf(5, 4, 32))),
    ("gated_norm", ValueError, lambda: dict(kind="batch")),
    ("gated_norm", ValueError, lambda: dict(h=_bf(6, 41))),
    ("gated_norm", ValueError, lambda: dict(gate=torch.zeros(3, 40))),
    ("gated_norm", ValueError, lambda: dict(shift=torch.zeros(2, 41))),
    ("gated_norm", TypeError, lambda: dict(scale=_bf(2, 40))),
    ("gated_norm", TypeError, lambda: dict(weight=torch.zeros(41))),
    ("gated_norm", TypeError, lambda: dict(post_weight=_bf(40))),
    ("gated_norm", TypeError, lambda: dict(x_out=_bf(6, 40))),
    ("gated_norm", ValueError, lambda: dict(y=_bf(5, 40))),
    ("gated_norm", TypeError, lambda: dict(y=torch.zeros(6, 40, dtype=torch.float16))),
]


@needs_library
@pytest.mark.parametrize("i", range(len(BAD)))
def test_bindings_refuse(ops, i):
    fn, exc, change = BAD[i]
    with pytest.raises(exc):
        getattr(ops, fn)(**{**_calls(ops)[fn], **change()}, stream=_NoStream())


@needs_library
@pytest.mark.parametrize("fn", ["cache_append", "cache_read", "cache_attention", "rotary_axes", "gated_norm"])
def test_host_memory_is_refused_before_any_launch(ops, fn):
    with pytest.raises(ops.W4A4Error) as e:
        getattr(ops, fn)(**_calls(ops)[fn], stream=_NoStream())
    assert e.value.status == -1 and "NULL" in str(e.value)


ELSEWHERE = [(fn, name) for fn, names in
             (("cache_append", "v slots"), ("cache_read", "v slots"), ("cache_attention", "table lens out workspace"),
              ("rotary_axes", "k pos q_out k_out"),
              ("gated_norm", "h gate scale shift post_weight weight bias x_out y")) for name in names.split()]


@needs_library
@pytest.mark.parametrize("fn,name", ELSEWHERE)
def test_an_operand_elsewhere_is_refused(ops, fn, name):
    kw = _calls(ops)[fn]
    kw[name] = kw[name].to("meta")
    with pytest.raises(ValueError, match=name):
        getattr(ops, fn)(**kw, stream=_NoStream())


@needs_library
def test_another_device_than_the_current_one_is_refused(ops, monkeypatch):
    class There:
        device = torch.device("cuda", 1)

        def get_device(self):
            return 1

    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        ops._stream_for(There(), _NoStream())
    monkeypatch.setattr(ops, "_current_device", lambda: 1)
    assert ops._stream_for(There(), _NoStream()) == 0


@needs_library
def test_rotary_table_keeps_48_bits(ops):
    import math
    t = ops.make_rotary_table([3, 2], 5000.0, device="cpu")
    want = [5000.0 ** (-i / s) / (2 * math.pi) for s in (3, 2) for i in range(s)]
    got = t.turns.double().sum(1)
    assert t.sections == (3, 2) and t.turns.shape == (5, 2)
    for g, w in zip(got.tolist(), want):
        assert abs(g - w) <= 2.0 ** -48 * w        # two roundings to 24 bits, the second of what the first lost
    freqs = [1.0, 0.5, 0.25]
    assert torch.equal(ops.make_rotary_table([1, 2], freqs=freqs, device="cpu").turns,
                       ops.make_rotary_table([3], freqs=torch.tensor(freqs), device="cpu").turns)
    with pytest.raises(ValueError):
        ops.make_rotary_table([2, 2], freqs=freqs, device="cpu")
    with pytest.raises(ValueError):
        ops.make_rotary_table([1] * 5, device="cpu")


@needs_library
def test_what_a_call_was_packed_from_is_fixed(ops):
    c = _calls(ops)["cache_append"]["cache"]
    t = ops.make_rotary_table([3, 2], device="cpu")
    for x, names in ((c, "k_codes v_scales k_scale D page n_pages"), (t, "sections turns")):
        for name in names.split():
            with pytest.raises(AttributeError, match=name):
                setattr(x, name, getattr(x, name))


@needs_library
def test_a_copied_cache_is_packed_from_its_own_tensors(ops):
    import copy
    c = _calls(ops)["cache_append"]["cache"]
    d = copy.deepcopy(c)
    assert d.k_codes.data_ptr() != c.k_codes.data_ptr() and (d.k_scale, d.v_scale, d.page) == (c.k_scale, c.v_scale, c.page)
    make, args = c.__reduce__()
    assert make is ops.KVCache and all(a is getattr(c, n) for a, n in zip(args, ("k_codes", "k_scales", "v_codes", "v_scales")))
