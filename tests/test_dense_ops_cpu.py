"""Refusals of the 16-bit operators: the C entry points' checks built for the
host under AddressSanitizer and UndefinedBehaviorSanitizer, and the Python
binding's own checks (no GPU needed)."""
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
    exe = str(tmp_path / "dense_sanitize")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I" + ROCM_INC, os.path.join(CSRC, "abi.cpp"),
           os.path.join(CSRC, "abi_dense.cpp"), os.path.join(SAN, "stubs.cpp"), os.path.join(SAN, "dense_driver.cpp"),
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and "ok: 0 failures" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


@pytest.fixture(scope="module")
def ops():
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@needs_library
def test_attention_binding_refuses(ops):
    good = dict(q=_bf(2, 3, 4, 64), k_prefix=_bf(9, 2, 64), v_prefix=_bf(9, 2, 64), k_own=_bf(2, 5, 2, 64),
                v_own=_bf(2, 5, 2, 64))
    bad = [
        (TypeError, dict(q=torch.zeros(2, 3, 4, 64))),
        (ValueError, dict(v_prefix=_bf(8, 2, 64))),
        (ValueError, dict(k_own=_bf(3, 5, 2, 64))),
        (ValueError, dict(v_own=_bf(2, 5, 2, 128)[..., ::2])),
        (ValueError, dict(out=_bf(2, 3, 4, 32))),
        (TypeError, dict(own_len=torch.zeros(2, dtype=torch.int64))),
        (TypeError, dict(own_len=torch.zeros(3, dtype=torch.int32))),
        (TypeError, dict(prefix_keep=torch.zeros(9))),
        (TypeError, dict(prefix_keep=torch.zeros(8, dtype=torch.bool))),
    ]
    for exc, change in bad:
        with pytest.raises(exc):
            ops.prefix_attention(**{**good, **change}, stream=_NoStream())
    with pytest.raises(ops.W4A4Error) as e:      # reaches the library, which refuses before any launch
        ops.prefix_attention(**{**good, "q": _bf(2, 3, 5, 64)}, stream=_NoStream())
    assert e.value.status == -2 and "query heads" in str(e.value)


@needs_library
def test_linear_and_norm_bindings_refuse(ops):
    x, w = _bf(3, 16), _bf(8, 16)
    for exc, kw in [(TypeError, dict(x=torch.zeros(3, 16))), (ValueError, dict(w=_bf(8, 24))),
                    (ValueError, dict(act="tanh")), (ValueError, dict(bias=torch.zeros(7))),
                    (TypeError, dict(residual=torch.zeros(3, 8))), (ValueError, dict(w=_bf(7, 16), act="swiglu")),
                    (ValueError, dict(y=_bf(3, 9)))]:
        with pytest.raises(exc):
            ops.bf16_linear(**{**dict(x=x, w=w), **kw}, stream=_NoStream())
    with pytest.raises(ops.W4A4Error) as e:
        ops.bf16_linear(_bf(3, 12), _bf(8, 12), stream=_NoStream())
    assert e.value.status == -2
    with pytest.raises(ops.W4A4Error):           # a broadcast row is not a row stride
        ops.bf16_linear(_bf(1, 16).expand(3, 16), w, stream=_NoStream())
    f = torch.zeros(2, 4, 12)
    for kw in [dict(x=f.double()), dict(x=f.transpose(1, 2)), dict(weight=torch.zeros(11)), dict(out=_bf(2, 4, 12))]:
        with pytest.raises(TypeError):
            ops.group_norm_act(**{**dict(x=f, groups=3), **kw}, stream=_NoStream())
    with pytest.raises(ops.W4A4Error) as e:
        ops.group_norm_act(f, 5, stream=_NoStream())
    assert e.value.status == -2


class _NoStream:
    cuda_stream = 0
