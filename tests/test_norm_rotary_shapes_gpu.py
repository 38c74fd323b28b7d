"""Gated norms wider than a thread's eight channels a row, over runs of rows with
changing modulations, and rotary heads whose pairs no eight-channel vector splits.
References in 64 bits; rows of a long call equal the same rows called by themselves."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_cache_ops_gpu as R  # noqa: E402  (references and tolerances)

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    from w4a4_post_quantized_channel_amd import ops as _ops
    return _ops


# more rows than workgroups at once: several of each, and modulation rows that end inside a run
@pytest.mark.parametrize("M,C,rows,kind,post,x,h,y", [
    (2100, 16384, 7, "layer", True, F32, BF, BF), (2100, 16384, 700, "rms", False, BF, BF, BF),
    (1995, 16383, 19, "rms", True, BF, F32, F32), (2001, 8193, 2001, "layer", True, BF, BF, BF),
    (1800, 8200, 5, "layer", False, F32, F32, F32), (1999, 8185, 1, "rms", True, F32, BF, BF),
    (1536, 9001, 3, "layer", True, BF, BF, F32)])
def test_wide_rows_in_runs(ops, M, C, rows, kind, post, x, h, y):
    xs, hs = R._rand(1, M, C).to(x).to(DEV), (R._rand(2, M, C) * torch.exp(R._rand(3, 1, C))).to(h).to(DEV)
    mod = (R._rand(4, rows, 3, C) * 0.3).to(DEV)
    vec = [(1 + 0.2 * R._rand(5 + n, C)).to(DEV) for n in range(3)]
    kw = dict(post_weight=vec[0] if post else None, weight=vec[1], bias=vec[2], kind=kind)
    xo, yo = ops.gated_norm(xs, hs, gate=mod[:, 2], scale=mod[:, 1], shift=mod[:, 0], y_dtype=y, **kw)
    per = M // rows
    for r in sorted({0, 1 % rows, rows // 2, rows - 2 if rows > 1 else 0, rows - 1}):
        at = slice(r * per, min(r * per + 300, (r + 1) * per))
        one = mod[r:r + 1]
        wx, wy = ops.gated_norm(xs[at], hs[at], gate=one[:, 2], scale=one[:, 1], shift=one[:, 0], y_dtype=y, **kw)
        assert torch.equal(xo[at], wx) and torch.equal(yo[at], wy)
    some = torch.arange(0, M, 97)                      # rows of many workgroups, against 64 bits
    each = mod[(some // per).to(DEV)]
    ref = R._gated_reference(xs[some.to(DEV)], hs[some.to(DEV)], each[:, 2], 1.0, kw["post_weight"], kind, vec[1], vec[2],
                             each[:, 1], each[:, 0], 1e-6)
    R._assert_gated(xo[some.to(DEV)], yo[some.to(DEV)], ref, post)


@pytest.mark.parametrize("M,Hq,Hk,D,sections", [(1, 5, 1, 72, [36]), (400, 16, 4, 72, [36]), (1561, 5, 2, 72, [12, 12, 12]),
                                                (33, 2, 2, 80, [12]), (50, 3, 1, 64, [20, 8])])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_pairs_that_are_no_multiple_of_eight(ops, M, Hq, Hk, D, sections, dtype, inter):
    big = R._rand(40, M, Hq + Hk, D).to(dtype).to(DEV)
    q, k = big[:, :Hq], big[:, Hq:]
    pos = torch.randint(0, 2000, (M, len(sections)), generator=torch.Generator().manual_seed(M)).int()
    table = ops.make_rotary_table(sections, device=DEV)
    q0, k0 = q.clone(), k.clone()
    out = ops.rotary_axes(q, k, pos.to(DEV), table, interleaved=inter)
    for x, got in zip((q0, k0), out):
        R._assert_rotary(got, x, pos, sections, inter)
    ops.rotary_axes(q, k, pos.to(DEV), table, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, out[0]) and torch.equal(k, out[1])
