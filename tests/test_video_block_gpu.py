"""The operators around the 4-bit cache run together, as a video block runs them:
every call that a step makes is held to its definition on the inputs that the
step gave it, the history to what the step wrote, and a captured step to the
eager one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_cache_ops_gpu as R  # noqa: E402  (references and tolerances)

BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
DIM, HQ, HKV, D, F = 256, 4, 2, 64, 512
SECTIONS = [12, 10, 10]


class _Recorded:
    """The package's operators, each call kept with copies of what it was given."""

    def __init__(self, ops, monkeypatch):
        self.calls = []
        for name in ("gated_norm", "rotary_axes", "cache_append", "cache_attention"):
            monkeypatch.setattr(ops, name, self._wrap(name, getattr(ops, name)))

    def _wrap(self, name, fn):
        def call(*args, **kw):
            copy = lambda t: t.clone() if isinstance(t, torch.Tensor) else t  # noqa: E731
            given, named = [copy(a) for a in args], {k: copy(v) for k, v in kw.items()}
            out = fn(*args, **kw)
            held = tuple(copy(o) for o in out) if isinstance(out, tuple) else copy(out)
            self.calls.append((name, given, named, held))
            return out
        return call


def _rnd(seed, *s):
    return R._rand(seed, *s).to(DEV)


@pytest.fixture
def vb():
    from w4a4_post_quantized_channel_amd import video_block
    return video_block


@pytest.mark.parametrize("fmt,dtype,causal,page", [(None, BF, False, 16), ("int8", F32, True, 32), ("int4", BF, False, 64)])
def test_every_call_of_a_step(vb, monkeypatch, fmt, dtype, causal, page):
    B, H, W, frames = 2, 3, 7, 3
    T = H * W
    block = vb.random_block(DIM, HQ, HKV, D, F, SECTIONS, fmt)
    hist = vb.History(B, frames * T + 5, page, HKV, D, 2.0 ** -8, 2.0 ** -8)
    rec = _Recorded(vb.ops, monkeypatch)
    mod = 0.3 * _rnd(1, B, 6, DIM)
    for f in range(frames):
        x = _rnd(10 + f, B, T, DIM).to(dtype)
        pos = vb.frame_positions(f, 1, H, W).repeat(B, 1)
        assert pos[T - 1].tolist() == [f, H - 1, W - 1] and torch.equal(pos[:T], pos[T:])
        slots = hist.slots(T)
        rec.calls.clear()
        y = block.step(x, pos, mod, hist, slots, causal=causal)
        assert [c[0] for c in rec.calls] == ["gated_norm", "rotary_axes", "cache_append", "cache_attention",
                                             "gated_norm", "gated_norm"]
        norm1, rot, app, att, norm2, norm3 = rec.calls
        for (_, given, kw, out), post, with_h in ((norm1, None, False), (norm2, block.post_attn, True), (norm3, None, True)):
            ref = R._gated_reference(given[0], given[1] if with_h else None, kw.get("gate"), 1.0, post, "layer", None,
                                     None, kw.get("scale"), kw.get("shift"), 1e-6)
            R._assert_gated(out[0], out[1], ref, post is not None)
        assert torch.equal(norm1[1][0], x.view(B * T, DIM))              # the stream runs through all three
        assert torch.equal(norm2[1][0], norm1[1][0]) and torch.equal(norm3[1][0], norm2[3][0])
        assert torch.equal(y, norm3[3][0].view(B, T, DIM))
        for i in (0, 1):
            R._assert_rotary(rot[3][i], rot[1][i], pos, SECTIONS, True)
        # the cache holds what was appended, in every sequence's slots
        k, v = app[1][1], app[1][2]
        assert torch.equal(k, rot[3][1]) and int(hist.lens[0]) == (f + 1) * T
        for s_b in range(B):
            for t in range(T):
                j = f * T + t
                assert int(slots[s_b * T + t]) == int(hist.table[s_b, j // page]) * page + j % page
        for t, codes, scales in ((k, hist.cache.k_codes, hist.cache.k_scales), (v, hist.cache.v_codes, hist.cache.v_scales)):
            nib, e, _, _ = R.O.quantize_nvfp4(t.float().cpu().numpy().reshape(-1, D), np.float32(2.0 ** -8))
            at = slots.long().cpu()
            got = codes.cpu()[at // page, :, at % page].reshape(-1, D // 2).numpy()
            assert np.array_equal(got, R.O.pack_nibbles(nib))
            assert np.array_equal(scales.cpu()[at // page, :, at % page].reshape(-1, D // 16).numpy(), e)
        q = att[1][0]
        assert torch.equal(q.reshape(B * T, HQ, D), rot[3][0])
        ref = R._attention_reference(q, hist.cache, hist.table, hist.lens, causal, D ** -0.5)
        vmax = float(v.abs().max()) * 1.2 + 1.0                          # earlier frames' values are alike
        R._assert_attention(att[3], ref, frames * T + page, vmax)


def test_a_captured_step_follows_its_inputs(vb):
    B, H, W = 2, 2, 5
    T = H * W
    block = vb.random_block(DIM, HQ, HKV, D, F, SECTIONS, "int8")
    mod = 0.3 * _rnd(1, B, 6, DIM)

    def history():
        h = vb.History(B, 4 * T, 16, HKV, D, 2.0 ** -8, 2.0 ** -8)
        for f in range(2):
            block.step(_rnd(f, B, T, DIM).to(BF), vb.frame_positions(f, 1, H, W).repeat(B, 1), mod, h, h.slots(T))
        return h

    hist, again = history(), history()
    x, pos = _rnd(5, B, T, DIM).to(BF), vb.frame_positions(2, 1, H, W).repeat(B, 1)
    slots = hist.slots(T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, pos, mod, hist, slots)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, pos, mod, hist, slots)
    eager_slots = again.slots(T)
    for n in range(3):
        x.copy_(_rnd(20 + n, B, T, DIM).to(BF))
        mod.copy_(0.2 * _rnd(30 + n, B, 6, DIM))
        want = block.step(x, pos, mod, again, eager_slots)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert torch.equal(hist.cache.k_codes[hist.table.long().view(-1)][:1], again.cache.k_codes[again.table.long().view(-1)][:1])


def test_a_dropped_page_is_not_seen_and_a_full_history_grows_no_further(vb):
    B, T = 1, 16
    block = vb.random_block(DIM, HQ, HKV, D, F, SECTIONS, None)
    hist = vb.History(B, 3 * T, 16, HKV, D, 2.0 ** -8, 2.0 ** -8)
    mod = 0.3 * _rnd(1, B, 6, DIM)
    for f in range(3):
        slots = hist.slots(T)
        y = block.step(_rnd(f, B, T, DIM).to(BF), vb.frame_positions(f, 1, 4, 4), mod, hist, slots)
    again = block.step(_rnd(2, B, T, DIM).to(BF), vb.frame_positions(2, 1, 4, 4), mod, hist, slots)
    assert torch.equal(y, again)
    hist.cache.v_scales[int(hist.table[0, 1])] = 0x7E                   # loud values in the second page
    loud = block.step(_rnd(2, B, T, DIM).to(BF), vb.frame_positions(2, 1, 4, 4), mod, hist, slots)
    hist.table[0, 1] = -1
    dropped = block.step(_rnd(2, B, T, DIM).to(BF), vb.frame_positions(2, 1, 4, 4), mod, hist, slots)
    assert not torch.equal(loud, y) and not torch.equal(dropped, loud)
    full = hist.cache.k_codes.clone()
    assert bool((hist.slots(T) == -1).all())
    block.step(_rnd(3, B, T, DIM).to(BF), vb.frame_positions(3, 1, 4, 4), mod, hist, torch.full((T,), -1, dtype=torch.int32, device=DEV))
    assert torch.equal(hist.cache.k_codes, full)


def test_main_runs(vb, capsys):
    vb.main()
    out = capsys.readouterr().out
    assert "video block: a frame of 1560 tokens over 12480" in out and "nan" not in out
