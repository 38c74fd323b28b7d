"""What a video block's step leaves in its history, captured, and which keys it sees
once pages are dropped."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_cache_ops_gpu as R  # noqa: E402  (references and tolerances)
from test_video_block_gpu import BF, D, DEV, DIM, F, HKV, HQ, SECTIONS, _Recorded, _rnd, vb  # noqa: E402, F401


def test_a_captured_step_appends_its_tokens(vb):  # noqa: F811
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
    slots, eager_slots = hist.slots(T), again.slots(T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, pos, mod, hist, slots)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, pos, mod, hist, slots)
    whole = hist.table.view(B, -1, 1) * 16 + torch.arange(16, device=DEV, dtype=torch.int32)
    whole = whole.view(B, -1)[:, :3 * T].reshape(-1).contiguous()        # every token so far, in both histories
    before = None
    for n in range(3):
        x.copy_(_rnd(20 + n, B, T, DIM).to(BF))
        want = block.step(x, pos, mod, again, eager_slots)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        k, v = vb.ops.cache_read(hist.cache, slots)
        for got, ref in zip((k, v), vb.ops.cache_read(again.cache, eager_slots)):
            assert torch.equal(got, ref)
        for got, ref in zip(vb.ops.cache_read(hist.cache, whole), vb.ops.cache_read(again.cache, whole)):
            assert torch.equal(got, ref)
        if before is not None:                         # other inputs, other tokens
            assert not torch.equal(k, before[0]) and not torch.equal(v, before[1])
        before = k, v


@pytest.mark.parametrize("B,causal,drop", [(1, False, [1]), (2, True, [0, 2]), (2, False, [0, 1, 2, 3])])
def test_a_step_sees_the_pages_that_are_left(vb, monkeypatch, B, causal, drop):  # noqa: F811
    T, frames = 16, 4
    block = vb.random_block(DIM, HQ, HKV, D, F, SECTIONS, None)
    hist = vb.History(B, frames * T, 16, HKV, D, 2.0 ** -8, 2.0 ** -8)
    mod = 0.3 * _rnd(1, B, 6, DIM)
    for f in range(frames):
        slots = hist.slots(T)
        x, pos = _rnd(f, B, T, DIM).to(BF), vb.frame_positions(f, 1, 4, 4).repeat(B, 1)
        block.step(x, pos, mod, hist, slots, causal=causal)
    for p in drop:                                     # gone, and loud: the last sequence alone
        hist.cache.v_scales[int(hist.table[B - 1, p])] = 0x7E
        hist.table[B - 1, p] = -1
    rec = _Recorded(vb.ops, monkeypatch)
    gone = slots.clone()
    if 3 in drop:
        gone.view(B, T)[B - 1] = -1                    # (the new tokens' own page)
    block.step(x, pos, mod, hist, gone, causal=causal)
    att = next(c for c in rec.calls if c[0] == "cache_attention")
    ref = R._attention_reference(att[1][0], hist.cache, hist.table, hist.lens, causal, D ** -0.5)
    assert torch.equal(att[1][2], hist.table) and hist.lens.tolist() == [frames * T] * B
    R._assert_attention(att[3], ref, frames * T + 16, float(np.abs(ref[0].numpy()).max()) + 8.0)
