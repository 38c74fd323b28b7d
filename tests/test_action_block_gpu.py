"""The action block: its 16-bit form against a 64-bit composition, its
quantized form against the same calls made one by one, and graph replays."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DIM, HQ, HKV, D, F, B, T, C, S = 256, 4, 2, 64, 320, 3, 7, 48, 90


@pytest.fixture(scope="module")
def blk():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a4_post_quantized_channel_amd import action_block
    return action_block


def _inputs():
    g = torch.Generator().manual_seed(7)
    feats = torch.randn(S, C, generator=g).bfloat16()
    norm_w, norm_b = 1 + 0.2 * torch.randn(C, generator=g), 0.2 * torch.randn(C, generator=g)
    w, b = (torch.randn(DIM, C, generator=g) / C ** 0.5).bfloat16(), 0.1 * torch.randn(DIM, generator=g)
    x = torch.randn(B, T, DIM, generator=g).bfloat16()
    keep = torch.rand(S, generator=g) < 0.8
    return feats, norm_w, norm_b, w, b, x, keep


def _run(blk, fmt):
    feats, norm_w, norm_b, w, b, x, keep = _inputs()
    tok = blk.FeatureTokens(8, norm_w.cuda(), norm_b.cuda(), w.cuda(), b.cuda())
    block = blk.random_block(DIM, HQ, HKV, D, F, fmt, seed=3)
    tokens = tok(feats.cuda())
    k, v = block.observe(tokens)
    return block, tokens, k, v, x.cuda(), keep.cuda(), block.step(x.cuda(), k, v, keep.cuda())


def test_sixteen_bit_block_against_64_bits(blk):
    block, tokens, _, _, x, keep, y = _run(blk, None)
    feats, norm_w, norm_b, w, b, x, keep = _inputs()
    f64 = lambda t: t.detach().cpu().double()
    # features -> tokens
    v = feats.double().view(S, 8, C // 8)
    h = (v - v.mean(dim=(0, 2), keepdim=True)) / torch.sqrt(v.var(dim=(0, 2), unbiased=False, keepdim=True) + 1e-5)
    h = h.reshape(S, C) * norm_w.double() + norm_b.double()
    tk = (h * torch.sigmoid(h)) @ w.double().t() + b.double()

    # every 16-bit value on the way is rounded to 8 significant bits; the sums below do not amplify that
    def close(got, want, steps):
        err = (f64(got) - want).abs()
        assert float(err.max()) <= steps * 2.0 ** -8 * float(want.abs().max()), float(err.max())

    close(tokens, tk, 2)
    kv = (tk @ f64(block.wkv).t()).view(S, 2, HKV, D)

    def norm(z):
        return (z - z.mean(-1, keepdim=True)) / torch.sqrt(z.var(-1, unbiased=False, keepdim=True) + 1e-5)

    z = x.double().view(B * T, DIM)
    qkv = (norm(z) @ f64(block.qkv).t()).view(B, T, HQ + 2 * HKV, D)
    a = torch.zeros(B, T, HQ, D, dtype=torch.float64)
    for bb in range(B):
        for hh in range(HQ):
            kk = torch.cat([kv[keep, 0, hh // 2], qkv[bb, :, HQ + hh // 2]])
            vv = torch.cat([kv[keep, 1, hh // 2], qkv[bb, :, HQ + HKV + hh // 2]])
            a[bb, :, hh] = torch.softmax(qkv[bb, :, hh] @ kk.t() / math.sqrt(D), -1) @ vv
    z = z + a.view(B * T, HQ * D) @ f64(block.wo).t() + f64(block.bo)
    gu = norm(z) @ f64(block.w_gate_up).t()
    z = z + (gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]) @ f64(block.w_down).t()
    close(y.view(B * T, DIM), z, 6)


def test_quantized_block_is_its_calls(blk):
    from w4a4_post_quantized_channel_amd import ops
    block, _, k, v, x, keep, y = _run(blk, "int4")
    flat = x.view(B * T, DIM)
    h = ops.group_norm_act(flat.view(B * T, 1, DIM), 1, act="none").view(B * T, DIM)
    q = block.qkv.forward(h).view(B, T, HQ + 2 * HKV, D)
    ws = block._workspaces(B, T, S, x.device)
    a = ops.prefix_attention(q[:, :, :HQ], k, v, q[:, :, HQ:HQ + HKV], q[:, :, HQ + HKV:], prefix_keep=keep,
                             workspace=ws["attn"])
    z = ops.bf16_linear(a.view(B * T, HQ * D), block.wo, bias=block.bo, residual=flat, workspace=ws["o"])
    h = ops.group_norm_act(z.view(B * T, 1, DIM), 1, act="none").view(B * T, DIM)
    g = ops.bf16_linear(h, block.w_gate_up, act="swiglu", workspace=ws["gate_up"])
    z = ops.bf16_linear(g, block.w_down, residual=z, workspace=ws["down"])
    torch.cuda.synchronize()
    assert torch.equal(y.view(B * T, DIM).view(torch.int16), z.view(torch.int16))
    assert torch.isfinite(y.float()).all()


def test_step_replays_from_a_graph(blk):
    block, _, k, v, x, keep, _ = _run(blk, "int4")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, k, v, keep)
    for i in range(3):
        x.mul_(-0.75)
        graph.replay()
        got = y.clone()
        want = block.step(x, k, v, keep)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), i
