"""A block of an autoregressive video model whose history is a 4-bit cache.

What stands between the quantized linears of such a block, put together as a
model runs it, frame after frame (or action token after action token):

* gated norm: the modulated norm in front of the projections, and the gated
  residual behind them fused with the next one;
* quantized query / key / value projection;
* rotary positions over time, height and width on queries and keys;
* the new keys and values appended to the paged NVFP4 cache;
* attention of the new tokens over the whole history in the cache;
* quantized output projection, and a SwiGLU feed-forward in 16 bits.

``python -m w4a4_post_quantized_channel_amd.video_block`` runs a frame over a
history on the GPU, captures it in a HIP graph and prints its time.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import ops
from .pipeline import QuantizedLinear


class History:
    """The cached keys and values of B sequences in one block, and where they lie.

    Every sequence has room for ``max_len`` tokens, in pages of its own in order;
    ``table`` and ``lens`` are what ops.cache_attention takes.  Writing -1 to an
    entry of the table drops that page: its keys are no longer seen.
    """

    def __init__(self, B: int, max_len: int, page: int, Hkv: int, D: int, k_scale: float, v_scale: float, device="cuda"):
        pages = -(-max_len // page)
        self.cache = ops.make_kv_cache(B * pages, page, Hkv, D, k_scale, v_scale, device=device)
        self.table = torch.arange(B * pages, dtype=torch.int32, device=device).view(B, pages)
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)
        self.max_len = max_len

    def slots(self, T: int) -> torch.Tensor:
        """Token slots int32[B * T] of the next T tokens of every sequence; grows the history by them.
        (Tokens past max_len have no slot: they are not cached, and not seen.)"""
        pos = self.lens.unsqueeze(1) + torch.arange(T, dtype=torch.int32, device=self.lens.device)
        at = torch.clamp(pos // self.cache.page, max=self.table.shape[1] - 1)
        page = torch.gather(self.table, 1, at.long())
        slots = torch.where((pos < self.max_len) & (page >= 0), page * self.cache.page + pos % self.cache.page, -1)
        self.lens += T
        return slots.view(-1)


class VideoBlock:
    """A transformer block over a 4-bit history.

    wqkv [(Hq + 2 Hkv) D, dim] and wo [dim, Hq D] are packed once as ``fmt``
    codes (None: kept as 16-bit products); w_gate_up [2 F, dim], w_down [dim, F]
    are bf16.  post_attn fp32[dim] or None: the norm behind the attention.
    Intermediates come from the allocator on the stream of the call, none is
    kept.
    """

    def __init__(self, Hq: int, Hkv: int, D: int, sections, wqkv: torch.Tensor, wo: torch.Tensor,
                 w_gate_up: torch.Tensor, w_down: torch.Tensor, fmt: Optional[str] = "int8",
                 post_attn: Optional[torch.Tensor] = None, theta: float = 10000.0):
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.table = ops.make_rotary_table(sections, theta, device=wqkv.device)
        pack = (lambda w: QuantizedLinear(w.float(), None, None, fmt)) if fmt else (lambda w: w.bfloat16())
        self.qkv, self.wo, self.w_gate_up, self.w_down = pack(wqkv), pack(wo), w_gate_up, w_down
        self.post_attn = post_attn

    @staticmethod
    def _linear(w, x, **kw):
        if isinstance(w, QuantizedLinear):
            return w.with_own_buffers().forward(x)
        ws = ops.make_bf16_linear_workspace(x.shape[0], w.shape[0] // (2 if kw.get("act") == "swiglu" else 1), x.shape[1],
                                            kw.get("act", "none"), device=x.device)
        return ops.bf16_linear(x, w, workspace=ws, **kw)

    def step(self, x: torch.Tensor, pos: torch.Tensor, mod: torch.Tensor, history: History, slots: torch.Tensor, *,
             causal: bool = False) -> torch.Tensor:
        """The residual stream after the block.

        x [B, T, dim] (fp32 or bf16) are the new tokens, pos int32 [B * T, axes]
        their positions, slots what history.slots(T) gave for them, mod fp32
        [B, 6, dim] the timestep's shift, scale and gate of both halves.
        causal: a token sees the new tokens up to itself, else all of them.
        """
        B, T, dim = x.shape
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        x = x.reshape(B * T, dim)
        _, h = ops.gated_norm(x, shift=mod[:, 0], scale=mod[:, 1])
        qkv = self._linear(self.qkv, h).view(B * T, Hq + 2 * Hkv, D)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        ops.rotary_axes(q, k, pos, self.table, q_out=q, k_out=k)
        ops.cache_append(history.cache, k, v, slots)
        ws = ops.make_cache_attention_workspace(B, T, Hq, Hkv, D, history.max_len, device=x.device)
        a = ops.cache_attention(qkv.view(B, T, Hq + 2 * Hkv, D)[:, :, :Hq], history.cache, history.table, history.lens,
                                causal=causal, max_len=history.max_len, workspace=ws)
        o = self._linear(self.wo, a.view(B * T, Hq * D))
        x, h = ops.gated_norm(x, o, gate=mod[:, 2], post_weight=self.post_attn, shift=mod[:, 3], scale=mod[:, 4])
        f = self._linear(self.w_down, self._linear(self.w_gate_up, h, act="swiglu"))
        x, _ = ops.gated_norm(x, f, gate=mod[:, 5], norm=False)
        return x.view(B, T, dim)


def random_block(dim: int, Hq: int, Hkv: int, D: int, F: int, sections, fmt: Optional[str], seed: int = 0, device="cuda",
                 post: bool = True) -> VideoBlock:
    """A VideoBlock with seeded random weights."""
    g = torch.Generator().manual_seed(seed)

    def w(n, k):
        return (torch.randn(n, k, generator=g) / k ** 0.5).bfloat16().to(device)

    wqkv, wo, gu, dn = w((Hq + 2 * Hkv) * D, dim), w(dim, Hq * D), w(2 * F, dim), w(dim, F)
    p = (1 + 0.1 * torch.randn(dim, generator=g)).to(device) if post else None
    return VideoBlock(Hq, Hkv, D, sections, wqkv, wo, gu, dn, fmt, p)


def frame_positions(first: int, frames: int, height: int, width: int, device="cuda") -> torch.Tensor:
    """int32 [frames * height * width, 3]: time, row and column of every token, time from ``first`` on."""
    t = torch.arange(first, first + frames, dtype=torch.int32, device=device)
    h, w = (torch.arange(n, dtype=torch.int32, device=device) for n in (height, width))
    return torch.stack(torch.meshgrid(t, h, w, indexing="ij"), dim=-1).view(-1, 3)


def main():
    dim, Hq, Hkv, D, F, B, H, W, past = 2048, 16, 16, 128, 8192, 1, 30, 52, 7
    T = H * W
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    block = random_block(dim, Hq, Hkv, D, F, [22, 21, 21], "int8")
    history = History(B, (past + 1) * T, 64, Hkv, D, 2.0 ** -8, 2.0 ** -8)
    mod = 0.3 * rnd(B, 6, dim)
    for f in range(past):
        block.step(rnd(B, T, dim), frame_positions(f, 1, H, W).repeat(B, 1), mod, history, history.slots(T))
    x, pos, slots = rnd(B, T, dim), frame_positions(past, 1, H, W).repeat(B, 1), history.slots(T)
    block.step(x, pos, mod, history, slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, pos, mod, history, slots)
    graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(50):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"video block: a frame of {T} tokens over {past * T + T} in a 4-bit cache, {start.elapsed_time(end) * 20:.1f} us, "
          f"output rms {float(y.float().pow(2).mean().sqrt()):.3f}")


if __name__ == "__main__":
    main()
