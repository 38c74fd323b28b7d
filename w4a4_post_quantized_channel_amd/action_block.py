"""One step of an action expert over a shared observation, on this library.

What stands between the low-bit linears of a world-action model, put together
as a step uses it:

* ``FeatureTokens``: autoencoder features -> group norm with SiLU -> a 16-bit
  product with bias -> tokens of the observation;
* ``ActionBlock``: the observation's keys and values (computed once), and per
  step for a batch of sampled action chunks: layer norm, quantized query /
  key / value projection, attention over observation and chunk, and the 16-bit
  output, SwiGLU and down projections that write the residual stream.

``python -m w4a4_post_quantized_channel_amd.action_block`` runs a step on the
GPU, captures it in a HIP graph and prints its time.
"""
from __future__ import annotations

import functools
from typing import Optional

import torch

from . import ops
from .pipeline import QuantizedLinear


@functools.lru_cache(maxsize=256)
def _scratch_bytes(B: int, T: int, P: int, dim: int, F: int, Hq: int, Hkv: int, D: int) -> int:
    """Bytes that cover every 16-bit call of a step (a host query of five plans)."""
    M = B * T
    return max(ops.bf16_linear_workspace_size(M, (Hq + 2 * Hkv) * D, dim),
               ops.prefix_attention_workspace_size(B, T, Hq, Hkv, D, P, T),
               ops.bf16_linear_workspace_size(M, dim, Hq * D), ops.bf16_linear_workspace_size(M, F, dim, "swiglu"),
               ops.bf16_linear_workspace_size(M, dim, F))


class FeatureTokens:
    """tokens = (silu(group_norm(features)) W^T + b) for channels-last features [S, C]."""

    def __init__(self, groups: int, norm_w: torch.Tensor, norm_b: torch.Tensor, w: torch.Tensor, b: torch.Tensor):
        self.groups, self.norm_w, self.norm_b, self.w, self.b = groups, norm_w, norm_b, w, b

    def __call__(self, features: torch.Tensor, stream=None) -> torch.Tensor:
        S, C = features.shape
        with torch.cuda.stream(stream):
            ws = ops.make_group_norm_workspace(1, S, C, self.groups, device=features.device)
            h = ops.group_norm_act(features.unsqueeze(0), self.groups, self.norm_w, self.norm_b, act="silu",
                                   workspace=ws)[0]
            ws = ops.make_bf16_linear_workspace(S, self.w.shape[0], C, device=features.device)
            return ops.bf16_linear(h, self.w, bias=self.b, workspace=ws)


class ActionBlock:
    """A transformer block of the action expert.

    wqkv   [(Hq + 2 Hkv) D, dim] float, packed once as ``fmt`` codes (None: kept as a 16-bit product);
    wkv    [2 Hkv D, dim] bf16, the observation's keys and values;
    wo     [dim, Hq D], bo [dim];  w_gate_up [2 F, dim];  w_down [dim, F] (bf16, bias fp32).

    Each call takes its intermediates, partial sums and result from the
    allocator on the stream that it runs on (``stream``, or the current one)
    and keeps none, so calls on several streams, in several threads or in
    captured graphs may overlap.
    """

    def __init__(self, Hq: int, Hkv: int, D: int, wqkv: torch.Tensor, wkv: torch.Tensor, wo: torch.Tensor,
                 bo: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, fmt: Optional[str] = "int4"):
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.qkv = QuantizedLinear(wqkv.float(), None, None, fmt) if fmt else wqkv.bfloat16()
        self.wkv, self.wo, self.bo, self.w_gate_up, self.w_down = wkv, wo, bo, w_gate_up, w_down

    def _workspaces(self, B: int, T: int, P: int, device):
        """One buffer for the step's calls, which follow each other on a stream."""
        nbytes = _scratch_bytes(B, T, P, self.wo.shape[0], self.w_down.shape[1], self.Hq, self.Hkv, self.D)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
        return dict.fromkeys(("qkv", "attn", "o", "gate_up", "down"), ws)

    def observe(self, tokens: torch.Tensor, stream=None):
        """Keys and values [P, Hkv, D] of the observation, shared by every sequence and step."""
        with torch.cuda.stream(stream):
            ws = ops.make_bf16_linear_workspace(tokens.shape[0], self.wkv.shape[0], tokens.shape[1],
                                                device=tokens.device)
            kv = ops.bf16_linear(tokens, self.wkv, workspace=ws)
        kv = kv.view(-1, 2, self.Hkv, self.D)
        return kv[:, 0], kv[:, 1]

    def _norm(self, x: torch.Tensor) -> torch.Tensor:
        # layer norm of every token: group norm with one group and one position a sample
        M, dim = x.shape
        return ops.group_norm_act(x.view(M, 1, dim), 1, act="none").view(M, dim)

    def step(self, x: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor, keep: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
        """The block's output for chunks x [B, T, dim] (bf16) that see the kept
        observation tokens and their own chunk."""
        with torch.cuda.stream(stream):
            return self._step(x, k_prefix, v_prefix, keep)

    def _step(self, x, k_prefix, v_prefix, keep):
        B, T, dim = x.shape
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        ws = self._workspaces(B, T, k_prefix.shape[0], x.device)
        x = x.reshape(B * T, dim)
        h = self._norm(x)
        if isinstance(self.qkv, QuantizedLinear):
            qkv = self.qkv.with_own_buffers().forward(h)
        else:
            qkv = ops.bf16_linear(h, self.qkv, workspace=ws["qkv"])
        qkv = qkv.view(B, T, Hq + 2 * Hkv, D)
        a = ops.prefix_attention(qkv[:, :, :Hq], k_prefix, v_prefix, qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:],
                                 prefix_keep=keep, workspace=ws["attn"])
        x = ops.bf16_linear(a.view(B * T, Hq * D), self.wo, bias=self.bo, residual=x, workspace=ws["o"])
        g = ops.bf16_linear(self._norm(x), self.w_gate_up, act="swiglu", workspace=ws["gate_up"])
        return ops.bf16_linear(g, self.w_down, residual=x, workspace=ws["down"]).view(B, T, dim)


def random_block(dim: int, Hq: int, Hkv: int, D: int, F: int, fmt: Optional[str], seed: int = 0, device="cuda"):
    """An ActionBlock with seeded random weights."""
    g = torch.Generator().manual_seed(seed)

    def w(n, k):
        return (torch.randn(n, k, generator=g) / k ** 0.5).bfloat16().to(device)

    return ActionBlock(Hq, Hkv, D, w((Hq + 2 * Hkv) * D, dim), w(2 * Hkv * D, dim), w(dim, Hq * D),
                       (torch.randn(dim, generator=g) * 0.1).to(device), w(2 * F, dim), w(dim, F), fmt)


def main():
    dim, Hq, Hkv, D, F, B, T, C = 2048, 16, 4, 128, 8192, 8, 50, 384
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    to_tokens = FeatureTokens(32, 1 + 0.1 * rnd(C), 0.1 * rnd(C), (rnd(dim, C) / C ** 0.5).bfloat16(), 0.1 * rnd(dim))
    block = random_block(dim, Hq, Hkv, D, F, "int4")
    k, v = block.observe(to_tokens(rnd(2040, C).bfloat16()))
    x = rnd(B, T, dim).bfloat16()
    block.step(x, k, v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, k, v)
    graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"action step: {B} chunks of {T} tokens over {k.shape[0]} observation tokens, "
          f"{start.elapsed_time(end) * 10:.1f} us, output rms {float(y.float().pow(2).mean().sqrt()):.3f}")


if __name__ == "__main__":
    main()
