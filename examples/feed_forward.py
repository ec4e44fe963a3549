"""A gated feed-forward block on libgbmm: forward, backward, and the same block with 8-bit
weights and activations.

    python examples/feed_forward.py         # differences between the two forms, times

y = (silu(x Wg^T) * (x Wu^T)) Wd^T.  PyTorch holds the memory and, between the 8-bit products, evaluates the gate;
every other step is a call of the library.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples.moe_layer import NAMES, gemm, milliseconds, stream  # noqa: E402
from gemv_moe_expert_gb300 import binding as gb  # noqa: E402


class FeedForward:
    """`hidden` wide rows through an inner width of `inner`; gate and up projection in one [2 inner, hidden] matrix."""

    def __init__(self, hidden, inner, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.inner, self.dtype, self.name = hidden, inner, dtype, NAMES[dtype]
        self.w_in = (torch.randn(2 * inner, hidden, generator=g, device="cuda") / hidden ** 0.5).to(dtype)
        self.w_out = (torch.randn(hidden, inner, generator=g, device="cuda") / inner ** 0.5).to(dtype)
        self.q_in, self.q_out = self.quantise(self.w_in), self.quantise(self.w_out)

    def new(self, *shape, dtype=None):
        return torch.empty(*shape, dtype=dtype or self.dtype, device="cuda")

    def scratch(self, answer):
        gb.check(answer[0])
        return self.new(max(answer[1], 1), dtype=torch.uint8), answer[1]

    def gated(self, x, keep):
        """h, and with `keep` both projections side by side in one [m, 2 inner] matrix."""
        m, n, k = x.shape[0], self.inner, self.hidden
        h, both = self.new(m, n), self.new(m, 2 * n) if keep else None
        gate, up = (both, both[:, n:]) if keep else (None, None)
        room, need = self.scratch(gb.gbmm_gated_scratch_bytes(self.name, m, n, k, True))
        gb.check(gb.gbmm_gated(self.name, gb.GATE_SILU, m, n, k, x, k, self.w_in, self.w_in[n:], k, h, n, gate, up, 2 * n,
                               room, need, stream()))
        return h, both

    def forward(self, x):
        """y, and what backward() needs."""
        h, both = self.gated(x, True)
        return gemm(h, self.w_out, self.new(x.shape[0], self.hidden), transpose_b=True), (x, h, both)

    def backward(self, kept, d_y):
        """Gradients of x, w_in and w_out."""
        x, h, both = kept
        m, n, k = x.shape[0], self.inner, self.hidden
        d_w_out = gemm(d_y, h, self.new(k, n), transpose_a=True)
        d_h = gemm(d_y, self.w_out, self.new(m, n))
        d_x, d_w_in = self.new(m, k), self.new(2 * n, k)
        room, need = self.scratch(gb.gbmm_gated_backward_scratch_bytes(self.name, m, n, k, True))
        gb.check(gb.gbmm_gated_backward(self.name, gb.GATE_SILU, m, n, k, x, k, self.w_in, self.w_in[n:], k, both,
                                        both[:, n:], 2 * n, d_h, n, d_x, k, d_w_in, d_w_in[n:], k, room, need,
                                        stream()))
        return d_x, d_w_in, d_w_out

    def quantise(self, rows):
        """8-bit codes and a scale for each row."""
        m, k = rows.shape
        q, scale = self.new(m, k, dtype=torch.int8), self.new(m, dtype=torch.float32)
        gb.check(gb.gbmm_quantize_i8(self.name, m, k, rows, k, q, k, scale, stream()))
        return q, scale

    def product_i8(self, x, weights, out):
        """out = x w^T from 8-bit codes of both."""
        (q, scale), (w, w_scale) = self.quantise(x), weights
        (m, n), k = out.shape, x.shape[1]
        room, need = self.scratch(gb.gbmm_gemm_i8_scratch_bytes(m, n, k, k % 16 == 0))
        gb.check(gb.gbmm_gemm_i8(NAMES[out.dtype], m, n, k, q, k, scale, w, k, w_scale, out, n, room, need, stream()))
        return out

    def serve(self, x):
        """The block with 8-bit weights and activations; nothing waits for the device."""
        m, n = x.shape[0], self.inner
        both = self.product_i8(x, self.q_in, self.new(m, 2 * n))
        h = torch.nn.functional.silu(both[:, :n]) * both[:, n:]
        return self.product_i8(h, self.q_out, self.new(m, self.hidden))


def main():
    block = FeedForward(hidden=4096, inner=11008)
    x = torch.randn(2048, block.hidden, device="cuda").to(block.dtype)
    y, kept = block.forward(x)
    block.backward(kept, torch.randn_like(y))
    few = x[:8].contiguous()
    print("2048 tokens, %d x %d, bf16" % (block.inner, block.hidden))
    print("8-bit block against bf16, 8 tokens: relative difference %.3f" %
          ((block.serve(few).float() - y[:8].float()).norm() / y[:8].float().norm()).item())
    print("forward   %8.3f ms" % milliseconds(lambda: block.forward(x)))
    print("backward  %8.3f ms" % milliseconds(lambda: block.backward(kept, y)))
    print("8 bits    %8.3f ms" % milliseconds(lambda: block.serve(x)))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        block.serve(few)
    print("8 tokens in 8 bits, replayed from a graph %8.3f ms" % milliseconds(graph.replay))


if __name__ == "__main__":
    main()
