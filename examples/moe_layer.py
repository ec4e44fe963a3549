"""A mixture-of-experts layer on libgbmm: router, expert order, expert products and
combine, forward and backward, and the same layer for a few tokens with 4-bit weights.

    python examples/moe_layer.py            # sizes, differences between the two forms, times

y[t] = sum over the chosen experts e of w[t,e] * W2[e] silu(W1[e] x[t]).  PyTorch holds the
memory and evaluates silu; every other step is a call of the library.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gemv_moe_expert_gb300 import binding as gb  # noqa: E402

NAMES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}


def stream():
    return torch.cuda.current_stream().cuda_stream


def gemm(a, b, out, transpose_a=False, transpose_b=False):
    """out = op(a) op(b) for 2-D tensors whose rows are contiguous."""
    m, n = out.shape
    k = a.shape[0] if transpose_a else a.shape[1]
    gb.check(gb.gbmm_gemm(NAMES[out.dtype], 1, m, n, k, transpose_a, transpose_b, a, 0, a.stride(0), 0, b, 0,
                          b.stride(0), 0, out, 0, out.stride(0), 0, stream()))
    return out


def silu_gradient(h, d_a):
    s = torch.sigmoid(h)
    return d_a * s * (1 + h * (1 - s))


def quantise(w, group):
    """4-bit codes, f16 scales and zero points of w [..., n, k], k even and a multiple of
    `group`: the group's range divided into 15 steps."""
    cut = w.float().unflatten(-1, (-1, group))
    low, high = cut.amin(-1, keepdim=True).clamp(max=0), cut.amax(-1, keepdim=True).clamp(min=0)
    scale = ((high - low) / 15).clamp_min(1e-6).half()
    zero = (-low / scale.float()).round().clamp(0, 15)
    code = ((cut / scale.float()).round() + zero).clamp(0, 15).to(torch.uint8).flatten(-2)
    return (code[..., 0::2] | code[..., 1::2] << 4).contiguous(), scale.squeeze(-1), zero.squeeze(-1).to(torch.uint8)


class MoeLayer:
    """`hidden` wide rows through `top_k` of `experts` experts of width `inner`."""

    def __init__(self, hidden, inner, experts, top_k, dtype=torch.bfloat16, group=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") / shape[-1] ** 0.5).to(dtype)
        self.hidden, self.inner, self.experts, self.top_k, self.group = hidden, inner, experts, top_k, group
        self.dtype, self.name = dtype, NAMES[dtype]
        self.router = normal(experts, hidden)
        self.w1, self.w2 = normal(experts, inner, hidden), normal(experts, hidden, inner)
        self.q1, self.q2 = quantise(self.w1, group), quantise(self.w2, group)

    def new(self, *shape, dtype=None):
        return torch.empty(*shape, dtype=dtype or self.dtype, device="cuda")

    def route(self, x):
        m = x.shape[0]
        logits = gemm(x, self.router, self.new(m, self.experts), transpose_b=True)
        ids, w = self.new(m, self.top_k, dtype=torch.int32), self.new(m, self.top_k, dtype=torch.float32)
        gb.check(gb.gbmm_moe_route(self.name, m, self.experts, self.top_k, gb.SOFTMAX_ALL, logits, self.experts, None,
                                   ids, w, stream()))
        return logits, ids, w

    def segments(self, offsets):
        """(expert, first place, end) of the experts that have rows; waits for the device."""
        o = offsets.tolist()
        return [(e, o[e], o[e + 1]) for e in range(self.experts) if o[e] < o[e + 1]]

    def forward(self, x):
        """y, and what backward() needs."""
        m, rows = x.shape[0], x.shape[0] * self.top_k
        logits, ids, w = self.route(x)
        offsets = self.new(self.experts + 1, dtype=torch.int32)
        order, position = self.new(rows, dtype=torch.int32), self.new(rows, dtype=torch.int32)
        status, nbytes = gb.gbmm_moe_sort_scratch_bytes(m, self.top_k, self.experts)
        gb.check(status)
        scratch = self.new(nbytes, dtype=torch.uint8)
        gb.check(gb.gbmm_moe_sort(m, self.top_k, self.experts, ids, offsets, order, position, scratch, nbytes,
                                  stream()))
        xs, h, ys = self.new(rows, self.hidden), self.new(rows, self.inner), self.new(rows, self.hidden)
        gb.check(gb.gbmm_moe_dispatch(self.name, m, self.top_k, self.experts, self.hidden, x, self.hidden, position,
                                      offsets, xs, self.hidden, stream()))
        parts = self.segments(offsets)
        for e, b0, b1 in parts:
            gemm(xs[b0:b1], self.w1[e], h[b0:b1], transpose_b=True)
        a = torch.nn.functional.silu(h)
        for e, b0, b1 in parts:
            gemm(a[b0:b1], self.w2[e], ys[b0:b1], transpose_b=True)
        y = self.new(m, self.hidden)
        gb.check(gb.gbmm_moe_combine(self.name, m, self.top_k, self.experts, self.hidden, ys, self.hidden, w, position,
                                     offsets, y, self.hidden, stream()))
        return y, (x, logits, ids, w, offsets, position, parts, xs, h, a, ys)

    def backward(self, kept, d_y):
        """Gradients of x, router, w1 and w2."""
        x, logits, ids, w, offsets, position, parts, xs, h, a, ys = kept
        m, rows = x.shape[0], xs.shape[0]
        d_ys, d_w = self.new(rows, self.hidden), self.new(m, self.top_k, dtype=torch.float32)
        gb.check(gb.gbmm_moe_combine_backward(self.name, m, self.top_k, self.experts, self.hidden, ys, self.hidden, w,
                                              position, offsets, d_y, self.hidden, d_ys, self.hidden, d_w, stream()))
        d_w1, d_w2 = torch.zeros_like(self.w1), torch.zeros_like(self.w2)
        d_a, d_xs = self.new(rows, self.inner), self.new(rows, self.hidden)
        for e, b0, b1 in parts:
            gemm(d_ys[b0:b1], a[b0:b1], d_w2[e], transpose_a=True)
            gemm(d_ys[b0:b1], self.w2[e], d_a[b0:b1])
        d_h = silu_gradient(h, d_a)
        for e, b0, b1 in parts:
            gemm(d_h[b0:b1], xs[b0:b1], d_w1[e], transpose_a=True)
            gemm(d_h[b0:b1], self.w1[e], d_xs[b0:b1])
        d_x, d_logits = self.new(m, self.hidden), self.new(m, self.experts)
        gb.check(gb.gbmm_moe_dispatch_backward(self.name, m, self.top_k, self.experts, self.hidden, d_xs, self.hidden,
                                               position, offsets, d_x, self.hidden, stream()))
        gb.check(gb.gbmm_moe_route_backward(self.name, m, self.experts, self.top_k, gb.SOFTMAX_ALL, logits,
                                            self.experts, None, ids, w, d_w, d_logits, self.experts, stream()))
        d_router = gemm(d_logits, x, self.new(self.experts, self.hidden), transpose_a=True)
        d_x += gemm(d_logits, self.router, self.new(m, self.hidden))
        return d_x, d_router, d_w1, d_w2

    def product_q4(self, q, n, k, layout, x, ids):
        """Routed rows [m, top_k, n]: each row of x times its expert's 4-bit matrix."""
        codes, scales, zeros = q
        m = ids.shape[0]
        out = self.new(m, self.top_k, n)
        gb.check(gb.gbmm_matmul_id_q4(self.name, m, n, k, self.top_k, self.experts, layout, self.group, codes,
                                      codes.stride(1), codes.stride(0), scales, "f16", zeros, x, ids, out, stream()))
        return out

    def decode(self, x):
        """The layer with 4-bit weights, for a few tokens: rows stay in routed order, and
        nothing waits for the device (the step can be captured into a CUDA graph)."""
        m = x.shape[0]
        _, ids, w = self.route(x)
        h = self.product_q4(self.q1, self.inner, self.hidden, gb.INPUT_SHARED_PER_TOKEN, x, ids)
        a = torch.nn.functional.silu(h)
        ys = self.product_q4(self.q2, self.hidden, self.inner, gb.INPUT_SLOTTED, a, ids)
        y = self.new(m, self.hidden)
        gb.check(gb.gbmm_moe_combine(self.name, m, self.top_k, self.experts, self.hidden, ys, self.hidden, w, None,
                                     None, y, self.hidden, stream()))
        return y


def milliseconds(f, times=20):
    for _ in range(3):
        f()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(times):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / times


def main():
    layer = MoeLayer(hidden=2048, inner=1408, experts=64, top_k=8)
    x = torch.randn(2048, layer.hidden, device="cuda").to(layer.dtype)
    y, kept = layer.forward(x)
    layer.backward(kept, torch.randn_like(y))
    few = x[:4].contiguous()
    q4 = layer.decode(few)
    torch.cuda.synchronize()
    print("2048 tokens, 8 of 64 experts, %d x %d, bf16" % (layer.inner, layer.hidden))
    print("4-bit weights against bf16, 4 tokens: relative difference %.3f" %
          ((q4.float() - y[:4].float()).norm() / y[:4].float().norm()).item())
    print("forward   %8.3f ms" % milliseconds(lambda: layer.forward(x)))
    print("backward  %8.3f ms" % milliseconds(lambda: layer.backward(kept, y)))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        layer.decode(few)
    print("decode of 4 tokens with 4-bit weights, replayed from a graph %8.3f ms" % milliseconds(graph.replay))


if __name__ == "__main__":
    main()
