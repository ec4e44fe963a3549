"""The example layer (examples/moe_layer.py) against a 64-bit layer with the same chosen
experts: router, expert order, dispatch, expert products, combine and their gradients,
and the step with 4-bit weights.

Bounds, on norms.  f32: each value passes through at most six sums of at most K = 256
products or 12 slots; a sum is off by at most K u of the sum of magnitudes, which for random
signs is sqrt(K) times the result: 6 * 256 * 16 * 2^-24 < 1.5e-3.  bf16: at most 16 stored
values lie between the inputs and any result (2^-9 each), and the logits' rounding
moves weights by 2^-9 times their magnitude (below 8) both ways: 32 * 2^-9 = 2^-4.
"""

from __future__ import annotations

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

BOUND = {torch.float32: 1.5e-3, torch.bfloat16: 2.0 ** -4, torch.float16: 2.0 ** -4}
CASES = [(torch.float32, 192, 160, 12, 3, 32, 70), (torch.bfloat16, 256, 128, 16, 4, 64, 33),
         (torch.float16, 128, 256, 5, 5, 128, 9), (torch.float32, 256, 128, 40, 1, 64, 1)]


def exact(x, router, w1, w2, ids):
    """The layer in the operands' precision, its experts given."""
    p = torch.softmax(x @ router.T, dim=1).gather(1, ids.long())
    y = torch.zeros_like(x)
    for e in range(router.shape[0]):
        t, s = (ids == e).nonzero(as_tuple=True)
        out = torch.nn.functional.silu(x[t] @ w1[e].T) @ w2[e].T
        y = y.index_add(0, t, p[t, s][:, None] * out)
    return y


def close(got, ref, bound, what):
    err = (got.double() - ref).norm() / ref.norm()
    assert err.item() <= bound, f"{what}: {err.item():.3g} > {bound:.3g}"


@pytest.mark.parametrize("dtype,hidden,inner,experts,top_k,group,m", CASES)
def test_layer(dtype, hidden, inner, experts, top_k, group, m):
    from moe_layer import MoeLayer
    layer = MoeLayer(hidden, inner, experts, top_k, dtype, group)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, hidden, generator=g, device="cuda").to(dtype)
    d_y = torch.randn(m, hidden, generator=g, device="cuda").to(dtype)
    y, kept = layer.forward(x)
    grads = layer.backward(kept, d_y)
    leaves = [v.double().requires_grad_() for v in (x, layer.router, layer.w1, layer.w2)]
    ref = exact(*leaves, kept[2])
    ref.backward(d_y.double())
    close(y, ref.detach(), BOUND[dtype], "y")
    for got, leaf, what in zip(grads, leaves, ("d_x", "d_router", "d_w1", "d_w2")):
        close(got, leaf.grad, BOUND[dtype], what)


@pytest.mark.parametrize("dtype,hidden,inner,experts,top_k,group,m", CASES)
def test_decode(dtype, hidden, inner, experts, top_k, group, m):
    from moe_layer import MoeLayer
    layer = MoeLayer(hidden, inner, experts, top_k, dtype, group)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(m, hidden, generator=g, device="cuda").to(dtype)

    def widen(q):
        codes, scales, zeros = q
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double().unflatten(-1, (-1, group))
        return ((c - zeros[..., None].double()) * scales[..., None].double()).flatten(-2)
    w1, w2 = widen(layer.q1), widen(layer.q2)
    assert (w1 - layer.w1.double()).norm() < 0.2 * layer.w1.double().norm()  # the codes stand for the weights
    _, ids, _ = layer.route(x)
    close(layer.decode(x), exact(x.double(), layer.router.double(), w1, w2, ids), BOUND[dtype], "y")


def test_decode_from_a_graph():
    from moe_layer import MoeLayer
    layer = MoeLayer(128, 256, 8, 2, torch.bfloat16, 64)
    x = torch.randn(3, 128, device="cuda").to(torch.bfloat16)
    want = layer.decode(x)
    held = torch.zeros_like(x)
    layer.decode(held)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        out = layer.decode(held)
    held.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
