"""The example block (examples/feed_forward.py) against a 64-bit block: the gated projection, the
products with the down projection, their gradients, and the 8-bit form.

Bounds, on norms.  f32: each value passes through at most four sums of at most K = 512 products; a sum is off by
at most K u of the sum of magnitudes, which for random signs is sqrt(K) times the result: 4 * 512 * 23 * 2^-24
< 3e-3.  16 bits: at most eight stored values lie between the inputs and any result (2^-9 each for bf16): 2^-6.
8 bits: each factor is off by at most half a code, 1/254 of its row's largest value.  A row of K normal values
has a largest one below 4.5 times their root mean square (K <= 512, all seeds here), a row of h one below
16 times (products of two such values), and an error that is uniform over a code has 1 / sqrt(3) of its bound as
its root mean square; errors of independent signs add in squares: x and w_in give 4.5 / 254 / sqrt(3) = 1.03 %
each, both times sqrt(2) into h (two projections), h and w_out 3.7 % and 1 %: below 5 % together.
"""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

pytestmark = pytest.mark.gpu

BOUND = {torch.float32: 3e-3, torch.bfloat16: 2.0 ** -6, torch.float16: 2.0 ** -6}


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemv_moe_expert_gb300 import build
    build.build()
    from examples import feed_forward
    return feed_forward


def close(got, ref, bound, what):
    off = (got.double() - ref).norm() / ref.norm()
    assert off <= bound, (what, off.item())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hidden,inner,m", [(256, 320, 1), (256, 320, 70), (512, 264, 300)])
def test_block(example, dtype, hidden, inner, m):
    block = example.FeedForward(hidden, inner, dtype)
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, hidden, generator=g, device="cuda").to(dtype)
    d_y = torch.randn(m, hidden, generator=g, device="cuda").to(dtype)
    y, kept = block.forward(x)
    grads = block.backward(kept, d_y)
    leaves = [v.double().requires_grad_() for v in (x, block.w_in, block.w_out)]
    both = leaves[0] @ leaves[1].T
    ref = (torch.nn.functional.silu(both[:, :inner]) * both[:, inner:]) @ leaves[2].T
    close(y, ref.detach(), BOUND[dtype], "y")
    for name, got, want in zip(("x", "w_in", "w_out"), grads, torch.autograd.grad(ref, leaves, d_y.double())):
        close(got, want, BOUND[dtype], name)
    close(block.serve(x), ref.detach(), 0.05 + BOUND[dtype], "8 bits")


def test_serve_replays_from_a_graph(example):
    block = example.FeedForward(256, 320)
    x, other = (torch.randn(9, 256, device="cuda").bfloat16() for _ in range(2))
    want = block.serve(other).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.serve(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = block.serve(x)
    x.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_host_threads_at_once(example):
    """Four host threads, a stream each, whose first calls of every kernel of the block meet."""
    import threading
    sizes = [(9, 256, 320), (70, 256, 320), (300, 520, 264), (1, 512, 264)]
    blocks = [example.FeedForward(h, i, torch.float16) for _, h, i in sizes]
    xs = [torch.randn(m, h, device="cuda").half() for m, h, _ in sizes]
    torch.cuda.synchronize()
    gate, got, failed = threading.Barrier(len(sizes)), [None] * len(sizes), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait(30)
                y, kept = blocks[i].forward(xs[i])
                got[i] = (y, *blocks[i].backward(kept, xs[i]), blocks[i].serve(xs[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for block, x, out in zip(blocks, xs, got):
        y, kept = block.forward(x)
        assert all(torch.equal(a, b) for a, b in zip(out, (y, *block.backward(kept, x), block.serve(x))))


def test_example_runs(example, capsys):
    example.main()
    assert "replayed from a graph" in capsys.readouterr().out
