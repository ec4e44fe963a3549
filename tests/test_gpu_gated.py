"""GPU parity of the gated projection and its gradients against plain 64-bit
definitions.

Tolerances, from the arithmetic (u = 2^-24; uo = half a step of the type relative to
its value; A the sum of a product's magnitudes):
  projections  (k + 16) u A.  A sum of k products in f32 in any order is off by k u A at
               most; a tensor-core step adds 16 of them and may truncate (2^-22 of the
               partial sum a step: k / 16 * 2^-22 = k u / 4); a few partial sums are added
  h            1.2 e_g |up| + |act| e_u + 1.2 e_g e_u + 16 u |gate up|, e_g and e_u the
               projections' bounds, 1.2 above every activation's slope (1.13 at most), 16 u
               |gate| above what evaluating the activation in f32 costs
  d_gate       16 u |d_h up| (the slope, below 1.2, in f32) + uo |d_gate|, rounded to the type
  d_up         16 u |d_h gate| + uo |d_up|, rounded to the type
  d_x, d_w     the errors of d_gate and d_up through the products' magnitudes, plus
               (length + 16) u A, the length of the contraction (2 n for d_x, m for d_w)
Each stored result adds uo |value| and the absolute half spacing below the type's normal range.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_moe_expert_gb300 import binding as gb  # noqa: E402
from tests import ffn_ref  # noqa: E402
from tests.gpu_util import DevBuf  # noqa: E402
from tests.test_gpu_moe import TINY, U, UO, empty, fetch, near, strided  # noqa: E402

pytestmark = pytest.mark.gpu

CODE = {name: i for i, name in enumerate(ffn_ref.ACTS)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemv_moe_expert_gb300 import build
    build.build()
    gb.load()
    torch.cuda.init()


def scratch_for(fn, dtype, m, n, k):
    st, need = fn(dtype, m, n, k, False)
    gb.check(st)
    return DevBuf(max(need, 1)), need


class Block:
    """Operands of one block; `pad` elements between rows hold NaN, `off` elements before them."""

    def __init__(self, dtype, m, n, k, seed=0, pad=0, off=0, scale=1.0):
        rng = np.random.default_rng(seed + 31 * m + 7 * n + k)
        self.dtype, self.m, self.n, self.k, self.pad, self.off = dtype, m, n, k, pad, off
        self.ldk, self.ldn = max(k, 1) + pad, max(n, 1) + pad
        w = scale / max(k, 1) ** 0.5
        self.xb, self.xp, self.x = strided(rng.standard_normal((m, k)), self.ldk, dtype, offset=off)
        self.gb, self.gp, self.wg = strided(w * rng.standard_normal((n, k)), self.ldk, dtype, offset=off)
        self.ub, self.up, self.wu = strided(w * rng.standard_normal((n, k)), self.ldk, dtype, offset=off)
        self.rng = rng

    def forward(self, act, save=False, scratch=True, stream=None):
        m, n, k = self.m, self.n, self.k
        outs = [empty(m, self.ldn, self.dtype, self.off) for _ in range(3 if save else 1)]
        sb, need = scratch_for(gb.gbmm_gated_scratch_bytes, self.dtype, m, n, k) if scratch else (None, 0)
        ptr = [o[1] for o in outs] + [None] * (3 - len(outs))
        gb.check(gb.gbmm_gated(self.dtype, CODE[act], m, n, k, self.xp, self.ldk, self.gp, self.up, self.ldk, ptr[0],
                               self.ldn, ptr[1], ptr[2], self.ldn, sb and sb.ptr, need, stream))
        got = [fetch(o[0], m, n, self.ldn, self.dtype, self.off) for o in outs]
        assert sb is None or sb.guards_intact()
        assert gb.gbmm_device_error()[0] == gb.GBMM_OK
        return got

    def check_forward(self, act, got):
        h, g, u = ffn_ref.forward(act, self.x, self.wg, self.wu)
        e = (self.k + 16) * U
        eg, eu = (e * np.abs(self.x) @ np.abs(w).T for w in (self.wg, self.wu))
        uo, tiny = UO[self.dtype], TINY[self.dtype]
        tol = 1.2 * eg * np.abs(u) + np.abs(ffn_ref.act(act, g)) * eu + 1.2 * eg * eu + 16 * U * np.abs(g * u)
        near(got[0], h, tol * (1 + uo) + uo * np.abs(h) + tiny, "h")
        if len(got) > 1:
            near(got[1], g, eg * (1 + uo) + uo * np.abs(g) + tiny, "gate")
            near(got[2], u, eu * (1 + uo) + uo * np.abs(u) + tiny, "up")

    def backward(self, act, d_x=True, d_w=True):
        m, n, k, dt = self.m, self.n, self.k, self.dtype
        self.saved = [strided(self.rng.standard_normal((m, n)), self.ldn, dt, offset=self.off) for _ in range(3)]
        (_, gp, self.g), (_, up, self.u), (_, hp, self.d_h) = self.saved
        dx = empty(m, self.ldk, dt, self.off) if d_x else (None, None)
        dg, du = (empty(n, self.ldk, dt, self.off) if d_w else (None, None) for _ in range(2))
        sb, need = scratch_for(gb.gbmm_gated_backward_scratch_bytes, dt, m, n, k)
        gb.check(gb.gbmm_gated_backward(dt, CODE[act], m, n, k, self.xp if d_w else None, self.ldk,
                                        self.gp if d_x else None, self.up if d_x else None, self.ldk, gp, up, self.ldn,
                                        hp, self.ldn, dx[1], self.ldk, dg[1], du[1], self.ldk, sb.ptr, need))
        got = [o[0] and fetch(o[0], rows, k, self.ldk, dt, self.off) for o, rows in ((dx, m), (dg, n), (du, n))]
        assert sb.guards_intact() and gb.gbmm_device_error()[0] == gb.GBMM_OK
        return got

    def check_backward(self, act, got):
        dt = self.dtype
        uo, tiny = UO[dt], TINY[dt]
        dx, dwg, dwu, dg, du = ffn_ref.backward(act, self.x, self.wg, self.wu, self.g, self.u, self.d_h)
        eg = 16 * U * np.abs(self.d_h * self.u) * (1 + uo) + uo * np.abs(dg) + tiny
        eu = 16 * U * np.abs(self.d_h * self.g) * (1 + uo) + uo * np.abs(du) + tiny
        ag, au = np.abs(dg) + eg, np.abs(du) + eu  # what is multiplied is at most this
        wg, wu, x = np.abs(self.wg), np.abs(self.wu), np.abs(self.x)
        if got[0] is not None:
            tol = eg @ wg + eu @ wu + (2 * self.n + 16) * U * (ag @ wg + au @ wu)
            near(got[0], dx, tol * (1 + uo) + uo * np.abs(dx) + tiny, "d_x")
        for name, out, ref, e, a in (("d_w_gate", got[1], dwg, eg, ag), ("d_w_up", got[2], dwu, eu, au)):
            if out is not None:
                tol = e.T @ x + (self.m + 16) * U * (a.T @ x)
                near(out, ref, tol * (1 + uo) + uo * np.abs(ref) + tiny, name)


SIZES = [(1, 1, 1), (1, 5, 8), (1, 64, 512), (1, 131, 4097), (2, 33, 130), (3, 128, 1024), (5, 7, 200), (7, 257, 264),
         (8, 40, 40), (9, 65, 33), (15, 300, 512), (16, 128, 64), (17, 129, 72), (33, 200, 640), (64, 256, 128),
         (65, 130, 1000), (100, 64, 2056), (128, 300, 256), (129, 127, 65), (147, 513, 520), (260, 264, 192)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_forward_sizes(dtype, m, n, k):
    act = ffn_ref.ACTS[(m + n + k) % 4]
    b = Block(dtype, m, n, k)
    b.check_forward(act, b.forward(act, save=(m + n) % 2 == 0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [1, 12, 80, 300])
@pytest.mark.parametrize("pad,off", [(0, 1), (3, 0), (8, 0), (8, 8), (4, 4)])
def test_forward_layouts(dtype, m, pad, off):
    b = Block(dtype, m, 136, 328, pad=pad, off=off)
    b.check_forward("silu", b.forward("silu", save=True))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,pad", [(30, 133, 261, 3), (300, 133, 261, 3), (300, 1030, 1030, 2), (600, 1025, 513, 7)])
def test_columns_that_end_inside_16_bytes_of_aligned_rows(dtype, m, n, k, pad):
    """What lies behind the last column of each row of every output stays as it was."""
    b = Block(dtype, m, n, k, pad=pad)
    b.check_forward("silu", b.forward("silu", save=True))
    b.check_backward("gelu", b.backward("gelu"))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,pad,off", [(2, 4100, 8200, 0, 0), (5, 4096, 2104, 0, 0), (5, 4100, 2104, 8, 8),
                                           (8, 4099, 1801, 3, 1), (4, 4099, 4097, 0, 0), (3, 300, 40000, 0, 0)])
def test_forward_few_rows_of_large_weights(dtype, m, n, k, pad, off):
    """Weights for which few rows go to the tensor cores, and rows that are laid out again for them."""
    b = Block(dtype, m, n, k, pad=pad, off=off)
    b.check_forward("silu", b.forward("silu", save=True))
    if pad or k % 8:
        b.check_forward("silu", b.forward("silu", scratch=False))


@pytest.mark.parametrize("m", [12, 300])
def test_forward_rows_that_start_anywhere_without_scratch(m):
    b = Block("bf16", m, 70, 130, pad=1, off=1)
    b.check_forward("gelu", b.forward("gelu", save=True, scratch=False))


@pytest.mark.parametrize("act", ffn_ref.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [3, 40, 300])
def test_forward_activations_over_their_range(act, dtype, m):
    b = Block(dtype, m, 72, 64, scale=12.0)  # gates of both signs up to about 50
    b.check_forward(act, b.forward(act, save=True))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(512, 2000, 576), (1000, 1300, 1032), (700, 5504, 64), (2049, 264, 520)])
def test_forward_many_tiles(dtype, m, n, k):
    b = Block(dtype, m, n, k)
    b.check_forward("gelu_tanh", b.forward("gelu_tanh", save=True))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("m", [1, 20, 300])
def test_forward_of_nothing_writes_zeros(dtype, m):
    b = Block(dtype, m, 40, 0)
    for out in b.forward("silu", save=True):
        assert (out == 0).all()


@pytest.mark.parametrize("m", [1, 30, 200])
def test_forward_carries_nan_and_infinity(m):
    """A NaN in one row of x reaches that row of h and no other; so does an infinite gate."""
    n, k = 40, 128
    x, w = torch.ones(m, k, device="cuda").bfloat16(), torch.full((n, k), 0.125, device="cuda").bfloat16()
    x[m // 2, 5] = float("nan")
    h = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
    for act in range(4):
        gb.check(gb.gbmm_gated("bf16", act, m, n, k, x, k, w, w, k, h, n, None, None, 0, None, 0))
        bad = torch.isnan(h).all(dim=1)
        assert bad[m // 2] and bad.sum() == 1 and not torch.isnan(h[~bad]).any()
    x.fill_(1.0)
    x[m // 2, 5] = float("inf")
    gb.check(gb.gbmm_gated("bf16", 0, m, n, k, x, k, w, w, k, h, n, None, None, 0, None, 0))
    assert torch.isinf(h[m // 2]).all() and torch.isinf(h).sum() == n


@pytest.mark.parametrize("m", [6, 40, 300])
def test_projections_side_by_side(m):
    """w_gate and w_up as the halves of one [2 n, k] matrix, gate and up as those of one [m, 2 n]."""
    n, k = 264, 320
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, k, generator=g, device="cuda").half()
    w = (torch.randn(2 * n, k, generator=g, device="cuda") / k ** 0.5).half()
    both, h = torch.empty(m, 2 * n, device="cuda").half(), torch.empty(m, n, device="cuda").half()
    apart, h2 = [torch.empty(m, n, device="cuda").half() for _ in range(2)], torch.empty_like(h)
    gb.check(gb.gbmm_gated("f16", 0, m, n, k, x, k, w, w[n:], k, h, n, both, both[:, n:], 2 * n, None, 0))
    gb.check(gb.gbmm_gated("f16", 0, m, n, k, x, k, w, w[n:].clone(), k, h2, n, *apart, n, None, 0))
    assert torch.equal(h, h2) and torch.equal(both, torch.cat(apart, dim=1))


@pytest.mark.parametrize("m", [2, 20, 200])
def test_offsets_past_32_bits(m):
    """Weights and gradients with rows 2^30 elements apart (both weights side by side), outputs 2^24 apart."""
    n, k, ldw, ldh = 6, 72, 1 << 30, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w = torch.randn(m, k, generator=g, device="cuda").half(), torch.randn(n, 2 * k, generator=g, device="cuda").half()
    wide = torch.empty((n - 1) * ldw + 2 * k, dtype=torch.float16, device="cuda").as_strided((n, 2 * k), (ldw, 1))
    wide.copy_(w)
    outs = torch.empty((m - 1) * ldh + 3 * n, dtype=torch.float16, device="cuda").as_strided((m, 3 * n), (ldh, 1))
    gb.check(gb.gbmm_gated("f16", 0, m, n, k, x, k, wide, wide[:, k:], ldw, outs, ldh, outs[:, n:], outs[:, 2 * n:], ldh,
                           None, 0))
    tight = torch.empty(3, m, n, device="cuda").half()
    halves = [w[:, :k].contiguous(), w[:, k:].contiguous()]
    gb.check(gb.gbmm_gated("f16", 0, m, n, k, x, k, *halves, k, tight[0], n, tight[1], tight[2], n, None, 0))
    assert torch.equal(outs.reshape(m, 3, n).transpose(0, 1), tight)
    d_h = torch.randn(m, n, generator=g, device="cuda").half()
    need = gb.gbmm_gated_backward_scratch_bytes("f16", m, n, k, False)[1]
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    dw = torch.empty((n - 1) * ldw + 2 * k, dtype=torch.float16, device="cuda").as_strided((n, 2 * k), (ldw, 1))
    dx, dx2, dw2 = torch.empty_like(x), torch.empty_like(x), torch.empty(2, n, k, device="cuda").half()
    gb.check(gb.gbmm_gated_backward("f16", 0, m, n, k, x, k, wide, wide[:, k:], ldw, tight[1], tight[2], n, d_h, n, dx, k,
                                    dw, dw[:, k:], ldw, scratch, need))
    gb.check(gb.gbmm_gated_backward("f16", 0, m, n, k, x, k, *halves, k, tight[1], tight[2], n, d_h, n, dx2, k, dw2[0],
                                    dw2[1], k, scratch, need))
    assert torch.equal(dx, dx2) and torch.equal(dw[:, :k], dw2[0]) and torch.equal(dw[:, k:], dw2[1])


BACK_SIZES = [(1, 1, 1), (1, 64, 128), (3, 5, 7), (7, 40, 264), (16, 64, 64), (33, 129, 65), (64, 128, 256),
              (100, 72, 520), (147, 257, 129), (128, 512, 1000), (300, 264, 328)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", BACK_SIZES)
def test_backward_sizes(dtype, m, n, k):
    act = ffn_ref.ACTS[(m + n + k) % 4]
    b = Block(dtype, m, n, k)
    b.check_backward(act, b.backward(act))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,off", [(0, 1), (3, 0), (8, 0), (8, 8), (4, 4)])
def test_backward_layouts(dtype, pad, off):
    b = Block(dtype, 90, 136, 200, pad=pad, off=off)
    b.check_backward("silu", b.backward("silu"))


@pytest.mark.parametrize("act", ffn_ref.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_backward_activations(act, dtype):
    b = Block(dtype, 40, 48, 56)
    b.check_backward(act, b.backward(act))


@pytest.mark.parametrize("d_x,d_w", [(True, False), (False, True)])
def test_backward_of_one_side(d_x, d_w):
    b = Block("bf16", 70, 96, 104)
    got = b.backward("gelu", d_x, d_w)
    assert (got[0] is None) != d_x and (got[1] is None) != d_w
    b.check_backward("gelu", got)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1100, 1000, 840), (512, 2056, 1032), (2500, 520, 264)])
def test_backward_many_tiles(dtype, m, n, k):
    b = Block(dtype, m, n, k)
    b.check_backward("silu", b.backward("silu"))


@pytest.mark.parametrize("d_w", [True, False])
@pytest.mark.parametrize("m,n,k,pad", [(1, 1290, 72, 0), (16, 1300, 264, 3), (20, 1285, 128, 3), (64, 1290, 70, 2),
                                       (70, 3205, 133, 3), (130, 3300, 136, 0), (300, 3208, 640, 8)])
def test_backward_over_many_rows_of_weights(m, n, k, pad, d_w):
    """Few tokens and columns, a long contraction for d_x."""
    b = Block("bf16" if m % 4 else "f16", m, n, k, pad=pad)
    b.check_backward("gelu", b.backward("gelu", True, d_w))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,pad,off", [(1, 1, 1, 0, 0), (1, 200, 200, 0, 0), (2, 128, 1032, 3, 0), (3, 33, 255, 0, 1),
                                           (4, 95, 264, 8, 8), (4, 700, 512, 0, 0), (3, 1025, 2049, 0, 0),
                                           (4, 65, 257, 4, 4)])
def test_weights_gradients_of_few_tokens_round_once(dtype, m, n, k, pad, off):
    """Up to four tokens: d_gate and d_up enter the weights' gradients in f32, off by 16 u |d_h up| and 16 u |d_h gate|."""
    b = Block(dtype, m, n, k, pad=pad, off=off)
    for d_x in (True, False):
        got = b.backward("silu", d_x, True)
        b.check_backward("silu", got)
        _, dwg, dwu, dg, du = ffn_ref.backward("silu", b.x, b.wg, b.wu, b.g, b.u, b.d_h)
        x = np.abs(b.x)
        for out, ref, d, other in ((got[1], dwg, dg, b.u), (got[2], dwu, du, b.g)):
            e = 16 * U * np.abs(b.d_h * other)
            tol = e.T @ x + (m + 16) * U * ((np.abs(d) + e).T @ x)
            near(out, ref, tol * (1 + UO[dtype]) + UO[dtype] * np.abs(ref) + TINY[dtype], "d_w")


@pytest.mark.parametrize("d_x,d_w", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("m,n,k", [(2570, 300, 2100), (520, 2600, 1300), (1300, 1290, 1290)])
def test_backward_tiles_of_both_products(m, n, k, d_x, d_w):
    """More tiles than pairs of CTAs, and rounds that end between."""
    b = Block("bf16", m, n, k)
    b.check_backward("relu", b.backward("relu", d_x, d_w))


# A product just under half a step of f32 beyond 1: added one after the other, every one that is added to 8192 or more
# is rounded down, and 16384 of them end 2e-4 too low.
LOST = float(np.float32(1 + 2.0 ** -11 - 2.0 ** -22))


@pytest.mark.parametrize("m", [1, 20, 70, 300])
def test_long_sums_in_f32(m):
    """A projection's sum is made of runs of at most 512 products, and of at most k / 512 + 16 sums of runs:
    (512 + k / 512 + 16) u of the magnitudes, 4e-5 at k = 32768 and not 2e-3."""
    n, k = 70, 32768
    x, w = torch.full((m, k), LOST, device="cuda"), torch.ones(n, k, device="cuda")
    st, need = gb.gbmm_gated_scratch_bytes("f32", m, n, k, False)
    gb.check(st)
    scratch, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(3, m, n, device="cuda")
    gb.check(gb.gbmm_gated("f32", CODE["relu"], m, n, k, x, k, w, w, k, out[0], n, out[1], out[2], n, scratch, need))
    r = (512 + k / 512 + 16) * U
    assert (out[1:].double() / (k * LOST) - 1).abs().max() <= r
    assert (out[0].double() / (k * LOST) ** 2 - 1).abs().max() <= 2 * r + r * r + 16 * U


@pytest.mark.parametrize("d_x,d_w", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("m,n,k", [(16384, 40, 72), (16384, 300, 1100), (40, 16384, 72), (300, 16384, 1100)])
def test_long_sums_of_gradients_in_f32(m, n, k, d_x, d_w):
    """As above, over 2 n products for x and over m for the weights."""
    x, w = torch.ones(m, k, device="cuda"), torch.ones(n, k, device="cuda")
    one, d_h = torch.ones(m, n, device="cuda"), torch.full((m, n), LOST, device="cuda")
    dx, dw = torch.empty(m, k, device="cuda"), torch.empty(2, n, k, device="cuda")
    st, need = gb.gbmm_gated_backward_scratch_bytes("f32", m, n, k, True)
    gb.check(st)
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    gb.check(gb.gbmm_gated_backward("f32", CODE["relu"], m, n, k, x if d_w else None, k, w if d_x else None,
                                    w if d_x else None, k, one, one, n, d_h, n, dx if d_x else None, k,
                                    dw[0] if d_w else None, dw[1] if d_w else None, k, scratch, need))
    for on, out, length in ((d_x, dx, 2 * n), (d_w, dw, m)):
        if on:
            assert (out.double() / (length * LOST) - 1).abs().max() <= (512 + length / 512 + 16) * U


@pytest.mark.parametrize("d_x,d_w", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("m,n,k,pad", [(21, 640, 64, 8), (1000, 64, 70, 1), (1300, 128, 256, 0), (16, 1409, 513, 0),
                                       (256, 512, 512, 0), (3, 1500, 100, 3), (1, 1, 300, 0)])
def test_backward_of_few_tiles_in_f32(m, n, k, pad, d_x, d_w):
    """Contractions divided over clusters: of one product, of both, of neither."""
    b = Block("f32", m, n, k, pad=pad)
    b.check_backward("silu", b.backward("silu", d_x, d_w))


def test_backward_of_nothing_writes_zeros():
    t = torch.full((3, 8, 16), 7.0, device="cuda")
    gb.check(gb.gbmm_gated_backward("f32", 0, 0, 8, 16, None, 16, t, t, 16, None, None, 8, None, 8, None, 16, t[0],
                                    t[1], 16, None, 0))
    assert (t[:2] == 0).all() and (t[2] == 7).all()
    t.fill_(7.0)
    gb.check(gb.gbmm_gated_backward("f32", 0, 8, 0, 16, None, 16, None, None, 16, None, None, 0, None, 0, t[0], 16,
                                    None, None, 16, None, 0))
    assert (t[0] == 0).all() and (t[1:] == 7).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradient_against_differences(act):
    """<gradient, v> against central differences of the definition in 64 bits along v, through forward and
    backward calls in f32.  The differences are off by 1e-10 of the sum of magnitudes at a step of 1e-5 (its square
    times a third derivative of order 1, and 2^-53 / 1e-5); the f32 gradients and saved projections by less
    than (2 n + m + k + 100) 2^-24 of the magnitudes."""
    m, n, k = 12, 24, 40
    b = Block("f32", m, n, k, seed=5)
    _, gate, up = b.forward(act, save=True)
    d_h = b.rng.standard_normal((m, n)).astype(np.float32).astype(np.float64)

    def up_(v):
        return torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda()
    x, wg, wu, g, u, dh = (up_(v) for v in (b.x, b.wg, b.wu, gate, up, d_h))
    out = [torch.empty_like(v) for v in (x, wg, wu)]
    st, need = gb.gbmm_gated_backward_scratch_bytes("f32", m, n, k, True)
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    gb.check(gb.gbmm_gated_backward("f32", CODE[act], m, n, k, x, k, wg, wu, k, g, u, n, dh, n, out[0], k, out[1],
                                    out[2], k, scratch, need))
    torch.cuda.synchronize()
    grads, at, eps = [o.double().cpu().numpy() for o in out], (b.x, b.wg, b.wu), 1e-5
    for i in range(3):
        v = b.rng.standard_normal(at[i].shape)
        far = [(d_h * ffn_ref.forward(act, *[a + (s * eps * v if j == i else 0) for j, a in enumerate(at)])[0]).sum()
               for s in (1, -1)]
        got, ref = (grads[i] * v).sum(), (far[0] - far[1]) / (2 * eps)
        # magnitudes of what the gradient's entry sums
        mag = np.abs(v) * (np.abs(d_h * up) @ np.abs(b.wg) + np.abs(d_h * gate) @ np.abs(b.wu)) if i == 0 else \
            np.abs(v) * (1.2 * np.abs(d_h * (up if i == 1 else gate)).T @ np.abs(b.x))
        assert abs(got - ref) <= (2 * n + m + k + 100) * U * 1.2 * mag.sum() + 1e-9 * mag.sum(), (i, got, ref)


@pytest.mark.parametrize("order", [("dwg", "dwu", "x", "scratch"), ("dwu", "dwg", "scratch", "x"),
                                   ("dwg", "scratch", "dwu", "x"), ("dwu", "x", "dwg", "scratch"), "rows"])
def test_backward_wherever_the_gradients_lie(order):
    """Both weights' gradients next to each other, in either order, with an operand between them, and row by row."""
    m, n, k = 80, 136, 200
    b = Block("bf16", m, n, k)
    ref = b.backward("silu")
    need = gb.gbmm_gated_backward_scratch_bytes("bf16", m, n, k, True)[1]
    size = {"dwg": n * k * 2, "dwu": n * k * 2, "x": m * k * 2, "scratch": need}
    size = {name: -(-v // 256) * 256 for name, v in size.items()}
    buf = torch.full((sum(size.values()) + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    base = -(-buf.data_ptr() // 256) * 256
    at, ld = {}, k
    for name in order if order != "rows" else ("x", "scratch", "dwg", "dwu"):
        at[name] = base + sum(size[v] for v in at)
    if order == "rows":
        at["dwu"], ld = at["dwg"] + k * 2, 2 * k
    off = at["x"] - buf.data_ptr()
    buf[off:off + m * k * 2].copy_(torch.from_numpy(b.x.astype(np.float32)).bfloat16().cuda().reshape(-1).view(torch.uint8))
    gb.check(gb.gbmm_gated_backward("bf16", CODE["silu"], m, n, k, at["x"], k, b.gp, b.up, b.ldk, b.saved[0][1],
                                    b.saved[1][1], b.ldn, b.saved[2][1], b.ldn, None, k, at["dwg"], at["dwu"], ld,
                                    at["scratch"], need))
    torch.cuda.synchronize()
    for name, want in (("dwg", ref[1]), ("dwu", ref[2])):
        off = at[name] - buf.data_ptr()
        got = buf[off:off + ((n - 1) * ld + k) * 2].view(torch.bfloat16)
        got = got.as_strided((n, k), (ld, 1)).double().cpu().numpy()
        assert np.array_equal(got, want), name


def make(dtype, m, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    t = {"x": new(m, k), "wg": new(n, k) / k ** 0.5, "wu": new(n, k) / k ** 0.5, "dh": new(m, n)}
    t |= {name: torch.zeros(m, n, dtype=dt, device="cuda") for name in ("h", "gate", "up")}
    t |= {"dx": torch.zeros_like(t["x"]), "dwg": torch.zeros_like(t["wg"]), "dwu": torch.zeros_like(t["wu"])}
    t["need"] = max(fn(dtype, m, n, k, False)[1] for fn in (gb.gbmm_gated_scratch_bytes, gb.gbmm_gated_backward_scratch_bytes))
    t["scratch"] = torch.empty(t["need"] + 1, dtype=torch.uint8, device="cuda")
    return t


def step(dtype, m, n, k, t, stream=None):
    """Forward and backward as a training step makes them, one workspace for both."""
    gb.check(gb.gbmm_gated(dtype, 0, m, n, k, t["x"], k, t["wg"], t["wu"], k, t["h"], n, t["gate"], t["up"], n,
                           t["scratch"], t["need"], stream))
    gb.check(gb.gbmm_gated_backward(dtype, 0, m, n, k, t["x"], k, t["wg"], t["wu"], k, t["gate"], t["up"], n, t["dh"],
                                    n, t["dx"], k, t["dwg"], t["dwu"], k, t["scratch"], t["need"], stream))
    return [t[name].clone() for name in ("h", "gate", "up", "dx", "dwg", "dwu")]


STEPS = [("f32", 20, 72, 136), ("f16", 12, 264, 520), ("bf16", 100, 200, 320), ("bf16", 600, 1032, 520),
         ("f16", 130, 77, 33), ("f16", 3, 264, 520), ("bf16", 40, 1400, 264), ("f16", 7, 3001, 133),
         ("f32", 2000, 72, 136), ("f32", 90, 1300, 500)]


@pytest.mark.parametrize("dtype,m,n,k", STEPS)
def test_steps_do_not_change_from_call_to_call(dtype, m, n, k):
    t = make(dtype, m, n, k, 3)
    first = step(dtype, m, n, k, t)
    for _ in range(3):
        t["scratch"].fill_(255)
        assert all(torch.equal(a, b) for a, b in zip(first, step(dtype, m, n, k, t)))


@pytest.mark.parametrize("dtype,m,n,k", STEPS)
def test_steps_replay_from_a_graph(dtype, m, n, k):
    t, other = make(dtype, m, n, k, 4), make(dtype, m, n, k, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(dtype, m, n, k, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step(dtype, m, n, k, t)
    want = step(dtype, m, n, k, other)
    for name in ("x", "wg", "wu", "dh"):
        t[name].copy_(other[name])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_two_streams_at_once():
    cases = [("bf16", 600, 1032, 520), ("f16", 12, 264, 520), ("bf16", 40, 1400, 264), ("f32", 2000, 72, 136)]
    sets = [make(*c, seed) for seed, c in enumerate(cases)]
    want = [step(*c, t) for c, t in zip(cases, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        got = []
        for c, t, s in zip(cases, sets, streams):
            with torch.cuda.stream(s):
                got.append(step(*c, t, s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(300, 264, 328), (2049, 2003, 64), (1000, 4101, 136)])
@pytest.mark.parametrize("pad_h,pad_saved", [(0, 1), (1, 0), (0, 0)])
def test_outputs_whose_rows_tma_can_and_cannot_write(dtype, m, n, k, pad_h, pad_saved):
    """h or the saved projections in rows on multiples of 16 bytes and the others not, and last columns that end inside
    16 bytes of aligned rows: pieces that leave by TMA and by plain stores alternate.  The same values whatever the rows."""
    b = Block(dtype, m, n, k)
    outs = {}
    for ld_h, ld_saved in ((n | 1, n | 1), (-(-n // 8) * 8 + pad_h, -(-n // 8) * 8 + pad_saved)):
        for turn in range(4):
            bufs = [empty(m, ld, dtype, 0) for ld in (ld_h, ld_saved, ld_saved)]
            gb.check(gb.gbmm_gated(dtype, CODE["silu"], m, n, k, b.xp, b.ldk, b.gp, b.up, b.ldk, bufs[0][1], ld_h,
                                   bufs[1][1], bufs[2][1], ld_saved, None, 0))
            got = [fetch(o[0], m, n, ld, dtype, 0) for o, ld in zip(bufs, (ld_h, ld_saved, ld_saved))]
            if not outs:
                b.check_forward("silu", got)
                outs["first"] = got
            assert all(np.array_equal(a, c) for a, c in zip(outs["first"], got))
    assert gb.gbmm_device_error()[0] == gb.GBMM_OK


F32_PLANS = [(26, 9664, 64), (2346, 892, 300), (3000, 64, 1400), (1000, 1100, 515), (132, 3000, 420), (2444, 192, 1100),
             (6605, 70, 200), (700, 1546, 1200), (5, 700, 5003)]


@pytest.mark.parametrize("m,n,k", F32_PLANS)
@pytest.mark.parametrize("d_x,d_w,pad", [(True, True, 0), (True, True, 3), (True, False, 0), (False, True, 0)])
def test_f32_gradients_however_they_are_divided(m, n, k, d_x, d_w, pad):
    b = Block("f32", m, n, k, pad=pad)
    b.check_backward("silu", b.backward("silu", d_x, d_w))


def test_f32_gradients_are_divided_in_different_ways():
    plans = {gb.gbmm_test_gradient_plan(*s, True, True, torch.cuda.get_device_properties(0).multi_processor_count)[1]
             for s in F32_PLANS}
    assert len({p[0] for p in plans}) == 2 and len({p[1] for p in plans}) > 2 and len({p[2] for p in plans}) > 2
    assert len({p[3] for p in plans}) == 2


F32_TILES = [(10, 2795, 512), (44, 3169, 300), (707, 216, 656), (512, 1408, 2048), (512, 2816, 1024), (6469, 131, 61),
             (454, 145, 25), (12, 40, 5000), (1300, 1668, 259)]


@pytest.mark.parametrize("m,n,k", F32_TILES)
@pytest.mark.parametrize("pad", [0, 3])
def test_f32_projections_however_they_are_divided(m, n, k, pad):
    b = Block("f32", m, n, k, pad=pad)
    b.check_forward("gelu", b.forward("gelu", save=True))


def test_f32_projections_are_divided_in_different_ways():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plans = {gb.gbmm_test_gated_plan(*s, sms)[1] for s in F32_TILES}
    assert {p[0] for p in plans} == {64, 128} and len({p[1] for p in plans}) > 3


def exact_gates(dtype, act):
    """Gates of the type's own values over the range in which the activation's far ends are normal numbers in f32."""
    most = {"gelu_tanh": 9.0, "relu": 100.0}.get(act, 12.0)
    v = np.concatenate([np.linspace(-most, most, 997), np.linspace(-1, 1, 203)])
    return strided(v[None, :], v.size, dtype)[2][0]


def activation_bound(act, v):
    """What evaluating the activation may be off by, relative to v times its sigmoid (or normal distribution): 2^-18, and
    the rounding of the exponent in front of the exponential, four steps of its own size (gelu v^2 / 2; silu v; the tanh
    form its argument)."""
    exponent = {"gelu": v * v / 2, "silu": np.abs(v), "gelu_tanh": 2 * ffn_ref.C * np.abs(v + 0.044715 * v ** 3),
                "relu": 0 * v}[act]
    return 2.0 ** -18 + 8 * U * exponent


@pytest.mark.parametrize("act", ffn_ref.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,pad", [(3, 0), (40, 0), (300, 0), (300, 1)])
def test_far_ends_of_activations(m, pad, dtype, act):
    """Rows of x pick single columns of w_gate, and w_up is 1, so that h is the activation of exact gates: off by half a
    step and activation_bound() relative to h itself, whichever way the number of rows takes."""
    v = exact_gates(dtype, act)
    n, k = v.size // 8, 8
    b = Block(dtype, m, n, k, pad=pad)
    x = np.zeros((m, k))
    x[np.arange(m), np.arange(m) % k] = 1
    xb, xp, _ = strided(x, b.ldk, dtype, fill=0.0)
    gate = v.reshape(k, n)
    gb_, gp, _ = strided(gate.T, b.ldk, dtype, fill=0.0)
    ub, up, _ = strided(np.ones((n, k)), b.ldk, dtype, fill=0.0)
    h = empty(m, n, dtype, 0)
    sb, need = scratch_for(gb.gbmm_gated_scratch_bytes, dtype, m, n, k)
    gb.check(gb.gbmm_gated(dtype, CODE[act], m, n, k, xp, b.ldk, gp, up, b.ldk, h[1], n, None, None, 0, sb.ptr, need))
    g = gate[np.arange(m) % k]
    want = ffn_ref.act(act, g) if act != "gelu" else 0.5 * g * ffn_ref.erfc(-g / 2 ** 0.5)
    if act == "gelu_tanh":
        want = g * ffn_ref._sigmoid(2 * ffn_ref.C * (g + 0.044715 * g ** 3))
    tol = np.abs(want) * (UO[dtype] + activation_bound(act, g) * (1 + UO[dtype])) + TINY[dtype]
    near(fetch(h[0], m, n, n, dtype, 0), want, tol, "h")


@pytest.mark.parametrize("act", ffn_ref.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [4, 40, 300])
def test_far_ends_of_slopes(m, dtype, act):
    """d_h and up of 1 and rows of x that pick single columns: the weights' gradients are the slopes and the activations
    of exact gates, rounded to the type (twice above four rows: once more where they are stored)."""
    v = exact_gates(dtype, act)
    n, k = v.size // 4, 4
    gate = np.zeros((m, n))
    gate[:4] = v[:4 * n].reshape(4, n)
    x = np.zeros((m, k))
    x[np.arange(4), np.arange(4)] = 1
    (xb, xp, _), (sb_, sp, _) = strided(x, k, dtype), strided(gate, n, dtype)
    (ub, up, _), (hb, hp, _) = (strided(np.ones((m, n)), n, dtype) for _ in range(2))
    dg, du = empty(n, k, dtype, 0), empty(n, k, dtype, 0)
    sb, need = scratch_for(gb.gbmm_gated_backward_scratch_bytes, dtype, m, n, k)
    gb.check(gb.gbmm_gated_backward(dtype, CODE[act], m, n, k, xp, k, None, None, k, sp, up, n, hp, n, None, k, dg[1],
                                    du[1], k, sb.ptr, need))
    g = gate[:4]
    bound = activation_bound(act, g)
    if act == "gelu":
        share, far, lever = 0.5 * ffn_ref.erfc(-g / 2 ** 0.5), g * np.exp(-0.5 * g * g) / (2 * np.pi) ** 0.5, g
    elif act == "relu":
        share, far, lever = (g > 0).astype(float), 0 * g, g
    else:
        a = g if act == "silu" else 2 * ffn_ref.C * (g + 0.044715 * g ** 3)
        share = ffn_ref._sigmoid(a)
        lever = g if act == "silu" else 2 * ffn_ref.C * (g + 3 * 0.044715 * g ** 3)
        far = share * ffn_ref._sigmoid(-a) * lever
    for out, want, size in ((dg, share + far, np.abs(share) + np.abs(far)), (du, g * share, np.abs(g * share))):
        # 1 - sigmoid is off by a step of the sigmoid, times what it is multiplied with in the slope
        tol = 2 * UO[dtype] * np.abs(want) + bound * size + 4 * U * np.abs(lever) * share + 2 * TINY[dtype]
        near(fetch(out[0], n, k, k, dtype, 0).T, want, tol, "slope")


def test_weights_gradients_of_268_million_tokens():
    """One tile whose contraction takes longer than any single wait may: every 2^20th row and the last hold ones, which
    the gradients count."""
    m, n = 1 << 28, 8
    rows = torch.zeros(m, n, dtype=torch.float16, device="cuda")
    rows[7::1 << 20] = 1
    rows[-1] = 1
    st, need = gb.gbmm_gated_backward_scratch_bytes("f16", m, n, n, True)
    gb.check(st)
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    d_w = torch.empty(2, n, n, dtype=torch.float16, device="cuda")
    gb.check(gb.gbmm_gated_backward("f16", gb.GATE_RELU, m, n, n, rows, n, None, None, n, rows, rows, n, rows, n, None, n,
                                    d_w[0], d_w[1], n, scratch, need))
    assert gb.gbmm_device_error()[0] == gb.GBMM_OK
    assert (d_w == m // (1 << 20) + 1).all()
    del rows, scratch
    torch.cuda.empty_cache()
