"""GPU parity of the quantisation to 8 bits and of the 8-bit integer product
against plain 64-bit definitions.

Codes and scales have to be equal.  The product's sum is that of integers, exactly;
rounded to f32, multiplied by two scales and stored: off by 2^-24 of the value three
times, and by half a step of the type (4 * 2^-24 covers the terms of second order)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_moe_expert_gb300 import binding as gb  # noqa: E402
from tests import ffn_ref  # noqa: E402
from tests.gpu_util import DevBuf  # noqa: E402
from tests.test_gpu_moe import TINY, U, UO, empty, fetch, floats, near, strided  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemv_moe_expert_gb300 import build
    build.build()
    gb.load()
    torch.cuda.init()


def bytes_of(values, ld, offset=0):
    """A device buffer of [rows, cols] codes with rows ld bytes apart; the gaps hold 77."""
    rows, cols = values.shape
    flat = np.full(offset + max(rows - 1, 0) * ld + cols, 77, np.int8)
    for i in range(rows):
        flat[offset + i * ld:offset + i * ld + cols] = values[i]
    buf = DevBuf(max(flat.size, 1), host=flat)
    return buf, buf.ptr + offset


def quantize(values, dtype, pad=0, off=0, qpad=0, qoff=0):
    m, k = values.shape
    xb, xp, x = strided(values, max(k, 1) + pad, dtype, offset=off)
    ldq = max(k, 1) + qpad
    qb, sb = DevBuf(qoff + m * ldq), DevBuf(4 * m)
    gb.check(gb.gbmm_quantize_i8(dtype, m, k, xp, max(k, 1) + pad, qb.ptr + qoff, ldq, sb.ptr))
    torch.cuda.synchronize()
    raw = qb.read(np.int8)
    at = qoff + np.arange(m)[:, None] * ldq + np.arange(k)[None, :]
    rest = np.ones(raw.size, bool)
    rest[at.reshape(-1)] = False
    assert (raw[rest] == np.int8(0xA5 - 256)).all() and qb.guards_intact() and sb.guards_intact()
    q, scale = ffn_ref.quantize(x)
    got = sb.read(np.float32)
    assert np.array_equal(got, scale, equal_nan=True), (got, scale)
    assert np.array_equal(raw[at], q), (x[raw[at] != q][:4], raw[at][raw[at] != q][:4], q[raw[at] != q][:4])
    return raw[at], got


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 7), (3, 64), (5, 129), (2, 1000), (70, 256), (9, 2048), (4, 4097),
                                 (3, 11008), (2, 40001), (1000, 72)])
def test_quantize_sizes(dtype, m, k):
    rng = np.random.default_rng(m + k)
    quantize(rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1))), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,off,qpad,qoff", [(8, 0, 8, 0), (8, 8, 16, 16), (1, 0, 0, 0), (0, 1, 0, 0), (8, 0, 1, 0),
                                               (8, 0, 0, 3), (8, 0, 4, 4), (5, 3, 7, 1)])
def test_quantize_layouts(dtype, pad, off, qpad, qoff):
    quantize(np.random.default_rng(pad).standard_normal((6, 336)), dtype, pad, off, qpad, qoff)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_middles_of_two_codes(dtype):
    """Values at, just below and just above the middle of two codes, for scales that are and are not exact."""
    rows = []
    for most in (127.0, 254.0, 1.0, 1.5, 100.0, 3.0):
        mid = (np.arange(-127, 127) + 0.5) * most / 127
        eps = 2.0 ** -23 if dtype == "f32" else 2.0 ** -10 if dtype == "f16" else 2.0 ** -7
        rows.append(np.concatenate([[most], mid, mid * (1 + eps), mid * (1 - eps), [most / 2, -most / 2]]))
    quantize(np.array(rows), dtype)


@pytest.mark.parametrize("k", [9, 600, 5000])
def test_quantize_rows_of_zeros_nan_and_infinity(k):
    for dtype in ("f32", "f16", "bf16"):
        x = np.random.default_rng(3).standard_normal((7, k))
        x[1], x[3, k // 2], x[4, 0], x[5, k - 1] = 0, np.nan, np.inf, -np.inf
        q, scale = quantize(x, dtype)
        assert scale[1] == 0 and np.isnan(scale[3:6]).all() and (q[[1, 3, 4, 5]] == 0).all()


def test_quantize_far_magnitudes():
    """From the largest values down to rows whose scale is below f32's normal range, or 0."""
    rng = np.random.default_rng(8)
    x = rng.uniform(-1, 1, (9, 200)) * np.array([3e38, 1e30, 1e-30, 1e-36, 1e-38, 1e-40, 1e-42, 1e-43, 1e-45])[:, None]
    quantize(x, "f32")
    quantize(x[:7], "bf16")


def codes(rng, m, k, low=-127):
    return rng.integers(low, 128, (m, k)).astype(np.int8)


class Product:
    def __init__(self, m, n, k, pad=0, off=0, seed=0, scales=True):
        rng = np.random.default_rng(seed + m + 3 * n + 7 * k)
        self.m, self.n, self.k = m, n, k
        self.a, self.b = codes(rng, m, k, -128), codes(rng, n, k, -128)
        self.ld = max(k, 1) + pad
        (self.ab, self.ap), (self.bb, self.bp) = bytes_of(self.a, self.ld, off), bytes_of(self.b, self.ld, off)
        self.sa = rng.uniform(0.5, 2, m).astype(np.float32) if scales else None
        self.sb = rng.uniform(-0.02, 0.02, n).astype(np.float32) if scales else None
        self.sab, self.sbb = (None if s is None else floats(s) for s in (self.sa, self.sb))

    def run(self, dtype, cpad=0, coff=0):
        m, n, k = self.m, self.n, self.k
        ldc = n + cpad
        cb, cp = empty(m, ldc, dtype, coff)
        st, need = gb.gbmm_gemm_i8_scratch_bytes(m, n, k, False)
        gb.check(st)
        scratch = DevBuf(max(need, 1))
        gb.check(gb.gbmm_gemm_i8(dtype, m, n, k, self.ap, self.ld, self.sab and self.sab.ptr, self.bp, self.ld,
                                 self.sbb and self.sbb.ptr, cp, ldc, scratch.ptr, need))
        got = fetch(cb, m, n, ldc, dtype, coff)
        assert scratch.guards_intact() and gb.gbmm_device_error()[0] == gb.GBMM_OK
        return got

    def check(self, dtype, got):
        # sums below 2^53: exact in f64 whatever the order
        ref = self.a.astype(np.float64) @ self.b.astype(np.float64).T
        if self.sa is not None:
            ref = ref * self.sa.astype(np.float64)[:, None] * self.sb.astype(np.float64)
        near(got, ref, (4 * U + UO[dtype]) * np.abs(ref) + TINY[dtype], dtype)


SIZES = [(1, 1, 1), (1, 9, 15), (1, 64, 512), (1, 131, 4099), (2, 33, 130), (3, 128, 1024), (4, 17, 16), (5, 7, 200),
         (7, 257, 264), (8, 40, 2048), (9, 65, 33), (15, 300, 512), (16, 128, 64), (17, 129, 72), (33, 200, 640),
         (64, 256, 128), (65, 130, 1000), (100, 64, 2056), (128, 300, 256), (129, 127, 65), (147, 513, 1025),
         (260, 264, 192), (300, 520, 3000)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_sizes(m, n, k):
    p = Product(m, n, k)
    for dtype in ("f32", "f16", "bf16"):
        p.check(dtype, p.run(dtype))


@pytest.mark.parametrize("m", [1, 6, 30, 200])
@pytest.mark.parametrize("pad,off", [(0, 1), (3, 0), (4, 4), (16, 16), (1, 5), (8, 8)])
def test_product_layouts(m, pad, off):
    p = Product(m, 130, 272, pad, off)
    p.check("f16", p.run("f16", pad, off))


@pytest.mark.parametrize("m", [40, 300, 700])
@pytest.mark.parametrize("n,cpad", [(133, 3), (1030, 2), (33, 3), (35, 1)])
def test_product_columns_that_end_inside_16_bytes_of_aligned_rows(m, n, cpad):
    p = Product(m, n, 272)
    for dtype in ("f32", "f16", "bf16"):
        p.check(dtype, p.run(dtype, cpad))


@pytest.mark.parametrize("m,n,k,pad,off", [(8, 4096, 3001, 0, 0), (4, 8200, 4096, 0, 0), (3, 4099, 11000, 0, 0),
                                           (5, 4100, 2003, 1, 1), (40, 70, 20000, 0, 0), (100, 70, 20001, 0, 0),
                                           (12, 40, 66000, 0, 0), (250, 600, 9000, 0, 0), (300, 130, 4100, 16, 16)])
def test_product_of_large_weights_and_long_sums(m, n, k, pad, off):
    """Few rows on the tensor cores, and sums over several accumulators."""
    p = Product(m, n, k, pad, off)
    p.check("f32", p.run("f32"))


@pytest.mark.parametrize("m,n,k", [(512, 2000, 576), (1000, 1300, 2100), (700, 5504, 64), (2049, 264, 1031)])
def test_product_many_tiles(m, n, k):
    p = Product(m, n, k)
    for dtype in ("f32", "bf16"):
        p.check(dtype, p.run(dtype, 8))


@pytest.mark.parametrize("m", [1, 5, 40, 300])
@pytest.mark.parametrize("k", [1024, 1025, 4096, 20000, 131071])
def test_product_of_extreme_codes_is_exact(m, k):
    """Sums up to the last that 32 bits hold, and their alternating forms, equal to the integers rounded to f32."""
    n = 40
    rng = np.random.default_rng(k)
    a = np.full((m, k), -128, np.int8)
    b = np.full((n, k), -128, np.int8)
    b[1::4] = 127
    b[2::4, ::2] = 127
    b[3::4] = codes(rng, len(b[3::4]), k, -128)
    a[1::3] = codes(rng, len(a[1::3]), k, -128)
    st, need = gb.gbmm_gemm_i8_scratch_bytes(m, n, k, False)
    ad, bd = torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()
    c, scratch = torch.empty(m, n, device="cuda"), torch.empty(need + 1, dtype=torch.uint8, device="cuda")
    gb.check(gb.gbmm_gemm_i8("f32", m, n, k, ad, k, None, bd, k, None, c, n, scratch, need))
    want = (a.astype(np.float64) @ b.astype(np.float64).T).astype(np.float32)
    assert np.array_equal(c.cpu().numpy(), want)


@pytest.mark.parametrize("m", [1, 30, 300])
def test_product_of_nothing_and_scales_that_are_not_finite(m):
    p = Product(m, 40, 0)
    assert (p.run("f16") == 0).all()
    p = Product(m, 40, 100)
    p.sab.t[4096:4096 + 4 * m].copy_(torch.from_numpy(np.where(np.arange(m) == m // 2, np.nan, 1).astype(np.float32)
                                                      .view(np.uint8).copy()))
    bad = np.isnan(p.run("f32"))
    assert bad[m // 2].all() and bad.sum() == 40


@pytest.mark.parametrize("m", [2, 20, 200, 600])
def test_offsets_past_32_bits(m):
    """Codes with rows 2^30 bytes apart, values and outputs 2^24 elements apart."""
    n, k, ldb, ldc = 6, 144, 1 << 30, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(m)
    wide = torch.empty((m - 1) * ldc + k, dtype=torch.bfloat16, device="cuda").as_strided((m, k), (ldc, 1))
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    wide.copy_(x)
    q = [torch.empty(m, k, dtype=torch.int8, device="cuda"),
         torch.empty((m - 1) * ldc + k, dtype=torch.int8, device="cuda").as_strided((m, k), (ldc, 1))]
    s = torch.empty(2, m, device="cuda")
    gb.check(gb.gbmm_quantize_i8("bf16", m, k, x, k, q[0], k, s[0]))
    gb.check(gb.gbmm_quantize_i8("bf16", m, k, wide, ldc, q[1], ldc, s[1]))
    assert torch.equal(q[0], q[1]) and torch.equal(s[0], s[1])
    b = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    far = torch.empty((n - 1) * ldb + k, dtype=torch.int8, device="cuda").as_strided((n, k), (ldb, 1))
    far.copy_(b)
    y = torch.empty((m - 1) * ldc + n, device="cuda").as_strided((m, n), (ldc, 1))
    need = gb.gbmm_gemm_i8_scratch_bytes(m, n, k, False)[1]
    scratch = torch.empty(need + 1, dtype=torch.uint8, device="cuda")
    gb.check(gb.gbmm_gemm_i8("f32", m, n, k, q[1], ldc, None, far, ldb, None, y, ldc, scratch, need))
    assert torch.equal(y, (q[0].double() @ b.double().T).float())


def layer(m, n, k, t, stream=None):
    """A linear layer as a program makes it: its activations quantised, then the product."""
    gb.check(gb.gbmm_quantize_i8("bf16", m, k, t["x"], k, t["q"], k, t["s"], stream))
    gb.check(gb.gbmm_gemm_i8("bf16", m, n, k, t["q"], k, t["s"], t["w"], k, t["ws"], t["y"], n, t["scratch"],
                             t["need"], stream))
    return t["y"].clone()


def make(m, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = {"x": torch.randn(m, k, generator=g, device="cuda").bfloat16(), "need": gb.gbmm_gemm_i8_scratch_bytes(m, n, k, False)[1]}
    w = torch.randn(n, k, generator=g, device="cuda").bfloat16()
    t |= {"q": torch.empty(m, k, dtype=torch.int8, device="cuda"), "s": torch.empty(m, device="cuda"),
          "w": torch.empty(n, k, dtype=torch.int8, device="cuda"), "ws": torch.empty(n, device="cuda"),
          "y": torch.empty(m, n, device="cuda").bfloat16(), "full": w,
          "scratch": torch.empty(t["need"] + 1, dtype=torch.uint8, device="cuda")}
    gb.check(gb.gbmm_quantize_i8("bf16", n, k, w, k, t["w"], k, t["ws"]))
    return t


LAYERS = [(1, 200, 520), (24, 264, 1032), (300, 520, 2056), (600, 1032, 520)]


@pytest.mark.parametrize("m,n,k", LAYERS)
def test_layer(m, n, k):
    """Quantised layer against the same layer in 64 bits: each factor is off by half a code at most."""
    t = make(m, n, k, 1)
    y = layer(m, n, k, t).double().cpu().numpy()
    x, w = t["x"].double().cpu().numpy(), t["full"].double().cpu().numpy()
    dx = 0.5 * np.abs(x).max(axis=1, keepdims=True) / 127 * (1 + 1e-6)
    dw = 0.5 * np.abs(w).max(axis=1, keepdims=True) / 127 * (1 + 1e-6)
    ref = x @ w.T
    tol = dx * np.abs(w).sum(axis=1) + np.abs(x).sum(axis=1, keepdims=True) * dw.T + k * dx * dw.T
    near(y, ref, tol * 1.01 + UO["bf16"] * np.abs(ref), "layer")


@pytest.mark.parametrize("m,n,k", LAYERS)
def test_layer_repeats_and_replays(m, n, k):
    t, other = make(m, n, k, 2), make(m, n, k, 3)
    first = layer(m, n, k, t)
    t["scratch"].fill_(255)
    assert torch.equal(first, layer(m, n, k, t))
    want = layer(m, n, k, other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(m, n, k, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = layer(m, n, k, t)
    for name in ("x", "w", "ws"):
        t[name].copy_(other[name])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_two_streams_at_once():
    sets = [make(*s, seed) for seed, s in enumerate(LAYERS[1:3])]
    want = [layer(*s, t) for s, t in zip(LAYERS[1:3], sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = []
        for s, t, st in zip(LAYERS[1:3], sets, streams):
            with torch.cuda.stream(st):
                got.append(layer(*s, t, st))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("m,n,k", [(40, 3584, 18944), (64, 2500, 24576), (33, 3584, 16385), (64, 2600, 16384)])
def test_long_sums_of_some_tens_of_tokens_in_more_ctas_than_sms(m, n, k):
    """Tiles of 64 and of 128 tokens on both sides of the limit of 64's tensor memory, clusters of six to eight over all SMs."""
    st, (tokens, cluster, _, _) = gb.gbmm_test_few_plan(1, m, n, k, 152)
    gb.check(st)
    assert cluster >= 6 and -(-n // 128) * cluster > 152 and tokens == (64 if k <= 16384 else 128)
    p = Product(m, n, k)
    p.check("f32", p.run("f32"))
