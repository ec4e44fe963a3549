"""GPU parity of the 4-bit matrix-vector products against the dequantised
product in 64 bits.

Tolerance, from the arithmetic: a group's sum of g integer-times-x products runs
in f32 over steps of 16 (a tensor-core accumulation may truncate: 2^-22 of the
partial sum a step, and x in f32 takes three steps), the groups' scaled sums are
added in f32 (k/32 + 16 additions at most): relative to sum |w x|
    tau = (3 if f32 else 1) * ceil(g / 16) * 2^-22 + (k / 32 + 16) * 2^-24
plus the rounding of the stored result.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_moe_expert_gb300 import binding as gb  # noqa: E402
from gemv_moe_expert_gb300 import synth  # noqa: E402
from tests import moe_ref  # noqa: E402
from tests.gpu_util import DevBuf, to_f64  # noqa: E402
from tests.test_gpu_moe import TINY, UO, empty, fetch, ints, near, strided  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemv_moe_expert_gb300 import build
    build.build()
    gb.load()
    torch.cuda.init()


class Weights:
    """Packed matrices [E, n, k] with rows ldq and experts stride bytes apart; the
    bytes between rows hold 0xFF, and the last row ends with the buffer."""

    def __init__(self, E, n, k, group, scale_dt, zeros, rng, ldq=None, stride_pad=0, offset=0):
        nb, G = (k + 1) // 2, -(-k // group)
        self.ldq = ldq or nb
        self.stride = n * self.ldq + stride_pad
        codes = rng.integers(0, 16, (E, n, k)).astype(np.uint8)
        packed = moe_ref.pack_q4(codes)
        flat = np.full(offset + max(0, (E - 1) * self.stride + (n - 1) * self.ldq + nb), 0xFF, np.uint8)
        for e in range(E):
            for j in range(n):
                at = offset + e * self.stride + j * self.ldq
                flat[at:at + nb] = packed[e, j]
        self.qb = DevBuf(max(flat.size, 1), host=flat)
        self.q = self.qb.ptr + offset
        s = synth._store((rng.uniform(0.5, 1.5, (E, n, G)) * 0.01).astype(np.float32), scale_dt)
        self.sb = DevBuf(max(s.nbytes, 4), host=s)
        self.scale_dt = scale_dt
        z = rng.integers(0, 17, (E, n, G)).astype(np.uint8) if zeros else None
        if zeros == "far":
            z = rng.integers(0, 256, (E, n, G)).astype(np.uint8)
        self.zb = None if z is None else DevBuf(max(z.nbytes, 1), host=z)
        s64 = to_f64(s, scale_dt)
        self.w = moe_ref.q4_matrix(packed, s64, z, k, group) if k else np.zeros((E, n, 0))

    @property
    def zeros(self):
        return None if self.zb is None else self.zb.ptr


def tau(dtype, k, group):
    return (3 if dtype == "f32" else 1) * -(-group // 16) * 2.0 ** -22 + (k / 32 + 16) * 2.0 ** -24


def check(got, x, w, dtype, k, group, what):
    ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    near(got, ref, tau(dtype, k, group) * mag + UO[dtype] * np.abs(ref) + TINY[dtype], what)


def dense(dtype, m, n, k, group, scale_dt="f16", zeros=False, ldq=None, offset=0, xpad=0, ypad=0, xoff=0, seed=0):
    rng = np.random.default_rng(seed + n * 7 + k)
    wts = Weights(1, n, k, group, scale_dt, zeros, rng, ldq, 0, offset)
    xb, xp, x = strided(rng.standard_normal((m, k)), k + xpad, dtype, offset=xoff)
    out, outp = empty(m, n + ypad, dtype)
    gb.check(gb.gbmm_gemv_q4(dtype, m, n, k, group, wts.q, wts.ldq, wts.sb.ptr, scale_dt, wts.zeros, xp, k + xpad,
                             outp, n + ypad))
    check(fetch(out, m, n, n + ypad, dtype), x, wts.w[0], dtype, k, group, (dtype, m, n, k, group))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 64, 128), (1, 33, 257), (2, 17, 1024), (3, 100, 2050), (8, 48, 512),
                                   (9, 31, 96), (16, 16, 640), (27, 5, 130), (1, 130, 4096), (5, 16, 9000)])
def test_gemv_q4(dtype, group, zeros, m, n, k):
    dense(dtype, m, n, k, group, zeros=zeros)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale_dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemv_q4_scale_types_and_far_zero_points(dtype, scale_dt, group):
    dense(dtype, 2, 40, 520, group, scale_dt=scale_dt, zeros="far")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("k,ldq,offset", [(512, 256, 0), (512, 272, 16), (512, 260, 0), (512, 256, 4), (512, 257, 0),
                                          (512, 256, 1), (500, 256, 0), (501, 256, 0), (1000, 512, 8), (2050, 1040, 0)])
def test_gemv_q4_row_alignments(dtype, group, k, ldq, offset):
    """Every alignment of the packed rows; the last row ends with the buffer."""
    dense(dtype, 3, 37, k, group, zeros=True, ldq=ldq, offset=offset, xpad=3, ypad=5, xoff=1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gemv_q4_empty_contraction_writes_zeros(dtype):
    out, outp = empty(3, 10, dtype)
    gb.check(gb.gbmm_gemv_q4(dtype, 3, 10, 0, 32, None, 0, None, "f16", None, None, 0, outp, 10))
    assert (fetch(out, 3, 10, 10, dtype) == 0).all()


def test_gemv_q4_f32_inputs_keep_their_precision():
    """x with all 24 bits in use and weights that cancel it: an x rounded to 16
    bits would be off by about 2^-9 of a term."""
    k, n = 256, 16
    x = np.zeros((1, k), np.float32)
    x[0, 0], x[0, 1] = np.float32(1 + 2.0 ** -23), np.float32(-1)
    codes = np.full((1, n, k), 8, np.uint8)
    codes[0, :, :2] = 9
    packed = moe_ref.pack_q4(codes)
    qb, sb = DevBuf(packed.nbytes, host=packed), DevBuf(n * 2 * 4, host=np.ones(n * 2, np.float32))
    xb, xp, _ = strided(x, k, "f32")
    out, outp = empty(1, n, "f32")
    gb.check(gb.gbmm_gemv_q4("f32", 1, n, k, 128, qb.ptr, k // 2, sb.ptr, "f32", None, xp, k, outp, n))
    assert (fetch(out, 1, n, n, "f32") == 2.0 ** -23).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gemv_q4_infinities_and_nan_reach_only_their_row(dtype):
    rng = np.random.default_rng(1)
    m, n, k = 4, 20, 300
    wts = Weights(1, n, k, 64, "f16", False, rng)
    vals = rng.standard_normal((m, k))
    vals[1, 7], vals[2, 299] = np.nan, np.inf
    xb, xp, x = strided(vals, k, dtype)
    out, outp = empty(m, n, dtype)
    gb.check(gb.gbmm_gemv_q4(dtype, m, n, k, 64, wts.q, wts.ldq, wts.sb.ptr, "f16", None, xp, k, outp, n))
    got = fetch(out, m, n, n, dtype)
    assert np.isnan(got[1]).all()
    with np.errstate(invalid="ignore"):
        ref = x[2] @ wts.w[0].T
    assert np.array_equal(np.isnan(got[2]), np.isnan(ref))
    fine = ~np.isnan(ref)
    assert np.array_equal(got[2][fine], ref[fine])  # infinities with their signs
    for t in (0, 3):
        check(got[t:t + 1], x[t:t + 1], wts.w[0], dtype, k, 64, t)


# ---------------------------------------------------------------------------
# per expert id
# ---------------------------------------------------------------------------

def experts(dtype, m, n, k, top_k, E, group, layout=0, zeros=False, scale_dt="f16", ids=None, ldq=None, stride_pad=0,
            offset=0, seed=0):
    rng = np.random.default_rng(seed + n + k + m)
    wts = Weights(E, n, k, group, scale_dt, zeros, rng, ldq, stride_pad, offset)
    ids = rng.integers(0, E, (m, top_k)).astype(np.uint32) if ids is None else np.asarray(ids, np.uint32)
    rows = m * top_k
    xrows = m if layout == 0 else rows
    xb, xp, x = strided(rng.standard_normal((xrows, k)), max(k, 1), dtype)
    out, outp = empty(rows, n, dtype)
    ib = ints(ids)
    gb.check(gb.gbmm_matmul_id_q4(dtype, m, n, k, top_k, E, layout, group, wts.q, wts.ldq, wts.stride, wts.sb.ptr,
                                  scale_dt, wts.zeros, xp, ib.ptr, outp))
    got = fetch(out, rows, n, n, dtype)
    for r, e in enumerate(ids.reshape(-1)):
        if e >= E:
            assert (got[r] == 0).all(), r
        else:
            at = r // top_k if layout == 0 else r
            check(got[r:r + 1], x[at:at + 1], wts.w[e], dtype, k, group, (r, int(e)))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("m,n,k,top_k,E", [(1, 48, 256, 2, 4), (1, 1, 1, 1, 1), (4, 33, 130, 8, 16), (16, 20, 128, 4, 5),
                                           (40, 16, 64, 3, 2), (7, 70, 2048, 2, 64)])
def test_matmul_id_q4(dtype, group, layout, m, n, k, top_k, E):
    experts(dtype, m, n, k, top_k, E, group, layout, zeros=bool(group == 64))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_matmul_id_q4_ids_without_expert_and_repeats(dtype):
    E = 6
    ids = [[0, 0, 0], [E, 2, 0xFFFFFFFF], [5, 5, E + 1], [E, E, E]]
    experts(dtype, 4, 35, 200, 3, E, 32, ids=ids)
    experts(dtype, 4, 35, 200, 3, E, 32, layout=1, ids=np.full((4, 3), E))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_matmul_id_q4_strides(dtype):
    experts(dtype, 3, 18, 300, 2, 5, 64, ldq=160, stride_pad=48, offset=16, zeros=True, scale_dt="bf16")
    experts(dtype, 3, 18, 300, 2, 5, 64, ldq=151, stride_pad=5, offset=3, zeros=True, scale_dt="f32")


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("ldq,offset,stride_pad", [(2064, 0, 0), (2048, 16, 16), (2045, 3, 1)])
def test_matmul_id_q4_odd_sizes(dtype, group, ldq, offset, stride_pad):
    """Rows that end inside an access, the last one at the end of the memory."""
    experts(dtype, 6, 161, 4090, 2, 3, group, ldq=ldq, offset=offset, stride_pad=stride_pad, zeros=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_matmul_id_q4_more_rows_than_a_window(dtype):
    experts(dtype, 400, 17, 96, 6, 9, 32)


def test_matmul_id_q4_many_experts():
    experts("bf16", 150, 16, 64, 8, 1024, 64)


def test_matmul_id_q4_empty_contraction_writes_zeros():
    out, outp = empty(6, 10, "bf16")
    ib = ints([[0, 1], [2, 3], [0, 9]])
    gb.check(gb.gbmm_matmul_id_q4("bf16", 3, 10, 0, 2, 4, 0, 32, None, 0, 0, None, "f16", None, None, ib.ptr, outp))
    assert (fetch(out, 6, 10, 10, "bf16") == 0).all()


def test_q4_in_a_cuda_graph_on_another_stream():
    rng = np.random.default_rng(2)
    n, k, E = 64, 512, 8
    wts = Weights(E, n, k, 128, "f16", False, rng)
    x = torch.randn(2, k, device="cuda")
    ids = torch.tensor([[1, 5], [5, 3]], dtype=torch.int32, device="cuda")
    out = torch.empty(2, 2, n, device="cuda")

    def step(stream):
        gb.check(gb.gbmm_matmul_id_q4("f32", 2, n, k, 2, E, 0, 128, wts.q, wts.ldq, wts.stride, wts.sb.ptr, "f16", None,
                                      x, ids, out, stream))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    x.copy_(torch.randn(2, k, device="cuda"))
    ids.copy_(torch.tensor([[7, 0], [E, 7]], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got, xv = out.double().cpu().numpy(), x.double().cpu().numpy()
    for t in range(2):
        for s, e in enumerate(ids[t].tolist()):
            if e == E:
                assert (got[t, s] == 0).all()
            else:
                check(got[t, s][None], xv[t:t + 1], wts.w[e], "f32", k, 128, (t, s))
