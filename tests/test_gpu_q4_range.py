"""GPU parity of the 4-bit matrix-vector products where values are very large or
small, and where the weights are zero or x has one sign, against the dequantised product
in 64 bits.

Tolerances are those of test_gpu_q4.py, relative to sum |w x| (so a result is exactly 0 where
every weight is 0).  A row of x that is
computed in plain f32 (an infinity, a NaN or a magnitude of 2^112 and more) rounds each
weight and each product once and adds up within the groups of g columns, then the
groups: (g + ceil(k / g) + 2) 2^-24 of sum |w x|.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_moe_expert_gb300 import binding as gb  # noqa: E402
from gemv_moe_expert_gb300 import synth  # noqa: E402
from tests import moe_ref  # noqa: E402
from tests.gpu_util import DevBuf, to_f64  # noqa: E402
from tests.test_gpu_moe import TINY, UO, empty, fetch, ints, near, strided  # noqa: E402
from tests.test_gpu_q4 import tau  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemv_moe_expert_gb300 import build
    build.build()
    gb.load()
    torch.cuda.init()


def signed(rng, shape, low, high):
    """Magnitudes between low and high, of either sign."""
    return rng.choice([-1.0, 1.0], shape) * rng.uniform(low, high, shape)


def product(dtype, x, codes, scales, scale_dt, group, zeros=None, by_id=False):
    """The library's result, x and the matrix in 64 bits; codes [n, k], scales and zeros [n, G].
    by_id: through the per-expert call, as the second of two experts."""
    m, (n, k) = x.shape[0], codes.shape
    xb, xp, xv = strided(x, k, dtype)
    packed = moe_ref.pack_q4(codes)
    stored = synth._store(scales.astype(np.float32), scale_dt)
    w = moe_ref.q4_matrix(packed, to_f64(stored, scale_dt), zeros, k, group)
    copies = 2 if by_id else 1
    qb = DevBuf(packed.nbytes * copies, host=np.stack([packed] * copies))
    sb = DevBuf(stored.nbytes * copies, host=np.stack([stored] * copies))
    zb = None if zeros is None else DevBuf(zeros.nbytes * copies, host=np.stack([zeros] * copies))
    out, outp = empty(m, n, dtype)
    ldq, z = (k + 1) // 2, None if zb is None else zb.ptr
    if by_id:
        ib = ints(np.ones((m, 1)))
        gb.check(gb.gbmm_matmul_id_q4(dtype, m, n, k, 1, 2, gb.INPUT_SHARED_PER_TOKEN, group, qb.ptr, ldq, n * ldq,
                                      sb.ptr, scale_dt, z, xp, ib.ptr, outp))
    else:
        gb.check(gb.gbmm_gemv_q4(dtype, m, n, k, group, qb.ptr, ldq, sb.ptr, scale_dt, z, xp, k, outp, n))
    return fetch(out, m, n, n, dtype), xv, w


def agree(got, x, w, dtype, relative, what, extra=0.0):
    ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    near(got, ref, relative * mag + UO[dtype] * np.abs(ref) + TINY[dtype] * (mag > 0) + extra, what)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale_dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("by_id", [False, True])
def test_large_values_times_large_scales(dtype, scale_dt, group, by_id):
    """Eight values of x a row up to 2^116, scales from 4 up, up to 2^119 together: every sum of terms stays
    below 2^127.1 whatever the signs, so the results are finite."""
    rng = np.random.default_rng(11)
    n, k = 40, 512
    for e, t in ((116, 2), (112, 6), (104, 15), (116, 3)):
        x = np.zeros((3, k))
        for row in x:
            row[rng.choice(k, 8, replace=False)] = signed(rng, 8, 1.0, 1.5) * 2.0 ** e
        codes = rng.integers(0, 16, (n, k)).astype(np.uint8)
        codes[0], codes[1] = 0, 15
        scales = rng.uniform(1.0, 1.5, (n, k // group)) * 2.0 ** t
        got, xv, w = product(dtype, x, codes, scales, scale_dt, group, by_id=by_id)
        agree(got, xv, w, dtype, tau(dtype, k, group), (e, t))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale_dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_values_near_the_largest_of_f32(dtype, scale_dt, group):
    """Up to 2^126.6 times scales of 2^-14: a group's sum of codes times x passes the range of
    f32, the results do not."""
    rng = np.random.default_rng(12)
    n, k = 37, 300
    x = signed(rng, (3, k), 1.0, 1.5) * 2.0 ** 126
    x[1] *= 2.0 ** -8
    x[2] = rng.standard_normal(k)
    codes = rng.integers(0, 16, (n, k)).astype(np.uint8)
    scales = rng.uniform(1.0, 1.5, (n, -(-k // group))) * 2.0 ** -14
    zeros = rng.integers(0, 256, scales.shape).astype(np.uint8)
    for z in (None, zeros):
        got, xv, w = product(dtype, x, codes, scales, scale_dt, group, z)
        agree(got[:2], xv[:2], w, dtype, (group + -(-k // group) + 2) * 2.0 ** -24, "plain")
        agree(got[2:], xv[2:], w, dtype, tau(dtype, k, group), "another row")


ALIGNED = [(512, 48), (500, 33), (517, 5)]  # packed rows on 32 bytes; anywhere, a ragged last group


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("by_id", [False, True])
@pytest.mark.parametrize("k,n", ALIGNED)
def test_weights_of_zero_give_zero(dtype, group, by_id, k, n):
    """Codes that equal their zero point are weights of exactly 0."""
    rng = np.random.default_rng(13)
    scales, zeros = rng.uniform(0.5, 1.5, (n, -(-k // group))), rng.integers(0, 16, (n, -(-k // group))).astype(np.uint8)
    for x in (rng.uniform(0.5, 1.5, (9, k)), rng.standard_normal((1, k)) * 1000, rng.uniform(1.0, 2.0, (2, k))):
        for scale_dt in ("f16", "f32"):
            got, _, w = product(dtype, x, np.full((n, k), 8, np.uint8), scales, scale_dt, group, by_id=by_id)
            assert (w == 0).all() and (got == 0).all()
            codes = np.repeat(zeros, group, axis=1)[:, :k]
            got, _, w = product(dtype, x, codes, scales, scale_dt, group, zeros, by_id=by_id)
            assert (w == 0).all() and (got == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("k,n", ALIGNED)
def test_few_weights_that_are_not_zero(dtype, group, k, n):
    """x of one sign everywhere; a row of the matrix has three weights that are not zero."""
    rng = np.random.default_rng(14)
    scales, zeros = rng.uniform(0.5, 1.5, (n, -(-k // group))), rng.integers(1, 15, (n, -(-k // group))).astype(np.uint8)
    x = rng.uniform(0.5, 1.5, (4, k))
    for z in (None, zeros):
        codes = np.full((n, k), 8, np.uint8) if z is None else np.repeat(z, group, axis=1)[:, :k].copy()
        for row in codes:
            at = rng.choice(k, 3, replace=False)
            row[at] += rng.choice([-1, 1], 3).astype(np.int8).view(np.uint8)
        got, xv, w = product(dtype, x, codes, scales, "f16", group, z)
        assert ((w != 0).sum(axis=1) == 3).all()
        agree(got, xv, w, dtype, tau(dtype, k, group), z is None)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("k,n", ALIGNED)
def test_rows_of_one_sign(dtype, group, k, n):
    rng = np.random.default_rng(15)
    codes = rng.integers(0, 16, (n, k)).astype(np.uint8)
    scales = rng.uniform(0.005, 0.015, (n, -(-k // group)))
    x = rng.uniform(0.5, 1.5, (5, k)) * np.array([1.0, -1.0, 1.0, -30.0, 0.01])[:, None]
    far = rng.integers(0, 256, scales.shape).astype(np.uint8)
    for z in (None, rng.integers(0, 16, scales.shape).astype(np.uint8), far):
        got, xv, w = product(dtype, x, codes, scales, "f16", group, z)
        agree(got, xv, w, dtype, tau(dtype, k, group), "one sign")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("factor", [2.0 ** 6, 2.0 ** 12])
def test_one_outlier_a_group(dtype, group, factor):
    """One value of x a group is `factor` times the others'; every other row of the matrix
    has a weight of 0 there.  (x keeps all its bits next to it.)"""
    rng = np.random.default_rng(16)
    n, k = 40, 640
    codes = rng.integers(0, 16, (n, k)).astype(np.uint8)
    scales = rng.uniform(0.005, 0.015, (n, k // group))
    x = signed(rng, (3, k), 0.5, 1.0)
    at = np.arange(0, k, group) + rng.integers(0, group, k // group)
    x[:, at] *= factor
    codes[::2, at] = 8
    got, xv, w = product(dtype, x, codes, scales, "f16", group)
    agree(got, xv, w, dtype, tau(dtype, k, group), factor)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("exponent", [-149, -140, -133, -126, -110])
def test_subnormal_values(dtype, group, exponent):
    """x from the smallest subnormals on, times scales that bring the results back."""
    rng = np.random.default_rng(17)
    n, k = 20, 256
    codes = rng.integers(0, 16, (n, k)).astype(np.uint8)
    scales = rng.uniform(1.0, 2.0, (n, k // group)) * 2.0 ** 100
    x = signed(rng, (2, k), 1.0, 8.0) * 2.0 ** exponent
    got, xv, w = product(dtype, x, codes, scales, "f32", group)
    # a group's sum of (q - z) x, before its scale, is held in f32: 2^-150 is half its last bit there
    agree(got, xv, w, dtype, tau(dtype, k, group), exponent, extra=k // group * 2.0 ** (101 - 150))


def test_matmul_id_q4_more_windows_than_a_grid_has():
    """67 million routed rows: more windows of 1024 than one launch takes."""
    m, E, tail = 65535 * 1024 + 1500, 2, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-8, 9, (m, 1), generator=g, device="cuda", dtype=torch.int8).half()
    ids = torch.randint(0, E + 1, (m, 1), generator=g, device="cuda", dtype=torch.int32)
    q = torch.tensor([11, 2], dtype=torch.uint8, device="cuda")  # 3 and -6
    scales = torch.ones(E, 1, 1, dtype=torch.float16, device="cuda")
    out = torch.full((m + tail,), 77.0, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    gb.check(gb.gbmm_matmul_id_q4("f16", m, 1, 1, 1, E, gb.INPUT_SHARED_PER_TOKEN, 128, q, 1, 1, scales, "f16", None, x,
                                  ids, out))
    torch.cuda.synchronize()
    w = torch.tensor([3.0, -6.0, 0.0], dtype=torch.float16, device="cuda")
    assert torch.equal(out[:m], (x * w[ids.long()])[:, 0])
    assert (out[m:] == 77.0).all()
