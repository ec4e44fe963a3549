"""GPU parity of the mixture-of-experts layer's router, expert order, dispatch
and combine, and their gradients, against plain 64-bit definitions.

Tolerances, from the arithmetic (f32 throughout, one rounding per output; u =
2^-24, uo = half an ulp of the output type relative to its value):
  weights     relative u * (D + E/32 + 24): D = the largest |l - max| (rounding of
              the subtraction, through exp), exp and the division a few u, the sum
              at most E/32 additions in a lane and 5 across lanes
  d_logits    the same factor + 8 on p * (|g| + sum w |d|), plus uo |value|
  combine     u * (top_k + 1) * sum |w y|, plus uo |y|
  d_weights   u * (n + 1) * sum |d_y y| (any order of a sum of n products)
  d_ys        one product and its rounding: (u + uo) |value|
  copies, ids, permutations: exact.
Values below the output type's normal range get its absolute half spacing.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_moe_expert_gb300 import binding as gb  # noqa: E402
from gemv_moe_expert_gb300 import synth  # noqa: E402
from tests import moe_ref  # noqa: E402
from tests.gpu_util import NP_DT, SENTINEL, DevBuf, to_f64  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UO = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemv_moe_expert_gb300 import build
    build.build()
    gb.load()
    torch.cuda.init()


def strided(values, ld, dtype, fill=np.nan, offset=0):
    """A device buffer holding [rows, cols] values with rows ld elements apart
    (gaps hold `fill`), the matrix starting `offset` elements into it."""
    rows, cols = values.shape
    flat = np.full(offset + max(rows, 1) * ld, fill, np.float32)
    at = offset + np.arange(rows)[:, None] * ld + np.arange(cols)[None, :]
    flat[at] = values
    with np.errstate(invalid="ignore", over="ignore"):
        stored = synth._store(flat, dtype)
    buf = DevBuf(stored.nbytes, host=stored)
    return buf, buf.ptr + offset * synth.ITEMSIZE[dtype], to_f64(stored, dtype)[at]


def empty(rows, ld, dtype, offset=0):
    buf = DevBuf((offset + max(rows, 1) * ld) * synth.ITEMSIZE[dtype])
    return buf, buf.ptr + offset * synth.ITEMSIZE[dtype]


def fetch(buf, rows, cols, ld, dtype, offset=0):
    """[rows, cols] as f64; everything around it must be untouched."""
    torch.cuda.synchronize()
    raw = buf.read(NP_DT[dtype])
    at = offset + np.arange(rows)[:, None] * ld + np.arange(cols)[None, :]
    rest = np.ones(raw.size, bool)
    rest[at.reshape(-1)] = False
    assert (raw[rest].view(np.uint8) == SENTINEL).all(), "wrote between or past the rows"
    assert buf.guards_intact()
    return to_f64(raw, dtype)[at]


def ints(values):
    a = np.ascontiguousarray(values, np.uint32)
    return DevBuf(max(a.nbytes, 4), host=a)


def floats(values):
    a = np.ascontiguousarray(values, np.float32)
    return DevBuf(max(a.nbytes, 4), host=a)


def near(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], ref[bad][:3], np.broadcast_to(tol, ref.shape)[bad][:3])


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------

def run_route(logits, dtype, top_k, selected, bias=None, ld=None, offset=0):
    m, E = logits.shape
    ld = ld or E
    lb, lp, vals = strided(logits, ld, dtype, offset=offset)
    ids, w = DevBuf(m * top_k * 4), DevBuf(m * top_k * 4)
    bb = None if bias is None else floats(bias)
    gb.check(gb.gbmm_moe_route(dtype, m, E, top_k, int(selected), lp, ld, None if bb is None else bb.ptr, ids.ptr,
                               w.ptr))
    torch.cuda.synchronize()
    assert ids.guards_intact() and w.guards_intact()
    return (vals, ids.read(np.uint32).reshape(m, top_k).astype(np.int64),
            w.read(np.float32).reshape(m, top_k).astype(np.float64), (lb, lp, bb, ids, w))


def run_route_backward(held, m, E, top_k, selected, dtype, ld, d_w, ld_out, offset=0):
    lb, lp, bb, ids, w = held
    dw = floats(d_w)
    out, outp = empty(m, ld_out, dtype, offset)
    logits = (None, 0) if selected else (lp, ld)
    gb.check(gb.gbmm_moe_route_backward(dtype, m, E, top_k, int(selected), logits[0], logits[1],
                                        None if bb is None or selected else bb.ptr, ids.ptr, w.ptr, dw.ptr, outp,
                                        ld_out))
    return fetch(out, m, E, ld_out, dtype, offset)


def weight_factor(vals, live):
    l = np.where(live & np.isfinite(vals), vals, np.nan)
    with np.errstate(invalid="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            D = np.nan_to_num(np.nanmax(l, axis=1) - np.nanmin(l, axis=1)) if l.size else np.zeros(len(l))
    D = np.minimum(D, 110)  # exp(-104) is 0 in f32: what lies further down has no weight
    return U * (D[:, None] + vals.shape[1] / 32 + 24)


def check_route(logits, dtype, top_k, selected, bias=None, ld=None, offset=0, seed=0):
    m, E = logits.shape
    ld = ld or E
    vals, ids, w, held = run_route(logits, dtype, top_k, selected, bias, ld, offset)
    rid, rw, rp, live = moe_ref.route(vals.astype(np.float32), bias, top_k, selected)
    assert np.array_equal(ids, rid)
    f = weight_factor(vals, live)
    near(w, rw, f * rw + 2.0 ** -126, "weights")
    d_w = np.random.default_rng(seed).standard_normal((m, top_k)).astype(np.float32)
    got = run_route_backward(held, m, E, top_k, selected, dtype, ld, d_w, E + 3, offset)
    d64 = d_w.astype(np.float64)
    ref = moe_ref.route_backward(ids, rw, rp, d64, E)
    mag = rp * (rw * np.abs(d64)).sum(axis=1, keepdims=True)
    for t in range(m):
        for s in range(top_k):
            if rid[t, s] < E:
                mag[t, rid[t, s]] += rw[t, s] * abs(d64[t, s])
    near(got, ref, 2 * (f + 8 * U) * mag + UO[dtype] * np.abs(ref) + TINY[dtype] + 2.0 ** -126, "d_logits")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("m,E,top_k", [(1, 1, 1), (1, 64, 8), (3, 5, 5), (9, 33, 3), (17, 64, 32), (8, 128, 8),
                                       (5, 257, 7), (3, 1000, 16), (2, 1024, 32), (65, 11, 2)])
def test_route(dtype, selected, m, E, top_k):
    rng = np.random.default_rng(m * 1000 + E)
    check_route(rng.standard_normal((m, E)) * 2, dtype, top_k, selected)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("E", [8, 96, 130])
def test_route_bias_strides_offsets(dtype, selected, E):
    rng = np.random.default_rng(E)
    check_route(rng.standard_normal((19, E)), dtype, 6, selected, bias=rng.standard_normal(E).astype(np.float32),
                ld=E + 5, offset=3)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_ties_take_the_lowest_index(dtype, selected):
    rng = np.random.default_rng(5)
    logits = rng.integers(-2, 3, (40, 77)).astype(np.float64)
    logits[0] = 0.0
    logits[1] = np.where(np.arange(77) % 2, 0.0, -0.0)  # -0 and +0 are equal
    check_route(logits, dtype, 9, selected)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_route_masked_experts_and_empty_rows(dtype, selected):
    rng = np.random.default_rng(6)
    E, lowest = 70, {"f32": -3.4028234663852886e38, "f16": -65504.0, "bf16": -3.3895313892515355e38}[dtype]
    logits = rng.standard_normal((12, E))
    logits[0, :] = -np.inf                  # nobody
    logits[1, :] = np.nan
    logits[2, 3:] = -np.inf                 # fewer than top_k
    logits[3, ::2] = np.nan
    logits[4, 5:] = lowest                  # the type's lowest value is an ordinary logit
    logits[5, :] = lowest
    logits[6, :E - 1] = -np.inf             # one expert
    bias = np.zeros(E, np.float32)
    bias[10:20] = -np.inf                   # masked for every token
    logits[7, 10:20] = np.nan               # whatever stands in masked places
    logits[8, 10:20] = np.inf
    bias[20] = np.nan
    check_route(logits, dtype, 5, selected, bias=bias)


@pytest.mark.parametrize("dtype,E,top_k,selected", [("f32", 128, 8, False), ("f32", 6, 3, True), ("bf16", 64, 1, False),
                                                    ("f16", 101, 7, True), ("bf16", 200, 8, False), ("f32", 40, 16, True), ("f16", 256, 13, False), ("f32", 300, 6, True)])
def test_route_many_tokens(dtype, E, top_k, selected):
    """A batch from which a warp takes several tokens, the last warp fewer; equal,
    masked and empty rows lie among the others."""
    rng = np.random.default_rng(E)
    m = 64 * torch.cuda.get_device_properties(0).multi_processor_count + 3
    logits = rng.standard_normal((m, E))
    logits[1::9] = rng.integers(-1, 2, logits[1::9].shape)
    logits[2::9] = -np.inf
    logits[3::9, top_k // 2:] = -np.inf
    logits[4::9, ::2] = np.nan
    bias = rng.standard_normal(E).astype(np.float32)
    bias[E // 2] = -np.inf
    check_route(logits, dtype, top_k, selected, bias=bias if E != 128 else None, ld=E + E % 4)


def test_route_many_waves_of_tokens():
    rng = np.random.default_rng(8)
    m = 256 * torch.cuda.get_device_properties(0).multi_processor_count + 5
    check_route(rng.standard_normal((m, 12)), "f16", 2, False)


def test_route_infinite_live_logit_gives_nan_weights():
    logits = np.zeros((1, 8))
    logits[0, 3] = np.inf
    _, ids, w, _ = run_route(logits, "f32", 2, True)
    assert ids[0].tolist() == [3, 0]
    assert np.isnan(w).all()


def test_route_gradient_against_differences():
    """Central differences of sum(c * weights) in the logits.  Logits are 1/8
    apart and the step is 1/64, so the selection stays; the error is the third
    derivative (at most 1 per unit of c) times h^2 / 6, and the weights' rounding
    (at most 64 u) over h."""
    rng = np.random.default_rng(3)
    m, E, top_k, h = 2, 24, 4, 1 / 64
    logits = np.stack([rng.permutation(E) for _ in range(m)]) / 8.0
    c = rng.standard_normal((m, top_k)).astype(np.float32)
    for selected in (False, True):
        _, _, _, held = run_route(logits, "f32", top_k, selected)
        got = run_route_backward(held, m, E, top_k, selected, "f32", E, c, E)
        for e in range(E):
            up, down = logits.copy(), logits.copy()
            up[:, e] += h
            down[:, e] -= h
            diff = (run_route(up, "f32", top_k, selected)[2] - run_route(down, "f32", top_k, selected)[2]) / (2 * h)
            near(got[:, e], (c * diff).sum(axis=1), np.abs(c).sum(axis=1) * (h * h / 6 + 64 * U / h), e)


# ---------------------------------------------------------------------------
# sort
# ---------------------------------------------------------------------------

def run_sort(ids, E):
    m, top_k = ids.shape
    rows = m * top_k
    st, need = gb.gbmm_moe_sort_scratch_bytes(m, top_k, E)
    gb.check(st)
    scratch = DevBuf(max(need, 4))
    off, order, pos = DevBuf((E + 1) * 4), DevBuf(max(rows, 1) * 4), DevBuf(max(rows, 1) * 4)
    ib = ints(ids)
    gb.check(gb.gbmm_moe_sort(m, top_k, E, ib.ptr, off.ptr, order.ptr, pos.ptr, scratch.ptr if need else None, need))
    torch.cuda.synchronize()
    for b in (off, order, pos, scratch):
        assert b.guards_intact()
    return (off.read(np.uint32).astype(np.int64), order.read(np.uint32)[:rows].astype(np.int64),
            pos.read(np.uint32)[:rows].astype(np.int64), (off, order, pos))


@pytest.mark.parametrize("m,top_k,E", [(0, 2, 5), (1, 1, 1), (1, 8, 64), (3, 5, 4), (33, 1, 7), (500, 3, 11),
                                       (511, 8, 128), (513, 8, 129), (4096, 8, 128), (5000, 7, 1024), (777, 6, 1000),
                                       (20000, 9, 37)])
def test_sort(m, top_k, E):
    rng = np.random.default_rng(m + E)
    ids = rng.integers(0, E, (m, top_k)).astype(np.uint32)
    check_sort(ids, E)


def check_sort(ids, E):
    got = run_sort(ids, E)
    key = np.minimum(ids.astype(np.int64).reshape(-1), E)
    order = np.argsort(key, kind="stable")
    assert np.array_equal(got[1], order)
    assert np.array_equal(got[2][order], np.arange(order.size))
    assert np.array_equal(got[0], np.searchsorted(key[order], np.arange(E + 1)))


@pytest.mark.parametrize("kind", ["one expert", "none", "some without", "last", "ramp"])
@pytest.mark.parametrize("m", [2, 300, 9000])
def test_sort_distributions(kind, m):
    E, top_k = 96, 4
    rng = np.random.default_rng(m)
    ids = rng.integers(0, E, (m, top_k)).astype(np.uint32)
    if kind == "one expert":
        ids[:] = 17
    elif kind == "none":
        ids[:] = np.where(rng.random(ids.shape) < 0.5, E, 0xFFFFFFFF)
    elif kind == "some without":
        ids[rng.random(ids.shape) < 0.4] = E + 3
    elif kind == "last":
        ids[:] = E - 1
    else:
        ids[:] = (np.arange(m * top_k).reshape(m, top_k) * E // (m * top_k)).astype(np.uint32)
    check_sort(ids, E)
    if m == 2:
        off, order, pos = moe_ref.sort(ids, E)
        got = run_sort(ids, E)
        assert np.array_equal(got[0], off) and np.array_equal(got[1], order) and np.array_equal(got[2], pos)


# ---------------------------------------------------------------------------
# dispatch and combine
# ---------------------------------------------------------------------------

class Rows:
    """A sorted batch: ids with rows that have no expert, positions and offsets."""

    def __init__(self, m, top_k, E, drop, seed, sorted_rows=True):
        rng = np.random.default_rng(seed)
        self.m, self.top_k, self.E, self.rng = m, top_k, E, rng
        ids = rng.integers(0, E, (m, top_k)).astype(np.uint32)
        ids[rng.random(ids.shape) < drop] = E
        if sorted_rows:
            self.off, _, self.pos, (ob, _, pb) = run_sort(ids, E)
            self.hold = (ob, pb)
            self.position, self.offsets, self.valid = pb.ptr, ob.ptr, int(self.off[-1])
        else:
            self.pos, self.valid = np.arange(m * top_k), m * top_k
            self.position = self.offsets = None
        self.rows = m * top_k


SHAPES = [  # m, top_k, E, n, pad, offset (elements): row starts of every alignment
    (1, 1, 1, 1, 0, 0), (1, 8, 64, 2048, 0, 0), (4, 8, 64, 256, 0, 0), (7, 3, 5, 33, 0, 0), (5, 2, 4, 1537, 7, 0),
    (6, 4, 9, 130, 2, 0), (3, 9, 16, 1000, 0, 1), (2, 33, 40, 64, 0, 0), (130, 1, 3, 40, 8, 0), (3, 2, 8, 9001, 0, 0),
    (2, 16, 8, 4100, 4, 4)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,top_k,E,n,pad,offset", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_dispatch_and_its_gradient(dtype, m, top_k, E, n, pad, offset, drop):
    b = Rows(m, top_k, E, drop, n)
    ld = n + pad
    xb, xp, x = strided(b.rng.standard_normal((m, n)), ld, dtype, offset=offset)
    out, outp = empty(b.rows, ld, dtype, offset)
    gb.check(gb.gbmm_moe_dispatch(dtype, m, top_k, E, n, xp, ld, b.position, b.offsets, outp, ld))
    assert np.array_equal(fetch(out, b.rows, n, ld, dtype, offset), moe_ref.dispatch(x, b.pos, b.valid, top_k))

    g = b.rng.standard_normal((b.rows, n))
    g[b.valid:] = np.nan  # rows without an expert are not read
    gbuf, gp, gv = strided(g, ld, dtype, offset=offset)
    dx, dxp = empty(m, ld, dtype, offset)
    gb.check(gb.gbmm_moe_dispatch_backward(dtype, m, top_k, E, n, gp, ld, b.position, b.offsets, dxp, ld))
    ref, mag = moe_ref.combine(np.nan_to_num(gv), None, b.pos, b.valid, m, top_k)
    near(fetch(dx, m, n, ld, dtype, offset), ref, U * (top_k + 1) * mag + UO[dtype] * np.abs(ref) + TINY[dtype], "d_x")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,top_k,E,n,pad,offset", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_combine_and_its_gradient(dtype, m, top_k, E, n, pad, offset, drop):
    check_combine(Rows(m, top_k, E, drop, n + 1), dtype, n, n + pad, offset)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,top_k,n", [(1, 8, 2048), (5, 3, 77), (64, 4, 128)])
def test_rows_in_routed_order(dtype, m, top_k, n):
    b = Rows(m, top_k, 6, 0.0, n, sorted_rows=False)
    check_combine(b, dtype, n, n, 0)
    xb, xp, x = strided(b.rng.standard_normal((m, n)), n, dtype)
    out, outp = empty(b.rows, n, dtype)
    gb.check(gb.gbmm_moe_dispatch(dtype, m, top_k, 6, n, xp, n, None, None, outp, n))
    assert np.array_equal(fetch(out, b.rows, n, n, dtype), np.repeat(x, top_k, axis=0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,top_k,E,n,pad,offset", [(9, 5, 7, 64, 1, 1), (6, 8, 8, 71, 0, 3), (5, 3, 4, 257, 2, 0),
                                                    (3, 4, 4, 4097, 0, 0), (40, 2, 9, 333, 5, 2)])
def test_rows_that_start_anywhere(dtype, m, top_k, E, n, pad, offset):
    """Row starts of every alignment in one call, with whole accesses between the rows' ends."""
    test_dispatch_and_its_gradient(dtype, m, top_k, E, n, pad, offset, 0.2)
    check_combine(Rows(m, top_k, E, 0.2, n + 1), dtype, n, n + pad, offset)


def check_combine(b, dtype, n, ld, offset):
    m, top_k, E = b.m, b.top_k, b.E
    ys = b.rng.standard_normal((b.rows, n))
    ys[b.valid:] = np.nan
    w = b.rng.standard_normal((m, top_k)).astype(np.float32)
    yb, yp, yv = strided(ys, ld, dtype, offset=offset)
    wb = floats(w)
    out, outp = empty(m, ld, dtype, offset)
    gb.check(gb.gbmm_moe_combine(dtype, m, top_k, E, n, yp, ld, wb.ptr, b.position, b.offsets, outp, ld))
    w64 = w.astype(np.float64)
    ref, mag = moe_ref.combine(np.nan_to_num(yv), w64, b.pos, b.valid, m, top_k)
    near(fetch(out, m, n, ld, dtype, offset), ref, U * (top_k + 1) * mag + UO[dtype] * np.abs(ref) + TINY[dtype], "y")

    gbuf, gp, g = strided(b.rng.standard_normal((m, n)), ld, dtype, offset=offset)
    dys, dysp = empty(b.rows, ld, dtype, offset)
    dw = DevBuf(b.rows * 4)
    gb.check(gb.gbmm_moe_combine_backward(dtype, m, top_k, E, n, yp, ld, wb.ptr, b.position, b.offsets, gp, ld, dysp,
                                          ld, dw.ptr))
    rdys, rdw, mag = moe_ref.combine_backward(np.nan_to_num(yv), w64, g, b.pos, b.valid, top_k)
    got = fetch(dys, b.rows, n, ld, dtype, offset)
    near(got, rdys, (U + UO[dtype]) * np.abs(rdys) + TINY[dtype], "d_ys")
    assert dw.guards_intact()
    near(dw.read(np.float32).reshape(m, top_k), rdw, U * (n + 1) * mag + 2.0 ** -149, "d_weights")


def test_gradients_are_adjoint_to_their_forward():
    """<dispatch(x), g> = <x, d_x(g)> and differences of combine in w and ys: both
    maps are linear, so a difference has no truncation error; small integers make
    every value exact."""
    b = Rows(9, 3, 5, 0.2, 1)
    n = 40
    integers = lambda *s: b.rng.integers(-4, 5, s).astype(np.float64)  # noqa: E731
    xb, xp, x = strided(integers(9, n), n, "f32")
    gbuf, gp, g = strided(integers(b.rows, n), n, "f32")
    xs, xsp = empty(b.rows, n, "f32")
    dx, dxp = empty(9, n, "f32")
    gb.check(gb.gbmm_moe_dispatch("f32", 9, 3, 5, n, xp, n, b.position, b.offsets, xsp, n))
    gb.check(gb.gbmm_moe_dispatch_backward("f32", 9, 3, 5, n, gp, n, b.position, b.offsets, dxp, n))
    live = np.arange(b.rows)[:, None] < b.valid
    assert (fetch(xs, b.rows, n, n, "f32") * g * live).sum() == (x * fetch(dx, 9, n, n, "f32")).sum()

    ys, w, dy = integers(b.rows, n), integers(9, 3), integers(9, n)

    def loss(ys, w):
        yb, yp, _ = strided(ys, n, "f32")
        wb = floats(w)
        out, outp = empty(9, n, "f32")
        gb.check(gb.gbmm_moe_combine("f32", 9, 3, 5, n, yp, n, wb.ptr, b.position, b.offsets, outp, n))
        return (fetch(out, 9, n, n, "f32") * dy).sum()

    yb, yp, _ = strided(ys, n, "f32")
    wb = floats(w)
    db, dp, _ = strided(dy, n, "f32")
    dys, dysp = empty(b.rows, n, "f32")
    dw = DevBuf(b.rows * 4)
    gb.check(gb.gbmm_moe_combine_backward("f32", 9, 3, 5, n, yp, n, wb.ptr, b.position, b.offsets, dp, n, dysp, n,
                                          dw.ptr))
    d_ys, d_w = fetch(dys, b.rows, n, n, "f32"), dw.read(np.float32).reshape(9, 3)
    for t, s in ((0, 0), (4, 2), (8, 1)):
        step = np.zeros_like(w)
        step[t, s] = 1
        assert loss(ys, w + step) - loss(ys, w) == d_w[t, s]
    for at, i in ((0, 0), (b.valid - 1, n - 1), (b.rows - 1, 3)):
        step = np.zeros_like(ys)
        step[at, i] = 1
        assert loss(ys + step, w) - loss(ys, w) == d_ys[at, i]


def test_empty_rows_and_zero_length():
    wb, dw = floats(np.ones((3, 2))), DevBuf(24)
    gb.check(gb.gbmm_moe_combine_backward("f16", 3, 2, 4, 0, None, 0, wb.ptr, None, None, None, 0, None, 0, dw.ptr))
    torch.cuda.synchronize()
    assert (dw.read(np.float32) == 0).all() and dw.guards_intact()


def test_offsets_past_32_bits():
    """Rows whose element offset passes 2^32: a wide leading dimension, f16."""
    free, _ = torch.cuda.mem_get_info()
    m, top_k, n, ld = 3, 3, 24, (1 << 29) + 8
    if free < 3 * m * top_k * ld * 2:
        pytest.skip("needs free device memory")
    ys = torch.empty(m * top_k * ld, dtype=torch.float16, device="cuda")
    dys = torch.empty(m * top_k * ld, dtype=torch.float16, device="cuda")
    b = Rows(m, top_k, 4, 0.0, 2)
    vals = torch.randn(b.rows, n, device="cuda").half()
    torch.as_strided(ys, (b.rows, n), (ld, 1)).copy_(vals)
    w = np.ones((m, top_k), np.float32)
    wb = floats(w)
    y = torch.empty(m, n, dtype=torch.float16, device="cuda")
    gb.check(gb.gbmm_moe_combine("f16", m, top_k, 4, n, ys, ld, wb.ptr, b.position, b.offsets, y, n))
    ref, mag = moe_ref.combine(vals.double().cpu().numpy(), w.astype(np.float64), b.pos, b.valid, m, top_k)
    near(y.double().cpu().numpy(), ref, U * (top_k + 1) * mag + UO["f16"] * np.abs(ref) + TINY["f16"], "y")
    dw = DevBuf(b.rows * 4)
    gb.check(gb.gbmm_moe_combine_backward("f16", m, top_k, 4, n, ys, ld, wb.ptr, b.position, b.offsets, y, n, dys, ld,
                                          dw.ptr))
    got = torch.as_strided(dys, (b.rows, n), (ld, 1)).double().cpu().numpy()
    assert np.array_equal(got, moe_ref.dispatch(y.double().cpu().numpy(), b.pos, b.valid, top_k))
    gb.check(gb.gbmm_moe_dispatch("f16", m, top_k, 4, n, y, n, b.position, b.offsets, ys, ld))
    got = torch.as_strided(ys, (b.rows, n), (ld, 1)).double().cpu().numpy()
    assert np.array_equal(got, moe_ref.dispatch(y.double().cpu().numpy(), b.pos, b.valid, top_k))


def test_another_stream_and_graph_capture():
    """The calls run on the stream they are given, and replay from a CUDA graph
    with new inputs."""
    m, E, top_k, n = 50, 12, 3, 72
    dev = torch.device("cuda")
    logits = torch.randn(m, E, device=dev)
    x = torch.randn(m, n, device=dev)
    ids = torch.empty(m, top_k, dtype=torch.int32, device=dev)
    w = torch.empty(m, top_k, device=dev)
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    order, pos = (torch.empty(m * top_k, dtype=torch.int32, device=dev) for _ in range(2))
    xs, y = torch.empty(m * top_k, n, device=dev), torch.empty(m, n, device=dev)
    need = gb.gbmm_moe_sort_scratch_bytes(m, top_k, E)[1]
    scratch = torch.empty(max(need, 4), dtype=torch.uint8, device=dev)

    def step(stream):
        gb.check(gb.gbmm_moe_route("f32", m, E, top_k, 1, logits, E, None, ids, w, stream))
        gb.check(gb.gbmm_moe_sort(m, top_k, E, ids, off, order, pos, scratch, need, stream))
        gb.check(gb.gbmm_moe_dispatch("f32", m, top_k, E, n, x, n, pos, off, xs, n, stream))
        gb.check(gb.gbmm_moe_combine("f32", m, top_k, E, n, xs, n, w, pos, off, y, n, stream))

    def verify():
        # the weights of a token sum to 1, so the way there and back returns x
        assert torch.allclose(y, x, rtol=0, atol=float(x.abs().max()) * (top_k + 8) * U * 4)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for seed in range(2):
        logits.copy_(torch.randn(m, E, device=dev))
        x.copy_(torch.randn(m, n, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        verify()


@pytest.mark.parametrize("m,n", [(40, 96), (2500, 1024), (40000, 24)])
def test_calls_back_to_back_on_the_same_buffers(m, n):
    """Router to combine and back again and again without a wait in between, every
    buffer overwritten by the next turn: the results are those of turns on their own."""
    E, k, turns = 16, 4, 12
    g = torch.Generator(device="cuda").manual_seed(m)
    xs_in = torch.randn(turns, m, n, generator=g, device="cuda")
    logits_in = torch.randn(turns, m, E, generator=g, device="cuda")
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    x, logits, y, d_x = new(m, n), new(m, E), new(m, n), new(m, n)
    ids, w, d_w = new(m, k, dtype=torch.int32), new(m, k), new(m, k)
    offsets, order, position = (new(c, dtype=torch.int32) for c in (E + 1, m * k, m * k))
    xs, d_xs = new(m * k, n), new(m * k, n)
    st, nbytes = gb.gbmm_moe_sort_scratch_bytes(m, k, E)
    gb.check(st)
    scratch = new(max(nbytes, 1), dtype=torch.uint8)

    def turn(i):
        x.copy_(xs_in[i])
        logits.copy_(logits_in[i])
        gb.check(gb.gbmm_moe_route("f32", m, E, k, gb.SOFTMAX_ALL, logits, E, None, ids, w))
        gb.check(gb.gbmm_moe_sort(m, k, E, ids, offsets, order, position, scratch, nbytes))
        gb.check(gb.gbmm_moe_dispatch("f32", m, k, E, n, x, n, position, offsets, xs, n))
        gb.check(gb.gbmm_moe_combine("f32", m, k, E, n, xs, n, w, position, offsets, y, n))
        gb.check(gb.gbmm_moe_combine_backward("f32", m, k, E, n, xs, n, w, position, offsets, y, n, d_xs, n, d_w))
        gb.check(gb.gbmm_moe_dispatch_backward("f32", m, k, E, n, d_xs, n, position, offsets, d_x, n))
        return y.clone(), d_x.clone(), d_w.clone()
    alone = []
    for i in range(turns):
        alone.append(turn(i))
        torch.cuda.synchronize()
    together = [turn(i) for i in range(turns)]
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    total = torch.softmax(logits_in[-1].double(), 1).topk(k).values.sum(1, keepdim=True)
    assert ((together[-1][0].double() - total * xs_in[-1].double()).abs() <= 1e-5 * xs_in[-1].abs() + 1e-30).all()
