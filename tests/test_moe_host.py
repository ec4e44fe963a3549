"""Host-only refusals of the mixture-of-experts and 4-bit entry points: every
rule of include/gbmm.h is checked before the first launch.  The pointers are
fake, aligned addresses, and every kernel is made unavailable, so a call that
passes its checks answers GBMM_ERR_KERNEL_UNAVAILABLE."""

import pytest

from gemv_moe_expert_gb300 import binding as gb
from gemv_moe_expert_gb300 import build as gbuild

BAD, OVERLAP, DTYPE = gb.GBMM_ERR_INVALID_ARGUMENT, gb.GBMM_ERR_OVERLAP, gb.GBMM_ERR_UNSUPPORTED_DTYPE
PASSES = gb.GBMM_ERR_KERNEL_UNAVAILABLE
BASE, STEP = 1 << 40, 1 << 24
A, B, C, D, E, F, G = (BASE + i * STEP for i in range(7))


@pytest.fixture(autouse=True)
def _no_kernel_may_launch():
    gbuild.build()
    gb.load()
    gb.gbmm_test_inject_kernel_failure("*")
    gb.gbmm_test_reset_launch_count()
    yield
    assert gb.gbmm_test_launch_count() == 0
    gb.gbmm_test_inject_kernel_failure(None)


def call(fn, defaults, over):
    args = dict(defaults)
    assert set(over) <= set(args), over
    args.update(over)
    return fn(*args.values(), stream=0)


ROUTE = dict(dt="f32", m=4, E=64, k=8, softmax=0, logits=A, ld=64, bias=B, ids=C, weights=D)
ROUTE_BACK = dict(dt="f32", m=4, E=64, k=8, softmax=0, logits=A, ld=64, bias=B, ids=C, weights=D, dw=E, dl=F, ldd=64)
SORT = dict(m=4, k=8, E=64, ids=A, offsets=B, order=C, position=D, scratch=E, nbytes=1 << 20)
DISPATCH = dict(dt="f32", m=4, k=8, E=64, n=32, x=A, ldx=32, position=B, offsets=C, xs=D, ldxs=32)
DISPATCH_BACK = dict(dt="f32", m=4, k=8, E=64, n=32, dxs=A, ldxs=32, position=B, offsets=C, dx=D, ldx=32)
COMBINE = dict(dt="f32", m=4, k=8, E=64, n=32, ys=A, ldys=32, weights=B, position=C, offsets=D, y=E, ldy=32)
COMBINE_BACK = dict(dt="f32", m=4, k=8, E=64, n=32, ys=A, ldys=32, weights=B, position=C, offsets=D, dy=E, lddy=32,
                    dys=F, lddys=32, dw=G)
GEMV = dict(dt="f16", m=4, n=32, k=64, group=32, q=A, ldq=32, scales=B, sdt="f16", zeros=C, x=D, ldx=64, y=E, ldy=32)
MID = dict(dt="f16", m=4, n=32, k=64, top_k=2, E=8, layout=0, group=32, q=A, ldq=32, stride=1024, scales=B, sdt="f16",
           zeros=C, x=D, ids=E, out=F)
CALLS = {"route": (gb.gbmm_moe_route, ROUTE), "route_backward": (gb.gbmm_moe_route_backward, ROUTE_BACK),
         "sort": (gb.gbmm_moe_sort, SORT), "dispatch": (gb.gbmm_moe_dispatch, DISPATCH),
         "dispatch_backward": (gb.gbmm_moe_dispatch_backward, DISPATCH_BACK),
         "combine": (gb.gbmm_moe_combine, COMBINE), "combine_backward": (gb.gbmm_moe_combine_backward, COMBINE_BACK),
         "gemv_q4": (gb.gbmm_gemv_q4, GEMV), "matmul_id_q4": (gb.gbmm_matmul_id_q4, MID)}
NAMES = {"route": "gbmm_moe_route", "route_backward": "gbmm_moe_route_backward", "sort": "gbmm_moe_sort",
         "dispatch": "gbmm_moe_dispatch", "dispatch_backward": "gbmm_moe_dispatch_backward",
         "combine": "gbmm_moe_combine", "combine_backward": "gbmm_moe_combine_backward", "gemv_q4": "gbmm_gemv_q4",
         "matmul_id_q4": "gbmm_matmul_id_q4"}


@pytest.mark.parametrize("name", CALLS)
def test_accepts_and_names_the_kernel(name):
    assert call(*CALLS[name], {}) == PASSES
    assert NAMES[name] in gb.gbmm_last_error()


REFUSED = [
    ("route", dict(dt=5), DTYPE), ("route", dict(E=0, k=1), BAD), ("route", dict(k=0), BAD),
    ("route", dict(E=1025, ld=1025), BAD), ("route", dict(k=33), BAD), ("route", dict(E=4, k=5), BAD),
    ("route", dict(softmax=2), BAD), ("route", dict(ld=63), BAD), ("route", dict(ld=-1), BAD),
    ("route", dict(m=1 << 31), BAD), ("route", dict(m=1 << 28), BAD), ("route", dict(ld=1 << 61), BAD),
    ("route", dict(logits=0), BAD), ("route", dict(logits=A + 2), BAD), ("route", dict(ids=0), BAD),
    ("route", dict(weights=D + 1), BAD), ("route", dict(bias=B + 2), BAD), ("route", dict(ids=A + 1020), OVERLAP),
    ("route", dict(weights=C + 124), OVERLAP), ("route", dict(ids=B), OVERLAP),
    ("route_backward", dict(dt=9), DTYPE), ("route_backward", dict(ld=63), BAD), ("route_backward", dict(ldd=63), BAD),
    ("route_backward", dict(logits=0), BAD), ("route_backward", dict(ids=0), BAD), ("route_backward", dict(dw=0), BAD),
    ("route_backward", dict(dl=A), OVERLAP), ("route_backward", dict(dl=E - 4), OVERLAP),
    ("route_backward", dict(dl=0), BAD), ("route_backward", dict(softmax=7), BAD),
    ("sort", dict(k=0), BAD), ("sort", dict(E=0), BAD), ("sort", dict(E=1025), BAD), ("sort", dict(m=1 << 30), BAD),
    ("sort", dict(ids=0), BAD), ("sort", dict(offsets=B + 2), BAD), ("sort", dict(order=0), BAD),
    ("sort", dict(order=A), OVERLAP), ("sort", dict(position=C), OVERLAP), ("sort", dict(offsets=D + 124), OVERLAP),
    ("dispatch", dict(dt=3), DTYPE), ("dispatch", dict(n=-1), BAD), ("dispatch", dict(ldx=31), BAD),
    ("dispatch", dict(ldxs=31), BAD), ("dispatch", dict(offsets=0), BAD), ("dispatch", dict(position=0), BAD),
    ("dispatch", dict(x=0), BAD), ("dispatch", dict(x=A + 2), BAD), ("dispatch", dict(xs=A + 16), OVERLAP),
    ("dispatch", dict(xs=C), OVERLAP), ("dispatch", dict(m=1 << 29), BAD), ("dispatch", dict(ldx=1 << 62), BAD),
    ("dispatch", dict(E=0), BAD), ("dispatch", dict(E=2000), BAD),
    ("dispatch_backward", dict(dt=3), DTYPE), ("dispatch_backward", dict(dx=A), OVERLAP),
    ("dispatch_backward", dict(ldx=0), BAD), ("dispatch_backward", dict(dxs=0), BAD),
    ("combine", dict(weights=0), BAD), ("combine", dict(weights=B + 2), BAD), ("combine", dict(ldys=5), BAD),
    ("combine", dict(y=A), OVERLAP), ("combine", dict(y=B), OVERLAP), ("combine", dict(dt=-1), DTYPE),
    ("combine", dict(position=0), BAD), ("combine", dict(k=0), BAD),
    ("combine_backward", dict(dw=0), BAD), ("combine_backward", dict(dw=B), OVERLAP),
    ("combine_backward", dict(dys=A), OVERLAP), ("combine_backward", dict(dys=E), OVERLAP),
    ("combine_backward", dict(lddys=31), BAD), ("combine_backward", dict(lddy=31), BAD),
    ("combine_backward", dict(dys=0), BAD), ("combine_backward", dict(dw=F + 16), OVERLAP),
    ("gemv_q4", dict(dt=3), DTYPE), ("gemv_q4", dict(sdt=3), DTYPE), ("gemv_q4", dict(group=16), BAD),
    ("gemv_q4", dict(group=0), BAD), ("gemv_q4", dict(n=-1), BAD), ("gemv_q4", dict(k=-1), BAD),
    ("gemv_q4", dict(k=1 << 31, ldq=1 << 30, ldx=1 << 31), BAD), ("gemv_q4", dict(ldq=31), BAD),
    ("gemv_q4", dict(ldx=63), BAD), ("gemv_q4", dict(ldy=31), BAD), ("gemv_q4", dict(q=0), BAD),
    ("gemv_q4", dict(scales=0), BAD), ("gemv_q4", dict(scales=B + 1), BAD), ("gemv_q4", dict(x=0), BAD),
    ("gemv_q4", dict(x=D + 1), BAD), ("gemv_q4", dict(y=D), OVERLAP), ("gemv_q4", dict(y=A + 992), OVERLAP),
    ("gemv_q4", dict(y=B - 2), OVERLAP), ("gemv_q4", dict(y=C), OVERLAP), ("gemv_q4", dict(ldq=1 << 62), BAD),
    ("gemv_q4", dict(m=1 << 31), BAD),
    ("matmul_id_q4", dict(dt=3), DTYPE), ("matmul_id_q4", dict(layout=2), BAD), ("matmul_id_q4", dict(stride=1023), BAD),
    ("matmul_id_q4", dict(stride=-1), BAD), ("matmul_id_q4", dict(top_k=0), BAD), ("matmul_id_q4", dict(E=0), BAD),
    ("matmul_id_q4", dict(E=1025), BAD), ("matmul_id_q4", dict(group=96), BAD), ("matmul_id_q4", dict(ids=0), BAD),
    ("matmul_id_q4", dict(ids=E + 2), BAD), ("matmul_id_q4", dict(out=E), OVERLAP), ("matmul_id_q4", dict(out=D), OVERLAP),
    ("matmul_id_q4", dict(out=A + 8 * 1024 - 2), OVERLAP), ("matmul_id_q4", dict(stride=1 << 62), BAD),
    ("matmul_id_q4", dict(m=1 << 31), BAD),
]


@pytest.mark.parametrize("name,over,status", REFUSED, ids=[f"{n}-{o}" for n, o, _ in REFUSED])
def test_refuses(name, over, status):
    assert call(*CALLS[name], over) == status, gb.gbmm_last_error()
    assert gb.gbmm_last_error() != ""


@pytest.mark.parametrize("name,over", [
    ("route", dict(bias=0)), ("route", dict(k=32)), ("route", dict(E=1024, ld=1024)),
    ("route_backward", dict(bias=0)), ("route_backward", dict(softmax=1, logits=0, ld=0, bias=0)),
    ("route_backward", dict(softmax=1, logits=3, bias=1)),
    ("dispatch", dict(position=0, offsets=0)), ("combine", dict(position=0, offsets=0)),
    ("combine_backward", dict(n=0, ys=0, ldys=0, dy=0, lddy=0, dys=0, lddys=0)),
    ("gemv_q4", dict(zeros=0)), ("gemv_q4", dict(k=0, q=0, ldq=0, scales=0, zeros=0, x=0, ldx=0)),
    ("gemv_q4", dict(q=A + 1, ldq=33)), ("matmul_id_q4", dict(layout=1)), ("matmul_id_q4", dict(zeros=0)),
    ("sort", dict(m=0, ids=0, order=0, position=0)),
])
def test_optional_operands(name, over):
    assert call(*CALLS[name], over) == PASSES, gb.gbmm_last_error()


@pytest.mark.parametrize("name", [n for n in CALLS if n != "sort"])
def test_no_tokens_is_a_no_op(name):
    assert call(*CALLS[name], dict(m=0)) == gb.GBMM_OK


@pytest.mark.parametrize("name", ["dispatch", "dispatch_backward", "combine", "gemv_q4", "matmul_id_q4"])
def test_no_columns_is_a_no_op(name):
    assert call(*CALLS[name], dict(n=0)) == gb.GBMM_OK


def test_sort_scratch():
    assert gb.gbmm_moe_sort_scratch_bytes(4, 0, 8)[0] == BAD
    assert gb.gbmm_moe_sort_scratch_bytes(1 << 30, 2, 8)[0] == BAD
    sizes = []
    for m in (0, 1, 1000, 100000, 1000000):
        st, need = gb.gbmm_moe_sort_scratch_bytes(m, 8, 1024)
        assert st == gb.GBMM_OK
        sizes.append(need)
        if need:
            assert call(*CALLS["sort"], dict(m=m, E=1024, nbytes=need - 1)) == gb.GBMM_ERR_SCRATCH
            assert call(*CALLS["sort"], dict(m=m, E=1024, nbytes=need, scratch=0)) == gb.GBMM_ERR_SCRATCH
    assert sizes == sorted(sizes)
    st, need = gb.gbmm_moe_sort_scratch_bytes(100000, 8, 64)
    far = dict(m=100000, order=BASE + 8 * STEP, position=BASE + 16 * STEP, nbytes=need)
    assert call(*CALLS["sort"], {**far, "scratch": BASE + 16 * STEP}) == OVERLAP
    assert call(*CALLS["sort"], {**far, "scratch": BASE + 24 * STEP + 2}) == BAD
    assert call(*CALLS["sort"], {**far, "scratch": BASE + 24 * STEP}) == PASSES
