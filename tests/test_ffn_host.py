"""Host-only refusals of the gated projection, the quantisation and the 8-bit
product: every rule of include/gbmm.h is checked before the first launch.  The
pointers are fake, aligned addresses, and every kernel is made unavailable, so a
call that passes its checks answers GBMM_ERR_KERNEL_UNAVAILABLE."""

import pytest

from gemv_moe_expert_gb300 import binding as gb
from gemv_moe_expert_gb300 import build as gbuild

BAD, OVERLAP, DTYPE, SCRATCH = (gb.GBMM_ERR_INVALID_ARGUMENT, gb.GBMM_ERR_OVERLAP, gb.GBMM_ERR_UNSUPPORTED_DTYPE,
                                gb.GBMM_ERR_SCRATCH)
PASSES = gb.GBMM_ERR_KERNEL_UNAVAILABLE
BASE, STEP = 1 << 40, 1 << 24
A, B, C, D, E, F, G, H, I, J, K = (BASE + i * STEP for i in range(11))


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


GATED = dict(dt="bf16", act=0, m=4, n=32, k=64, x=A, ldx=64, wg=B, wu=C, ldw=64, h=D, ldh=32, gate=E, up=F, lds=32,
             scratch=G, nbytes=1 << 20)
BACK = dict(dt="bf16", act=0, m=4, n=32, k=64, x=A, ldx=64, wg=B, wu=C, ldw=64, gate=D, up=E, lds=32, dh=F, lddh=32,
            dx=G, lddx=64, dwg=H, dwu=I, lddw=64, scratch=J, nbytes=1 << 20)
QUANT = dict(dt="f16", m=4, k=64, x=A, ldx=64, q=B, ldq=64, scale=C)
GEMM = dict(dt="f16", m=4, n=32, k=64, a=A, lda=64, sa=B, b=C, ldb=64, sb=D, c=E, ldc=32, scratch=F, nbytes=1 << 20)
CALLS = {"gated": (gb.gbmm_gated, GATED), "back": (gb.gbmm_gated_backward, BACK),
         "quant": (gb.gbmm_quantize_i8, QUANT), "gemm": (gb.gbmm_gemm_i8, GEMM)}
NAMES = {"gated": "gbmm_gated", "back": "gbmm_gated_backward", "quant": "gbmm_quantize_i8", "gemm": "gbmm_gemm_i8"}


@pytest.mark.parametrize("name", CALLS)
def test_accepts_and_names_the_kernel(name):
    assert call(*CALLS[name], {}) == PASSES
    assert NAMES[name] in gb.gbmm_last_error()


REFUSED = [
    ("gated", dict(dt=3), DTYPE), ("gated", dict(act=4), BAD), ("gated", dict(m=-1), BAD), ("gated", dict(n=-1), BAD),
    ("gated", dict(k=-1), BAD), ("gated", dict(m=1 << 31), BAD), ("gated", dict(k=1 << 31, ldx=1 << 31, ldw=1 << 31), BAD),
    ("gated", dict(ldx=63), BAD), ("gated", dict(ldw=63), BAD), ("gated", dict(ldh=31), BAD),
    ("gated", dict(lds=31), BAD), ("gated", dict(gate=0), BAD), ("gated", dict(up=0), BAD), ("gated", dict(x=0), BAD),
    ("gated", dict(wg=0), BAD), ("gated", dict(wu=0), BAD), ("gated", dict(h=0), BAD), ("gated", dict(x=A + 1), BAD),
    ("gated", dict(wu=C + 1), BAD), ("gated", dict(h=D + 1), BAD), ("gated", dict(ldx=1 << 62), BAD),
    ("gated", dict(h=A), OVERLAP), ("gated", dict(h=B + 4094), OVERLAP), ("gated", dict(h=E), OVERLAP),
    ("gated", dict(gate=F), OVERLAP), ("gated", dict(gate=F + 32), OVERLAP), ("gated", dict(up=C), OVERLAP),
    ("gated", dict(scratch=A), OVERLAP), ("gated", dict(scratch=D - 8), OVERLAP),
    ("gated", dict(lds=64, up=E + 62), OVERLAP), ("gated", dict(lds=64, up=E + 66), OVERLAP),
    ("back", dict(dt=9), DTYPE), ("back", dict(act=9), BAD), ("back", dict(m=-1), BAD), ("back", dict(n=1 << 31), BAD),
    ("back", dict(ldx=63), BAD), ("back", dict(ldw=63), BAD), ("back", dict(lds=31), BAD), ("back", dict(lddh=31), BAD),
    ("back", dict(lddx=63), BAD), ("back", dict(lddw=63), BAD), ("back", dict(dwg=0), BAD), ("back", dict(dwu=0), BAD),
    ("back", dict(x=0), BAD), ("back", dict(wg=0), BAD), ("back", dict(wu=0), BAD), ("back", dict(gate=0), BAD),
    ("back", dict(up=0), BAD), ("back", dict(dh=0), BAD), ("back", dict(dh=F + 1), BAD), ("back", dict(dx=G + 1), BAD),
    ("back", dict(dx=A), OVERLAP), ("back", dict(dwg=B), OVERLAP), ("back", dict(dwg=I + 2), OVERLAP),
    ("back", dict(dwu=J + 100), OVERLAP), ("back", dict(dx=F), OVERLAP), ("back", dict(scratch=C), OVERLAP),
    ("back", dict(scratch=0), SCRATCH), ("back", dict(nbytes=100), SCRATCH), ("back", dict(lddw=1 << 62), BAD),
    ("quant", dict(dt=3), DTYPE), ("quant", dict(m=-1), BAD), ("quant", dict(k=-1), BAD), ("quant", dict(ldx=63), BAD),
    ("quant", dict(ldq=63), BAD), ("quant", dict(x=0), BAD), ("quant", dict(q=0), BAD), ("quant", dict(scale=0), BAD),
    ("quant", dict(scale=C + 2), BAD), ("quant", dict(x=A + 1), BAD), ("quant", dict(q=A), OVERLAP),
    ("quant", dict(scale=A), OVERLAP), ("quant", dict(scale=B + 252), OVERLAP), ("quant", dict(m=1 << 31), BAD),
    ("gemm", dict(dt=3), DTYPE), ("gemm", dict(m=-1), BAD), ("gemm", dict(n=-1), BAD), ("gemm", dict(k=-1), BAD),
    ("gemm", dict(k=131072, lda=131072, ldb=131072), BAD), ("gemm", dict(lda=63), BAD), ("gemm", dict(ldb=63), BAD),
    ("gemm", dict(ldc=31), BAD), ("gemm", dict(a=0), BAD), ("gemm", dict(b=0), BAD), ("gemm", dict(c=0), BAD),
    ("gemm", dict(c=E + 1), BAD), ("gemm", dict(sa=B + 2), BAD), ("gemm", dict(sb=D + 1), BAD),
    ("gemm", dict(c=A), OVERLAP), ("gemm", dict(c=B), OVERLAP), ("gemm", dict(c=C + 2046), OVERLAP),
    ("gemm", dict(c=D + 124), OVERLAP), ("gemm", dict(scratch=C), OVERLAP), ("gemm", dict(lda=1 << 62), BAD),
]


@pytest.mark.parametrize("name,over,status", REFUSED, ids=[f"{n}-{o}" for n, o, _ in REFUSED])
def test_refuses(name, over, status):
    assert call(*CALLS[name], over) == status, gb.gbmm_last_error()
    assert gb.gbmm_last_error() != ""


@pytest.mark.parametrize("name,over", [
    ("gated", dict(gate=0, up=0)), ("gated", dict(gate=0, up=0, lds=0)), ("gated", dict(scratch=0, nbytes=0)),
    ("gated", dict(k=0, x=0, wg=0, wu=0, ldx=0, ldw=0)),
    ("gated", dict(lds=64, up=E + 64)),            # both projections in one [m, 2 n] matrix
    ("gated", dict(lds=64, gate=E + 64, up=E)),
    ("gated", dict(ldh=96, lds=96, h=D, gate=D + 64, up=D + 128)),
    ("gated", dict(wu=B + 64 * 64 * 2)), ("gated", dict(ldw=128, wu=B + 128)),
    ("back", dict(dx=0, lddx=0)), ("back", dict(dx=0, wg=0, wu=0, ldw=0)), ("back", dict(dwg=0, dwu=0, lddw=0)),
    ("back", dict(dwg=0, dwu=0, x=0, ldx=0)), ("back", dict(lddw=128, dwu=H + 128)),
    ("back", dict(m=0, x=0, gate=0, up=0, dh=0, scratch=0, nbytes=0)),
    ("back", dict(n=0, wg=0, wu=0, gate=0, up=0, dh=0, scratch=0, nbytes=0)),
    ("quant", dict(k=0, x=0, q=0, ldx=0, ldq=0)), ("quant", dict(q=B + 1, ldq=67)),
    ("gemm", dict(sa=0, sb=0)), ("gemm", dict(a=A + 1, lda=65, b=C + 3, ldb=71)), ("gemm", dict(k=131071, lda=131071, ldb=131071)),
    ("gemm", dict(k=0, a=0, b=0, lda=0, ldb=0)),
])
def test_optional_operands(name, over):
    assert call(*CALLS[name], over) == PASSES, gb.gbmm_last_error()


@pytest.mark.parametrize("name,over", [
    ("gated", dict(m=0)), ("gated", dict(n=0)), ("back", dict(k=0)), ("back", dict(dx=0, dwg=0, dwu=0)),
    ("back", dict(m=0, dwg=0, dwu=0)), ("back", dict(n=0, dx=0)), ("back", dict(m=0, n=0)), ("quant", dict(m=0)),
    ("gemm", dict(m=0)), ("gemm", dict(n=0)),
])
def test_nothing_to_do_is_a_no_op(name, over):
    assert call(*CALLS[name], over) == gb.GBMM_OK, gb.gbmm_last_error()


def test_scratch_sizes():
    for fn in (gb.gbmm_gated_scratch_bytes, gb.gbmm_gated_backward_scratch_bytes):
        assert fn(5, 4, 4, 4, True)[0] == DTYPE
        assert fn("bf16", -1, 4, 4, True)[0] == BAD
        assert fn("bf16", 4, 1 << 31, 4, True)[0] == BAD
        assert fn("bf16", (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1, False)[0] == BAD
        for aligned in (False, True):
            sizes = [fn("bf16", m, 1000, 1000, aligned) for m in (0, 1, 1000, 100000)]
            assert all(st == gb.GBMM_OK for st, _ in sizes) and [v for _, v in sizes] == sorted(v for _, v in sizes)
        assert fn("bf16", 1000, 1000, 1000, True)[1] < fn("bf16", 1000, 1000, 1000, False)[1]
        assert fn("f32", 1000, 1000, 1000, True)[1] == fn("f32", 1000, 1000, 1000, False)[1]
    # few rows times few weights need none, many do
    assert gb.gbmm_gated_scratch_bytes("f16", 8, 1000, 1000, False) == (gb.GBMM_OK, 0)
    assert gb.gbmm_gated_scratch_bytes("f16", 8, 10000, 10000, False)[1] > 2 * 2 * 10000 * 10000
    assert gb.gbmm_gemm_i8_scratch_bytes(8, 1000, 1000, False) == (gb.GBMM_OK, 0)
    assert gb.gbmm_gemm_i8_scratch_bytes(8, 10000, 10000, False)[1] > 10000 * 10000
    # rows that do not start on multiples of 16 bytes
    need = gb.gbmm_gated_scratch_bytes("bf16", 40, 32, 64, False)[1]
    over = dict(m=40, ldx=65, ldw=65)
    assert call(*CALLS["gated"], dict(over, nbytes=need)) == PASSES
    assert call(*CALLS["gated"], dict(over, nbytes=need - 1)) == SCRATCH
    assert call(*CALLS["gated"], dict(over, scratch=0, nbytes=0)) == PASSES
    need = gb.gbmm_gated_backward_scratch_bytes("bf16", 4, 32, 64, False)[1]
    over = dict(ldx=65, ldw=65)
    assert call(*CALLS["back"], dict(over, nbytes=need)) == PASSES
    assert call(*CALLS["back"], dict(over, nbytes=need - 1)) == SCRATCH
    assert gb.gbmm_gemm_i8_scratch_bytes(1, 1, gb.I8_MAX_K + 1, True)[0] == BAD
    assert gb.gbmm_gemm_i8_scratch_bytes(-1, 1, 1, True)[0] == BAD
    assert gb.gbmm_gemm_i8_scratch_bytes(1 << 31, 1, 1, True)[0] == BAD
    for m, n, k in ((4, 32, 64), (40, 32, 64), (40, 33, 1003), (100, 7, 131071), (1000, 1001, 1003), (100000, 7, 131071)):
        sizes = []
        for ld in (-(-k // 16) * 16, k | 1):
            st, need = gb.gbmm_gemm_i8_scratch_bytes(m, n, k, ld % 16 == 0)
            assert st == gb.GBMM_OK
            far = dict(m=m, n=n, k=k, lda=ld, ldb=ld, ldc=n, a=BASE, b=BASE << 1, c=BASE << 2, scratch=BASE << 3, sa=0,
                       sb=0)
            assert call(*CALLS["gemm"], dict(far, nbytes=need)) == PASSES
            if need:
                assert call(*CALLS["gemm"], dict(far, nbytes=need - 1)) == SCRATCH
                assert call(*CALLS["gemm"], dict(far, nbytes=need, scratch=0)) == SCRATCH
            sizes.append(need)
        assert sizes[0] <= sizes[1]
    st, need = gb.gbmm_gated_backward_scratch_bytes("bf16", 4, 32, 64, True)
    assert call(*CALLS["back"], dict(nbytes=need)) == PASSES
    assert call(*CALLS["back"], dict(nbytes=need - 1)) == SCRATCH


@pytest.mark.parametrize("kernel", ["gbmm_gated_backward", "gbmm_fill_zero"])
def test_backward_asks_for_its_kernels_first(kernel):
    gb.gbmm_test_inject_kernel_failure(kernel)
    assert call(*CALLS["back"], {}) == PASSES and kernel in gb.gbmm_last_error()
    gb.gbmm_test_inject_kernel_failure("*")


GATED_FORM, CODES_FORM, SUM_FORM = 0, 1, 2


def needed_columns(form, tokens, cluster, k):
    """Tensor-memory columns of one CTA: one f32 accumulator of `tokens` columns; for codes one for each 1024 of its
    share of k, in whole blocks of 128, beside 128 columns of weights."""
    if form != CODES_FORM:
        return tokens
    share = -(-(-(-k // 128)) // cluster)
    return 128 + -(-share // 8) * tokens


@pytest.mark.parametrize("sms", [152, 148, 16, 2, 1])
@pytest.mark.parametrize("form", [GATED_FORM, CODES_FORM, SUM_FORM])
def test_ctas_of_an_sm_share_its_tensor_memory(form, sms):
    """A CTA that waits for columns waits without a limit: the CTAs that an SM holds never ask for more than 512."""
    edges = [e + d for e in (1, 8, 16, 32, 64, 128, 256, 512, 600) for d in (-1, 0, 1) if e + d > 0]
    lengths = [1, 64, 127, 128, 129, 1000, 1024, 1025, 2048, 4096, 11008]
    lengths += [1024 * e + d for e in (8, 12, 16, 20, 24, 32, 48, 64, 96, 120) for d in (-1, 0, 1)]
    lengths += [18944, 20000, 131071]
    seen = 0
    for m in edges:
        for n in (1, 70, 128, 1000, 2048, 3584, 4096, 8192, 11008, 100000):
            for k in lengths:
                st, (tokens, cluster, columns, held) = gb.gbmm_test_few_plan(form, m, n, k, sms)
                assert st == gb.GBMM_OK
                if tokens == 0:
                    continue
                seen += 1
                size = (m, n, k)
                assert tokens in (16, 32, 64, 128) and 1 <= cluster <= 8 and held in (1, 2), size
                assert needed_columns(form, tokens, cluster, k) <= columns, size
                assert columns >= 32 and columns & (columns - 1) == 0 and columns * held <= 512, size
    assert seen > 500


def test_the_long_sums_of_some_tens_of_tokens_take_wide_tiles():
    """33 to 64 tokens over more than 16384 codes: three accumulators of 64 tokens would fill an SM's tensor memory
    twice over, so that such tiles are 128 tokens wide and have their SM to themselves."""
    for m in (33, 40, 48, 64):
        for k in (16385, 18944, 20000, 24576):
            assert gb.gbmm_test_few_plan(CODES_FORM, m, 3584, k, 152)[1][0] == 128
        assert gb.gbmm_test_few_plan(CODES_FORM, m, 3584, 16384, 152)[1][0] == 64
        assert gb.gbmm_test_few_plan(CODES_FORM, m, 3584, 24577, 152)[1][0] == 0
    assert gb.gbmm_test_few_plan(3, 1, 1, 1, 152)[0] == BAD and gb.gbmm_test_few_plan(0, 0, 1, 1, 152)[0] == BAD


@pytest.mark.parametrize("need_x,need_w", [(True, True), (True, False), (False, True)])
def test_no_chain_of_an_f32_gradient_outlasts_an_equal_share(need_x, need_w):
    """A block's work, in products of a step, against an SM's share of all: at most twice that (two blocks lie on an
    SM), or a contraction divided by eight, or, where there is little to do, 64 steps of a small tile.
    Where blocks wait for a place, chains that are much longer come first."""
    sms = 152
    for m in (1, 5, 26, 49, 130, 500, 1000, 2346, 4000, 8192):
        for n in (64, 192, 512, 892, 1408, 3136, 5504, 9664, 11008):
            for k in (64, 320, 384, 686, 960, 2048, 4096, 11008):
                st, (edge, x_parts, w_parts, w_first) = gb.gbmm_test_gradient_plan(m, n, k, need_x, need_w, sms)
                assert st == gb.GBMM_OK and edge in (64, 128) and 1 <= x_parts <= 8 and 1 <= w_parts <= 8
                x_tiles = -(-m // edge) * -(-k // edge) * need_x
                w_tiles = -(-n // 64) * -(-k // edge) * need_w
                x_steps, w_steps = 2 * -(-n // 16), -(-m // 16)
                x_cost, w_cost = edge * edge, 2 * 64 * edge  # of a step
                share = (x_tiles * x_steps * x_cost + w_tiles * w_steps * w_cost) / sms
                x_chain, w_chain = -(-x_steps // x_parts) * x_cost * need_x, -(-w_steps // w_parts) * w_cost * need_w
                for chain, parts, cost in ((x_chain, x_parts, x_cost), (w_chain, w_parts, w_cost)):
                    assert chain <= 2 * share or parts == 8 or chain <= 64 * 64 * 64, (m, n, k, edge, x_parts, w_parts)
                blocks = x_tiles * x_parts + w_tiles * w_parts
                if need_x and need_w and blocks > 2 * sms and max(x_chain, w_chain) > 2.5 * min(x_chain, w_chain):
                    assert w_first == (w_chain > x_chain), (m, n, k)
    assert gb.gbmm_test_gradient_plan(1, 1, 1, False, False, sms)[0] == BAD
    assert gb.gbmm_test_gradient_plan(0, 1, 1, True, True, sms)[0] == BAD


def test_f32_projections_are_divided_about_evenly():
    """Tiles of 128 or 64 rows (1394 and 819 ns a step), divided over one to eight CTAs (the exchange as six steps): the
    rounds of the plan taken come to at most 1.4 times the least of all of them, and two steps."""
    sms = 152

    def time(m, n, k, height, parts):
        tiles = -(-m // height) * -(-n // 64)
        steps = -(--(-k // 16) // parts) + (6 if parts > 1 else 0)
        return -(-tiles * parts // sms) * steps * (1394 if height == 128 else 819)

    for m in (9, 10, 44, 66, 143, 272, 512, 890, 2512, 4356, 6469):
        for n in (64, 203, 231, 704, 1408, 2816, 4217, 7374, 10169):
            for k in (25, 64, 512, 1408, 2048, 2512, 4928, 7616):
                st, (height, parts) = gb.gbmm_test_gated_plan(m, n, k, sms)
                assert st == gb.GBMM_OK and height in (64, 128) and 1 <= parts <= 8
                least = min(time(m, n, k, h, p) for h in (64, 128) for p in range(1, 9))
                assert time(m, n, k, height, parts) <= 1.4 * least + 2 * 1394, (m, n, k, height, parts)
    assert gb.gbmm_test_gated_plan(8, 1, 1, sms)[0] == BAD
