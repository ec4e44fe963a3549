"""GPU tests of the token sort's launches: refusals before the first of several, and
the largest clusters of the one-launch form."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_moe_expert_gb300 import binding as gb  # noqa: E402
from tests.gpu_util import SENTINEL, DevBuf  # noqa: E402
from tests.test_gpu_moe import check_sort, ints  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemv_moe_expert_gb300 import build
    build.build()
    gb.load()
    torch.cuda.init()


def test_a_sort_that_cannot_finish_launches_nothing():
    m, top_k, E = 6000, 8, 16
    ib = ints(np.random.default_rng(5).integers(0, E, (m, top_k)))
    need = gb.gbmm_moe_sort_scratch_bytes(m, top_k, E)[1]
    assert need > 0  # the form with several launches
    outs = [DevBuf((E + 1) * 4), DevBuf(m * top_k * 4), DevBuf(m * top_k * 4), DevBuf(need)]
    args = (m, top_k, E, ib.ptr, *(b.ptr for b in outs), need)
    gb.gbmm_test_reset_launch_count()
    gb.gbmm_test_inject_kernel_failure("gbmm_moe_sort_place")
    assert gb.gbmm_moe_sort(*args) == gb.GBMM_ERR_KERNEL_UNAVAILABLE
    assert gb.gbmm_test_launch_count() == 0
    torch.cuda.synchronize()
    for b in outs:
        assert (b.read(np.uint8) == SENTINEL).all()
    gb.check(gb.gbmm_moe_sort(*args))
    assert gb.gbmm_test_launch_count() == 3


@pytest.mark.parametrize("m,top_k,E", [(4096, 8, 1024), (2341, 7, 1024), (32768, 1, 1023), (3750, 8, 1000)])
def test_clusters_of_the_most_ctas_with_the_most_experts(m, top_k, E):
    """9 to 16 CTAs, each with nearly all of an SM's shared memory."""
    rng = np.random.default_rng(m + E)
    check_sort(rng.integers(0, E + 1, (m, top_k)).astype(np.uint32), E)
