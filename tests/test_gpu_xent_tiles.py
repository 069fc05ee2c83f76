"""Every test of the linear layer with cross entropy again with its 256 x 256
tiles at every size (small ones otherwise run the few-token kernels), and both
ways around the sizes where they change."""

import pytest

from tests.test_gpu_xent import *  # noqa: F401,F403
from tests.test_gpu_xent import _gpu, check, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _tiles(_gpu, request):
    from ternary_weight_quantization_amd import binding as B

    B.bitnet_set_test_knobs(no_skinny=0 if "either_side" in request.node.name else 1)
    yield
    B.bitnet_set_test_knobs()


# 512 groups of 64 tokens and 64 columns are the most the few-token kernels take
@pytest.mark.parametrize("T,V", [(65, 16384), (65, 16385), (128, 16384), (129, 10880), (129, 10881), (256, 8192),
                                 (257, 8192), (512, 4096), (513, 3700), (1000, 2048), (1000, 2049), (3000, 640),
                                 (3000, 705), (32768, 1), (32769, 1), (5000, 100)])
def test_either_side_of_the_choice(T, V):
    check(*make(T, V, 136, seed=T + V, ignored=T // 4))


@pytest.mark.parametrize("T", [65, 79, 80, 81, 127, 129, 191, 192, 193, 250])
def test_either_side_groups_of_tokens(T):
    """Broken groups of 64 and of 16 tokens, with and without rows that do not
    count, widths that are padded."""
    check(*make(T, 700, 200, seed=T))
    check(*make(T, 6500, 72, seed=T, ignored=T // 2), reduction="mean")
    check(*make(T, 333, 77, seed=T, ignored=3), reduction="sum")


@pytest.mark.parametrize("T", [1, 16, 17, 33, 49, 64, 70, 200])
@pytest.mark.parametrize("V,D", [(1, 9), (63, 203), (130, 2555), (2000, 77), (25000, 75)])
def test_either_side_odd_widths(T, V, D):
    """Rows that are not whole chunks, read in place by the loss, each number
    of groups and both tile heights."""
    check(*make(T, V, D, seed=T + V, ignored=T // 3), reduction="sum")
