"""GPU tests of the group norm's gradients for a bias without a weight, with the
bounds of the running error analysis."""

import pytest

from tests.test_gpu_group_norm import F32, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,T,G,D", [(1, 1, 16, 128), (1, 2, 16, 80), (2, 5, 3, 40), (1, 100, 16, 128), (1, 1024, 2, 520),
                                     (1, 7, 1, 2048)])
def test_a_bias_alone(B, T, G, D, shared):
    i = make(T, B, T, G, D, F32, shared=shared, gated=False)
    i["w"] = None
    check(i, G, "silu", False)
