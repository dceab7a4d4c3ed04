"""Windows of ``paged_prompt_attention`` that hide nothing, up to the largest number, for sequences with fewer tokens than rows."""
import pytest
import torch

from test_gpu_prompt_attention import _check

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# (any larger window is taken as 2^31 - 1)
@pytest.mark.parametrize("window", [2 ** 40, 2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 200, 4096, 150])
@pytest.mark.parametrize("sinks", [0, 3])
@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_rows_before_the_first_token(window, sinks, cache):
    _check([5], [3], 4, 2, 64, 16, cache, window, sinks)
    _check([200, 300, 7], [150, 1, 7], 4, 2, 64, 16, cache, window, sinks)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 130, 1300])
def test_long_contexts_among_them(window):
    # 1300 tokens fill 82 pages but 12 slots: a window of 1300 hides nothing either
    _check([130, 4, 40], [129, 1300, 9], 4, 2, 128, 16, BF16, window, 2)
