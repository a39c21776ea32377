"""The serving operators where a launch's workgroups take more than one share each."""
import numpy as np
import pytest

from test_gpu_cache_plan import check as check_plan
from test_gpu_cache_plan import make as make_plan
from test_gpu_lora import check as check_lora
from test_gpu_lora import make as make_lora
from test_gpu_lora import run as run_lora

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_of_more_tokens_than_threads(in_place):
    # threads of 512 workgroups (two per compute unit) at most: 262,144
    case = make_plan([8], 400, 16, 400, 0.97, 5500)
    total = int(np.maximum(case[1], 0).sum())
    assert total > 262144
    check_plan(case, 16, total + 1000, in_place=in_place)


@pytest.mark.parametrize("x16", [True, False])
def test_adapters_of_more_rows_than_a_grid_dimension_of_the_row_kernels(x16):
    tokens = 65535 + 300
    ids = np.random.default_rng(5).integers(-1, 3, tokens)
    c = make_lora([51], [(16, 24)], 5, tokens, 3, ids, x16, x16)
    check_lora(c, run_lora(c))
    check_lora(c, run_lora(c, in_place=True))


def test_adapters_of_very_many_rows_on_the_matrix_cores():
    tokens = 70001
    ids = np.random.default_rng(6).integers(-1, 4, tokens)
    c = make_lora([52], [(64, 72)], 16, tokens, 4, ids)
    check_lora(c, run_lora(c))
