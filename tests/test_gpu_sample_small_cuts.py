"""Cuts so small that only whole numbers of 2^-44 of the largest weight are left of them."""
import math

import pytest
import torch

from test_gpu_sample import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("e", [39, 40, 41, 42, 43, 44, 50, 149])
def test_min_p_of_exactly_a_weight(dtype, e):
    """min_p = 2^-e; weights of 1, of 2^-min(e, 44) and of a quarter of that: with T = log2(e) a weight is 2^x, to 2^-18 of itself,
    which its rounding to whole 2^-44 takes away. What is kept ends with the tokens that have the bound's own weight (a bound below
    2^-44 counts as that); u = 1 takes the last of them."""
    t = float(torch.tensor(1 / math.log(2), dtype=torch.float32))
    low = min(e, 44)
    x = torch.full((1, 300), -80.0)
    x[0, 7], x[0, 20], x[0, 31], x[0, 100] = 0.0, -float(low), -float(low), -float(low + 2)
    tokens, _ = run(x.to(dtype), [1.0], temperature=[t], min_p=[2.0**-e])
    assert tokens.tolist() == [31]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_top_p_and_u_next_to_nothing(dtype):
    """The least numbers there are: the first token alone passes any top_p that is so small, and any u."""
    x = torch.full((4, 200), -3.0)
    x[:, 9] = 1.0
    tokens, _ = run(x.to(dtype), [2.0**-149, 2.0**-41, 0.5, 0.999], top_p=[1.0, 1.0, 2.0**-44, 2.0**-149])
    assert tokens.tolist() == [9] * 4
