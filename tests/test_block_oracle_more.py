"""CPU pins of the optimizer's random bits against the definition that the measured cases
have, where those are: below 2^32 places."""

import numpy as np
import pytest
import torch

from oracle import block_oracle as o
from perf import more_operators as cases


@pytest.mark.parametrize("seed,step", [(0, 1), (9, 1), (0x123456789ABC, 7), (2 ** 63, 2 ** 33 + 5)])
def test_random_bits_are_those_of_the_cases(seed, step):
    n = 5000
    for bits in (cases._random_bits(n, seed, step, torch.device("cpu")),
                 cases._exact_bits(n, seed, step, torch.device("cpu"))):
        x, y = (z.numpy() for z in bits)
        m, v, p = o.random_bits(np.arange(n), seed, step)
        assert np.array_equal(x & 0xFFFF, m) and np.array_equal(x >> 16, v)
        assert np.array_equal(y & 0xFFFF, p)
