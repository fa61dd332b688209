"""A pin of oracle/evict.py on the CPU: how NaN and -inf rank."""
import math

import numpy as np
import pytest

from oracle import evict as OE


@pytest.mark.parametrize("low", [(math.nan, -math.inf), (-math.inf, math.nan), (math.nan, math.nan), (-math.inf, -math.inf)])
@pytest.mark.parametrize("at", [(0, 2), (17, 63)])
def test_nan_and_minus_infinity_rank_alike_and_the_first_of_them_stays(low, at):
    """One key of 64 goes: the later of the two lowest, whichever of them is the NaN."""
    w = np.random.default_rng(2).random((1, 1, 64))
    w[0, 0, list(at)] = low
    w[0, 0, [5, 6]] = [math.inf, -0.0]
    keep, _ = OE.select(w, [64], 63, 0)
    assert keep[0, 0].tolist() == [j for j in range(64) if j != at[1]]
    keep, _ = OE.select(w, [64], 62, 0)
    assert keep[0, 0].tolist() == [j for j in range(64) if j not in at]
