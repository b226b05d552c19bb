"""Values that are not finite where rows see them, in one and in several blocks of keys, seen by all rows
of a tile or by some: the rows that see them have them, the others are as without."""
import math

import pytest
import torch

from tests.test_prompt import BF16, F16, call, compare, inputs, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lq,lk", [([900], [900]), ([300, 500], [300, 500]), ([5], [9000]), ([4, 3], [900, 2500]),
                                   ([40] * 12, [40] * 12)])
@pytest.mark.parametrize("causal", [True, False])
def test_seen(dtype, lq, lk, causal):
    for places in ((0,), (1,), (-1,), (0.5,), (0.1, 0.9), (0.0, 0.3, 0.5, -2, -1), (0.2, 0.21, 0.6)):
        q, k, v = inputs(lq, lk, 8, 2, dtype, seed=len(places))
        v = v.clone()
        Tk = sum(lk)
        for i, at in enumerate(places):
            j = at if isinstance(at, int) else int(at * Tk)
            v[j, i % 2, 7 + 16 * i] = (math.inf, -math.inf, math.nan)[i % 3]
            v[j, 1, 100] = math.inf
        compare(call(q, k, v, lq, lk, causal), reference(q, k, v, lq, lk, causal))
