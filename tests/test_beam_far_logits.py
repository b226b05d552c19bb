"""Scores of rows whose logits lie far from zero, spread over chunks and parts: the sums of each are taken
beside its own greatest logit and joined.  Tolerances are those of tests/test_beam.py."""
import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa
from tests.test_beam import BF16, F32, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low,step", [(2_000_000.0, 0.5), (-10_000_000.0, 1.0), (1_048_576.0, 0.5), (-1_048_575.0, -0.75),
                                      (1_048_575.0, 1.5), (33_554_432.0, 4.0), (-2.0 ** 80, 0.0)])
@pytest.mark.parametrize("G,V", [(1, 16384), (1, 400_000), (300, 30_000)])
def test_two_halves(low, step, G, V):
    """A row's first half at one logit, its second a little above: parts, or chunks of one part."""
    st = ssa.BeamState(G, 2)
    st.scores.zero_()
    x = torch.full((2 * G, V), low, device="cuda")
    x[:, V // 2:] += step
    check(x, st)


@pytest.mark.parametrize("base", [2.0 ** 19.99, 2.0 ** 20, 2.0 ** 20.5, 2.0 ** 21, 2.0 ** 22, 2.0 ** 23, 2.0 ** 24, 2.0 ** 40, 2.0 ** 127])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_spread_over_chunks_and_parts(base, sign, dtype):
    for G in (2, 100):
        x, st = make(G, 4, 60_000, F32, seed=G)
        check((sign * base + x).to(dtype), st)
        # every chunk a little above those before it
        up = torch.linspace(-3, 3, 60_000, device="cuda")
        check((sign * base + up + 0.1 * x).to(dtype), st)
        # a row's parts far from one another and next to one another
        far = torch.randint(0, 4, (4 * G, 15), device="cuda").repeat_interleave(4000, 1)
        check((sign * base + x + 5e5 * far).to(dtype), st)


@pytest.mark.parametrize("rows", [1, 2])
def test_sums_of_the_largest_vocabulary(rows):
    """2^23 logits, all but each part's first chunk two octaves above it."""
    V, chunk = 1 << 23, 4096
    room = 4 * torch.cuda.get_device_properties(0).multi_processor_count // rows
    per_part = -(-(V // chunk) // room)
    st = ssa.BeamState(1, rows)
    st.scores.zero_()
    for low in (-1.4, -0.7):
        x = torch.zeros((rows, V // chunk, chunk), device="cuda")
        x[:, ::per_part] = low
        x = x.view(rows, V)
        check(x, st)
