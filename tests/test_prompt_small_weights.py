"""Prompt attention in fp16 where most of a row's weights are far below its greatest.

Tolerance: that of tests/test_prompt.py but for the small weights' steps.  Weights are rounded as p = w /
(reference's weight), 2^7 or more for the row's greatest; steps below 2^-14 are 2^-24, so a weight is off by
at most 2^-25 / 2^7 of the greatest, which is at most 1 of the sum: 2^-32 sum_j |v_j| in place of 2^-25 |v| a
key."""
import math

import pytest
import torch

from tests.test_prompt import F16, D, call, reference

pytestmark = pytest.mark.gpu


def compare(q, k, v, lq, lk, causal):
    out, lse = call(q, k, v, lq, lk, causal)
    o, s, tol, ltol = reference(q, k, v, lq, lk, causal)
    G, b, a = q.shape[1] // k.shape[1], 0, 0
    for n, m in zip(lq, lk):
        mag = v[b:b + m].double().abs()
        steps = (2.0 ** -32 * mag.sum(0) - 2.0 ** -25 * m * mag.amax()).repeat_interleave(G, 0)
        tol[a:a + n] += steps
        a, b = a + n, b + m
    err = (out.double() - o).abs() - tol
    assert (err <= 0).all(), f"{err.max().item():.3e} above the tolerance"
    assert ((lse.double() - s).abs() <= ltol).all()
    return o


@pytest.mark.parametrize("nats", [10.0, 15.0, 17.0, 18.1, 20.0])
@pytest.mark.parametrize("lq,lk", [([1], [65536]), ([300], [9000]), ([2, 3], [30000, 20000])])
def test_one_key_above_the_others(nats, lq, lk):
    """The first key of each sequence is `nats` above all others, whose sum still counts."""
    Tq, Tk = sum(lq), sum(lk)
    q, k, v = (torch.zeros((T, H, D), dtype=F16, device="cuda") for T, H in ((Tq, 4), (Tk, 2), (Tk, 2)))
    q[..., 3] = 16.0
    k[..., 3] = -0.25
    v[:] = torch.linspace(0.5, 2.0, D, device="cuda")
    for first in [sum(lk[:i]) for i in range(len(lk))]:
        k[first, :, 3] += nats * math.sqrt(D) / 16.0
        v[first] = 0.0
    o = compare(q, k, v, lq, lk, False)
    assert o.min() > 0
    compare(q, k, v, lq, lk, True)


@pytest.mark.parametrize("causal", [True, False])
def test_spread_scores(causal):
    """Scores over some 30 nats, greatest first, last or in the middle."""
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn((n, h, D), generator=g, device="cuda") for n, h in ((700, 8), (5000, 2), (5000, 2)))
    q[..., 0] = 8.0
    at = torch.arange(5000, device="cuda")
    for ramp in (at / 5000, 1 - at / 5000, 1 - (at / 2500 - 1).abs()):
        kr = 0.2 * k
        kr[..., 0] = (ramp * 30 * math.sqrt(D) / 8 - 20)[:, None]
        compare(q.to(F16), kr.to(F16), v.abs().to(F16), [700], [5000], causal)
