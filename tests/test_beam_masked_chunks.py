"""The selection where some chunks of a part hold nothing that can win, NaN (a mask) among it.

The CTA's warps decide after each chunk whether anything was listed.  A model of their barriers on the
CPU: warps run in any order, add to the list's size, and must meet at the same barriers.  On the GPU:
parts of many chunks against the scores of all candidates in 64 bits (tests/test_beam.py)."""
import math
import random

import pytest
import torch

from tests.test_beam import BF16, F16, F32, check, make

WARPS = 3


def warp(w, chunks, between, size):
    """One warp's way: yields None after a step, or (barrier, its vote) and gets the votes' or."""
    for i, (lists, nan) in enumerate(chunks):
        mine = w == i % WARPS
        if lists and mine:
            size[0] += 1
            yield None
        if not (yield ("flags", i), (lists or nan) and mine):
            continue
        if between:
            found = size[0]
            yield None
        if (yield ("sums", i), nan and mine):
            yield ("greatest", i), False
            if between:
                yield ("greatest read", i), False
        if not between:
            yield None
            found = size[0]
        if found:
            yield ("list", i), False
            if w == 0:
                size[0] = 0
            yield ("list done", i), False


def run(chunks, between, rng):
    """All warps over `chunks`, each (some warp lists a value, some warp has a NaN), in a random order.
    `between`: the list's size is read between two barriers, else after the last of them.  "apart": they
    wait at different barriers, or some have gone."""
    size = [0]
    live = {w: warp(w, chunks, between, size) for w in range(WARPS)}
    at, votes = {}, {w: None for w in live}
    while live:
        running = [w for w in live if w not in at]
        if running:
            w = rng.choice(running)
            try:
                stop = live[w].send(votes[w])
                votes[w] = None
                if stop:
                    at[w] = stop
            except StopIteration:
                del live[w]
        elif len(live) < WARPS or len({name for name, _ in at.values()}) > 1:
            return "apart"
        else:
            votes = dict.fromkeys(live, any(vote for _, vote in at.values()))
            at = {}
    return "done"


CHUNKS = [(True, False), (False, True), (True, False), (False, True), (False, False), (True, True)]


def test_warps_decide_together():
    assert {run(CHUNKS, True, random.Random(i)) for i in range(500)} == {"done"}


def test_the_model_sees_a_late_decision():
    assert "apart" in {run(CHUNKS, False, random.Random(i)) for i in range(500)}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("K", [1, 4, 32])
def test_nan_between_chunks(dtype, K):
    """A part's first chunk holds its best; later ones are masked, by NaN or -infinity or both, or low."""
    G, V, chunk = 320 // K, 300_000, (4096 if dtype is F32 else 8192)
    x, st = make(G, K, V, dtype, seed=K)
    best = x[:, :2000].clone()
    x.clamp_(max=-3.0)
    x[:, :2000] = best + 4
    g = torch.Generator(device="cuda").manual_seed(1)
    n = (V + chunk - 1) // chunk
    kind = torch.randint(0, 5, (G * K, n), generator=g, device="cuda")
    kind[:, 0] = 0
    kind = kind.repeat_interleave(chunk, 1)[:, :V]
    some = torch.rand((G * K, V), generator=g, device="cuda") < 0.001
    x[(kind == 1) & some] = math.nan            # a few NaN among low logits
    x[kind == 2] = math.nan                     # nothing else
    x[kind == 3] = -math.inf
    x[(kind == 3) & some] = math.nan
    for _ in range(20):
        check(x, st)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_logits_among_masked_chunks(dtype):
    """No K-th best yet: rows with a logit or two in some chunks, the others masked, by NaN too."""
    K, V = 8, 200_000
    x, st = make(40, K, V, dtype, seed=5)
    keep = torch.rand((40 * K, V), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) < 2e-5
    odd = torch.arange(V, device="cuda") % 3 == 0
    x = torch.where(keep, x, torch.where(odd, math.nan, -math.inf).to(dtype))
    for _ in range(20):
        check(x, st)
