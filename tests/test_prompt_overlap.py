"""ssa_prompt_attention refuses results that share an element with its inputs or with one another, and takes
those that lie between their rows.  No kernel runs: a call without sequences ends after the checks."""
import ctypes
import random

import numpy as np
import pytest

import sparse_attention_decode_indexer_gb300 as ssa

D, FAR = 128, 1 << 40


def call(q, k, v, out, nq, nk):
    """Tensors as (element offset, heads, token stride, head stride)."""
    t = [ctypes.byref(ssa.SsaPromptTensor(FAR + 2 * at, heads, (ctypes.c_int64 * 2)(tok, head)))
         for at, heads, tok, head in (q, k, v, out)]
    return ssa.lib().ssa_prompt_attention(0, D, 0, nq, nk, *t, FAR, FAR, 1, 0.1, None, None, FAR, None)


def elements(x, n):
    at, heads, tok, head = x
    rows = at + (np.arange(n) * tok)[:, None] + (np.arange(heads) * head)[None]
    return (rows[..., None] + np.arange(D)).ravel()


AWAY = [(10_000_000 * i, 2, 2 * D, D) for i in range(1, 5)]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_out_over_an_input(which):
    n = 8
    t = [(0, 4, 512, D)] + [(x[0], 2, 256, D) for x in AWAY[:2]]
    # begins inside of it: its second token, its last head, one row of the type's alignment on
    for at in (512, 512 * 7 + 3 * D, 8, 120, 0):
        base = t[which][0]
        width = t[which][1]
        out = (base + at % (256 * n if width == 2 else 512 * n), 4, 512, D)
        assert call(*t, out, n, n) == -1
        # and it in the result
        moved = list(t)
        moved[which] = (base + 3 * 512 + 8, *t[which][1:])
        assert call(*moved, (base, 4, 512, D), n, n) == -1
    assert call(*t, (AWAY[3][0], 4, 512, D), n, n) == 0


def test_slices_of_one_buffer():
    """[T][q, k, v, out] in one buffer, tokens first or heads first."""
    n = 50
    Hq, H = 8, 2
    W = (2 * Hq + 2 * H) * D
    tensors = [(0, Hq, W, D), (Hq * D, H, W, D), ((Hq + H) * D, H, W, D), ((Hq + 2 * H) * D, Hq, W, D)]
    assert call(*tensors, n, n) == 0
    assert call(*tensors[:3], (tensors[3][0] - D, Hq, W, D), n, n) == -1
    assert call(*tensors[:3], (tensors[3][0] + 8, Hq, W, D), n, n) == -1       # its last row in the next token's q
    heads = [(at // D * n * D, h, D, n * D) for at, h, _, _ in tensors]
    assert call(*heads, n, n) == 0
    assert call(*heads[:3], (heads[3][0] - 8, Hq, D, n * D), n, n) == -1
    # one query token: its stride says nothing
    assert call(*tensors[:3], (tensors[3][0], Hq, 8, D), 1, n) == 0
    # token strides that differ, between each other's rows
    assert call(*tensors[:3], (tensors[3][0], Hq, 2 * W, D), n, n) == -1


def test_out_over_itself():
    q, k, v, away = AWAY
    at = away[0]
    for tok, head in ((256, 64), (64, 1 << 20), (8, D), (D, D), (D + 8, 2 * D)):
        assert call((q[0], 2, 256, D), k, v, (at, 2, tok, head), 3, 3) == -1
    for tok, head in ((256, D), (D, 3 * D), (384, D), (256, 3 * 256 + D), (4 * D, 2 * D)):
        assert call((q[0], 2, 256, D), k, v, (at, 2, tok, head), 3, 3) == 0
    assert call((q[0], 1, 256, D), (k[0], 1, 256, D), (v[0], 1, 256, D), (at, 1, 8, 8), 1, 3) == 0


def test_as_the_elements_say():
    rng = random.Random(3)
    seen = {0: 0, -1: 0}
    for _ in range(4000):
        nq, nk = rng.randint(1, 5), rng.randint(1, 5)
        H, G = rng.randint(1, 3), rng.randint(1, 2)
        tok = 8 * rng.choice([16, 32, 48, rng.randint(1, 80)])
        k_head, o_head = (8 * rng.choice([16, 32, 80, rng.randint(1, 40)]) for _ in range(2))
        q, v = (10_000_000, G * H, 256, D), (20_000_000, H, 256, D)
        k = (4096, H, tok, k_head)
        out = (4096 + 8 * rng.randint(-200, 200), G * H, tok, o_head)
        o = elements(out, nq)
        want = -1 if len(np.unique(o)) < len(o) or np.intersect1d(o, elements(k, nk)).size else 0
        assert call(q, k, v, out, nq, nk) == want, (q, k, v, out, nq, nk)
        seen[want] += 1
    assert min(seen.values()) > 400


def test_no_such_memory():
    big = (0, 2, (1 << 38) - 8, D)
    assert call(big, AWAY[0], AWAY[1], AWAY[2], 1 << 29, 3) == -1
