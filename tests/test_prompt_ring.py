"""The ring of K and V blocks of prompt attention, as a model on the CPU: waiters know a barrier by the
parity of its phase alone, and copies land in any order.  The roles follow the kernel's: one that copies, two
that multiply (K by `full`, V by `clean`), and those that look through V."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_decode_indexer_gb300", "csrc")
STAGES, LOOKS = 5, 4


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        assert self.pending > 0
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def done(self, parity):               # what a wait on a parity sees
        return (self.phase & 1) != parity


def run(blocks, every_use, rng):
    """Runs the roles in a random order.  Returns "done", "stuck", or "early" if something is read that has
    not landed.  `every_use`: the looking roles wait for K as well, and release the stages with the others."""
    full = [Barrier(1) for _ in range(STAGES)]
    empty = [Barrier(2 + LOOKS if every_use else 2) for _ in range(STAGES)]
    clean = [Barrier(LOOKS) for _ in range(STAGES)]
    holds = [None] * STAGES
    flying, early = [], []

    def copy():
        for it in range(2 * blocks):
            st, use = it % STAGES, it // STAGES
            if use:
                yield lambda: empty[st].done((use - 1) & 1)
            holds[st] = None
            flying.append((st, it))

    def multiply():
        for it in range(2 * blocks):
            st, use = it % STAGES, it // STAGES
            if it & 1:
                n = sum(1 for o in range(1, it, 2) if o % STAGES == st)      # V's uses of this stage before
                yield lambda: clean[st].done(n & 1)
            else:
                yield lambda: full[st].done(use & 1)
            if holds[st] != it:
                early.append(it)
            empty[st].arrive()

    def look():
        for it in range(2 * blocks):
            st, use = it % STAGES, it // STAGES
            if not it & 1 and not every_use:
                continue
            yield lambda: full[st].done(use & 1)
            if holds[st] != it:
                early.append(it)
            if it & 1:
                clean[st].arrive()
            if every_use:
                empty[st].arrive()

    roles = [copy(), multiply(), multiply()] + [look() for _ in range(LOOKS)]
    waits = {r: (lambda: True) for r in roles}
    while waits or flying:
        ready = [r for r, w in waits.items() if w()]
        if not ready and not flying:
            return "stuck"
        if flying and (not ready or rng.random() < 0.1):
            st, it = flying.pop(rng.randrange(len(flying)))
            holds[st] = it
            full[st].arrive()
            continue
        r = rng.choice(ready)
        try:
            waits[r] = next(r)
        except StopIteration:
            del waits[r]
        if early:
            return "early"
    return "done"


@pytest.mark.parametrize("blocks", [1, 2, 3, 5, 7, 23])
def test_every_use_is_waited_for(blocks):
    assert {run(blocks, True, random.Random(seed)) for seed in range(200)} == {"done"}


def test_a_use_left_out_is_seen_by_the_model():
    """The roles that look for V alone pass a stage whose K has not landed yet."""
    assert "early" in {run(7, False, random.Random(seed)) for seed in range(200)}


def test_source_waits_for_every_use():
    with open(os.path.join(CSRC, "prompt.cu")) as f:
        body = re.sub(r"//[^\n]*", "", f.read())
    assert int(re.search(r"kStages = (\d+)", body).group(1)) == STAGES
    assert int(re.search(r"kLooks = (\d+)", body).group(1)) == LOOKS
    assert "mbar_init(&sh.empty[threadIdx.x], 2 + kLooks)" in body
    look = body.split("} else if (warp >= kLook) {")[1].split("} else if (warp < 8) {")[0]
    steps = re.findall(r"mbar_wait\(&sh\.full\[st\], ph|seen\(nullptr\)|seen\(&sh\.clean\[st\]\)", look)
    assert [s.split("(")[0] for s in steps] == ["mbar_wait", "seen", "mbar_wait", "seen"]
    assert "mbar_arrive(&sh.empty[st])" in look
