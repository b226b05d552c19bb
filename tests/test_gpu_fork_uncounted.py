"""Forks over tables with pages that rows hold and nothing counts: lengths that grew in place over pages
assigned beforehand, after the references were counted.  Such a page is kept, counted and flagged; it is
never a new page of another row."""
import numpy as np
import pytest
import torch

from tests.test_pages import BAD_ID, Model, _dev, _setup, ssa  # noqa: F401

pytestmark = pytest.mark.gpu


def _rows(bt, lens, P):
    return [[int(x) for x in r[:-(-int(n) // P)]] for r, n in zip(bt, lens)]


@pytest.mark.parametrize("kw", [dict(), dict(host=True), dict(fmt="bf16", P=32, Hkv=1), dict(B=1),
                                dict(Lp=6000, B=60, nmax=90, L=1, Hkv=1)],      # several blocks plan
                         ids=str)
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_uncounted_pages_stay_with_their_rows(ssa, kw, seed):  # noqa: F811
    c, table, ws, status, rng = _setup(ssa, seed=seed, **kw)
    lay = c.layout
    B, P, nmax, Lp = lay.batch, lay.page_size, lay.max_pages, lay.logical_pages
    for step in range(4):
        old = _rows(table.block_table.cpu().numpy(), table.seq_lens.cpu().numpy(), P)
        mine = [i for i in range(B) if rng.random() < 0.6]                      # rows that go on
        lost = {x for i in mine for x in old[i] if rng.random() < 0.3}
        if lost:
            table.ref[torch.tensor(sorted(lost), device="cuda")] = 0
        parent = np.array([i if i in mine else rng.integers(-1, B) for i in range(B)], np.int32)
        new = rng.integers(0, nmax * P + 1, B).astype(np.int32)
        new[rng.random(B) < 0.4] = 0
        slab = {n: getattr(c, n).cpu().numpy().copy() for n in Model.SLAB}
        status.zero_()
        ssa.ssa_fork_requests(c, table, _dev(parent), _dev(new), status, ws)
        now = _rows(table.block_table.cpu().numpy(), table.seq_lens.cpu().numpy(), P)
        ref = table.ref.cpu().numpy()
        kept = {x for i, j in enumerate(parent) if j >= 0 for x in old[j]}
        shared = {x for i, j in enumerate(parent) if j >= 0 and j != i for x in old[j]}
        if lost - shared:                        # (a page that another row took up counts again)
            assert int(status.item()) & BAD_ID
        elif not lost:
            assert not int(status.item()) & BAD_ID
        assert lost <= kept
        held = [set(old[j]) if j >= 0 else set() for j in parent]               # before copies and growth
        for i in range(B):
            assert len(set(now[i])) == len(now[i])
            fresh = set(now[i]) - held[i]
            for k in range(B):                   # a new page is nobody else's, nor was it held
                assert not fresh & held[k] and (k == i or not fresh & set(now[k]))
            for x in now[i]:
                assert ref[x] >= 1
        for i in mine:                           # what a row went on holding is where and as it was
            n = max(len(old[i]) - 1, 0)
            assert now[i][:n] == old[i][:n]
            for name, t in slab.items():
                np.testing.assert_array_equal(getattr(c, name).cpu().numpy()[:, old[i][:n]], t[:, old[i][:n]])
        ssa.ssa_page_refs(table)
    # counted again, the calls are the definition's to the byte, and nothing is left in the workspace
    status.zero_()
    m = Model(c, table)
    for step in range(2):
        parent = rng.integers(-1, B, B).astype(np.int32)
        m.fork(parent, None)
        ssa.ssa_fork_requests(c, table, _dev(parent), None, status, ws)
        m.check(status)


def test_a_runner_whose_lengths_grew_in_place(ssa):  # noqa: F811
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    P = 16
    lay = ssa.Layout(P, 2, 2, 128, False, 2, 12, 12, 3, 4, 2)
    bt = np.array([[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11]], np.int32)       # assigned beforehand
    run = DecodeRunner(lay, host_tier=False, identity=True, block_table=bt,
                       seq_lens=np.array([P, P, 0], np.int32))
    assert run.table.ref.tolist() == [1, 0, 0, 0, 1] + [0] * 7
    x = torch.randn((2, P, 2, 128), device="cuda").bfloat16()
    run.seq_lens[0] = 3 * P                                                     # past pages 1 and 2
    for pg in (0, 1, 2):
        run.store(0, 2, x, x, torch.arange(pg * P, pg * P + P, device="cuda"))
    sums = run.cache.slab_sum.clone()
    run.fork(_dev([0, 1, 2]), _dev([0, 0, 2 * P]))                              # row 2 is admitted
    assert run.block_table[0].tolist() == [0, 1, 2, -1] and run.block_table[2].tolist() == [3, 5, -1, -1]
    assert run.table.ref.tolist() == [1, 1, 1, 1, 1, 1] + [0] * 6
    assert torch.equal(run.cache.slab_sum[:, :3], sums[:, :3])
    assert int(run.status.item()) == BAD_ID
    run.status.zero_()
    run.fork(_dev([0, 0, 2]))
    assert run.table.ref.tolist() == [2, 2, 2, 1, 0, 1] + [0] * 6 and int(run.status.item()) == 0


def test_a_partly_filled_page_that_nothing_counts(ssa):  # noqa: F811
    c, table, ws, status, rng = _setup(ssa, Lp=12, B=4, nmax=4, lens=np.array([20, 16, 0, 0]))
    a = table.block_table[0].tolist()
    table.ref[a[1]] = 0
    ssa.ssa_fork_requests(c, table, _dev([0, 0, 2, 3]), _dev([0, 0, 48, 0]), status, ws)
    bt = table.block_table.tolist()
    assert bt[0][:2] == a[:2] and bt[1][0] == a[0]
    ids = bt[0][:2] + bt[1][1:2] + bt[2][:3]
    assert len(set(ids)) == 6 and all(table.ref[i] >= 1 for i in ids)
    status.zero_()
    table.block_table[0, 1] = -1                 # a row that goes on names no page
    ssa.ssa_fork_requests(c, table, _dev([0, 1, 2, 3]), None, status, ws)
    assert int(status.item()) == BAD_ID and int(table.block_table[0, 1]) == -1
