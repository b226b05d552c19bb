"""Ids and positions out of range are flagged and nothing is written through them: pools, mirrors, scales,
slab rows and slot tables stay as they were, those of a page and a slot behind the last ones among them."""
import numpy as np
import pytest
import torch

from tests.test_pages import BAD_ID, Model, _dev, _setup, ssa  # noqa: F401

pytestmark = pytest.mark.gpu
D = 128
BAD_POS = 16


class _Guarded:
    """A cache whose layout leaves out the last page and the last slot of every layer's arrays of one layer:
    what is written behind them is seen."""

    def __init__(self, ssa, fmt, P, H, Lp, host):  # noqa: F811
        big = ssa.Layout(P, H, H, D, fmt != "bf16", 1, Lp + 1, Lp + 1, 1, Lp, 1, kv_format=fmt)
        self.cache = c = ssa.KVCache(big, host)
        ssa.ssa_lru_init(c, True)
        small = ssa.Layout(P, H, H, D, fmt != "bf16", 1, Lp, Lp, 1, Lp, 1, kv_format=fmt)
        c.layout, c._lay = small, small.c()
        g = torch.Generator().manual_seed(P)
        for n in self.names():
            t = getattr(c, n)
            if n in ("k_pool", "v_pool", "k_mirror", "v_mirror"):
                t.copy_(torch.randint(0, 120, t.shape, generator=g, dtype=torch.uint8))
            elif n in ("slab_cnt", "slab"):
                t.copy_(torch.randint(1, 9, t.shape, generator=g).to(t.dtype))
            elif t.dtype == torch.float32:
                t.copy_(torch.rand(t.shape, generator=g) + 0.5)
        for n in ("k_pool", "v_pool", "k_scale", "v_scale"):   # slot s holds page s, the mirror's bytes
            m = getattr(c, Model.mname(n))
            if m is not None:
                m.copy_(getattr(c, n))
        self.before = {n: getattr(c, n).cpu().clone() for n in self.names()}

    def names(self):
        ns = list(Model.KV) + list(Model.SLAB) + [Model.mname(n) for n in Model.KV]
        return [n for n in ns + ["slot_of", "page_of", "last_use"] if getattr(self.cache, n) is not None]

    def check_untouched(self, pages):
        """Every page but `pages` (and the guards) as before, in every array."""
        torch.cuda.synchronize()
        keep = [i for i in range(self.before["slot_of"].shape[1]) if i not in pages]
        for n, t in self.before.items():
            got = getattr(self.cache, n).cpu()
            assert torch.equal(got[:, keep], t[:, keep]), n


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8_page_head", "e4m3_page_head"])
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("host", [False, True])
def test_store_writes_nothing_at_bad_positions(ssa, fmt, P, T, host):  # noqa: F811
    """Tokens before the first page, of the page behind the last, and far behind it, around tokens of page 1."""
    Lp = 4
    n = min(T - 2, P - 1)                        # page 1 from its second row on
    rest = T - n
    below = -np.arange(rest // 2, 0, -1) - 1
    above = Lp * P + np.arange(rest - rest // 2)
    above[len(above) // 2:] += 1 << 40           # (a page number that passes 32 bits)
    pos = np.concatenate([below, P + 1 + np.arange(n), above])
    assert len(pos) == T and (np.diff(pos) > 0).all()
    gd = _Guarded(ssa, fmt, P, 2, Lp, host)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((1, T, 2, D), generator=g).bfloat16().cuda() for _ in range(2))
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    ssa.ssa_store_kv_mirror(gd.cache, 0, 1, k, v, torch.from_numpy(pos).cuda(), status)
    gd.check_untouched([1] if n else [])
    assert int(status.item()) == BAD_ID
    cnt = gd.cache.slab_cnt.cpu()[0]
    assert int(cnt[1]) == int(gd.before["slab_cnt"][0, 1]) + n


@pytest.mark.parametrize("fmt", ["int8_page_head", "e4m3_page_head"])
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("T", [2, 300])
def test_store_in_no_order_stays_in_its_pages(ssa, fmt, P, T):  # noqa: F811
    """Positions that fall, or come twice: flagged; no other page is written."""
    Lp = 6
    rng = np.random.default_rng(T)
    for pos in (np.full(T, P + 3), np.sort(rng.integers(P, 3 * P, T))[::-1].copy(), rng.integers(P, 3 * P, T)):
        gd = _Guarded(ssa, fmt, P, 2, Lp, False)
        k, v = (torch.ones((1, T, 2, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        status = torch.zeros((1,), dtype=torch.int32, device="cuda")
        ssa.ssa_store_kv_mirror(gd.cache, 0, 1, k, v, torch.from_numpy(pos).cuda(), status)
        gd.check_untouched([1, 2])
        assert bool(int(status.item()) & BAD_POS) == bool((np.diff(pos) <= 0).any())


@pytest.mark.parametrize("host", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "int8_page_head"])
def test_forks_follow_no_bad_id(ssa, fmt, host):  # noqa: F811
    c, table, ws, status, rng = _setup(ssa, fmt=fmt, Lp=12, B=3, nmax=3, host=host, lens=np.array([40, 20, 16]))
    table.block_table[0, 1] = 99                 # a full page out of range
    table.block_table[1, 1] = -7                 # the partly filled page out of range
    m = Model(c, table)
    bt = m.bt.copy()
    ssa.ssa_fork_requests(c, table, _dev([0, 0, 1]), None, status, ws)
    torch.cuda.synchronize()
    assert int(status.item()) == BAD_ID
    now = table.block_table.cpu().numpy()
    # row 1 continues row 0 (a full page, 99, a copy of its last page), row 2 row 1's old pages
    assert now[0].tolist() == bt[0].tolist() and now[1, :2].tolist() == bt[0, :2].tolist()
    assert now[2].tolist() == [bt[1, 0], -7, -1]
    new = int(now[1, 2])
    assert new not in set(bt.flatten().tolist()) - {int(bt[2, 0])}      # free, or what row 2 let go
    for n, t in m.a.items():                     # nothing but the copy, and the slots of free pages
        got = getattr(c, n).cpu().numpy()
        if n in Model.SLAB or n.endswith("_mirror"):
            keep = [i for i in range(12) if i != new]
            np.testing.assert_array_equal(got[:, keep], t[:, keep], err_msg=n)
            if n in Model.SLAB:
                np.testing.assert_array_equal(got[:, new], t[:, bt[0, 2]], err_msg=n)
        elif n in Model.KV:
            for l in range(m.L):
                keep = [s for s in range(m.S) if s != m.slot(l, new) or host]
                np.testing.assert_array_equal(got[l, keep], t[l, keep], err_msg=n)
        elif host:                               # let go: the page of row 2, and the new one
            gone = {new, int(bt[2, 0])}
            for l in range(m.L):
                free = {m.slot(l, p) for p in gone}
                keep = [i for i in range(t.shape[1]) if i not in (gone if n == "slot_of" else free)]
                np.testing.assert_array_equal(got[l, keep], t[l, keep], err_msg=n)
        else:
            np.testing.assert_array_equal(got, t, err_msg=n)


@pytest.mark.parametrize("host", [False, True])
def test_compaction_follows_no_bad_id(ssa, host):  # noqa: F811
    c, table, ws, status, rng = _setup(ssa, Lp=12, B=3, nmax=3, host=host, lens=np.array([40, 20, 16]))
    ssa.ssa_compact_pages(c, table, status, ws)  # the pages in use are the lowest: nothing is left to move
    assert int(status.item()) == 0
    table.block_table[0, 1] = 99
    table.block_table[1, 1] = -7
    m = Model(c, table)
    ssa.ssa_compact_pages(c, table, status, ws)
    m.status = BAD_ID
    m.check(status)


def test_copies_follow_no_bad_id(ssa):  # noqa: F811
    gd = _Guarded(ssa, "int8_page_head", 16, 2, 4, True)
    c = gd.cache
    ws = torch.zeros((ssa.ssa_workspace_size(c.layout),), dtype=torch.uint8, device="cuda")
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    src, dst = [4, 1, 2 ** 31 - 1, 0], [1, 4, 2, 2 ** 30]
    ssa.ssa_copy_pages(c, _dev(src), _dev(dst), status, ws)
    gd.check_untouched([])
    assert int(status.item()) == BAD_ID
    ssa.ssa_copy_pages(c, _dev(src * 20), _dev(dst * 20), status, ws)   # with a launch that checks
    gd.check_untouched([])
