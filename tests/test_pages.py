"""Owners of the pages (copy; fork, grow and free; compaction) against a plain model of the definitions
in include/ssa.h: every table, count, slot, slab row, pool and mirror byte equal after each call."""
import collections
import ctypes

import numpy as np
import pytest
import torch

BAD_ID, UNRESOLVED, BAD_POS, NO_PAGES = 2, 8, 16, 128


@pytest.fixture(scope="module")
def ssa():
    from sparse_attention_decode_indexer_gb300 import build
    build.build()
    import sparse_attention_decode_indexer_gb300 as m
    return m


class Model:
    """Numpy copies of the cache's arrays and the table, and the definitions, page by page."""
    SLAB = ("slab", "slab_scale", "slab_sum", "slab_cnt")
    KV = ("k_pool", "v_pool", "k_scale", "v_scale")

    def __init__(self, cache, table):
        self.cache, self.table = cache, table
        lay = cache.layout
        self.L, self.P, self.B, self.nmax = lay.n_layers, lay.page_size, lay.batch, lay.max_pages
        self.Lp, self.S = lay.logical_pages, lay.pool_slots
        self.kv = [n for n in self.KV if getattr(cache, n) is not None]
        self.mir = cache.k_mirror is not None
        names = self.kv + list(self.SLAB) + ["slot_of", "page_of", "last_use"]
        if self.mir:
            names += [self.mname(n) for n in self.kv]
        self.a = {n: getattr(cache, n).cpu().numpy().copy() for n in names}
        self.bt, self.lens, self.ref = (t.cpu().numpy().copy() for t in (table.block_table, table.seq_lens, table.ref))
        self.status = 0

    @staticmethod
    def mname(n):
        return n.replace("_pool", "_mirror") if n.endswith("_pool") else n + "_mirror"

    def check(self, status):
        torch.cuda.synchronize()
        assert int(status.item()) == self.status
        for n, t in (("block_table", self.bt), ("seq_lens", self.lens), ("ref", self.ref)):
            np.testing.assert_array_equal(getattr(self.table, n).cpu().numpy(), t, err_msg=n)
        for n, t in self.a.items():
            np.testing.assert_array_equal(getattr(self.cache, n).cpu().numpy(), t, err_msg=n)

    def pages(self, n):
        return -(-n // self.P)

    def slot(self, l, p):
        s = self.a["slot_of"][l, p]
        return s if 0 <= s < self.S else -1

    def copy(self, src, dst, dst_slot=True):
        for l in range(self.L):
            ss, sd = self.slot(l, src), self.slot(l, dst) if dst_slot else -1
            if (ss >= 0 or self.mir) and (sd >= 0 or self.mir):
                for n in self.kv:
                    x = (self.a[n][l, ss] if ss >= 0 else self.a[self.mname(n)][l, src]).copy()
                    if self.mir:
                        self.a[self.mname(n)][l, dst] = x
                    if sd >= 0:
                        self.a[n][l, sd] = x
            else:
                self.status |= UNRESOLVED
            for n in self.SLAB:
                self.a[n][l, dst] = self.a[n][l, src]

    def release(self, p):
        for l in range(self.L):
            s = self.a["slot_of"][l, p]
            if s >= 0:
                self.a["page_of"][l, s] = self.a["last_use"][l, s] = -1
                self.a["slot_of"][l, p] = -1

    def copy_pages(self, src, dst):
        before = {n: t.copy() for n, t in self.a.items()}
        todo = []
        for i, (s, d) in enumerate(zip(src, dst)):
            if s < 0 or d < 0:
                continue
            clash = any(dst[j] == d and src[j] >= 0 for j in range(i)) or \
                any(src[j] == d and dst[j] >= 0 for j in range(len(src)) if j != i)
            if s >= self.Lp or d >= self.Lp or clash:
                self.status |= BAD_ID
            elif s != d:
                todo.append((s, d))
        del before
        for s, d in todo:
            self.copy(s, d)

    def fork(self, parent, new_lens):
        old_bt, old_len = self.bt.copy(), self.lens.copy()
        B = self.B
        par = []
        for i in range(B):
            j = int(parent[i])
            if j < -1 or j >= B:
                self.status |= BAD_ID
                j = i
            par.append(j)
        refs = self.ref
        for i, j in enumerate(par):
            if j != i:
                for p in range(self.pages(old_len[i])):
                    refs[old_bt[i, p]] -= 1
        held = {}                                  # partly filled page -> rows that continue it
        for i, j in enumerate(par):
            n = old_len[j] if j >= 0 else 0
            if j != i:
                for p in range(self.pages(n)):
                    refs[old_bt[j, p]] += 1
            if n % self.P:
                held.setdefault(int(old_bt[j, n // self.P]), []).append(i)
        keep, need = [True] * B, [0] * B
        for g, rows in held.items():
            left = refs[g] - len(rows)
            for i in rows:
                keep[i] = i == min(rows) and left <= 0
            refs[g] = max(left, 1)
        free = [p for p in range(self.Lp) if refs[p] <= 0]
        freed = [old_bt[i, p] for i, j in enumerate(par) if j != i for p in range(self.pages(old_len[i]))]
        free_now = set(free)
        freed = [p for p in freed if p in free_now]
        free = collections.deque(free)
        copies = []
        for i, j in enumerate(par):
            n = int(old_len[j]) if j >= 0 else 0
            want = int(new_lens[i]) if new_lens is not None else 0
            if want > self.nmax * self.P:
                self.status |= BAD_POS
                want = self.nmax * self.P
            nlen = max(n, want)
            row = [int(x) for x in old_bt[j, :self.pages(n)]] if j >= 0 else []
            short = False
            if not keep[i]:
                g = row.pop()
                if free:
                    row.append(free.popleft())
                    refs[row[-1]] = 1
                    copies.append((g, row[-1]))
                else:
                    short = True
            while not short and len(row) < self.pages(nlen):
                if not free:
                    short = True
                    break
                row.append(free.popleft())
                refs[row[-1]] = 1
                for n_ in self.SLAB:
                    self.a[n_][:, row[-1]] = 0
                if self.mir:
                    self.release(row[-1])
            if short:
                self.status |= NO_PAGES
                nlen = min(nlen, len(row) * self.P)
            self.bt[i] = -1
            self.bt[i, :len(row)] = row
            self.lens[i] = nlen
        if self.mir:
            for p in freed:
                self.release(p)
        for g, d in copies:
            if self.mir:
                self.release(d)
            self.copy(g, d, dst_slot=not self.mir)

    def compact(self):
        live = self.ref > 0
        n = int(live.sum())
        src, dst = np.flatnonzero(live & (np.arange(self.Lp) >= n)), np.flatnonzero(~live & (np.arange(self.Lp) < n))
        to = dict(zip(src.tolist(), dst.tolist()))
        for i in range(self.B):
            for p in range(self.pages(self.lens[i])):
                self.bt[i, p] = to.get(int(self.bt[i, p]), self.bt[i, p])
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
            for l in range(self.L):
                sa, sb = self.a["slot_of"][l, a], self.a["slot_of"][l, b]
                if self.mir:
                    for m in self.kv:
                        self.a[self.mname(m)][l, b] = self.a[m][l, sa] if sa >= 0 else self.a[self.mname(m)][l, a]
                for m in self.SLAB:
                    self.a[m][l, b] = self.a[m][l, a]
                self.a["slot_of"][l, b], self.a["slot_of"][l, a] = sa, sb
                if sa >= 0:
                    self.a["page_of"][l, sa] = b
                if sb >= 0:
                    self.a["page_of"][l, sb] = a
        return src, dst


def _setup(ssa, fmt="int8_page_head", P=16, Hkv=2, L=3, Lp=40, S=None, B=5, nmax=7, host=False, seed=0, lens=None):
    """A cache of random bytes, pages in random slots, requests on random pages."""
    rng = np.random.default_rng(seed)
    S = Lp if S is None else S
    lay = ssa.Layout(P, Hkv, Hkv, 128, fmt != "bf16", L, Lp, S, B, nmax, 1, kv_format=fmt)
    c = ssa.KVCache(lay, host)
    ssa.ssa_lru_init(c, False)
    for n in ("k_pool", "v_pool", "k_mirror", "v_mirror"):
        t = getattr(c, n)
        if t is not None:
            t.copy_(torch.from_numpy(rng.integers(0, 256, t.shape, dtype=np.uint8)))
    for n in ("k_scale", "v_scale", "k_scale_mirror", "v_scale_mirror", "slab_scale", "slab_sum"):
        t = getattr(c, n)
        if t is not None:
            t.copy_(torch.from_numpy(rng.random(t.shape, dtype=np.float32)))
    c.slab.copy_(torch.from_numpy(rng.integers(-127, 128, c.slab.shape, dtype=np.int8)))
    c.slab_cnt.copy_(torch.from_numpy(rng.integers(1, P + 1, c.slab_cnt.shape, dtype=np.int32)))
    for l in range(L):
        n = S if not host else min(S, Lp) * 2 // 3          # some pages hold no slot, some slots no page
        pg, sl = rng.permutation(Lp)[:n], rng.permutation(S)[:n]
        so, po, lu = np.full(Lp, -1, np.int32), np.full(S, -1, np.int32), np.full(S, -1, np.int32)
        so[pg], po[sl], lu[sl] = sl, pg, rng.integers(0, 9, n)
        for name, x in (("slot_of", so), ("page_of", po), ("last_use", lu)):
            getattr(c, name)[l].copy_(torch.from_numpy(x))
        if host:                                            # a bound slot holds its page's bytes
            for n_ in ("k_pool", "v_pool", "k_scale", "v_scale"):
                if getattr(c, n_) is not None:
                    getattr(c, n_)[l][torch.from_numpy(sl).cuda()] = getattr(c, Model.mname(n_))[l][torch.from_numpy(pg)].cuda()
    if lens is None:
        lens = rng.integers(0, nmax * P + 1, B)
        lens[rng.integers(B)] = 0
        lens[rng.integers(B)] = nmax * P
    used = [-(-int(n) // P) for n in lens]
    while sum(used) > Lp:
        i = int(np.argmax(used))
        lens[i] -= P
        used[i] -= 1
    ids = rng.permutation(Lp)
    bt = np.full((B, nmax), -1, np.int32)
    at = 0
    for i, n in enumerate(used):
        bt[i, :n] = ids[at:at + n]
        at += n
    table = ssa.RequestTable(lay, bt, np.asarray(lens, np.int32))
    ws = torch.zeros((ssa.ssa_workspace_size(lay),), dtype=torch.uint8, device="cuda")
    return c, table, ws, torch.zeros((1,), dtype=torch.int32, device="cuda"), rng


def _dev(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


CACHES = [dict(), dict(host=True), dict(fmt="bf16", P=32, Hkv=1), dict(fmt="fp8", host=True, Hkv=4, S=30),
          dict(fmt="e4m3_page_head", P=128, Hkv=8, L=1, host=True), dict(Lp=700, B=33, nmax=19, L=1),
          dict(B=1, nmax=1, Lp=2, host=True)]


@pytest.mark.gpu
@pytest.mark.parametrize("kw", CACHES, ids=str)
def test_refs_count_the_rows(ssa, kw):
    c, table, ws, status, rng = _setup(ssa, **kw)
    want = np.zeros(c.layout.logical_pages, np.int32)
    bt, lens = table.block_table.cpu().numpy(), table.seq_lens.cpu().numpy()
    for i, n in enumerate(lens):
        for p in range(-(-int(n) // c.layout.page_size)):
            want[bt[i, p]] += 1
    np.testing.assert_array_equal(table.ref.cpu().numpy(), want)
    table.ref.fill_(77)
    ssa.ssa_page_refs(table, status)
    np.testing.assert_array_equal(table.ref.cpu().numpy(), want)
    assert int(status.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kw", CACHES[:6], ids=str)
def test_copy_pages(ssa, kw):
    c, table, ws, status, rng = _setup(ssa, **kw)
    Lp = c.layout.logical_pages
    m = Model(c, table)
    perm = rng.permutation(Lp)
    n = Lp // 2
    src, dst = perm[:n].astype(np.int32), perm[n:2 * n].astype(np.int32)
    src[1] = src[0]                              # one page copied twice
    src[2], dst[3] = -1, -5                      # padding
    dst[4] = src[4]                              # onto itself
    ssa.ssa_copy_pages(c, _dev(src), _dev(dst), status, ws)
    m.copy_pages(src, dst)
    m.check(status)
    # pairs that would depend on their order, and ids out of range
    src, dst = perm[:8].astype(np.int32), perm[8:16].astype(np.int32)
    dst[5] = dst[1]
    dst[2] = src[6]
    src[3], dst[7] = Lp, Lp + 5
    ssa.ssa_copy_pages(c, _dev(src), _dev(dst), status, ws)
    m.copy_pages(src, dst)
    m.check(status)
    assert m.status & BAD_ID
    ssa.ssa_copy_pages(c, _dev([]), _dev([]), status, ws)
    m.check(status)


@pytest.mark.gpu
def test_copy_many_pairs(ssa):
    """More pairs than one block checks, clashes far apart."""
    c, table, ws, status, rng = _setup(ssa, Lp=1500, L=1, B=2, nmax=2)
    m = Model(c, table)
    perm = rng.permutation(1500)
    src, dst = perm[:700].astype(np.int32), perm[700:1400].astype(np.int32)
    dst[650] = dst[3]
    dst[10] = src[690]
    ssa.ssa_copy_pages(c, _dev(src), _dev(dst), status, ws)
    m.copy_pages(src, dst)
    m.check(status)


@pytest.mark.gpu
def test_copy_without_slot_or_mirror(ssa):
    c, table, ws, status, rng = _setup(ssa, L=2)
    c.slot_of[1, 4] = -1
    c.slot_of[0, 9] = -1
    m = Model(c, table)
    ssa.ssa_copy_pages(c, _dev([4, 2, 7]), _dev([5, 9, 8]), status, ws)
    m.copy_pages([4, 2, 7], [5, 9, 8])
    m.check(status)
    assert m.status == UNRESOLVED


@pytest.mark.gpu
@pytest.mark.parametrize("kw", CACHES, ids=str)
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_fork_grow_free_and_compact_in_turn(ssa, kw, seed):
    """Random calls one after another on one state, with a pinned page that comes and goes."""
    c, table, ws, status, rng = _setup(ssa, seed=seed, **kw)
    lay = c.layout
    B, nmax, P, Lp = lay.batch, lay.max_pages, lay.page_size, lay.logical_pages
    m = Model(c, table)
    pin = None
    for step in range(8):
        kind = rng.integers(4)
        parent = np.arange(B, dtype=np.int32)
        if kind == 0:                            # some rows end
            parent[rng.random(B) < 0.5] = -1
        elif kind == 1:                          # beam search
            parent = rng.integers(0, B, B).astype(np.int32)
        elif kind == 2:                          # mixed
            parent = rng.integers(-1, B, B).astype(np.int32)
        new = None
        if rng.random() < 0.6:
            new = rng.integers(-3, nmax * P + 1, B).astype(np.int32)
            new[rng.random(B) < 0.5] = 0
        m.fork(parent, new)
        ssa.ssa_fork_requests(c, table, _dev(parent), None if new is None else _dev(new), status, ws)
        m.check(status)
        if rng.random() < 0.5:
            if pin is None:
                pin = int(rng.integers(Lp))
                m.ref[pin] += 1
                table.ref[pin] += 1
            else:
                m.ref[pin] -= 1
                table.ref[pin] -= 1
                pin = None
            m.check(status)
        if rng.random() < 0.5:
            src, dst = m.compact()
            frm, to = (torch.full((Lp,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
            n = torch.zeros((1,), dtype=torch.int32, device="cuda")
            ssa.ssa_compact_pages(c, table, status, ws, frm, to, n)
            m.check(status)
            assert int(n.item()) == len(src)
            np.testing.assert_array_equal(frm.cpu().numpy()[:len(src)], src)
            np.testing.assert_array_equal(to.cpu().numpy()[:len(src)], dst)
            assert bool((frm[len(src):] == -9).all())
            if pin is not None:
                pin = dict(zip(src.tolist(), dst.tolist())).get(pin, pin)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    # more pages than the plan keeps bits of on chip, more new pages than its list holds there, and
    # tables that take several blocks to count (pages without a slot: their copies are flagged)
    dict(Lp=135000, B=60, nmax=2100, S=50, L=1, Hkv=1),
    # more requests than a block has threads
    dict(Lp=4000, B=1300, nmax=3, L=1, Hkv=1),
], ids=["pages", "requests"])
def test_large_tables(ssa, kw):
    c, table, ws, status, rng = _setup(ssa, seed=9, **kw)
    B, nmax, P = kw["B"], kw["nmax"], 16
    m = Model(c, table)
    everyone = np.arange(B, dtype=np.int32)
    beams = rng.integers(0, B, B).astype(np.int32)
    steps = [(np.where(rng.random(B) < 0.4, -1, everyone), None), "compact",
             (everyone, rng.integers(0, nmax * P + 1, B)), (beams, None), "compact",
             (np.where(rng.random(B) < 0.2, -1, beams), rng.integers(0, nmax * P + 1, B))]
    for step in steps:
        if step == "compact":
            m.compact()
            ssa.ssa_compact_pages(c, table, status, ws)
        else:
            parent, new = step
            m.fork(parent, new)
            ssa.ssa_fork_requests(c, table, _dev(parent), None if new is None else _dev(new), status, ws)
        m.check(status)


@pytest.mark.gpu
@pytest.mark.parametrize("host", [False, True])
def test_fork_cases_one_by_one(ssa, host):
    P = 16
    kw = dict(Lp=12, B=4, nmax=4, host=host)

    def go(lens, parent, new=None, pin=None, bt=None):
        c, table, ws, status, rng = _setup(ssa, lens=np.array(lens), seed=7, **kw)
        if bt is not None:
            table.block_table.copy_(_dev(bt))
            ssa.ssa_page_refs(table)
        if pin is not None:
            table.ref[int(table.block_table[pin])] += 1
        m = Model(c, table)
        before = m.bt.copy()
        m.fork(np.array(parent), None if new is None else np.array(new))
        ssa.ssa_fork_requests(c, table, _dev(parent), None if new is None else _dev(new), status, ws)
        m.check(status)
        return m, before
    m, b = go([P + 3, P, 5, 0], [0, 1, 2, 3])                    # nothing changes
    assert (m.bt == b).all()
    m, b = go([P + 3, P, 5, 0], [0, 0, 2, 3])                    # a fork: one shared page, one copy
    assert m.bt[1, 0] == b[0, 0] and m.bt[1, 1] not in (b[0, 1], -1) and m.ref[b[0, 0]] == 2
    m, b = go([P + 3, P, 5, 0], [1, 0, 2, 3])                    # two rows trade places: no copy
    assert (m.bt[[1, 0]] == b[[0, 1]]).all() and m.status == 0
    m, b = go([P + 3, P, 5, 0], [0, 1, 0, 0], pin=(0, 1))        # a pinned partly filled page: copies only
    assert all(m.bt[i, 1] != b[0, 1] for i in (0, 2, 3)) and m.ref[b[0, 1]] == 1
    m, b = go([3 * P, 2 * P + 1, 0, 0], [0, 1, 2, 3], bt=[[3, 4, 5, -1], [3, 4, 5, -1], [-1] * 4, [-1] * 4])
    assert m.bt[1, 2] != 5 and m.bt[0, 2] == 5                   # full for one row, partly filled for another
    m, b = go([4 * P, 4 * P, 4 * P, 0], [0, 1, 2, 3], new=[0, 0, 0, P])          # no page left
    assert m.status == NO_PAGES and m.lens[3] == 0
    m, b = go([3 * P + 1, 4 * P, 3 * P, 0], [0, 1, 2, 0], new=[0, 0, 4 * P, 4 * P])  # the copy's page goes first
    m, b = go([4 * P, 4 * P, 4 * P, 0], [-1, 1, 2, 3], new=[0, 0, 0, 4 * P])     # pages let go serve at once
    assert m.status == 0 and set(m.bt[3]) == set(b[0])
    m, b = go([5, 0, 0, 0], [0, 9, -2, 3], new=[4 * P + 1, 0, 0, 0])
    assert m.status == BAD_ID | BAD_POS and m.lens[0] == 4 * P
    m, b = go([5, 7, 9, 11], [-1] * 4)
    assert (m.bt == -1).all() and (m.lens == 0).all() and (m.ref == 0).all()


@pytest.mark.gpu
def test_bad_tables_are_flagged_and_not_followed(ssa):
    c, table, ws, status, rng = _setup(ssa, Lp=12, B=3, nmax=3, lens=np.array([40, 20, 16]))
    table.block_table[0, 1] = 99                 # a full page out of range
    table.block_table[1, 1] = -7                 # the partly filled page out of range
    ref = table.ref.clone()
    slabs = {n: getattr(c, n).clone() for n in Model.SLAB}
    ssa.ssa_fork_requests(c, table, _dev([0, 0, 1]), None, status, ws)
    assert int(status.item()) & BAD_ID
    bt = table.block_table.cpu().numpy()
    assert bt[1, 1] == 99 and bt[2, 1] == -7     # carried along
    assert int((table.ref - ref).abs().max()) <= 2
    status.zero_()
    ssa.ssa_compact_pages(c, table, status, ws)
    assert int(status.item()) & BAD_ID
    del slabs
    table.seq_lens[2] = 1000
    status.zero_()
    ssa.ssa_page_refs(table, status)
    assert int(status.item()) & BAD_POS


@pytest.mark.gpu
def test_captured_fork_replays(ssa):
    """The same captured call, replayed, follows the tables as they are then."""
    c, table, ws, status, rng = _setup(ssa, B=4, nmax=5, Lp=40, lens=np.array([70, 33, 5, 48]))
    parent = _dev([0, 0, 2, 3])
    m = Model(c, table)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        ssa.ssa_fork_requests(c, table, parent, None, status, ws)      # sets what a capture may not
        m.fork(parent.cpu().numpy(), None)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            ssa.ssa_fork_requests(c, table, parent, None, status, ws)
            ssa.ssa_compact_pages(c, table, status, ws)
    for p in ([0, 0, 2, 3], [1, 1, -1, 2], [3, 0, 1, -1]):
        parent.copy_(_dev(p))
        g.replay()
        m.fork(np.array(p), None)
        m.compact()
        m.check(status)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,host", [("int8_page_head", True), ("bf16", False), ("fp8", True)])
def test_forked_requests_decode_alike(ssa, fmt, host):
    """As a serving loop uses them together: rope, store, step; fork; grow and append; compact; free.  A
    fork's output equals its parent's, and a request that other forks and moves go past keeps its own."""
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    P, Hq, Hkv, L, B, nmax, Lp, k = 16, 8, 2, 2, 4, 6, 40, 2
    lay = ssa.Layout(P, Hq, Hkv, 128, True, L, Lp, Lp, B, nmax, k, kv_format=fmt)
    bt = np.full((B, nmax), -1, np.int32)
    ids = np.random.default_rng(0).permutation(Lp)
    bt[0, :4], bt[1, :3] = ids[:4], ids[4:7]
    lens = np.array([3 * P + 5, 2 * P + 9, 0, 0], np.int32)
    plan = ssa.RopePlan(128, 64)
    run = DecodeRunner(lay, host_tier=host, identity=not host, block_table=bt, seq_lens=lens, rope=plan)
    g = torch.Generator().manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=g).bfloat16().cuda()

    def append(rows, tokens):
        """Store tokens [L][n][H][D] of the rows' last positions (lengths already grown)."""
        t, n = run.block_table.cpu().numpy(), run.seq_lens.cpu().numpy()
        at = [(int(t[r, (n[r] - 1) // P]) * P + (n[r] - 1) % P, int(n[r]) - 1) for r in rows]
        order = sorted(range(len(rows)), key=lambda i: at[i][0])
        dev = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")  # noqa: E731
        run.store(0, L, tokens[0][:, order].contiguous(), tokens[1][:, order].contiguous(),
                  dev([at[i][0] for i in order]), positions=dev([at[i][1] for i in order]))

    for r in (0, 1):
        n = int(lens[r])
        pos = torch.from_numpy(np.array([int(bt[r, i // P]) * P + i % P for i in range(n)]))
        order = torch.argsort(pos)
        kk, vv = rand(L, n, Hkv, 128), rand(L, n, Hkv, 128)
        run.store(0, L, kk[:, order].contiguous(), vv[:, order].contiguous(), pos[order].cuda(),
                  positions=order.cuda())
    q1 = rand(L, 1, Hq, 128).expand(L, B, Hq, 128).contiguous()

    def same(x, y):
        """Two rows' outputs for the same context.  Rows are cut into pieces at other places, so the
        weights' rounding (bf16, half a step 2^-8, at worst) and the output's differ: each output is off
        by at most 2 * 2^-8 of the weighted mean of |V| (below max |V|, 5 of 10^5 normal values) and by
        2^-8 of itself."""
        return bool(((x - y).abs() <= 2 * (2 * 2.0 ** -8 * 5 + 2.0 ** -8 * y.abs())).all())
    run.step(q1)
    first = run.out.clone().float()
    assert bool((first[:, 2:] == 0).all())                   # rows without a token
    run.fork(_dev([0, 1, 0, 0]))
    run.step(q1)
    out = run.out.float()
    assert torch.equal(out[:, :2], first[:, :2])
    for r in (2, 3):
        assert torch.equal(run.sel[:, r], run.sel[:, 0]) and same(out[:, r], out[:, 0])
    # rows 2 and 3 grow by the same token, row 0 by another; row 1 stays
    run.fork(_dev([0, 1, 2, 3]), _dev([3 * P + 6, 0, 3 * P + 6, 3 * P + 6]))
    a, b = (rand(L, 1, Hkv, 128), rand(L, 1, Hkv, 128)), (rand(L, 1, Hkv, 128), rand(L, 1, Hkv, 128))
    b[1].add_(40)                                            # a value the output cannot miss
    append([0, 2, 3], [torch.cat((x, y, y), 1) for x, y in zip(a, b)])
    run.step(q1)
    grown, sel = run.out.clone().float(), run.sel.clone()
    assert torch.equal(grown[:, 1], first[:, 1])
    assert bool(((grown[:, 2] - grown[:, 3]).abs() <= 10 * 2 * 3 * 2.0 ** -8 * 5).all())   # |V| up to 45
    assert float((grown[:, 2] - first[:, 0]).abs().max()) > 2 * float((grown[:, 0] - first[:, 0]).abs().max())
    # the page space compacts, row 0 ends and row 1 is forked into its place
    run.compact()
    run.step(q1)
    assert torch.equal(run.out.float(), grown) and torch.equal(run.sel, sel)
    run.fork(_dev([1, 1, 2, -1]))
    run.compact()
    n_live = int((run.table.ref > 0).sum())
    assert int(run.block_table.max()) < n_live
    run.step(q1)
    out = run.out.float()
    assert torch.equal(run.sel[:, 0], sel[:, 1]) and same(out[:, 0], grown[:, 1])
    assert torch.equal(out[:, 1:3], grown[:, 1:3]) and bool((out[:, 3] == 0).all())
    assert int(run.status.item()) == 0


@pytest.mark.gpu
def test_a_runner_counts_its_table_outside_captures(ssa):
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    lay = ssa.Layout(16, 2, 2, 128, False, 1, 8, 8, 2, 3, 1)
    bt = torch.tensor([[0, 1, -1], [2, -1, -1]])
    run = DecodeRunner(lay, host_tier=False, identity=True, block_table=bt, seq_lens=torch.tensor([20, 16]))
    parent, x = torch.tensor([1, 1], dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        x.add_(1)
        with pytest.raises(RuntimeError):
            run.fork(parent)
    assert run.table.ref.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
    run.table.ref[0] += 1
    run.fork(torch.arange(2, dtype=torch.int32, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run.fork(parent)
    g.replay()
    g.replay()
    assert run.table.ref.tolist() == [1, 0, 2, 0, 0, 0, 0, 0]
    assert run.block_table.tolist() == [[2, -1, -1], [2, -1, -1]] and int(run.status.item()) == 0


def test_refusals(ssa):
    """On the host, before anything is enqueued."""
    lib, p, INVALID, UNSUPPORTED = ssa.lib(), 0x10000, -1, -3
    lay = ssa.Layout(64, 16, 2, 128, True, 2, 100, 80, 1, 100, 32).c()
    c = ssa.SsaCache(*([p] * 16))
    r = ssa.SsaRequests(p, p, p)
    assert lib.ssa_page_refs(lay, ssa.SsaRequests(p, None, p), None, None) == INVALID
    assert lib.ssa_copy_pages(lay, c, p, p, -1, None, p, None) == INVALID
    assert lib.ssa_copy_pages(lay, c, None, p, 1, None, p, None) == INVALID
    assert lib.ssa_copy_pages(lay, c, p, p, 1, None, None, None) == INVALID
    assert lib.ssa_copy_pages(lay, c, p, p, 16385, None, p, None) == UNSUPPORTED
    assert lib.ssa_fork_requests(lay, c, r, None, None, None, p, None) == INVALID
    assert lib.ssa_fork_requests(lay, c, r, p, None, None, None, None) == INVALID
    assert lib.ssa_fork_requests(lay, c, None, p, None, None, p, None) == INVALID
    assert lib.ssa_compact_pages(lay, c, ssa.SsaRequests(p, p, None), None, None, None, None, p, None) == INVALID
    assert lib.ssa_compact_pages(lay, c, r, None, None, None, None, None, None) == INVALID
    bad = ssa.SsaCache(*([p] * 16))
    bad.slab_cnt = None
    assert lib.ssa_fork_requests(lay, bad, r, p, None, None, p, None) == INVALID
    part = ssa.SsaCache(*([p] * 16))
    part.v_mirror = None
    assert lib.ssa_copy_pages(lay, part, p, p, 1, None, p, None) == -4
    lay.kv_dtype = 4
    assert lib.ssa_fork_requests(lay, c, r, p, None, None, p, None) == UNSUPPORTED
    assert ssa.status_str(128) == "no_pages"


def test_binding_refusals(ssa):
    lay = ssa.Layout(16, 2, 2, 128, True, 1, 8, 8, 2, 3, 1)
    z = lambda n, **kw: torch.zeros((n,), dtype=kw.get("dtype", torch.int32))  # noqa: E731
    with pytest.raises(ValueError):
        ssa.RequestTable(lay, z(5), z(2), ref=z(8), device="cpu")
    with pytest.raises(ValueError):
        ssa.RequestTable(lay, z(6).view(2, 3), z(3), ref=z(8), device="cpu")
    with pytest.raises(ValueError):
        ssa.RequestTable(lay, z(6).view(2, 3), z(2), ref=z(7), device="cpu")
    t = ssa.RequestTable(lay, z(6).view(2, 3), z(2), ref=z(8), device="cpu")
    c = ssa.KVCache(lay, False, device="cpu")
    st, ws = z(1), z(1)
    other = ssa.KVCache(ssa.Layout(16, 2, 2, 128, True, 1, 9, 9, 2, 3, 1), False, device="cpu")
    for f in (lambda: ssa.ssa_fork_requests(c, t, z(3), None, st, ws),
              lambda: ssa.ssa_fork_requests(c, t, z(2, dtype=torch.int64), None, st, ws),
              lambda: ssa.ssa_fork_requests(c, t, z(2), z(4)[::2], st, ws),
              lambda: ssa.ssa_fork_requests(other, t, z(2), None, st, ws),
              lambda: ssa.ssa_compact_pages(c, t, st, ws, z(3)),
              lambda: ssa.ssa_compact_pages(c, t, st, ws, n_moved=z(2)),
              lambda: ssa.ssa_copy_pages(c, z(2), z(3), st, ws),
              lambda: ssa.ssa_copy_pages(c, z(2).float(), z(2), st, ws)):
        with pytest.raises(ValueError):
            f()
    assert ctypes.sizeof(ssa.SsaRequests) == 24
