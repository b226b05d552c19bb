"""Residency shared by the layers under everything a serving loop does: stores into pages that hold a slot,
forks, growth, freed rows, compaction.  A runner in that mode and one with a state per layer are handed the
same calls; selections, outputs, tables and mirrors are the same bits, and every slot that the shared state
binds to a page in use holds its bytes in every layer."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8_page_head", "e4m3_page_head"])
@pytest.mark.parametrize("identity", [False, True])
@pytest.mark.parametrize("by_layer", [False, True])
def test_shared_residency_in_a_serving_loop(fmt, identity, by_layer):
    import sparse_attention_decode_indexer_gb300 as ssa
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    P, Hq, Hkv, L, B, nmax, k = 16, 4, 2, 3, 4, 8, 1
    Lp = S = 40                                  # as few slots as the calls allow
    lay = ssa.Layout(P, Hq, Hkv, 128, fmt != "bf16", L, Lp, S, B, nmax, k, kv_format=fmt)
    lens = np.array([5 * P + 3, 3 * P, 0, 0], np.int32)
    bt = np.full((B, nmax), -1, np.int32)
    ids = np.random.default_rng(1).permutation(Lp)
    bt[0, :6], bt[1, :3] = ids[:6], ids[6:9]
    runs = [DecodeRunner(lay, host_tier=True, identity=identity, block_table=bt, seq_lens=lens,
                         shared_residency=shared) for shared in (True, False)]
    g = torch.Generator().manual_seed(2)

    def store(rows, at):
        """The tokens `at` of the rows, the same in both runners."""
        t = runs[0].block_table.cpu().numpy()
        pos = torch.tensor([int(t[r, i // P]) * P + int(i) % P for r, i in zip(rows, at)], dtype=torch.int64)
        order = torch.argsort(pos)
        kk, vv = (torch.randn((L, len(pos), Hkv, 128), generator=g).bfloat16()[:, order].cuda() for _ in range(2))
        for run in runs:
            for l in range(L) if by_layer else [0]:
                n = 1 if by_layer else L
                run.store(l, n, kk[l:l + n], vv[l:l + n], pos[order].cuda())

    def step():
        q = torch.randn((L, B, Hq, 128), generator=g).bfloat16().cuda()
        for run in runs:
            run.step(q)
        torch.cuda.synchronize()
        a, b = runs
        assert int(a.status.item()) == int(b.status.item()) == 0
        assert torch.equal(a.sel, b.sel) and torch.equal(a.out, b.out)
        for n in ("block_table", "seq_lens"):
            assert torch.equal(getattr(a, n), getattr(b, n))
        names = ["k", "v"] + (["k_scale", "v_scale"] if fmt != "bf16" else [])
        slots = a.cache.page_of[0].cpu().numpy()
        live = a.table.ref.cpu().numpy() > 0     # (a free page's bytes are nobody's)
        at = np.flatnonzero((slots >= 0) & live[np.maximum(slots, 0)])
        assert len(at)
        for n in names:
            pool = getattr(a.cache, n + ("_pool" if len(n) == 1 else "")).cpu()
            mir = getattr(a.cache, n + "_mirror")
            assert torch.equal(mir, getattr(b.cache, n + "_mirror")), n
            assert torch.equal(pool[:, at], mir[:, slots[at]]), n
        assert bool((a.cache.slot_of[1:] == -1).all()) and bool((a.cache.page_of[1:] == -1).all())

    store([0] * int(lens[0]) + [1] * int(lens[1]), list(range(lens[0])) + list(range(lens[1])))
    step()
    for run in runs:
        run.fork(_dev([0, 1, 0, 0]), _dev([lens[0] + 1, lens[1] + 1, lens[0] + 1, 0]))
    store([0, 1, 2], [lens[0], lens[1], lens[0]])           # into pages that hold a slot, and new ones
    step()
    for t in range(3):
        new = runs[0].seq_lens.cpu().numpy() + 1
        for run in runs:
            run.fork(_dev([0, 1, 2, 3]), _dev(new))
        store([0, 1, 2, 3], list(new - 1))
        step()
        if t == 1:
            for run in runs:
                run.compact()
            step()
    for run in runs:
        run.fork(_dev([1, 1, -1, 3]))
        run.compact()
    step()
    ref = runs[0].table.ref
    assert torch.equal(ref, runs[1].table.ref) and int(ref.sum()) > 0


@pytest.mark.parametrize("form", ["per_layer", "preload"])
@pytest.mark.parametrize("identity", [False, True])
def test_steps_by_each_layers_state_keep_it(form, identity):
    """A runner made for shared residency whose steps go by each layer's own state (per-layer steps, preload):
    its stores do too, over an evicting pool."""
    import sparse_attention_decode_indexer_gb300 as ssa
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    P, Hq, Hkv, L, B, nmax, k = 16, 4, 2, 3, 2, 16, 1
    lay = ssa.Layout(P, Hq, Hkv, 128, True, L, B * nmax, 20, B, nmax, k, kv_format="int8_page_head")
    bt = np.arange(B * nmax, dtype=np.int32).reshape(B, nmax)
    lens = np.array([nmax * P - 9, 7 * P + 5], np.int32)
    runs = [DecodeRunner(lay, host_tier=True, identity=identity, block_table=bt, seq_lens=lens,
                         shared_residency=shared, preload_width=3 if form == "preload" else 0)
            for shared in (True, False)]
    g = torch.Generator().manual_seed(4)

    def store(pos):
        x = torch.randn((2, L, len(pos), Hkv, 128), generator=g).bfloat16().cuda()
        for run in runs:
            run.store(0, L, x[0], x[1], torch.tensor(pos, device="cuda"))
    store([r * nmax * P + i for r in range(B) for i in range(lens[r])])
    for t in range(8):
        q = torch.randn((L, B, Hq, 128), generator=g).bfloat16().cuda()
        for run in runs:
            run.step(q, per_layer=form == "per_layer")
        torch.cuda.synchronize()
        a, b = runs
        assert int(a.status.item()) == int(b.status.item()) == 0
        assert torch.equal(a.out, b.out)
        for n in ("slot_of", "page_of", "last_use", "k_pool", "v_pool", "k_scale", "v_scale"):
            assert torch.equal(getattr(a.cache, n), getattr(b.cache, n)), n
        for run in runs:
            run.seq_lens += 1
        store([int(r * nmax * P + n) for r, n in enumerate(lens)])
        lens += 1
