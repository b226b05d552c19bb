"""The page_head KV formats (e4m3 or int8 codes, one fp32 scale per page and KV head): the write path
bit for bit against the definition, the attention against 64 bits, and the whole step with a host
tier in each of its forms (copy, deferred fetch, host tail, preload, shared residency)."""
import numpy as np
import pytest
import torch

from tests.page_head_ref import RefPages, attend, sm_scale

pytestmark = pytest.mark.gpu
FORMATS = ["int8_page_head", "e4m3_page_head"]
D = 128


def _layout(fmt, P=64, Hq=8, Hkv=2, L=2, Lp=12, S=None, B=2, nmax=6, k=2):
    import sparse_attention_decode_indexer_gb300 as ssa
    return ssa.Layout(P, Hq, Hkv, D, True, L, Lp, Lp if S is None else S, B, nmax, k, kv_format=fmt)


def _bf16(rng, *shape, scale=1.0):
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16()
    return t, t.float().numpy()


def _cache(lay, host_tier=False, identity=True):
    import sparse_attention_decode_indexer_gb300 as ssa
    c = ssa.KVCache(lay, host_tier)
    ssa.ssa_lru_init(c, identity)
    return c, torch.zeros((1,), dtype=torch.int32, device="cuda")


def _pages(c, l, where="pool"):
    """(k, v, ks, vs) blocks of one layer: by slot for the pool, by page for the mirror."""
    lay = c.layout
    H, P = lay.n_kv_heads, lay.page_size
    n = lambda t: t[l].cpu().numpy()  # noqa: E731
    k = n(getattr(c, "k_" + where)).reshape(-1, H, P, D)
    v = n(getattr(c, "v_" + where)).reshape(-1, H, D, P).transpose(0, 1, 3, 2)
    tail = "" if where == "pool" else "_mirror"
    return k, v, n(getattr(c, "k_scale" + tail)), n(getattr(c, "v_scale" + tail))


def _same_pages(ref, got, ids, at):
    for name, r, g in zip(("k", "v", "k_scale", "v_scale"), (ref.k, ref.v, ref.ks, ref.vs), got):
        np.testing.assert_array_equal(r[ids], g[at], err_msg=name)


def _same_slab(ref, c, l):
    for name, r in (("slab_sum", ref.sums), ("slab_cnt", ref.cnt), ("slab_scale", ref.slab_scale),
                    ("slab", ref.slab)):
        np.testing.assert_array_equal(r, getattr(c, name)[l].cpu().numpy(), err_msg=name)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("P,Hkv", [(16, 1), (32, 8), (64, 2), (128, 4)])
@pytest.mark.parametrize("host", [False, True])
def test_store_in_pieces_equals_the_definition(fmt, P, Hkv, host):
    """Prefill, ragged pieces and single tokens, growing magnitudes (so that scales grow and old codes
    are rounded again), gaps inside a page, resident and not."""
    import sparse_attention_decode_indexer_gb300 as ssa
    L, Lp = 2, 7
    lay = _layout(fmt, P=P, Hq=Hkv, Hkv=Hkv, L=L, Lp=Lp, B=1, nmax=Lp, k=1)
    c, status = _cache(lay, host_tier=host, identity=not host)
    if host:                                     # every other page holds a slot
        for l in range(L):
            c.slot_of[l, ::2] = torch.arange(0, (Lp + 1) // 2, dtype=torch.int32, device="cuda")
            c.page_of[l, :(Lp + 1) // 2] = torch.arange(0, Lp, 2, dtype=torch.int32, device="cuda")
    refs = [RefPages(fmt, Lp, Hkv, P) for _ in range(L)]
    rng = np.random.default_rng([P, Hkv, host])
    total = Lp * P
    cuts = [0, 1, 2, P // 2 + 1, P, 3 * P, 3 * P + 5, 4 * P - 1, total - 3]
    pieces = [np.arange(a, b) for a, b in zip(cuts, cuts[1:])]
    pieces.append(np.array([total - 3, total - 1]))          # a gap
    for i, pos in enumerate(pieces):
        k, kf = _bf16(rng, L, len(pos), Hkv, D, scale=1.5 ** i)
        v, vf = _bf16(rng, L, len(pos), Hkv, D, scale=0.6 ** i)
        ssa.ssa_store_kv_mirror(c, 0, L, k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), status)
        for l in range(L):
            refs[l].store(kf[l], vf[l], pos)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for l in range(L):
        slots = c.slot_of[l].cpu().numpy()
        ids = np.flatnonzero(slots >= 0)
        _same_pages(refs[l], _pages(c, l), ids, slots[ids])
        if host:
            _same_pages(refs[l], _pages(c, l, "mirror"), np.arange(Lp), np.arange(Lp))
        _same_slab(refs[l], c, l)


@pytest.mark.parametrize("fmt", FORMATS)
def test_store_long_call_and_odd_values(fmt):
    """A call of over 4,096 tokens (page-sized chunks) that starts inside a page and skips pages; zero
    pages, values of very different size, infinities and NaN (which leave the scale alone)."""
    import sparse_attention_decode_indexer_gb300 as ssa
    P, H, Lp = 64, 2, 90
    lay = _layout(fmt, P=P, Hq=H, Hkv=H, L=1, Lp=Lp, B=1, nmax=Lp, k=1)
    c, status = _cache(lay)
    rng = np.random.default_rng(5)
    pos = np.arange(17, Lp * P - 30)
    pos = pos[(pos // P) % 9 != 4]
    assert len(pos) >= 4096
    k, _ = _bf16(rng, 1, len(pos), H, D)
    v, _ = _bf16(rng, 1, len(pos), H, D)
    k *= torch.from_numpy(2.0 ** rng.integers(-20, 20, (1, len(pos), 1, 1))).bfloat16()
    k[0, :P] = 0
    v[0, 100:400, 1] = 0
    v[0, 1000, 0, 3] = float("inf")
    v[0, 1001, 1, 4] = float("nan")
    v[0, 1002, 1, 5] = -float("inf")
    ssa.ssa_store_kv_mirror(c, 0, 1, k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), status)
    ref = RefPages(fmt, Lp, H, P)
    with np.errstate(invalid="ignore"):
        ref.store(k.float().numpy()[0], v.float().numpy()[0], pos)
    assert int(status.item()) == 0
    kr, vr, ks, vs = _pages(c, 0)
    if fmt == "e4m3_page_head":                  # NaN: either sign's code
        vr, ref.v = np.where(vr == 0xFF, 0x7F, vr), np.where(ref.v == 0xFF, 0x7F, ref.v)
    _same_pages(ref, (kr, vr, ks, vs), np.arange(Lp), np.arange(Lp))
    _same_slab(ref, c, 0)


@pytest.mark.parametrize("P,H", [(16, 8), (64, 4), (128, 1)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [511, 512, 700, 4095])
def test_store_of_short_and_long_runs_in_one_call(fmt, P, H, T):
    """Calls between an append and a prefill: single tokens, short runs, the longest short run and the
    shortest long one, and whole pages side by side, on pages with and without earlier tokens."""
    import sparse_attention_decode_indexer_gb300 as ssa
    rng = np.random.default_rng([P, T])
    lengths, page = [], 0
    pos = []
    while len(pos) < T:
        n = int(rng.choice([1, 1, 2, 8, 9, P, P, P - 1]))
        n = min(n, P, T - len(pos))
        j = int(rng.integers(0, P - n + 1)) if n < P else 0
        pos += [page * P + j + i for i in range(n)]
        lengths.append(n)
        page += int(rng.integers(1, 3))
    pos, Lp = np.array(pos), page + 1
    lay = _layout(fmt, P=P, Hq=H, Hkv=H, L=1, Lp=Lp, B=1, nmax=1, k=1)
    c, status = _cache(lay)
    ref = RefPages(fmt, Lp, H, P)
    for i in range(2):                            # the second call writes over the first's rows
        k, kf = _bf16(rng, 1, T, H, D, scale=3.0 ** i)
        v, vf = _bf16(rng, 1, T, H, D)
        ssa.ssa_store_kv_mirror(c, 0, 1, k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), status)
        ref.store(kf[0], vf[0], pos)
    assert int(status.item()) == 0
    _same_pages(ref, _pages(c, 0), np.arange(Lp), np.arange(Lp))
    _same_slab(ref, c, 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("P", [16, 32])
def test_store_of_a_prefill_and_single_tokens_in_many_layers(fmt, P):
    """Whole pages, single tokens of other requests behind them and a run of a page and a half, in so
    many layers that one CTA looks after more than 32 tokens."""
    import sparse_attention_decode_indexer_gb300 as ssa
    L, whole, single = 36, 2560 // P, 900
    Lp = whole + single + 2
    lay = _layout(fmt, P=P, Hq=1, Hkv=1, L=L, Lp=Lp, B=1, nmax=Lp, k=1)
    c, status = _cache(lay)
    rng = np.random.default_rng(P)
    ones = (whole + np.arange(single)) * P + rng.integers(0, P, single)
    pos = np.concatenate([np.arange(whole * P), ones, np.arange((Lp - 2) * P, (Lp - 2) * P + P + P // 2)])
    assert len(pos) * L > 2048 * 48
    k, kf = _bf16(rng, L, len(pos), 1, D)
    v, vf = _bf16(rng, L, len(pos), 1, D)
    ssa.ssa_store_kv_mirror(c, 0, L, k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), status)
    assert int(status.item()) == 0
    for l in (0, 17, L - 1):
        ref = RefPages(fmt, Lp, 1, P)
        ref.store(kf[l], vf[l], pos)
        _same_pages(ref, _pages(c, l), np.arange(Lp), c.slot_of[l].cpu().numpy())
        _same_slab(ref, c, l)


def test_store_flags_bad_positions():
    import sparse_attention_decode_indexer_gb300 as ssa
    lay = _layout("int8_page_head", P=16, Hq=1, Hkv=1, L=1, Lp=3, B=1, nmax=3, k=1)
    x = torch.ones((1, 2, 1, D), dtype=torch.bfloat16, device="cuda")
    for pos, bits in (([48, 49], ssa.ST_BAD_ID), ([-1, 0], ssa.ST_BAD_ID), ([5, 5], ssa.ST_BAD_POS),
                      ([5, 4], ssa.ST_BAD_POS)):
        c, status = _cache(lay)
        ssa.ssa_store_kv_mirror(c, 0, 1, x, x, torch.tensor(pos, device="cuda"), status)
        assert int(status.item()) & bits, pos


def _filled(fmt, lay, rng, host_tier=False, identity=True, lens=None, spread=3.0):
    """A cache with every logical page stored, and the reference states."""
    import sparse_attention_decode_indexer_gb300 as ssa
    c, status = _cache(lay, host_tier, identity)
    L, H, P, Lp = lay.n_layers, lay.n_kv_heads, lay.page_size, lay.logical_pages
    refs = [RefPages(fmt, Lp, H, P) for _ in range(L)]
    pos = np.arange(Lp * P)
    for l in range(L):
        mag = torch.from_numpy(2.0 ** rng.uniform(-spread, spread, (1, Lp, 1, H, 1))).bfloat16()
        k, _ = _bf16(rng, 1, Lp * P, H, D)
        v = (_bf16(rng, 1, Lp, P, H, D)[0] * mag).reshape(1, Lp * P, H, D)
        ssa.ssa_store_kv_mirror(c, l, 1, k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), status)
        refs[l].store(k.float().numpy()[0], v.float().numpy()[0], pos)
    assert int(status.item()) == 0
    return c, status, refs


def _check_attention(lay, refs, q, sel, bt, lens, out, fmt):
    P, H, G = lay.page_size, lay.n_kv_heads, lay.n_q_heads // lay.n_kv_heads
    out = out.float().cpu().numpy()
    qn = q.float().cpu().numpy()
    for l in range(sel.shape[0]):
        for b in range(sel.shape[1]):
            s = sel[l, b]
            s = s[s >= 0]
            ids = bt[b, s]
            live = (s[:, None] * P + np.arange(P)) < lens[b]
            for h in range(H):
                want, bound = attend(fmt, refs[l].k[ids, h], refs[l].v[ids, h], refs[l].ks[ids, h],
                                     refs[l].vs[ids, h], qn[l, b, h * G:(h + 1) * G], sm_scale(), live)
                got = out[l, b, h * G:(h + 1) * G]
                assert np.all(np.abs(got - want) <= bound), (l, b, h, np.max(np.abs(got - want) / bound))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("P,Hq,Hkv,k,lens", [
    (16, 8, 1, 3, (1, 95, 0)),                   # one token; a request without any
    (32, 5, 1, 5, (192, 33, 32)),                # an odd group
    (64, 16, 2, 2, (384, 65, 300)),
    (128, 64, 8, 1, (257, 640, 129)),
    (64, 4, 4, 47, (384, 384, 7)),               # every page selected
])
def test_attention_against_64_bits(fmt, P, Hq, Hkv, k, lens):
    import sparse_attention_decode_indexer_gb300 as ssa
    B, L = len(lens), 2
    nmax = max(-(-n // P) for n in lens)
    lay = _layout(fmt, P=P, Hq=Hq, Hkv=Hkv, L=L, Lp=B * nmax, B=B, nmax=nmax, k=k)
    rng = np.random.default_rng([P, Hq, k])
    c, status, refs = _filled(fmt, lay, rng)
    bt = np.arange(B * nmax, dtype=np.int32).reshape(B, nmax)
    W = lay.max_sel
    sel = np.full((L, B, W), -1, np.int32)
    for l in range(L):
        for b in range(B):
            n = -(-lens[b] // P)
            pick = rng.permutation(max(n - 1, 0))[:k]
            s = np.sort(np.append(pick, n - 1)) if n else np.empty(0, np.int64)
            sel[l, b, :len(s)] = s
    phys = np.where(sel >= 0, np.take_along_axis(np.broadcast_to(bt, (L, B, nmax)), np.maximum(sel, 0), -1), -1)
    q, _ = _bf16(rng, L, B, Hq, D, scale=2.0)
    q = q.cuda()
    out = torch.full((L, B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros((ssa.ssa_workspace_size(lay),), dtype=torch.uint8, device="cuda")
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x.astype(np.int32))).cuda()  # noqa: E731
    args = (dev(sel), dev(phys), dev(np.asarray(lens)), sm_scale())
    ssa.ssa_sparse_paged_decode(c, 0, L, q, *args, out, status, ws)
    first = out.clone()
    ssa.ssa_sparse_paged_decode(c, 0, L, q, *args, out, status, ws)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(first, out)               # the same bits twice
    _check_attention(lay, refs, q, sel, bt, lens, out, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("P,B", [(16, 3), (32, 3), (16, 40), (32, 40)])
def test_attention_over_small_pages_with_holes(fmt, P, B):
    """Rows of more entries than the kernel compacts at a time, padding and unresolved pages anywhere in
    them, requests that end inside a page, one selected page, none; then the same pages from the host."""
    import sparse_attention_decode_indexer_gb300 as ssa
    L, Hkv, Hq, nmax, k = 2, 2, 6, 61, 47
    rng = np.random.default_rng([P, B])
    lay = _layout(fmt, P=P, Hq=Hq, Hkv=Hkv, L=L, Lp=nmax, B=B, nmax=nmax, k=k)
    c, status, refs = _filled(fmt, lay, rng, host_tier=True)
    bt = np.broadcast_to(np.arange(nmax, dtype=np.int32), (B, nmax))      # the requests share their pages
    lens = rng.integers(1, nmax * P + 1, B)
    lens[:2] = nmax * P - 3, 1
    W = lay.max_sel
    sel, phys = np.full((L, B, W), -1, np.int32), np.full((L, B, W), -1, np.int32)
    slot_of = c.slot_of.cpu().numpy()
    for l in range(L):
        for b in range(B):
            n = -(-int(lens[b]) // P)
            s = np.sort(rng.permutation(n)[:k + 1])
            at = np.sort(rng.permutation(W)[:len(s)])                     # padding between the entries
            sel[l, b, at] = s
            phys[l, b, at] = slot_of[l, s]
    holes = (sel >= 0) & (rng.random(sel.shape) < 0.2)
    holes[:, 2] = sel[:, 2] >= 0                                          # a row without any page
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x.astype(np.int32))).cuda()  # noqa: E731
    q = _bf16(rng, L, B, Hq, D)[0].cuda()
    ws = torch.zeros((ssa.ssa_workspace_size(lay),), dtype=torch.uint8, device="cuda")
    out = torch.full((L, B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ssa.ssa_sparse_paged_decode(c, 0, L, q, dev(sel), dev(np.where(holes, -1, phys)), dev(lens), sm_scale(),
                                out, status, ws)
    assert int(status.item()) == ssa.ST_UNRESOLVED
    assert not bool(out[:, 2].any())
    left = np.where(holes, -1, sel)
    some = [0, 1, 3] if B > 3 else [0, 1]
    _check_attention(lay, refs, q[:, some], left[:, some], bt, lens[some], out[:, some], fmt)
    status.zero_()
    tail = torch.empty_like(out)
    ssa.ssa_sparse_paged_decode(c, 0, L, q, dev(sel), dev(phys), dev(lens), sm_scale(), out, status, ws)
    c.slot_of[:, 1::3] = -1
    ssa.ssa_sparse_paged_decode_host_tail(c, 0, L, q, dev(sel), dev(bt), dev(lens), sm_scale(), tail, status, ws)
    assert int(status.item()) == 0
    assert torch.equal(out, tail)
    _check_attention(lay, refs, q[:, some], sel[:, some], bt, lens[some], out[:, some], fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heavy", [0, 1, 2, 3])
def test_attention_over_pages_of_very_different_scale(fmt, heavy):
    """V of 2^-28, 2^-14, 1 and 2^26 by page, an all-zero page, and nearly all weight on one page: a
    small page beside large ones keeps its precision."""
    import sparse_attention_decode_indexer_gb300 as ssa
    P, Hq, n = 32, 4, 5
    lay = _layout(fmt, P=P, Hq=Hq, Hkv=1, L=1, Lp=n, B=1, nmax=n, k=n)
    rng = np.random.default_rng(heavy)
    c, status = _cache(lay)
    ref = RefPages(fmt, n, 1, P)
    k, _ = _bf16(rng, 1, n * P, 1, D, scale=0.05)
    v, _ = _bf16(rng, 1, n * P, 1, D)
    order = np.array([2.0 ** -14, 2.0 ** 26, 2.0 ** -28, 1.0, 0.0], np.float32)
    v = (v.view(1, n, P, 1, D) * torch.from_numpy(order).view(1, n, 1, 1, 1).bfloat16()).view(1, n * P, 1, D)
    q, _ = _bf16(rng, 1, 1, Hq, D)
    # the heavy page's keys lie along q: its scores are about 90 above the others'
    k.view(n, P, D)[heavy] += (q[0, 0].float().mean(0) * 16).bfloat16()
    ssa.ssa_store_kv_mirror(c, 0, 1, k.cuda(), v.cuda(), torch.arange(n * P, device="cuda"), status)
    ref.store(k.float().numpy()[0], v.float().numpy()[0], np.arange(n * P))
    sel = torch.full((1, 1, lay.max_sel), -1, dtype=torch.int32, device="cuda")
    sel[..., :n] = torch.arange(n)
    lens = torch.tensor([n * P], dtype=torch.int32, device="cuda")
    out = torch.empty((1, 1, Hq, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros((ssa.ssa_workspace_size(lay),), dtype=torch.uint8, device="cuda")
    ssa.ssa_sparse_paged_decode(c, 0, 1, q.cuda(), sel, sel, lens, sm_scale(), out, status, ws)
    assert int(status.item()) == 0
    _check_attention(lay, [ref], q, sel.cpu().numpy(), np.arange(n)[None], [n * P], out, fmt)


def test_pool_beyond_4_gib():
    """Store, attention and page copy at slots whose byte offsets pass 2^32 (two pools of 9.2 GB)."""
    import sparse_attention_decode_indexer_gb300 as ssa
    fmt, P, H, S, L = "int8_page_head", 64, 8, 70000, 2
    lay = _layout(fmt, P=P, Hq=H, Hkv=H, L=L, Lp=S, S=S, B=1, nmax=4, k=3)
    c, status = _cache(lay)
    ws = torch.zeros((ssa.ssa_workspace_size(lay),), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(2)
    ids = np.array([3, S - 9, S - 2, S - 1])
    T = 3 * P + 9
    order = np.concatenate([i * P + np.arange(P) for i in ids])[:T]
    for step in (300, 0):                         # enough tokens for the whole-page kernel, or not
        k, kf = _bf16(rng, L, T + step, H, D)
        v, vf = _bf16(rng, L, T + step, H, D)
        pos = np.concatenate([order[:P], 10 * P + np.arange(step), order[P:]])
        c.slab_cnt.zero_()
        c.slab_sum.zero_()
        ssa.ssa_store_kv_mirror(c, 0, L, k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), status)
        keep = np.concatenate([np.arange(P), P + step + np.arange(T - P)])
        refs = []
        for l in range(L):
            ref = RefPages(fmt, 4, H, P)
            ref.store(kf[l][keep], vf[l][keep], np.arange(T))
            refs.append(ref)
            got = [getattr(c, n)[l, torch.from_numpy(ids).cuda()].cpu().numpy()
                   for n in ("k_pool", "v_pool", "k_scale", "v_scale")]
            got[0] = got[0].reshape(4, H, P, D)
            got[1] = got[1].reshape(4, H, D, P).transpose(0, 1, 3, 2)
            _same_pages(ref, got, np.arange(4), np.arange(4))
    sel = torch.full((L, 1, lay.max_sel), -1, dtype=torch.int32, device="cuda")
    phys = sel.clone()
    sel[..., :4] = torch.arange(4)
    phys[..., :4] = torch.from_numpy(ids.astype(np.int32))
    q, _ = _bf16(rng, L, 1, H, D)
    out = torch.empty((L, 1, H, D), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    ssa.ssa_sparse_paged_decode(c, 0, L, q.cuda(), sel, phys, lens, sm_scale(), out, status, ws)
    _check_attention(lay, refs, q, sel.cpu().numpy(), np.arange(4)[None], [T], out, fmt)
    ssa.ssa_copy_pages(c, torch.tensor([S - 1, 3], dtype=torch.int32, device="cuda"),
                       torch.tensor([7, S - 5], dtype=torch.int32, device="cuda"), status, ws)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for n in ("k_pool", "v_pool", "k_scale", "v_scale", "slab", "slab_sum", "slab_cnt"):
        t = getattr(c, n)
        assert torch.equal(t[:, 7], t[:, S - 1]) and torch.equal(t[:, S - 5], t[:, 3]), n


def test_captured_store_and_attention_replay():
    """A store and an attention captured on a stream of their own: the replay stores what k, v and pos
    hold then, into pages that were cleared, and attends over it."""
    import sparse_attention_decode_indexer_gb300 as ssa
    fmt, P = "int8_page_head", 64
    lay = _layout(fmt, P=P, Hq=8, Hkv=2, L=1, Lp=6, B=1, nmax=6, k=5)
    rng = np.random.default_rng(8)
    for T in (1, 300):
        c, status = _cache(lay)
        k, v = (torch.zeros((1, T, 2, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pos = torch.arange(T, device="cuda")
        q = _bf16(rng, 1, 1, 8, D)[0]
        qd = q.cuda()
        sel = torch.full((1, 1, lay.max_sel), -1, dtype=torch.int32, device="cuda")
        n = -(-T // P)
        sel[..., :n] = torch.arange(n)
        lens = torch.tensor([T], dtype=torch.int32, device="cuda")
        out = torch.empty((1, 1, 8, D), dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros((ssa.ssa_workspace_size(lay),), dtype=torch.uint8, device="cuda")

        def calls():
            c.slab_cnt.zero_()
            c.slab_sum.zero_()
            ssa.ssa_store_kv_mirror(c, 0, 1, k, v, pos, status)
            ssa.ssa_sparse_paged_decode(c, 0, 1, qd, sel, sel, lens, sm_scale(), out, status, ws)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            calls()
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                calls()
        for scale in (4.0, 0.5):
            kk, kf = _bf16(rng, 1, T, 2, D, scale=scale)
            vv, vf = _bf16(rng, 1, T, 2, D, scale=scale)
            k.copy_(kk)
            v.copy_(vv)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            ref = RefPages(fmt, 6, 2, P)
            ref.store(kf[0], vf[0], np.arange(T))
            assert int(status.item()) == 0
            _same_slab(ref, c, 0)
            _check_attention(lay, [ref], q, sel.cpu().numpy(), np.arange(6)[None], [T], out, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_unselected_bytes_do_not_matter(fmt):
    """Codes behind a request's last token (NaN codes and large ones) leave the output as it is."""
    import sparse_attention_decode_indexer_gb300 as ssa
    lay = _layout(fmt, P=64, Hq=8, Hkv=1, L=1, Lp=2, B=1, nmax=2, k=1)
    rng = np.random.default_rng(3)
    c, status, refs = _filled(fmt, lay, rng)
    lens = torch.tensor([64 + 21], dtype=torch.int32, device="cuda")
    sel = torch.full((1, 1, lay.max_sel), -1, dtype=torch.int32, device="cuda")
    sel[..., :2] = torch.tensor([0, 1])
    q = _bf16(rng, 1, 1, 8, D)[0].cuda()
    ws = torch.zeros((ssa.ssa_workspace_size(lay),), dtype=torch.uint8, device="cuda")
    outs = []
    for byte in (0x00, 0x7F, 0xFF, 0x80):
        c.k_pool.view(1, 2, 64, D)[0, 1, 21:] = byte
        c.v_pool.view(1, 2, D, 64)[0, 1, :, 21:] = byte
        out = torch.empty((1, 1, 8, D), dtype=torch.bfloat16, device="cuda")
        ssa.ssa_sparse_paged_decode(c, 0, 1, q, sel, sel, lens, sm_scale(), out, status, ws)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs)
    assert bool(outs[0].isfinite().all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("form", ["copy", "fetch", "overlap", "preload", "shared", "per_layer", "graphs"])
def test_decode_steps_with_a_host_tier(fmt, form):
    """Runner steps over an evicting pool: after each step every bound slot holds its page's mirror bytes
    and scales, and the attention over the selection is that of 64 bits."""
    import sparse_attention_decode_indexer_gb300 as ssa
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    P, Hq, Hkv, L, B, nmax, k = 32, 16, 4, 3, 2, 14, 3
    lens = (14 * P, 9 * P + 5)
    # 28 pages in use; 28 slots a layer (fewer than the 60 logical pages), or all of them shared
    lay = _layout(fmt, P=P, Hq=Hq, Hkv=Hkv, L=L, Lp=B * nmax if form == "shared" else 60, S=28, B=B,
                  nmax=nmax, k=k)
    rng = np.random.default_rng(11)
    bt = np.arange(B * nmax, dtype=np.int32).reshape(B, nmax)
    run = DecodeRunner(lay, host_tier=True, identity=False, block_table=bt, seq_lens=np.asarray(lens),
                       preload_width=5 if form == "preload" else 0, shared_residency=form == "shared",
                       fetch_in_attention=form == "fetch", graphs=form == "graphs",
                       overlap_groups=2 if form == "overlap" else 0)
    c = run.cache
    refs = [RefPages(fmt, lay.logical_pages, Hkv, P) for _ in range(L)]
    pos = np.arange(B * nmax * P)
    k_, _ = _bf16(rng, L, len(pos), Hkv, D)
    v_, _ = _bf16(rng, L, len(pos), Hkv, D)
    run.store(0, L, k_.cuda(), v_.cuda(), torch.from_numpy(pos).cuda())
    for l in range(L):
        refs[l].store(k_.float().numpy()[l], v_.float().numpy()[l], pos)
    q = torch.empty((L, B, Hq, D), dtype=torch.bfloat16, device="cuda")
    missed = 0
    for step in range(6):
        q.copy_(_bf16(rng, L, B, Hq, D)[0])
        run.step(q, per_layer=form == "per_layer")
        torch.cuda.synchronize()
        assert int(run.status.item()) == 0
        missed += int(run.n_miss[:1 if form == "shared" else L].sum())
        sel = run.sel.cpu().numpy()
        _check_attention(lay, refs, q, sel, bt, lens, run.out, fmt)
        for l in range(L):
            own = c.page_of[0 if form == "shared" else l].cpu().numpy()
            slots = np.flatnonzero(own >= 0)
            _same_pages(refs[l], _pages(c, l), own[slots], slots)
    assert missed > 0
    # zero-copy host tail over the same selection: same pages, same arithmetic
    if form == "copy":
        out = torch.empty_like(run.out)
        ssa.ssa_sparse_paged_decode_host_tail(c, 0, L, q, run.sel, run.block_table, run.seq_lens,
                                              sm_scale(), out, run.status, run.ws)
        c.slot_of.fill_(-1)
        out2 = torch.empty_like(run.out)
        ssa.ssa_sparse_paged_decode_host_tail(c, 0, L, q, run.sel, run.block_table, run.seq_lens,
                                              sm_scale(), out2, run.status, run.ws)
        torch.cuda.synchronize()
        assert int(run.status.item()) == 0
        assert torch.equal(out, run.out) and torch.equal(out2, run.out)


def test_layout_formats_and_refusals():
    import sparse_attention_decode_indexer_gb300 as ssa
    with pytest.raises(ValueError):
        _layout("int4")
    lay = _layout("int8_page_head")
    c, status = _cache(lay)
    x = torch.zeros((2 * 2 * 2 * D + 4,), dtype=torch.bfloat16, device="cuda")[1:1 + 2 * 2 * 2 * D]
    with pytest.raises(ssa.SsaError):            # not 16-byte aligned
        ssa.ssa_store_kv_mirror(c, 0, 2, x, x, torch.zeros((2,), dtype=torch.int64, device="cuda"), status)
