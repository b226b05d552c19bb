"""ssa_beam_select against the scores of all candidates in 64 bits.

Scores: an exponential is off by at most 2^-21 of itself, a thread's fp32 sum of 32 of them by 32 *
2^-24, so the logarithm of the sum by less than 2^-18, and the score rounded to fp32 by 2^-24 of
itself more.  Candidates whose scores in 64 bits are further apart than twice that must come in their
order; equal ones (the same logit, rows that are alike) in that of their row and token.
"""
import ctypes
import math

import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
gpu = pytest.mark.gpu
EPS = 2.0 ** -18


def candidates(x, scores, finished, eos):
    """[B][V] scores in 64 bits, -inf where there is none."""
    x = x.double()
    x = torch.where(x.isnan(), -math.inf, x.clamp(max=2.0 ** 126))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    # rows that are alike must have equal sums, whatever order torch adds them in: to 2^-40
    ln = ((x - m).exp().sum(-1, keepdim=True).log() * 2.0 ** 40).round() * 2.0 ** -40
    # (x - m first: beside a mask of 1e38 the logarithm would be lost)
    c = torch.where(x > -math.inf, x - m - ln + scores.double()[:, None], -math.inf)
    if finished is not None:
        stay = torch.full_like(c, -math.inf)
        stay[:, eos] = scores.double()
        c = torch.where(finished.bool()[:, None], stay, c)
    return torch.where(c.isnan(), -math.inf, c)


def make(G, K, V, dtype=F32, seed=0, max_len=0, eos=-1, pad=0, shift=0, wide=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = G * K
    x = wide * 3 * torch.randn((B, V + pad + shift), generator=g, device="cuda")
    x = x.to(dtype)[:, shift:shift + V]
    st = ssa.BeamState(G, K, max_len=max_len, finished=eos >= 0)
    st.scores.copy_(-9 * torch.rand((B,), generator=g, device="cuda"))
    if eos >= 0:
        st.finished.copy_(torch.rand((B,), generator=g, device="cuda") < 0.3)
    if max_len:
        st.history.copy_(torch.randint(0, V, (B, max_len), generator=g, device="cuda"))
        st.hist_len.copy_(torch.randint(0, max_len, (G,), generator=g, device="cuda"))
    return x, st


def copy_of(st):
    out = ssa.BeamState(st.groups, st.beams, st.max_len, st.finished is not None)
    for name in ("scores", "finished", "history", "hist_len"):
        if getattr(st, name) is not None:
            getattr(out, name).copy_(getattr(st, name))
    return out


def select(x, st, eos=-1, out=None, lens=None, ws=None, expect=0):
    B = st.groups * st.beams
    parent, token = (torch.full((B,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    new = torch.full((B,), 77, dtype=torch.int32, device="cuda") if lens is not None else None
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.zeros((ssa.ssa_beam_workspace_size(st.groups, st.beams),), dtype=torch.uint8, device="cuda")
    ssa.ssa_beam_select(x, st, parent, token, status, ws, out=out, eos=eos, seq_lens=lens, new_lens=new)
    assert status.item() == expect
    return parent, token, new


def check(x, st, eos=-1, in_place=False, exact=False, expect=0):
    """One call against the definition, states and all."""
    G, K, V = st.groups, st.beams, x.shape[1]
    before = copy_of(st)
    out = st if in_place else copy_of(st)
    if not in_place and out.history is not None:
        out.history.fill_(-5)
    lens = torch.randint(1, 1000, (G * K,), device="cuda", dtype=torch.int32)
    parent, token, new = select(x, st, eos, out=None if in_place else out, lens=lens, expect=expect)
    if not in_place:
        assert torch.equal(st.scores.view(torch.int32), before.scores.view(torch.int32))
    cand = candidates(x, before.scores, before.finished, eos).view(G, K * V)
    val, idx = cand.sort(dim=-1, descending=True, stable=True)
    if val.shape[1] < K:
        val = torch.nn.functional.pad(val, (0, K - val.shape[1]), value=-math.inf)
        idx = torch.nn.functional.pad(idx, (0, K - idx.shape[1]))
    val, idx = val[:, :K], idx[:, :K]
    row, tok = parent.view(G, K).long(), token.view(G, K).long()
    none = val == -math.inf
    assert torch.equal(row == -1, none) and torch.equal(tok == -1, none)
    sc = out.scores.view(G, K)
    assert (sc[none] == -math.inf).all()
    tol = EPS + 2.0 ** -24 * val.abs()
    assert torch.where(none, True, (sc.double() - val).abs() <= tol).all()
    first = torch.arange(G, device="cuda")[:, None] * K
    at = torch.where(none, 0, (row - first) * V + tok)
    assert ((at >= 0) & (at < K * V)).all()
    # what was chosen is, in 64 bits, as good as what should have been
    assert torch.where(none, True, (cand.gather(1, at) - val).abs() <= 2 * tol).all()
    for g in range(G):
        got = at[g][~none[g]].tolist()
        assert len(set(got)) == len(got)
    if exact:
        assert torch.equal(torch.where(none, -1, at), torch.where(none, -1, idx))
    # the states follow
    par = parent.long().clamp(min=0)
    live = parent >= 0
    assert torch.equal(new, torch.where(live, lens[par] + 1, 0).int())
    if eos >= 0:
        want = torch.where(live, (before.finished[par].bool() | (token == eos)), False)
        assert torch.equal(out.finished.bool(), want)
    if before.history is not None:
        n = before.hist_len.clamp(0, st.max_len)
        full = (before.hist_len < 0) | (before.hist_len >= st.max_len)
        c = torch.arange(st.max_len, device="cuda")
        rn, rf = n.repeat_interleave(K)[:, None], full.repeat_interleave(K)[:, None]
        was = before.history if in_place else torch.full_like(before.history, -5)
        want = torch.where(c < rn, before.history[par], was)
        want = torch.where((c == rn) & ~rf, token[:, None], want)
        want = torch.where(live[:, None], want, was)
        assert torch.equal(out.history, want)
        assert torch.equal(out.hist_len, torch.where(full, n, n + 1).int())


@gpu
@pytest.mark.parametrize("V", [1, 2, 7, 8, 100, 1023, 8191, 8192, 8193, 32000, 100003])
@pytest.mark.parametrize("K", [1, 2, 5, 8])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_sizes(V, K, dtype):
    x, st = make(3, K, V, dtype, seed=V + K)
    check(x, st)


@gpu
@pytest.mark.parametrize("G,K,V", [(1, 32, 262144), (2, 31, 5000), (300, 1, 999), (70, 4, 20000), (1, 1, 1 << 23),
                                   (1, 16, 40)])
def test_large_and_many(G, K, V):
    x, st = make(G, K, V, BF16, seed=K)
    check(x, st)


@gpu
@pytest.mark.parametrize("pad,shift", [(5, 0), (8, 0), (0, 1), (3, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [8192, 9001])
def test_strided_rows(pad, shift, dtype, V):
    x, st = make(2, 4, V, dtype, seed=pad, pad=pad, shift=shift)
    check(x, st)


@gpu
@pytest.mark.parametrize("max_len", [1, 3, 500, 4096])
@pytest.mark.parametrize("in_place", [False, True])
def test_states(max_len, in_place):
    x, st = make(5, 6, 3000, BF16, seed=max_len, max_len=max_len, eos=11)
    check(x, st, eos=11, in_place=in_place)


@gpu
def test_full_and_bad_histories_are_flagged():
    x, st = make(4, 2, 500, seed=1, max_len=16)
    st.hist_len.copy_(torch.tensor([16, -1, 40, 3]))
    check(x, st, in_place=True, expect=ssa.ST_BAD_POS)


@gpu
def test_rows_beyond_4_gib():
    x, st = make(1, 3, 9000, BF16, seed=6)
    far = torch.empty((3, 1_200_000_000), dtype=BF16, device="cuda")[:, :9000]
    far.copy_(x)
    check(far, st)


@gpu
def test_ties_go_to_the_lowest_row_and_token():
    G, K, V = 3, 4, 20000
    x = torch.zeros((G * K, V), device="cuda")
    st = ssa.BeamState(G, K)
    st.scores.zero_()
    x[4:8, 17000:] = 2.0                    # equal rows, equal best tokens late in the row
    x[8:12, 5::7] = 1.5
    st.scores[8:12] = torch.tensor([-1.0, -0.5, -0.5, -3.0])
    check(x, st, exact=True)
    # one row only: its first tokens
    first = ssa.BeamState(G, K)
    check(x, first, exact=True)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_equal_logits_in_unaligned_rows(dtype):
    """Rows that are alike give the same sums wherever they start."""
    K, V = 8, 9001
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((1, V), generator=g, device="cuda").to(dtype).expand(K, V).contiguous()
    st = ssa.BeamState(1, K)
    st.scores.fill_(-2.0)
    check(x, st, exact=True)


@gpu
def test_masked_logits_and_dead_rows():
    x, st = make(6, 3, 5000, seed=4, eos=7)
    st.finished.zero_()
    x[0:3] = -math.inf                      # a group without any candidate
    x[3:6, 10:] = -math.inf                 # ten tokens left in each
    x[6:9] = -math.inf
    x[7, 4321] = 1.0                        # one candidate in the group
    x[9, 5] = math.nan                      # a NaN is masked, the rest stays
    x[10, 9] = math.inf
    st.scores[12:15] = -math.inf            # dead rows
    st.scores[13] = math.nan
    st.scores[15] = -math.inf
    st.finished[16] = 1
    check(x, st, eos=7)


@gpu
def test_all_ended():
    x, st = make(2, 4, 300, seed=8, eos=0, max_len=9)
    st.finished.fill_(1)
    check(x, st, eos=0, in_place=True)


@gpu
def test_large_logits():
    x, st = make(2, 4, 4000, F32, seed=9, wide=1e4)
    check(x, st)
    x, st = make(2, 4, 4000, F32, seed=9, wide=1e-4)
    check(x, st)


@gpu
def test_same_bits_graph_and_workspace_left_clean():
    x, st = make(7, 4, 50000, BF16, seed=2, max_len=40, eos=3)
    st.hist_len.clamp_(max=30)              # room for the steps below
    ws = torch.zeros((ssa.ssa_beam_workspace_size(7, 4),), dtype=torch.uint8, device="cuda")
    a, b = copy_of(st), copy_of(st)
    pa, ta, _ = select(x, st, 3, out=a, ws=ws)
    pb, tb = torch.empty_like(pa), torch.empty_like(ta)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ssa.ssa_beam_select(x, st, pb, tb, None, ws, out=b, eos=3, stream=side)
    side.synchronize()
    assert torch.equal(pa, pb) and torch.equal(ta, tb) and torch.equal(a.scores, b.scores)
    g = torch.cuda.CUDAGraph()
    live = copy_of(st)
    with torch.cuda.graph(g):
        ssa.ssa_beam_select(x, live, pb, tb, None, ws, eos=3)
    for _ in range(3):          # each replay goes on from the last one's states
        want = copy_of(live)
        p, t, _ = select(x, want, 3, ws=ws)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(pb, p) and torch.equal(tb, t)
        for name in ("scores", "finished", "history", "hist_len"):
            assert torch.equal(getattr(live, name), getattr(want, name))


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [40000, 300000])
@pytest.mark.parametrize("K", [3, 32])
def test_rising_equal_and_masked_by_a_number(dtype, V, K):
    """Every logit better than those before it; all equal; a mask of one finite value."""
    G = 40 if V == 40000 else 2
    st = ssa.BeamState(G, K)
    st.scores.copy_(-torch.arange(G * K, device="cuda") * 0.25)
    up = torch.linspace(-8, 8, V, device="cuda").to(dtype).expand(G * K, V).contiguous()
    check(up, copy_of(st))
    check(torch.full_like(up, -1.5), copy_of(st), exact=True)
    low = torch.full_like(up, torch.finfo(dtype).min)
    low[::2, 777::5000] = 3.0
    check(low, copy_of(st))


def _cpu(G=2, K=3, V=10, eos=-1, max_len=0, **kw):
    st = ssa.BeamState(G, K, max_len, eos >= 0, device="cpu")
    i32 = dict(dtype=torch.int32)
    z = dict(logits=torch.zeros((G * K, V)), state=st, parent=torch.zeros((G * K,), **i32),
             token=torch.zeros((G * K,), **i32), status=None, eos=eos,
             ws=torch.zeros((ssa.ssa_beam_workspace_size(G, K),), dtype=torch.uint8))
    z.update(kw)
    ssa.ssa_beam_select(**z)


@pytest.mark.parametrize("kw,match", [
    (dict(logits=torch.zeros((6, 10), dtype=torch.float64)), "logits"),
    (dict(logits=torch.zeros((5, 10))), "logits"),
    (dict(logits=torch.zeros((6, 20))[:, ::2]), "logits"),
    (dict(parent=torch.zeros((6,), dtype=torch.int64)), "parent"),
    (dict(token=torch.zeros((5,), dtype=torch.int32)), "token"),
    (dict(eos=3, state=ssa.BeamState(2, 3, device="cpu")), "eos"),
    (dict(state=ssa.BeamState(2, 3, finished=True, device="cpu")), "eos"),
    (dict(out=ssa.BeamState(3, 2, device="cpu")), "other sizes"),
    (dict(out=ssa.BeamState(2, 3, 5, device="cpu")), "other sizes"),
    (dict(seq_lens=torch.zeros((6,), dtype=torch.int32)), "both or none"),
    (dict(ws=torch.zeros((8,), dtype=torch.uint8)), "ws"),
    (dict(), "current CUDA device"),
])
def test_refusals(kw, match):
    with pytest.raises(ValueError, match=match):
        _cpu(**kw)


def test_state():
    st = ssa.BeamState(2, 3, 4, True, device="cpu")
    assert st.scores.tolist() == [0, -math.inf, -math.inf] * 2
    with pytest.raises(AttributeError, match="in place"):
        st.scores = torch.zeros((6,))


def test_c_refusals():
    L, p = ssa.lib(), 0x10000
    assert L.ssa_beam_workspace_size(0, 1) == 0 and L.ssa_beam_workspace_size(1, 33) == 0

    def go(dtype=0, G=2, K=3, V=100, x=p, stride=100, i=(p, None, None, None), o=None, max_len=0, eos=-1, par=p,
           tok=p, lens=None, new=None, ws=p):
        i = ssa.SsaBeams(*i)
        o = i if o is None else ssa.SsaBeams(*o)
        return L.ssa_beam_select(dtype, G, K, V, x, stride, ctypes.byref(i), ctypes.byref(o), max_len, eos, par, tok,
                                 lens, new, None, ws, None)
    assert go(dtype=3) == -3 and go(K=33) == -3 and go(V=(1 << 23) + 1, stride=1 << 24) == -3 and go(G=70000) == -3
    assert go(G=0) == -1 and go(K=0) == -1 and go(V=0) == -1 and go(max_len=-1) == -1
    assert go(eos=100) == -1 and go(eos=-2) == -1
    assert go(x=None) == -1 and go(x=p + 1) == -1 and go(stride=99) == -1 and go(ws=None) == -1 and go(ws=p + 16) == -1
    assert go(i=(None,) * 4) == -1 and go(par=None) == -1 and go(tok=None) == -1
    assert go(eos=3) == -1 and go(i=(p, p, None, None)) == -1
    assert go(max_len=4) == -1 and go(i=(p, None, p, None)) == -1 and go(max_len=4, i=(p, None, p, None)) == -1
    assert go(lens=p) == -1 and go(new=p) == -1
