"""The operators at both ends of the serving loop as a runner calls them: prompts in (norms,
positions, attention, store), decode steps over what was stored, beams on.

The prompt's attention and a decode step over all of a request's pages are the same sum for the
prompt's last token; each is within its own tolerance of the 64-bit result (that of
tests/test_prompt.py; the 1e-2 that the decode attention's parity is held to for bf16)."""
import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa
from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
from tests.test_beam import candidates
from tests.test_prompt import offsets, reference

pytestmark = pytest.mark.gpu
BF16, D, P = torch.bfloat16, 128, 16


def make(kv_format="bf16", lens=(100, 33, 1, 64), L=2, Hq=8, Hkv=2, host_tier=False, norm=True, n=9, **kw):
    B = len(lens)
    lay = ssa.Layout(P, Hq, Hkv, D, kv_format != "bf16", L, B * n, B * n, B, n, n, kv_format=kv_format)
    g = torch.Generator().manual_seed(3)
    hn = ssa.HeadNorm(1 + 0.2 * torch.randn((L, D), generator=g), 1 + 0.2 * torch.randn((L, D), generator=g))
    run = DecodeRunner(lay, host_tier=host_tier, identity=not host_tier,
                       block_table=torch.arange(B * n).view(B, n), seq_lens=torch.tensor(lens),
                       rope=ssa.RopePlan(D), norm=hn if norm else None, **kw)
    return run, hn


def prompts(run, lens, seed=0):
    lay = run.layout
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    x = torch.randn((T, lay.n_q_heads + 2 * lay.n_kv_heads, D), generator=g, device="cuda").to(BF16)
    q, k, v = x.split([lay.n_q_heads, lay.n_kv_heads, lay.n_kv_heads], 1)
    at = torch.cat([torch.arange(n) for n in lens]).cuda()
    pos = torch.cat([torch.arange(n) + i * lay.max_pages * P for i, n in enumerate(lens)]).cuda()
    return q, k, v, pos, at


@pytest.mark.parametrize("kv_format", ["bf16", "fp8", "int8_page_head"])
@pytest.mark.parametrize("norm", [True, False])
def test_prompts_in_and_the_first_step(kv_format, norm):
    lens = (100, 33, 1, 64)
    run, hn = make(kv_format, lens, norm=norm)
    by_hand, _ = make(kv_format, lens, norm=norm)
    lay = run.layout
    last = torch.tensor(lens).cumsum(0).cuda() - 1
    q_last, want = [], []
    for l in range(lay.n_layers):
        q, k, v, pos, at = prompts(run, lens, seed=l)
        out = run.prefill(l, q, k, v, pos, offsets(list(lens)), positions=at)
        # the same by the calls themselves
        qr, kr = torch.empty(q.shape, dtype=BF16, device="cuda"), torch.empty(k.shape, dtype=BF16, device="cuda")
        if norm:
            ssa.ssa_norm_rope(run.rope, hn, at, q, k, q_out=qr, k_out=kr, layer0=l)
        else:
            ssa.ssa_rope(run.rope, at, q, k, q_out=qr, k_out=kr)
        o, _, tol, _ = reference(qr, kr, v, list(lens), list(lens), True)
        assert ((out.double() - o).abs() <= tol).all()
        by_hand.store(l, 1, k[None], v[None], pos, positions=at)
        q_last.append(q[last])
        want.append(o[last])
    for name in ("k_pool", "v_pool", "k_scale", "v_scale", "slab", "slab_cnt"):
        a, b = getattr(run.cache, name), getattr(by_hand.cache, name)
        assert a is None or torch.equal(a, b)
    # block_topk covers every page: the step attends over the whole prompt
    got = run.step(torch.stack(q_last))
    assert run.status.item() == 0
    err = (got.double() - torch.stack(want)).abs().max().item()
    assert err < (1e-2 if kv_format == "bf16" else 3e-2 * torch.stack(want).abs().max().item() + 3e-2)


def test_queries_are_normed_by_layer():
    """A step with norms is the step on queries that were normed by the call; layer by layer too."""
    lens = (40, 17)
    run, hn = make("bf16", lens)
    plain, _ = make("bf16", lens, norm=False)
    L = run.layout.n_layers
    for l in range(L):
        q, k, v, pos, at = prompts(run, lens, seed=l)
        run.prefill(l, q, k, v, pos, offsets(list(lens)), positions=at)
    for name in ("k_pool", "v_pool", "slab", "slab_scale", "slab_sum", "slab_cnt"):
        getattr(plain.cache, name).copy_(getattr(run.cache, name))
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn((L, 2, 8, D), generator=g, device="cuda").to(BF16)
    q1 = torch.empty_like(q)
    ssa.ssa_norm_rope(run.rope, hn, run.seq_lens, q, q_out=q1, offset=-1)
    plain.rope = None
    want = plain.step(q1).clone()
    assert torch.equal(run.step(q), want)
    assert torch.equal(run.step(q, per_layer=True), want)


@pytest.mark.parametrize("eos", [-1, 5])
def test_beams_follow_their_pages(eos):
    """Beam steps of a runner against the selection in 64 bits and a second runner's forks."""
    G, K, V, T = 2, 3, 50, 6
    lens = [30, 0, 0, 7, 0, 0]
    run, _ = make("bf16", lens, n=6)
    other, _ = make("bf16", lens, n=6)
    state = ssa.BeamState(G, K, max_len=T, finished=eos >= 0)
    scores = state.scores.double().clone()
    ended = torch.zeros((G * K,), dtype=torch.uint8, device="cuda") if eos >= 0 else None
    texts = [[] for _ in range(G * K)]
    g = torch.Generator(device="cuda").manual_seed(4)
    for t in range(T):
        x = 2 * torch.randn((G * K, V), generator=g, device="cuda")
        if eos >= 0 and t == 2:
            x[:, eos] += 5
        cand = candidates(x, scores, ended, eos).view(G, K * V)
        val, idx = cand.sort(dim=-1, descending=True, stable=True)
        val, idx = val[:, :K].flatten(), idx[:, :K].flatten()
        row = idx // V + torch.arange(G, device="cuda").repeat_interleave(K) * K
        tok = idx % V
        parent, token = run.beam_step(x, state, eos=eos)
        assert torch.equal(parent.long(), row) and torch.equal(token.long(), tok)
        other.fork(row.int(), other.seq_lens[row] + 1)
        assert torch.equal(run.block_table, other.block_table) and torch.equal(run.seq_lens, other.seq_lens)
        assert torch.equal(run.table.ref, other.table.ref)
        scores = val
        texts = [texts[r] + [k] for r, k in zip(row.tolist(), tok.tolist())]
        if eos >= 0:
            ended = (ended[row].bool() | (tok == eos)).to(torch.uint8)
            assert torch.equal(state.finished, ended)
    assert run.status.item() == 0
    assert state.history.tolist() == texts
    assert (state.scores.double() - scores).abs().max() < T * 2.0 ** -18


def test_beam_step_in_a_graph():
    lens = [30, 30, 9, 9]
    run, _ = make("bf16", lens, n=6)
    eager, _ = make("bf16", lens, n=6)
    a, b = (ssa.BeamState(2, 2, max_len=8) for _ in range(2))
    x = torch.randn((4, 700), device="cuda")
    with pytest.raises(RuntimeError, match="before a capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            run.beam_step(x, a)
    run.beam_step(x, a)
    eager.beam_step(x, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        parent, token = run.beam_step(x, a)
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        g.replay()
        p, t = eager.beam_step(x, b)
        assert torch.equal(parent, p) and torch.equal(token, t)
        assert torch.equal(run.block_table, eager.block_table) and torch.equal(a.history, b.history)


def test_no_beam_step_is_captured_beside_a_preload():
    lens = [30, 30]
    run, _ = make("bf16", lens, n=6, host_tier=True)
    state = ssa.BeamState(1, 2)
    x = torch.randn((2, 90), device="cuda")
    run.beam_step(x, state)
    run.enable_preload(2)
    with pytest.raises(RuntimeError, match="preload"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            run.beam_step(x, state)


def test_refusals():
    run, hn = make()
    with pytest.raises(ValueError, match="positions"):
        q, k, v, pos, at = prompts(run, (5,))
        run.prefill(0, q, k, v, pos, offsets([5]))
    with pytest.raises(ValueError, match="groups"):
        run.beam_step(torch.zeros((4, 9), device="cuda"), ssa.BeamState(3, 1))
    lay = run.layout
    kw = dict(host_tier=False, identity=True, block_table=run.block_table, seq_lens=run.seq_lens)
    with pytest.raises(ValueError, match="with rope"):
        DecodeRunner(lay, norm=hn, **kw)
    with pytest.raises(ValueError, match="norm: 3 layers"):
        DecodeRunner(lay, rope=run.rope, norm=ssa.HeadNorm(torch.ones(3, D), torch.ones(3, D)), **kw)
