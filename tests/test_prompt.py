"""ssa_prompt_attention against softmax attention in 64 bits: packed sequences, grouped heads,
causal or not, keys before the query tokens, rows without keys, splits over the keys.

Tolerance of out, per element, from the kernel's roundings (u: half a step of the type,
torch.finfo(t).eps / 2):
  * each weight rounded to the type: u * A, with A = sum_j w_j |v_j|;
  * fp32 scores: a sum of 128 exact products is off by at most 130 * 2^-23 of the sum of their
    magnitudes (times sm_scale); exp turns that into the same relative error of a weight, once
    above and once below the division; the exponential itself and its argument add less than
    2^-18 (score magnitudes below 2^4);
  * fp16 weights below 2^-14 have steps of 2^-24 beside a sum of at least one: 2^-25 |v| a key;
  * the result's own rounding: u * |out|, or u times the least normal number where |out| is below
    it and the steps get no smaller.
"""
import ctypes
import math

import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa

D = 128
BF16, F16 = torch.bfloat16, torch.float16
gpu = pytest.mark.gpu


def offsets(lens, device="cuda"):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=device)


def reference(q, k, v, lq, lk, causal, scale=None):
    """out, lse and out's tolerance, lse's tolerance, in 64 bits; what a row does not see is not
    touched at all."""
    Tq, Hq, _ = q.shape
    H = k.shape[1]
    G = Hq // H
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    u = torch.finfo(q.dtype).eps / 2
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((Tq, Hq), -math.inf, dtype=torch.float64, device=q.device)
    ltol = torch.zeros_like(lse)
    a = b = 0
    for n, m in zip(lq, lk):
        qs = q[a:a + n].double().view(n, H, G, D).permute(1, 2, 0, 3)          # [H][G][n][D]
        ks, vs = (x[b:b + m].double().transpose(0, 1)[:, None] for x in (k, v))  # [H][1][m][D]
        rows, b, a = slice(a, a + n), b + m, a + n
        if not n or not m:
            continue
        s = (qs @ ks.transpose(-1, -2)) * scale
        mag = (qs.abs().nan_to_num() @ ks.abs().nan_to_num(posinf=0.0).transpose(-1, -2)) * abs(scale)
        see = torch.ones((n, m), dtype=torch.bool, device=q.device)
        if causal:
            see = torch.arange(m, device=q.device) <= torch.arange(n, device=q.device)[:, None] + (m - n)
        s = s.masked_fill(~see, -math.inf)
        e_s = 130 * 2.0 ** -23 * mag.masked_fill(~see, 0.0).amax(-1, keepdim=True)
        top = s.amax(-1, keepdim=True)
        w = torch.where(see, (s - torch.where(top == -math.inf, 0.0, top)).exp(), 0.0)
        z = w.sum(-1, keepdim=True)
        w = torch.where(z > 0, w / z, 0.0)

        def mix(w, x):
            # 0 times an infinity that a row does not see is no part of it
            o = w @ x.nan_to_num(0.0, 0.0, 0.0)
            bad = ~x.isfinite()
            if bad.any():
                for j in bad.any(-1).any(0).any(0).nonzero()[:, 0].tolist():
                    hit = torch.where(bad[:, :, j], x[:, :, j], 0.0)[:, :, None]   # [H][1][1][D]
                    o = torch.where(see[:, j][:, None], o + hit, o)
            return o
        o = mix(w, vs)
        vabs = vs.abs().nan_to_num(0.0, 0.0, 0.0)
        t = (u + 2 * e_s + 2.0 ** -18) * (w @ vabs) + u * o.abs().clamp(min=torch.finfo(q.dtype).tiny)
        if q.dtype == F16:
            t = t + 2.0 ** -25 * m * vabs.amax()
        out[rows] = o.permute(2, 0, 1, 3).reshape(n, Hq, D)
        tol[rows] = t.permute(2, 0, 1, 3).reshape(n, Hq, D)
        lse[rows] = (top + z.log())[..., 0].permute(2, 0, 1).reshape(n, Hq)
        ltol[rows] = (e_s + 2.0 ** -18)[..., 0].permute(2, 0, 1).reshape(n, Hq)
    return out, lse, tol, ltol


def inputs(lq, lk, Hq, Hkv, dtype, seed=0, packed=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Tq, Tk = sum(lq), sum(lk)
    if packed:
        x = torch.randn((Tq, Hq + 2 * Hkv, D), generator=g, device="cuda").to(dtype)
        return x.split([Hq, Hkv, Hkv], 1)
    return tuple(torch.randn((T, H, D), generator=g, device="cuda").to(dtype)
                 for T, H in ((Tq, Hq), (Tk, Hkv), (Tk, Hkv)))


def workspace():
    # no clearing is asked for: anything may be in it
    return torch.full((ssa.ssa_prompt_workspace_size(),), 0xFF, dtype=torch.uint8, device="cuda")


def call(q, k, v, lq, lk, causal=True, **kw):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    ssa.ssa_prompt_attention(q, k, v, offsets(lq), out, status, workspace(), cu_k=offsets(lk),
                             causal=causal, lse=lse, **kw)
    assert status.item() == 0
    return out, lse


def compare(got, want):
    (out, lse), (o, s, tol, ltol) = got, want
    empty = s == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert (out[empty] == 0).all()
    odd = ~o.isfinite()
    assert torch.equal(out.double()[odd].nan_to_num(nan=5.0), o[odd].nan_to_num(nan=5.0))
    err = torch.where(odd, 0.0, (out.double() - o).abs() - tol)
    assert (err <= 0).all(), f"{err.max().item():.3e} above the tolerance"
    lerr = torch.where(empty, 0.0, (lse.double() - s).abs() - ltol)
    assert (lerr <= 0).all()


def check(lq, lk, Hq, Hkv, dtype=BF16, causal=True, seed=0, packed=False):
    q, k, v = inputs(lq, lk, Hq, Hkv, dtype, seed, packed)
    compare(call(q, k, v, lq, lk, causal), reference(q, k, v, lq, lk, causal))


@gpu
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 640, 1300])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(n, causal):
    check([n], [n], 8, 1, causal=causal, seed=n)


@gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (4, 2), (6, 2), (5, 1), (12, 2), (7, 1), (16, 2), (32, 4),
                                    (64, 8), (16, 1), (100, 1), (128, 1)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_head_groups(Hq, Hkv, dtype):
    check([150, 61], [150, 61], Hq, Hkv, dtype, seed=Hq)


@gpu
@pytest.mark.parametrize("lens", [[0], [0, 5], [5, 0], [1] * 70, [3, 0, 0, 200, 1, 129, 0, 40], [700, 1, 300],
                                  [1, 2000, 1], list(range(40))])
@pytest.mark.parametrize("causal", [True, False])
def test_packed(lens, causal):
    check(lens, lens, 16, 2, causal=causal, seed=len(lens))


@gpu
@pytest.mark.parametrize("lq,lk", [
    ([1], [1]), ([1], [20000]), ([8], [9000]), ([33], [5000]),               # keys before the queries: split
    ([7, 1, 1], [7, 4000, 600]), ([40, 3], [1, 0]), ([9, 200], [3, 100]),    # rows without keys
    ([0, 4, 0], [300, 0, 20]), ([500, 20], [900, 6000]), ([2, 0, 3], [300, 3000, 20]), ([9, 0, 0, 200], [9, 700, 1500, 200])])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (3, 3)])
def test_other_keys(lq, lk, causal, Hq, Hkv):
    check(lq, lk, Hq, Hkv, causal=causal, seed=sum(lk))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_views_of_a_projection(dtype):
    check([300, 90], [300, 90], 12, 4, dtype, packed=True)


@gpu
def test_many_rows_and_a_long_sequence():
    # more tiles than SMs; far rows alone are compared
    lq, H = [6000, 1, 2100], 8
    q, k, v = inputs(lq, lq, 4 * H, H, BF16)
    out, lse = call(q, k, v, lq, lq)
    for h in (0, 5):
        one = (q[:, 4 * h:4 * h + 4], k[:, h:h + 1], v[:, h:h + 1])
        compare((out[:, 4 * h:4 * h + 4], lse[:, 4 * h:4 * h + 4]), reference(*one, lq, lq, True))


@gpu
@pytest.mark.parametrize("lq,lk", [([300, 200], [300, 200]), ([4, 3], [900, 2500])])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_not_finite_where_nothing_is_seen(lq, lk, dtype):
    """Infinities and NaN in keys and values behind a row's last key, and in other sequences'."""
    q, k, v = inputs(lq, lk, 16, 2, dtype)
    k, v, b = k.clone(), v.clone(), lk[0]
    for i, bad in enumerate((math.nan, math.inf, -math.inf)):
        v[b - 1 - i, :, 5 + i] = bad          # the first sequence's last keys
        k[b - 1 - i, 1, 9] = bad
        v[sum(lk) - 1 - i, 0, 100 + i] = bad
    # the reference is told the same, but for keys with a row's own score
    out, lse = call(q, k, v, lq, lk)
    clean_k = k.clone()
    clean_k[b - 3:b, 1, 9] = 0
    o, s, tol, ltol = reference(q, clean_k, v, lq, lk, True)
    # rows of head 1 that see one of the changed keys are not compared
    sees = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    sees[max(0, lq[0] - 3):lq[0], 8:] = True
    keep = ~sees
    compare((out[keep], lse[keep]), (o[keep], s[keep], tol[keep], ltol[keep]))


@gpu
def test_scores_that_grow_along_the_keys():
    """The reference of the softmax moves many times, up and far: large scores come last."""
    n = 1500
    q, k, v = inputs([n], [n], 8, 1, BF16)
    k = k * torch.linspace(0.05, 6.0, n, device="cuda")[:, None, None].to(BF16)
    for causal in (True, False):
        compare(call(q, k, v, [n], [n], causal), reference(q, k, v, [n], [n], causal))


@gpu
@pytest.mark.parametrize("scale", [0.0, 0.3])
def test_scale(scale):
    q, k, v = inputs([200], [200], 4, 2, F16)
    compare(call(q, k, v, [200], [200], sm_scale=scale), reference(q, k, v, [200], [200], True, scale))


@gpu
def test_rows_outside_the_sequences_stay():
    q, k, v = inputs([100], [100], 8, 2, BF16)
    out, lse = torch.full_like(q, 3.0), torch.full((100, 8), 3.0, device="cuda")
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    cu = torch.tensor([10, 40, 40, 90], dtype=torch.int32, device="cuda")
    ssa.ssa_prompt_attention(q, k, v, cu, out, status, workspace(), lse=lse)
    assert status.item() == 0
    compare((out[10:90], lse[10:90]), reference(q[10:90], k[10:90], v[10:90], [30, 0, 50], [30, 0, 50], True))
    for x in (out, lse):
        assert (x[:10] == 3.0).all() and (x[90:] == 3.0).all()


@gpu
def test_rows_outside_the_sequences_stay_in_a_split():
    q, k, v = inputs([12], [6000], 8, 2, BF16)
    out, lse = torch.full_like(q, 3.0), torch.full((12, 8), 3.0, device="cuda")
    cq, ck = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([2, 7, 7, 10], [100, 3000, 3500, 5900]))
    ssa.ssa_prompt_attention(q, k, v, cq, out, None, workspace(), cu_k=ck, lse=lse)
    want = reference(q[2:10], k[100:5900], v[100:5900], [5, 0, 3], [2900, 500, 2400], True)
    compare((out[2:10], lse[2:10]), want)
    for x in (out, lse):
        assert (x[:2] == 3.0).all() and (x[10:] == 3.0).all()


@gpu
def test_keys_by_head_and_tokens_far_apart():
    """K and V laid out head by head; query and result rows more than 4 GiB from the first."""
    n, far = 50, 100_000_000
    q, k, v = inputs([n], [n], 8, 2, BF16)
    k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))
    store = [torch.empty((n * far,), dtype=BF16, device="cuda") for _ in range(2)]
    qf, out = (x.as_strided((n, 8, D), (far, D, 1)) for x in store)
    qf.copy_(q)
    lse = torch.empty((n, 8), device="cuda")
    ssa.ssa_prompt_attention(qf, k, v, offsets([n]), out, None, workspace(), lse=lse)
    compare((out, lse), reference(q, k, v, [n], [n], True))


@gpu
def test_no_keys_at_all():
    check([5, 200], [0, 0], 8, 2)


@gpu
def test_many_sequences():
    """More sequences than the kernel holds on chip."""
    lens = [(7 * i) % 23 for i in range(700)]
    check(lens, lens, 4, 2)


@gpu
@pytest.mark.parametrize("cu", [[0, 60, 40, 100], [0, 50, 100, 130], [-5, 50, 80, 100]])
def test_bad_tables_are_flagged_and_stay_inside(cu):
    q, k, v = inputs([100], [100], 8, 2, BF16)
    big = torch.full((300, 8, D), 3.0, dtype=BF16, device="cuda")
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    ssa.ssa_prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), big[100:200],
                             status, workspace())
    assert status.item() == ssa.ST_BAD_POS
    assert (big[:100] == 3.0).all() and (big[200:] == 3.0).all()


@gpu
def test_same_bits_and_graph_replay():
    lq, lk = [6, 1], [3000, 700]
    q, k, v = inputs(lq, lk, 16, 2, BF16)
    first, lse = call(q, k, v, lq, lk)
    out, ws = torch.zeros_like(q), workspace()
    cq, ck = offsets(lq), offsets(lk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssa.ssa_prompt_attention(q, k, v, cq, out, None, ws, cu_k=ck)
    side.synchronize()
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssa.ssa_prompt_attention(q, k, v, cq, out, None, ws, cu_k=ck)
    # other inputs and another split of the same tokens in the captured buffers
    q2, k2, v2 = inputs([2, 5], [1200, 2500], 16, 2, BF16, seed=9)
    for a, b in ((q, q2), (k, k2), (v, v2), (cq, offsets([2, 5])), (ck, offsets([1200, 2500]))):
        a.copy_(b)
    for _ in range(2):
        out.zero_()
        g.replay()
        o, s, tol, _ = reference(q2, k2, v2, [2, 5], [1200, 2500], True)
        assert ((out.double() - o).abs() <= tol).all()


def _call_cpu(**kw):
    z = dict(q=torch.zeros((6, 4, D), dtype=BF16), k=torch.zeros((6, 2, D), dtype=BF16),
             v=torch.zeros((6, 2, D), dtype=BF16), cu_q=torch.tensor([0, 6], dtype=torch.int32),
             out=torch.zeros((6, 4, D), dtype=BF16), status=None,
             ws=torch.zeros((ssa.ssa_prompt_workspace_size(),), dtype=torch.uint8))
    z.update(kw)
    ssa.ssa_prompt_attention(**z)


@gpu
@pytest.mark.parametrize("n,ctx", [(8, 16376), (8, 65528), (700, 3000)])
def test_keys_and_values_from_cold_memory(n, ctx):
    """Copies that come from memory and not from the cache land out of order: a V before the K that had
    its stage.  Every call finds the cache full of something else, and gives the bits of the first."""
    gen = torch.Generator(device="cuda").manual_seed(n + ctx)
    q, k, v = (torch.randn((t, h, D), generator=gen, device="cuda").to(BF16)
               for t, h in ((n, 16), (n + ctx, 2), (n + ctx, 2)))
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu_q, cu_k = offsets([n]), offsets([n + ctx])
    outs, ws = [torch.zeros_like(q) for _ in range(30)], workspace()
    for i, out in enumerate(outs):
        other.fill_(i)
        ssa.ssa_prompt_attention(q, k, v, cu_q, out, status, ws, cu_k=cu_k)
    assert status.item() == 0
    assert all(torch.equal(o, outs[0]) for o in outs)
    ref, _, tol, _ = reference(q, k, v, [n], [n + ctx], True)
    assert ((outs[0].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("kw,match", [
    (dict(q=torch.zeros((6, 4, D))), "bfloat16 or float16"),
    (dict(k=torch.zeros((6, 2, D), dtype=F16)), "k: "),
    (dict(v=torch.zeros((6, 2, D))), "v: "),
    (dict(v=torch.zeros((5, 2, D), dtype=BF16)), "alike"),
    (dict(v=torch.zeros((6, 1, D), dtype=BF16)), "alike"),
    (dict(out=torch.zeros((6, 2, D), dtype=BF16)), "alike"),
    (dict(out=torch.zeros((5, 4, D), dtype=BF16)), "alike"),
    (dict(out=torch.zeros((6, 4, D), dtype=F16)), "out: "),
    (dict(q=torch.zeros((6, 4, 2 * D), dtype=BF16)[..., ::2]), "contiguous"),
    (dict(cu_q=torch.tensor([0, 6])), "cu_q"),
    (dict(cu_q=torch.zeros((0,), dtype=torch.int32)), "cu_q"),
    (dict(cu_k=torch.tensor([0, 3, 6], dtype=torch.int32)), "cu_k"),
    (dict(lse=torch.zeros((6, 2))), "lse"),
    (dict(ws=torch.zeros((16,), dtype=torch.uint8)), "ws"),
    (dict(), "current CUDA device"),
])
def test_refusals(kw, match):
    with pytest.raises(ValueError, match=match):
        _call_cpu(**kw)


def test_c_refusals():
    L, p = ssa.lib(), 0x10000
    t = {}

    def go(dtype=0, D=128, n=1, nq=6, nk=6, Hq=4, Hk=2, Hv=None, Ho=None, scale=0.1, cu=p, ws=p, data=p, st=512):
        q, k, v, o = (ssa.SsaPromptTensor(data, h, (ctypes.c_int64 * 2)(st, 128))
                      for h in (Hq, Hk, Hk if Hv is None else Hv, Hq if Ho is None else Ho))
        t.update(q=q, k=k)
        b = ctypes.byref
        return L.ssa_prompt_attention(dtype, D, n, nq, nk, b(q), b(k), b(v), b(o), cu, p, 1, scale, None, None,
                                      ws, None)
    assert go(dtype=2) == -3 and go(dtype=-1) == -3
    assert go(D=64) == -3
    assert go(n=-1) == -1 and go(nq=-1) == -1 and go(nk=-1) == -1
    assert go(cu=None) == -1 and go(ws=None) == -1 and go(ws=p + 4) == -1
    assert go(scale=-0.5) == -1 and go(scale=math.nan) == -1 and go(scale=math.inf) == -1
    assert go(Hv=1) == -1 and go(Ho=2) == -1
    assert go(Hq=5) == -3 and go(Hq=258, Hk=2) == -3
    assert go(data=None) == -1 and go(data=p + 2) == -1
    assert go(st=516) == -1 and go(st=0) == -1 and go(st=-512) == -1
    assert go() == -1                               # out over its inputs
    assert go(nq=0) == 0                            # nothing to do, nothing launched
