"""Rotary positions: the frequency table and the refusals on the CPU, the kernel against 64 bits."""
import ctypes
import math

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def ssa():
    from sparse_attention_decode_indexer_gb300 import build
    build.build()
    import sparse_attention_decode_indexer_gb300 as m
    return m


def _theta(rd, base, kind="plain", factor=1.0, original_len=0, low=1.0, high=32.0):
    """The definitions of include/ssa.h, pair by pair."""
    if kind == "ntk" and rd > 2:
        base = base * factor ** (rd / (rd - 2))
    th = [base ** (-2 * i / rd) for i in range(rd // 2)]
    if kind == "linear":
        th = [x / factor for x in th]
    if kind == "bands":
        for i, x in enumerate(th):
            n = original_len * x / (2 * math.pi)
            mix = 0.0 if n <= low else 1.0 if n >= high else (n - low) / (high - low)
            th[i] = mix * x + (1 - mix) * x / factor
    if kind == "yarn":
        pair = lambda r: rd * math.log(original_len / (2 * math.pi * r)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rd - 1)
        for i, x in enumerate(th):
            ramp = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            th[i] = x / factor * ramp + x * (1 - ramp)
    return th, 0.1 * math.log(factor) + 1 if kind == "yarn" else 1.0


SCALINGS = [dict(kind="plain"), dict(kind="linear", factor=4), dict(kind="ntk", factor=8),
            dict(kind="bands", factor=8, original_len=8192, low=1, high=4),
            dict(kind="yarn", factor=16, original_len=4096, low=1, high=32),
            dict(kind="yarn", factor=2, original_len=64, low=1, high=32)]


@pytest.mark.parametrize("rd", [2, 58, 64, 128])
@pytest.mark.parametrize("sc", SCALINGS, ids=lambda s: s["kind"] + str(s.get("factor", "")))
def test_frequencies(ssa, rd, sc):
    """The table to within a few roundings of 64-bit arithmetic (pow, exp and log within an ulp or two of
    2^-53, amplified by log(base) * 2 and by the blend): 2^-45 relative, or one step of 2^-64 turns."""
    th, m = _theta(rd, 500000.0, **sc)
    plan = ssa.RopePlan(128, rd, 500000.0, scaling=ssa.RopeScaling(**sc), device="cpu")
    got = plan.freq.numpy().view(np.uint64)
    want = np.array(th) / (2 * math.pi)
    assert np.all(np.abs(got.astype(np.float64) * 2.0 ** -64 - want) <= want * 2.0 ** -45 + 2.0 ** -64)
    assert abs(plan.factor - m) < 1e-12


def test_given_theta(ssa):
    plan = ssa.RopePlan(4, theta=[2.0, -7.0], device="cpu")
    got = plan.freq.numpy().view(np.uint64).astype(np.float64) * 2.0 ** -64
    np.testing.assert_allclose(got, [2 / (2 * math.pi), (-7 / (2 * math.pi)) % 1.0], atol=1e-15)


def test_refusals(ssa):
    lib, INVALID, UNSUPPORTED = ssa.lib(), -1, -3
    buf = (ctypes.c_uint64 * 64)()
    f = lambda *a: lib.ssa_rope_frequencies(*a, buf, None)  # noqa: E731
    assert f(128, 10000.0, 0, 1.0, 0.0, 1.0, 32.0) == 0
    for bad in ((3, 1e4, 0, 1.0, 0.0, 1.0, 32.0), (0, 1e4, 0, 1.0, 0.0, 1.0, 32.0),
                (1026, 1e4, 0, 1.0, 0.0, 1.0, 32.0), (64, 1.0, 0, 1.0, 0.0, 1.0, 32.0),
                (64, float("inf"), 0, 1.0, 0.0, 1.0, 32.0), (64, 1e4, 1, 0.5, 0.0, 1.0, 32.0),
                (64, 1e4, 3, 2.0, 0.0, 1.0, 4.0), (64, 1e4, 4, 2.0, 4096.0, 4.0, 4.0),
                (64, 1e4, 1, float("nan"), 0.0, 1.0, 4.0)):
        assert f(*bad) == INVALID, bad
    assert f(64, 1e4, 5, 2.0, 4096.0, 1.0, 4.0) == UNSUPPORTED
    for bad in (dict(rotary_dim=3), dict(rotary_dim=130), dict(theta=[1.0]),
                dict(theta=[float("nan")] * 64), dict(scaling=ssa.RopeScaling("other"))):
        with pytest.raises(ValueError):
            ssa.RopePlan(128, **bad)
    # the C call, before any launch
    p = 0x10000
    t = lambda i=p, o=p, h=2, ist=(0, 256, 128), ost=(0, 256, 128): ssa.SsaRopeTensor(  # noqa: E731
        i, o, h, (ctypes.c_int64 * 3)(*ist), (ctypes.c_int64 * 3)(*ost))
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    call = lambda dtype=0, D=128, rd=128, freq=p, L=1, T=4, pos=p, q=t(), k=None: lib.ssa_rope(  # noqa: E731
        dtype, D, rd, 0, 0, freq, 1.0, L, T, pos, 0, 0, ref(q), k, None)
    assert call(dtype=3) == UNSUPPORTED and call(D=4096, rd=2048) == UNSUPPORTED
    for bad in (dict(rd=130), dict(rd=5), dict(rd=0), dict(freq=None), dict(pos=None), dict(L=0), dict(T=-1),
                dict(q=None), dict(q=t(h=0)), dict(q=t(i=None)), dict(q=t(o=None)), dict(q=t(i=p + 1)),
                dict(q=t(ost=(0, 512, 128))), dict(q=t(o=2 * p, ost=(0, 0, 128)))):
        assert call(**bad) == INVALID, bad
    assert call(T=0) == 0                       # nothing to do, nothing launched
    # the binding
    plan = ssa.RopePlan(128, device="cpu")
    x, pos = torch.zeros((2, 3, 4, 128), dtype=torch.bfloat16), torch.zeros((3,), dtype=torch.int64)
    for a, kw in (((pos,), {}), ((pos, x.double()), {}), ((pos.float(), x), {}), ((pos[:2], x), {}),
                  ((pos, x[..., :64]), {}), ((pos, x.transpose(-1, -2)), {}), ((pos, x, x.float()), {}),
                  ((pos, x, x[:1]), {}), ((pos, x), dict(q_out=x[:1])), ((pos, x, x[0]), {})):
        with pytest.raises(ValueError):
            ssa.ssa_rope(plan, *a, **kw)


def test_q_and_k_on_the_same_elements_are_refused(ssa):
    P = 0x10000
    t = lambda i, o: ctypes.byref(ssa.SsaRopeTensor(  # noqa: E731
        i * P, o * P, 2, (ctypes.c_int64 * 3)(0, 256, 128), (ctypes.c_int64 * 3)(0, 256, 128)))
    for q, k in (((1, 1), (1, 1)), ((1, 2), (3, 2)), ((1, 2), (2, 3)), ((3, 2), (4, 3))):
        assert ssa.lib().ssa_rope(0, 128, 128, 0, 0, P, 1.0, 1, 4, P, 0, 0, t(*q), t(*k), None) == -1


def _exact(x, pos, theta, m, rd, inter, inverse):
    ang = pos.double()[:, None] * torch.tensor(theta, dtype=torch.float64)
    c, s = m * ang.cos()[:, None], m * ang.sin()[:, None]
    s = -s if inverse else s
    y = x.double().clone()
    i = torch.arange(rd // 2)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def _close(got, x, pos, theta, m, rd, inter, inverse):
    """Per pair of length r = m |(a, b)|: cos and sin in fp32 (the turn's rest 2^-24, sincospif 2 ulp, the
    factor) 2^-21 in all, three fp32 roundings 2^-22, the output's rounding; the 64-bit reference itself
    has angles off by 2^-53 pos theta."""
    want = _exact(x.cpu(), pos.cpu(), theta, m, rd, inter, inverse)
    g = got.double().cpu()
    half = torch.finfo(x.dtype).eps / 2
    i = torch.arange(rd // 2)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
    r = m * torch.hypot(x.double().cpu()[..., ia], x.double().cpu()[..., ib])
    e = 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -52 * float(pos.abs().max().clamp(min=1)) * max(map(abs, theta))
    tiny = torch.finfo(x.dtype).smallest_normal * half
    for idx in (ia, ib):
        d = (g[..., idx] - want[..., idx]).abs()
        assert bool((d <= half * want[..., idx].abs() + r * e + tiny).all()), float((d - half * want[..., idx].abs()).max())
    assert torch.equal(g[..., rd:], x.double().cpu()[..., rd:])       # untouched, not rounded


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D,rd,inter", [(128, 128, False), (128, 64, True), (64, 32, False), (80, 80, True),
                                        (96, 58, False), (128, 2, True), (256, 200, False), (576, 64, True),
                                        (66, 66, False), (1200, 1024, False)])
@pytest.mark.parametrize("L,T,Hq,Hkv", [(1, 1, 1, 1), (3, 5, 7, 2), (2, 513, 4, 1)])
def test_against_64_bits(ssa, dtype, D, rd, inter, L, T, Hq, Hkv):
    g = torch.Generator().manual_seed(D * 1000 + T)
    q = torch.randn((L, T, Hq, D), generator=g).to(dtype).cuda()
    k = torch.randn((L, T, Hkv, D), generator=g).to(dtype).cuda()
    pos = torch.randint(0, 1 << 21, (T,), generator=g).cuda()
    sc = SCALINGS[(D + T) % len(SCALINGS)]
    th, m = _theta(rd, 10000.0, **sc)
    plan = ssa.RopePlan(D, rd, interleaved=inter, scaling=ssa.RopeScaling(**sc))
    qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    inverse = T == 5
    q0, k0 = q.clone(), k.clone()
    ssa.ssa_rope(plan, pos, q, k, q_out=qo, k_out=ko, inverse=inverse)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    for x, y in ((q, qo), (k, ko)):
        _close(y, x, pos, th, m, rd, inter, inverse)
    # in place, one tensor alone, and int32 positions with an offset: the same bits
    ssa.ssa_rope(plan, (pos - 3).int(), q=q, offset=3, inverse=inverse)
    ssa.ssa_rope(plan, pos, k=k, inverse=inverse)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 1, -1, -4097, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31), 1 << 40])
def test_far_and_negative_positions(ssa, at):
    """The angle keeps its accuracy (frequencies whose product with the position is exact in 64 bits)."""
    th = [2 * math.pi * f for f in (0.25, 2.0 ** -10, 3 * 2.0 ** -12, 2.0 ** -20)]
    plan = ssa.RopePlan(8, theta=th)
    x = torch.randn((1, 1, 1, 8), generator=torch.Generator().manual_seed(1)).cuda()
    pos = torch.tensor([at], device="cuda")
    y = torch.empty_like(x)
    ssa.ssa_rope(plan, pos, q=x, q_out=y)
    turns = [(at * f) % 1.0 for f in (0.25, 2.0 ** -10, 3 * 2.0 ** -12, 2.0 ** -20)]
    _close(y, x, torch.tensor([1]), [2 * math.pi * t for t in turns], 1.0, 8, False, False)


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1])
def test_strided_views(ssa, offset):
    """q and k as slices of a fused projection (aligned and not), layers and heads in other orders."""
    L, T, Hq, Hkv, D = 2, 9, 3, 2, 64
    g = torch.Generator().manual_seed(3)
    buf = torch.randn((T, L, (Hq + 2 * Hkv) * D + 3), generator=g).bfloat16().cuda()
    before = buf.clone()
    q = buf[..., offset:offset + Hq * D].unflatten(-1, (Hq, D)).transpose(0, 1)
    k = buf[..., offset + Hq * D:offset + (Hq + Hkv) * D].unflatten(-1, (Hkv, D)).transpose(0, 1)
    pos = torch.arange(T, device="cuda") * 1000
    plan = ssa.RopePlan(D, 32, interleaved=True)
    th, m = _theta(32, 10000.0)
    qo = torch.empty((L, Hq, T, D), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    ko = torch.empty((L, T, Hkv, D), dtype=torch.bfloat16, device="cuda")
    ssa.ssa_rope(plan, pos, q, k, q_out=qo, k_out=ko)
    assert torch.equal(buf, before)
    _close(qo, q, pos, th, m, 32, True, False)
    _close(ko, k, pos, th, m, 32, True, False)
    qc, kc = qo.clone(), ko.clone()
    ssa.ssa_rope(plan, pos, q, k)               # in place in the projection: the rest stays
    assert torch.equal(q, qc) and torch.equal(k, kc)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[..., offset:offset + (Hq + Hkv) * D] = False
    assert torch.equal(buf[rest], before[rest])


@pytest.mark.gpu
def test_inverse_is_the_gradient(ssa):
    """d(sum(w * rope(x)))/dx by central differences of the 64-bit form, and the way back."""
    D, T = 16, 4
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn((T, 2, D), generator=g), torch.randn((T, 2, D), generator=g)
    pos = torch.tensor([0, 7, 100, 5000])
    th, m = _theta(D, 10000.0)
    grad = torch.empty((T, 2, D)).cuda()
    plan = ssa.RopePlan(D)
    ssa.ssa_rope(plan, pos.cuda(), q=w.cuda(), q_out=grad, inverse=True)
    f = lambda y: (_exact(y, pos, th, m, D, False, False) * w.double()).sum()  # noqa: E731
    h = 2.0 ** -10
    for idx in ((0, 0, 0), (1, 1, 5), (2, 0, 9), (3, 1, 15)):
        e = torch.zeros_like(x, dtype=torch.float64)
        e[idx] = h
        num = (f(x.double() + e) - f(x.double() - e)) / (2 * h)      # linear: exact but for rounding
        assert abs(float(grad[idx]) - float(num)) < 2.0 ** -19 * float(w.abs().max()) * 2
    y = torch.empty_like(grad)
    ssa.ssa_rope(plan, pos.cuda(), q=x.cuda(), q_out=y)
    ssa.ssa_rope(plan, pos.cuda(), q=y, inverse=True)
    assert float((y.cpu() - x).abs().max()) < 2.0 ** -19 * float(x.abs().max()) * 2


@pytest.mark.gpu
def test_streams_graphs_and_no_tokens(ssa):
    plan = ssa.RopePlan(128)
    x = torch.randn((2, 6, 4, 128), device="cuda").bfloat16()
    pos = torch.arange(6, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    ssa.ssa_rope(plan, pos, q=x, q_out=y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ssa.ssa_rope(plan, pos, q=x, q_out=z, stream=s)
    s.synchronize()
    assert torch.equal(y, z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssa.ssa_rope(plan, pos, q=x, q_out=z)
    pos.add_(100)
    g.replay()
    ssa.ssa_rope(plan, pos, q=x, q_out=y)
    assert torch.equal(y, z)
    n = ssa.launch_count()
    ssa.ssa_rope(plan, pos[:0], q=x[:, :0])
    assert ssa.launch_count() == n


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["plain", "graphs", "preload", "overlap", "per_layer", "fetch"])
def test_runner_with_rope_equals_rotating_by_hand(ssa, form):
    """A runner with a plan gives the selection and outputs of one that is handed rotated tensors."""
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    P, Hq, Hkv, L, B, nmax, k = 32, 8, 2, 2, 2, 9, 2
    lens = torch.tensor([9 * P - 3, 5 * P + 1])
    lay = ssa.Layout(P, Hq, Hkv, 128, False, L, B * nmax, B * nmax, B, nmax, k, kv_format="int8_page_head")
    bt = torch.arange(B * nmax).view(B, nmax)
    g = torch.Generator().manual_seed(5)
    plan = ssa.RopePlan(128, 64, scaling=ssa.RopeScaling("yarn", 4.0, 64, 1.0, 32.0))
    kw = dict(host_tier=True, identity=False, block_table=bt, seq_lens=lens,
              graphs=form == "graphs", preload_width=4 if form == "preload" else 0,
              overlap_groups=2 if form == "overlap" else 0, fetch_in_attention=form == "fetch")
    a, b = DecodeRunner(lay, rope=plan, **kw), DecodeRunner(lay, **kw)
    pos = torch.cat([torch.arange(int(n)) + i * nmax * P for i, n in enumerate(lens)]).cuda()
    at = torch.cat([torch.arange(int(n)) for n in lens]).cuda()
    kk = torch.randn((L, len(pos), Hkv, 128), generator=g).bfloat16().cuda()
    vv = torch.randn((L, len(pos), Hkv, 128), generator=g).bfloat16().cuda()
    before = kk.clone()
    a.store(0, L, kk, vv, pos, positions=at)
    assert torch.equal(kk, before)
    with pytest.raises(ValueError):
        a.store(0, L, kk, vv, pos)
    kr = torch.empty_like(kk)
    ssa.ssa_rope(plan, at, k=kk, k_out=kr)
    b.store(0, L, kr, vv, pos)
    q, qr = (torch.empty((L, B, Hq, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for _ in range(4):
        q.copy_(torch.randn((L, B, Hq, 128), generator=g).bfloat16())
        ssa.ssa_rope(plan, lens.cuda() - 1, q=q, q_out=qr)
        a.step(q, per_layer=form == "per_layer")
        b.step(qr, per_layer=form == "per_layer")
        torch.cuda.synchronize()
        assert torch.equal(a.sel, b.sel) and torch.equal(a.out, b.out)
    assert int(a.status.item()) == 0
