"""ssa_norm_rope against the norm and the rotation in 64 bits.

Tolerance, from the kernel's roundings: the sum of D squares in fp32 is off by at most D * 2^-24
of itself, its root by half of that, the reciprocal root and the products by a few 2^-24 more; a
cosine or sine by 2^-22 (its angle is a 25-bit fraction of a turn's eighth, the functions are good
to about 2^-23).  A rotated element a c - b s is then off by (|a| + |b|) times their sum, and the
result's own rounding adds u * |out|, u half a step of the type -- of the least normal number
where |out| is below it: the steps get no smaller there (fp16: 2^-24, so a value below 2^-14 is off
by up to 2^-25 = 2^-11 * 2^-14, whatever its size).
"""
import ctypes
import math

import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
gpu = pytest.mark.gpu


def reference(x, w, eps, theta, pos, rd, inter, factor=1.0):
    """x [L][T][H][D], w [L][D] or None, theta [rd / 2] doubles, pos [T]: the result and its
    tolerance."""
    D = x.shape[-1]
    y = x.double()
    y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.double()[:, None, None]
    ang = (pos.double()[:, None] * theta)[:, None]
    c, s = ang.cos() * factor, ang.sin() * factor
    i = torch.arange(rd // 2, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + rd // 2)
    out, size = y.clone(), y.abs()
    a, b = y[..., lo], y[..., hi]
    out[..., lo], out[..., hi] = a * c - b * s, b * c + a * s
    size[..., lo] = size[..., hi] = (a.abs() + b.abs()) * factor
    u, least = torch.finfo(x.dtype).eps / 2, torch.finfo(x.dtype).tiny
    return out, size * ((D / 2 + 16) * 2.0 ** -24 + 2.0 ** -22) + u * out.abs().clamp(min=least)


def check(got, want):
    (out, tol), got = want, got.double()
    assert got.shape == out.shape
    bad = (got - out).abs() - tol
    assert (bad <= 0).all(), f"{bad.max().item():.3e} above the tolerance"


def run(L, T, Hq, Hkv, D, rd, inter, dtype, weights="layers", in_place=False, packed=False, pos64=True,
        eps=1e-6, seed=0, offset=0, shift=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if packed:
        x = scale * torch.randn((L, T, (Hq + 2 * Hkv) * D + shift), generator=g, device="cuda")
        x = x.to(dtype)[..., shift:].unflatten(-1, (Hq + 2 * Hkv, D))
        q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    else:
        q = (scale * torch.randn((L, T, Hq, D), generator=g, device="cuda")).to(dtype)
        k = (scale * torch.randn((L, T, Hkv, D), generator=g, device="cuda")).to(dtype)
    shape = {"layers": (L, D), "shared": (D,), "none": None}[weights]
    w = [None if shape is None else 1 + 0.3 * torch.randn(shape, generator=g, device="cuda") for _ in range(2)]
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
    plan = ssa.RopePlan(D, rotary_dim=rd, base=10000.0, interleaved=inter)
    theta = 10000.0 ** (-2.0 * torch.arange(rd // 2, dtype=torch.float64, device="cuda") / rd)
    norm = ssa.HeadNorm(*w, eps=eps)
    wl = [None if x is None else x.expand(L, D) for x in w]
    want = [reference(x, y, eps, theta, pos + offset, rd, inter) for x, y in zip((q, k), wl)]
    p = pos if pos64 else pos.int()
    if in_place:
        ssa.ssa_norm_rope(plan, norm, p, q, k, offset=offset)
        out = (q, k)
    else:
        out = torch.empty((L, T, Hq, D), dtype=dtype, device="cuda"), torch.empty((L, T, Hkv, D), dtype=dtype, device="cuda")
        keep = q.clone()
        ssa.ssa_norm_rope(plan, norm, p, q, k, q_out=out[0], k_out=out[1], offset=offset)
        assert torch.equal(q, keep)
    for a, b in zip(out, want):
        check(a, b)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rd", [(128, 128), (128, 64), (64, 64), (80, 80), (96, 64), (192, 192), (256, 256),
                                  (256, 6), (70, 34), (33, 2), (128, 36), (512, 512), (1030, 1024)])
def test_sizes(D, rd, inter, dtype):
    run(2, 9, 6, 2, D, rd, inter, dtype, seed=D + rd)


@gpu
@pytest.mark.parametrize("L,T,Hq,Hkv", [(1, 1, 1, 1), (12, 1, 16, 2), (3, 1, 5, 1), (1, 5000, 4, 1), (2, 700, 32, 8),
                                        (5, 33, 7, 7), (40, 2, 1, 1), (1, 6000, 3, 1)])
@pytest.mark.parametrize("weights", ["layers", "shared", "none"])
def test_rows(L, T, Hq, Hkv, weights):
    run(L, T, Hq, Hkv, 128, 128, False, BF16, weights=weights, seed=T)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_views_and_in_place(dtype, shift, in_place, inter):
    """Slices of a fused projection, 16-byte aligned or one element off."""
    run(2, 65, 8, 2, 128, 64, inter, dtype, packed=True, shift=shift, in_place=in_place, pos64=False, offset=-1)


@gpu
@pytest.mark.parametrize("shift", [0, 1])
def test_tokens_beyond_4_gib(shift):
    T, far = 5, 600_000_000
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((1, T, 4, 128), generator=g, device="cuda").to(BF16)
    x = torch.empty((T * far + 8,), dtype=BF16, device="cuda")[shift:].as_strided((T, 4, 128), (far, 128, 1))
    x.copy_(q[0])
    plan, norm, pos = ssa.RopePlan(128), ssa.HeadNorm(eps=1e-6), torch.arange(T, device="cuda")
    theta = 10000.0 ** (-2.0 * torch.arange(64, dtype=torch.float64, device="cuda") / 128)
    ssa.ssa_norm_rope(plan, norm, pos, x)
    check(x[None], reference(q, None, 1e-6, theta, pos, 128, False))


@gpu
@pytest.mark.parametrize("scale,eps", [(1e-4, 1e-5), (300.0, 1e-6), (1.0, 0.0), (1e-3, 1e3)])
def test_magnitudes(scale, eps):
    run(1, 40, 4, 2, 128, 128, False, BF16, scale=scale, eps=eps)


@gpu
def test_rows_of_zeros_and_of_nan():
    q = torch.randn((3, 4, 128), device="cuda").to(BF16)
    q[1, 2] = 0
    q[2, 0, 5] = math.nan
    plan, norm = ssa.RopePlan(128), ssa.HeadNorm()
    pos = torch.arange(3, device="cuda")
    out = torch.empty_like(q)
    ssa.ssa_norm_rope(plan, norm, pos, q, q_out=out)
    assert (out[1, 2] == 0).all() and out[2, 0].isnan().all()
    nan = torch.zeros((3, 4), dtype=torch.bool, device="cuda")
    nan[2, 0] = True
    assert out[~nan].isfinite().all()


@gpu
def test_alone_offset_weights_and_a_layer_of_many():
    """k alone; weights about zero; one layer of a norm that has a vector for each."""
    g = torch.Generator(device="cuda").manual_seed(5)
    k = torch.randn((50, 3, 128), generator=g, device="cuda").to(BF16)
    w = [0.2 * torch.randn((4, 128), generator=g, device="cuda").to(BF16) for _ in range(2)]
    plan, norm = ssa.RopePlan(128), ssa.HeadNorm(*w, eps=1e-5, offset=1.0)
    pos = torch.arange(50, device="cuda")
    theta = 10000.0 ** (-2.0 * torch.arange(64, dtype=torch.float64, device="cuda") / 128)
    want = reference(k[None], 1 + w[1][2:3].double(), 1e-5, theta, pos, 128, False)
    out = torch.empty_like(k)
    ssa.ssa_norm_rope(plan, norm, pos, k=k, k_out=out, layer0=2)
    # (the weights are kept in fp32: 1 + w is one rounding more)
    check(out[None], (want[0], want[1] + 2.0 ** -24 * want[0].abs()))


@gpu
def test_graph_and_stream():
    q = torch.randn((2, 8, 4, 128), device="cuda").to(F16)
    plan, norm = ssa.RopePlan(128), ssa.HeadNorm(torch.rand(128) + 0.5, torch.rand(128) + 0.5)
    pos = torch.arange(8, device="cuda", dtype=torch.int32)
    want, out = torch.empty_like(q), torch.empty_like(q)
    ssa.ssa_norm_rope(plan, norm, pos, q, q_out=want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ssa.ssa_norm_rope(plan, norm, pos, q, q_out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssa.ssa_norm_rope(plan, norm, pos, q, q_out=out)
    out.zero_()
    g.replay()
    assert torch.equal(out, want)


def _fake_plan(D=128, rd=128):
    plan = ssa.RopePlan.__new__(ssa.RopePlan)
    plan.head_dim, plan.rotary_dim, plan.interleaved, plan.factor = D, rd, False, 1.0
    plan.freq = torch.zeros((rd // 2,), dtype=torch.int64)
    plan._freq, plan._dev = plan.freq.data_ptr(), -1
    return plan


def test_refusals():
    plan, pos = _fake_plan(), torch.arange(4)
    q = torch.zeros((2, 4, 8, 128), dtype=BF16)
    norm = ssa.HeadNorm(torch.ones(2, 128), torch.ones(2, 128), device="cpu")
    with pytest.raises(ValueError, match="q or k"):
        ssa.ssa_norm_rope(plan, norm, pos)
    with pytest.raises(ValueError, match="the same"):
        ssa.ssa_norm_rope(plan, norm, pos, q.double())
    with pytest.raises(ValueError, match="positions"):
        ssa.ssa_norm_rope(plan, norm, pos.float(), q)
    with pytest.raises(ValueError, match="layers 1 to 3"):
        ssa.ssa_norm_rope(plan, norm, pos, q, layer0=1)
    with pytest.raises(ValueError, match="norm: weights of 64"):
        ssa.ssa_norm_rope(plan, ssa.HeadNorm(torch.ones(64), device="cpu"), pos, q)
    with pytest.raises(ValueError, match="current CUDA device"):
        ssa.ssa_norm_rope(plan, norm, pos, q)
    with pytest.raises(ValueError, match="the same for both"):
        ssa.HeadNorm(torch.ones(64), torch.ones(2, 64), device="cpu")
    with pytest.raises(ValueError, match=r"\[D\] or"):
        ssa.HeadNorm(torch.ones(1, 2, 64), device="cpu")
    with pytest.raises(ValueError, match="eps"):
        ssa.HeadNorm(eps=-1.0, device="cpu")
    with pytest.raises(ValueError, match="offset"):
        ssa.HeadNorm(torch.ones(64), offset=1.0, device="cpu")


def test_c_refusals():
    L, p = ssa.lib(), 0x10000
    x = ssa.SsaRopeTensor(p, p, 4, (ctypes.c_int64 * 3)(4096, 512, 128), (ctypes.c_int64 * 3)(4096, 512, 128))

    def go(dtype=0, D=128, rd=128, L_=1, T=4, freq=p, q=x, k=None, wq=p, wk=p, step=128, eps=1e-6):
        return L.ssa_norm_rope(dtype, D, rd, 0, freq, 1.0, L_, T, p, 1, 0, q and ctypes.byref(q),
                               k and ctypes.byref(k), wq, wk, step, eps, None)
    assert go(dtype=3) == -3 and go(rd=127) == -1 and go(rd=130) == -1 and go(D=20000) == -3
    assert go(L_=0) == -1 and go(T=-1) == -1 and go(q=None) == -1 and go(freq=None) == -1
    assert go(eps=-1.0) == -1 and go(eps=math.nan) == -1 and go(eps=math.inf) == -1
    assert go(step=-1) == -1 and go(wq=p + 2) == -1
    assert go(k=x) == -1                              # both on the same elements
    assert go(T=0) == 0
