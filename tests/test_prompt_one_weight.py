"""Prompt attention where one key has nearly all of a row's weight.

The weights w_j (1 + d_j), |d_j| at most u (half a step of the type), are divided by their own sum, so the
result is off by sum_j w_j d_j (v_j - out) / (1 + sum_j w_j d_j): at most u / (1 - u) sum_j w_j |v_j - out|,
where tests/test_prompt.py allows u sum_j w_j |v_j|.  The rest of its tolerance is as there: scores and
exponentials (2 e_s + 2^-18) sum_j w_j |v_j|, and the rounding of the result."""
import math

import pytest
import torch

from tests.test_prompt import BF16, F16, D, call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,ctx", [(40, 260), (3, 12000)])
@pytest.mark.parametrize("at", [0, 70, 200])
def test_one_key(dtype, n, ctx, at):
    """The key lies up to 7 octaves above the others, in steps that no 16-bit weight hits."""
    H, G, Tk = 4, 2, n + ctx
    g = torch.Generator(device="cuda").manual_seed(at)
    q, k, v = (0.2 * torch.randn((T, h, D), generator=g, device="cuda") for T, h in ((n, G * H), (Tk, H), (Tk, H)))
    v = 5 * v
    u = torch.finfo(dtype).eps / 2
    q[..., 0] = 8.0
    octaves = math.log(2) * math.sqrt(D) / 8
    for step in range(12):
        kk = k.clone()
        kk[..., 0] = 0
        kk[at, :, 0] = (math.log2(Tk) + 5 + 0.27 * step) * octaves
        if at:                  # a key before it that the reference starts from
            kk[0, :, 0] = (math.log2(Tk) - 1.6) * octaves
        qq, kk, vv = (x.to(dtype) for x in (q, kk, v))
        out, _ = call(qq, kk, vv, [n], [Tk], False)
        s = torch.einsum("ihd,jhd->hij", qq.double(), kk.double().repeat_interleave(G, 1)) / math.sqrt(D)
        mag = torch.einsum("ihd,jhd->hij", qq.double().abs(), kk.double().abs().repeat_interleave(G, 1)) / math.sqrt(D)
        w, x = s.softmax(-1), vv.double().repeat_interleave(G, 1)
        o = torch.einsum("hij,jhd->ihd", w, x)
        e_s = 130 * 2.0 ** -23 * mag.amax(-1).T[..., None]
        spread = torch.stack([(w[:, i, :, None] * (x.transpose(0, 1) - o[i][:, None]).abs()).sum(1) for i in range(n)])
        tol = u / (1 - u) * spread + (2 * e_s + 2.0 ** -18) * torch.einsum("hij,jhd->ihd", w, x.abs())
        tol = tol + u * o.abs().clamp(min=torch.finfo(dtype).tiny)
        if dtype is F16:        # the steps of small weights, 2^-32 of the greatest
            tol = tol + 2.0 ** -32 * x.abs().sum(0)
        err = (out.double() - o).abs() - tol
        assert (err <= 0).all(), f"{err.max().item():.3e} above the tolerance"
