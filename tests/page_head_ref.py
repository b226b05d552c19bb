"""A plain implementation of the page_head formats for the tests: the write path step by step in
numpy (IEEE fp32, one operation at a time, as the definition states it), the attention in 64 bits.

State arrays of one layer, by logical page (the tests compare them with pool or mirror blocks):
k [Lp][H][P][D], v [Lp][H][P][D] code bytes, ks, vs [Lp][H] fp32, sums [Lp][H*D], cnt [Lp]."""
import math

import numpy as np
import torch

QMAX = {"int8_page_head": np.float32(127), "e4m3_page_head": np.float32(448)}


def quant(fmt, x):
    """fp32 values -> code bytes."""
    x = np.asarray(x, np.float32)
    if fmt == "int8_page_head":
        r = np.clip(np.rint(x), -127, 127)
        return np.where(np.isnan(x), 0, r).astype(np.int8).view(np.uint8)
    t = torch.from_numpy(np.ascontiguousarray(np.clip(x, np.float32(-448), np.float32(448))))
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def values(fmt, codes):
    c = np.ascontiguousarray(codes)
    if fmt == "int8_page_head":
        return c.view(np.int8).astype(np.float32)
    return torch.from_numpy(c).view(torch.float8_e4m3fn).float().numpy()


class RefPages:
    def __init__(self, fmt, Lp, H, P, D=128):
        self.fmt, self.P = fmt, P
        self.k = np.zeros((Lp, H, P, D), np.uint8)
        self.v = np.zeros((Lp, H, P, D), np.uint8)
        self.ks = np.zeros((Lp, H), np.float32)
        self.vs = np.zeros((Lp, H), np.float32)
        self.sums = np.zeros((Lp, H * D), np.float32)
        self.cnt = np.zeros((Lp,), np.int32)
        self.slab = np.zeros((Lp, H * D), np.int8)
        self.slab_scale = np.zeros((Lp,), np.float32)

    def store(self, k, v, pos):
        """k, v: fp32 holding bf16 values [T][H][D]; pos strictly increasing."""
        pages = pos // self.P
        for pg in np.unique(pages):
            at = np.flatnonzero(pages == pg)
            j = pos[at] % self.P
            for x, codes, scale in ((k[at], self.k, self.ks), (v[at], self.v, self.vs)):
                a = np.where(np.isfinite(x), np.abs(x), np.float32(0)).max(axis=(0, 2))
                need = (a / QMAX[self.fmt]).astype(np.float32)
                for h in range(x.shape[1]):
                    old, s = scale[pg, h], need[h]
                    if self.cnt[pg] > 0:
                        s = max(old, s)
                        if s > old:
                            ratio = np.float32(old / s)
                            codes[pg, h] = quant(self.fmt, values(self.fmt, codes[pg, h]) * ratio)
                    scale[pg, h] = s
                    codes[pg, h, j] = quant(self.fmt, x[:, h] / s) if s > 0 else 0
            for r in at:                       # token order
                self.sums[pg] = self.sums[pg] + k[r].reshape(-1)
            self.cnt[pg] += len(at)
            mean = self.sums[pg] / np.float32(self.cnt[pg])
            amax = np.abs(mean).max()
            s = np.float32(amax / np.float32(127))
            self.slab_scale[pg] = s
            self.slab[pg] = np.clip(np.rint(mean / s), -127, 127).astype(np.int8) if amax > 0 else 0


def attend(fmt, kcodes, vcodes, ks, vs, q, sm_scale, live):
    """One request and KV head in 64 bits: codes [N][P][D], scales [N], q [G][D], live [N][P].
    Returns the output [G][D] and a bound on the kernel's error.

    The bound, by the roundings the kernel makes (u = 2^-24 fp32, half steps):
      * q enters as f16 (int8 codes: exact to 2^-28 of |q|max) or as two e4m3 terms (e4m3 codes: off
        by at most 2^-17 of |q|max: the low term keeps 4 of the bits the high one drops);
      * a score is a sum of 128 products in fp32, and is scaled three times: 131 u of sum |q k|;
        its exponent x = score * log2(e) moves by that, and the exponential by another 2^-21;
      * the weight p * v_scale is rounded to f16 (2^-11);
      * the sums over t tokens in fp32: (t + 16) u each, and the rescales of the pieces;
    a weighted mean of values with weights off by a factor 1 + e moves by at most 2 e sum w|v|, and
    the result is rounded to bf16 (2^-8)."""
    K = values(fmt, kcodes).astype(np.float64) * ks[:, None, None].astype(np.float64)
    V = values(fmt, vcodes).astype(np.float64) * vs[:, None, None].astype(np.float64)
    K, V = K[live], V[live]
    G, D = q.shape
    if not len(K):
        return np.zeros((G, D)), np.zeros((G, D))
    q = q.astype(np.float64)
    s = sm_scale * (q @ K.T)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    out = w @ V
    u = 2.0 ** -24
    qe = (2.0 ** -28 if fmt == "int8_page_head" else 2.0 ** -17) * np.abs(q).max()
    es = sm_scale * (qe * np.abs(K).sum(-1).max() + 131 * u * (np.abs(q) @ np.abs(K).T).max(-1))
    e = es + np.abs(s).max(-1) * 4 * u + 2.0 ** -21 + 2.0 ** -11 + (len(K) + 16) * u
    bound = 2.0 ** -8 * np.abs(out) + 2 * e[:, None] * (w @ np.abs(V)) * (1 + 2.0 ** -7) + 1e-30
    return out, bound


def sm_scale(D=128):
    return 1.0 / math.sqrt(D)
