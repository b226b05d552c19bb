"""Cases of the operators around the paged KV cache: rotary positions of queries and new keys,
the 8-bit cache with one scale per page and KV head (its write path and the sparse attention
that reads it), and the page operations (copy; fork, grow and free requests; compaction).

Each case runs in a plain form (elementary torch operations) or, with ``own`` set, as a user's
program calls the package.  Cache tensors have the layouts of the package's KVCache:
k_pool [L][S][Hkv][P][D], 8-bit v_pool [L][S][Hkv][D][P], scales [L][S][Hkv] (page_head
formats) or [L][S][P] (per token), slab rows [L][Lp][Hkv*D].  Every shape is synthetic.
"""
import math

import numpy as np
import torch

own = False
D = 128          # the package's head size (rotary positions take others too)

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # rotary: the newest token of one request, every layer in one call (decode, latency)
        dict(name="rope_decode_1", op="rope", dtype="bf16", T=1, L=12, Hq=16, Hkv=2, D=128, rd=128,
             inter=False, scaling="none", packed=False, inverse=False, maxpos=65536),
        # rotary: a prefill chunk out of a fused QKV projection, interleaved pairs, positions
        # stretched for a long context
        dict(name="rope_prefill_32k", op="rope", dtype="bf16", T=32768, L=1, Hq=32, Hkv=4, D=128,
             rd=64, inter=True, scaling="yarn", packed=True, inverse=False, maxpos=131072),
        # cache write: one token per request and layer into partly filled pages (decode append)
        dict(name="append_int8_64", op="store", fmt="int8_page_head", T=64, L=12, Hkv=4, P=64,
             fresh=False),
        # cache write: a prefill chunk into new pages
        dict(name="prefill_e4m3_32k", op="store", fmt="e4m3_page_head", T=32768, L=12, Hkv=4, P=64,
             fresh=True),
        # attention: one request, one layer (latency), 16-token pages
        dict(name="attend_int8_1", op="attend", fmt="int8_page_head", B=1, L=1, ctx=4096, P=16, Hq=8,
             Hkv=1, topk=16, empty=False),
        # attention: 4 requests x 12 layers at 64K, the default decode workload's shape
        dict(name="attend_e4m3_4x12", op="attend", fmt="e4m3_page_head", B=4, L=12, ctx=65536, P=64,
             Hq=16, Hkv=2, topk=32, empty=False),
        # attention: 32 requests x 12 layers at 128K, ragged, one request without a token
        dict(name="attend_int8_32x12", op="attend", fmt="int8_page_head", B=32, L=12, ctx=131072, P=64,
             Hq=32, Hkv=4, topk=32, empty=True),
        # pages: a prefix hit copies one page of two layers
        dict(name="copy_1", op="copy", fmt="bf16", n=1, L=2, Lp=96, Hkv=2, P=16),
        # pages: 400 pages of 12 layers duplicated (a request's context copied out)
        dict(name="copy_400", op="copy", fmt="int8_page_head", n=400, L=12, Lp=1031, Hkv=4, P=64),
        # pages: one beam-search step of 8 beams
        dict(name="fork_beam_8", op="fork", fmt="e4m3_page_head", B=8, beam=4, L=2, nmax=64, Hkv=2,
             P=64),
        # pages: one beam-search step of 16 groups of 4 beams at up to 8K tokens, 12 layers
        dict(name="fork_beam_64", op="fork", fmt="e4m3_page_head", B=64, beam=4, L=12, nmax=130,
             Hkv=2, P=64),
        # pages: half the requests end, the page space is compacted, new ones are admitted; twice
        dict(name="turnover_32", op="turnover", fmt="bf16", B=32, L=12, nmax=250, Hkv=2, P=16),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["rope", "store", "attend", "attend", "copy", "fork", "turnover"])
    fmt8 = rng.choice(["int8_page_head", "e4m3_page_head"])
    fmt = rng.choice(["bf16", "fp8", "int8_page_head", "e4m3_page_head"])
    Hkv = rng.choice([1, 2, 4, 8])
    P = rng.choice([16, 32, 64, 128])
    L = rng.randint(1, 12)
    if op == "rope":
        Dr = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rd = rng.choice([Dr, Dr, Dr // 2, 2 * rng.randint(1, Dr // 2)])
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), T=_logint(rng, 1, 16384),
                    L=L, Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=Dr, rd=rd, inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]),
                    packed=rng.random() < 0.3, inverse=rng.random() < 0.2,
                    maxpos=_logint(rng, 16, 1 << 21))
    if op == "store":
        return dict(op=op, fmt=fmt8, T=_logint(rng, 1, 16384), L=L, Hkv=Hkv, P=P,
                    fresh=rng.random() < 0.5)
    if op == "attend":
        return dict(op=op, fmt=fmt8, B=_logint(rng, 1, 32), L=L, ctx=_logint(rng, 1, 131072), P=P,
                    Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, topk=rng.choice([1, 5, 16, 32, 47]),
                    empty=rng.random() < 0.3)
    if op == "copy":
        return dict(op=op, fmt=fmt, n=_logint(rng, 1, 400), L=L, Lp=rng.randint(800, 1600), Hkv=Hkv,
                    P=P)
    if op == "fork":
        return dict(op=op, fmt=fmt, B=_logint(rng, 1, 64), beam=rng.randint(1, 8), L=L,
                    nmax=_logint(rng, 1, 130), Hkv=Hkv, P=P)
    return dict(op=op, fmt=fmt, B=_logint(rng, 2, 40), L=L, nmax=_logint(rng, 1, 250), Hkv=Hkv, P=16)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), work(c)["bytes"])
    while True:
        c = _draw(rng)
        if c["op"] == "fork" and _pool_bytes(c) > 4 << 30:
            continue
        if work(c)["bytes"] <= most[c["op"]]:
            return c


def _esz(fmt):
    return 2 if fmt == "bf16" else 1


def _page_bytes(c):
    """K, V and scales of one page, and one page's slab row."""
    kv = 2 * c["Hkv"] * c["P"] * D * _esz(c["fmt"])
    sc = {"bf16": 0, "fp8": 8 * c["P"]}.get(c["fmt"], 8 * c["Hkv"])
    return kv + sc, c["Hkv"] * D * 5 + 8


def _fork_pages(c):
    return c["B"] * (c["nmax"] + 1)


def _pool_bytes(c):
    return c["L"] * _fork_pages(c) * _page_bytes(c)[0]


def work(case):
    c = case
    if c["op"] == "rope":
        esz = 4 if c["dtype"] == "f32" else 2
        n = c["L"] * c["T"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 2 * n * esz + 8 * c["T"], "flops": 3 * c["L"] * c["T"] * (c["Hq"] + c["Hkv"]) * c["rd"]}
    if c["op"] == "store":
        # bf16 K, V in, codes out; slab sums in (partly filled pages) and out, slab codes out
        n = c["L"] * c["T"] * c["Hkv"] * D
        pages = c["T"] if not c["fresh"] else -(-c["T"] // c["P"])
        slab = c["L"] * pages * (c["Hkv"] * (D * 9 + 16) + 16)
        return {"bytes": 2 * n * 3 + slab + 8 * c["T"], "flops": 6 * n}
    if c["op"] == "attend":
        n_sel = min(-(-c["ctx"] // c["P"]), c["topk"] + 1)
        tok = c["L"] * c["B"] * n_sel * c["P"]
        io = c["L"] * c["B"] * (c["Hq"] * D * 4 + 8 * n_sel)
        return {"bytes": tok * c["Hkv"] * D * 2 + c["L"] * c["B"] * n_sel * c["Hkv"] * 8 + io,
                "flops": 4 * tok * c["Hq"] * D}
    kv, slab = _page_bytes(c)
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * c["L"] * (kv + slab) + 8 * c["n"], "flops": 0}
    if c["op"] == "fork":
        # about one beam in three is a copy: its last page in every layer; the tables once
        table = 8 * c["B"] * c["nmax"] + 8 * _fork_pages(c)
        return {"bytes": 2 * (-(-c["B"] // 3)) * c["L"] * (kv + slab) + table, "flops": 0}
    # turnover: about a quarter of the pages move in each compaction, a quarter are cleared
    pages = c["B"] * c["nmax"] // 4
    return {"bytes": 2 * pages * c["L"] * (3 * slab + 24) + 48 * c["B"] * c["nmax"], "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_FIELDS = ("k_pool", "v_pool", "k_scale", "v_scale", "slab", "slab_scale", "slab_sum", "slab_cnt",
           "slot_of", "page_of", "last_use", "clock")
_QMAX = {"int8_page_head": 127.0, "e4m3_page_head": 448.0}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _scaling(c):
    """(kind, numbers) of the case's position scaling."""
    return {"none": {}, "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
            "bands": dict(factor=8.0, original_len=8192, low=1.0, high=4.0),
            "yarn": dict(factor=8.0, original_len=8192, low=1.0, high=32.0)}[c["scaling"]]


def _theta(c, base=500000.0):
    """Radians per position of each pair (double) and the factor on cos and sin."""
    rd, kind, s = c["rd"], c["scaling"], _scaling(c)
    if kind == "ntk" and rd > 2:
        base = base * s["factor"] ** (rd / (rd - 2))
    i = torch.arange(rd // 2, dtype=torch.float64)
    th, m = base ** (-2.0 * i / rd), 1.0
    if kind == "linear":
        th = th / s["factor"]
    elif kind == "bands":
        # long wavelengths are stretched, short ones kept, a linear blend between
        mix = ((s["original_len"] * th / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        th = th * mix + th / s["factor"] * (1 - mix)
    elif kind == "yarn":
        # the pair index whose wavelength turns r times over the original length
        def at(r):
            return rd * math.log(s["original_len"] / (2 * math.pi * r)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(s["high"])), 0), min(math.ceil(at(s["low"])), rd - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        th = th / s["factor"] * ramp + th * (1 - ramp)
        m = 0.1 * math.log(s["factor"]) + 1.0
    return th, m


def _prepare_rope(c, seed):
    g, dt = _gen(seed), _TORCH[c["dtype"]]
    L, T, Hq, Hkv, Dr = c["L"], c["T"], c["Hq"], c["Hkv"], c["D"]
    # q and k beside v in one projection's output, or tensors of their own
    W = (Hq + 2 * Hkv) * Dr if c["packed"] else (Hq + Hkv) * Dr
    x = torch.randn((L, T, W), generator=g, device="cuda").to(dt)
    if not c["packed"]:
        q = x[..., :Hq * Dr].contiguous().view(L, T, Hq, Dr)
        k = x[..., Hq * Dr:].contiguous().view(L, T, Hkv, Dr)
    else:
        q = x[..., :Hq * Dr].unflatten(-1, (Hq, Dr))
        k = x[..., Hq * Dr:(Hq + Hkv) * Dr].unflatten(-1, (Hkv, Dr))
    if T > 64:      # a chunk of consecutive tokens that ends at maxpos
        pos = torch.arange(T, device="cuda") + max(0, c["maxpos"] - T)
    else:           # one token of each request
        pos = torch.randint(0, c["maxpos"], (T,), generator=g, device="cuda")
    st = dict(q=q, k=k, pos=pos.to(torch.int64))
    th, m = _theta(c)
    st["theta"], st["m"] = th.cuda(), m
    if own:
        import sparse_attention_decode_indexer_gb300 as ssa
        sc = ssa.RopeScaling(c["scaling"], **_scaling(c)) if c["scaling"] != "none" else None
        st["plan"] = ssa.RopePlan(c["D"], rotary_dim=c["rd"], base=500000.0, interleaved=c["inter"],
                                  scaling=sc)
        st["q_out"] = torch.empty((L, T, Hq, Dr), dtype=dt, device="cuda")
        st["k_out"] = torch.empty((L, T, Hkv, Dr), dtype=dt, device="cuda")
    return st


def _own_cache(c, S, Lp, B, nmax, topk, tensors, L):
    """The package's cache holding the prepared tensors, which then name its own buffers."""
    import sparse_attention_decode_indexer_gb300 as ssa
    lay = ssa.Layout(c["P"], c.get("Hq", c["Hkv"]), c["Hkv"], D, c["fmt"] != "bf16", L, Lp, S, B, nmax,
                     topk, kv_format=c["fmt"])
    cache = ssa.KVCache(lay, host_tier=False)
    for n in _FIELDS:
        t = getattr(cache, n)
        if t is not None and n in tensors:
            t.copy_(tensors[n])
            tensors[n] = t
    ws = torch.zeros((max(ssa.ssa_workspace_size(lay), 256),), dtype=torch.uint8, device="cuda")
    return dict(lay=lay, cache=cache, ws=ws, status=torch.zeros((1,), dtype=torch.int32, device="cuda"))


def _quant(fmt, v):
    """Codes (as bytes) of values already divided by their scale."""
    if fmt == "int8_page_head":
        return v.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(fmt, codes):
    """The numbers that code bytes stand for (before their scale), fp32."""
    return codes.view(torch.int8 if fmt == "int8_page_head" else torch.float8_e4m3fn).float()


def _random_pages(c, L, S, g, spread=True):
    """[L][S] pages of quantised normal K and V with their page_head scales."""
    H, P, fmt = c["Hkv"], c["P"], c["fmt"]
    pools, scales = [], []
    qmax = torch.tensor(_QMAX[fmt], device="cuda")
    for _ in range(2):
        pool = torch.empty((L, S, H * P * D), dtype=torch.uint8, device="cuda")
        scale = torch.empty((L, S, H), device="cuda")
        for l in range(L):
            x = torch.randn((S, H, P * D), generator=g, device="cuda")
            if spread:     # heads and pages of different magnitude
                x = x * torch.exp2(torch.randn((S, H, 1), generator=g, device="cuda"))
            scale[l] = x.abs().amax(-1) / qmax
            pool[l] = _quant(fmt, x / scale[l][..., None]).view(S, -1)
        pools.append(pool)
        scales.append(scale)
    return dict(k_pool=pools[0], v_pool=pools[1], k_scale=scales[0], v_scale=scales[1])


def _store_sizes(c):
    if c["fresh"]:
        return -(-c["T"] // c["P"])
    return c["T"]


def _prepare_store(c, seed):
    g = _gen(seed)
    L, T, H, P, S = c["L"], c["T"], c["Hkv"], c["P"], _store_sizes(c)
    if c["fresh"]:
        t = dict(k_pool=torch.zeros((L, S, H * P * D), dtype=torch.uint8, device="cuda"),
                 v_pool=torch.zeros((L, S, H * P * D), dtype=torch.uint8, device="cuda"),
                 k_scale=torch.zeros((L, S, H), device="cuda"), v_scale=torch.zeros((L, S, H), device="cuda"))
        cnt = torch.zeros((S,), dtype=torch.int32, device="cuda")
        pos = torch.arange(T, device="cuda")
    else:
        t = _random_pages(c, L, S, g, spread=False)
        cnt = torch.randint(1, P, (S,), generator=g, device="cuda", dtype=torch.int32)
        pos = torch.arange(S, device="cuda") * P + cnt
    t["slab_cnt"] = cnt.expand(L, S).contiguous()
    t["slab_sum"] = torch.randn((L, S, H * D), generator=g, device="cuda") * t["slab_cnt"][..., None].float().sqrt()
    t["slab"] = torch.zeros((L, S, H * D), dtype=torch.int8, device="cuda")
    t["slab_scale"] = torch.zeros((L, S), device="cuda")
    t["slot_of"] = torch.stack([torch.randperm(S, generator=g, device="cuda") for _ in range(L)]).int()
    t["page_of"] = torch.argsort(t["slot_of"].long(), -1).int()
    st = dict(t=t, pos=pos.to(torch.int64), fresh=c["fresh"],
              k=torch.randn((L, T, H, D), generator=g, device="cuda").bfloat16(),
              v=torch.randn((L, T, H, D), generator=g, device="cuda").bfloat16())
    if own:
        st["own"] = _own_cache(c, S, S, 1, 1, 1, t, L)
    return st


def _prepare_attend(c, seed):
    g = _gen(seed)
    L, B, P, k = c["L"], c["B"], c["P"], c["topk"]
    nmax, W = -(-c["ctx"] // P), 2 * c["topk"] + 8
    n_sel = min(nmax, k + 1)
    lens = c["ctx"] - torch.randint(0, max(1, c["ctx"] // 4), (B,), generator=g, device="cuda")
    if c["empty"]:
        lens[B // 2] = 0
    S = B * n_sel
    t = _random_pages(c, L, S, g)
    # the selection: random pages before the last one, the last one, ascending, -1 padded
    n = (lens + P - 1) // P
    keys = torch.rand((L, B, nmax), generator=g, device="cuda")
    p = torch.arange(nmax, device="cuda")
    keys = keys.masked_fill(p == n[:, None] - 1, 2.0).masked_fill(p >= n[:, None], -1.0)
    top = keys.topk(n_sel, -1)
    pages = torch.where(top.values >= 0, top.indices, nmax).sort(-1).values
    sel = torch.full((L, B, W), -1, dtype=torch.int32, device="cuda")
    sel[..., :n_sel] = torch.where(pages < nmax, pages, -1).int()
    slots = torch.stack([torch.randperm(S, generator=g, device="cuda") for _ in range(L)]).int()
    phys = torch.full_like(sel, -1)
    phys[..., :n_sel] = torch.where(pages < nmax, slots.view(L, B, n_sel), -1).int()
    st = dict(t=t, sel=sel, phys=phys, lens=lens.int(), n_sel=n_sel,
              q=torch.randn((L, B, c["Hq"], D), generator=g, device="cuda").bfloat16())
    if own:
        st["own"] = _own_cache(c, S, S, B, nmax, k, t, L)
        st["out"] = torch.empty_like(st["q"])
    return st


def _page_tensors(c, L, Lp, g):
    """A resident cache of random bytes: every logical page in a slot of its own."""
    H, P, fmt = c["Hkv"], c["P"], c["fmt"]
    pb = H * P * D * _esz(fmt)

    def rand(*shape):
        n = math.prod(shape)
        words = torch.randint(-(1 << 62), 1 << 62, (-(-n // 8),), generator=g, device="cuda")
        return words.view(torch.uint8)[:n].view(*shape)
    t = dict(k_pool=rand(L, Lp, pb), v_pool=rand(L, Lp, pb))
    if fmt != "bf16":
        ns = P if fmt == "fp8" else H
        t["k_scale"] = torch.rand((L, Lp, ns), generator=g, device="cuda")
        t["v_scale"] = torch.rand((L, Lp, ns), generator=g, device="cuda")
    t["slab"] = rand(L, Lp, H * D).view(torch.int8)
    t["slab_sum"] = torch.randn((L, Lp, H * D), generator=g, device="cuda")
    t["slab_scale"] = torch.rand((L, Lp), generator=g, device="cuda")
    t["slab_cnt"] = torch.randint(1, P + 1, (L, Lp), generator=g, device="cuda", dtype=torch.int32)
    t["slot_of"] = torch.stack([torch.randperm(Lp, generator=g, device="cuda") for _ in range(L)]).int()
    t["page_of"] = torch.argsort(t["slot_of"].long(), -1).int()
    return t


def _prepare_copy(c, seed):
    g = _gen(seed)
    t = _page_tensors(c, c["L"], c["Lp"], g)
    perm = torch.randperm(c["Lp"], generator=g, device="cuda").int()
    st = dict(t=t, src=perm[:c["n"]].contiguous(), dst=perm[c["n"]:2 * c["n"]].contiguous())
    if own:
        st["own"] = _own_cache(c, c["Lp"], c["Lp"], 1, 1, 1, t, c["L"])
    return st


def _prepare_fork(c, seed):
    g = _gen(seed)
    B, P, nmax, Lp = c["B"], c["P"], c["nmax"], _fork_pages(c)
    t = _page_tensors(c, c["L"], Lp, g)
    lens = torch.randint(1, nmax * P + 1, (B,), generator=g, device="cuda").int()
    n = (lens + P - 1) // P
    pages = torch.randperm(Lp, generator=g, device="cuda")[:B * nmax].view(B, nmax).int()
    bt = torch.where(torch.arange(nmax, device="cuda") < n[:, None], pages, -1)
    # beam search: every beam continues some beam of its group
    row = torch.arange(B, device="cuda")
    first = row // c["beam"] * c["beam"]
    width = (B - first).clamp(max=c["beam"])
    parent = (first + (torch.rand((B,), generator=g, device="cuda") * width).long()).clamp(max=B - 1).int()
    st = dict(t=t, bt=bt.contiguous(), lens=lens, parent=parent, ref=_refs(bt, lens, P, Lp))
    if own:
        import sparse_attention_decode_indexer_gb300 as ssa
        st["own"] = _own_cache(c, Lp, Lp, B, nmax, 1, t, c["L"])
        st["table"] = ssa.RequestTable(st["own"]["lay"], bt, lens, ref=st["ref"])
    return st


def _prepare_turnover(c, seed):
    g = _gen(seed)
    B, P, nmax = c["B"], c["P"], c["nmax"]
    Lp = B * nmax + 1
    t = _page_tensors(c, c["L"], Lp, g)
    lens = torch.randint(max(1, nmax * P // 2), nmax * P + 1, (B,), generator=g, device="cuda").int()
    n = (lens + P - 1) // P
    pages = torch.randperm(Lp, generator=g, device="cuda")[:B * nmax].view(B, nmax).int()
    bt = torch.where(torch.arange(nmax, device="cuda") < n[:, None], pages, -1)
    row = torch.arange(B, device="cuda", dtype=torch.int32)
    st = dict(t=t, bt=bt.contiguous(), lens=lens, ref=_refs(bt, lens, P, Lp))
    # a quarter of the requests ends and is admitted anew, then another quarter
    for h in range(2):
        turn = (row % 4) == h
        st["end%d" % h] = torch.where(turn, -1, row)
        st["new%d" % h] = torch.where(turn, lens, 0)
    if own:
        import sparse_attention_decode_indexer_gb300 as ssa
        st["own"] = _own_cache(c, Lp, Lp, B, nmax, 1, t, c["L"])
        st["table"] = ssa.RequestTable(st["own"]["lay"], bt, lens, ref=st["ref"])
    return st


def _refs(bt, lens, P, Lp):
    """References of each page by the requests' rows."""
    used = torch.arange(bt.shape[1], device=bt.device) < ((lens + P - 1) // P)[:, None]
    return torch.bincount(bt[used].long(), minlength=Lp)[:Lp].int()


def prepare(case, seed):
    st = {"rope": _prepare_rope, "store": _prepare_store, "attend": _prepare_attend,
          "copy": _prepare_copy, "fork": _prepare_fork, "turnover": _prepare_turnover}[case["op"]](case, seed)
    st["case"] = case
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_rope(st):
    c = st["case"]
    ang = st["pos"].double()[:, None] * st["theta"]            # [T][rd/2], 64 bits: far positions
    cos, sin = (ang.cos() * st["m"]).float()[:, None], (ang.sin() * st["m"]).float()[:, None]
    if c["inverse"]:
        sin = -sin

    def turn(x):
        xr, rest = x[..., :c["rd"]].float(), x[..., c["rd"]:]
        a, b = (xr[..., 0::2], xr[..., 1::2]) if c["inter"] else xr.chunk(2, -1)
        ra, rb = a * cos - b * sin, b * cos + a * sin
        y = torch.stack((ra, rb), -1).flatten(-2) if c["inter"] else torch.cat((ra, rb), -1)
        return torch.cat((y.to(x.dtype), rest), -1)
    return [turn(st["q"]), turn(st["k"])]


def _plain_store(st):
    c, t = st["case"], st["t"]
    L, T, H, P, fmt = c["L"], c["T"], c["Hkv"], c["P"], c["fmt"]
    page, j = st["pos"] // P, st["pos"] % P
    up, inv, count = page.unique_consecutive(return_inverse=True, return_counts=True)
    n = up.numel()
    lay = torch.arange(L, device="cuda")[:, None]
    slot = t["slot_of"][:, up].long()                           # [L][n]
    cnt = t["slab_cnt"][:, up]
    fresh = (cnt == 0)[..., None]
    qmax = torch.tensor(_QMAX[fmt], device="cuda")
    tslot = slot[:, inv]                                        # [L][T]
    for x, is_v, pool, scale in ((st["k"].float(), False, t["k_pool"], t["k_scale"]),
                                 (st["v"].float(), True, t["v_pool"], t["v_scale"])):
        amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)                       # [L][T][H]
        need = torch.zeros((L, n, H), device="cuda").scatter_reduce(
            1, inv[None, :, None].expand(L, T, H), amax, "amax") / qmax
        old = scale[lay, slot]
        s = torch.where(fresh, need, torch.maximum(old, need))
        scale[lay, slot] = s
        view = pool.view(L, -1, H, D, P) if is_v else pool.view(L, -1, H, P, D)
        gl, gp = ((s > old) & ~fresh).any(-1).nonzero(as_tuple=True)
        if gl.numel():           # pages whose scale grew: their codes again, at the new scale
            gs = slot[gl, gp]
            r = torch.where((s > old)[gl, gp], old[gl, gp] / s[gl, gp], 1.0)[..., None, None]
            view[gl, gs] = _quant(fmt, _values(fmt, view[gl, gs]) * r)
        sx = s[:, inv][..., None]
        codes = _quant(fmt, torch.where(sx > 0, x / sx, 0.0))                          # [L][T][H][D]
        if is_v:
            view[lay, tslot, :, :, j] = codes
        else:
            view[lay, tslot, :, j] = codes
    # the slab: fp32 running sums of the bf16 keys, in token order by definition
    x = st["k"].float().view(L, T, H * D)
    most = int(count.max())
    start = torch.cumsum(count, 0) - count
    at = torch.arange(most, device="cuda")[:, None]
    take = (start + at).clamp(max=T - 1)
    sums = t["slab_sum"][:, up]
    for r in range(most):
        sums = sums + torch.where((r < count)[:, None], x[:, take[r]], 0.0)
    cnt = cnt + count.int()
    mean = sums / cnt[..., None].float()
    amax = mean.abs().amax(-1)
    s = amax / torch.tensor(127.0, device="cuda")
    code = torch.where(amax[..., None] > 0, (mean / s[..., None]).round().clamp(-127, 127), 0.0)
    t["slab_sum"][:, up], t["slab_cnt"][:, up] = sums, cnt
    t["slab_scale"][:, up], t["slab"][:, up] = s, code.to(torch.int8)


def _store_outputs(st):
    t, fmt = st["t"], st["case"]["fmt"]
    as_values = torch.float8_e4m3fn if fmt == "e4m3_page_head" else torch.int8
    return {"k": t["k_pool"].view(as_values), "v": t["v_pool"].view(as_values), "k_scale": t["k_scale"],
            "v_scale": t["v_scale"], "slab": t["slab"], "slab_sum": t["slab_sum"],
            "slab_scale": t["slab_scale"], "slab_cnt": t["slab_cnt"]}


def _plain_attend(st):
    c, t, n = st["case"], st["t"], st["n_sel"]
    L, B, P, Hq, H = c["L"], c["B"], c["P"], c["Hq"], c["Hkv"]
    page, slot = st["sel"][..., :n].long(), st["phys"][..., :n].long()
    ok = (page >= 0) & (slot >= 0)
    lay, slot = torch.arange(L, device="cuda")[:, None, None], slot.clamp(min=0)

    def gather(pool, scale, shape):
        x = _values(c["fmt"], pool.view(L, -1, H, *shape)[lay, slot])          # [L][B][n][H]...
        return x * scale[lay, slot][..., None, None]
    k = gather(t["k_pool"], t["k_scale"], (P, D)).transpose(2, 3).reshape(L, B, H, n * P, D)
    v = gather(t["v_pool"], t["v_scale"], (D, P)).permute(0, 1, 3, 2, 5, 4).reshape(L, B, H, n * P, D)
    q = st["q"].float().view(L, B, H, Hq // H, D)
    s = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(D))
    tok = page[..., None] * P + torch.arange(P, device="cuda")
    live = (ok[..., None] & (tok < st["lens"][:, None, None])).view(L, B, 1, 1, n * P)
    s = s.masked_fill(~live, -math.inf)
    e = torch.where(live, (s - s.amax(-1, keepdim=True)).exp(), 0.0)
    z = e.sum(-1, keepdim=True)
    o = torch.where(z > 0, (e / z) @ v, 0.0)                      # no token: zeros
    return o.reshape(L, B, Hq, D).bfloat16()


def _copy_content(t, src, dst):
    """Pages dst[i] := src[i] in every layer (distinct pages; no pair reads another's page)."""
    src, dst = src.long(), dst.long()
    lay = torch.arange(t["slot_of"].shape[0], device="cuda")[:, None]
    a, b = t["slot_of"][:, src].long(), t["slot_of"][:, dst].long()
    for name in ("k_pool", "v_pool", "k_scale", "v_scale"):
        if name in t:
            t[name][lay, b] = t[name][lay, a]
    for name in ("slab", "slab_scale", "slab_sum", "slab_cnt"):
        t[name][:, dst] = t[name][:, src]


def _count(ref, ids, add):
    ref.scatter_add_(0, ids.long(), torch.full_like(ids, add))


def _plain_fork(st, parent, new_lens):
    """Row i continues old row parent[i] (-1: an empty one), grown to new_lens[i] tokens."""
    c, t, bt, lens, ref = st["case"], st["t"], st["bt"], st["lens"], st["ref"]
    P, nmax = c["P"], bt.shape[1]
    col = torch.arange(nmax, device="cuda")
    par = parent.clamp(min=0).long()
    plen = torch.where(parent >= 0, lens[par], 0)
    nlen = plen if new_lens is None else torch.maximum(plen, new_lens)
    old_n, pn, nn, full = (lens + P - 1) // P, (plen + P - 1) // P, (nlen + P - 1) // P, plen // P
    pb = bt[par]
    partial = plen % P > 0
    _count(ref, bt[col < old_n[:, None]], -1)
    _count(ref, pb[col < pn[:, None]], 1)
    # the partly filled last page: the first row that continues it keeps it, unless another
    # reference stays; every other row gets a copy
    g = torch.where(partial, pb.gather(1, full.clamp(max=nmax - 1).long()[:, None])[:, 0], -1)
    same = (g[:, None] == g) & partial[:, None]
    first = partial & ~same.tril(-1).any(1)
    others = ref[g.clamp(min=0).long()] - same.sum(1).int()
    keep = first & (others <= 0)
    copy = partial & ~keep
    ref[g[first].long()] = others[first].clamp(min=1)
    # new pages: the lowest free ids, in row order
    free = (ref <= 0).nonzero()[:, 0].int()
    need = copy.int() + nn - pn
    base = torch.cumsum(need, 0).int() - need
    grown = (col >= pn[:, None]) & (col < nn[:, None])
    tail = (col == full[:, None]) & copy[:, None]
    rank = torch.where(tail, base[:, None], base[:, None] + copy.int()[:, None] + col.int() - pn[:, None])
    got = free[rank.clamp(0, free.numel() - 1).long()]
    bt.copy_(torch.where(grown | tail, got, torch.where(col < pn[:, None], pb, -1)))
    lens.copy_(nlen)
    fresh = got[grown].long()
    ref[got[grown | tail].long()] = 1
    for name in ("slab", "slab_scale", "slab_sum", "slab_cnt"):
        t[name][:, fresh] = 0
    _copy_content(t, g[copy], got[tail])


def _plain_compact(st):
    """Live pages move down to the lowest ids: the k-th live page at or above the number of live
    pages goes to the k-th free id below it; the two trade slots, so no pool bytes move."""
    t, bt, ref = st["t"], st["bt"], st["ref"]
    Lp = ref.numel()
    live = ref > 0
    ids = torch.arange(Lp, device="cuda")
    n_live = live.sum()
    src, dst = (live & (ids >= n_live)).nonzero()[:, 0], (~live & (ids < n_live)).nonzero()[:, 0]
    to = ids.clone()
    to[src] = dst
    bt.copy_(torch.where(bt >= 0, to[bt.clamp(min=0).long()].int(), -1))
    ref[dst], ref[src] = ref[src], 0
    for name in ("slab", "slab_scale", "slab_sum", "slab_cnt"):
        t[name][:, dst] = t[name][:, src]
    a, b = t["slot_of"][:, src], t["slot_of"][:, dst]
    t["slot_of"][:, dst], t["slot_of"][:, src] = a, b
    t["page_of"].scatter_(1, a.long(), dst.int().expand_as(a))
    t["page_of"].scatter_(1, b.long(), src.int().expand_as(b))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if own:
        import sparse_attention_decode_indexer_gb300 as ssa
        o = st.get("own")
    if op == "rope":
        if not own:
            return _plain_rope(st)
        ssa.ssa_rope(st["plan"], st["pos"], st["q"], st["k"], q_out=st["q_out"], k_out=st["k_out"],
                     inverse=c["inverse"])
        return [st["q_out"], st["k_out"]]
    if op == "store":
        t = st["t"]
        if st["fresh"]:            # new pages come with cleared slab rows
            t["slab_cnt"].zero_()
            t["slab_sum"].zero_()
        if own:
            ssa.ssa_store_kv_mirror(o["cache"], 0, c["L"], st["k"], st["v"], st["pos"], o["status"])
        else:
            _plain_store(st)
        return _store_outputs(st)
    if op == "attend":
        if not own:
            return _plain_attend(st)
        ssa.ssa_sparse_paged_decode(o["cache"], 0, c["L"], st["q"], st["sel"], st["phys"], st["lens"],
                                    1.0 / math.sqrt(D), st["out"], o["status"], o["ws"])
        return st["out"]
    t = st["t"]
    if op == "copy":
        if own:
            ssa.ssa_copy_pages(o["cache"], st["src"], st["dst"], o["status"], o["ws"])
        else:
            _copy_content(t, st["src"], st["dst"])
        return dict(t)
    if op == "fork":
        if own:
            ssa.ssa_fork_requests(o["cache"], st["table"], st["parent"], None, o["status"], o["ws"])
            tb = st["table"]
            return dict(t, bt=tb.block_table, lens=tb.seq_lens, ref=tb.ref)
        _plain_fork(st, st["parent"], None)
        return dict(t, bt=st["bt"], lens=st["lens"], ref=st["ref"])
    for end, new in ((st["end0"], st["new0"]), (st["end1"], st["new1"])):
        if own:
            ssa.ssa_fork_requests(o["cache"], st["table"], end, None, o["status"], o["ws"])
            ssa.ssa_compact_pages(o["cache"], st["table"], o["status"], o["ws"])
            ssa.ssa_fork_requests(o["cache"], st["table"], end, new, o["status"], o["ws"])
        else:
            _plain_fork(st, end, None)
            _plain_compact(st)
            _plain_fork(st, end, new)
    tb = st.get("table")
    rows = dict(bt=tb.block_table, lens=tb.seq_lens, ref=tb.ref) if own else \
        dict(bt=st["bt"], lens=st["lens"], ref=st["ref"])
    return dict({n: t[n] for n in ("slab", "slab_scale", "slab_sum", "slab_cnt", "slot_of", "page_of")}, **rows)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rope(c, st):
    # a pair as a complex number, turned by the unit number of its angle
    ang = np.outer(st["pos"].cpu().numpy().astype(np.float64), st["theta"].cpu().numpy())
    turn = torch.from_numpy(st["m"] * np.exp((-1j if c["inverse"] else 1j) * ang)).cuda()[:, None, :]
    i = torch.arange(c["rd"] // 2, device="cuda")
    lo, hi = (2 * i, 2 * i + 1) if c["inter"] else (i, i + c["rd"] // 2)
    outs = []
    for x in (st["q"], st["k"]):
        y = x.double().clone()
        z = torch.complex(y[..., lo], y[..., hi]) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        outs.append(y)
    return outs


def _exact_attend(c, st):
    t, n, P, G = st["t"], st["n_sel"], c["P"], c["Hq"] // c["Hkv"]
    kind = torch.int8 if c["fmt"] == "int8_page_head" else torch.float8_e4m3fn
    out = torch.zeros((c["L"], c["B"], c["Hq"], D), dtype=torch.float64, device="cuda")
    kp = t["k_pool"].view(kind).view(c["L"], -1, c["Hkv"], P, D)
    vp = t["v_pool"].view(kind).view(c["L"], -1, c["Hkv"], D, P)
    lens = st["lens"].tolist()
    for l in range(c["L"]):
        for b in range(c["B"]):
            page, slot = st["sel"][l, b, :n].long(), st["phys"][l, b, :n].long()
            page, slot = page[page >= 0], slot[page >= 0]
            live = (page[:, None] * P + torch.arange(P, device="cuda")).flatten() < lens[b]
            if not page.numel():
                continue
            k = kp[l].view(torch.uint8)[slot].view(kind).double() * t["k_scale"][l, slot].double()[..., None, None]
            v = vp[l].view(torch.uint8)[slot].view(kind).double() * t["v_scale"][l, slot].double()[..., None, None]
            k = k.permute(1, 0, 2, 3).flatten(1, 2).repeat_interleave(G, 0)
            v = v.permute(1, 0, 3, 2).flatten(1, 2).repeat_interleave(G, 0)
            w = torch.einsum("hd,htd->ht", st["q"][l, b].double(), k) / math.sqrt(D)
            out[l, b] = torch.einsum("ht,htd->hd", w[:, live].softmax(-1), v[:, live])
    return out


def _exact_store(c, st):
    t, P, H, L = st["t"], c["P"], c["Hkv"], c["L"]
    pos = st["pos"].cpu().numpy()
    page = pos // P
    edge = np.flatnonzero(np.diff(page, prepend=-1))
    res = {}
    seg = torch.from_numpy(np.repeat(np.arange(edge.size), np.diff(np.append(edge, pos.size)))).cuda()
    pg = torch.from_numpy(page[edge]).cuda()
    lay = torch.arange(L, device="cuda")[:, None]
    slot = t["slot_of"].long()[:, pg]
    fresh = (t["slab_cnt"][:, pg] == 0)[..., None]
    for name, x in (("k_scale", st["k"]), ("v_scale", st["v"])):
        big = x.double().abs().amax(-1)
        per = torch.stack([torch.zeros((edge.size, H), dtype=torch.float64, device="cuda").index_reduce_(
            0, seg, big[l], "amax") for l in range(L)]) / _QMAX[c["fmt"]]
        out = t[name].double().clone()
        out[lay, slot] = torch.where(fresh, per, torch.maximum(out[lay, slot], per))
        res[name] = out
    sums = t["slab_sum"].double().clone()
    add = torch.zeros((L, edge.size, H * D), dtype=torch.float64, device="cuda")
    add.index_add_(1, seg, st["k"].double().view(L, pos.size, H * D))
    sums[:, pg] += add
    cnt = t["slab_cnt"].double()
    cnt[:, pg] += torch.from_numpy(np.diff(np.append(edge, pos.size))).cuda().double()
    scale = t["slab_scale"].double().clone()
    scale[:, pg] = (sums[:, pg] / cnt[:, pg][..., None]).abs().amax(-1) / 127
    return {"k": None, "v": None, **res, "slab": None, "slab_sum": sums, "slab_scale": scale, "slab_cnt": None}


def exact(case, seed):
    if case["op"] not in ("rope", "store", "attend"):
        return None                       # bytes, ids and counts: compared as they are
    st = prepare(case, seed)
    return {"rope": _exact_rope, "store": _exact_store, "attend": _exact_attend}[case["op"]](case, st)
