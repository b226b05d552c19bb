"""Cases of the operators at both ends of a serving loop around the paged cache: a prompt's way in
(norms of queries and keys with the rotary positions in the same pass; attention over whole prompts,
packed sequences of different lengths) and the choice of the next tokens (selection over beams and
vocabulary, with the token histories reordered).

Each case runs in a plain form (elementary torch operations) or, with ``own`` set, as a user's
program calls the package.  Every shape is synthetic.
"""
import math
import random

import torch

own = False
D = 128          # the package's head size (the norms and positions take others too)

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # prompt attention: one very short prompt (latency)
        dict(name="prompt_17", op="prompt", dtype="bf16", n=1, total=17, ctx=0, Hq=8, Hkv=1, causal=True,
             packed=False, lens_seed=0),
        # prompt attention: eight new tokens behind a long context (a short turn, drafted tokens)
        dict(name="prompt_tail_8", op="prompt", dtype="bf16", n=1, total=8, ctx=65528, Hq=16, Hkv=2,
             causal=True, packed=False, lens_seed=0),
        # prompt attention: a batch of prompts of different lengths out of a fused projection
        dict(name="prompt_packed_24", op="prompt", dtype="bf16", n=24, total=24576, ctx=0, Hq=32, Hkv=4,
             causal=True, packed=True, lens_seed=1),
        # prompt attention: four texts, every token sees the whole text, seven query heads per KV head
        dict(name="prompt_full_f16", op="prompt", dtype="f16", n=4, total=9001, ctx=0, Hq=14, Hkv=2,
             causal=False, packed=False, lens_seed=2),
        # prompt attention: one long prompt
        dict(name="prompt_24k", op="prompt", dtype="bf16", n=1, total=24576, ctx=0, Hq=16, Hkv=2,
             causal=True, packed=False, lens_seed=0),
        # norm and positions: the newest token of one request, every layer in one call (decode)
        dict(name="norm_rope_1", op="norm", dtype="bf16", T=1, L=12, Hq=16, Hkv=2, D=128, rd=128,
             inter=False, packed=False, maxpos=65536),
        # norm and positions: a prefill chunk out of a fused projection
        dict(name="norm_rope_32k", op="norm", dtype="bf16", T=32768, L=1, Hq=32, Hkv=4, D=128, rd=128,
             inter=False, packed=True, maxpos=131072),
        # norm and positions: fp32, a head of 96 of which 64 turn in interleaved pairs, three layers
        dict(name="norm_rope_f32_96", op="norm", dtype="f32", T=4099, L=3, Hq=12, Hkv=4, D=96, rd=64,
             inter=True, packed=False, maxpos=8192),
        # selection: four beams of one request (latency)
        dict(name="beam_1x4", op="beam", dtype="f32", groups=1, beams=4, V=32000, pad=0, hist=512,
             eos=True),
        # selection: one beam, greedy decoding of 64 requests
        dict(name="beam_64x1", op="beam", dtype="f16", groups=64, beams=1, V=131072, pad=0, hist=0,
             eos=False),
        # selection: 16 requests of four beams, an odd vocabulary in padded rows
        dict(name="beam_16x4", op="beam", dtype="f32", groups=16, beams=4, V=100003, pad=29, hist=512,
             eos=True),
        # selection: 32 requests of eight beams, long histories
        dict(name="beam_32x8", op="beam", dtype="bf16", groups=32, beams=8, V=160000, pad=0, hist=4096,
             eos=True),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["prompt", "prompt", "norm", "beam"])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "prompt":
        total = _logint(rng, 1, 32768)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]), n=min(total, _logint(rng, 1, 64)),
                    total=total, ctx=_logint(rng, 1, 65536) if rng.random() < 0.35 else 0,
                    Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, causal=rng.random() < 0.8,
                    packed=rng.random() < 0.3, lens_seed=rng.randrange(1 << 30))
    if op == "norm":
        Dr = rng.choice([64, 80, 96, 128, 128, 192, 256])
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), T=_logint(rng, 1, 32768),
                    L=rng.choice([1, 1, rng.randint(2, 12)]), Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=Dr,
                    rd=rng.choice([Dr, Dr, Dr // 2, 2 * rng.randint(1, Dr // 2)]),
                    inter=rng.random() < 0.5, packed=rng.random() < 0.3, maxpos=_logint(rng, 16, 1 << 21))
    return dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]), groups=_logint(rng, 1, 64),
                beams=rng.choice([1, 2, 3, 4, 5, 8, 16]), V=_logint(rng, 100, 200000),
                pad=rng.choice([0, 0, rng.randint(1, 64)]), hist=rng.choice([0, _logint(rng, 2, 4096)]),
                eos=rng.random() < 0.6)


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for key in ("bytes", "flops"):
            most[c["op"], key] = max(most.get((c["op"], key), 0), w[key])
    while True:
        c = _draw(rng)
        w = work(c)
        if c["op"] == "beam" and c["groups"] * c["beams"] * c["V"] > 256 * 160000:
            continue
        if all(w[key] <= most[c["op"], key] for key in w):
            return c


def _lens(c):
    """(query tokens, keys) of each sequence: ragged, some of them empty where there are many."""
    rng = random.Random(c["lens_seed"])
    n, total = c["n"], c["total"]
    if n == 1:
        lq = [total]
    else:
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lq = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    ctx = c["ctx"] // n
    lk = [x + (ctx if n == 1 else rng.randint(0, 2 * ctx)) for x in lq]
    return lq, lk


def _pairs(c):
    """(query, key) pairs of one head."""
    return sum(a * b - (a * (a - 1) // 2 if c["causal"] else 0) for a, b in zip(*_lens(c)))


_ESZ = {"bf16": 2, "f16": 2, "f32": 4}


def work(case):
    c = case
    if c["op"] == "prompt":
        lq, lk = _lens(c)
        return {"bytes": 4 * D * (sum(lq) * c["Hq"] + sum(lk) * c["Hkv"]) + 4 * sum(lq) * c["Hq"],
                "flops": 4 * D * c["Hq"] * _pairs(c)}
    if c["op"] == "norm":
        n = c["L"] * c["T"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 2 * n * c["D"] * _ESZ[c["dtype"]] + 8 * c["T"], "flops": n * (4 * c["D"] + 3 * c["rd"])}
    rows = c["groups"] * c["beams"]
    # logits once; the tokens so far (half of the longest history, on average) in and out
    return {"bytes": rows * (c["V"] * _ESZ[c["dtype"]] + 4 * c["hist"] + 32), "flops": 4 * rows * c["V"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _qkv(c, g, shape, width, dt):
    """q, k (and v): views of one projection's output, or tensors of their own."""
    Hq, Hkv = c["Hq"], c["Hkv"]
    x = torch.randn((*shape, (Hq + 2 * Hkv) * width), generator=g, device="cuda").to(dt)
    parts = x.split([Hq * width, Hkv * width, Hkv * width], -1)
    parts = [p.unflatten(-1, (-1, width)) for p in parts]
    return parts if c["packed"] else [p.contiguous() for p in parts]


def _prepare_prompt(c, seed):
    g, dt = _gen(seed), _TORCH[c["dtype"]]
    lq, lk = _lens(c)
    Tq, Tk = sum(lq), sum(lk)
    if Tq == Tk:
        q, k, v = _qkv(c, g, (Tq,), D, dt)
    else:
        q = torch.randn((Tq, c["Hq"], D), generator=g, device="cuda").to(dt)
        k, v = (torch.randn((Tk, c["Hkv"], D), generator=g, device="cuda").to(dt) for _ in range(2))
    cu = [torch.tensor([sum(x[:i]) for i in range(len(x) + 1)], dtype=torch.int32, device="cuda")
          for x in (lq, lk)]
    st = dict(q=q, k=k, v=v, lq=lq, lk=lk, cu_q=cu[0], cu_k=cu[1])
    if own:
        import sparse_attention_decode_indexer_gb300 as ssa
        st["out"] = torch.empty((Tq, c["Hq"], D), dtype=dt, device="cuda")
        st["lse"] = torch.empty((Tq, c["Hq"]), device="cuda")
        st["status"] = torch.zeros((1,), dtype=torch.int32, device="cuda")
        st["ws"] = torch.zeros((ssa.ssa_prompt_workspace_size(),), dtype=torch.uint8, device="cuda")
    return st


def _theta(c):
    i = torch.arange(c["rd"] // 2, dtype=torch.float64)
    return 500000.0 ** (-2.0 * i / c["rd"])


def _prepare_norm(c, seed):
    g, dt = _gen(seed), _TORCH[c["dtype"]]
    L, T, Dr = c["L"], c["T"], c["D"]
    q, k, _ = _qkv(c, g, (L, T), Dr, dt)
    # learned weights: about one, one vector per layer for q and one for k
    wq, wk = (1.0 + 0.2 * torch.randn((L, Dr), generator=g, device="cuda") for _ in range(2))
    if T > 64:      # a chunk of consecutive tokens that ends at maxpos
        pos = torch.arange(T, device="cuda") + max(0, c["maxpos"] - T)
    else:           # one token of each request
        pos = torch.randint(0, c["maxpos"], (T,), generator=g, device="cuda")
    st = dict(q=q, k=k, wq=wq, wk=wk, pos=pos, theta=_theta(c).cuda(), eps=1e-6)
    if own:
        import sparse_attention_decode_indexer_gb300 as ssa
        st["plan"] = ssa.RopePlan(Dr, rotary_dim=c["rd"], base=500000.0, interleaved=c["inter"])
        st["norm"] = ssa.HeadNorm(wq, wk, eps=st["eps"])
        st["q_out"] = torch.empty((L, T, c["Hq"], Dr), dtype=dt, device="cuda")
        st["k_out"] = torch.empty((L, T, c["Hkv"], Dr), dtype=dt, device="cuda")
    return st


def _prepare_beam(c, seed):
    g, dt = _gen(seed), _TORCH[c["dtype"]]
    G, K, V = c["groups"], c["beams"], c["V"]
    B = G * K
    x = 2.5 * torch.randn((B, V + c["pad"]), generator=g, device="cuda")
    # a few tokens that the model holds for likely
    at = torch.randint(0, V, (B, 6), generator=g, device="cuda")
    x.scatter_add_(1, at, 6.0 + 2.0 * torch.rand((B, 6), generator=g, device="cuda"))
    st = dict(logits=x.to(dt)[:, :V], eos=V // 3 if c["eos"] else -1)
    # beams some tokens along: their sums of log-probabilities, a tenth of them ended
    st["scores"] = -20.0 * torch.rand((B,), generator=g, device="cuda") - 2.0
    st["finished"] = (torch.rand((B,), generator=g, device="cuda") < (0.1 if c["eos"] else 0.0)).to(torch.uint8)
    h = c["hist"]
    st["history"] = torch.randint(0, V, (B, h), generator=g, device="cuda", dtype=torch.int32)
    st["hist_len"] = torch.randint(0, h, (G,), generator=g, device="cuda", dtype=torch.int32) if h else None
    st["seq_lens"] = torch.randint(1, 131072, (B,), generator=g, device="cuda", dtype=torch.int32)
    if own:
        import sparse_attention_decode_indexer_gb300 as ssa
        st["beams"] = ssa.BeamState(G, K, max_len=h, finished=c["eos"])
        st["next"] = ssa.BeamState(G, K, max_len=h, finished=c["eos"])
        for name in ("scores", "finished", "history", "hist_len"):
            t = getattr(st["beams"], name)
            if t is not None:
                t.copy_(st[name])
        for name in ("parent", "token", "new_lens"):
            st[name] = torch.empty((B,), dtype=torch.int32, device="cuda")
        st["status"] = torch.zeros((1,), dtype=torch.int32, device="cuda")
        st["ws"] = torch.zeros((ssa.ssa_beam_workspace_size(G, K),), dtype=torch.uint8, device="cuda")
    return st


def prepare(case, seed):
    st = {"prompt": _prepare_prompt, "norm": _prepare_norm, "beam": _prepare_beam}[case["op"]](case, seed)
    st["case"] = case
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_prompt(st):
    c = st["case"]
    Hq, H = c["Hq"], c["Hkv"]
    G = Hq // H
    out, lse, q0, k0 = [], [], 0, 0
    for lq, lk in zip(st["lq"], st["lk"]):
        q, k, v = st["q"][q0:q0 + lq].float(), st["k"][k0:k0 + lk].float(), st["v"][k0:k0 + lk].float()
        q0, k0 = q0 + lq, k0 + lk
        k, v = k.permute(1, 2, 0)[:, None], v.transpose(0, 1)[:, None]        # [H][1][D][lk], [H][1][lk][D]
        step = max(1, (1 << 28) // (Hq * max(lk, 1)))
        for a in range(0, lq, step):
            b = min(a + step, lq)
            n = b + lk - lq if c["causal"] else lk                            # keys that these rows see
            s = q[a:b].view(b - a, H, G, D).permute(1, 2, 0, 3) @ k[..., :n] * (1.0 / math.sqrt(D))
            if c["causal"]:
                i = torch.arange(a, b, device="cuda")[:, None] + (lk - lq)
                s = s.masked_fill(torch.arange(n, device="cuda") > i, -math.inf)
            m = s.amax(-1, keepdim=True)
            e = (s - m).exp()
            z = e.sum(-1, keepdim=True)
            o = (e / z) @ v[:, :, :n]                                          # [H][G][rows][D]
            out.append(o.permute(2, 0, 1, 3).reshape(b - a, Hq, D).to(st["q"].dtype))
            lse.append((m + z.log())[..., 0].permute(2, 0, 1).reshape(b - a, Hq))
    return [torch.cat(out), torch.cat(lse)]


def _plain_norm(st):
    c = st["case"]
    ang = st["pos"].double()[:, None] * st["theta"]            # [T][rd/2], 64 bits: far positions
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + st["eps"]) * w[:, None, None]
        yr, rest = y[..., :c["rd"]], y[..., c["rd"]:]
        a, b = (yr[..., 0::2], yr[..., 1::2]) if c["inter"] else yr.chunk(2, -1)
        ra, rb = a * cos - b * sin, b * cos + a * sin
        z = torch.stack((ra, rb), -1).flatten(-2) if c["inter"] else torch.cat((ra, rb), -1)
        return torch.cat((z, rest), -1).to(x.dtype)
    return [one(st["q"], st["wq"]), one(st["k"], st["wk"])]


def _beam_outputs(st, row, token, score):
    """What follows from the chosen (row of the batch, token): states reordered."""
    c = st["case"]
    res = dict(parent=row, token=token, scores=score, new_lens=st["seq_lens"][row.long()] + 1)
    if c["eos"]:
        res["finished"] = st["finished"][row.long()] | (token == st["eos"]).to(torch.uint8)
    if c["hist"]:
        at = torch.arange(c["hist"], device="cuda")
        n = st["hist_len"].repeat_interleave(c["beams"])[:, None]
        h = torch.where(at < n, st["history"][row.long()], 0)
        res["history"] = torch.where(at == n, token[:, None], h)
        res["hist_len"] = st["hist_len"] + 1
    return res


def _plain_beam(st):
    c = st["case"]
    G, K, V = c["groups"], c["beams"], c["V"]
    # 64 bits: scores of different beams that lie next to one another
    x = st["logits"].double()
    m = x.amax(-1, keepdim=True)
    cand = x - (m + (x - m).exp().sum(-1, keepdim=True).log()) + st["scores"].double()[:, None]
    if c["eos"]:       # a beam that has ended goes on as it is
        ended = st["finished"].bool()[:, None]
        stay = torch.arange(V, device="cuda") == st["eos"]
        cand = torch.where(ended, torch.where(stay, st["scores"].double()[:, None], -math.inf), cand)
    cand = cand.view(G, K * V)
    val, idx = cand.sort(dim=-1, descending=True, stable=True)       # ties: the lowest beam, then token
    val, idx = val[:, :K], idx[:, :K]
    row = (idx // V + torch.arange(G, device="cuda")[:, None] * K).flatten().int()
    return _beam_outputs(st, row, (idx % V).flatten().int(), val.flatten().float())


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    st, c = state, state["case"]
    if not own:
        return {"prompt": _plain_prompt, "norm": _plain_norm, "beam": _plain_beam}[c["op"]](st)
    import sparse_attention_decode_indexer_gb300 as ssa
    if c["op"] == "prompt":
        ssa.ssa_prompt_attention(st["q"], st["k"], st["v"], st["cu_q"], st["out"], st["status"], st["ws"],
                                 cu_k=st["cu_k"], causal=c["causal"], lse=st["lse"])
        return [st["out"], st["lse"]]
    if c["op"] == "norm":
        ssa.ssa_norm_rope(st["plan"], st["norm"], st["pos"], st["q"], st["k"], q_out=st["q_out"],
                          k_out=st["k_out"])
        return [st["q_out"], st["k_out"]]
    new = st["next"]
    ssa.ssa_beam_select(st["logits"], st["beams"], st["parent"], st["token"], st["status"], st["ws"],
                        out=new, eos=st["eos"], seq_lens=st["seq_lens"], new_lens=st["new_lens"])
    res = dict(parent=st["parent"], token=st["token"], scores=new.scores, new_lens=st["new_lens"])
    if c["eos"]:
        res["finished"] = new.finished
    if c["hist"]:
        res["history"], res["hist_len"] = new.history, new.hist_len
    return res


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_prompt(c, st):
    if _pairs(c) * c["Hq"] > 6e9:       # 64-bit products at about 1 TFLOP/s
        return None
    group = c["Hq"] // c["Hkv"]
    out = torch.zeros((sum(st["lq"]), c["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(st["lq"]), c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    q_end = k_end = 0
    for n_q, n_k in zip(st["lq"], st["lk"]):
        q_end, k_end = q_end + n_q, k_end + n_k
        for h in range(c["Hq"]):
            key = st["k"][k_end - n_k:k_end, h // group].double()
            val = st["v"][k_end - n_k:k_end, h // group].double()
            # rows in pieces counted from the sequence's end, where the last row sees every key
            for hi in range(n_q, 0, -2048):
                lo = max(0, hi - 2048)
                sees = n_k - (n_q - hi) if c["causal"] else n_k
                w = torch.einsum("id,jd->ij", st["q"][q_end - n_q + lo:q_end - n_q + hi, h].double(), key[:sees])
                w /= math.sqrt(D)
                if c["causal"]:
                    w += torch.full_like(w, -math.inf).triu(sees - (hi - lo) + 1)
                lse[q_end - n_q + lo:q_end - n_q + hi, h] = torch.logsumexp(w, -1)
                out[q_end - n_q + lo:q_end - n_q + hi, h] = torch.softmax(w, -1) @ val[:sees]
    return [out, lse]


def _exact_norm(c, st):
    # a pair as a complex number, turned by the unit number of its angle
    ang = torch.outer(st["pos"].double(), st["theta"])
    turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]
    i = torch.arange(c["rd"] // 2, device="cuda")
    lo, hi = (2 * i, 2 * i + 1) if c["inter"] else (i, i + c["rd"] // 2)
    outs = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        y = x.double()
        size = torch.linalg.vector_norm(y, dim=-1, keepdim=True)
        y = y * w.double()[:, None, None] / (size * size / c["D"] + st["eps"]).sqrt()
        z = torch.complex(y[..., lo], y[..., hi]) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        outs.append(y)
    return outs


def _exact_beam(c, st):
    G, K, V = c["groups"], c["beams"], c["V"]
    row, token, score = [], [], []
    for g in range(G):
        first = g * K
        cand = torch.log_softmax(st["logits"][first:first + K].double(), -1)
        cand += st["scores"][first:first + K, None].double()
        for b in range(K):
            if c["eos"] and st["finished"][first + b]:
                cand[b] = -math.inf
                cand[b, st["eos"]] = st["scores"][first + b].double()
        flat = cand.flatten()
        for _ in range(K):          # the best that is left, the first of equals
            best = flat.max()
            j = int((flat == best).nonzero()[0])
            row.append(first + j // V)
            token.append(j % V)
            score.append(best.clone())
            flat[j] = -math.inf
    i32 = dict(dtype=torch.int32, device="cuda")
    res = _beam_outputs(st, torch.tensor(row, **i32), torch.tensor(token, **i32), torch.stack(score))
    # whole numbers: compared as they are
    return {name: t if name == "scores" else None for name, t in res.items()}


def exact(case, seed):
    st = prepare(case, seed)
    return {"prompt": _exact_prompt, "norm": _exact_norm, "beam": _exact_beam}[case["op"]](case, st)
