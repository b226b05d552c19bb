"""Views of a fused projection as the store's input: the runner stores what they name, the call itself takes
contiguous tensors and refuses others."""
import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa

L, T, H, D, P = 2, 21, 2, 128, 16


def _layout(fmt):
    return ssa.Layout(P, 4, H, D, fmt != "bf16", L, 3, 3, 1, 3, 1, kv_format=fmt)


@pytest.mark.parametrize("fmt", ["bf16", "int8_page_head"])
def test_the_call_refuses_what_it_would_misread(fmt):
    c = ssa.KVCache(_layout(fmt), False, device="cpu")
    x = torch.zeros((L, T, H, D), dtype=torch.bfloat16)
    pos, status = torch.arange(T), torch.zeros((1,), dtype=torch.int32)
    wide = torch.zeros((L, T, 3 * H, D), dtype=torch.bfloat16)
    for k, v, at in ((wide[:, :, :H], x, pos), (x, wide[:, :, H:2 * H], pos), (x.float(), x, pos),
                     (x, x.half(), pos), (x[:, :-1].contiguous(), x, pos), (x, x[:1], pos),
                     (x, x, pos.int()), (x, x, torch.arange(2 * T)[::2])):
        with pytest.raises(ValueError):
            ssa.ssa_store_kv_mirror(c, 0, L, k, v, at, status)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8_page_head", "e4m3_page_head"])
@pytest.mark.parametrize("rope", [False, True])
def test_a_runner_stores_views(fmt, rope):
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    plan = ssa.RopePlan(D, 64) if rope else None
    qkv = torch.randn((L, T, 3 * H, D), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    k, v = qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
    pos = torch.arange(T, device="cuda")
    runs = []
    for kk, vv in ((k, v), (k.contiguous(), v.contiguous())):
        run = DecodeRunner(_layout(fmt), host_tier=False, identity=True, block_table=torch.arange(3)[None],
                           seq_lens=torch.tensor([T]), rope=plan)
        run.store(0, L, kk, vv, pos, positions=pos if rope else None)
        runs.append(run.cache)
    a, b = runs
    assert bool(a.v_pool.any())
    for n in ("k_pool", "v_pool", "k_scale", "v_scale", "slab", "slab_sum", "slab_cnt"):
        if getattr(a, n) is not None:
            assert torch.equal(getattr(a, n), getattr(b, n)), n


@pytest.mark.gpu
def test_bits_of_another_type_are_the_same_input():
    k, v = (torch.randn((L, T, H, D), generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in (1, 2))
    pos = torch.arange(T, device="cuda")
    caches = []
    for bits in (torch.bfloat16, torch.int16, torch.uint8, torch.int32):
        c, status = ssa.KVCache(_layout("int8_page_head"), False), torch.zeros((1,), dtype=torch.int32, device="cuda")
        ssa.ssa_lru_init(c, True)
        ssa.ssa_store_kv_mirror(c, 0, L, k.view(bits), v.view(bits), pos, status)
        assert int(status.item()) == 0
        caches.append(c)
    for c in caches[1:]:
        assert torch.equal(c.k_pool, caches[0].k_pool) and torch.equal(c.v_pool, caches[0].v_pool)
