"""What a runner's calls do about a preload that still runs on its own stream: they write slots and slot
tables that it reads and writes, so they wait for it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _runner(width=4):
    import sparse_attention_decode_indexer_gb300 as ssa
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    P, n, B = 16, 6, 2
    lay = ssa.Layout(P, 2, 2, 128, True, 1, B * n, B * n, B, n, 2, kv_format="int8_page_head")
    run = DecodeRunner(lay, host_tier=True, identity=False, block_table=torch.arange(B * n).view(B, n),
                       seq_lens=torch.tensor([n * P - 1, 3 * P]), preload_width=width)
    x = torch.randn((1, 2 * P, 2, 128), device="cuda").bfloat16()
    run.store(0, 1, x, x, torch.arange(2 * P, device="cuda"))
    return run, torch.randn((1, B, 2, 128), device="cuda").bfloat16(), x


@pytest.mark.parametrize("call", ["store", "fork", "compact", "off"])
def test_calls_wait_for_the_preload(call):
    run, q, x = _runner()
    run.table, run.step(q)
    last = torch.tensor([95], device="cuda")
    torch.cuda.synchronize()
    # a preload that takes its time: some 10 ms of clock ticks before it writes
    flag = torch.zeros((1,), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(run.side):
        torch.cuda._sleep(20_000_000)
        flag.fill_(1)
        run.ev_preload.record(run.side)
    if call == "store":
        run.store(0, 1, x[:, :1], x[:, :1], last)
    elif call == "fork":
        run.fork(torch.arange(2, dtype=torch.int32, device="cuda"))
    elif call == "compact":
        run.compact()
    else:
        run.enable_preload(0)
    seen = flag.clone()
    torch.cuda.synchronize()
    assert float(seen) == 1.0 and int(run.status.item()) == 0


def test_captures_beside_a_preload():
    run, q, x = _runner()
    run.table, run.step(q)
    last = torch.tensor([95], device="cuda")
    parent, y = torch.arange(2, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y.add_(1)
        for f in (lambda: run.fork(parent), run.compact):
            with pytest.raises(RuntimeError, match="preload"):
                f()
    g.replay()
    assert y.tolist() == [1, 1, 1, 1]            # the capture went on
    run.enable_preload(0)
    torch.cuda.synchronize()
    with torch.cuda.graph(g2 := torch.cuda.CUDAGraph()):
        run.fork(parent)
        run.store(0, 1, x[:, :1], x[:, :1], last)
    g2.replay()
    torch.cuda.synchronize()
    assert int(run.status.item()) == 0 and int(run.cache.slab_cnt[0, 5]) == 1
