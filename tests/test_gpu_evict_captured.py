"""Choice and moves of an eviction in a captured call."""
import pytest

from tests.test_gpu_slots import PAGE, i32, ops_for, some_slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_diffusion_drafter_context_gb300.build import build
    build()


@pytest.mark.parametrize("d,dtype,cap,budget", [(64, "bf16", 640, 500), (128, "f32", 1024, 100)])
def test_replays_are_eager_calls(d, dtype, cap, budget):
    """evict, and move_slots alone, captured once and replayed on other weights
    and lengths: K, V, weights, positions and lengths as of eager calls."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    L, B, nkv = 2, 3, 2
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pages = cap // PAGE
    k = torch.randn(L, B * pages, nkv, PAGE, d, device="cuda").to(dt)
    v = torch.randn(L, B * pages, nkv, d, PAGE, device="cuda").to(dt)
    kv = PagedKV.from_tensors(k, v, torch.randperm(B * pages, device="cuda").to(torch.int32).view(B, pages))
    ops = ops_for(nkv, d, dtype)
    s = some_slots(L, B, nkv, cap, budget, 1, "any")
    ctx, seq = i32([cap, budget + 1, budget]), i32([cap + 10, budget + 11, budget + 10])
    state = [k, v, s.weights, s.positions]
    first = [x.clone() for x in state]
    moves, counts, _ = ops.plan_eviction(s, ctx, seq, budget, recent=9, first=3)
    ops.move_slots(kv, s, moves, counts)
    torch.cuda.synchronize()
    both, alone = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(both):
        left = ops.evict(kv, s, ctx, seq, budget, recent=9, first=3)
    with torch.cuda.graph(alone):
        ops.move_slots(kv, s, moves, counts)
    for seed, lens in ((2, [cap, budget + 1, budget]), (3, [budget - 1, cap - 70, cap - 1])):
        other = some_slots(L, B, nkv, cap, budget, seed, "any")
        begin = first[:2] + [other.weights, other.positions]

        def reset():
            for x, y in zip(state, begin):
                x.copy_(y)

        ctx.copy_(i32(lens))
        seq.copy_(ctx + 10)
        reset()
        moves_e, counts_e, want = ops.plan_eviction(s, ctx, seq, budget, recent=9, first=3)
        ops.move_slots(kv, s, moves_e, counts_e)
        ref = [x.clone() for x in state]
        assert any(not torch.equal(x, y) for x, y in zip(ref, begin))
        reset()
        both.replay()
        assert torch.equal(left, want) and all(torch.equal(x, y) for x, y in zip(state, ref))
        reset()
        moves.copy_(moves_e)
        counts.copy_(counts_e)
        alone.replay()
        assert all(torch.equal(x, y) for x, y in zip(state, ref))
    assert ops.status() == 0
