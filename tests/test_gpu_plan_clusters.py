"""Eviction plans of clusters, some of whose lists have nothing to drop."""
import pytest

from tests.test_gpu_slots import i32, ops_for, plan_on_device, some_slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_diffusion_drafter_context_gb300.build import build
    build()


@pytest.mark.parametrize("cap,budget,spare", [(20001, 9000, 0), (20001, 19997, 3), (70000, 35000, 1), (120000, 100, 7)])
def test_lists_with_and_without_something_to_drop(cap, budget, spare):
    """Requests above the budget, at it, below it and empty, in one call; the
    moves of the last three, and what lies behind a list's count, are -1.  The
    room for moves ends anywhere among a cluster's threads."""
    import torch
    from block_diffusion_drafter_context_gb300 import binding as B
    nkv = 2
    s = some_slots(1, 4, nkv, cap, budget, 5, "any")
    ctx = i32([cap, budget, budget // 2, 0])
    ops = ops_for(nkv)
    top = min(budget, cap - budget) + spare
    moves = torch.full((1, 4, nkv, 2, top), 77, dtype=torch.int32, device="cuda")
    counts, left = torch.full((1, 4, nkv), 77, dtype=torch.int32, device="cuda"), torch.full_like(ctx, 77)
    into, source = plan_on_device(s, ctx, ctx + 10, 0, 0, budget)
    for _ in range(5):
        moves.fill_(77)
        B.dflash_plan_eviction(ops.heads, s.struct, layer=0, n_layers=1, ctx_len=ctx, seq_len=ctx + 10, batch=4, first=0,
                               recent=0, budget=budget, moves=moves, top=top, counts=counts, ctx_out=left,
                               workspace=ops.workspace, workspace_bytes=ops.ws_bytes)
        assert ops.status() == 0
        got = torch.where(moves >= 0, moves, cap)
        n = min(top, cap)
        assert torch.equal(got[..., 0, :n].long(), into[..., :n]) and torch.equal(got[..., 1, :n].long(), source[..., :n])
        assert (moves[:, 1:] == -1).all() and left.tolist() == [budget, budget, budget // 2, 0]
        assert torch.equal(counts.long(), (source < cap).sum(-1)) and not counts[:, 1:].any()
