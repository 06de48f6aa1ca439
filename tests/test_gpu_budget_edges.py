"""Edges of the shared prefix and the cache with a budget on the GPU: how many
keys share the wanted one's leading bits, pools past 2^32 elements, the wrappers
under their C names, other streams."""
import numpy as np
import pytest

from block_diffusion_drafter_context_gb300 import binding as B
from tests.test_gpu_shared import Shared
from tests.test_gpu_slots import Weighed, i32, np32, ops_for, plan_on_device, some_slots
from tests.test_gpu_target import PAGE, U, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_diffusion_drafter_context_gb300.build import build
    build()


@pytest.mark.parametrize("nkv,batch,cap", [
    (2, 2, 4500),        # a CTA per list, few threads
    (8, 12, 9000),       # a CTA of many threads per list
    (1, 2, 20000)])      # clusters
@pytest.mark.parametrize("near", [1, 2, 31, 255, 256, 257, 1024, 2047, 2048, 2049, 4000])
@pytest.mark.parametrize("ties", [False, True])
def test_plan_with_keys_that_lie_close(nkv, batch, cap, near, ties):
    """`near` weights between 1 and 1.25, whose leading bits are alike, some
    heavier ones, the rest lighter; the last that stays is the first, a middle
    one or the last of the near ones."""
    import torch
    from block_diffusion_drafter_context_gb300.target import SlotWeights
    g = torch.Generator("cuda").manual_seed(near + cap)
    heavy, ops = 170, ops_for(nkv)
    shape = (1, batch, nkv, cap)
    order = torch.rand(shape, generator=g, device="cuda").argsort(-1)
    close = 1 + torch.rand(shape, generator=g, device="cuda") / 4
    if ties:
        close = 1 + torch.randint(0, 3, shape, generator=g, device="cuda").float() / 16
    else:
        close = close.clamp(max=1.2499)
    w = torch.where(order < heavy, 4 + close, torch.where(order < heavy + near, close, 0.01 * close))
    s = SlotWeights.from_tensors(w, torch.zeros(shape, dtype=torch.int32, device="cuda"))
    ctx = i32([cap - 3 * b for b in range(batch)])
    lost = 3 * batch        # of the heavy and the near ones, behind a request's end
    for keep in sorted({heavy + 1, heavy + (near + 1) // 2, max(heavy + 1, heavy + near - lost), heavy + near}):
        moves, counts, left = ops.plan_eviction(s, ctx, ctx + 10, keep)
        into, source = plan_on_device(s, ctx, ctx + 10, 0, 0, keep)
        top = moves.shape[-1]
        got = torch.where(moves >= 0, moves, cap)
        assert torch.equal(got[..., 0, :].long(), into[..., :top]) and torch.equal(got[..., 1, :].long(), source[..., :top])
        assert torch.equal(counts.long(), (source < cap).sum(-1)) and torch.equal(left, ctx.clamp(max=keep))
    assert ops.status() == 0


@pytest.mark.parametrize("kind", ["any", "ties", "zeros", "same"])
@pytest.mark.parametrize("B,nkv,cap,budget,recent,first", [
    (20, 8, 45000, 40000, 100, 5),       # a CTA per list, more than 1024 slots for each of its warps
    (1, 2, 300001, 150000, 3000, 0),     # the same in clusters
    (1, 2, 49153, 20000, 0, 64),         # clusters of two or more by length
    (2, 2, 1500, 900, 0, 0), (2, 1, 3000, 2500, 7, 1), (1, 1, 2048, 1, 0, 0)])   # 8 and 16 slots to a lane
def test_plan_of_every_stretch(kind, B, nkv, cap, budget, recent, first):
    import torch
    s = some_slots(1, B, nkv, cap, budget, 11, kind)
    ctx = i32([cap - 13 * b for b in range(B)])
    ops = ops_for(nkv)
    moves, counts, left = ops.plan_eviction(s, ctx, ctx + 10, budget, recent=recent, first=first)
    into, source = plan_on_device(s, ctx, ctx + 10, first, recent, budget)
    top = moves.shape[-1]
    got = torch.where(moves >= 0, moves, cap)
    assert torch.equal(got[..., 0, :].long(), into[..., :top]) and torch.equal(got[..., 1, :].long(), source[..., :top])
    assert torch.equal(counts.long(), (source < cap).sum(-1)) and torch.equal(left, ctx.clamp(max=budget))
    assert ops.status() == 0


@pytest.mark.parametrize("nq,nkv,d,ctx,new,launches", [
    (2, 2, 64, [40, 3, 0, 70], [1, 1, 1, 1], 1), (8, 2, 128, [9, 300], [3, 1], 1), (8, 1, 64, [0, 1], [1, 1], 2),
    (12, 4, 128, [5], [5], 2)])
def test_few_rows_have_exact_probabilities(nq, nkv, d, ctx, new, launches):
    """bf16, up to 16 rows per kv head: P as two bf16 parts, each off by half a
    step, 2^-8 of 2^-8.  The other terms as in Shared.check."""
    c = Shared(nq, nkv, d, "bf16", 5, ctx, new, seed=d + nq)
    B.dflash_debug_shared_launches(launches)
    try:
        out = np64(c.attend()[0])
    finally:
        B.dflash_debug_shared_launches(0)
    ref, _, spread = c.attend_ref()
    size = np.abs(np64(c.q)).reshape(c.T, nq, d).sum(-1).max() * np.nanmax(np.abs(np64(c.k[1]))) * d ** -0.5
    e = 2 * d * 2.0 ** -24 * size + max(a + b for a, b in zip(c.ctx, c.new)) * 2.0 ** -24 + 2.0 ** -19
    assert c.ops.status() == 0
    assert (np.abs(out - ref) <= (2.0 ** -16 + e) * spread + U["bf16"] * np.abs(ref) + 1e-30).all()


def far(c, pages, used):
    """The batch's second layer on the last pages of a large pool."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    assert 2 * pages * c.nkv * PAGE * c.d > 2 ** 32
    k = torch.empty(2, pages, c.nkv, PAGE, c.d, dtype=c.dt, device="cuda")
    v = torch.empty(2, pages, c.nkv, c.d, PAGE, dtype=c.dt, device="cuda")
    k[1, -used:], v[1, -used:] = c.k[1], c.v[1]
    table = torch.from_numpy(np.where(c.table >= 0, c.table + pages - used, -1).astype(np.int32)).cuda()
    return k, v, PagedKV.from_tensors(k, v, table)


@pytest.mark.parametrize("nq,nkv,d,dtype,pages", [(16, 8, 128, "bf16", 33500), (40, 8, 128, "bf16", 33500),
                                                  (64, 16, 64, "bf16", 33500), (8, 4, 128, "f32", 66000)])
def test_pages_past_32_bits_of_elements(nq, nkv, d, dtype, pages):
    import torch
    shared = Shared(nq, nkv, d, dtype, 3, [300, 65, 0], [5, 1, 16], seed=d, stale=0.0)
    kv = far(shared, pages, shared.k.shape[1])[2]
    for launches in (1, 2):
        B.dflash_debug_shared_launches(launches)
        try:
            out, lse = shared.attend()
            out2, lse2 = shared.ops.attend_shared(kv, 1, shared.q, shared.cu_d, shared.ctx_d, shared.prefix, want_lse=True)
        finally:
            B.dflash_debug_shared_launches(0)
        assert shared.ops.status() == 0 and torch.equal(out2, out) and torch.equal(lse2, lse)
    del kv
    c = Weighed(nq, nkv, d, dtype, [300, 65, 0], [5, 1, 16], seed=d, stale=0.0, commit=[3, 1, 16], first=2)
    used = c.k.shape[1]
    k, v, kv = far(c, pages, used)
    c.add()
    want = c.slots.weights.clone()
    left = c.ops.evict(c.kv, c.slots, c.ctx_d + i32(c.commit), c.ctx_d + i32(c.commit), 60, recent=7, first=2, layer=1)
    after, positions = c.slots.weights.clone(), c.slots.positions.clone()
    c.reset()
    c.ops.add_weights(kv, 1, c.slots, c.q, c.lse, c.cu_d, c.ctx_d, n_commit=c.commit_d, first=2)
    assert torch.equal(c.slots.weights, want)
    assert torch.equal(c.ops.evict(kv, c.slots, c.ctx_d + c.commit_d, c.ctx_d + c.commit_d, 60, recent=7, first=2, layer=1), left)
    assert torch.equal(c.slots.weights, after) and torch.equal(c.slots.positions, positions)
    assert not torch.equal(after, want) and c.ops.status() == 0
    assert torch.equal(k[1, -used:], c.k[1]) and torch.equal(v[1, -used:], c.v[1])


@pytest.mark.parametrize("nq,nkv,d,dtype", [(8, 2, 128, "bf16"), (4, 2, 64, "f32")])
def test_the_wrappers_give_what_the_objects_give(nq, nkv, d, dtype):
    """Named by their C arguments, on torch's current stream and on another."""
    import torch
    c = Shared(nq, nkv, d, dtype, 2, [70, 3, 100], [5, 1, 9], seed=1, stale=0.0)
    s = some_slots(2, 3, nkv, c.table.shape[1] * PAGE, 160, 5, "any")
    commit, budget = i32([4, 1, 0]), 160
    seq = c.ctx_d + 1000
    k0, v0, w0, p0 = c.k.clone(), c.v.clone(), s.weights.clone(), s.positions.clone()
    state = [c.k, c.v, s.weights, s.positions]

    def reset():
        for x, y in zip(state, [k0, v0, w0, p0]):
            x.copy_(y)
        torch.cuda.synchronize()

    def objects(stream):
        q = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k, pos=seq, stream=stream)
        out, lse = c.ops.attend_shared(c.kv, 1, q, c.cu_d, c.ctx_d, c.prefix, scale=0.07, want_lse=True, stream=stream)
        c.ops.add_weights(c.kv, 1, s, q, lse, c.cu_d, c.ctx_d, pos=seq, n_commit=commit, first=c.prefix, scale=0.07,
                          stream=stream)
        got = c.ops.plan_eviction(s, now, seq + commit, budget, recent=20, first=c.prefix, layer=1, stream=stream)
        assert c.ops.evict(c.kv, s, now, seq + commit, budget, recent=20, first=c.prefix, layer=1,
                           stream=stream) is not None
        torch.cuda.synchronize()
        return [q, out, lse, *got] + [x.clone() for x in state]

    now = c.ctx_d + commit
    want = objects(None)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        reset()
        assert all(torch.equal(a, b) for a, b in zip(objects(stream), want))
    later, heads = seq + commit, c.ops.heads
    for stream in (None, side, side.cuda_stream):
        reset()
        q, out, lse, moves, counts, left = (torch.zeros_like(x) for x in want[:6])
        torch.cuda.synchronize()
        ws = dict(workspace=c.ops.workspace, workspace_bytes=c.ops.ws_bytes, stream=stream)
        batch = dict(cu_new=c.cu_d, total_new=c.T, ctx_len=c.ctx_d, batch=3)
        B.dflash_append_kv_at(heads, c.kv.struct, layer=1, qkv=c.qkv, row_stride=c.qkv.stride(0), g_q=c.g_q, g_k=c.g_k,
                              eps=1e-6, rope_base=1e6, pos=seq, q_out=q, **batch, **ws)
        B.dflash_shared_attention(heads, c.kv.struct, layer=1, q=q, q_stride=nq * d, max_new=16, shared_len=c.prefix,
                                  scale=0.07, out=out, lse=lse, rows=c.ops.rows, rows_bytes=c.ops.rows_bytes, **batch, **ws)
        B.dflash_add_weights(heads, c.kv.struct, s.struct, layer=1, q=q, q_stride=nq * d, lse=lse, pos=seq, n_commit=commit,
                             max_new=16, first=c.prefix, scale=0.07, **batch, **ws)
        B.dflash_plan_eviction(heads, s.struct, layer=1, n_layers=1, ctx_len=now, seq_len=later, batch=3, first=c.prefix,
                               recent=20, budget=budget, moves=moves, top=moves.shape[-1], counts=counts, ctx_out=left, **ws)
        B.dflash_move_slots(heads, c.kv.struct, s.struct, layer=1, n_layers=1, moves=moves, top=moves.shape[-1],
                            counts=counts, batch=3, **ws)
        torch.cuda.synchronize()
        assert c.ops.status() == 0
        for got, ref in zip([q, out, lse, moves, counts, left] + state, want):
            assert torch.equal(got, ref)
    assert np32(want[4]).any()
