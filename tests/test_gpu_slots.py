"""The cache with a budget on the GPU: weights of the slots, the choice of what
stays, the moves, and steps that run them together, against the fp64 oracle."""
import numpy as np
import pytest

from oracle import target_oracle as O
from tests.test_gpu_target import PAGE, U, Batch, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_diffusion_drafter_context_gb300.build import build
    build()


def i32(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def np32(t):
    return t.cpu().numpy()


class Weighed(Batch):
    """A Batch (layer 1 of two) with slots of random weights and the lse of its
    attention."""

    def __init__(self, *a, commit=None, turn=None, first=0, **kw):
        import torch
        from block_diffusion_drafter_context_gb300.target import SlotWeights
        super().__init__(*a, **kw)
        B, cap = len(self.ctx), self.table.shape[1] * PAGE
        self.commit = list(self.new) if commit is None else commit
        self.turn = list(self.ctx) if turn is None else turn
        self.commit_d, self.turn_d = (None if x is None else i32(x) for x in (commit, turn))
        self.first = first
        g = torch.Generator("cuda").manual_seed(1)
        self.slots = SlotWeights.from_tensors(torch.rand(2, B, self.nkv, cap, generator=g, device="cuda") * 4,
                                              torch.arange(cap, dtype=torch.int32, device="cuda").expand(
                                                  2, B, self.nkv, cap).contiguous())
        self.w0, self.p0 = self.slots.weights.clone(), self.slots.positions.clone()
        self.lse = self.ops.attend(self.kv, 1, self.q, self.cu_d, self.ctx_d, want_lse=True)[1]
        self.ops.status()

    def add(self, **kw):
        a = dict(pos=self.turn_d, n_commit=self.commit_d, first=self.first)
        a.update(kw)
        q, lse = a.pop("q", self.q), a.pop("lse", self.lse)
        self.ops.add_weights(self.kv, 1, self.slots, q, lse, a.pop("cu", self.cu_d), a.pop("ctx", self.ctx_d), **a)

    def reset(self):
        self.slots.weights.copy_(self.w0)
        self.slots.positions.copy_(self.p0)

    def check(self, q=None, lse=None):
        """|w - ref| <= e added + 2^-23 |ref|, e the relative error of a row's
        exp: its score's fp32 sum of d products, 2 d 2^-24 sum |q k| scale (the
        tensor cores cut off instead of rounding), the arguments' roundings
        (|s| + |lse|) 2^-22, exp2 and the sum over rows 2^-20."""
        q, lse = np64(self.q if q is None else q), np64(self.lse if lse is None else lse)
        ref, pos, added = O.add_weights(np64(self.w0[1]), np32(self.p0[1]), np64(self.k[1]), self.table, q, lse, self.nq,
                                        self.nkv, self.d, self.cu, self.ctx, self.turn, self.commit, self.first,
                                        self.d ** -0.5)
        kmax = np.nanmax(np.abs(np64(self.k[1])))
        size = np.nanmax(np.abs(q[:self.T].reshape(self.T, self.nq, self.d)).sum(-1)) * kmax * self.d ** -0.5
        e = 2 * self.d * 2.0 ** -24 * size + 2 * size * 2.0 ** -22 + 2.0 ** -20
        got = np64(self.slots.weights[1])
        assert (np.abs(got - ref) <= e * added + 2.0 ** -23 * np.abs(ref)).all(), np.nanmax(np.abs(got - ref) / (e * added + 1e-30))
        assert np.array_equal(np32(self.slots.positions[1]), pos)
        # the other layer, and what nobody paid attention to
        assert np.array_equal(np32(self.slots.weights[0]), np32(self.w0[0]))
        assert np.array_equal(np32(self.slots.positions[0]), np32(self.p0[0]))
        for b in range(len(self.ctx)):
            for part in (slice(0, self.first), slice(self.ctx[b] + self.commit[b], None)):
                assert np.array_equal(got[b, :, part], np64(self.w0[1])[b, :, part])


SHAPES = [(8, 2, 128, "bf16"), (5, 1, 128, "bf16"), (16, 2, 64, "bf16"), (4, 4, 64, "bf16"), (4, 2, 64, "f32"),
          (6, 1, 128, "f32"), (2, 2, 128, "f32")]


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("nq,nkv,d,dtype", SHAPES)
@pytest.mark.parametrize("ctx,new,commit,turn,first", [
    ([0], [1], None, None, 0),                                                 # a single token, of itself alone
    ([0, 63, 64, 127, 190], [1, 1, 1, 1, 1], None, None, 0),                   # decode at page and pair borders
    ([70, 3, 200, 64], [16, 0, 5, 9], [3, 0, 5, 0], [500, 0, 200, 7], 0),       # verification, some or none committed
    ([150, 129, 10], [16, 16, 16], [16, 1, 7], None, 67),                      # from a slot inside a page; one behind all
])
def test_weights_match_oracle(nq, nkv, d, dtype, ctx, new, commit, turn, first):
    c = Weighed(nq, nkv, d, dtype, ctx, new, seed=nq + d, commit=commit, turn=turn, first=first, pad_rows=2)
    c.add()
    assert c.ops.status() == 0
    c.check()


@pytest.mark.parametrize("nq,nkv,d,dtype,batch,ctx,new", [
    (40, 8, 128, "bf16", 24, 3000, 16), (32, 8, 128, "bf16", 100, 700, 1), (16, 4, 64, "bf16", 9, 9000, 8),
    (4, 2, 64, "f32", 30, 1500, 5), (8, 8, 128, "f32", 3, 4000, 16), (8, 1, 128, "bf16", 200, 90, 3)])
def test_weights_over_a_full_gpu(nq, nkv, d, dtype, batch, ctx, new):
    """Runs that cross many requests and heads, against fp64 on the device, and
    three calls with the same bits.  Tolerances as in Weighed.check."""
    import torch
    lens = [ctx - ctx * b // (2 * batch) for b in range(batch)]
    news = [1 + (b * 3) % new for b in range(batch)]
    c = Weighed(nq, nkv, d, dtype, lens, news, seed=5, stale=0.0, commit=[(n + 1) // 2 for n in news], first=5)
    c.add()
    assert c.ops.status() == 0
    got = c.slots.weights.clone()
    for _ in range(2):
        c.reset()
        c.add()
        assert torch.equal(c.slots.weights, got)
    ref, added = c.w0[1].double(), torch.zeros_like(c.w0[1], dtype=torch.float64)
    table = torch.from_numpy(c.table).cuda()
    for b in range(batch):
        m, n = c.commit[b], lens[b] + c.commit[b]
        ref[b, :, lens[b]:n] = 0
        k = c.k[1, table[b, :-(-n // PAGE)].long()].double().transpose(0, 1).reshape(nkv, -1, d)[:, :n]
        rows = slice(int(c.cu[b]), int(c.cu[b]) + m)
        s = torch.einsum("ihgd,htd->higt", c.q[rows].double().view(m, nkv, -1, d), k) * d ** -0.5
        p = (s - c.lse[rows].double().view(m, nkv, -1).transpose(0, 1)[..., None]).exp()
        hide = torch.arange(n, device="cuda") > lens[b] + torch.arange(m, device="cuda")[:, None]
        added[b, :, 5:n] = p.masked_fill_(hide[None, :, None], 0).sum((1, 2))[:, 5:]
    ref += added
    size = float(c.q.double().abs().view(c.T, nq, d).sum(-1).max() * c.k[1].abs().max()) * d ** -0.5
    e = 2 * d * 2.0 ** -24 * size + 2 * size * 2.0 ** -22 + 2.0 ** -20
    assert ((got[1].double() - ref).abs() <= e * added + 2.0 ** -23 * ref.abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_of_rows_that_saw_nothing_and_of_nan_rows(dtype):
    import torch
    c = Weighed(4, 2, 64, dtype, [100, 20], [3, 2], seed=4)
    lse = c.lse.clone()
    lse[0, 1] = -float("inf")
    c.add(lse=lse)
    c.check(lse=lse)
    c.reset()
    lse[1, 0] = float("nan")
    c.add(lse=lse)
    got = c.slots.weights[1]
    assert torch.isnan(got[0, 0, :102]).all() and not torch.isnan(got[0, 0, 102:]).any()   # slot 102 is not seen by row 1
    assert not torch.isnan(got[0, 1]).any() and not torch.isnan(got[1]).any() and c.ops.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_with_missing_pages_and_invalid_requests(dtype):
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    c = Weighed(4, 1, 128, dtype, [300, 70, 130], [2, 3, 1], seed=6)
    c.table[0, 0], c.table[0, 3], c.table[2, 2] = -1, 10 ** 6, -5
    c.kv = PagedKV.from_tensors(c.k, c.v, torch.from_numpy(c.table).cuda())
    c.add()
    assert c.ops.status() == -7
    c.check()
    for kw in (dict(n_commit=i32([2, 4, 1])), dict(n_commit=i32([2, -1, 1])), dict(ctx=i32([300, -1, 130])),
               dict(ctx=i32([300, 10 ** 6, 130])), dict(max_new=2)):
        c.reset()
        c.add(**kw)
        assert c.ops.status() == -7
        got, pos = c.slots.weights.clone(), c.slots.positions.clone()
        assert torch.equal(got[1, 1], c.w0[1, 1]) and torch.equal(pos[1, 1], c.p0[1, 1])
        c.reset()
        c.add()
        c.ops.status()
        assert torch.equal(got[1, 0], c.slots.weights[1, 0]) and torch.equal(got[1, 2], c.slots.weights[1, 2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_of_a_slice_and_in_a_graph(dtype):
    """A part of a batch by slices, a captured call replayed with other
    queries, other streams: as the eager call on the same inputs."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    from block_diffusion_drafter_context_gb300.target import SlotWeights
    c = Weighed(8, 2, 64, dtype, [30, 400, 64, 100], [3, 16, 1, 5], seed=8)
    c.add()
    want, pos = c.slots.weights.clone(), c.slots.positions.clone()
    c.reset()
    table = torch.from_numpy(c.table).cuda()
    for lo, hi in ((0, 1), (1, 3), (3, 4)):
        part = SlotWeights.from_tensors(c.slots.weights[1:2, lo:hi].contiguous(), c.slots.positions[1:2, lo:hi].contiguous())
        kv = PagedKV.from_tensors(c.k[1:2], c.v[1:2], table[lo:hi].contiguous())
        c.ops.add_weights(kv, 0, part, c.q, c.lse, c.cu_d[lo:hi + 1].contiguous(), c.ctx_d[lo:hi].contiguous())
        assert torch.equal(part.weights[0], want[1, lo:hi]) and torch.equal(part.positions[0], pos[1, lo:hi])
    q = c.q.clone()
    c.add(q=q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.add(q=q)
    for x in (torch.randn_like(q), c.q):
        c.reset()
        c.add(q=x)
        eager = c.slots.weights.clone()
        c.reset()
        q.copy_(x)
        g.replay()
        assert torch.equal(c.slots.weights, eager)
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        c.reset()
        torch.cuda.synchronize()
        c.add(stream=s)
        side.synchronize()
        assert torch.equal(c.slots.weights, want)
    assert c.ops.status() == 0


# ------------------------------------------------------------------ choice
def some_slots(L, B, nkv, cap, budget, seed, kind):
    import torch
    from block_diffusion_drafter_context_gb300.target import SlotWeights
    g = torch.Generator("cuda").manual_seed(seed)
    w = torch.randn(L, B, nkv, cap, generator=g, device="cuda").mul_(2).exp_()
    if kind == "ties":
        w = torch.randint(0, 4, w.shape, generator=g, device="cuda").float() * 0.5
    elif kind == "zeros":
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.9] = 0
    elif kind == "odd":
        w = torch.randn(w.shape, generator=g, device="cuda")
        for value in (float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-44, 3.0):
            w[torch.rand(w.shape, generator=g, device="cuda") < 0.08] = value
    elif kind == "same":
        w.fill_(0.25)
    # the tokens of the slots below the budget in no order, the newest behind
    near = torch.rand(L, B, nkv, min(budget, cap), generator=g, device="cuda").argsort(-1)
    far = torch.arange(min(budget, cap), cap, device="cuda").expand(L, B, nkv, -1)
    return SlotWeights.from_tensors(w, (torch.cat([near, far], -1) + 10).to(torch.int32))


def ops_for(nkv, d=64, dtype="bf16", **kw):
    from block_diffusion_drafter_context_gb300.target import TargetOps
    return TargetOps(nkv, nkv, d, dtype=dtype, **kw)


@pytest.mark.parametrize("kind", ["any", "ties", "zeros", "odd", "same"])
@pytest.mark.parametrize("L,B,nkv,cap,budget,recent,first", [
    (1, 1, 1, 64, 1, 0, 0), (1, 1, 1, 2, 1, 1, 0), (2, 3, 2, 200, 130, 20, 4), (1, 4, 2, 333, 320, 0, 0),
    (3, 2, 1, 100, 99, 99, 0), (1, 2, 2, 1000, 300, 100, 200), (1, 2, 1, 5000, 4000, 100, 3999 - 100),
    (1, 1, 2, 20000, 7777, 500, 64), (1, 2, 1, 64, 64, 0, 0), (1, 2, 1, 64, 100, 0, 10)])
def test_plan_matches_oracle(kind, L, B, nkv, cap, budget, recent, first):
    s = some_slots(L, B, nkv, cap, budget, cap + first, kind)
    w0, p0 = s.weights.clone(), s.positions.clone()
    ctx = [max(0, cap - 7 * b * b) for b in range(B)]
    if B > 2:
        ctx[2] = budget + 1
    ops = ops_for(nkv)
    moves, counts, left = ops.plan_eviction(s, i32(ctx), i32([c + 10 for c in ctx]), budget, recent=recent, first=first)
    assert ops.status() == 0
    assert left.tolist() == [min(c, budget) for c in ctx]
    w, p, moves, counts = np32(s.weights), np32(s.positions), np32(moves), np32(counts)
    assert moves.shape[-1] == max(0, min(budget - first, cap - budget))
    for layer in range(L):
        for b in range(B):
            for h in range(nkv):
                ref = O.plan_eviction(w[layer, b, h], p[layer, b, h], ctx[b], ctx[b] + 10, first, recent, budget)
                n = counts[layer, b, h]
                assert n == len(ref)
                assert [tuple(m) for m in moves[layer, b, h, :, :n].T] == ref
                assert (moves[layer, b, h, :, n:] == -1).all()
    assert np.array_equal(np32(w0), w, equal_nan=True) and np.array_equal(np32(p0), p)


def plan_on_device(s, ctx, seq, first, recent, budget):
    """The kept slots and the moves by a stable sort (no NaN)."""
    import torch
    cap = s.capacity
    slot = torch.arange(cap, device="cuda")
    ctx_, seq_ = ctx.view(1, -1, 1, 1), seq.view(1, -1, 1, 1)
    free = (slot >= first) & (slot < ctx_)
    x = torch.where(free, torch.where(s.positions >= seq_ - recent, float("inf"), s.weights), -float("inf"))
    order = torch.sort(x, dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    kept = free & (rank < budget - first)
    over = ctx_ > budget
    into = torch.where(over & free & ~kept & (slot < budget), slot, cap).sort(-1)[0]
    source = torch.where(over & kept & (slot >= budget), slot, cap).sort(-1)[0]
    return into, source


@pytest.mark.parametrize("kind", ["any", "zeros"])
@pytest.mark.parametrize("L,B,nkv,cap,budget,recent,first", [
    (1, 1, 8, 131072, 65536, 4096, 0),        # clusters, all keys in shared memory
    (1, 64, 4, 60000, 30000, 100, 64),        # a CTA per list, more keys than it can hold
    (8, 16, 8, 4160, 4096, 256, 4),           # a step in every layer
    (1, 1, 1, 1000000, 600000, 1000, 0)])     # one list, more than a cluster can hold
def test_plan_of_long_lists(kind, L, B, nkv, cap, budget, recent, first):
    import torch
    s = some_slots(L, B, nkv, cap, budget, 3, kind)
    ctx = i32([cap - 11 * b for b in range(B)])
    ops = ops_for(nkv)
    moves, counts, left = ops.plan_eviction(s, ctx, ctx + 10, budget, recent=recent, first=first)
    into, source = plan_on_device(s, ctx, ctx + 10, first, recent, budget)
    top = moves.shape[-1]
    got = torch.where(moves >= 0, moves, cap)
    assert torch.equal(got[..., 0, :].long(), into[..., :top]) and torch.equal(got[..., 1, :].long(), source[..., :top])
    assert torch.equal(counts.long(), (source < cap).sum(-1)) and torch.equal(left, ctx.clamp(max=budget))
    assert ops.status() == 0


def test_plan_of_one_layer_bad_lengths_and_in_a_graph():
    import torch
    s = some_slots(3, 3, 2, 300, 200, 1, "any")
    ops = ops_for(2)
    ctx, seq = i32([300, 250, 201]), i32([310, 260, 211])
    every = ops.plan_eviction(s, ctx, seq, 200, recent=9, first=3)
    for layer in range(3):
        one = ops.plan_eviction(s, ctx, seq, 200, recent=9, first=3, layer=layer)
        assert torch.equal(one[0][0], every[0][layer]) and torch.equal(one[1][0], every[1][layer])
    assert ops.status() == 0
    moves, counts, left = ops.plan_eviction(s, i32([300, 301, -1]), seq, 200, recent=9, first=3)
    assert ops.status() == -7 and left.tolist() == [200, 301, -1]
    assert torch.equal(moves[:, 0], every[0][:, 0]) and (moves[:, 1:] == -1).all() and (counts[:, 1:] == 0).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = ops.plan_eviction(s, ctx, seq, 200, recent=9, first=3)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(again, every))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = ops.plan_eviction(s, ctx, seq, 200, recent=9, first=3, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, every))


# ------------------------------------------------------------------ moves
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "f32"), (128, "f32")])
@pytest.mark.parametrize("L,B,nkv,cap,budget,first", [(1, 1, 1, 128, 64, 0), (2, 3, 2, 640, 500, 7), (1, 2, 3, 1024, 100, 64),
                                                      (3, 1, 1, 192, 130, 128)])
def test_moves_match_numpy(d, dtype, L, B, nkv, cap, budget, first):
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    s = some_slots(L, B, nkv, cap, budget, 7, "any")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pages = cap // PAGE
    ids = np.random.default_rng(d).permutation(B * pages + 2)[:B * pages].reshape(B, pages).astype(np.int32)
    k = torch.randn(L, B * pages + 2, nkv, PAGE, d, device="cuda").to(dt)
    v = torch.randn(L, B * pages + 2, nkv, d, PAGE, device="cuda").to(dt)
    kv = PagedKV.from_tensors(k, v, torch.from_numpy(ids).cuda())
    ops = ops_for(nkv, d, dtype)
    ctx = [cap - 5 * b for b in range(B)]
    recent = min(3, budget - first)      # more would be refused
    moves, counts, _ = ops.plan_eviction(s, i32(ctx), i32([c + 10 for c in ctx]), budget, recent=recent, first=first)
    want = [np64(k).copy(), np64(v).copy(), np32(s.weights).copy(), np32(s.positions).copy()]
    for layer in range(L):
        for b in range(B):
            for h in range(nkv):
                for i in range(int(counts[layer, b, h])):
                    to, of = (int(x) for x in moves[layer, b, h, :, i])
                    p0, p1 = ids[b, to // PAGE], ids[b, of // PAGE]
                    want[0][layer, p0, h, to % PAGE] = want[0][layer, p1, h, of % PAGE]
                    want[1][layer, p0, h, :, to % PAGE] = want[1][layer, p1, h, :, of % PAGE]
                    want[2][layer, b, h, to], want[3][layer, b, h, to] = want[2][layer, b, h, of], want[3][layer, b, h, of]
    state = [k, v, s.weights, s.positions]
    before = [x.clone() for x in state]

    def same():
        assert ops.status() == 0
        assert np.array_equal(np64(k), want[0]) and np.array_equal(np64(v), want[1])
        assert np.array_equal(np32(s.weights), want[2]) and np.array_equal(np32(s.positions), want[3])
        for x, y in zip(state, before):
            x.copy_(y)

    ops.move_slots(kv, s, moves, counts)
    same()
    for layer in range(L):       # layer by layer
        ops.move_slots(kv, s, moves[layer:layer + 1], counts[layer:layer + 1], layer=layer)
    same()
    assert ops.evict(kv, s, i32(ctx), i32([c + 10 for c in ctx]), budget, recent=recent, first=first).tolist() == \
        [min(c, budget) for c in ctx]
    same()


def test_bad_moves_are_dropped():
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    k = torch.randn(1, 4, 1, PAGE, 64, device="cuda").bfloat16()
    v = torch.randn(1, 4, 1, 64, PAGE, device="cuda").bfloat16()
    table = i32([[0, 1, 9], [2, 3, -1]])
    kv = PagedKV.from_tensors(k, v, table)
    s = some_slots(1, 2, 1, 192, 100, 1, "any")
    ops = ops_for(1)
    k0, w0 = k.clone(), s.weights.clone()
    # into a missing page, from one, outside the cache, below 0; one good move among them
    moves = torch.stack([i32([[130, 5, 1, 7, -1, 3], [1, 2, 3, 4, 5, 6]]),
                         i32([[70, 140, 192, 1 << 24, 66, 65], [71, 72, 73, 74, 75, 76]])], 1).view(1, 2, 1, 2, 6)
    ops.move_slots(kv, s, moves, i32([[[6], [7]]]))
    assert ops.status() == -7
    k0[0, 0, 0, 3] = k0[0, 1, 0, 1]                       # request 0: slot 3 from 65; request 1's count is no count
    w0[0, 0, 0, 3] = w0[0, 0, 0, 65]
    assert torch.equal(k, k0) and torch.equal(s.weights, w0)


# ------------------------------------------------------------------ positions of the append
@pytest.mark.parametrize("nq,nkv,d,dtype", [(8, 2, 128, "bf16"), (4, 2, 64, "f32")])
def test_append_at_other_positions(nq, nkv, d, dtype):
    import torch
    c = Batch(nq, nkv, d, dtype, [0, 60, 130], [3, 17, 1], seed=3, pad_rows=1)
    turn = [1000, 61, 2 ** 24 - 1]
    k0, v0 = np64(c.k[1]), np64(c.v[1])
    q = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k, pos=i32(turn))
    assert c.ops.status() == 0
    kr, vr, qr = O.append(k0, v0, c.table, np64(c.qkv), nq, nkv, d, np64(c.g_q), np64(c.g_k), 1e-6, 1e6, c.cu, c.ctx, turn)
    # a pair is off by its fp32 operations, its angle's error (1.5e-6 at the far end) and the rounding to the type
    for got, ref in ((np64(q)[:c.T].reshape(c.T, nq, d), qr[:c.T].reshape(c.T, nq, d)), (np64(c.k[1]), kr)):
        live = ~np.isnan(ref)
        half = d // 2
        pair = np.sqrt(ref[..., :half] ** 2 + ref[..., half:] ** 2)
        tol = U[dtype] * np.abs(ref) + (16 * 2.0 ** -24 + 1.5e-6) * np.concatenate([pair, pair], -1)
        assert (np.abs(got - ref) <= tol)[live].all() and (np.isnan(got) == ~live).all()
    assert np.array_equal(np64(c.v[1]), vr, equal_nan=True)
    same = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k, pos=c.ctx_d)
    plain = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k)
    assert torch.equal(same[:c.T], plain[:c.T]) and c.ops.status() == 0
    k1 = c.k.clone()
    for bad in ([-1, 61, 5], [5, 61, 2 ** 24], [2 ** 31 - 1, 61, 5]):
        c.k.copy_(k1)
        c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k, pos=i32(bad))
        assert c.ops.status() == -7


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("nq,nkv,d,dtype,prefix", [(8, 2, 64, "bf16", 0), (4, 2, 64, "f32", 0), (4, 1, 128, "bf16", 128),
                                                   (4, 2, 128, "f32", 64)])
def test_steps_with_a_budget(nq, nkv, d, dtype, prefix):
    """Several steps of append, attention, weights of the committed tokens and
    eviction, on a cache with a budget and a (shared) prefix that stays: the
    cache's contents are the tokens that the plan kept, with their own
    positions, and the attention is the oracle's over them."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    from block_diffusion_drafter_context_gb300.target import SlotWeights, TargetOps
    B, L, budget, recent = 3, 2, prefix + 70, 20
    pages = -(-(budget + 16) // PAGE)
    n0 = prefix // PAGE
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator("cuda").manual_seed(d + prefix)
    table = np.arange(B * pages, dtype=np.int32).reshape(B, pages)
    table[1:, :n0] = table[0, :n0]
    k = torch.randn(L, B * pages, nkv, PAGE, d, generator=g, device="cuda").to(dt)
    v = torch.randn(L, B * pages, nkv, d, PAGE, generator=g, device="cuda").to(dt)
    kv = PagedKV.from_tensors(k, v, torch.from_numpy(table).cuda())
    slots = SlotWeights(L, B, nkv, pages * PAGE)
    ops = TargetOps(nq, nkv, d, dtype=dtype, max_batch=B, shared_prefix=True)
    seq = [prefix + 50, prefix + 9, prefix + 60]      # tokens so far; the slots hold them in order
    ctx = list(seq)
    # what every (layer, request, head) ought to hold: slot -> (position, K, V)
    at = lambda l, b, h, s: (l, int(table[b, s // PAGE]), h, s % PAGE)   # noqa: E731
    held = {(l, b, h): {s: (s, k[at(l, b, h, s)].clone(), v[l, int(table[b, s // PAGE]), h, :, s % PAGE].clone())
                        for s in range(ctx[b])} for l in range(L) for b in range(B) for h in range(nkv)}
    rng = np.random.default_rng(1)
    for step in range(7):
        new = [int(n) for n in rng.integers(0, 17, B)]
        new[0] = 16
        commit = [int(rng.integers(1, n + 1)) if n else 0 for n in new]
        cu = np.concatenate([[0], np.cumsum(new)])
        T = int(cu[-1])
        cu_d, ctx_d, seq_d, com_d = i32(cu.tolist()), i32(ctx), i32(seq), i32(commit)
        for l in range(L):
            qkv = torch.randn(T, (nq + 2 * nkv) * d, generator=g, device="cuda").to(dt)
            q = ops.append_kv(kv, l, qkv, cu_d, ctx_d, pos=seq_d)
            out, lse = ops.attend_shared(kv, l, q, cu_d, ctx_d, prefix, want_lse=True)
            ref, rlse, spread = O.attend(np64(k[l]), np64(v[l]), table, np64(q), nq, nkv, d, cu, ctx, 0, d ** -0.5)
            # as in the attention's own tests, |q| |k| d^-0.5 below 400, some 300 positions
            e = 2 * d * 2.0 ** -24 * 400 + 300 * 2.0 ** -24 + 2.0 ** -19
            tol = ((U["bf16"] if dtype == "bf16" else 0) + e) * spread + U[dtype] * np.abs(ref)
            assert (np.abs(np64(out) - ref) <= tol).all()
            before = np64(slots.weights[l])
            ops.add_weights(kv, l, slots, q, lse, cu_d, ctx_d, pos=seq_d, n_commit=com_d, first=prefix)
            wref, pref, added = O.add_weights(before, np32(slots.positions[l]), np64(k[l]), table, np64(q), np64(lse), nq,
                                              nkv, d, cu, ctx, seq, commit, prefix, d ** -0.5)
            got = np64(slots.weights[l])
            assert (np.abs(got - wref) <= (e + 800 * 2.0 ** -22) * added + 2.0 ** -23 * np.abs(wref)).all()
            # every committed token's weights over the heads and its slots add up to less than the heads
            assert added.sum() <= sum(commit) * nq * (1 + 1e-3)
            for b in range(B):
                for h in range(nkv):
                    for i in range(commit[b]):
                        s = ctx[b] + i
                        kk = O.head_norm_rope(np64(qkv[int(cu[b]) + i, (nq + h) * d:(nq + h + 1) * d]), None, 0, 1e6, seq[b] + i)
                        assert np.abs(np64(k[at(l, b, h, s)]) - kk).max() <= (2 * U[dtype] + 1e-5) * np.abs(kk).max() * 1.5
                        held[l, b, h][s] = (seq[b] + i, k[at(l, b, h, s)].clone(),
                                            v[l, int(table[b, s // PAGE]), h, :, s % PAGE].clone())
        ctx, seq = [c + m for c, m in zip(ctx, commit)], [s + m for s, m in zip(seq, commit)]
        w, p = np32(slots.weights).copy(), np32(slots.positions).copy()
        left = ops.evict(kv, slots, i32(ctx), i32(seq), budget, recent=recent, first=prefix)
        for (l, b, h), tokens in held.items():
            assert all(p[l, b, h, s] == tokens[s][0] for s in range(prefix, ctx[b]))
            for into, source in O.plan_eviction(w[l, b, h], p[l, b, h], ctx[b], seq[b], prefix, recent, budget):
                tokens[into] = tokens[source]
            for s in range(min(ctx[b], budget), ctx[b]):
                del tokens[s]
        ctx = [min(c, budget) for c in ctx]
        assert left.tolist() == ctx and ops.status() == 0
        p = np32(slots.positions)
        for (l, b, h), tokens in held.items():
            assert sorted(tokens) == list(range(ctx[b]))
            assert len({t[0] for t in tokens.values()}) == ctx[b]
            assert all(x in {t[0] for t in tokens.values()} for x in range(max(0, seq[b] - recent), seq[b]))
            for s, (pos, kk, vv) in tokens.items():
                assert s < prefix or p[l, b, h, s] == pos
                assert torch.equal(k[at(l, b, h, s)], kk) and torch.equal(v[l, int(table[b, s // PAGE]), h, :, s % PAGE], vv)
