"""The operators of a long or shared cache on the target model's side, as measured cases.

They stand beside append and attention on the same paged cache:

  shared   causal attention of the newest tokens of a batch whose requests share
           a long prefix (a system prompt, examples), the prefix computed once
           for all of them
  weights  the attention weight that each cached token received from the newest
           tokens, added up per kv head
  plan     which tokens a cache that outgrew its budget keeps, by accumulated
           weight: the moves that fill the freed slots below the budget
  move     those moves carried out on K, V, weights and positions

``own`` False computes them in elementary torch operations, ``own`` True calls
the library.  K pages are [page][kv head][slot][d] and V pages
[page][kv head][d][slot], 64 slots each, as everywhere in this repository.
"""
import math
import types

import torch

own = False

PAGE = 64
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few samples of one short prompt, token by token: latency
        dict(name="shared 4x1 on 1k", op="shared", dtype="bf16", nq=32, nkv=8, d=128, batch=4, prefix=1024, ctx_lo=5,
             ctx_hi=100, new_lo=1, new_hi=1),
        # ordinary decoding of a serving batch behind a long system prompt
        dict(name="shared 64x1 on 8k", op="shared", dtype="bf16", nq=32, nkv=8, d=128, batch=64, prefix=8192, ctx_lo=60,
             ctx_hi=1000, new_lo=1, new_hi=1),
        # verification of 16-token blocks behind a prefix of documents: the largest
        dict(name="shared 64x16 on 32k", op="shared", dtype="bf16", nq=40, nkv=8, d=128, batch=64, prefix=32768,
             ctx_lo=100, ctx_hi=2000, new_lo=16, new_hi=16),
        # the small fp32 model, mixed 0..16 tokens per request
        dict(name="shared f32 ragged", op="shared", dtype="f32", nq=4, nkv=2, d=64, batch=9, prefix=640, ctx_lo=0,
             ctx_hi=300, new_lo=0, new_hi=16),
        # one sequence decoding token by token
        dict(name="weights 1x1 ctx 2k", op="weights", dtype="bf16", nq=32, nkv=8, d=128, batch=1, ctx_lo=2048,
             ctx_hi=2048, new_lo=1, new_hi=1, first=0),
        # verification at long contexts, 1..16 tokens of each block committed: the largest
        dict(name="weights 64x16 16k-32k", op="weights", dtype="bf16", nq=40, nkv=8, d=128, batch=64, ctx_lo=16384,
             ctx_hi=32768, new_lo=16, new_hi=16, first=0),
        # the small fp32 model, mixed 0..16 tokens, the first tokens left out
        dict(name="weights f32 ragged", op="weights", dtype="f32", nq=4, nkv=2, d=64, batch=9, ctx_lo=70, ctx_hi=900,
             new_lo=0, new_hi=16, first=37),
        # every step of a small batch at its budget: all layers in one call
        dict(name="plan step 36 layers", op="plan", layers=36, nkv=8, batch=8, ctx_lo=4097, ctx_hi=4112, cap=4160,
             first=4, recent=256, budget=4096, zeros=0.0),
        # prompts cut down to the budget after they were read; many tokens that no row attended to (ties)
        dict(name="plan prompts 64x32k", op="plan", layers=1, nkv=8, batch=64, ctx_lo=16000, ctx_hi=32768, cap=32768,
             first=64, recent=1024, budget=4096, zeros=0.3),
        # one very long prompt: few lists, all of the time in each
        dict(name="plan prompt 1x128k", op="plan", layers=1, nkv=8, batch=1, ctx_lo=131071, ctx_hi=131071, cap=131072,
             first=0, recent=4096, budget=65536, zeros=0.0),
        # a step's few moves in every layer
        dict(name="move step 8 layers", op="move", dtype="bf16", layers=8, nkv=8, d=128, batch=16, ctx_lo=4097,
             ctx_hi=4112, cap=4160, first=4, budget=4096),
        # a batch of prompts cut down to the budget: nearly every slot below it is filled anew
        dict(name="move prompts 32x16k", op="move", dtype="bf16", layers=1, nkv=8, d=128, batch=32, ctx_lo=9000,
             ctx_hi=16384, cap=16384, first=64, budget=4096),
    ]


def _log(rng, lo, hi):
    """An integer spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "weights", "plan", "move"])
    nkv = rng.choice([1, 2, 4, 8])
    if op in ("shared", "weights"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d = rng.choice([64, 128, 128])
        g = rng.randint(1, min(8, 40 // nkv))
        batch = _log(rng, 1, 64)
        new_hi = rng.choice([1, 1, rng.randint(2, 16)])
        case = dict(op=op, dtype=dtype, nq=g * nkv, nkv=nkv, d=d, batch=batch)
        if op == "shared":
            top = 512 if dtype == "bf16" else 32
            ctx_hi = _log(rng, 1, 2000)
            return dict(case, prefix=PAGE * _log(rng, 1, top), ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi,
                        new_lo=rng.randint(0, new_hi), new_hi=new_hi)
        ctx_hi = _log(rng, 1, 32768 if dtype == "bf16" else 4096)
        return dict(case, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, new_lo=rng.randint(0, new_hi), new_hi=new_hi,
                    first=rng.choice([0, 0, 4, rng.randint(0, ctx_hi)]))
    batch = _log(rng, 1, 32)
    layers = _log(rng, 1, 8) if batch <= 8 else 1
    cap = PAGE * _log(rng, 2, 256 if op == "plan" and batch * layers <= 32 else 128)
    budget = rng.randint(2, cap - 1)
    first = rng.choice([0, 4, 64, rng.randint(0, budget)])
    first = min(first, budget - 1)
    ctx_hi = rng.randint(budget + 1, cap)
    case = dict(op=op, layers=layers, nkv=nkv, batch=batch, ctx_lo=rng.randint(budget // 2, ctx_hi), ctx_hi=ctx_hi,
                cap=cap, first=first, budget=budget)
    if op == "plan":
        return dict(case, recent=rng.randint(0, budget - first), zeros=rng.choice([0.0, 0.0, 0.5, 0.95]))
    return dict(case, dtype=rng.choice(["bf16", "bf16", "f32"]), d=rng.choice([64, 128]))


def _spread(lo, hi, n):
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)] if n > 1 else [hi]


def _lengths(case):
    """Tokens before the new ones (behind the prefix, where there is one), new
    tokens and committed ones: evenly spread over their ranges (the seed only
    permutes the requests), at least one token new."""
    n = case["batch"]
    ctx, new = _spread(case["ctx_lo"], case["ctx_hi"], n), _spread(case["new_lo"], case["new_hi"], n)[::-1]
    new[0] = max(1, new[0])
    return ctx, new, [1 + i * 7 % m if m else 0 for i, m in enumerate(new)]


def _moves_of(case):
    """Moves of each request of a `move` case: what random weights make of the
    slots that may be freed, the slots above the budget."""
    out = []
    for c in _spread(case["ctx_lo"], case["ctx_hi"], case["batch"]):
        over, room = max(0, c - case["budget"]), case["budget"] - case["first"]
        out.append(max(1, room * over // (room + over)) if over else 0)
    return out


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    st = types.SimpleNamespace(case=case)
    {"shared": _make_rows, "weights": _make_rows, "plan": _make_slots, "move": _make_slots}[case["op"]](st, _gen(seed), seed)
    return st


def _make_rows(st, g, seed):
    """A ragged batch over a scattered cache: queries, lengths, and for
    `weights` the log-sum-exp that the attention before gave."""
    c = st.case
    dt, nq, nkv, d = DT[c["dtype"]], c["nq"], c["nkv"], c["d"]
    host = torch.Generator().manual_seed(seed)
    ctx, new, commit = _lengths(c)
    order = torch.randperm(len(ctx), generator=host).tolist()
    ctx, new, commit = ([v[i] for i in order] for v in (ctx, new, commit))
    shared = c.get("prefix", 0) // PAGE
    ctx = [shared * PAGE + x for x in ctx]
    pages = [-(-(x + n) // PAGE) for x, n in zip(ctx, new)]
    pool = shared + sum(p - shared for p in pages) + 3
    ids = torch.randperm(pool, generator=host).to(torch.int32)
    table = torch.full((len(ctx), max(1, max(pages))), -1, dtype=torch.int32)
    table[:, :shared] = ids[:shared]
    at = shared
    for b, p in enumerate(pages):
        table[b, shared:p] = ids[at:at + p - shared]
        at += p - shared
    cu = torch.tensor([0] + new).cumsum(0).tolist()
    st.table, st.ctx, st.cu, st.most = table.cuda(), _i32(ctx), _i32(cu), max(new)
    st.k = torch.empty(1, pool, nkv, PAGE, d, dtype=dt, device="cuda").normal_(generator=g)
    st.v = torch.empty(1, pool, nkv, d, PAGE, dtype=dt, device="cuda").normal_(generator=g)
    st.q = (torch.randn(cu[-1], nq * d, generator=g, device="cuda") * 2).to(dt)
    if c["op"] == "weights":
        st.commit, st.pos = _i32(commit), _i32([x + 100 * i for i, x in enumerate(ctx)])
        st.lse = torch.empty(cu[-1], nq, device="cuda")
        for b, x in enumerate(ctx):
            n = x + new[b]
            if new[b]:
                k = st.k[0, st.table[b, :pages[b]].long()].transpose(0, 1).reshape(nkv, -1, d)[:, :n].float()
                q = st.q[cu[b]:cu[b + 1]].float().view(new[b], nkv, -1, d).transpose(0, 1).reshape(nkv, -1, d)
                s = (q @ k.transpose(1, 2) * d ** -0.5).view(nkv, new[b], -1, n)
                hide = torch.arange(n, device="cuda") > x + torch.arange(new[b], device="cuda")[:, None]
                s.masked_fill_(hide[:, None], -math.inf)
                st.lse[cu[b]:cu[b + 1]] = torch.logsumexp(s, -1).transpose(0, 1).reshape(new[b], nq)
        rows = (1, len(ctx), nkv, table.shape[1] * PAGE)
        st.weights = torch.rand(rows, generator=g, device="cuda") * 3
        st.positions = torch.arange(rows[3], dtype=torch.int32, device="cuda").expand(rows).contiguous()
    if own:
        _handle(st, c["dtype"], len(ctx), nq, nkv, d, max(1, st.most))


def _make_slots(st, g, seed):
    """Weights and positions of every slot; for `move` the cache and a plan."""
    c = st.case
    L, B, nkv, cap = c["layers"], c["batch"], c["nkv"], c["cap"]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
    ctx = [_spread(c["ctx_lo"], c["ctx_hi"], B)[i] for i in order]
    st.ctx = _i32(ctx)
    # heavy-tailed, as accumulated weights are
    st.weights = torch.randn(L, B, nkv, cap, generator=g, device="cuda").mul_(1.5).exp_()
    # slots below the budget were refilled before: their tokens lie in no strict order
    jitter = torch.rand(L, B, nkv, c["budget"], generator=g, device="cuda") * min(300, c["budget"])
    near = (torch.arange(c["budget"], device="cuda") + jitter).argsort(-1)
    far = torch.arange(c["budget"], cap, device="cuda").expand(L, B, nkv, -1)
    st.positions = (torch.cat([near, far], -1) + 777).to(torch.int32)
    st.seq = st.ctx + 777
    st.top = min(c["budget"] - c["first"], cap - c["budget"])     # most moves of a list
    if c["op"] == "plan":
        st.weights[torch.rand(st.weights.shape, generator=g, device="cuda") < c["zeros"]] = 0
        if own:
            _handle(st, "bf16", B, nkv, nkv, 128, 1)
        return
    moved = [_moves_of(c)[i] for i in order]
    st.counts = _i32(moved).view(1, B, 1).expand(L, B, nkv).contiguous()

    def pick(lo, hi, n):   # n[b] slots of lo .. hi[b] - 1, ascending
        u = torch.rand(L, B, nkv, cap, generator=g, device="cuda")
        slot = torch.arange(cap, device="cuda")
        u = torch.where((slot >= lo) & (slot < hi.view(1, B, 1, 1)), u, 2.0)
        at = u.argsort(-1)[..., :st.top]
        live = torch.arange(st.top, device="cuda") < n[..., None]
        return torch.where(live, at, cap).sort(-1)[0].where(live, torch.tensor(-1, device="cuda")).to(torch.int32)

    into = pick(c["first"], torch.full_like(st.ctx, c["budget"]), st.counts)
    st.moves = torch.stack([into, pick(c["budget"], st.ctx, st.counts)], 3).contiguous()
    pages = [-(-x // PAGE) for x in ctx]
    pool = sum(pages) + 3
    ids = torch.randperm(pool, generator=torch.Generator().manual_seed(seed + 1)).to(torch.int32)
    table = torch.full((B, cap // PAGE), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = ids[at:at + p]
        at += p
    st.table = table.cuda()
    dt = DT[c["dtype"]]
    st.k = torch.empty(L, pool, nkv, PAGE, c["d"], dtype=dt, device="cuda").normal_(generator=g)
    st.v = torch.empty(L, pool, nkv, c["d"], PAGE, dtype=dt, device="cuda").normal_(generator=g)
    if own:
        _handle(st, c["dtype"], B, nkv, nkv, c["d"], 1)


def _handle(st, dtype, batch, nq, nkv, d, most):
    """What a program keeps between calls: the operators' handle, the cache and
    its slots' weights."""
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    from block_diffusion_drafter_context_gb300.target import SlotWeights, TargetOps
    st.ops = TargetOps(nq, nkv, d, dtype=dtype, max_batch=batch, max_new=most, shared_prefix=st.case["op"] == "shared")
    if hasattr(st, "k"):
        st.kv = PagedKV.from_tensors(st.k, st.v, st.table)
    if hasattr(st, "weights"):
        st.slots = SlotWeights.from_tensors(st.weights, st.positions)


# ------------------------------------------------------------------ one pass
def run(st):
    return {"shared": _shared, "weights": _weights, "plan": _plan, "move": _move}[st.case["op"]](st)


def _rows(st):
    """The batch padded to [B, S] tokens: row of each, whether it is one, its position."""
    i = torch.arange(st.most, device="cuda")
    row = st.cu[:-1, None] + i
    return row.clamp(max=st.q.shape[0] - 1), row < st.cu[1:, None], st.ctx[:, None] + i


def _shared(st):
    c = st.case
    if own:
        out, lse = st.ops.attend_shared(st.kv, 0, st.q, st.cu, st.ctx, c["prefix"], max_new=st.most, want_lse=True)
        return {"out": out, "lse": lse}
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    B, S, g, T = c["batch"], st.most, nq // nkv, st.q.shape[0]
    scale, n0 = d ** -0.5, c["prefix"] // PAGE
    # the prefix: every row of the batch against the same keys
    head = st.table[0, :n0].long()
    k = st.k[0][head].float().transpose(0, 1).reshape(nkv, -1, d)
    v = st.v[0][head].float().permute(1, 2, 0, 3).reshape(nkv, d, -1)
    q = st.q.float().view(T, nkv, g, d).transpose(0, 1).reshape(nkv, T * g, d)
    s = (q @ k.transpose(1, 2)).mul_(scale)
    m0 = s.amax(-1, keepdim=True)
    p = s.sub_(m0).exp_()
    z0, o0 = p.sum(-1, keepdim=True), p @ v.transpose(1, 2)
    # each request's own part, padded
    row, real, pos = _rows(st)
    pages = st.table[:, n0:].clamp(min=0).long()
    n = pages.shape[1] * PAGE
    k = st.k[0][pages].float().transpose(1, 2).reshape(B, nkv, n, d)
    v = st.v[0][pages].float().permute(0, 2, 3, 1, 4).reshape(B, nkv, d, n)
    q = st.q[row].float().view(B, S, nkv, g, d).transpose(1, 2).reshape(B, nkv, S * g, d)
    s = (q @ k.transpose(2, 3)).mul_(scale).view(B, nkv, S, g, n)
    see = torch.arange(n, device="cuda") + c["prefix"] <= pos[:, :, None]
    s = s.masked_fill_(~see[:, None, :, None], -math.inf).view(B, nkv, S * g, n)
    m1 = s.amax(-1, keepdim=True)
    p = s.sub_(m1).exp_()
    z1, o1 = p.sum(-1, keepdim=True), p @ v.transpose(2, 3)

    def pad(x):   # [nkv, T g, w] -> [B, nkv, S g, w]
        return x.view(nkv, T, g, -1)[:, row].permute(1, 0, 2, 3, 4).reshape(B, nkv, S * g, -1)

    m0, z0, o0 = pad(m0), pad(z0), pad(o0)
    m = torch.maximum(m0, m1)
    a, b = (m0 - m).exp(), (m1 - m).exp()
    z = a * z0 + b * z1
    o = (a * o0 + b * o1) / z
    o = o.view(B, nkv, S, g, d).transpose(1, 2).reshape(B, S, nq * d)
    lse = (m + z.log()).view(B, nkv, S, g).transpose(1, 2).reshape(B, S, nq)
    return {"out": o[real].to(st.q.dtype), "lse": lse[real]}


def _weights(st):
    c = st.case
    if own:
        st.ops.add_weights(st.kv, 0, st.slots, st.q, st.lse, st.cu, st.ctx, pos=st.pos, n_commit=st.commit,
                           max_new=st.most, first=c["first"])
        return {"weights": st.weights, "positions": st.positions}
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    B, S, g = c["batch"], st.most, nq // nkv
    row, _, pos = _rows(st)
    pages = st.table.clamp(min=0).long()
    n = pages.shape[1] * PAGE
    k = st.k[0][pages].float().transpose(1, 2).reshape(B, nkv, n, d)
    q = st.q[row].float().view(B, S, nkv, g, d).transpose(1, 2).reshape(B, nkv, S * g, d)
    s = (q @ k.transpose(2, 3)).mul_(d ** -0.5).view(B, nkv, S, g, n)
    s = s.sub_(st.lse[row].view(B, S, nkv, g).transpose(1, 2)[..., None])
    key, i = torch.arange(n, device="cuda"), torch.arange(S, device="cuda")
    see = (key <= pos[:, :, None]) & (i < st.commit[:, None])[:, :, None]
    add = s.exp_().masked_fill_(~see[:, None, :, None], 0).sum((2, 3))
    ctx, end = st.ctx[:, None, None], (st.ctx + st.commit)[:, None, None]
    live, fresh = (key >= c["first"]) & (key < end), (key >= ctx) & (key < end)
    w = torch.where(fresh, 0, st.weights[0])
    st.weights[0] = torch.where(live, w + add, st.weights[0])
    at = (st.pos[:, None, None] + key - ctx).to(torch.int32)
    st.positions[0] = torch.where(live & fresh, at, st.positions[0])
    return {"weights": st.weights, "positions": st.positions}


def _plan(st):
    c = st.case
    if own:
        moves, counts, left = st.ops.plan_eviction(st.slots, st.ctx, st.seq, c["budget"], recent=c["recent"],
                                                   first=c["first"])
        return {"moves": moves, "counts": counts, "ctx": left}
    slot = torch.arange(c["cap"], device="cuda")
    ctx, seq = st.ctx.view(1, -1, 1, 1), st.seq.view(1, -1, 1, 1)
    keep = ctx.clamp(max=c["budget"])
    free = (slot >= c["first"]) & (slot < ctx)
    w = torch.where(st.positions >= seq - c["recent"], math.inf, st.weights)
    order = torch.where(free, w, -math.inf).sort(dim=-1, descending=True, stable=True)[1]   # equal weights: the lower slot first
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    kept = free & (rank < keep - c["first"])
    into = torch.where(free & ~kept & (slot < keep), slot, c["cap"])
    source = torch.where(kept & (slot >= keep), slot, c["cap"])
    moves = torch.stack([into.sort(-1)[0], source.sort(-1)[0]], 3)[..., :st.top]
    counts = (source < c["cap"]).sum(-1)
    return {"moves": torch.where(moves < c["cap"], moves, -1).int(), "counts": counts.int(), "ctx": keep.view(-1).int()}


def _move(st):
    c = st.case
    if own:
        st.ops.move_slots(st.kv, st.slots, st.moves, st.counts)
        return {"k": st.k, "v": st.v, "weights": st.weights, "positions": st.positions}
    layer, b, h, i = (st.moves[:, :, :, 0] >= 0).nonzero(as_tuple=True)
    into, source = st.moves[layer, b, h, 0, i].long(), st.moves[layer, b, h, 1, i].long()
    p0, p1 = st.table[b, into // PAGE].long(), st.table[b, source // PAGE].long()
    s0, s1 = into % PAGE, source % PAGE
    st.k[layer, p0, h, s0] = st.k[layer, p1, h, s1]
    st.v[layer, p0, h, :, s0] = st.v[layer, p1, h, :, s1]
    st.weights[layer, b, h, into] = st.weights[layer, b, h, source]
    st.positions[layer, b, h, into] = st.positions[layer, b, h, source]
    return {"k": st.k, "v": st.v, "weights": st.weights, "positions": st.positions}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, nkv = case["op"], case["nkv"]
    size = 4 if case.get("dtype") == "f32" else 2
    if op in ("plan", "move"):
        lists = case["layers"] * nkv
        if op == "plan":   # weight and position of every slot that may go, the moves; a comparison per slot
            slots = sum(max(0, n - case["first"])
                        for n in _spread(case["ctx_lo"], case["ctx_hi"], case["batch"]) if n > case["budget"])
            top = min(case["budget"] - case["first"], case["cap"] - case["budget"])
            return {"bytes": lists * (8 * slots + (8 * top + 4) * case["batch"]) + 12 * case["batch"],
                    "flops": 2 * lists * slots}
        n = lists * sum(_moves_of(case))
        return {"bytes": max(1, n * (4 * case["d"] * size + 16 + 8)), "flops": 0}
    nq, d = case["nq"], case["d"]
    ctx, new, commit = _lengths(case)
    T = sum(new)
    if op == "shared":
        pairs = sum(n * case["prefix"] + sum(c + i + 1 for i in range(n)) for c, n in zip(ctx, new))
        keys = case["prefix"] + sum(c + n for c, n in zip(ctx, new) if n)
        return {"bytes": 2 * keys * nkv * d * size + T * nq * (2 * d * size + 4), "flops": 4 * pairs * nq * d}
    keys = sum(max(0, c + m - case["first"]) for c, m in zip(ctx, commit) if m)
    pairs = sum(sum(max(0, c + i + 1 - case["first"]) for i in range(m)) for c, m in zip(ctx, commit))
    return {"bytes": keys * nkv * (d * size + 8) + sum(commit) * nq * (d * size + 4), "flops": 2 * pairs * nq * d}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def exact(case, seed):
    st = prepare(case, seed)
    return {"shared": _exact_shared, "weights": _exact_weights, "plan": lambda st: None, "move": _exact_move}[case["op"]](st)


def _keys(st, b, n):
    """K [nkv][n][d] and V [nkv][n][d] of a request's first n slots."""
    pages = st.table[b, :-(-n // PAGE)].long()
    nkv, d = st.case["nkv"], st.case["d"]
    return (st.k[0, pages].double().permute(1, 0, 2, 3).reshape(nkv, -1, d)[:, :n],
            st.v[0, pages].double().permute(1, 0, 3, 2).reshape(nkv, -1, d)[:, :n])


def _exact_shared(st):
    c = st.case
    nkv, d, n0 = c["nkv"], c["d"], c["prefix"]
    ctx, cu = st.ctx.tolist(), st.cu.tolist()
    out = torch.empty(cu[-1], nkv, c["nq"] // nkv, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(cu[-1], nkv, c["nq"] // nkv, dtype=torch.float64, device="cuda")
    for b in range(len(ctx)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        k, v = _keys(st, b, ctx[b] + n)
        q = st.q[cu[b]:cu[b + 1]].double().view(n, nkv, -1, d)
        for h in range(nkv):
            s = torch.einsum("igd,td->igt", q[:, h], k[h]) / math.sqrt(d)
            for i in range(n - 1):
                s[i, :, ctx[b] + i + 1:] = -math.inf
            l = torch.logsumexp(s, -1)
            lse[cu[b]:cu[b + 1], h] = l
            out[cu[b]:cu[b + 1], h] = torch.einsum("igt,td->igd", (s - l[..., None]).exp(), v[h])
    return {"out": out.reshape(cu[-1], -1), "lse": lse.reshape(cu[-1], -1)}


def _exact_weights(st):
    c = st.case
    ctx, cu, commit = st.ctx.tolist(), st.cu.tolist(), st.commit.tolist()
    w = st.weights.double()
    for b in range(len(ctx)):
        m = commit[b]
        if m == 0:
            continue
        end = ctx[b] + m
        w[0, b, :, max(ctx[b], c["first"]):end] = 0
        k = _keys(st, b, end)[0]
        for i in range(m):
            q = st.q[cu[b] + i].double().view(c["nkv"], -1, c["d"])
            seen = ctx[b] + i + 1
            s = torch.einsum("hgd,htd->hgt", q, k[:, :seen]) / math.sqrt(c["d"])
            p = (s - st.lse[cu[b] + i].double().view(c["nkv"], -1, 1)).exp().sum(1)
            w[0, b, :, c["first"]:seen] += p[:, c["first"]:]
    return {"weights": w, "positions": None}


def _exact_move(st):
    c = st.case
    k, v, w = st.k.double(), st.v.double(), st.weights.double()
    table = st.table.cpu()
    for layer in range(c["layers"]):
        for b in range(c["batch"]):
            for h in range(c["nkv"]):
                n = int(st.counts[layer, b, h])
                to, of = st.moves[layer, b, h, :, :n].long().cpu()
                at, by = (table[b, to // PAGE].long(), to % PAGE), (table[b, of // PAGE].long(), of % PAGE)
                k[layer, at[0], h, at[1]] = st.k[layer, by[0], h, by[1]].double()
                v[layer, at[0], h, :, at[1]] = st.v[layer, by[0], h, :, by[1]].double()
                w[layer, b, h, to] = st.weights[layer, b, h, of].double()
    return {"k": k, "v": v, "weights": w, "positions": None}
