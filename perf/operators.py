"""The operators of the target model's side of a speculative step, as measured cases.

One step of speculative decoding needs, beside the drafter, one pass of the
target model over the tokens to be verified.  Three operators of that pass
work on the same paged cache and token layout as the drafter:

  append     q / k norm and rotation of a fused q | k | v projection, K and V
             appended to the paged cache, the rotated queries returned
  attend     causal attention of the 1..16 newest tokens of each request over
             its paged cache (grouped heads, optional sliding window)
  logprobs   log probability, entropy and rank of given tokens under their
             logits, with the 16 most probable alternatives

``own`` False computes them in elementary torch operations, ``own`` True calls
the library.  K pages are [page][kv head][slot][d] and V pages
[page][kv head][d][slot], 64 slots each, as everywhere in this repository.
"""
import math
import types

import torch

own = False

PAGE = 64
BASE = 1e6
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence decoding token by token: the smallest append
        dict(name="append 1x1", op="append", dtype="bf16", nq=32, nkv=8, d=128, batch=1, ctx_lo=2048, ctx_hi=2048,
             new_lo=1, new_hi=1, norm=True, pad=0),
        # a full serving batch appending a drafted block per request, far positions, a row stride wider than the row
        dict(name="append 64x16 far", op="append", dtype="bf16", nq=40, nkv=8, d=128, batch=64, ctx_lo=16384,
             ctx_hi=32768, new_lo=16, new_hi=16, norm=True, pad=64),
        # prompts of different lengths entering an empty cache
        dict(name="append prompts", op="append", dtype="bf16", nq=32, nkv=8, d=128, batch=5, ctx_lo=0, ctx_hi=0,
             new_lo=1024, new_hi=8192, norm=True, pad=0),
        # the small fp32 model: ragged pieces at odd offsets inside their pages, no norm
        dict(name="append f32 ragged", op="append", dtype="f32", nq=4, nkv=2, d=64, batch=5, ctx_lo=3, ctx_hi=777,
             new_lo=1, new_hi=37, norm=False, pad=4),
        # one sequence, one token: the latency of a decode step
        dict(name="attend 1x1 ctx 2k", op="attend", dtype="bf16", nq=32, nkv=8, d=128, batch=1, ctx_lo=2048,
             ctx_hi=2048, new_lo=1, new_hi=1, window=0),
        # ordinary decoding: 32 ragged requests, one token each
        dict(name="attend 32x1 ctx 1k-8k", op="attend", dtype="bf16", nq=32, nkv=8, d=128, batch=32, ctx_lo=1024,
             ctx_hi=8192, new_lo=1, new_hi=1, window=0),
        # verification of 16-token blocks at long contexts: the largest
        dict(name="attend 64x16 ctx 16k-32k", op="attend", dtype="bf16", nq=40, nkv=8, d=128, batch=64, ctx_lo=16384,
             ctx_hi=32768, new_lo=16, new_hi=16, window=0),
        # a single very long sequence verifying a 5-token block: the split over the length is all there is
        dict(name="attend 1x5 ctx 128k", op="attend", dtype="bf16", nq=32, nkv=8, d=128, batch=1, ctx_lo=131071,
             ctx_hi=131071, new_lo=5, new_hi=5, window=0),
        # the small fp32 model with a sliding window, mixed 0..16 tokens per request
        dict(name="attend f32 window", op="attend", dtype="f32", nq=4, nkv=2, d=64, batch=9, ctx_lo=0, ctx_hi=900,
             new_lo=0, new_hi=16, window=200),
        # the committed tokens of one request
        dict(name="logprobs 16 rows", op="logprobs", dtype="f32", rows=16, live=16, vocab=151936, pad=0, temp=1.0,
             masked=0.0),
        # a serving batch of 64 blocks of 16 positions, the unaccepted ones padded with -1
        dict(name="logprobs 1024 rows", op="logprobs", dtype="f32", rows=1024, live=640, vocab=151936, pad=0, temp=0.8,
             masked=0.0),
        # bf16 logits (many ties), odd vocabulary and row stride, a grammar mask over part of the vocabulary
        dict(name="logprobs bf16 odd", op="logprobs", dtype="bf16", rows=480, live=480, vocab=40001, pad=2, temp=1.0,
             masked=0.3),
    ]


def _log(rng, lo, hi):
    """An integer spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "logprobs"])
    if op == "logprobs":
        rows = _log(rng, 1, 1024)
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), rows=rows, live=rng.randint((rows + 1) // 2, rows),
                    vocab=_log(rng, 1000, 151936), pad=rng.choice([0, 1, 3, 8, 64]),
                    temp=rng.choice([0.5, 0.8, 1.0, 1.3]), masked=rng.choice([0.0, 0.0, 0.5, 0.95]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    nkv = rng.choice([1, 2, 4, 8])
    g = rng.randint(1, 8)
    batch = _log(rng, 1, 64)
    if op == "append":
        top = 8192 if batch <= 5 else 256 if batch <= 32 else 16
        new_hi = _log(rng, 1, top)
        ctx_hi = rng.randint(0, 32768)
        return dict(op=op, dtype=dtype, nq=g * nkv, nkv=nkv, d=d, batch=batch, ctx_lo=rng.randint(0, ctx_hi),
                    ctx_hi=ctx_hi, new_lo=rng.randint(0, new_hi), new_hi=new_hi, norm=rng.random() < 0.7,
                    pad=rng.choice([0, 8, 64]))
    top = 32768 if dtype == "bf16" else 4096
    ctx_hi = 131072 if dtype == "bf16" and batch <= 4 and rng.random() < 0.3 else _log(rng, 1, top)
    new_hi = rng.choice([1, 1, rng.randint(2, 16)])
    return dict(op=op, dtype=dtype, nq=g * nkv, nkv=nkv, d=d, batch=batch, ctx_lo=rng.randint(0, ctx_hi),
                ctx_hi=ctx_hi, new_lo=rng.randint(0, new_hi), new_hi=new_hi,
                window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]))


def _lengths(case):
    """Context lengths and new tokens of the batch: evenly spread over their
    ranges (the seed only permutes the requests), at least one token new."""
    n = case["batch"]

    def spread(lo, hi):
        return [lo + (hi - lo) * i // (n - 1) for i in range(n)] if n > 1 else [hi]

    ctx, new = spread(case["ctx_lo"], case["ctx_hi"]), spread(case["new_lo"], case["new_hi"])[::-1]
    new[0] = max(1, new[0])
    return ctx, new


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _batch(case, seed):
    """The batch in a random order: contexts, prefix sums of the new tokens."""
    ctx, new = _lengths(case)
    order = torch.randperm(len(ctx), generator=torch.Generator().manual_seed(seed)).tolist()
    ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return ctx, new, cu


def _table(first, last, seed):
    """Page table rows holding pages first[b]..last[b]-1 of each request,
    scattered over the pool; other entries are never read and hold -1."""
    used = sum(max(0, e - s) for s, e in zip(first, last))
    pool = used + 3
    ids = torch.randperm(pool, generator=torch.Generator().manual_seed(seed + 1)).to(torch.int32)
    table = torch.full((len(first), max(1, max(last))), -1, dtype=torch.int32)
    at = 0
    for b, (s, e) in enumerate(zip(first, last)):
        if e > s:
            table[b, s:e] = ids[at:at + e - s]
            at += e - s
    return table.cuda(), pool


def _handle(case, st):
    """What a program keeps between calls: the operators' handle and the cache."""
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    from block_diffusion_drafter_context_gb300.target import TargetOps
    st.kv = PagedKV.from_tensors(st.k, st.v, st.table)
    st.ops = TargetOps(case["nq"], case["nkv"], case["d"], dtype=case["dtype"], max_batch=case["batch"],
                       max_new=min(16, max(1, case["new_hi"])), rope_base=BASE, eps=EPS)


def prepare(case, seed):
    g = _gen(seed)
    st = types.SimpleNamespace(case=case)
    if case["op"] == "logprobs":
        rows, V = case["rows"], case["vocab"]
        x = torch.randn(rows, V + case["pad"], generator=g, device="cuda") * 2.5
        if case["masked"] > 0:
            x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < case["masked"], -math.inf)
        st.logits = x.to(DT[case["dtype"]])[:, :V]   # the row stride is V + pad
        # half of the tokens are what the row makes likely, the rest any token
        likely = st.logits.argmax(1)
        any_id = torch.randint(0, V, (rows,), generator=g, device="cuda")
        ids = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, likely, any_id)
        dead = torch.randperm(rows, generator=g, device="cuda")[case["live"]:]
        ids[dead] = -1
        st.ids = ids.to(torch.int32)
        return st
    dt, nq, nkv, d = DT[case["dtype"]], case["nq"], case["nkv"], case["d"]
    ctx, new, cu = _batch(case, seed)
    if case["op"] == "append":   # the pool holds the pages that are written
        first = [c // PAGE for c in ctx]
        last = [-(-(c + n) // PAGE) if n else c // PAGE for c, n in zip(ctx, new)]
    else:
        first = [0] * len(ctx)
        last = [-(-(c + n) // PAGE) for c, n in zip(ctx, new)]
    st.table, pool = _table(first, last, seed)
    st.k = torch.empty(1, pool, nkv, PAGE, d, dtype=dt, device="cuda").normal_(generator=g)
    st.v = torch.empty(1, pool, nkv, d, PAGE, dtype=dt, device="cuda").normal_(generator=g)
    st.ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    st.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    T = cu[-1]
    if case["op"] == "append":
        width = (nq + 2 * nkv) * d
        st.qkv = (torch.randn(T, width + case["pad"], generator=g, device="cuda") * 1.5).to(dt)[:, :width]
        st.g_q = 1 + 0.1 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None
        st.g_k = 1 + 0.1 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None
    else:
        st.q = (torch.randn(T, nq * d, generator=g, device="cuda") * 2).to(dt)
        st.most = max(new)
    if own:
        _handle(case, st)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return {"append": _append, "attend": _attend, "logprobs": _logprobs}[st.case["op"]](st)


def _place(st, T):
    """Request and position of every new token."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(st.cu[1:].contiguous(), t, right=True)
    return b, st.ctx[b].long() + t - st.cu[b]


def _append(st):
    c = st.case
    if own:
        q = st.ops.append_kv(st.kv, 0, st.qkv, st.cu, st.ctx, g_q=st.g_q, g_k=st.g_k)
        return {"q": q, "k": st.k, "v": st.v}
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    T = st.qkv.shape[0]
    b, pos = _place(st, T)
    x = st.qkv.float().view(T, nq + 2 * nkv, d)
    q, k, v = x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * st.g_q
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * st.g_k
    i = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    ang = pos.double()[:, None] * BASE ** (-2 * i / d)
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def rotate(y):
        a, z = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([a * cos - z * sin, z * cos + a * sin], -1)

    page, slot = st.table[b, pos // PAGE].long(), pos % PAGE
    st.k[0][page, :, slot] = rotate(k).to(st.k.dtype)
    st.v[0][page, :, :, slot] = v.to(st.v.dtype)
    return {"q": rotate(q).to(st.k.dtype).view(T, nq * d), "k": st.k, "v": st.v}


def _attend(st):
    c = st.case
    if own:
        out, lse = st.ops.attend(st.kv, 0, st.q, st.cu, st.ctx, max_new=st.most, window=c["window"], want_lse=True)
        return {"out": out, "lse": lse}
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    B, T, S = c["batch"], st.q.shape[0], st.most
    pages = st.table.clamp(min=0).long()
    n = pages.shape[1] * PAGE
    k = st.k[0][pages].float().transpose(1, 2).reshape(B, nkv, n, d)
    v = st.v[0][pages].float().permute(0, 2, 3, 1, 4).reshape(B, nkv, d, n)
    i = torch.arange(S, device="cuda")
    row = st.cu[:-1, None] + i                               # [B, S], past a request's tokens: any row, not kept
    real = row < st.cu[1:, None]
    q = st.q[row.clamp(max=T - 1)].float().view(B, S, nkv, nq // nkv, d).transpose(1, 2).reshape(B, nkv, -1, d)
    s = q @ k.transpose(2, 3) * d ** -0.5                    # [B, nkv, S * g, n]
    key, pos = torch.arange(n, device="cuda"), st.ctx[:, None] + i
    see = key <= pos[:, :, None]                             # [B, S, n]
    if c["window"]:
        see = see & (key > pos[:, :, None] - c["window"])
    s = s.view(B, nkv, S, -1, n).masked_fill_(~see[:, None, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = p.view(B, nkv, -1, n) @ v.transpose(2, 3) / z.view(B, nkv, -1, 1)
    o = o.view(B, nkv, S, nq // nkv, d).transpose(1, 2).reshape(B, S, nq * d)
    lse = (m + z.log()).view(B, nkv, S, -1).transpose(1, 2).reshape(B, S, nq)
    return {"out": o[real].to(st.q.dtype), "lse": lse[real]}


def _logprobs(st):
    c = st.case
    if own:
        from block_diffusion_drafter_context_gb300.target import token_logprobs
        return token_logprobs(st.logits, st.ids, temperature=c["temp"], n_top=16)
    x, V = st.logits, c["vocab"]
    live = st.ids >= 0
    tok = st.ids.clamp(min=0).long()[:, None]
    y = x.float() / c["temp"]
    m = y.amax(1, keepdim=True)
    e = (y - m).exp()
    z = e.sum(1, keepdim=True)
    lse = m + z.log()
    top, top_ids = torch.sort(x, dim=1, descending=True, stable=True)   # equal values: the lower id first
    mine = x.gather(1, tok)
    before = (x > mine) | ((x == mine) & (torch.arange(V, device="cuda") < tok))
    # entropy: log z - sum e (y - m) / z, a masked entry adds nothing
    ent = z.log()[:, 0] - torch.where(e > 0, e * (y - m), 0).sum(1) / z[:, 0]

    def of(v, dead):
        return torch.where(live.view(-1, *[1] * (v.dim() - 1)), v, dead)

    return {"logprob": of((mine.float() / c["temp"] - lse)[:, 0], 0.0), "entropy": of(ent, 0.0),
            "rank": of(before.sum(1).int(), -1), "top_ids": of(top_ids[:, :16].int(), -1),
            "top_logprobs": of(top[:, :16].float() / c["temp"] - lse, 0.0)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "logprobs":
        n = case["live"] * case["vocab"]
        # a scaling, an exp, two sums and a comparison for each logit
        return {"bytes": n * size + case["rows"] * (4 + 12 + 16 * 8), "flops": 6 * n}
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    ctx, new = _lengths(case)
    T = sum(new)
    if case["op"] == "append":
        return {"bytes": 2 * T * (nq + 2 * nkv) * d * size + 8 * case["batch"],
                "flops": T * (nq + nkv) * d * (3 + 4 * case["norm"])}
    w = case["window"] or 1 << 40
    seen = sum(min(c + n, w + n - 1) for c, n in zip(ctx, new) if n)
    pairs = sum(sum(min(c + i + 1, w) for i in range(n)) for c, n in zip(ctx, new))
    return {"bytes": 2 * seen * nkv * d * size + T * nq * (2 * d * size + 4), "flops": 4 * pairs * nq * d}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "logprobs": _exact_logprobs}[case["op"]](case, st)


def _exact_append(case, st):
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    k, v, q = st.k.double(), st.v.double(), []
    x = st.qkv.double()
    freq = torch.tensor([BASE ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device="cuda")
    ctx, cu, table = st.ctx.tolist(), st.cu.tolist(), st.table.tolist()
    turn = None

    def head(y, gain):
        if case["norm"]:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * gain.double()
        z = torch.complex(y[..., :d // 2].contiguous(), y[..., d // 2:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    for b in range(len(ctx)):
        at = cu[b]
        while at < cu[b + 1]:   # the tokens of one page at a time
            p0 = ctx[b] + at - cu[b]
            m = min(cu[b + 1] - at, PAGE - p0 % PAGE)
            page, s0 = table[b][p0 // PAGE], p0 % PAGE
            ang = torch.arange(p0, p0 + m, device="cuda").double()[:, None] * freq
            turn = torch.complex(ang.cos(), ang.sin())[:, None]
            y = x[at:at + m].view(m, -1, d)
            q.append(head(y[:, :nq], st.g_q).reshape(m, nq * d))
            k[0, page, :, s0:s0 + m] = head(y[:, nq:nq + nkv], st.g_k).transpose(0, 1)
            v[0, page, :, :, s0:s0 + m] = y[:, nq + nkv:].permute(1, 2, 0)
            at += m
    return {"q": torch.cat(q), "k": k, "v": v}


def _exact_attend(case, st):
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    ctx, cu = st.ctx.tolist(), st.cu.tolist()
    out, lse = [], []
    for b in range(len(ctx)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        L = ctx[b] + n
        pages = st.table[b, :-(-L // PAGE)].long()
        k = st.k[0, pages].double().permute(1, 0, 2, 3).reshape(nkv, -1, d)[:, :L]
        v = st.v[0, pages].double().permute(1, 0, 3, 2).reshape(nkv, -1, d)[:, :L]
        q = st.q[cu[b]:cu[b + 1]].double().view(n, nkv, nq // nkv, d)
        o_b, l_b = [], []
        for h in range(nkv):
            s = torch.einsum("igd,td->igt", q[:, h], k[h]) / math.sqrt(d)
            for i in range(n):
                lo = max(0, ctx[b] + i + 1 - case["window"]) if case["window"] else 0
                s[i, :, :lo] = -math.inf
                s[i, :, ctx[b] + i + 1:] = -math.inf
            l_b.append(torch.logsumexp(s, -1))
            o_b.append(torch.einsum("igt,td->igd", (s - l_b[-1][..., None]).exp(), v[h]))
        out.append(torch.stack(o_b, 1).reshape(n, nq * d))
        lse.append(torch.stack(l_b, 1).reshape(n, nq))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_logprobs(case, st):
    rows = case["rows"]
    got = {"logprob": torch.zeros(rows, dtype=torch.float64, device="cuda"),
           "entropy": torch.zeros(rows, dtype=torch.float64, device="cuda"), "rank": None, "top_ids": None,
           "top_logprobs": torch.zeros(rows, 16, dtype=torch.float64, device="cuda")}
    ids = st.ids.tolist()
    for r in range(rows):
        if ids[r] < 0:
            continue
        y = st.logits[r].double() / case["temp"]
        lp = y - torch.logsumexp(y, 0)
        got["logprob"][r] = lp[ids[r]]
        got["entropy"][r] = -torch.xlogy(lp.exp(), lp.exp()).sum()
        got["top_logprobs"][r] = lp.topk(16).values
    return got
