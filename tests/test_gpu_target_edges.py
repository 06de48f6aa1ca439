"""Target-side operators on the GPU where they can go wrong at the edges: rows
without a finite score, pages and requests that are not there in the form of
the attention that cuts its work into runs, positions near 2^24, rows of
logits with few tokens left.  The oracle is fp64; u(t) as in
test_gpu_target."""
import numpy as np
import pytest

from oracle import target_oracle as O
from tests.test_gpu_target import PAGE, U, Batch, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_diffusion_drafter_context_gb300.build import build
    build()


def widen(c, pages=300):
    """The same cache behind a page table `pages` wide: more than 16 pages for
    each of a cluster's 16 CTAs at most, so that the call cuts its pages into
    runs."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    table = np.full((len(c.ctx), max(pages, c.table.shape[1])), -1, dtype=np.int32)
    table[:, :c.table.shape[1]] = c.table
    c.table = table
    c.kv = PagedKV.from_tensors(c.k, c.v, torch.from_numpy(table).cuda())
    return c


FORMS = [(8, 2, 128, "bf16"), (16, 2, 64, "bf16"), (16, 2, 128, "bf16"), (4, 1, 128, "f32"), (4, 2, 64, "f32")]


@pytest.mark.parametrize("nq,nkv,d,dtype", FORMS)
@pytest.mark.parametrize("ctx,new,window", [([0], [1], 0), ([70, 200, 3], [1, 1, 1], 1), ([0, 63], [16, 3], 0),
                                            ([130, 0, 64], [16, 1, 2], 2), ([300, 1], [9, 1], 64)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), -3e38])
def test_a_row_of_nothing_but_infinite_scores_is_nan(nq, nkv, d, dtype, ctx, new, window, wide, value):
    """One component of every key is above 2, so that a query with an infinity
    there (or one whose products overflow) has every score at the same
    infinity: a score of -inf everywhere must not look like a row that sees
    nothing (out 0, lse -inf)."""
    import torch
    c = Batch(nq, nkv, d, dtype, ctx, new, seed=nq + d + len(ctx), window=window, max_new=max(new))
    c.k[..., 5] = c.k[..., 5].abs() + 2
    if wide:
        widen(c)
    good, good_lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, window=window, want_lse=True)
    q = c.q.clone()
    spoiled = torch.zeros_like(good, dtype=torch.bool)
    for row, head in ((0, nq - 1), (c.T - 1, 0)):
        q[row, head * d + 5] = value
        spoiled[row, head * d:(head + 1) * d] = True
    out, lse = c.ops.attend(c.kv, 1, q, c.cu_d, c.ctx_d, window=window, want_lse=True)
    assert c.ops.status() == 0
    assert torch.equal(out.isnan(), spoiled) and torch.equal(lse.isnan(), spoiled[:, ::d])
    c.check_attention(torch.where(spoiled, good, out), torch.where(spoiled[:, ::d], good_lse, lse))


@pytest.mark.parametrize("nq,nkv,d,dtype", FORMS)
@pytest.mark.parametrize("new", [1, 16])
@pytest.mark.parametrize("wide", [False, True])
def test_overflow_to_minus_infinity_at_some_keys_alone(nq, nkv, d, dtype, new, wide):
    """Scores of -inf beside finite ones have probability 0: the first 3 pages
    and every second key behind them, the newest token's finite."""
    import torch
    c = Batch(nq, nkv, d, dtype, [280, 260], [new, 1], seed=nq + new, max_new=new)
    c.q[..., 5::d] = -3e38
    c.k[..., 5] = 0
    for b in range(2):
        for p in range(-(-(c.ctx[b] + c.new[b]) // PAGE)):
            live = min(PAGE, c.ctx[b] + c.new[b] - p * PAGE)
            at = torch.arange(live, device="cuda")
            low = at < PAGE if p < 3 else (at % 2 == 1) & (p * PAGE + at < c.ctx[b])
            c.k[1, int(c.table[b, p]), :, :live, 5] = torch.where(low, 4.0, 0.0).to(c.dt)
    if wide:
        widen(c)
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == 0
    # the reference: keys with the component, left out (their V too), on the finite rest of the query
    q = c.q.clone()
    q[..., 5::d] = 0
    k, v = np64(c.k[1]), np64(c.v[1])
    ref, rlse, spread = [], [], []
    for b in range(2):
        for i in range(c.new[b]):
            t, keys = int(c.cu[b]) + i, np.arange(c.ctx[b] + i + 1)
            pages, slots = c.table[b, keys // PAGE], keys % PAGE
            keep = k[pages, 0, slots, 5] == 0
            for h in range(nq):
                kk, vv = k[pages[keep], h // (nq // nkv), slots[keep]], v[pages[keep], h // (nq // nkv), :, slots[keep]]
                s = kk @ np64(q[t, h * d:(h + 1) * d]) * d ** -0.5
                e = np.exp(s - s.max())
                ref.append(e @ vv / e.sum())
                spread.append(e @ np.abs(vv) / e.sum())
                rlse.append(s.max() + np.log(e.sum()))
    shape = (c.T, nq * d)
    ref, spread, rlse = np.reshape(ref, shape), np.reshape(spread, shape), np.reshape(rlse, (c.T, nq))
    # as in Batch.check_attention
    kmax = np.nanmax(np.abs(k))
    e = 2 * d * 2.0 ** -24 * np.abs(np64(q)).reshape(c.T, nq, d).sum(-1).max() * kmax * d ** -0.5 + 300 * 2.0 ** -24 + 2.0 ** -20
    tol = ((U["bf16"] if dtype == "bf16" else 0) + e) * spread + U[dtype] * np.abs(ref) + 1e-30
    assert (np.abs(np64(out) - ref) <= tol).all()
    assert (np.abs(np64(lse) - rlse) <= e + 2.0 ** -22 * (1 + np.abs(rlse))).all()


# ------------------------------------------------------------------ the form that cuts the pages into runs
def bad_pages(which, n):
    """Page numbers of a request of n pages.  A run is 2 pages at least (4 in
    the wider tiles), so 11 in a row are some CTA's whole part."""
    return {"first": [0], "last": [n - 1], "a whole part": list(range(20, 31)), "both ends": [0, 1, n - 2, n - 1],
            "every": list(range(n)), "alternate": list(range(0, n, 2))}[which]


@pytest.mark.parametrize("nq,nkv,d,dtype", FORMS)
@pytest.mark.parametrize("new", [1, 9])
@pytest.mark.parametrize("which", ["first", "last", "a whole part", "both ends", "every", "alternate"])
def test_missing_pages_in_runs(nq, nkv, d, dtype, new, which):
    """A request of 94 pages that lost some, between two whole ones: the lost
    positions drop out, a token left without any gets out 0 and lse -inf, the
    others keep their bits."""
    import torch
    c = widen(Batch(nq, nkv, d, dtype, [700, 6000, 90], [1, new, 2], seed=new + d, max_new=max(2, new)))
    whole, whole_lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == 0
    lost = bad_pages(which, -(-(6000 + new) // PAGE))
    c.table[1, lost] = [(-7, 1 << 20, c.k.shape[1])[i % 3] for i in range(len(lost))]
    widen(c)
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == -7 and c.ops.status() == 0
    c.check_attention(out, lse)
    rows = torch.ones(c.T, dtype=torch.bool, device="cuda")
    rows[1:1 + new] = False
    assert torch.equal(out[rows], whole[rows]) and torch.equal(lse[rows], whole_lse[rows])
    again, lse2 = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == -7 and torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("nq,nkv,d,dtype", FORMS)
@pytest.mark.parametrize("what", ["context", "too many", "capacity"])
def test_requests_out_of_range_in_runs(nq, nkv, d, dtype, what):
    """Invalid requests first, in the middle (two in a row) and last in a batch
    of long ones: reported, their rows unwritten, the others right."""
    import torch
    ctx, new = [400, 2500, 64, 1000, 3000, 200], [3, 2, 3, 3, 1, 3]
    c = widen(Batch(nq, nkv, d, dtype, ctx, new, seed=d, pad_rows=2))
    good, good_lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == 0
    c.check_attention(good, good_lse)
    bad, max_new, at = [0, 2, 3, 5], 16, c.ctx_d.clone()
    if what == "too many":
        max_new = 2
    else:   # 300 pages hold 19 200 positions
        at[bad] = torch.tensor([-1, 2 ** 31 - 1, -2 ** 31, 300 * PAGE - 2] if what == "context" else [300 * PAGE - 2] * 4,
                               dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(good, 7.0), torch.full_like(good_lse, 7.0)
    c.ops.attend(c.kv, 1, c.q, c.cu_d, at, max_new=max_new, out=out, lse=lse)
    assert c.ops.status() == -7 and c.ops.status() == 0
    left = torch.ones(c.T + 2, dtype=torch.bool, device="cuda")
    for b in (1, 4):
        left[int(c.cu[b]):int(c.cu[b + 1])] = False
    assert (out[left] == 7).all() and (lse[left] == 7).all()
    out[left], lse[left] = good[left], good_lse[left]
    c.check_attention(out, lse)


@pytest.mark.parametrize("nq,nkv,d,dtype", FORMS)
@pytest.mark.parametrize("new", [1, 6])
def test_a_common_prefix_in_runs(nq, nkv, d, dtype, new):
    """Three requests that share their first 40 pages."""
    c = Batch(nq, nkv, d, dtype, [3000, 2600, 4000], [new] * 3, seed=new, max_new=new)
    c.table[1:, :40] = c.table[0, :40]
    widen(c)
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == 0
    c.check_attention(out, lse)


# ------------------------------------------------------------------ far positions
@pytest.mark.parametrize("base", [1.0001, 2.0, 10.0, 1e4, 5e5, 1e6])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first,bound", [(0, 4e-7), (2 ** 17 - 4096, 4e-7), (2 ** 20 - 4096, 4e-7), (2 ** 22 - 8192, 4e-7),
                                         (2 ** 23 - 4096, 8.5e-7), (15339979 - 4096, 8.5e-7), (2 ** 24 - 8192, 8.5e-7)])
def test_rotation_angles(base, d, first, bound):
    """Heads of (1, 0) pairs come out as the cosines and sines themselves, so
    each is off by the angle's error and sincosf's 2 ulp (2^-23) at most: 8192
    positions from `first` on, every pair, against the angle in 64 bits."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    from block_diffusion_drafter_context_gb300.target import TargetOps
    n, page0 = 8192, first // PAGE
    table = torch.full((1, 2 ** 18), -1, dtype=torch.int32, device="cuda")
    count = (first + n - 1) // PAGE - page0 + 1
    table[0, page0:page0 + count] = torch.arange(count, device="cuda", dtype=torch.int32)
    k, v = (torch.zeros(1, count, 1, *s, device="cuda") for s in ((PAGE, d), (d, PAGE)))
    x = torch.zeros(n, 3 * d, device="cuda")
    x[:, :d // 2] = 1
    x[:, d:d + d // 2] = 1
    ops = TargetOps(1, 1, d, dtype="f32", max_batch=1, rope_base=base)
    q = ops.append_kv(PagedKV.from_tensors(k, v, table), 0, x, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                      torch.tensor([first], dtype=torch.int32, device="cuda"))
    assert ops.status() == 0
    # the base is an fp32 argument; fp64 angles are off by 2^24 * 2^-52 = 4e-9
    theta = float(np.float32(base)) ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d)
    pos = torch.arange(first, first + n, device="cuda")
    angle = pos.double()[:, None] * theta
    ref = torch.cat([angle.cos(), angle.sin()], 1)
    assert (q.double() - ref).abs().max() <= bound + 2.0 ** -23 + 1e-8
    assert torch.equal(k[0, (pos // PAGE) - page0, 0, pos % PAGE], q)     # the key's head is the same pairs


# ------------------------------------------------------------------ log probabilities with few tokens left
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(1, 151936), (5, 40001), (40, 20000), (650, 9000)])
@pytest.mark.parametrize("alive", [1, 2, 5, 15, 16, 17])
def test_logprobs_of_rows_with_few_finite_logits(dtype, rows, V, alive):
    """A grammar's mask: 1 to 17 finite logits in rows cut over clusters and in
    rows of one CTA; the places behind them are -inf logits, lowest ids first."""
    import torch
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    rng = np.random.default_rng(rows + V + alive)
    x = np.full((rows, V), -np.inf, dtype=np.float32)
    for r in range(rows):
        # the ends of the row and the first ids among them in every third row
        at = rng.choice(V, alive, replace=False)
        if r % 3 == 0:
            at = np.unique(np.concatenate([[0, V - 1, 3, V - 2], rng.choice(V, alive, replace=False)])[:alive])
        x[r, at] = rng.standard_normal(len(at)) * 3
    x = torch.from_numpy(x).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    ids = rng.integers(0, V, rows)
    ids[::2] = np64(x).argmax(1)[::2]
    got = token_logprobs(x, torch.from_numpy(ids.astype(np.int32)).cuda(), temperature=0.7)
    got = {k: v.cpu().numpy() for k, v in got.items()}
    x64 = np64(x)
    for r in list(range(min(rows, 6))) + ([rows - 1] if rows > 6 else []):
        lp, ent, rank, top, top_lp = O.token_logprobs(x64[r], ids[r], 0.7, 16)
        assert got["rank"][r] == rank and list(got["top_ids"][r]) == top, r
        # fp32: logits up to 15 / 0.7 scaled (2 roundings each), 17 summands, exp2 and log2 to 2^-21
        e = (6 * 22 + 17 + 32) * 2.0 ** -24
        assert got["logprob"][r] == lp if np.isinf(lp) else abs(got["logprob"][r] - lp) <= 2 * e
        assert abs(got["entropy"][r] - ent) <= 3 * e * 5
        inf = np.isinf(top_lp)
        assert np.array_equal(np.isneginf(got["top_logprobs"][r]), inf)
        assert (np.abs(got["top_logprobs"][r][~inf] - top_lp[~inf]) <= 2 * e).all()


# ------------------------------------------------------------------ streams
@pytest.mark.parametrize("nq,nkv,d,dtype", [(8, 2, 128, "bf16"), (16, 2, 128, "bf16"), (4, 2, 64, "f32")])
def test_a_new_object_is_used_on_another_stream_at_once(nq, nkv, d, dtype):
    """The workspace's memory held something else, and the stream it is made on
    is busy for a while: the first call on another stream finds it cleared."""
    import torch
    from block_diffusion_drafter_context_gb300.target import TargetOps
    new = 16 if dtype == "bf16" else 2
    c = widen(Batch(nq, nkv, d, dtype, [9000, 300], [new, 1], seed=3))
    want, want_lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    side = torch.cuda.Stream()
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    size = c.ops.ws_bytes
    del c.ops
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.full((size,), 0x55, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del old
    torch.cuda._sleep(200_000_000)      # about 0.1 s
    ops = TargetOps(nq, nkv, d, dtype=dtype, max_batch=2)
    ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, out=out, lse=lse, stream=side)
    torch.cuda.synchronize()
    assert ops.status() == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


# ------------------------------------------------------------------ a part of a batch
@pytest.mark.parametrize("nq,nkv,d,dtype", FORMS)
@pytest.mark.parametrize("new", [[3, 2, 1, 4, 2], [16, 16, 5, 7, 16], [30, 70, 9, 1, 50]])
@pytest.mark.parametrize("wide", [False, True])
def test_the_requests_of_a_slice(nq, nkv, d, dtype, new, wide):
    """Requests 2 and 3 alone, by slices of cu_new, ctx_len and the page table
    and the whole batch's rows: what the whole batch gives in their rows and
    slots, nothing reported, every other row and slot as it was."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    c = Batch(nq, nkv, d, dtype, [100, 7, 250, 60, 0], new, seed=d + new[0], stale=0.0, pad_rows=2)
    if wide:
        widen(c)
    k0, v0 = c.k.clone(), c.v.clone()
    few = max(new) <= 16
    q = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k)
    out = c.ops.attend(c.kv, 1, q, c.cu_d, c.ctx_d) if few else None
    k1, v1 = c.k.clone(), c.v.clone()
    c.k.copy_(k0), c.v.copy_(v0)
    kv = PagedKV.from_tensors(c.k, c.v, c.kv.page_table[2:4])
    cu, ctx = c.cu_d[2:5], c.ctx_d[2:4]
    q2 = torch.full_like(q, 7.0)
    c.ops.append_kv(kv, 1, c.qkv, cu, ctx, c.g_q, c.g_k, q_out=q2)
    assert c.ops.status() == 0
    mine = torch.zeros(c.T + 2, dtype=torch.bool, device="cuda")
    mine[int(c.cu[2]):int(c.cu[4])] = True
    assert torch.equal(q2[mine], q[mine]) and (q2[~mine] == 7).all()
    pages = [int(p) for b in (2, 3) for p in c.table[b] if p >= 0]
    rest = [p for p in range(c.k.shape[1]) if p not in pages]
    assert torch.equal(c.k[1, pages], k1[1, pages]) and torch.equal(c.v[1, pages], v1[1, pages])
    assert torch.equal(c.k[1, rest], k0[1, rest]) and torch.equal(c.v[1, rest], v0[1, rest])
    assert torch.equal(c.k[0], k0[0]) and torch.equal(c.v[0], v0[0])
    if few:
        out2, lse2 = torch.full_like(out, 7.0), torch.full((c.T + 2, nq), 7.0, device="cuda")
        c.ops.attend(kv, 1, q2, cu, ctx, out=out2, lse=lse2)
        assert c.ops.status() == 0
        assert (out2[~mine] == 7).all() and (lse2[~mine] == 7).all()
        out2[~mine], lse2[~mine] = 0, 0
        want, want_lse, spread = c.attend_ref(q)
        # the roundings of Batch.check_attention, kept apart because only two requests are there
        q64 = np64(q)[:c.T].reshape(c.T, nq, d)
        e = 2 * d * 2.0 ** -24 * np.abs(q64).sum(-1).max() * np.abs(np64(c.k[1])).max() * d ** -0.5 + 300 * 2.0 ** -24 + 2.0 ** -20
        at = mine.cpu().numpy()
        tol = ((U["bf16"] if dtype == "bf16" else 0) + e) * spread[at] + U[dtype] * np.abs(want[at]) + 1e-30
        assert (np.abs(np64(out2)[at] - want[at]) <= tol).all()
        assert (np.abs(np64(lse2)[at] - want_lse[at]) <= e + 2.0 ** -22 * (1 + np.abs(want_lse[at]))).all()


@pytest.mark.parametrize("which", ["default", "default's handle", "stream", "stream's handle", "current"])
def test_calls_follow_the_stream_they_are_given(which):
    """Inputs that a busy stream has still to write: every call on that stream
    (named as an object or a handle, 0 for the default one) sees them."""
    import torch
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    c = Batch(8, 2, 128, "bf16", [200, 70], [2, 3], seed=2, stale=0.0)
    x, ids = torch.randn(5, 5000, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda")
    k0, v0 = c.k.clone(), c.v.clone()
    q = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k)
    out = c.ops.attend(c.kv, 1, q, c.cu_d, c.ctx_d)
    lp = token_logprobs(x, ids)
    k1, v1 = c.k.clone(), c.v.clone()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    on = torch.cuda.default_stream() if which.startswith("default") else other if which == "current" else side
    given = {"default": on, "default's handle": on.cuda_stream, "stream": on, "stream's handle": on.cuda_stream,
             "current": None}[which]
    assert which != "default's handle" or given == 0
    qkv, logits = torch.zeros_like(c.qkv), torch.zeros_like(x)
    c.k.copy_(k0), c.v.copy_(v0)
    torch.cuda.synchronize()
    with torch.cuda.stream(on):
        torch.cuda._sleep(200_000_000)      # about 0.1 s
        qkv.copy_(c.qkv), logits.copy_(x)
    with torch.cuda.stream(other):          # the current stream, where the calls are not meant to go unless told nothing
        q2 = c.ops.append_kv(c.kv, 1, qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k, stream=given)
        out2 = c.ops.attend(c.kv, 1, q2, c.cu_d, c.ctx_d, stream=given)
        lp2 = token_logprobs(logits, ids, stream=given)
        status = c.ops.status(given)
    torch.cuda.synchronize()
    assert status == 0
    assert torch.equal(q2, q) and torch.equal(out2, out) and torch.equal(c.k, k1) and torch.equal(c.v, v1)
    for key in lp:
        assert torch.equal(lp2[key], lp[key]), key


# ------------------------------------------------------------------ large pools
@pytest.mark.parametrize("nq,nkv,d,dtype,pages", [(16, 8, 128, "bf16", 33500), (40, 8, 128, "bf16", 33500),
                                                  (64, 16, 64, "bf16", 33500), (8, 4, 128, "f32", 66000)])
def test_pages_past_32_bits_of_elements(nq, nkv, d, dtype, pages):
    """The last pages of the second layer of a pool of more than 2^32 elements:
    the same bits as in a small pool."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    c = Batch(nq, nkv, d, dtype, [300, 65, 0], [5, 1, 16], seed=d, stale=0.0)
    k0, v0 = c.k.clone(), c.v.clone()
    q = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k)
    out, lse = c.ops.attend(c.kv, 1, q, c.cu_d, c.ctx_d, want_lse=True)
    used = c.k.shape[1]
    assert 2 * pages * nkv * PAGE * d > 2 ** 32
    k = torch.empty(2, pages, nkv, PAGE, d, dtype=c.dt, device="cuda")
    v = torch.empty(2, pages, nkv, d, PAGE, dtype=c.dt, device="cuda")
    k[1, -used:], v[1, -used:] = k0[1], v0[1]
    table = torch.from_numpy(np.where(c.table >= 0, c.table + pages - used, -1).astype(np.int32)).cuda()
    kv = PagedKV.from_tensors(k, v, table)
    q2 = c.ops.append_kv(kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k)
    out2, lse2 = c.ops.attend(kv, 1, q2, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == 0
    assert torch.equal(q2, q) and torch.equal(out2, out) and torch.equal(lse2, lse)
    assert torch.equal(k[1, -used:], c.k[1]) and torch.equal(v[1, -used:], c.v[1])


@pytest.mark.parametrize("nq,nkv,d,dtype", FORMS)
@pytest.mark.parametrize("wide", [False, True])
def test_queries_with_a_row_stride(nq, nkv, d, dtype, wide):
    """Queries as columns of a wider buffer (a fused projection's, NaN around
    them): the bits of contiguous ones."""
    import torch
    c = Batch(nq, nkv, d, dtype, [300, 65, 0, 1000], [5, 0, 16, 1], seed=d, pad_rows=1)
    if wide:
        widen(c)
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    step = 16 // c.q.element_size()
    for before, behind in ((0, 2 * nkv * d), (step, 0), (3 * step, 5 * step)):
        buf = torch.full((c.T + 1, before + nq * d + behind), float("nan"), dtype=c.dt, device="cuda")
        buf[:, before:before + nq * d] = c.q
        out2, lse2 = c.ops.attend(c.kv, 1, buf[:, before:before + nq * d], c.cu_d, c.ctx_d, want_lse=True)
        assert c.ops.status() == 0
        assert torch.equal(out2[:c.T], out[:c.T]) and torch.equal(lse2[:c.T], lse[:c.T])
