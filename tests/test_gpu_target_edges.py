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
