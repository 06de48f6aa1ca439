"""Attention of a batch that shares a prefix, on the GPU against the fp64 oracle
of plain attention over each request's whole context.  u(t) is half a step of
type t (its rounding error relative to the value): bf16 2^-8, fp32 2^-24."""
import numpy as np
import pytest

from oracle import target_oracle as O
from tests.test_gpu_target import PAGE, U, Batch, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_diffusion_drafter_context_gb300.build import build
    build()


@pytest.fixture(autouse=True, params=[1, 2], ids=["one launch", "prefix apart"])
def launches(request, built):
    """Every test in both forms, whatever the prefix's length would choose."""
    from block_diffusion_drafter_context_gb300 import binding as B
    B.dflash_debug_shared_launches(request.param)
    yield request.param
    B.dflash_debug_shared_launches(0)


class Shared(Batch):
    """A Batch whose requests share their first `pages` pages: the kernels get
    them in the first request's row alone (the other rows hold -1 there)."""

    def __init__(self, nq, nkv, d, dtype, pages, own, new, **kw):
        from block_diffusion_drafter_context_gb300.drafter import PagedKV
        from block_diffusion_drafter_context_gb300.target import TargetOps
        import torch
        super().__init__(nq, nkv, d, dtype, [pages * PAGE + c for c in own], new, **kw)
        self.prefix = pages * PAGE
        self.table[1:, :pages] = -1
        self.kv = PagedKV.from_tensors(self.k, self.v, torch.from_numpy(self.table).cuda())
        self.table[1:, :pages] = self.table[0, :pages]      # what the oracle reads
        self.ops = TargetOps(nq, nkv, d, dtype=dtype, max_batch=len(own), max_new=kw.get("max_new", 16),
                             shared_prefix=True)

    def attend(self, q=None, **kw):
        return self.ops.attend_shared(self.kv, 1, self.q if q is None else q, self.cu_d, self.ctx_d, self.prefix,
                                      want_lse=True, **kw)

    def check(self, out, lse, rows=None, q=None, scale=None):
        """As Batch.check_attention, with 2^-20 more for the join's two factors
        (exp2 and the product before it, 2^-22 each) and its sums."""
        ref, rlse, spread = self.attend_ref(q, scale=scale)
        own = np.arange(self.T) if rows is None else np.asarray(rows)
        q64 = np64(self.q if q is None else q)[own].reshape(len(own), self.nq, self.d)
        sc = self.d ** -0.5 if scale is None else scale
        kmax = np.nanmax(np.abs(np64(self.k[1])))
        n = max(c + m for c, m in zip(self.ctx, self.new))
        e = 2 * self.d * 2.0 ** -24 * np.abs(q64).sum(-1).max() * kmax * sc + n * 2.0 ** -24 + 2.0 ** -19
        got, glse = np64(out)[own], np64(lse)[own]
        tol = ((U["bf16"] if self.dtype == "bf16" else 0) + e) * spread[own] + U[self.dtype] * np.abs(ref[own]) + 1e-30
        assert np.isfinite(got).all()
        assert (np.abs(got - ref[own]) <= tol).all(), np.max(np.abs(got - ref[own]) / tol)
        dead = np.isneginf(rlse[own])
        assert (np.isneginf(glse) == dead).all()
        assert (np.abs(glse[~dead] - rlse[own][~dead]) <= e + 2.0 ** -22 * (1 + np.abs(rlse[own][~dead]))).all()


SHAPES = [(8, 2, 128, "bf16"), (5, 1, 128, "bf16"), (16, 2, 64, "bf16"), (4, 4, 128, "bf16"), (14, 2, 128, "bf16"),
          (4, 2, 64, "f32"), (6, 1, 128, "f32"), (8, 8, 64, "f32")]


@pytest.mark.parametrize("nq,nkv,d,dtype", SHAPES)
@pytest.mark.parametrize("pages,own,new", [
    (1, [0, 5], [1, 1]),                                    # a row each, one page
    (3, [0, 63, 64, 130, 7], [1, 0, 1, 1, 1]),              # decode; a request without tokens
    (2, [10, 0, 200, 61, 64, 0], [16, 3, 0, 9, 1, 16]),     # verification
    (17, [0, 1, 2], [16, 16, 16]),                          # more pages than a cluster's share
])
def test_matches_oracle(nq, nkv, d, dtype, pages, own, new):
    c = Shared(nq, nkv, d, dtype, pages, own, new, seed=nq + d + pages)
    out, lse = c.attend()
    assert c.ops.status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("nq,nkv,d,batch,new,dtype", [
    (8, 1, 128, 40, 16, "bf16"), (5, 1, 128, 33, 13, "bf16"), (12, 4, 64, 61, 7, "bf16"), (7, 1, 64, 70, 1, "bf16"),
    (4, 2, 64, 30, 5, "f32")])
def test_many_rows(nq, nkv, d, batch, new, dtype):
    """Rows of many requests in the prefix's tiles, the last one not full."""
    own = [(37 * b) % 150 for b in range(batch)]
    c = Shared(nq, nkv, d, dtype, 9, own, [(b * 5) % new + 1 for b in range(batch)], seed=d, pad_rows=3)
    out, lse = c.attend()
    assert c.ops.status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_rows_and_slices(dtype):
    """A slice of a batch (cu_new not from 0): rows before and behind it hold
    NaN and their results stay as they were."""
    import torch
    c = Shared(8, 2, 64, dtype, 4, [3, 70, 0, 40, 5, 9], [3, 16, 2, 5, 1, 16], pad_rows=4, seed=3)
    for lo, hi in ((0, 6), (2, 5), (1, 2), (5, 6)):
        q = c.q.clone()
        a, b = int(c.cu[lo]), int(c.cu[hi])
        q[:a], q[b:] = float("nan"), float("nan")
        out = torch.full_like(q, 7.0)
        lse = torch.full((q.shape[0], 8), 7.0, device="cuda")
        from block_diffusion_drafter_context_gb300.drafter import PagedKV
        table = torch.from_numpy(c.table[lo:hi]).cuda()
        kv = PagedKV.from_tensors(c.k, c.v, table)
        c.ops.attend_shared(kv, 1, q, c.cu_d[lo:hi + 1].contiguous(), c.ctx_d[lo:hi].contiguous(), c.prefix, out=out,
                            lse=lse)
        assert c.ops.status() == 0
        c.check(out, lse, rows=range(a, b))
        left = torch.cat([out[:a], out[b:]])
        assert (left == 7.0).all() and (torch.cat([lse[:a], lse[b:]]) == 7.0).all()


def test_a_page_multiple_of_zero_is_plain_attention():
    import torch
    c = Shared(8, 2, 128, "bf16", 0, [100, 3], [16, 2])
    out, lse = c.attend()
    out2, lse2 = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def exact(c):
    """(out, lse, sum p |v|) in fp64 on the device."""
    import torch
    table = torch.from_numpy(c.table).cuda().long()
    out = torch.empty(c.T, c.nq, c.d, dtype=torch.float64, device="cuda")
    lse, spread = torch.empty(c.T, c.nq, dtype=torch.float64, device="cuda"), torch.empty_like(out)
    g = c.nq // c.nkv
    for b in range(len(c.ctx)):
        n, L = c.new[b], c.ctx[b] + c.new[b]
        if n == 0:
            continue
        pages = table[b, :-(-L // PAGE)]
        rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
        for h in range(c.nkv):
            k = c.k[1, pages, h].double().reshape(-1, c.d)[:L]
            v = c.v[1, pages, h].double().permute(0, 2, 1).reshape(-1, c.d)[:L]
            q = c.q[rows].double().view(n, c.nq, c.d)[:, h * g:(h + 1) * g]
            s = torch.einsum("igd,td->igt", q, k) * c.d ** -0.5
            hide = torch.arange(L, device="cuda") > c.ctx[b] + torch.arange(n, device="cuda")[:, None]
            s.masked_fill_(hide[:, None], -float("inf"))
            l = torch.logsumexp(s, -1)
            p = (s - l[..., None]).exp()
            out[rows, h * g:(h + 1) * g], spread[rows, h * g:(h + 1) * g] = p @ v, p @ v.abs()
            lse[rows, h * g:(h + 1) * g] = l
    return out, lse, spread


@pytest.mark.parametrize("nq,nkv,d,dtype,batch,pages,new", [
    (40, 8, 128, "bf16", 64, 33, 16),     # 160 tiles of 256 rows: one each and 8 that are cut, an odd number of pages
    (32, 8, 128, "bf16", 64, 128, 1),     # a tile per head, cut into 19
    (8, 8, 64, "bf16", 50, 300, 1),       # rows for less than a tile
    (8, 1, 128, "bf16", 21, 511, 7),      # one head, tiles that end inside
    (16, 2, 64, "bf16", 200, 16, 16),     # many tiles of few pages
    (6, 1, 128, "bf16", 3, 1025, 16),     # few rows on a long prefix
    (3, 3, 64, "bf16", 5, 40, 1),         # 16-row tiles
    (16, 8, 128, "f32", 40, 60, 1), (4, 1, 64, "f32", 12, 201, 16)])
def test_long_prefixes(nq, nkv, d, dtype, batch, pages, new):
    """Against fp64 on the device, tolerances as in Shared.check; three calls
    with the same bits."""
    import torch
    own = [(b * 61) % 300 for b in range(batch)]
    c = Shared(nq, nkv, d, dtype, pages, own, [1 + (b * 7) % new for b in range(batch)], seed=pages, stale=0.0)
    out, lse = c.attend()
    for _ in range(2):
        again = c.attend()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert c.ops.status() == 0
    ref, rlse, spread = exact(c)
    size = float(c.q.double().abs().view(c.T, nq, d).sum(-1).max() * c.k[1].abs().max()) * d ** -0.5
    e = 2 * d * 2.0 ** -24 * size + (max(c.ctx) + 16) * 2.0 ** -24 + 2.0 ** -19
    tol = ((U["bf16"] if dtype == "bf16" else 0) + e) * spread + U[dtype] * ref.abs() + 1e-30
    got = out.double().view(c.T, nq, d)
    assert ((got - ref).abs() <= tol).all(), float(((got - ref).abs() / tol).max())
    assert ((lse.double() - rlse).abs() <= e + 2.0 ** -22 * (1 + rlse.abs())).all()


def test_missing_pages_at_both_ends_of_a_long_prefix():
    """The first, the last and a pair of pages in between are not there, for rows
    of several tiles."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    c = Shared(8, 1, 128, "bf16", 31, [10 * b for b in range(40)], [9] * 40, seed=12, stale=0.0)
    for hole in (0, 12, 13, 30):
        c.table[:, hole] = -1
    c.kv = PagedKV.from_tensors(c.k, c.v, torch.from_numpy(c.table).cuda())
    out, lse = c.attend()
    assert c.ops.status() == -7
    c.check(out, lse)


def test_the_choice_by_length():
    """What the library chooses by itself agrees with both forms."""
    from block_diffusion_drafter_context_gb300 import binding as B
    B.dflash_debug_shared_launches(0)
    for pages, batch in ((2, 4), (400, 30)):
        c = Shared(8, 1, 128, "bf16", pages, [40] * batch, [2] * batch, seed=3, stale=0.0)
        out, lse = c.attend()
        ref, rlse, spread = exact(c)
        assert c.ops.status() == 0
        assert ((out.double().view(c.T, 8, 128) - ref).abs() <= 2.0 ** -7 * (spread + ref.abs())).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_missing_pages_and_bad_requests(dtype):
    """A hole in the prefix and one in an own part drop their positions; a
    request that lies before the prefix's end is left unwritten."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    c = Shared(4, 1, 128, dtype, 5, [70, 9, 130], [16, 4, 1], seed=5)
    c.table[:, 2] = -1
    c.table[2, 6] = 10 ** 6
    c.kv = PagedKV.from_tensors(c.k, c.v, torch.from_numpy(c.table).cuda())
    out, lse = c.attend()
    assert c.ops.status() == -7
    c.check(out, lse)
    ctx = c.ctx_d.clone()
    ctx[1] = c.prefix - 1
    out, lse = torch.full_like(c.q, 7.0), torch.full((c.T, 4), 7.0, device="cuda")
    c.ops.attend_shared(c.kv, 1, c.q, c.cu_d, ctx, c.prefix, out=out, lse=lse)
    assert c.ops.status() == -7
    c.check(out, lse, rows=[*range(16), 20])
    assert (out[16:20] == 7.0).all() and (lse[16:20] == 7.0).all()
    # nothing but holes: the prefix, and all of a request's own pages
    c.table[:, :5] = -1
    c.table[2] = -1
    c.kv = PagedKV.from_tensors(c.k, c.v, torch.from_numpy(c.table).cuda())
    out, lse = c.attend()
    assert c.ops.status() == -7 and (out[20] == 0).all() and torch.isneginf(lse[20]).all()
    c.check(out, lse)


def test_a_batch_with_too_many_rows():
    """A request above max_new pushes the others' rows behind batch * max_new:
    those are reported and left unwritten, the ones before are right."""
    import torch
    c = Shared(4, 1, 128, "bf16", 2, [5, 6, 7], [2, 9, 2], seed=8, max_new=2)
    out, lse = torch.full_like(c.q, 7.0), torch.full((c.T, 4), 7.0, device="cuda")
    c.ops.attend_shared(c.kv, 1, c.q, c.cu_d, c.ctx_d, c.prefix, out=out, lse=lse)
    assert c.ops.status() == -7
    c.check(out, lse, rows=[0, 1])
    assert (out[2:] == 7.0).all() and (lse[2:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_queries_stay_in_their_rows(dtype):
    import torch
    c = Shared(8, 1, 128, dtype, 3, [70, 9], [16, 16], seed=6)
    q = c.q.clone()
    q[3], q[20] = float("nan"), float("inf")
    out, lse = c.attend(q=q)
    for r in (3, 20):
        assert torch.isnan(out[r]).all() and torch.isnan(lse[r]).all()
    c.check(out, lse, rows=[r for r in range(32) if r not in (3, 20)])


def test_scores_that_grow_along_the_prefix():
    """Maxima that move by far more than 2^8 from page to page, and own parts
    far above and far below the prefix."""
    c = Shared(8, 2, 128, "bf16", 6, [70, 9, 200], [16, 4, 1], seed=7)
    for p in range(6):
        c.k[1, int(c.table[0, p])] *= 1.0 + p
    for p in range(6, 11):
        if c.table[2, p] >= 0:
            c.k[1, int(c.table[2, p])] *= 20
        if 0 <= c.table[0, p]:
            c.k[1, int(c.table[0, p])] *= 0.01
    out, lse = c.attend()
    c.check(out, lse)


@pytest.mark.parametrize("new,dtype", [(1, "bf16"), (16, "bf16"), (3, "f32")])
def test_same_bits_and_a_captured_call(new, dtype):
    """Three calls and replays of a captured one with other contents: the same
    bits as eager calls, on a workspace that plain attention uses in between."""
    import torch
    c = Shared(8, 2, 128, dtype, 20, [100 + 9 * b for b in range(20)], [new] * 20, seed=9)
    out, lse = c.attend()
    for _ in range(2):
        out2, lse2 = c.attend()
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    q = c.q.clone()
    o, l = torch.empty_like(out), torch.empty_like(lse)
    c.attend(q=q, out=o, lse=l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(q=q, out=o, lse=l)
    other = torch.randn_like(q)
    for x in (other, c.q):
        q.copy_(x)
        g.replay()
        eager, elser = c.attend(q=x)
        assert torch.equal(o, eager) and torch.equal(l, elser)
    assert c.ops.status() == 0
    c.check(o, l)


def test_on_another_stream():
    import torch
    c = Shared(8, 2, 128, "bf16", 8, [100, 3], [16, 2], seed=4)
    want, wl = c.attend()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        out, lse = c.attend(stream=s)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)


def test_strided_queries_and_scale():
    import torch
    c = Shared(8, 2, 64, "bf16", 3, [10, 80], [16, 5], seed=2)
    wide = torch.full((c.T, 8 * 64 + 24), float("nan"), dtype=c.dt, device="cuda")
    wide[:, :512] = c.q
    out, lse = c.attend(q=wide[:, :512], scale=0.3)
    c.check(out, lse, scale=0.3)
