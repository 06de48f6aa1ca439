"""Target-side operators on the GPU against the fp64 oracle: append to the
paged cache, attention over it, token log probabilities, and a step that runs
them together.  u(t) below is half a step of type t (its rounding error
relative to the value): bf16 2^-8, fp32 2^-24."""
import types

import numpy as np
import pytest

from oracle import target_oracle as O

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_diffusion_drafter_context_gb300.build import build
    build()


def np64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """A ragged batch over a scattered paged cache of normal values (two
    layers, the second one used), with NaN in every slot no token owns."""

    def __init__(self, nq, nkv, d, dtype, ctx, new, seed=0, pad_rows=0, hole=None, window=0, stale=float("nan"),
                 max_new=16):
        import torch
        from block_diffusion_drafter_context_gb300.drafter import PagedKV
        from block_diffusion_drafter_context_gb300.target import TargetOps
        self.nq, self.nkv, self.d, self.dtype = nq, nkv, d, dtype
        self.ctx, self.new, self.window = list(ctx), list(new), window
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.T = int(self.cu[-1])
        rng = np.random.default_rng(seed)
        need = [-(-(c + n) // PAGE) for c, n in zip(ctx, new)]
        pool = sum(need) + 2
        ids = rng.permutation(pool)
        self.table = np.full((len(ctx), max(max(need), 1) + 1), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dt = dt
        g = torch.Generator("cuda").manual_seed(seed)
        self.k = torch.full((2, pool, nkv, PAGE, d), stale, dtype=dt, device="cuda")
        self.v = torch.full((2, pool, nkv, d, PAGE), stale, dtype=dt, device="cuda")
        for b in range(len(ctx)):
            for p in range(need[b]):
                page, live = int(self.table[b, p]), min(PAGE, ctx[b] + new[b] - p * PAGE)
                self.k[1, page, :, :live] = torch.randn(nkv, live, d, generator=g, device="cuda").to(dt)
                self.v[1, page, :, :, :live] = torch.randn(nkv, d, live, generator=g, device="cuda").to(dt)
        if hole is not None:   # a page index outside the pool
            self.table[hole[0], hole[1]] = hole[2]
        rows = self.T + pad_rows
        self.qkv = (torch.randn(rows, (nq + 2 * nkv) * d, generator=g, device="cuda") * 1.5).to(dt)
        self.q = (torch.randn(rows, nq * d, generator=g, device="cuda") * 2).to(dt)
        self.g_q = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        self.g_k = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        self.cu_d = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        self.ctx_d = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.kv = PagedKV.from_tensors(self.k, self.v, torch.from_numpy(self.table).cuda())
        self.ops = TargetOps(nq, nkv, d, dtype=dtype, max_batch=len(ctx), max_new=max_new)

    def attend_ref(self, q=None, k=None, v=None, scale=None):
        k = np64(self.k[1]) if k is None else k
        v = np64(self.v[1]) if v is None else v
        return O.attend(k, v, self.table, np64(self.q if q is None else q), self.nq, self.nkv, self.d, self.cu,
                        self.ctx, self.window, self.d ** -0.5 if scale is None else scale)

    def check_attention(self, out, lse, q=None, scale=None):
        """|out - ref| <= u(bf16) (sum p|v|) for the rounded probabilities (bf16
        path) + u(type) |ref| for the output + e sum p|v|, where e bounds the
        relative error of a probability: the score's fp32 sum of d products,
        d 2^-24 sum |q k| scale, twice (score and maximum), the sums over n
        positions n 2^-24, exp2 and scaling 2^-20."""
        ref, rlse, spread = self.attend_ref(q, scale=scale)
        own = slice(0, self.T)
        q64 = np64(self.q if q is None else q)[own].reshape(self.T, self.nq, self.d)
        sc = self.d ** -0.5 if scale is None else scale
        kmax = np.nanmax(np.abs(np64(self.k[1])))
        n = max(c + m for c, m in zip(self.ctx, self.new))
        e = 2 * self.d * 2.0 ** -24 * np.abs(q64).sum(-1).max() * kmax * sc + n * 2.0 ** -24 + 2.0 ** -20
        got, glse = np64(out)[own], np64(lse)[own]
        tol = ((U["bf16"] if self.dtype == "bf16" else 0) + e) * spread[own] + U[self.dtype] * np.abs(ref[own]) + 1e-30
        assert np.isfinite(got).all()
        assert (np.abs(got - ref[own]) <= tol).all(), np.max(np.abs(got - ref[own]) / tol)
        dead = np.isneginf(rlse[own])
        assert (np.isneginf(glse) == dead).all()
        assert (np.abs(glse[~dead] - rlse[own][~dead]) <= e + 2.0 ** -22 * (1 + np.abs(rlse[own][~dead]))).all()


SHAPES = [(8, 2, 128, "bf16"), (5, 1, 128, "bf16"), (16, 2, 64, "bf16"), (4, 4, 128, "bf16"), (4, 2, 64, "f32"),
          (6, 1, 128, "f32"), (8, 8, 64, "f32")]


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("nq,nkv,d,dtype", SHAPES)
@pytest.mark.parametrize("norm", [True, False])
def test_append_matches_oracle(nq, nkv, d, dtype, norm):
    """Ragged pieces: one token, none, a piece that crosses pages, a prompt of
    several tiles; far positions and a padded row stride."""
    import torch
    c = Batch(nq, nkv, d, dtype, ctx=[0, 63, 5, 700, 64], new=[17, 1, 0, 90, 3], seed=nq + d, pad_rows=2)
    wide = torch.zeros(c.T + 2, c.qkv.shape[1] + 64, dtype=c.dt, device="cuda")
    wide[:, :c.qkv.shape[1]] = c.qkv
    k0, v0 = np64(c.k), np64(c.v)
    q_out = torch.full((c.T + 2, nq * d), 7.0, dtype=c.dt, device="cuda")
    q = c.ops.append_kv(c.kv, 1, wide[:, :c.qkv.shape[1]], c.cu_d, c.ctx_d, c.g_q if norm else None,
                        c.g_k if norm else None, q_out=q_out)
    assert c.ops.status() == 0 and q is q_out
    gq, gk = (np64(c.g_q), np64(c.g_k)) if norm else (None, None)
    kr, vr, qr = O.append(k0[1], v0[1], c.table, np64(c.qkv), nq, nkv, d, gq, gk, 1e-6, 1e6, c.cu, c.ctx)
    # values: rounded once, after ~12 fp32 operations on a pair (x, y) and an
    # angle off by 5e-7: 16 * 2^-24 + 5e-7 of the pair's length
    e = 16 * 2.0 ** -24 + 5e-7

    def close(got, ref):
        half = ref.shape[-1] // 2
        pair = np.sqrt(ref[..., :half] ** 2 + ref[..., half:] ** 2)
        tol = U[dtype] * np.abs(ref) + e * np.concatenate([pair, pair], -1)
        return (np.abs(got - ref) <= tol).all()

    assert close(np64(q)[:c.T].reshape(c.T, nq, d), qr[:c.T].reshape(c.T, nq, d))
    assert (np64(q)[c.T:] == 7.0).all()                       # rows behind the last request: left alone
    k1, v1 = np64(c.k), np64(c.v)
    assert np.array_equal(k1[0], k0[0], equal_nan=True) and np.array_equal(v1[0], v0[0], equal_nan=True)   # other layer
    live = ~np.isnan(kr)
    assert (np.isnan(k1[1]) == ~live).all() and (np.isnan(v1[1]) == np.isnan(vr)).all()
    assert close(np.where(live, k1[1], 0), np.where(live, kr, 0))
    assert np.array_equal(v1[1], vr, equal_nan=True)          # V is copied


@pytest.mark.parametrize("nq,nkv,d,dtype,ctx,new", [
    (8, 4, 128, "bf16", [0, 64, 8, 5], [1500, 700, 1000, 600]), (16, 8, 64, "bf16", [0, 128, 3], [5000, 4096, 2000]),
    (4, 4, 64, "f32", [0, 12, 66], [3000, 2500, 900]), (8, 8, 128, "f32", [0, 4], [2048, 8000])])
def test_append_of_prompts(nq, nkv, d, dtype, ctx, new):
    """Prompts long enough for every tile of tokens, at slots that are and are
    not on 16-byte boundaries: all rows against the formula in 64 bits."""
    import torch
    c = Batch(nq, nkv, d, dtype, ctx, new, seed=nq + d, stale=0.0, pad_rows=3)
    before = c.k.clone(), c.v.clone()
    q = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k)
    assert c.ops.status() == 0
    owner = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
    pos = c.ctx_d[owner].long() + torch.arange(c.T, device="cuda") - c.cu_d[owner]
    page, slot = c.kv.page_table[owner, pos // PAGE].long(), pos % PAGE
    x = c.qkv[:c.T].view(c.T, nq + 2 * nkv, d)
    assert torch.equal(c.v[1, page, :, :, slot], x[:, nq + nkv:])          # V is copied
    y = x[:, :nq + nkv].double()
    y = y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    y = y * torch.cat([c.g_q.expand(nq, d), c.g_k.expand(nkv, d)]).double()
    ang = pos.double()[:, None] * 1e6 ** (-2 * torch.arange(d // 2, device="cuda").double() / d)
    z = torch.complex(y[..., :d // 2].contiguous(), y[..., d // 2:].contiguous()) * torch.polar(torch.ones_like(ang), ang)[:, None]
    ref, size = torch.cat([z.real, z.imag], -1), torch.cat([z.abs(), z.abs()], -1)
    tol = U[dtype] * ref.abs() + (16 * 2.0 ** -24 + 5e-7) * size           # as in test_append_matches_oracle
    assert ((q[:c.T].double().view(c.T, nq, d) - ref[:, :nq]).abs() <= tol[:, :nq]).all()
    assert ((c.k[1, page, :, slot].double() - ref[:, nq:]).abs() <= tol[:, nq:]).all()
    # every other slot, and the other layer, as they were
    c.k[1, page, :, slot], c.v[1, page, :, :, slot] = before[0][1, page, :, slot], before[1][1, page, :, :, slot]
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])


def test_append_at_the_far_end_of_the_positions():
    """Positions up to 2^24 - 1 (2^18 pages): the angle keeps its accuracy."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    from block_diffusion_drafter_context_gb300.target import TargetOps
    d, ctx = 128, [2 ** 24 - 8, 2 ** 20 + 3, 131071]
    table = torch.full((3, 2 ** 18), -1, dtype=torch.int32)
    for b, c in enumerate(ctx):
        table[b, c // PAGE] = 2 * b
        if (c + 7) // PAGE != c // PAGE:
            table[b, (c + 7) // PAGE] = 2 * b + 1
    k = torch.zeros(1, 6, 1, PAGE, d, device="cuda")
    v = torch.zeros(1, 6, 1, d, PAGE, device="cuda")
    kv = PagedKV.from_tensors(k, v, table.cuda())
    ops = TargetOps(1, 1, d, dtype="f32", max_batch=3)
    x = torch.randn(24, 3 * d, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    cu = np.array([0, 8, 16, 24])
    q = ops.append_kv(kv, 0, x, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                      torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    assert ops.status() == 0
    for b, c in enumerate(ctx):
        for i in range(8):
            ref = O.head_norm_rope(np64(x[8 * b + i, :d]), None, 0, 1e6, c + i)
            assert np.abs(np64(q[8 * b + i]) - ref).max() <= 1.5e-6 * np.abs(np64(x[8 * b + i])).max() * 2 ** 0.5
            kref = O.head_norm_rope(np64(x[8 * b + i, d:2 * d]), None, 0, 1e6, c + i)
            page, slot = int(table[b, (c + i) // PAGE]), (c + i) % PAGE
            assert np.abs(np64(k[0, page, 0, slot]) - kref).max() <= 1.5e-6 * np.abs(np64(x[8 * b + i])).max() * 2 ** 0.5


def test_append_without_rotation_and_with_a_missing_page():
    """rope_base 0 and no gains: the rows are copied; a token whose page is
    outside the pool is reported and not appended."""
    import torch
    c = Batch(4, 2, 128, "bf16", ctx=[10, 60], new=[5, 9], hole=(1, 1, 1 << 20))
    c.ops.rope_base = 0.0
    before = np64(c.k)
    q = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d)
    assert c.ops.status() == -7 and c.ops.status() == 0
    assert torch.equal(q, c.qkv[:, :4 * 128])
    k = c.qkv[:, 4 * 128:6 * 128].view(-1, 2, 128)
    v = c.qkv[:, 6 * 128:].view(-1, 2, 128)
    pages = [int(c.table[0, 0]), int(c.table[1, 0])]
    for page, rows, slots in ((pages[0], slice(0, 5), slice(10, 15)), (pages[1], slice(5, 9), slice(60, 64))):
        assert torch.equal(c.k[1, page, :, slots], k[rows].transpose(0, 1))
        assert torch.equal(c.v[1, page, :, :, slots], v[rows].permute(1, 2, 0))
    rest = [p for p in range(c.k.shape[1]) if p not in pages]
    assert np.array_equal(np64(c.k)[1, rest], before[1, rest], equal_nan=True)


# ------------------------------------------------------------------ attention
LENGTHS = [
    ([0], [1]), ([0, 1, 63, 64, 65, 127, 128], [1] * 7), ([777], [1]), ([0, 300, 64, 5], [16, 1, 0, 7]),
    ([0] * 3, [16, 15, 1]), ([1000, 3, 129], [5, 5, 5]), ([2048] * 2, [1, 2]),
]


@pytest.mark.parametrize("nq,nkv,d,dtype", SHAPES)
@pytest.mark.parametrize("ctx,new", LENGTHS)
def test_attention_matches_oracle(nq, nkv, d, dtype, ctx, new):
    """From one position on, page borders, requests without new tokens, every
    row tile; NaN in every slot that no token owns."""
    import torch
    c = Batch(nq, nkv, d, dtype, ctx, new, seed=len(ctx) + d, pad_rows=3, max_new=max(new))
    out = torch.full((c.T + 3, nq * d), 7.0, dtype=c.dt, device="cuda")
    lse = torch.full((c.T + 3, nq), 7.0, device="cuda")
    o, l = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, out=out, lse=lse)
    assert c.ops.status() == 0 and o is out and l is lse
    c.check_attention(out, lse)
    assert (out[c.T:] == 7).all() and (lse[c.T:] == 7).all()     # rows behind the last request
    again, lse2 = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert torch.equal(again[:c.T], out[:c.T]) and torch.equal(lse2[:c.T], lse[:c.T])


@pytest.mark.parametrize("nq,nkv,d,dtype", [(8, 2, 128, "bf16"), (8, 1, 64, "bf16"), (4, 2, 64, "f32")])
@pytest.mark.parametrize("window", [1, 2, 64, 100, 5000])
def test_sliding_window(nq, nkv, d, dtype, window):
    c = Batch(nq, nkv, d, dtype, [0, 700, 64, 130], [16, 1, 3, 9], seed=window, window=window)
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, window=window, want_lse=True)
    assert c.ops.status() == 0
    c.check_attention(out, lse)


@pytest.mark.parametrize("nq,nkv,d,dtype,n", [(16, 2, 128, "bf16", 1), (16, 2, 128, "bf16", 16), (4, 1, 64, "f32", 3)])
def test_long_request_is_split_and_joined(nq, nkv, d, dtype, n):
    """One request whose pages are shared out over the whole GPU, beside an
    empty and a short one."""
    c = Batch(nq, nkv, d, dtype, [0, 9000, 30], [0, n, 1], seed=5, max_new=n)
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == 0
    c.check_attention(out, lse)


@pytest.mark.parametrize("nq,nkv,d,dtype,B,top,new,window", [
    (32, 8, 128, "bf16", 40, 6000, 1, 0), (40, 8, 128, "bf16", 24, 5000, 16, 0), (32, 8, 64, "bf16", 40, 4000, 8, 0),
    (16, 8, 64, "bf16", 64, 3000, 2, 700), (16, 4, 128, "f32", 24, 3000, 3, 0), (32, 8, 64, "f32", 16, 3000, 8, 900),
    (8, 1, 128, "bf16", 1, 120000, 1, 0), (8, 1, 128, "bf16", 1, 120000, 7, 0), (4, 4, 128, "bf16", 300, 90, 1, 0)])
def test_attention_of_a_full_gpu(nq, nkv, d, dtype, B, top, new, window):
    """Ragged batches that keep every SM's pipes busy, and one request over all
    of them: all rows against fp64 on the GPU (the same bounds), three calls
    with the same bits."""
    import torch
    rng = np.random.default_rng(B + d + new)
    ctx = sorted(int(v) for v in rng.integers(top // 8, top + 1, B))
    c = Batch(nq, nkv, d, dtype, ctx, [1 + (b * 7) % new for b in range(B)], seed=B, window=window, max_new=new)
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, window=window, want_lse=True)
    assert c.ops.status() == 0
    g, scale, unit = nq // nkv, d ** -0.5, U["bf16"] if dtype == "bf16" else 0.0
    for b in range(B):
        n, L = c.new[b], c.ctx[b] + c.new[b]
        pages = torch.from_numpy(c.table[b, :-(-L // PAGE)].astype(np.int64)).cuda()
        k = c.k[1, pages].permute(1, 0, 2, 3).reshape(nkv, -1, d)[:, :L].double()
        v = c.v[1, pages].permute(1, 0, 3, 2).reshape(nkv, -1, d)[:, :L].double()
        rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
        q = c.q[rows].double().view(n, nkv, g, d).permute(1, 0, 2, 3)        # [nkv, n, g, d]
        s = torch.einsum("hngd,htd->hngt", q, k) * scale
        size = torch.einsum("hngd,htd->hngt", q.abs(), k.abs()).max() * scale   # what a score's sum is made of
        pos, key = c.ctx[b] + torch.arange(n, device="cuda")[:, None], torch.arange(L, device="cuda")
        see = (key <= pos) & ((key > pos - window) if window else True)
        s = s.masked_fill(~see[None, :, None], -float("inf"))
        ref_lse = s.logsumexp(-1)
        w = (s - ref_lse[..., None]).exp()
        ref, spread = (torch.einsum("hngt,htd->hngd", w, x) for x in (v, v.abs()))
        e = float(2 * d * 2.0 ** -24 * size + L * 2.0 ** -24 + 2.0 ** -20)
        got = out[rows].double().view(n, nkv, g, d).permute(1, 0, 2, 3)
        assert ((got - ref).abs() <= (unit + e) * spread + U[dtype] * ref.abs() + 1e-30).all(), b
        got = lse[rows].double().view(n, nkv, g).permute(1, 0, 2)
        assert ((got - ref_lse).abs() <= e + 2.0 ** -22 * (1 + ref_lse.abs())).all(), b
    for _ in range(3):
        again = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, window=window, want_lse=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("B", [257, 1100, 4096])
def test_large_batches(B):
    """Batches past one and two steps of the lookups, many requests without new
    tokens, every request inside one page: append, then attention."""
    import torch
    rng = np.random.default_rng(B)
    new = rng.integers(0, 3, B)
    new[0], new[-1] = 1, 2
    c = Batch(2, 1, 64, "f32", rng.integers(0, 62, B).tolist(), new.tolist(), seed=B, stale=0.0, max_new=2)
    q = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k)
    out, lse = c.ops.attend(c.kv, 1, q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == 0
    owner = torch.repeat_interleave(torch.arange(B), torch.tensor(c.new)).cuda()
    pos = c.ctx_d[owner].long() + torch.arange(c.T, device="cuda") - c.cu_d[owner]
    page = c.kv.page_table[owner, 0].long()
    x = c.qkv.double().view(c.T, 4, 64)
    assert torch.equal(c.v[1, page, 0, :, pos].double(), x[:, 3])
    y = x[:, :3] / (x[:, :3].pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    y = y * torch.stack([c.g_q, c.g_q, c.g_k]).double()
    ang = pos.double()[:, None] * 1e6 ** (-2 * torch.arange(32, device="cuda").double() / 64)
    z = torch.complex(y[..., :32].contiguous(), y[..., 32:].contiguous()) * torch.polar(torch.ones_like(ang), ang)[:, None]
    y = torch.cat([z.real, z.imag], -1)
    assert (q.double().view(c.T, 2, 64) - y[:, :2]).abs().max() <= 1.5e-6 * 10
    assert (c.k[1, page, 0, pos].double() - y[:, 2]).abs().max() <= 1.5e-6 * 10
    s = torch.einsum("thd,tkd->thk", q.double().view(c.T, 2, 64), c.k[1, page, 0].double()) / 8
    s = s.masked_fill((torch.arange(64, device="cuda") > pos[:, None])[:, None], -float("inf"))
    ref = torch.einsum("thk,tdk->thd", s.softmax(-1), c.v[1, page, 0].double())
    # scores up to about 30 of 64 products: 2 * 64 * 2^-24 * 8 * 30 / 8 on a probability
    assert (out.double().view(c.T, 2, 64) - ref).abs().max() <= 3e-4
    assert (lse.double() - s.logsumexp(-1)).abs().max() <= 3e-4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_peaked_scores_and_large_values(dtype):
    """Scores far apart (the maximum moves by hundreds along the request)."""
    c = Batch(4, 2, 128, dtype, [400, 70], [4, 1], seed=3)
    c.q.mul_(12)
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, scale=0.25, want_lse=True)
    assert c.ops.status() == 0
    c.check_attention(out, lse, scale=0.25)


@pytest.mark.parametrize("nq,nkv,d,dtype", [(8, 2, 128, "bf16"), (8, 2, 64, "bf16"), (4, 2, 64, "f32")])
@pytest.mark.parametrize("new", [1, 5, 16])
def test_missing_pages_are_dropped_and_reported(nq, nkv, d, dtype, new):
    """Request 0 lost its second page, request 1 its only one: its tokens see
    nothing (out 0, lse -inf)."""
    c = Batch(nq, nkv, d, dtype, [200, 0], [new, 1], seed=new, hole=(0, 1, 1 << 20))
    c.table[1, 0] = -5
    c.kv.page_table[1, 0] = -5
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == -7
    c.check_attention(out, lse)
    assert c.ops.status() == 0


@pytest.mark.parametrize("nq,nkv,d,dtype", [(8, 2, 128, "bf16"), (16, 2, 64, "bf16"), (4, 2, 64, "f32"),
                                            (4, 1, 128, "f32")])
@pytest.mark.parametrize("ctx,new", [([70, 200, 3], [1, 1, 1]), ([70, 200, 3], [9, 16, 2]), ([20000, 70], [1, 1]),
                                     ([20000, 70], [9, 3]), ([64] * 90, [3] * 90)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row_alone(nq, nkv, d, dtype, ctx, new, value):
    """Few short requests, a long one cut over many CTAs, many short ones: a
    NaN or an infinity in one head of one token's query makes that row NaN,
    never a plausible 0, and leaves the other rows within their bounds."""
    import torch
    c = Batch(nq, nkv, d, dtype, ctx, new, seed=nq + len(ctx), max_new=max(new))
    good, good_lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    q = c.q.clone()
    for row, head in ((0, nq - 1), (c.T - 1, 0)):
        q[row, head * d + 5] = value
    out, lse = c.ops.attend(c.kv, 1, q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == 0
    spoiled = torch.zeros_like(good, dtype=torch.bool)
    for row, head in ((0, nq - 1), (c.T - 1, 0)):
        spoiled[row, head * d:(head + 1) * d] = True
    assert torch.equal(out.isnan(), spoiled) and torch.equal(lse.isnan(), spoiled[:, ::d])
    c.check_attention(torch.where(spoiled, good, out), torch.where(spoiled[:, ::d], good_lse, lse))


@pytest.mark.parametrize("new", [1, 6])
def test_requests_share_the_pages_of_a_common_prefix(new):
    import torch
    c = Batch(8, 2, 128, "bf16", [300, 300, 300], [new] * 3, seed=new, max_new=new)
    c.table[1:, :4] = c.table[0, :4]          # 256 tokens in common
    c.kv.page_table.copy_(torch.from_numpy(c.table))
    out, lse = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    assert c.ops.status() == 0
    c.check_attention(out, lse)


def test_requests_out_of_range_are_left_unwritten():
    import torch
    c = Batch(4, 2, 128, "bf16", [10, 20, 30], [1, 3, 2], max_new=4)
    good, _ = c.ops.attend(c.kv, 1, c.q, c.cu_d, c.ctx_d, want_lse=True)
    for change, touched in (("ctx", 1), ("new", 1)):
        ctx = c.ctx_d.clone()
        if change == "ctx":
            ctx[1] = -3
        out = torch.full_like(good, 7.0)
        if change == "new":     # more new tokens than the call's max_new
            c.ops.attend(c.kv, 1, c.q, c.cu_d, ctx, max_new=2, out=out)
        else:
            c.ops.attend(c.kv, 1, c.q, c.cu_d, ctx, out=out)
        assert c.ops.status() == -7
        assert (out[1:4] == 7).all()
        assert torch.equal(out[0], good[0]) and torch.equal(out[4:], good[4:])


# ------------------------------------------------------------------ log probabilities
def rows_of(kind, rows, V, rng):
    x = rng.standard_normal((rows, V)).astype(np.float32) * 2.5
    if kind == "masked":
        x[rng.random((rows, V)) < 0.9] = -np.inf
    elif kind == "lowest":
        x[rng.random((rows, V)) < 0.9] = np.finfo(np.float32).min
    elif kind == "ties":
        x = np.round(x)
    elif kind == "equal":
        x[:] = 0.25
    elif kind == "peaked":
        x[np.arange(rows), rng.integers(0, V, rows)] = 60.0
    elif kind == "far":
        x += 5e4
    elif kind == "ascending":      # every logit is above all before it
        x.sort(axis=1)
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V,pad", [(1, 1, 0), (3, 17, 0), (4, 1000, 3), (2, 4097, 1), (5, 40001, 0), (2, 9000, 7),
                                        (700, 300, 0)])
@pytest.mark.parametrize("kind", ["normal", "masked", "lowest", "ties", "equal", "peaked", "far", "ascending"])
def test_logprobs_match_oracle(dtype, rows, V, pad, kind):
    import torch
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    if rows > 10 and kind not in ("normal", "ties"):
        pytest.skip("many rows: two kinds are enough")
    rng = np.random.default_rng(rows * V + pad)
    x = torch.from_numpy(rows_of(kind, rows, V + pad, rng)).cuda()
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)[:, :V]
    T, n = (0.7, min(16, V)) if pad else (1.0, min(5, V))
    ids = rng.integers(0, V, rows)
    ids[::3] = np64(x).argmax(1)[::3]
    if rows > 2:
        ids[1] = -1
    got = token_logprobs(x, torch.from_numpy(ids.astype(np.int32)).cuda(), temperature=T, n_top=n)
    got = {k: v.cpu().numpy() for k, v in got.items()}
    x64 = np64(x)
    for r in range(min(rows, 25)):
        if ids[r] < 0:
            assert got["logprob"][r] == 0 and got["entropy"][r] == 0 and got["rank"][r] == -1
            assert (got["top_ids"][r] == -1).all() and (got["top_logprobs"][r] == 0).all()
            continue
        lp, ent, rank, top, top_lp = O.token_logprobs(x64[r], ids[r], T, n)
        assert got["rank"][r] == rank and list(got["top_ids"][r]) == top, r
        # fp32: a scaled logit y is off by 2 * 2^-24 |y| (product and the
        # maximum's), e^(y-m) by that, and the sum by (V / 256 + 16) * 2^-24
        # relative; the entropy sums terms of at most log V + 1
        big = np.abs(x64[r][np.isfinite(x64[r])]).max() / T if np.isfinite(x64[r]).any() else 0.0
        big = big if kind != "lowest" else np.abs(x64[r][x64[r] > -1e30]).max(initial=0) / T
        e = (6 * big + V / 256 + 32) * 2.0 ** -24
        for a, b in ((got["logprob"][r], lp), *zip(got["top_logprobs"][r], top_lp)):
            if abs(b) > np.finfo(np.float32).max:     # -inf, or past the output's range
                assert a == -np.inf
            else:
                assert abs(a - b) <= e + 4 * 2.0 ** -24 * abs(b), (r, a, b)
        assert abs(got["entropy"][r] - ent) <= 3 * e * (np.log(V) + 2), (r, got["entropy"][r], ent)


@pytest.mark.parametrize("dtype,rows,V", [("f32", 700, 151936), ("bf16", 700, 151936), ("f32", 64, 151936),
                                          ("bf16", 500, 40001), ("f32", 3, 1500000)])
def test_logprobs_of_a_full_gpu(dtype, rows, V):
    """Rows enough to keep every SM's memory pipes busy, and few long ones: all
    rows against fp64 sums, exact counts and a stable sort on the GPU."""
    import torch
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    g = torch.Generator("cuda").manual_seed(rows + V)
    x = (torch.randn(rows, V, generator=g, device="cuda") * 2.5).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    ids = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, x.argmax(1),
                      torch.randint(0, V, (rows,), generator=g, device="cuda"))
    ids[::7] = -1
    live = (ids >= 0).nonzero()[:, 0]
    first = None
    for _ in range(3):
        got = token_logprobs(x, ids.int(), temperature=0.8)
        if first is None:
            first = got
            at = torch.arange(V, device="cuda")
            for part in live.split(64):
                y, t = x[part].double() / 0.8, ids[part][:, None]
                lse = y.logsumexp(1, keepdim=True)
                mine, lp = x[part].gather(1, t), y - lse
                # fp32: as in the test above, logits up to 6 * 2.5 / 0.8
                e = (6 * 20 + V / 256 + 32) * 2.0 ** -24
                for key, ref, tol in (("logprob", lp.gather(1, t)[:, 0], 2 * e),
                                      ("entropy", -(lp.exp() * lp).sum(1), 3 * e * (np.log(V) + 2)),
                                      ("top_logprobs", lp.topk(16, dim=1).values, 2 * e)):
                    assert (got[key][part].double() - ref).abs().max() <= tol, key
                before = (x[part] > mine) | ((x[part] == mine) & (at < t))
                assert torch.equal(got["rank"][part].long(), before.sum(1))
                order = torch.sort(x[part], dim=1, descending=True, stable=True).indices[:, :16]
                assert torch.equal(got["top_ids"][part].long(), order)
        for key in got:      # the same bits on every call
            assert torch.equal(got[key], first[key]), key


def test_logprobs_of_rows_without_a_distribution():
    """Nothing but -inf: probability 0 everywhere; a NaN or +inf logit: NaN;
    an id past the vocabulary: NaN and rank -1."""
    import torch
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    x = torch.randn(6, 5000, device="cuda")
    x[0] = -float("inf")
    x[1, 77] = float("nan")
    x[2, 4999] = float("inf")
    x[3, 3] = -float("inf")
    ids = torch.tensor([4, 5, 6, 3, 5000, 9], dtype=torch.int32, device="cuda")
    got = {k: v.cpu() for k, v in token_logprobs(x, ids, n_top=4).items()}
    assert got["logprob"][0] == -float("inf") and got["entropy"][0] == 0 and got["rank"][0] == 4
    assert got["top_ids"][0].tolist() == [0, 1, 2, 3] and (got["top_logprobs"][0] == -float("inf")).all()
    for r in (1, 2):
        assert got["logprob"][r].isnan() and got["entropy"][r].isnan() and got["top_logprobs"][r].isnan().all()
        assert ((got["top_ids"][r] >= 0) & (got["top_ids"][r] < 5000)).all()
    assert got["logprob"][3] == -float("inf") and got["entropy"][3].isfinite() and got["rank"][3] == 4999
    assert got["logprob"][4].isnan() and got["rank"][4] == -1 and got["top_logprobs"][4].isfinite().all()
    assert got["logprob"][5].isfinite()


def test_logprobs_without_alternatives_and_top16_agrees():
    """n_top 0 gives the same sums; the alternatives are the library's top-16."""
    import torch
    from block_diffusion_drafter_context_gb300 import binding as Bd
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    x = torch.randn(9, 151936, generator=torch.Generator("cuda").manual_seed(2), device="cuda").mul_(3)
    ids = torch.randint(0, 151936, (9,), device="cuda").int()
    a, b = token_logprobs(x, ids, n_top=16), token_logprobs(x, ids, n_top=0)
    for k in ("logprob", "entropy", "rank"):
        assert torch.equal(a[k], b[k])
    assert b["top_ids"].shape == (9, 0)
    top, val = torch.empty(9, 16, dtype=torch.int32, device="cuda"), torch.empty(9, 16, device="cuda")
    Bd.dflash_topk16_noalloc(x, 9, 151936, top, val)
    assert torch.equal(a["top_ids"], top)


# ------------------------------------------------------------------ together
def test_a_verification_step_then_the_next():
    """Two steps of two layers on a second stream: append a block, attend,
    verify greedily, take the committed tokens' log probabilities, and append
    the next block over the rejected tokens' slots."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import Drafter
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    S, V = 6, 2000
    c = Batch(8, 2, 128, "bf16", ctx=[40, 7, 190], new=[S] * 3, seed=11, stale=0.0)
    c.table[:, :] = np.arange(c.table.size).reshape(c.table.shape)      # room for both steps
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    pool = c.table.size
    c.k = torch.zeros(2, pool, 2, PAGE, 128, dtype=c.dt, device="cuda")
    c.v = torch.zeros(2, pool, 2, 128, PAGE, dtype=c.dt, device="cuda")
    c.k[:, :, :, :, :].normal_(generator=torch.Generator("cuda").manual_seed(4))
    c.v.normal_(generator=torch.Generator("cuda").manual_seed(5))
    c.kv = PagedKV.from_tensors(c.k, c.v, torch.from_numpy(c.table).cuda())
    rng = np.random.default_rng(6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for step in range(2):
        k0, v0 = np64(c.k), np64(c.v)
        qkv = [(torch.randn(3 * S, 12 * 128, device="cuda") * 1.5).to(c.dt) for _ in range(2)]
        logits = torch.randn(3, S, V, device="cuda") * 3
        draft = torch.from_numpy(rng.integers(0, V, (3, S - 1)).astype(np.int32)).cuda()
        target = logits.argmax(-1).int()
        draft[0, :3] = target[0, :3]
        draft[2] = target[2, :S - 1]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            outs = []
            for l in range(2):
                q = c.ops.append_kv(c.kv, l, qkv[l], c.cu_d, c.ctx_d, c.g_q, c.g_k)
                outs.append((q, *c.ops.attend(c.kv, l, q, c.cu_d, c.ctx_d, want_lse=True)))
            acc, bonus, com = Drafter.verify_greedy(draft, target)
            lp = token_logprobs(logits.reshape(3 * S, V), com.reshape(-1))
        side.synchronize()
        assert c.ops.status(side) == 0
        for l in range(2):
            kr, vr, _ = O.append(k0[l], v0[l], c.table, np64(qkv[l]), 8, 2, 128, np64(c.g_q), np64(c.g_k), 1e-6, 1e6,
                                 c.cu, c.ctx)
            assert np.abs(np64(c.k[l]) - kr).max() <= 2.0 ** -8 * np.abs(kr).max() * 1.01
            assert np.array_equal(np64(c.v[l]), vr)
            one = types.SimpleNamespace(**{**c.__dict__})
            one.k, one.v = c.k[l:l + 1].repeat(2, 1, 1, 1, 1), c.v[l:l + 1].repeat(2, 1, 1, 1, 1)
            one.attend_ref = types.MethodType(Batch.attend_ref, one)
            Batch.check_attention(one, outs[l][1], outs[l][2], q=outs[l][0])
        com = com.cpu().numpy()
        assert (acc.cpu().numpy() >= [3, 0, S - 1]).all()
        for b in range(3):
            for i in range(S):
                if com[b, i] < 0:
                    assert lp["rank"][b * S + i] == -1
                else:     # committed tokens are the target's most probable ones
                    assert lp["rank"][b * S + i] == 0 and lp["top_ids"][b * S + i, 0] == com[b, i]
                    ref = O.token_logprobs(np64(logits[b, i]), com[b, i], 1.0, 1)
                    assert abs(float(lp["logprob"][b * S + i]) - ref[0]) <= 1e-5
        # the next step starts behind the accepted tokens: the rejected ones' slots are written again
        c.ctx_d += acc + 1
        c.ctx = c.ctx_d.tolist()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_captured_step_follows_its_buffers(dtype, d):
    """A graph of append + attend + log probabilities for a padded batch is
    replayed with other lengths, tokens and pages in the same buffers; an eager
    call on the same workspace in between changes nothing."""
    import torch
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    c = Batch(8, 2, d, dtype, ctx=[500, 3, 64], new=[5, 1, 4], seed=8, stale=0.0, pad_rows=6)
    logits = torch.randn(16, 3000, device="cuda")
    ids = torch.full((16,), -1, dtype=torch.int32, device="cuda")
    ids[:10] = 7
    out, lse = torch.zeros(16, 8 * d, dtype=c.dt, device="cuda"), torch.zeros(16, 8, device="cuda")
    q = torch.zeros(16, 8 * d, dtype=c.dt, device="cuda")

    def step():
        c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k, q_out=q)
        c.ops.attend(c.kv, 1, q, c.cu_d, c.ctx_d, out=out, lse=lse)
        return token_logprobs(logits, ids)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for ctx, new in (([500, 3, 64], [5, 1, 4]), ([130, 60, 0], [16, 0, 0]), ([0, 62, 5], [1, 1, 1])):   # each within its mapped pages
        c.ctx, c.new = ctx, new
        c.cu = np.concatenate([[0], np.cumsum(new)])
        c.T = int(c.cu[-1])
        c.ctx_d.copy_(torch.tensor(ctx))
        c.cu_d.copy_(torch.tensor(c.cu))
        ids.fill_(-1)
        ids[:c.T] = torch.randint(0, 3000, (c.T,), device="cuda").int()
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got, got_lse = out.clone(), lse.clone()
        lp = {k: v.clone() for k, v in captured.items()}
        assert c.ops.status() == 0
        c.check_attention(got, got_lse, q=q)
        assert (got[c.T:] == 7).all()
        eager = step()
        assert torch.equal(out[:c.T], got[:c.T])
        for k in lp:
            assert torch.equal(lp[k], eager[k])
            assert torch.equal(lp["rank"] >= 0, ids >= 0)


def test_wrapper_refuses_tensors_of_another_shape():
    import torch
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    c = Batch(4, 2, 128, "bf16", [10, 20], [1, 1])
    bad = [dict(q=c.q.float()), dict(q=c.q[:, :-8]), dict(q=c.q.cpu()), dict(q=c.q.t().contiguous().t()),
           dict(cu=c.cu_d.long()), dict(cu=c.cu_d[:-1]), dict(ctx=c.ctx_d.cpu()), dict(layer=2), dict(layer=-1),
           dict(out=torch.empty(2, 512, device="cuda")), dict(lse=torch.empty(2, 3, device="cuda"))]
    for kw in bad:
        a = dict(layer=1, q=c.q, cu=c.cu_d, ctx=c.ctx_d, out=None, lse=None)
        a.update(kw)
        with pytest.raises(ValueError):
            c.ops.attend(c.kv, a["layer"], a["q"], a["cu"], a["ctx"], out=a["out"], lse=a["lse"])
    with pytest.raises(ValueError):
        c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q.double(), c.g_k)
    three = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):       # more requests than the page table has rows
        c.ops.attend(c.kv, 1, c.q, three, three[:3])
    x = torch.zeros(2, 100, device="cuda")
    for logits, ids in ((x.half(), three[:2]), (x, three[:3]), (x, three[:2].long()), (x.t(), three[:2]),
                        (x[0], three[:2]), (x, three[:2].cpu())):
        with pytest.raises(ValueError):
            token_logprobs(logits, ids)
