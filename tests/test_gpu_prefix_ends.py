"""Many short tiles of a shared prefix in the launch of its own: what happens at
a tile's end, again and again."""
import pytest

from tests.test_gpu_shared import Shared
from tests.test_gpu_target import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def apart():
    """The prefix in its own launch, however short it is."""
    from block_diffusion_drafter_context_gb300 import binding as B
    from block_diffusion_drafter_context_gb300.build import build
    build()
    B.dflash_debug_shared_launches(2)
    yield
    B.dflash_debug_shared_launches(0)


@pytest.mark.parametrize("nq,nkv,d", [(64, 8, 128), (32, 8, 64), (5, 1, 128)])
@pytest.mark.parametrize("pages", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("missing", [False, True])
def test_short_tiles(nq, nkv, d, pages, missing):
    """Tiles of 1 to 5 pages, the last of them there or not, thirty times over:
    no wait runs out, the same bits, and right against fp64 (tolerances as in
    Shared.check; the pages that are not there are no positions)."""
    import torch
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    batch = 64 if nkv > 1 else 200
    c = Shared(nq, nkv, d, "bf16", pages, [(b * 11) % 70 for b in range(batch)], [16 - b % 5 for b in range(batch)],
               seed=pages + d, stale=0.0)
    if missing:
        table = c.table.copy()
        table[1:, :pages] = -1
        table[:, pages - 1] = -1
        c.kv = PagedKV.from_tensors(c.k, c.v, torch.from_numpy(table).cuda())
    want = -7 if missing else 0
    out, lse = c.attend()
    assert c.ops.status() == want
    for _ in range(30):
        again = c.attend()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert c.ops.status() == want
    hole = range((pages - 1) * 64, pages * 64) if missing else range(0)
    ref, rlse, spread = without(c, hole)
    size = float(c.q.double().abs().view(c.T, nq, d).sum(-1).max() * c.k[1].abs().max()) * d ** -0.5
    e = 2 * d * 2.0 ** -24 * size + (max(c.ctx) + 16) * 2.0 ** -24 + 2.0 ** -19
    tol = (U["bf16"] + e) * spread + U["bf16"] * ref.abs() + 1e-30
    got = out.double().view(c.T, nq, d)
    assert ((got - ref).abs() <= tol).all(), float(((got - ref).abs() / tol).max())
    assert ((lse.double() - rlse).abs() <= e + 2.0 ** -22 * (1 + rlse.abs())).all()


def without(c, hole):
    """(out, lse, sum p |v|) in fp64 on the device, the positions of `hole` left out."""
    import torch
    table = torch.from_numpy(c.table).cuda().long()
    g = c.nq // c.nkv
    out = torch.empty(c.T, c.nq, c.d, dtype=torch.float64, device="cuda")
    lse, spread = torch.empty(c.T, c.nq, dtype=torch.float64, device="cuda"), torch.empty_like(out)
    for b in range(len(c.ctx)):
        n, L = c.new[b], c.ctx[b] + c.new[b]
        rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
        pages = table[b, :-(-L // 64)]
        k = c.k[1, pages].double().transpose(0, 1).reshape(c.nkv, -1, c.d)[:, :L]
        v = c.v[1, pages].double().permute(1, 0, 3, 2).reshape(c.nkv, -1, c.d)[:, :L]
        q = c.q[rows].double().view(n, c.nkv, g, c.d)
        s = torch.einsum("ihgd,htd->ihgt", q, k) * c.d ** -0.5
        at = torch.arange(L, device="cuda")
        hide = (at > c.ctx[b] + torch.arange(n, device="cuda")[:, None]) | ((at >= hole.start) & (at < hole.stop))
        s.masked_fill_(hide[:, None, None], -float("inf"))
        l = torch.logsumexp(s, -1)
        p = (s - l[..., None]).exp()
        out[rows] = torch.einsum("ihgt,htd->ihgd", p, v).reshape(n, c.nq, c.d)
        spread[rows] = torch.einsum("ihgt,htd->ihgd", p, v.abs()).reshape(n, c.nq, c.d)
        lse[rows] = l.reshape(n, c.nq)
    return out, lse, spread


def test_the_largest_batch():
    """4096 requests behind one prefix, in both forms; tolerances as above."""
    import torch
    from block_diffusion_drafter_context_gb300 import binding as B
    nq, nkv, d, batch = 8, 1, 128, 4096
    c = Shared(nq, nkv, d, "bf16", 2, [(b * 37) % 90 for b in range(batch)], [1 + b % 2 for b in range(batch)], seed=1,
               stale=0.0)
    ref, rlse, spread = without(c, range(0))
    size = float(c.q.double().abs().view(c.T, nq, d).sum(-1).max() * c.k[1].abs().max()) * d ** -0.5
    e = 2 * d * 2.0 ** -24 * size + (max(c.ctx) + 16) * 2.0 ** -24 + 2.0 ** -19
    tol = (U["bf16"] + e) * spread + U["bf16"] * ref.abs() + 1e-30
    for launches in (1, 2):
        B.dflash_debug_shared_launches(launches)
        out, lse = c.attend()
        assert c.ops.status() == 0
        assert ((out.double().view(c.T, nq, d) - ref).abs() <= tol).all()
        assert ((lse.double() - rlse).abs() <= e + 2.0 ** -22 * (1 + rlse.abs())).all()
        assert torch.equal(c.attend()[0], out)
