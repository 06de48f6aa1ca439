"""The target-side operators' wrappers under their C names: every argument
reaches its place (refusals on the CPU, the same bits as TargetOps on the GPU)."""
import pytest

from block_diffusion_drafter_context_gb300 import binding as B
from block_diffusion_drafter_context_gb300 import build as BUILD
from tests.test_target_refusals import BIG, FAKE, cache, heads


@pytest.fixture(scope="module", autouse=True)
def built():
    BUILD.build()


def refused(code, call, args, **kw):
    a = dict(args)
    assert set(kw) <= set(a)
    a.update(kw)
    with pytest.raises(B.DflashError) as e:
        call(**a)
    assert e.value.code == code


APPEND = dict(layer=0, qkv=FAKE, row_stride=1536, g_q=FAKE, g_k=FAKE, eps=1e-6, rope_base=1e6, cu_new=FAKE, total_new=3,
              ctx_len=FAKE, batch=2, q_out=FAKE, workspace=FAKE, workspace_bytes=256, stream=0)
ATTEND = dict(layer=0, q=FAKE, q_stride=1024, cu_new=FAKE, total_new=3, ctx_len=FAKE, batch=2, max_new=4, window=0,
              scale=0.1, out=FAKE, lse=None, workspace=FAKE, workspace_bytes=BIG, stream=0)
LOGPROBS = dict(logits=FAKE, dtype=1, rows=2, vocab=100, row_stride=100, token_ids=FAKE, temperature=1.0, n_top=16,
                logprob=FAKE, entropy=FAKE, rank=FAKE, top_ids=FAKE, top_logprobs=FAKE, stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(layer=-1), -1), (dict(qkv=FAKE + 8), -3), (dict(row_stride=1537), -3), (dict(g_q=None), -1),
    (dict(g_k=FAKE + 2), -3), (dict(eps=-1.0), -1), (dict(rope_base=0.5), -1), (dict(cu_new=FAKE + 2), -3),
    (dict(total_new=-1), -1), (dict(ctx_len=FAKE + 1), -3), (dict(batch=4097), -1), (dict(q_out=FAKE + 4), -3),
    (dict(workspace=FAKE + 4), -3), (dict(workspace_bytes=255), -2)])
def test_append_kv(kw, code):
    refused(code, lambda **a: B.dflash_append_kv(heads(), cache(), **a), APPEND, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(layer=-1), -1), (dict(q=FAKE + 8), -3), (dict(q_stride=1023), -2), (dict(cu_new=FAKE + 2), -3),
    (dict(total_new=-1), -1), (dict(ctx_len=FAKE + 1), -3), (dict(batch=4097), -1), (dict(max_new=17), -1),
    (dict(window=-1), -1), (dict(scale=0.0), -1), (dict(out=FAKE + 8), -3), (dict(lse=FAKE + 2), -3),
    (dict(workspace=None), -1), (dict(workspace_bytes=1000), -2)])
def test_cache_attention(kw, code):
    refused(code, lambda **a: B.dflash_cache_attention(heads(), cache(), **a), ATTEND, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=FAKE + 2), -3), (dict(dtype=2), -1), (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(row_stride=99), -2),
    (dict(token_ids=FAKE + 1), -3), (dict(temperature=0.0), -1), (dict(n_top=17), -1), (dict(logprob=None), -1),
    (dict(entropy=FAKE + 2), -3), (dict(rank=None), -1), (dict(top_ids=None), -1), (dict(top_logprobs=FAKE + 1), -3)])
def test_token_logprobs(kw, code):
    refused(code, B.dflash_token_logprobs, LOGPROBS, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("nq,nkv,d,dtype", [(8, 2, 128, "bf16"), (4, 2, 64, "f32")])
def test_the_wrappers_give_what_the_objects_give(nq, nkv, d, dtype):
    """Named by their C arguments, on torch's current stream and on another."""
    import torch
    from block_diffusion_drafter_context_gb300.target import token_logprobs
    from tests.test_gpu_target import Batch
    c = Batch(nq, nkv, d, dtype, [70, 3, 300], [5, 1, 9], seed=1, window=100)
    q = c.ops.append_kv(c.kv, 1, c.qkv, c.cu_d, c.ctx_d, c.g_q, c.g_k)
    out, lse = c.ops.attend(c.kv, 1, q, c.cu_d, c.ctx_d, window=100, scale=0.07, want_lse=True)
    k, v = c.k.clone(), c.v.clone()
    x = torch.randn(c.T, 5000, device="cuda")
    ids = torch.arange(c.T, dtype=torch.int32, device="cuda")
    lp = token_logprobs(x, ids, temperature=0.6, n_top=7)
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        c.k[1, :, :, :, :] = 0
        c.v[1, :, :, :, :] = 0
        for b in range(3):      # the positions before the new ones
            for p in range(-(-(c.ctx[b] + c.new[b]) // 64)):
                page, live = int(c.table[b, p]), max(0, min(64, c.ctx[b] - p * 64))
                c.k[1, page, :, :live], c.v[1, page, :, :, :live] = k[1, page, :, :live], v[1, page, :, :, :live]
        q2, out2, lse2 = torch.zeros_like(q), torch.zeros_like(out), torch.zeros_like(lse)
        got = {key: torch.zeros_like(t) for key, t in lp.items()}
        torch.cuda.synchronize()
        ws = dict(workspace=c.ops.workspace, workspace_bytes=c.ops.ws_bytes, stream=stream)
        B.dflash_append_kv(c.ops.heads, c.kv.struct, layer=1, qkv=c.qkv, row_stride=c.qkv.stride(0), g_q=c.g_q, g_k=c.g_k,
                           eps=1e-6, rope_base=1e6, cu_new=c.cu_d, total_new=c.T, ctx_len=c.ctx_d, batch=3, q_out=q2, **ws)
        B.dflash_cache_attention(c.ops.heads, c.kv.struct, layer=1, q=q2, q_stride=nq * d, cu_new=c.cu_d, total_new=c.T,
                                 ctx_len=c.ctx_d, batch=3, max_new=16, window=100, scale=0.07, out=out2, lse=lse2, **ws)
        B.dflash_token_logprobs(logits=x, dtype=B.DFLASH_F32, rows=c.T, vocab=5000, row_stride=5000, token_ids=ids,
                                temperature=0.6, n_top=7, stream=stream, **got)
        torch.cuda.synchronize()
        assert c.ops.status() == 0
        assert torch.equal(q2, q) and torch.equal(out2, out) and torch.equal(lse2, lse)
        for key in lp:
            assert torch.equal(got[key], lp[key]), key
