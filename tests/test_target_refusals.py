"""Argument checks of the target-side operators (append to the paged cache,
attention over it, token log probabilities): every refusal below returns
before any device work, so it runs without a GPU."""
import ctypes

import pytest

from block_diffusion_drafter_context_gb300 import binding as B
from block_diffusion_drafter_context_gb300 import build as BUILD

FAKE = 0x10000      # an aligned address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.load()


def heads(**kw):
    h = dict(dtype=0, n_q_heads=8, n_kv_heads=2, head_dim=128)
    h.update(kw)
    return B.dflash_heads(*h.values())


def cache(**kw):
    c = dict(k_cache=FAKE, v_cache=FAKE, page_table=FAKE, num_pages=10, max_pages=4)
    c.update(kw)
    return B.dflash_kv(*c.values())


def append(lib, hs=None, kv=None, **kw):
    a = dict(layer=0, qkv=FAKE, ld=1536, g_q=FAKE, g_k=FAKE, eps=1e-6, base=1e6, cu=FAKE, total=3, ctx=FAKE, batch=2,
             q_out=FAKE, ws=FAKE, ws_bytes=256, stream=None)
    a.update(kw)
    return lib.dflash_append_kv(ctypes.byref(hs or heads()), ctypes.byref(kv or cache()), *a.values())


def attend(lib, hs=None, kv=None, **kw):
    a = dict(layer=0, q=FAKE, ld=1024, cu=FAKE, total=3, ctx=FAKE, batch=2, max_new=4, window=0, scale=0.1, out=FAKE,
             lse=None, ws=FAKE, ws_bytes=BIG, stream=None)
    a.update(kw)
    return lib.dflash_cache_attention(ctypes.byref(hs or heads()), ctypes.byref(kv or cache()), *a.values())


def logprobs(lib, **kw):
    a = dict(x=FAKE, dtype=1, rows=2, vocab=100, ld=100, ids=FAKE, temp=1.0, n_top=16, lp=FAKE, ent=FAKE, rank=FAKE,
             top=FAKE, top_lp=FAKE, stream=None)
    a.update(kw)
    return lib.dflash_token_logprobs(*a.values())


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("hs,code", [
    (dict(dtype=2), -1), (dict(n_q_heads=0), -2), (dict(n_kv_heads=0), -2), (dict(n_kv_heads=3), -2),
    (dict(n_kv_heads=-2), -2), (dict(head_dim=96), -4), (dict(head_dim=256), -4), (dict(n_q_heads=18), -4),
])
def test_heads(lib, call, hs, code):
    assert call(lib, hs=heads(**hs)) == code
    assert lib.dflash_last_error()


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("kv,code", [
    (dict(k_cache=None), -1), (dict(v_cache=None), -1), (dict(page_table=None), -1), (dict(num_pages=0), -2),
    (dict(max_pages=0), -2), (dict(max_pages=(1 << 18) + 1), -2), (dict(num_pages=1 << 23), -2),
    (dict(k_cache=FAKE + 8), -3), (dict(v_cache=FAKE + 2), -3), (dict(page_table=FAKE + 2), -3),
])
def test_cache(lib, call, kv, code):
    assert call(lib, kv=cache(**kv)) == code


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("kw,code", [
    (dict(cu=None), -1), (dict(ctx=None), -1), (dict(ws=None), -1), (dict(batch=-1), -1), (dict(batch=4097), -1),
    (dict(total=-1), -1), (dict(layer=-1), -1), (dict(ld=1000), -2), (dict(ld=-1536), -2), (dict(ld=1537), -3),
    (dict(ws=FAKE + 4), -3), (dict(ws_bytes=255), -2),
    (dict(total=(1 << 30) + 1), -1), (dict(cu=FAKE + 2), -3), (dict(ctx=FAKE + 1), -3),
])
def test_shared_arguments(lib, call, kw, code):
    assert call(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(qkv=None), -1), (dict(qkv=FAKE + 8), -3), (dict(g_q=None), -1), (dict(g_k=None), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(base=1.0), -1), (dict(base=-5.0), -1), (dict(base=float("inf")), -1),
    (dict(base=float("nan")), -1), (dict(q_out=FAKE + 4), -3), (dict(g_q=FAKE + 2), -3), (dict(g_k=FAKE + 2), -3),
])
def test_append(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(q=FAKE + 8), -3), (dict(out=None), -1), (dict(out=FAKE + 8), -3), (dict(max_new=0), -1),
    (dict(max_new=17), -1), (dict(window=-1), -1), (dict(scale=0.0), -1), (dict(scale=-0.1), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(scale=2.5e38), -1), (dict(lse=FAKE + 2), -3),
])
def test_attention(lib, kw, code):
    assert attend(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -1), (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(n_top=17), -1), (dict(n_top=-1), -1),
    (dict(vocab=10, n_top=11), -1), (dict(ld=99), -2), (dict(temp=0.0), -1), (dict(temp=-1.0), -1),
    (dict(temp=float("nan")), -1), (dict(temp=1e5), -1), (dict(x=None), -1), (dict(ids=None), -1), (dict(lp=None), -1),
    (dict(ent=None), -1), (dict(rank=None), -1), (dict(top=None), -1), (dict(top_lp=None), -1), (dict(x=FAKE + 2), -3),
    (dict(dtype=0, x=FAKE + 1), -3), (dict(rows=(1 << 27) + 1), -2),
    (dict(ids=FAKE + 1), -3), (dict(lp=FAKE + 2), -3), (dict(rank=FAKE + 2), -3), (dict(top=FAKE + 2), -3),
])
def test_logprobs(lib, kw, code):
    assert logprobs(lib, **kw) == code


def test_empty_calls_do_nothing(lib):
    none = dict(batch=0, cu=None, ctx=None)
    assert append(lib, **none) == 0 and append(lib, total=0, qkv=None) == 0
    assert append(lib, kv=cache(page_table=None), qkv=None, **none) == 0
    assert attend(lib, **none) == 0 and attend(lib, total=0, q=None, out=None) == 0
    assert attend(lib, kv=cache(page_table=None), q=None, **none) == 0
    assert logprobs(lib, rows=0, x=None) == 0


def test_workspace_size(lib):
    size = lib.dflash_target_workspace_bytes
    h = heads()
    one = size(ctypes.byref(h), 1, 1)
    assert one > 256 and one % 16 == 0
    assert size(ctypes.byref(h), 64, 16) >= one
    for batch, new in ((0, 1), (4097, 1), (1, 0), (1, 17)):
        assert size(ctypes.byref(h), batch, new) == 0
    assert size(ctypes.byref(heads(head_dim=80)), 1, 1) == 0 and size(None, 1, 1) == 0
    # a workspace for a smaller batch is refused
    assert attend(lib, batch=64, max_new=16, ws_bytes=one) == -2
    with pytest.raises(B.DflashError):
        B.dflash_target_workspace_bytes(h, 0, 1)


def test_wrapper_checks():
    torch = pytest.importorskip("torch")
    from block_diffusion_drafter_context_gb300 import target
    from block_diffusion_drafter_context_gb300.drafter import PagedKV
    k = torch.zeros(1, 3, 2, 64, 128, dtype=torch.bfloat16)
    v = torch.zeros(1, 3, 2, 128, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 2, dtype=torch.int32)
    for bad in ((k[0], v, table), (k, k, table), (k, v.float(), table), (k, v, table.long()),
                (k.half(), v.half(), table), (k, v.transpose(0, 1).contiguous().transpose(0, 1)[:, ::2], table),
                (k, v, table)):    # the last: not on a CUDA device
        with pytest.raises(ValueError):
            PagedKV.from_tensors(*bad)
    with pytest.raises(ValueError):
        target.TargetOps(8, 2, 128, dtype="f16")
    with pytest.raises(ValueError):
        target.token_logprobs(torch.zeros(2, 100), torch.zeros(2, dtype=torch.int32))
