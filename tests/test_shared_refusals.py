"""Argument checks of the attention behind a shared prefix: every refusal
returns before any device work, so it runs without a GPU."""
import ctypes

import pytest

from block_diffusion_drafter_context_gb300 import binding as B
from block_diffusion_drafter_context_gb300 import build as BUILD
from tests.test_target_refusals import BIG, FAKE, cache, heads

ARGS = dict(layer=0, q=FAKE, q_stride=1024, cu_new=FAKE, total_new=3, ctx_len=FAKE, batch=2, max_new=4, shared_len=64,
            scale=0.1, out=FAKE, lse=None, rows=FAKE, rows_bytes=BIG, workspace=FAKE, workspace_bytes=BIG, stream=0)


@pytest.fixture(scope="module", autouse=True)
def built():
    BUILD.build()


@pytest.mark.parametrize("kw,code", [
    (dict(layer=-1), -1), (dict(q=None), -1), (dict(q=FAKE + 8), -3), (dict(q_stride=1023), -2), (dict(cu_new=None), -1),
    (dict(cu_new=FAKE + 2), -3), (dict(total_new=-1), -1), (dict(ctx_len=FAKE + 1), -3), (dict(batch=4097), -1),
    (dict(max_new=0), -1), (dict(max_new=17), -1), (dict(shared_len=-64), -2), (dict(shared_len=63), -2),
    (dict(shared_len=1), -2), (dict(shared_len=4 * 64), -2), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=2.5e38), -1), (dict(out=None), -1), (dict(out=FAKE + 8), -3), (dict(lse=FAKE + 2), -3),
    (dict(rows=None), -1), (dict(rows=FAKE + 4), -3), (dict(rows_bytes=3 * 8 * 130 * 4 - 1), -2),
    (dict(workspace=None), -1), (dict(workspace_bytes=1000), -2)])
def test_refusals(kw, code):
    a = dict(ARGS)
    assert set(kw) <= set(a)
    a.update(kw)
    with pytest.raises(B.DflashError) as e:
        B.dflash_shared_attention(heads(), cache(), **a)
    assert e.value.code == code and "shared_attention" in str(e.value)


@pytest.mark.parametrize("hs,code", [(dict(dtype=2), -1), (dict(n_kv_heads=3), -2), (dict(head_dim=96), -4)])
def test_heads(hs, code):
    with pytest.raises(B.DflashError) as e:
        B.dflash_shared_attention(heads(**hs), cache(), **ARGS)
    assert e.value.code == code


def test_empty_calls_do_nothing():
    assert B.dflash_shared_attention(heads(), cache(), **{**ARGS, "batch": 0, "cu_new": None, "ctx_len": None}) == 0
    assert B.dflash_shared_attention(heads(), cache(), **{**ARGS, "total_new": 0, "q": None, "out": None, "rows": None}) == 0


def test_rows_size():
    h = heads()
    assert B.dflash_shared_rows_bytes(heads(dtype=1), 64, 16) == 64 * 16 * 8 * 130 * 4
    assert B.dflash_shared_rows_bytes(h, 64, 16) > 64 * 16 * 8 * 130 * 4      # and the partials of the tiles that are cut
    for batch, new in ((0, 1), (4097, 1), (1, 0), (1, 17)):
        with pytest.raises(B.DflashError):
            B.dflash_shared_rows_bytes(h, batch, new)
    assert B.load().dflash_shared_rows_bytes(None, 1, 1) == 0 and ctypes.sizeof(B.dflash_heads) == 16


def test_debug_launches():
    for bad in (-1, 3):
        with pytest.raises(B.DflashError):
            B.dflash_debug_shared_launches(bad)
    assert B.dflash_debug_shared_launches(0) == 0
