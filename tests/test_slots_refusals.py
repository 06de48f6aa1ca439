"""Argument checks of the cache with a budget (append at other positions,
weights of the slots, choice and moves): every refusal returns before any device
work, so it runs without a GPU."""
import pytest

from block_diffusion_drafter_context_gb300 import binding as B
from block_diffusion_drafter_context_gb300 import build as BUILD
from tests.test_target_refusals import FAKE, cache, heads


@pytest.fixture(scope="module", autouse=True)
def built():
    BUILD.build()


def slots(**kw):
    s = dict(weights=FAKE, positions=FAKE, batch_rows=2, capacity=256)
    s.update(kw)
    return B.dflash_slots(*s.values())


APPEND = dict(layer=0, qkv=FAKE, row_stride=1536, g_q=FAKE, g_k=FAKE, eps=1e-6, rope_base=1e6, cu_new=FAKE, total_new=3,
              ctx_len=FAKE, pos=FAKE, batch=2, q_out=FAKE, workspace=FAKE, workspace_bytes=256, stream=0)
ADD = dict(layer=0, q=FAKE, q_stride=1024, lse=FAKE, cu_new=FAKE, total_new=3, ctx_len=FAKE, pos=None, n_commit=None, batch=2,
           max_new=4, first=0, scale=0.1, workspace=FAKE, workspace_bytes=256, stream=0)
PLAN = dict(layer=0, n_layers=1, ctx_len=FAKE, seq_len=FAKE, batch=2, first=0, recent=0, budget=200, moves=FAKE, top=56,
            counts=FAKE, ctx_out=FAKE, workspace=FAKE, workspace_bytes=256, stream=0)
MOVE = dict(layer=0, n_layers=1, moves=FAKE, top=56, counts=FAKE, batch=2, workspace=FAKE, workspace_bytes=256, stream=0)
CALLS = {
    "append_kv_at": (lambda hs, kv, sl, **a: B.dflash_append_kv_at(hs, kv, **a), APPEND),
    "add_weights": (B.dflash_add_weights, ADD),
    "plan_eviction": (lambda hs, kv, sl, **a: B.dflash_plan_eviction(hs, sl, **a), PLAN),
    "move_slots": (B.dflash_move_slots, MOVE),
}


def refused(name, code, hs=None, kv=None, sl=None, **kw):
    call, args = CALLS[name]
    assert set(kw) <= set(args)
    with pytest.raises(B.DflashError) as e:
        call(hs or heads(), kv or cache(), sl or slots(), **{**args, **kw})
    assert e.value.code == code and name in str(e.value)


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("hs,code", [(dict(dtype=2), -1), (dict(n_kv_heads=3), -2), (dict(head_dim=96), -4)])
def test_heads(name, hs, code):
    refused(name, code, hs=heads(**hs))


@pytest.mark.parametrize("name", ["append_kv_at", "add_weights", "move_slots"])
@pytest.mark.parametrize("kv,code", [
    (dict(k_cache=None), -1), (dict(page_table=None), -1), (dict(num_pages=0), -2), (dict(max_pages=(1 << 18) + 1), -2),
    (dict(num_pages=1 << 23), -2), (dict(v_cache=FAKE + 2), -3), (dict(page_table=FAKE + 2), -3)])
def test_cache(name, kv, code):
    refused(name, code, kv=cache(**kv))


@pytest.mark.parametrize("name", ["add_weights", "plan_eviction", "move_slots"])
@pytest.mark.parametrize("sl,code", [
    (dict(weights=None), -1), (dict(positions=None), -1), (dict(weights=FAKE + 2), -3), (dict(positions=FAKE + 1), -3),
    (dict(batch_rows=1), -2), (dict(batch_rows=4097), -2), (dict(capacity=0), -2), (dict(capacity=(1 << 24) + 1), -2)])
def test_slots(name, sl, code):
    refused(name, code, sl=slots(**sl))


@pytest.mark.parametrize("kw,code", [
    (dict(pos=None), -1), (dict(pos=FAKE + 2), -3), (dict(layer=-1), -1), (dict(qkv=FAKE + 8), -3), (dict(g_q=None), -1),
    (dict(g_k=FAKE + 2), -3), (dict(eps=-1.0), -1), (dict(rope_base=0.5), -1), (dict(q_out=FAKE + 4), -3),
    (dict(cu_new=None), -1), (dict(workspace_bytes=255), -2)])
def test_append_kv_at(kw, code):
    refused("append_kv_at", code, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(layer=-1), -1), (dict(q=None), -1), (dict(q=FAKE + 8), -3), (dict(q_stride=1000), -2), (dict(lse=None), -1),
    (dict(lse=FAKE + 2), -3), (dict(cu_new=FAKE + 2), -3), (dict(total_new=-1), -1), (dict(ctx_len=None), -1),
    (dict(pos=FAKE + 1), -3), (dict(n_commit=FAKE + 2), -3), (dict(batch=4097), -1), (dict(max_new=0), -1),
    (dict(max_new=17), -1), (dict(first=-1), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(workspace=None), -1), (dict(workspace_bytes=255), -2)])
def test_add_weights(kw, code):
    refused("add_weights", code, **kw)


def test_add_weights_wants_a_slot_per_place_of_the_page_table():
    refused("add_weights", -2, sl=slots(capacity=255))


@pytest.mark.parametrize("kw,code", [
    (dict(layer=-1), -1), (dict(n_layers=-1), -1), (dict(batch=-1), -1), (dict(ctx_len=None), -1), (dict(seq_len=None), -1),
    (dict(ctx_out=None), -1), (dict(counts=None), -1), (dict(moves=None), -1), (dict(top=55), -2), (dict(budget=0), -1),
    (dict(budget=(1 << 24) + 1), -1), (dict(first=-1), -1), (dict(first=200), -1), (dict(recent=-1), -1),
    (dict(first=100, recent=101), -1), (dict(first=128, recent=3, budget=130), -1), (dict(recent=201), -1),
    (dict(recent=2 ** 31 - 1), -1), (dict(moves=FAKE + 2), -3), (dict(counts=FAKE + 1), -3), (dict(ctx_out=FAKE + 2), -3),
    (dict(seq_len=FAKE + 2), -3), (dict(workspace=None), -1), (dict(workspace=FAKE + 4), -3),
    (dict(workspace_bytes=255), -2), (dict(n_layers=1 << 27), -2)])
def test_plan_eviction(kw, code):
    refused("plan_eviction", code, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(layer=-1), -1), (dict(n_layers=-1), -1), (dict(moves=None), -1), (dict(counts=None), -1), (dict(top=-1), -1),
    (dict(top=(1 << 24) + 1), -1), (dict(moves=FAKE + 2), -3), (dict(counts=FAKE + 2), -3), (dict(batch=-1), -1),
    (dict(workspace=None), -1), (dict(workspace_bytes=0), -2), (dict(n_layers=1 << 27), -2)])
def test_move_slots(kw, code):
    refused("move_slots", code, **kw)


def test_empty_calls_do_nothing():
    none = dict(batch=0, cu_new=None, ctx_len=None)
    assert B.dflash_append_kv_at(heads(), cache(), **{**APPEND, **none, "pos": None}) == 0
    assert B.dflash_add_weights(heads(), cache(), slots(), **{**ADD, **none, "lse": None}) == 0
    assert B.dflash_add_weights(heads(), cache(), slots(), **{**ADD, "total_new": 0, "q": None, "lse": None}) == 0
    assert B.dflash_plan_eviction(heads(), slots(), **{**PLAN, "n_layers": 0, "counts": None, "moves": None}) == 0
    assert B.dflash_plan_eviction(heads(), slots(), **{**PLAN, "batch": 0, "ctx_len": None, "seq_len": None,
                                                       "ctx_out": None, "moves": None}) == 0
    assert B.dflash_move_slots(heads(), cache(), slots(), **{**MOVE, "top": 0, "moves": None, "counts": None}) == 0
    assert B.dflash_move_slots(heads(), cache(page_table=None), slots(), **{**MOVE, "batch": 0, "moves": None}) == 0


def test_wrapper_checks():
    torch = pytest.importorskip("torch")
    from block_diffusion_drafter_context_gb300.target import SlotWeights
    w, p = torch.zeros(1, 2, 2, 64), torch.zeros(1, 2, 2, 64, dtype=torch.int32)
    for bad in ((w[0], p[0]), (w.double(), p), (w, p.long()), (w, p[..., :32]), (w.transpose(1, 2), p), (w, p)):
        with pytest.raises(ValueError):      # the last: not on a CUDA device
            SlotWeights.from_tensors(*bad)
