"""The target model's side of a speculative step, on the drafter's paged-cache
layout: q / k norm + rotation + append, causal attention of the newest tokens,
and log probabilities of given tokens.

Marshalling and argument checks only: the arithmetic happens in libdflash.
A verification pass of one layer is

    q = ops.append_kv(kv, layer, qkv, cu_new, ctx_len, g_q, g_k)
    out = ops.attend(kv, layer, q, cu_new, ctx_len)

with ctx_len the tokens cached *before* the new ones (rejected tokens need no
undoing: the next step overwrites their slots), and after the last layer's
logits and the verification, ``token_logprobs(logits, committed.reshape(-1))``.
"""
from __future__ import annotations

from . import binding as B


def _torch():
    import torch
    return torch


def _dtype(name: str):
    torch = _torch()
    if name not in ("bf16", "f32"):
        raise ValueError(f"dtype must be 'bf16' or 'f32', not {name!r}")
    return torch.bfloat16 if name == "bf16" else torch.float32


def _on(stream):
    """``with`` context that makes `stream` (a torch stream or a raw handle)
    current, so that outputs are allocated for the stream that writes them."""
    torch = _torch()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class TargetOps:
    """The cache operators for one shape of attention layer: heads, dtype,
    rotation, and the workspace the calls share (ordered on one stream).

    max_batch, max_new: the largest batch and the most new tokens per request
    (1..16) of an ``attend`` call; ``append_kv`` takes any number of tokens.
    rope_base: 0 for layers without rotation."""

    def __init__(self, n_q_heads, n_kv_heads, head_dim, dtype="bf16", max_batch=64, max_new=16, rope_base=1e6,
                 eps=1e-6, device="cuda"):
        torch = _torch()
        self.dtype = _dtype(dtype)
        self.nq, self.nkv, self.d = int(n_q_heads), int(n_kv_heads), int(head_dim)
        self.heads = B.dflash_heads(B.DFLASH_BF16 if dtype == "bf16" else B.DFLASH_F32, self.nq, self.nkv, self.d)
        self.max_batch, self.max_new = int(max_batch), int(max_new)
        self.rope_base, self.eps = float(rope_base), float(eps)
        self.ws_bytes = B.dflash_target_workspace_bytes(self.heads, self.max_batch, self.max_new)
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=device)
        self.device = self.workspace.device

    def status(self, stream=None) -> int:
        """The device status word (0 = clean), read and cleared."""
        with _torch().cuda.device(self.device):
            return B.dflash_read_status(self.workspace, stream)

    def _rows(self, name, x, width):
        if x.dtype != self.dtype or x.device != self.device:
            raise ValueError(f"{name} must be {self.dtype} on {self.device}, not {x.dtype} on {x.device}")
        if x.dim() != 2 or x.shape[1] != width or (x.shape[1] > 1 and x.stride(1) != 1):
            raise ValueError(f"{name} must be [tokens][{width}] with contiguous rows, not {tuple(x.shape)} with "
                             f"strides {x.stride()}")
        return x.stride(0) if x.shape[0] > 1 else max(x.stride(0), width)

    def _cache(self, kv, layer, cu_new, ctx_len):
        torch = _torch()
        k = kv.k
        if k.dtype != self.dtype or k.device != self.device or k.shape[2] != self.nkv or k.shape[4] != self.d:
            raise ValueError(f"the cache is {k.dtype} {tuple(k.shape)} on {k.device}: these operators want "
                             f"{self.dtype}, {self.nkv} kv heads of {self.d} on {self.device}")
        if not 0 <= layer < k.shape[0]:
            raise ValueError(f"layer {layer} of a cache with {k.shape[0]}")
        batch = ctx_len.shape[0]
        if cu_new.dtype != torch.int32 or ctx_len.dtype != torch.int32 or cu_new.shape != (batch + 1,) \
                or cu_new.device != self.device or ctx_len.device != self.device \
                or not (cu_new.is_contiguous() and ctx_len.is_contiguous()):
            raise ValueError("cu_new and ctx_len must be contiguous int32 [batch + 1] and [batch] on the cache's device")
        if batch > kv.page_table.shape[0]:
            raise ValueError(f"{batch} requests, a page table of {kv.page_table.shape[0]}")
        return batch

    def _out(self, out, rows, what="out"):
        width = self.nq * self.d
        if out is None:
            return _torch().empty((rows, width), dtype=self.dtype, device=self.device)
        if out.dtype != self.dtype or out.device != self.device or out.shape != (rows, width) \
                or not out.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {self.dtype} [{rows}][{width}] on {self.device}")
        return out

    def append_kv(self, kv, layer, qkv, cu_new, ctx_len, g_q=None, g_k=None, q_out=None, stream=None):
        """K and V of the rows of qkv ([tokens][(nq + 2 nkv) d], the fused
        projection) into the pages of their requests, K normed (g_k) and
        rotated; returns the normed (g_q) and rotated queries [tokens][nq d].
        Rows from cu_new[batch] on are left alone, in q_out too."""
        if stream is not None:
            with _on(stream):
                return self.append_kv(kv, layer, qkv, cu_new, ctx_len, g_q, g_k, q_out)
        ld = self._rows("qkv", qkv, (self.nq + 2 * self.nkv) * self.d)
        batch = self._cache(kv, layer, cu_new, ctx_len)
        torch = _torch()
        for g in (g_q, g_k):
            if g is not None and (g.dtype != torch.float32 or g.shape != (self.d,) or g.device != self.device
                                  or not g.is_contiguous()):
                raise ValueError(f"g_q and g_k must be contiguous fp32 [{self.d}] on {self.device}")
        rows = qkv.shape[0]
        q_out = self._out(q_out, rows, "q_out")
        with B.on_device(self.device):
            B.dflash_append_kv(self.heads, kv.struct, layer, qkv, ld, g_q, g_k, self.eps, self.rope_base, cu_new,
                               rows, ctx_len, batch, q_out, self.workspace, self.ws_bytes)
        return q_out

    def attend(self, kv, layer, q, cu_new, ctx_len, max_new=None, window=0, scale=None, out=None, want_lse=False,
               lse=None, stream=None):
        """Causal attention of q ([tokens][nq d]; request b's rows
        cu_new[b]..cu_new[b+1]-1 at positions ctx_len[b]...) over the cache
        that already holds their K and V: out [tokens][nq d], with want_lse
        also the log-sum-exp [tokens][nq].  max_new: the most new tokens of a
        request in this call (default: the object's)."""
        if stream is not None:
            with _on(stream):
                return self.attend(kv, layer, q, cu_new, ctx_len, max_new, window, scale, out, want_lse, lse)
        ld = self._rows("q", q, self.nq * self.d)
        batch = self._cache(kv, layer, cu_new, ctx_len)
        rows = q.shape[0]
        out = self._out(out, rows)
        torch = _torch()
        if want_lse and lse is None:
            lse = torch.empty((rows, self.nq), dtype=torch.float32, device=self.device)
        elif lse is not None and (lse.dtype != torch.float32 or lse.shape != (rows, self.nq)
                                  or lse.device != self.device or not lse.is_contiguous()):
            raise ValueError(f"lse must be a contiguous fp32 [{rows}][{self.nq}] on {self.device}")
        with B.on_device(self.device):
            B.dflash_cache_attention(self.heads, kv.struct, layer, q, ld, cu_new, rows, ctx_len, batch,
                                     self.max_new if max_new is None else max_new, window,
                                     self.d ** -0.5 if scale is None else scale, out, lse, self.workspace,
                                     self.ws_bytes)
        return (out, lse) if lse is not None else out


def token_logprobs(logits, token_ids, temperature=1.0, n_top=16, stream=None) -> dict:
    """Log probability, entropy and rank of token_ids [rows] under logits
    [rows][vocab] (bf16 or fp32, any row stride), and the n_top (0..16) most
    probable tokens with theirs: a dict of logprob, entropy [rows] (fp32), rank
    [rows] (int32), top_ids (int32) and top_logprobs (fp32) [rows][n_top].
    Rows with a negative id (the padding of ``committed``) are skipped."""
    if stream is not None:
        with _on(stream):
            return token_logprobs(logits, token_ids, temperature, n_top)
    torch = _torch()
    if logits.dim() != 2 or logits.dtype not in (torch.bfloat16, torch.float32) or not logits.is_cuda:
        raise ValueError("logits must be a bf16 or fp32 CUDA tensor [rows][vocab]")
    rows, vocab = logits.shape
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("the rows of logits must be contiguous")
    if token_ids.dtype != torch.int32 or token_ids.shape != (rows,) or token_ids.device != logits.device \
            or not token_ids.is_contiguous():
        raise ValueError("token_ids must be contiguous int32 [rows] on the logits' device")
    dev = logits.device
    out = {"logprob": torch.empty(rows, dtype=torch.float32, device=dev),
           "entropy": torch.empty(rows, dtype=torch.float32, device=dev),
           "rank": torch.empty(rows, dtype=torch.int32, device=dev),
           "top_ids": torch.empty((rows, n_top), dtype=torch.int32, device=dev),
           "top_logprobs": torch.empty((rows, n_top), dtype=torch.float32, device=dev)}
    with B.on_device(dev):
        B.dflash_token_logprobs(logits, B.DFLASH_BF16 if logits.dtype == torch.bfloat16 else B.DFLASH_F32, rows, vocab,
                                logits.stride(0) if rows > 1 else vocab, token_ids, temperature, n_top, out["logprob"],
                                out["entropy"], out["rank"], out["top_ids"], out["top_logprobs"])
    return out
