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

import ctypes

from . import binding as B


def _torch():
    import torch
    return torch


def _dtype(name: str):
    torch = _torch()
    if name not in ("bf16", "f32"):
        raise ValueError(f"dtype must be 'bf16' or 'f32', not {name!r}")
    return torch.bfloat16 if name == "bf16" else torch.float32


def _on(stream, device):
    """``with`` context that makes `stream` (a torch stream or a raw handle;
    None: the device's current one) and its device current, so that outputs
    are allocated for the stream that writes them."""
    torch = _torch()
    if stream is None:
        return torch.cuda.device(device)
    if isinstance(stream, int):   # handle 0 is the default stream; ExternalStream(0) would be one of torch's own
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"a stream of {stream.device}, tensors on {device}")
    return torch.cuda.stream(stream)


class TargetOps:
    """The cache operators for one shape of attention layer: heads, dtype,
    rotation, and the workspace the calls share (ordered on one stream).

    max_batch, max_new: the largest batch and the most new tokens per request
    (1..16) of an ``attend`` call; ``append_kv`` takes any number of tokens.
    rope_base: 0 for layers without rotation.  shared_prefix: with the scratch
    that ``attend_shared`` wants, a row of fp32 outputs per token.  The object outlives its calls:
    one that is let go frees the workspace for the stream it was made on."""

    def __init__(self, n_q_heads, n_kv_heads, head_dim, dtype="bf16", max_batch=64, max_new=16, rope_base=1e6,
                 eps=1e-6, device="cuda", shared_prefix=False):
        torch = _torch()
        self.dtype = _dtype(dtype)
        self.nq, self.nkv, self.d = int(n_q_heads), int(n_kv_heads), int(head_dim)
        self.heads = B.dflash_heads(B.DFLASH_BF16 if dtype == "bf16" else B.DFLASH_F32, self.nq, self.nkv, self.d)
        self.max_batch, self.max_new = int(max_batch), int(max_new)
        self.rope_base, self.eps = float(rope_base), float(eps)
        self.ws_bytes = B.dflash_target_workspace_bytes(self.heads, self.max_batch, self.max_new)
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=device)
        self.device = self.workspace.device
        self.rows_bytes = B.dflash_shared_rows_bytes(self.heads, self.max_batch, self.max_new) if shared_prefix else 0
        self.rows = torch.empty(self.rows_bytes, dtype=torch.uint8, device=self.device) if shared_prefix else None
        with torch.cuda.device(self.device):     # the first call may be on another stream
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()
        self.layer_sig = (self.dtype, self.device, self.nkv, self.d)
        self._torch, self._lib, self._i32 = torch, B.load(), torch.int32
        self._heads, self._ws, self._scale = ctypes.byref(self.heads), self.workspace.data_ptr(), self.d ** -0.5

    def status(self, stream=None) -> int:
        """The device status word (0 = clean), read and cleared."""
        with _torch().cuda.device(self.device):
            return B.dflash_read_status(self.workspace, stream)

    # The checks below run before every launch, and a decode step's kernels take
    # a few microseconds: plain comparisons, no helper per tensor, the C function
    # called with addresses.
    def _rows(self, name, x, width):
        if x.dtype is not self.dtype or x.device != self.device:
            raise ValueError(f"{name} must be {self.dtype} on {self.device}, not {x.dtype} on {x.device}")
        shape = x.shape
        if len(shape) != 2 or shape[1] != width or x.stride(1) != 1:
            raise ValueError(f"{name} must be [tokens][{width}] with contiguous rows, not {tuple(shape)} with "
                             f"strides {x.stride()}")
        return x.stride(0) if shape[0] > 1 else width

    def _cache(self, kv, layer, cu_new, ctx_len):
        if kv.layer_sig != self.layer_sig:
            raise ValueError(f"the cache holds (dtype, device, kv heads, head dim) {kv.layer_sig}: these operators "
                             f"want {self.layer_sig}")
        if not 0 <= layer < kv.n_layers:
            raise ValueError(f"layer {layer} of a cache with {kv.n_layers}")
        batch = ctx_len.shape[0]
        if cu_new.dtype is not self._i32 or ctx_len.dtype is not self._i32 or cu_new.shape != (batch + 1,) \
                or cu_new.device != self.device or ctx_len.device != self.device \
                or not (cu_new.is_contiguous() and ctx_len.is_contiguous()):
            raise ValueError("cu_new and ctx_len must be contiguous int32 [batch + 1] and [batch] on the cache's device")
        if batch > kv.batch_rows:
            raise ValueError(f"{batch} requests, a page table of {kv.batch_rows}")
        return batch

    def _out(self, out, rows, what):
        width = self.nq * self.d
        if out.dtype is not self.dtype or out.device != self.device or out.shape != (rows, width) \
                or not out.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {self.dtype} [{rows}][{width}] on {self.device}")

    def _results(self, rows, out, want_lse, lse):
        torch = self._torch
        if out is None:
            out = torch.empty((rows, self.nq * self.d), dtype=self.dtype, device=self.device)
        else:
            self._out(out, rows, "out")
        if lse is None:
            if want_lse:
                lse = torch.empty((rows, self.nq), dtype=torch.float32, device=self.device)
        else:
            self._lse(lse, rows)
        return out, lse

    def _lse(self, lse, rows):
        if lse.dtype is not self._torch.float32 or lse.shape != (rows, self.nq) or lse.device != self.device \
                or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous fp32 [{rows}][{self.nq}] on {self.device}")

    def append_kv(self, kv, layer, qkv, cu_new, ctx_len, g_q=None, g_k=None, q_out=None, stream=None):
        """K and V of the rows of qkv ([tokens][(nq + 2 nkv) d], the fused
        projection) into the pages of their requests, K normed (g_k) and
        rotated; returns the normed (g_q) and rotated queries [tokens][nq d].
        Rows before cu_new[0] and from cu_new[batch] on are left alone, in
        q_out too."""
        torch = self._torch
        if stream is not None or torch.cuda.current_device() != self.device.index:
            with _on(stream, self.device):
                return self.append_kv(kv, layer, qkv, cu_new, ctx_len, g_q, g_k, q_out)
        ld = self._rows("qkv", qkv, (self.nq + 2 * self.nkv) * self.d)
        batch = self._cache(kv, layer, cu_new, ctx_len)
        for g in (g_q, g_k):
            if g is not None and (g.dtype is not torch.float32 or g.shape != (self.d,) or g.device != self.device
                                  or not g.is_contiguous()):
                raise ValueError(f"g_q and g_k must be contiguous fp32 [{self.d}] on {self.device}")
        rows = qkv.shape[0]
        if q_out is None:
            q_out = torch.empty((rows, self.nq * self.d), dtype=self.dtype, device=self.device)
        else:
            self._out(q_out, rows, "q_out")
        rc = self._lib.dflash_append_kv(
            self._heads, kv.struct_ref, layer, qkv.data_ptr(), ld, None if g_q is None else g_q.data_ptr(),
            None if g_k is None else g_k.data_ptr(), self.eps, self.rope_base, cu_new.data_ptr(), rows,
            ctx_len.data_ptr(), batch, q_out.data_ptr(), self._ws, self.ws_bytes, B.raw_stream(self.device.index))
        if rc:
            B._check(rc)
        return q_out

    def attend(self, kv, layer, q, cu_new, ctx_len, max_new=None, window=0, scale=None, out=None, want_lse=False,
               lse=None, stream=None):
        """Causal attention of q ([tokens][nq d]; request b's rows
        cu_new[b]..cu_new[b+1]-1 at positions ctx_len[b]...) over the cache
        that already holds their K and V: out [tokens][nq d], with want_lse
        also the log-sum-exp [tokens][nq].  max_new: the most new tokens of a
        request in this call (default: the object's); the narrower it is, the
        better the kernel fits.  In bf16 the probabilities are rounded to bf16
        for their product with V; sums, maxima and lse are fp32."""
        torch = self._torch
        if stream is not None or torch.cuda.current_device() != self.device.index:
            with _on(stream, self.device):
                return self.attend(kv, layer, q, cu_new, ctx_len, max_new, window, scale, out, want_lse, lse)
        ld = self._rows("q", q, self.nq * self.d)
        batch = self._cache(kv, layer, cu_new, ctx_len)
        rows = q.shape[0]
        out, lse = self._results(rows, out, want_lse, lse)
        rc = self._lib.dflash_cache_attention(
            self._heads, kv.struct_ref, layer, q.data_ptr(), ld, cu_new.data_ptr(), rows, ctx_len.data_ptr(), batch,
            self.max_new if max_new is None else max_new, window, self._scale if scale is None else scale,
            out.data_ptr(), None if lse is None else lse.data_ptr(), self._ws, self.ws_bytes,
            B.raw_stream(self.device.index))
        if rc:
            B._check(rc)
        return out if lse is None else (out, lse)

    def attend_shared(self, kv, layer, q, cu_new, ctx_len, shared_len, max_new=None, scale=None, out=None,
                      want_lse=False, lse=None, stream=None):
        """``attend`` (without a window) for requests that share their first
        shared_len tokens, whole pages: those are read and multiplied once for
        all of the batch's rows, from the pages of the first request's row of
        the page table.  ctx_len counts them in.  Needs an object made with
        shared_prefix=True."""
        torch = self._torch
        if stream is not None or torch.cuda.current_device() != self.device.index:
            with _on(stream, self.device):
                return self.attend_shared(kv, layer, q, cu_new, ctx_len, shared_len, max_new, scale, out, want_lse, lse)
        if self.rows is None:
            raise ValueError("these operators were made without shared_prefix=True")
        ld = self._rows("q", q, self.nq * self.d)
        batch = self._cache(kv, layer, cu_new, ctx_len)
        rows = q.shape[0]
        out, lse = self._results(rows, out, want_lse, lse)
        rc = self._lib.dflash_shared_attention(
            self._heads, kv.struct_ref, layer, q.data_ptr(), ld, cu_new.data_ptr(), rows, ctx_len.data_ptr(), batch,
            self.max_new if max_new is None else max_new, shared_len, self._scale if scale is None else scale,
            out.data_ptr(), None if lse is None else lse.data_ptr(), self.rows.data_ptr(), self.rows_bytes, self._ws,
            self.ws_bytes, B.raw_stream(self.device.index))
        if rc:
            B._check(rc)
        return out if lse is None else (out, lse)


def token_logprobs(logits, token_ids, temperature=1.0, n_top=16, stream=None) -> dict:
    """Log probability, entropy and rank of token_ids [rows] under logits
    [rows][vocab] (bf16 or fp32, any row stride), and the n_top (0..16) most
    probable tokens with theirs: a dict of logprob, entropy [rows] (fp32), rank
    [rows] (int32), top_ids (int32) and top_logprobs (fp32) [rows][n_top].
    Rows with a negative id (the padding of ``committed``) are skipped."""
    torch = _torch()
    dev = logits.device
    if logits.is_cuda and (stream is not None or torch.cuda.current_device() != dev.index):
        with _on(stream, dev):
            return token_logprobs(logits, token_ids, temperature, n_top)
    dtype = logits.dtype
    if logits.dim() != 2 or (dtype is not torch.float32 and dtype is not torch.bfloat16) or not logits.is_cuda:
        raise ValueError("logits must be a bf16 or fp32 CUDA tensor [rows][vocab]")
    rows, vocab = logits.shape
    if logits.stride(1) != 1 and vocab > 1:
        raise ValueError("the rows of logits must be contiguous")
    if token_ids.dtype is not torch.int32 or token_ids.shape != (rows,) or token_ids.device != dev \
            or not token_ids.is_contiguous():
        raise ValueError("token_ids must be contiguous int32 [rows] on the logits' device")
    if not 0 <= n_top <= 16:
        raise ValueError("n_top must be 0..16")
    logprob = torch.empty_like(token_ids, dtype=torch.float32)
    entropy = torch.empty_like(logprob)
    rank = torch.empty_like(token_ids)
    top_ids = torch.empty((rows, n_top), dtype=torch.int32, device=dev)
    top_logprobs = torch.empty_like(top_ids, dtype=torch.float32)
    rc = B.load().dflash_token_logprobs(
        logits.data_ptr(), B.DFLASH_F32 if dtype is torch.float32 else B.DFLASH_BF16, rows, vocab,
        logits.stride(0) if rows > 1 else vocab, token_ids.data_ptr(), temperature, n_top, logprob.data_ptr(),
        entropy.data_ptr(), rank.data_ptr(), top_ids.data_ptr(), top_logprobs.data_ptr(), B.raw_stream(dev.index))
    if rc:
        B._check(rc)
    return {"logprob": logprob, "entropy": entropy, "rank": rank, "top_ids": top_ids, "top_logprobs": top_logprobs}
