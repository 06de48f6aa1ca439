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


class SlotWeights:
    """What a cache with a budget keeps of every slot, per layer, request and kv
    head: the attention weight its token received (``add_weights``) and its
    position.  A new one counts every slot's position as its number and no
    weight, as after a prompt.  capacity: at least 64 slots per page of the page
    table's rows."""

    def __init__(self, n_layers, batch, n_kv_heads, capacity, device="cuda"):
        torch = _torch()
        shape = (int(n_layers), int(batch), int(n_kv_heads), int(capacity))
        self.weights = torch.zeros(shape, dtype=torch.float32, device=device)
        self.positions = torch.arange(shape[3], dtype=torch.int32, device=device).expand(shape).contiguous()
        self._describe()

    def _describe(self):
        self.n_layers, self.batch_rows, self.nkv, self.capacity = (int(n) for n in self.weights.shape)
        self.device = self.weights.device
        self.struct = B.dflash_slots(self.weights.data_ptr(), self.positions.data_ptr(), self.batch_rows, self.capacity)
        self.struct_ref = ctypes.byref(self.struct)

    @classmethod
    def from_tensors(cls, weights, positions):
        """Over tensors the caller already has: weights fp32 and positions int32
        [n_layers][batch][n_kv_heads][capacity], contiguous on one CUDA device."""
        torch = _torch()
        if weights.dim() != 4 or weights.dtype != torch.float32 or positions.dtype != torch.int32 \
                or positions.shape != weights.shape:
            raise ValueError("weights must be fp32 and positions int32, both [layers][batch][n_kv][capacity]")
        if not (weights.is_contiguous() and positions.is_contiguous() and weights.is_cuda
                and positions.device == weights.device):
            raise ValueError("weights and positions must be contiguous on one CUDA device")
        s = cls.__new__(cls)
        s.weights, s.positions = weights, positions
        s._describe()
        return s


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

    def _per_request(self, name, x, batch):
        if x.dtype is not self._i32 or x.shape != (batch,) or x.device != self.device or not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32 [{batch}] on {self.device}")
        return x.data_ptr()

    def _slots(self, slots, batch, layer):
        if slots.nkv != self.nkv or slots.device != self.device or slots.batch_rows < batch:
            raise ValueError(f"slots of {slots.batch_rows} requests x {slots.nkv} kv heads on {slots.device}: these "
                             f"operators want {batch} x {self.nkv} on {self.device}")
        if layer is None:
            return 0, slots.n_layers
        if not 0 <= layer < slots.n_layers:
            raise ValueError(f"layer {layer} of slots with {slots.n_layers}")
        return layer, 1

    def append_kv(self, kv, layer, qkv, cu_new, ctx_len, g_q=None, g_k=None, q_out=None, stream=None, pos=None):
        """K and V of the rows of qkv ([tokens][(nq + 2 nkv) d], the fused
        projection) into the pages of their requests, K normed (g_k) and
        rotated; returns the normed (g_q) and rotated queries [tokens][nq d].
        Rows before cu_new[0] and from cu_new[batch] on are left alone, in
        q_out too.  pos (int32 [batch]): the position of each request's first
        new token, where that is not its slot ctx_len (after an eviction)."""
        torch = self._torch
        if stream is not None or torch.cuda.current_device() != self.device.index:
            with _on(stream, self.device):
                return self.append_kv(kv, layer, qkv, cu_new, ctx_len, g_q, g_k, q_out, pos=pos)
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
        args = (self._heads, kv.struct_ref, layer, qkv.data_ptr(), ld, None if g_q is None else g_q.data_ptr(),
                None if g_k is None else g_k.data_ptr(), self.eps, self.rope_base, cu_new.data_ptr(), rows,
                ctx_len.data_ptr())
        end = (batch, q_out.data_ptr(), self._ws, self.ws_bytes, B.raw_stream(self.device.index))
        if pos is None:
            rc = self._lib.dflash_append_kv(*args, *end)
        else:
            rc = self._lib.dflash_append_kv_at(*args, self._per_request("pos", pos, batch), *end)
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

    def add_weights(self, kv, layer, slots, q, lse, cu_new, ctx_len, pos=None, n_commit=None, max_new=None, first=0,
                    scale=None, stream=None):
        """Adds to the slots' weights (a ``SlotWeights``) the attention that the
        committed new tokens paid to each cached token from slot `first` on.
        q, cu_new, ctx_len and scale as of the ``attend`` or ``attend_shared``
        before (without a window), lse what it gave.  n_commit (int32 [batch]):
        how many of each request's new tokens count, all by default; their own
        slots start from 0 and get the positions pos[b] ... (default: ctx_len)."""
        torch = self._torch
        if stream is not None or torch.cuda.current_device() != self.device.index:
            with _on(stream, self.device):
                return self.add_weights(kv, layer, slots, q, lse, cu_new, ctx_len, pos, n_commit, max_new, first, scale)
        ld = self._rows("q", q, self.nq * self.d)
        batch = self._cache(kv, layer, cu_new, ctx_len)
        self._slots(slots, batch, layer)
        rows = q.shape[0]
        self._lse(lse, rows)
        rc = self._lib.dflash_add_weights(
            self._heads, kv.struct_ref, slots.struct_ref, layer, q.data_ptr(), ld, lse.data_ptr(), cu_new.data_ptr(), rows,
            ctx_len.data_ptr(), None if pos is None else self._per_request("pos", pos, batch),
            None if n_commit is None else self._per_request("n_commit", n_commit, batch), batch,
            self.max_new if max_new is None else max_new, first, self._scale if scale is None else scale, self._ws,
            self.ws_bytes, B.raw_stream(self.device.index))
        if rc:
            B._check(rc)

    def plan_eviction(self, slots, ctx_len, seq_len, budget, recent=0, first=0, layer=None, stream=None):
        """What a cache keeps of requests with more than `budget` tokens, for one
        layer of `slots` or all: the first `first` slots, the positions from
        seq_len - recent on, then the heaviest.  Returns (moves
        [layers][batch][n_kv][2][top], counts [layers][batch][n_kv], ctx
        [batch]): slots moved into and from (-1 behind the count), and the
        tokens that are left, min(ctx_len, budget)."""
        torch = self._torch
        if stream is not None or torch.cuda.current_device() != self.device.index:
            with _on(stream, self.device):
                return self.plan_eviction(slots, ctx_len, seq_len, budget, recent, first, layer)
        batch = ctx_len.shape[0]
        layer, n = self._slots(slots, batch, layer)
        ctx, seq = self._per_request("ctx_len", ctx_len, batch), self._per_request("seq_len", seq_len, batch)
        top = max(0, min(budget - first, slots.capacity - budget))
        moves = torch.empty((n, batch, self.nkv, 2, top), dtype=torch.int32, device=self.device)
        counts = torch.empty((n, batch, self.nkv), dtype=torch.int32, device=self.device)
        left = torch.empty_like(ctx_len)
        rc = self._lib.dflash_plan_eviction(
            self._heads, slots.struct_ref, layer, n, ctx, seq, batch, first, recent, budget, moves.data_ptr(), top,
            counts.data_ptr(), left.data_ptr(), self._ws, self.ws_bytes, B.raw_stream(self.device.index))
        if rc:
            B._check(rc)
        return moves, counts, left

    def move_slots(self, kv, slots, moves, counts, layer=None, stream=None):
        """Carries out the moves of ``plan_eviction`` on K, V, weights and
        positions, in the layers that the plan was made for."""
        torch = self._torch
        if stream is not None or torch.cuda.current_device() != self.device.index:
            with _on(stream, self.device):
                return self.move_slots(kv, slots, moves, counts, layer)
        if kv.layer_sig != self.layer_sig:
            raise ValueError(f"the cache holds (dtype, device, kv heads, head dim) {kv.layer_sig}: these operators "
                             f"want {self.layer_sig}")
        batch = counts.shape[1] if counts.dim() == 3 else -1
        layer, n = self._slots(slots, batch, layer)
        if counts.shape != (n, batch, self.nkv) or moves.dim() != 5 or moves.shape[:4] != (n, batch, self.nkv, 2) \
                or moves.dtype is not self._i32 or counts.dtype is not self._i32 or moves.device != self.device \
                or counts.device != self.device or not (moves.is_contiguous() and counts.is_contiguous()):
            raise ValueError(f"moves and counts must be what plan_eviction gave for {n} layers: contiguous int32 "
                             "[layers][batch][n_kv][2][top] and [layers][batch][n_kv]")
        if layer + n > kv.n_layers or batch > kv.batch_rows:
            raise ValueError(f"{n} layers from {layer} on and {batch} requests, a cache of {kv.n_layers} and "
                             f"{kv.batch_rows}")
        rc = self._lib.dflash_move_slots(
            self._heads, kv.struct_ref, slots.struct_ref, layer, n, moves.data_ptr(), moves.shape[4], counts.data_ptr(),
            batch, self._ws, self.ws_bytes, B.raw_stream(self.device.index))
        if rc:
            B._check(rc)

    def evict(self, kv, slots, ctx_len, seq_len, budget, recent=0, first=0, layer=None, stream=None):
        """``plan_eviction`` and ``move_slots``: cuts requests with more than
        `budget` tokens down to it and returns the tokens that are left.  With
        pages that requests share, `first` is the shared prefix's length."""
        moves, counts, left = self.plan_eviction(slots, ctx_len, seq_len, budget, recent, first, layer, stream)
        if moves.shape[4]:
            self.move_slots(kv, slots, moves, counts, layer, stream)
        return left


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
