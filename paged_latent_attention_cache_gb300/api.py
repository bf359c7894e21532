"""User-facing operator object over the C ABI.

``PagedLatentAttention`` holds the operator parameters, the split-KV
workspace and the device error word, all allocated once at construction;
``forward`` then only enqueues the library's kernels (write phase, decode
phase for the decode-first sequences, prefill phase for the rest) and is
safe to record into a CUDA graph after one eager call.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import binding as B


class PagedLatentAttention:
    def __init__(self, *, dtype: torch.dtype, num_heads: int, head_size: int,
                 v_head_size: int = 0, rotary_offset: int = 0, rotary_dim: int = 0,
                 rotary_interleaved: int = 0, cos_rows: int = 1, block_size: int,
                 num_blocks: int, max_blocks_per_seq: int, scale: float = 0.0,
                 softcap: float = 0.0, local_window_size: int = -1, max_seqs: int,
                 max_tokens: int, device="cuda", portable: bool = False,
                 own_slots: bool = False, cache_dtype=None, k_scale: float = 1.0):
        self.dtype = dtype
        self.num_heads = num_heads
        self.head_size = head_size
        self.v_head_size = v_head_size or head_size
        self.params = B.make_params(
            dtype=dtype, num_heads=num_heads, head_size=head_size, v_head_size=v_head_size,
            rotary_offset=rotary_offset, rotary_dim=rotary_dim,
            rotary_interleaved=rotary_interleaved, cos_rows=cos_rows, block_size=block_size,
            num_blocks=num_blocks, max_blocks_per_seq=max_blocks_per_seq, scale=scale,
            softcap=softcap, local_window_size=local_window_size,
            flags=B.PA_FLAG_PORTABLE if portable else 0, cache_dtype=cache_dtype,
            k_scale=k_scale)
        s = B.pa_latent_validate(self.params)
        if s != B.PA_OK:
            raise B.PaError(s, B.last_error())
        # the same parameters for the first read call after the write phase
        # (own_slots: every slot is its token's own position, see
        # PA_FLAG_OWN_SLOTS)
        self.params_after_write = B.pa_latent_params.from_buffer_copy(self.params)
        self.params_after_write.flags |= B.PA_FLAG_AFTER_WRITE | (
            B.PA_FLAG_OWN_SLOTS if own_slots else 0)
        self.device = torch.device(device)
        self.max_seqs, self.max_tokens = max_seqs, max_tokens
        self.workspace = B.alloc_workspace(self.params, max_seqs, max_tokens, self.device)
        self.err_flags = torch.zeros(1, dtype=torch.int32, device=self.device)

    @classmethod
    def from_workload(cls, w, device="cuda", portable=False,
                      own_slots=True) -> "PagedLatentAttention":
        """Operator for a generated workload; its slot mappings point every
        token at its own position (see ``workloads.make_workload``)."""
        return cls(dtype=w.dtype, num_heads=w.num_heads, head_size=w.head_size,
                   v_head_size=w.v_head_size, rotary_offset=w.rotary_offset,
                   rotary_dim=w.rotary_dim, rotary_interleaved=w.rotary_interleaved,
                   cos_rows=w.cos_rows, block_size=w.block_size, num_blocks=w.num_blocks,
                   max_blocks_per_seq=w.max_blocks_per_seq, scale=w.scale, softcap=w.softcap,
                   local_window_size=w.local_window_size, max_seqs=w.num_seqs,
                   max_tokens=max(w.num_tokens, 1), device=device, portable=portable,
                   own_slots=own_slots, cache_dtype=w.cache_dtype, k_scale=w.k_scale)

    def kernel_family(self, phase: int) -> int:
        return B.pa_latent_kernel_family(self.params, phase)

    def write(self, key, cos_cache, sin_cache, slot_mapping, cumseq, past, key_cache,
              stream=None):
        B.pa_latent_write(self.params, key, cos_cache, sin_cache, slot_mapping, cumseq, past,
                          key_cache, self.err_flags, stream)

    def _read_params(self, after_write: bool):
        return self.params_after_write if after_write else self.params

    def decode(self, query, key_cache, cos_cache, sin_cache, cumseq, past, block_table, out,
               seq_begin=0, seq_end=None, stream=None, after_write: bool = False):
        """Decode phase over sequences [seq_begin, seq_end). ``after_write``:
        this call directly follows ``write`` on the same stream (see
        PA_FLAG_AFTER_WRITE)."""
        B.pa_latent_decode(self._read_params(after_write), query, key_cache, cos_cache, sin_cache, cumseq, past,
                           block_table, out, seq_begin, seq_end, self.workspace,
                           self.err_flags, stream)

    def prefill(self, query, key_cache, cos_cache, sin_cache, cumseq, past, block_table, out,
                seq_begin=0, seq_end=None, stream=None, after_write: bool = False):
        B.pa_latent_prefill(self._read_params(after_write), query, key_cache, cos_cache, sin_cache, cumseq, past,
                            block_table, out, seq_begin, seq_end, self.workspace,
                            self.err_flags, stream)

    def mixed(self, query, key_cache, cos_cache, sin_cache, cumseq, past, block_table, out,
              num_decode_seqs: int, stream=None, after_write: bool = False):
        """Read phase of the whole batch in one call: decode over
        [0, num_decode_seqs), prefill over the rest (see pa_latent_mixed)."""
        B.pa_latent_mixed(self._read_params(after_write), query, key_cache, cos_cache, sin_cache,
                          cumseq, past, block_table, out, num_decode_seqs, self.workspace,
                          self.err_flags, stream)

    def forward(self, query, key, key_cache, cos_cache, sin_cache, cumseq, past, block_table,
                slot_mapping, num_decode_seqs: int, out: Optional[torch.Tensor] = None,
                stream=None, one_call: bool = True) -> torch.Tensor:
        """Write phase over all tokens, then decode over sequences
        [0, num_decode_seqs) and prefill over the rest; returns ``out``. A
        batch with both kinds of sequences is read by one pa_latent_mixed
        call (``one_call=False``: a decode call and a prefill call)."""
        T = query.shape[0]
        nseq = past.shape[0]
        if out is None:
            out = torch.empty(T, self.num_heads * self.v_head_size, dtype=self.dtype,
                              device=query.device)
        self.write(key, cos_cache, sin_cache, slot_mapping, cumseq, past, key_cache, stream)
        if one_call and 0 < num_decode_seqs < nseq:
            self.mixed(query, key_cache, cos_cache, sin_cache, cumseq, past, block_table, out,
                       num_decode_seqs, stream, after_write=True)
            return out
        if num_decode_seqs > 0:
            self.decode(query, key_cache, cos_cache, sin_cache, cumseq, past, block_table, out,
                        0, num_decode_seqs, stream, after_write=True)
        if num_decode_seqs < nseq:
            self.prefill(query, key_cache, cos_cache, sin_cache, cumseq, past, block_table, out,
                         num_decode_seqs, nseq, stream, after_write=num_decode_seqs == 0)
        return out

    def error_flags(self) -> int:
        """Reads the device error word (synchronises with the device)."""
        return int(self.err_flags.item())

    def reset_error_flags(self):
        self.err_flags.zero_()


class SeparateAttention:
    """The op's SEPARATE mode (grouped-query attention over separate key and
    value caches, optional head sink and q/k RMSNorm) over the C ABI: holds
    the parameters, the decode workspace and the error word; ``forward``
    issues write -> decode -> prefill like ``PagedLatentAttention``."""

    def __init__(self, *, dtype: torch.dtype, num_heads: int, kv_num_heads: int, head_size: int,
                 v_head_size: int = 0, rotary_offset: int = 0, rotary_dim: int = 0,
                 rotary_interleaved: int = 0, cos_rows: int = 1, block_size: int,
                 num_blocks: int, max_blocks_per_seq: int, scale: float = 0.0,
                 softcap: float = 0.0, local_window_size: int = -1, rms_eps: float = 1e-6,
                 max_seqs: int, max_tokens: int, device="cuda", own_slots: bool = False):
        self.dtype = dtype
        self.num_heads = num_heads
        self.v_head_size = v_head_size or head_size
        self.params = B.make_separate_params(
            dtype=dtype, num_heads=num_heads, kv_num_heads=kv_num_heads, head_size=head_size,
            v_head_size=v_head_size, rotary_offset=rotary_offset, rotary_dim=rotary_dim,
            rotary_interleaved=rotary_interleaved, cos_rows=cos_rows, block_size=block_size,
            num_blocks=num_blocks, max_blocks_per_seq=max_blocks_per_seq, scale=scale,
            softcap=softcap, local_window_size=local_window_size, rms_eps=rms_eps)
        s = B.pa_separate_validate(self.params)
        if s != B.PA_OK:
            raise B.PaError(s, B.last_error())
        self.params_after_write = B.pa_separate_params.from_buffer_copy(self.params)
        self.params_after_write.flags |= B.PA_FLAG_AFTER_WRITE | (
            B.PA_FLAG_OWN_SLOTS if own_slots else 0)
        self.device = torch.device(device)
        n = B.pa_separate_workspace_size(self.params, max_seqs, max_tokens)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device) if n else None
        self.err_flags = torch.zeros(1, dtype=torch.int32, device=self.device)

    @classmethod
    def from_workload(cls, w, device="cuda", own_slots=True) -> "SeparateAttention":
        return cls(dtype=w.dtype, num_heads=w.num_heads, kv_num_heads=w.kv_num_heads,
                   head_size=w.head_size, v_head_size=w.v_head_size,
                   rotary_offset=w.rotary_offset, rotary_dim=w.rotary_dim,
                   rotary_interleaved=w.rotary_interleaved, cos_rows=w.cos_rows,
                   block_size=w.block_size, num_blocks=w.num_blocks,
                   max_blocks_per_seq=w.max_blocks_per_seq, scale=w.scale, softcap=w.softcap,
                   local_window_size=w.local_window_size, rms_eps=w.rms_eps,
                   max_seqs=w.num_seqs, max_tokens=max(w.num_tokens, 1), device=device,
                   own_slots=own_slots)

    def forward(self, query, key, value, key_cache, value_cache, cos_cache, sin_cache, cumseq,
                past, block_table, slot_mapping, num_decode_seqs: int, head_sink=None,
                q_norm_weight=None, k_norm_weight=None, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        T, nseq = query.shape[0], past.shape[0]
        if out is None:
            out = torch.empty(T, self.num_heads * self.v_head_size, dtype=self.dtype,
                              device=query.device)
        B.pa_separate_write(self.params, key, value, cos_cache, sin_cache, k_norm_weight,
                            slot_mapping, cumseq, past, key_cache, value_cache, self.err_flags,
                            stream)
        if num_decode_seqs > 0:
            B.pa_separate_decode(self.params_after_write, query, key_cache, value_cache,
                                 cos_cache, sin_cache, q_norm_weight, head_sink, cumseq, past,
                                 block_table, out, 0, num_decode_seqs, self.workspace,
                                 self.err_flags, stream)
        if num_decode_seqs < nseq:
            p = self.params_after_write if num_decode_seqs == 0 else self.params
            B.pa_separate_prefill(p, query, key_cache, value_cache, cos_cache, sin_cache,
                                  q_norm_weight, head_sink, cumseq, past, block_table, out,
                                  num_decode_seqs, nseq, self.workspace, self.err_flags, stream)
        return out

    def error_flags(self) -> int:
        return int(self.err_flags.item())


def _require(ok: bool, message: str):
    if not ok:
        raise B.PaError(B.PA_ERR_INVALID_ARGUMENT, message)


_NOTHING = contextlib.nullcontext()


def _device(index: int):
    """Makes a device current for a block (nothing to do where it is)."""
    return _NOTHING if torch.cuda.current_device() == index else torch.cuda.device(index)


def _allocating(stream, index: int):
    """What is allocated in this block is memory of ``stream``, a call's
    argument: a torch stream, a handle, or None for the current stream."""
    if stream is None:
        return _NOTHING
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=index) if handle else \
            torch.cuda.default_stream(index)
    return torch.cuda.stream(stream)


class _Filled:
    """Orders an object's first call behind what its constructor enqueued on
    the stream that was current then, whatever stream the call is given. (Not
    across a graph's borders: a capture starts behind everything, and could
    not wait for an event from outside.)"""

    def __init__(self, index: int):
        with _device(index):
            self.stream = B.raw_stream(None)
            self.captured = torch.cuda.is_current_stream_capturing()
            if not self.captured:
                self.event = torch.cuda.Event()
                self.event.record()

    def before(self, stream):
        """Makes ``stream`` wait."""
        raw = B.raw_stream(stream)
        if raw != self.stream and not self.captured:
            with _allocating(raw, torch.cuda.current_device()):
                if not torch.cuda.is_current_stream_capturing():
                    self.event.wait()


class DifferentialAttention:
    """Differential attention over paged caches (include/pa_diff.h): two query
    and key maps per head and one value, the difference of the two softmax
    maps with the layer's learned lambda, RMSNorm per head. Holds the
    parameters, the workspace and the error word; ``forward`` issues write ->
    decode -> prefill like ``PagedLatentAttention``. Calls of one object share
    its workspace: order them (one stream, or events).

    ``query`` [T, H*2*hs], ``key`` [T, kvH*2*hs], ``value`` [T, kvH*vhs],
    ``key_cache`` [num_blocks, bs, kvH, 2, hs], ``value_cache`` [num_blocks,
    bs, kvH, vhs], ``lambda_vectors`` float32 [4, hs], ``norm_weight`` [vhs];
    ``v_head_size`` 0 means 2 * hs. The block tables and slots can come from a
    ``PagePool`` over the two caches."""

    def __init__(self, *, dtype: torch.dtype, num_heads: int, kv_num_heads: int, head_size: int,
                 v_head_size: int = 0, rotary_offset: int = 0, rotary_dim: int = 0,
                 rotary_interleaved: int = 0, cos_rows: int = 1, block_size: int,
                 num_blocks: int, max_blocks_per_seq: int, scale: float = 0.0,
                 softcap: float = 0.0, local_window_size: int = -1, lambda_init: float,
                 norm_eps: float = 1e-5, max_seqs: int, max_tokens: int, device="cuda",
                 own_slots: bool = False):
        self.dtype = dtype
        self.num_heads, self.kv_num_heads = num_heads, kv_num_heads
        self.head_size, self.v_head_size = head_size, v_head_size or 2 * head_size
        self.params = B.make_diff_params(
            dtype=dtype, num_heads=num_heads, kv_num_heads=kv_num_heads, head_size=head_size,
            v_head_size=v_head_size, rotary_offset=rotary_offset, rotary_dim=rotary_dim,
            rotary_interleaved=rotary_interleaved, cos_rows=cos_rows, block_size=block_size,
            num_blocks=num_blocks, max_blocks_per_seq=max_blocks_per_seq, scale=scale,
            softcap=softcap, local_window_size=local_window_size, lambda_init=lambda_init,
            norm_eps=norm_eps)
        s = B.pa_diff_validate(self.params)
        if s != B.PA_OK:
            raise B.PaError(s, B.last_error())
        # as in PagedLatentAttention: the first read call after the write phase
        self.params_after_write = B.pa_diff_params.from_buffer_copy(self.params)
        self.params_after_write.flags |= B.PA_FLAG_AFTER_WRITE | (
            B.PA_FLAG_OWN_SLOTS if own_slots else 0)
        self.device = torch.empty(0, device=device).device
        self._index = self.device.index
        self.max_seqs, self.max_tokens = max_seqs, max_tokens
        with _device(self._index):
            n = B.pa_diff_workspace_size(self.params, max_seqs, max_tokens)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device) if n else None
        self.err_flags = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._filled = _Filled(self._index)

    def _begin(self, stream):
        filled = self._filled
        if filled is not None:  # (not taken by another thread meanwhile)
            filled.before(stream)
            self._filled = None

    # -- argument checks: types, devices and sizes the C side cannot see
    def _tensors(self, dtype, names, *tensors):
        index = self._index
        for t in tensors:
            if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
                name = names.split()[[x is t for x in tensors].index(True)]
                _require(False, f"{name} must be a contiguous {dtype} tensor on {self.device}")

    def _check_caches(self, key_cache, value_cache, cos_cache, sin_cache, cumseq, past):
        p, hs, vhs = self.params, self.head_size, self.v_head_size
        if p.rotary_dim:
            self._tensors(self.dtype, "key_cache value_cache cos_cache sin_cache", key_cache,
                          value_cache, cos_cache, sin_cache)
            half = p.rotary_dim // 2
            n = p.cos_rows * half
            _require(cos_cache.size(-1) == sin_cache.size(-1) == half
                     and cos_cache.numel() >= n and sin_cache.numel() >= n,
                     "cos_cache and sin_cache must be [cos_rows, rotary_dim / 2]")
        else:
            self._tensors(self.dtype, "key_cache value_cache", key_cache, value_cache)
        self._tensors(torch.int32, "cumseq past", cumseq, past)
        rows = p.num_blocks * p.block_size * p.kv_num_heads
        _require(key_cache.numel() == rows * 2 * hs and value_cache.numel() == rows * vhs,
                 "key_cache must be [num_blocks, bs, kvH, 2, hs], value_cache [num_blocks, bs, "
                 "kvH, vhs]")
        _require(cumseq.numel() == past.numel() + 1, "cumseq must be [num_seqs + 1]")

    def _check_write(self, key, value, slot_mapping):
        self._tensors(self.dtype, "key value", key, value)
        self._tensors(torch.int32, "slot_mapping", slot_mapping)
        n = key.size(0)
        _require(key.numel() == n * self.kv_num_heads * 2 * self.head_size
                 and value.size(0) == n and value.numel() == n * self.kv_num_heads * self.v_head_size
                 and slot_mapping.numel() == n,
                 "key must be [T, kvH*2*hs], value [T, kvH*vhs], slot_mapping [T]")

    def _check_read(self, query, lambda_vectors, norm_weight, past, block_table, out):
        self._tensors(self.dtype, "query norm_weight out", query, norm_weight, out)
        self._tensors(torch.int32, "block_table", block_table)
        self._tensors(torch.float32, "lambda_vectors", lambda_vectors)
        n = query.size(0)
        _require(query.numel() == n * self.num_heads * 2 * self.head_size
                 and out.size(0) == n and out.numel() == n * self.num_heads * self.v_head_size
                 and norm_weight.numel() == self.v_head_size
                 and lambda_vectors.numel() == 4 * self.head_size
                 and block_table.numel() == past.numel() * self.params.max_blocks_per_seq,
                 "query must be [T, H*2*hs], out [T, H*vhs], norm_weight [vhs], lambda_vectors "
                 "[4, hs], block_table [num_seqs, max_blocks_per_seq]")

    def _on_device(self):
        return _device(self._index)

    def write(self, key, value, key_cache, value_cache, cos_cache, sin_cache, slot_mapping,
              cumseq, past, stream=None):
        """Rotates the new keys and stores keys and values in their slots."""
        self._check_caches(key_cache, value_cache, cos_cache, sin_cache, cumseq, past)
        self._check_write(key, value, slot_mapping)
        with self._on_device():
            if self._filled is not None:
                self._begin(stream)
            B.pa_diff_write(self.params, key, value, cos_cache, sin_cache, slot_mapping, cumseq,
                            past, key_cache, value_cache, self.err_flags, stream)

    def _read(self, fn, args, seq_begin, seq_end, stream, after_write):
        fn(self.params_after_write if after_write else self.params, *args, seq_begin, seq_end,
           self.workspace, self.err_flags, stream)

    def _read_checked(self, fn, args, *rest):
        (query, key_cache, value_cache, cos_cache, sin_cache, lambda_vectors, norm_weight, cumseq,
         past, block_table, out) = args
        self._check_caches(key_cache, value_cache, cos_cache, sin_cache, cumseq, past)
        self._check_read(query, lambda_vectors, norm_weight, past, block_table, out)
        with self._on_device():
            if self._filled is not None:
                self._begin(rest[2])
            self._read(fn, args, *rest)

    def decode(self, query, key_cache, value_cache, cos_cache, sin_cache, lambda_vectors,
               norm_weight, cumseq, past, block_table, out, seq_begin=0, seq_end=None,
               stream=None, after_write: bool = False):
        """Sequences [seq_begin, seq_end) with one new token each.
        ``after_write``: this call directly follows ``write`` on the same
        stream (see PA_FLAG_AFTER_WRITE)."""
        self._read_checked(B.pa_diff_decode,
                           (query, key_cache, value_cache, cos_cache, sin_cache, lambda_vectors,
                            norm_weight, cumseq, past, block_table, out),
                           seq_begin, seq_end, stream, after_write)

    def prefill(self, query, key_cache, value_cache, cos_cache, sin_cache, lambda_vectors,
                norm_weight, cumseq, past, block_table, out, seq_begin=0, seq_end=None,
                stream=None, after_write: bool = False):
        """Sequences [seq_begin, seq_end) with any number of new tokens."""
        self._read_checked(B.pa_diff_prefill,
                           (query, key_cache, value_cache, cos_cache, sin_cache, lambda_vectors,
                            norm_weight, cumseq, past, block_table, out),
                           seq_begin, seq_end, stream, after_write)

    def forward(self, query, key, value, key_cache, value_cache, cos_cache, sin_cache,
                lambda_vectors, norm_weight, cumseq, past, block_table, slot_mapping,
                num_decode_seqs: int, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """Write phase over all tokens, then decode over sequences [0,
        num_decode_seqs) and prefill over the rest; returns ``out``."""
        nseq = past.size(0)
        _require(0 <= num_decode_seqs <= nseq, "num_decode_seqs must be in 0..num_seqs")
        with self._on_device():
            self._check_caches(key_cache, value_cache, cos_cache, sin_cache, cumseq, past)
            self._check_write(key, value, slot_mapping)
            _require(key.size(0) == query.size(0), "query and key must have a row per token")
            if out is None:
                shape = (query.size(0), self.num_heads * self.v_head_size)
                with _allocating(stream, self._index):
                    out = torch.empty(shape, dtype=self.dtype, device=self.device)
            stream = B.raw_stream(stream)
            self._check_read(query, lambda_vectors, norm_weight, past, block_table, out)
            if self._filled is not None:
                self._begin(stream)
            B.pa_diff_write(self.params, key, value, cos_cache, sin_cache, slot_mapping, cumseq,
                            past, key_cache, value_cache, self.err_flags, stream)
            args = (query, key_cache, value_cache, cos_cache, sin_cache, lambda_vectors,
                    norm_weight, cumseq, past, block_table, out)
            if num_decode_seqs > 0:
                self._read(B.pa_diff_decode, args, 0, num_decode_seqs, stream, True)
            if num_decode_seqs < nseq:
                self._read(B.pa_diff_prefill, args, num_decode_seqs, nseq, stream,
                           num_decode_seqs == 0)
        return out

    def error_flags(self) -> int:
        """Reads the device error word (synchronises with the device)."""
        return int(self.err_flags.item())

    def reset_error_flags(self):
        self.err_flags.zero_()


class PagePool:
    """Pages of a set of paged caches, kept on the device: which sequence
    holds which (``block_table``), how often each is held (``refcount``) and
    how many tokens each sequence has cached (``past``).

    ``caches``: the paged tensors that share the page ids, ``[num_blocks,
    block_size, ...]`` and contiguous in a page (the layers' ``key_cache`` /
    ``value_cache`` of the attention objects above). ``block_table`` [B, mb],
    ``past`` [B] and ``refcount`` [num_blocks] are int32 tensors: pass those in
    use, or leave them out for an empty pool of ``max_seqs`` sequences of up to
    ``max_blocks_per_seq`` pages. The three go to ``forward`` as they are.

    Every method only enqueues kernels on ``stream`` (the current stream of
    the pool's device by default) and can be captured in a CUDA graph after
    one eager call; calls on one pool have to be ordered by the caller. (The
    first call waits for the constructor's own fills; work on other streams
    that reads ``block_table``, ``past`` or ``refcount`` before it has to be
    ordered too.) See include/pa_pages.h for what each does with arguments
    that make no sense; ``error_flags`` reads what the device reported."""

    def __init__(self, caches, *, block_size: int, block_table: Optional[torch.Tensor] = None,
                 past: Optional[torch.Tensor] = None, refcount: Optional[torch.Tensor] = None,
                 max_seqs: Optional[int] = None, max_blocks_per_seq: Optional[int] = None):
        self.caches = list(caches)
        _require(len(self.caches) > 0, "a pool needs at least one cache")
        first = self.caches[0]
        _require(first.dim() >= 2 and first.shape[0] > 0, "caches need at least one page")
        self.device, self.num_blocks = first.device, int(first.shape[0])
        self._index = self.device.index
        _require(self.device.type == "cuda", "caches must be CUDA tensors")
        for c in self.caches:
            _require(c.device == self.device and c.dim() >= 2 and int(c.shape[0]) == self.num_blocks
                     and int(c.shape[1]) == block_size,
                     "every cache must be [num_blocks, block_size, ...] on one device")
            _require(c[0].numel() > 0, "cache rows must not be empty")
            _require(c[0].is_contiguous() and (self.num_blocks == 1 or c.stride(0) == c[0].numel()),
                     "caches must be contiguous")
            _require(c.data_ptr() % 16 == 0 and c[0, 0].numel() * c.element_size() % 16 == 0,
                     "cache rows must be multiples of 16 bytes, 16-byte aligned")
        if block_table is None:
            _require(max_seqs is not None and max_blocks_per_seq is not None,
                     "without a block_table, max_seqs and max_blocks_per_seq are needed")
            block_table = torch.full((max_seqs, max_blocks_per_seq), -1, dtype=torch.int32,
                                     device=self.device)
        _require(block_table.dim() == 2, "block_table must be [num_seqs, max_blocks_per_seq]")
        if past is None:
            past = torch.zeros(block_table.shape[0], dtype=torch.int32, device=self.device)
        if refcount is None:
            refcount = torch.zeros(self.num_blocks, dtype=torch.int32, device=self.device)
        self._ints("block_table past refcount", block_table, past, refcount)
        _require(past.numel() == block_table.shape[0], "past must be [num_seqs]")
        _require(refcount.numel() == self.num_blocks, "refcount must be [num_blocks]")
        self.block_table, self.past, self.refcount = block_table, past, refcount
        self.params = B.make_pages_params(num_blocks=self.num_blocks, block_size=block_size,
                                          max_blocks_per_seq=block_table.shape[1],
                                          num_seqs=block_table.shape[0])
        s = B.pa_pages_validate(self.params)
        if s != B.PA_OK:
            raise B.PaError(s, B.last_error())
        self._list = B.make_page_caches(self.caches)
        self.workspace = torch.empty(B.pa_pages_workspace_size(self.params), dtype=torch.uint8,
                                     device=self.device)
        self.err_flags = torch.zeros(1, dtype=torch.int32, device=self.device)
        #: pages held after the last ``compact`` (int32 [1] on the device)
        self.live = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._filled = _Filled(self._index)

    def _begin(self, stream):
        filled = self._filled
        if filled is not None:  # (not taken by another thread meanwhile)
            filled.before(stream)
            self._filled = None

    def _ints(self, names, *tensors):
        index = self._index
        for t in tensors:
            if t.dtype is not torch.int32 or t.get_device() != index or not t.is_contiguous():
                name = names.split()[[x is t for x in tensors].index(True)]
                _require(False, f"{name} must be a contiguous int32 tensor on {self.device}")

    def copy(self, src, dst, rows=None, stream=None):
        """Pages ``src[i]`` -> ``dst[i]`` (their first ``rows[i]`` rows) in every cache."""
        if rows is None:
            self._ints("src dst", src, dst)
        else:
            self._ints("src dst rows", src, dst, rows)
        _require(dst.numel() == src.numel() and (rows is None or rows.numel() == src.numel()),
                 "src, dst and rows must have one entry per pair")
        with _device(self._index):
            if self._filled is not None:
                self._begin(stream)
            B.pa_pages_copy(self.params, self._list, len(self.caches), src, dst, rows,
                            self.workspace, self.err_flags, stream)

    def fork(self, parents, children, stream=None):
        """Sequence ``children[i]`` becomes a copy of ``parents[i]``: full pages
        shared, the rows of the last one copied into a page of its own. A
        child's row has to be empty: beams that go on from one another fork
        into a second set of rows, and the first is freed behind that."""
        self._ints("parents children", parents, children)
        _require(parents.numel() == children.numel(), "parents and children must pair up")
        with _device(self._index):
            if self._filled is not None:
                self._begin(stream)
            B.pa_pages_fork(self.params, self._list, len(self.caches), parents, children,
                            self.block_table, self.past, self.refcount, self.workspace,
                            self.err_flags, stream)

    def free(self, seqs, stream=None):
        """Takes the pages of ``seqs`` back (their rows become -1, their past 0)."""
        self._ints("seqs", seqs)
        with _device(self._index):
            if self._filled is not None:
                self._begin(stream)
            B.pa_pages_free(self.params, seqs, self.block_table, self.past, self.refcount,
                            self.err_flags, stream)

    def reserve(self, cumseq, slot_mapping, stream=None) -> torch.Tensor:
        """Pages for the ``cumseq[b+1] - cumseq[b]`` next tokens of every
        sequence; fills ``slot_mapping`` [T] for the write phase and returns
        it. ``past`` stays (add the new tokens once they are written)."""
        self._ints("cumseq slot_mapping", cumseq, slot_mapping)
        _require(cumseq.numel() == self.past.numel() + 1, "cumseq must be [num_seqs + 1]")
        with _device(self._index):
            if self._filled is not None:
                self._begin(stream)
            B.pa_pages_reserve(self.params, cumseq, self.block_table, self.past, self.refcount,
                               slot_mapping, self.workspace, self.err_flags, stream)
        return slot_mapping

    def compact(self, stream=None) -> torch.Tensor:
        """Moves the held pages to the lowest ids; returns ``live`` (their
        number, on the device)."""
        with _device(self._index):
            if self._filled is not None:
                self._begin(stream)
            B.pa_pages_compact(self.params, self._list, len(self.caches), self.block_table,
                               self.refcount, self.live, self.workspace, self.err_flags, stream)
        return self.live

    def error_flags(self) -> int:
        """Reads the device error word (synchronises with the device)."""
        return int(self.err_flags.item())

    def reset_error_flags(self):
        self.err_flags.zero_()
