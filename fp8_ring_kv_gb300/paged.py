"""A paged FP8 KV cache for many sequences (include/kvring_paged.h).

``PagedKV`` owns one cache in a torch-allocated device workspace; ``append``
and ``attend`` check their tensors, enqueue the library's kernels on the
current (or given) stream and return at once.  Argument checks only: every
step of the path runs in the CUDA kernels of ``libkvring.so``.
"""
import ctypes

import torch

from . import kvring as _k
from .kvring import KVRingError, check, kvring_paged_config

_I32 = torch.int32
_get_device, _get_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_IN = {torch.bfloat16: _k.KVRING_IN_BF16, torch.float16: _k.KVRING_IN_F16}


def make_paged_config(kv_heads, q_heads, head_dim, n_pages, page_tokens, axis_dims, pos_min, pos_count,
                      rope_base=10000.0, dtype=torch.bfloat16, layers=1) -> kvring_paged_config:
    if dtype not in _IN:
        raise KVRingError(f"dtype: {dtype}; the kernels read bfloat16 or float16")
    if not 1 <= len(axis_dims) <= 3 or len(pos_min) != len(axis_dims) or len(pos_count) != len(axis_dims):
        raise KVRingError("axis_dims, pos_min and pos_count: one entry for each of 1 to 3 axes")
    c = kvring_paged_config()
    c.layers, c.kv_heads, c.q_heads, c.head_dim = int(layers), int(kv_heads), int(q_heads), int(head_dim)
    c.page_tokens, c.n_pages, c.in_dtype, c.n_axes = int(page_tokens), int(n_pages), _IN[dtype], len(axis_dims)
    for a in range(len(axis_dims)):
        c.axis_dims[a], c.pos_min[a], c.pos_count[a] = int(axis_dims[a]), int(pos_min[a]), int(pos_count[a])
    c.rope_base = float(rope_base)
    return c


def kvring_paged_workspace_bytes(cfg: kvring_paged_config) -> int:
    return int(_k.load().kvring_paged_workspace_bytes(ctypes.byref(cfg)))


def _as_stream(stream, device):
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(getattr(stream, "cuda_stream", stream))
    # torch takes 0, the default stream's handle, for a request for a new stream
    return torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)


def _bad_ints(t, shape, index, what):
    """Why an int32 tensor is not as the kernels read it (None in ``shape``: any size)."""
    if t.dtype is not torch.int32:
        return f"{what}: {t.dtype}; the kernels read torch.int32"
    if t.get_device() != index:
        return f"{what}: on {t.device}, the cache is on cuda:{index}"
    if not t.is_contiguous():
        return f"{what}: not contiguous"
    return f"{what}: shape {tuple(t.shape)}; [{', '.join('*' if w is None else str(w) for w in shape)}] is read"


def _bad_heads(t, n, heads, dim, dtype, index, what):
    """Why a tensor is not [n, heads, dim] with a token's heads side by side."""
    if t.dtype is not dtype:
        return f"{what}: {t.dtype}; the cache was made for {dtype}"
    if tuple(t.shape) != (n, heads, dim):
        return f"{what}: shape {tuple(t.shape)}; [{n}, {heads}, {dim}] is read"
    if t.get_device() != index:
        return f"{what}: on {t.device}, the cache is on cuda:{index}"
    return f"{what}: strides {t.stride()}; heads side by side and tokens a multiple of 8 elements apart"


class PagedKV:
    """One paged cache: ``layers`` pools of ``n_pages`` pages of
    ``page_tokens`` tokens.

    ``k_codes``, ``v_codes`` (uint8 [layers, n_pages, kv_heads, page_tokens,
    head_dim], e4m3) and ``k_scales``, ``v_scales`` (fp32 [layers, n_pages,
    kv_heads]) are views of the workspace; a cached value is code * scale.
    For inference: nothing here has a gradient.

    A workspace of its own is allocated on ``stream``.  Whoever uses the cache
    on other streams keeps it until their work is done, as with any tensor."""

    def __init__(self, kv_heads, q_heads, head_dim, n_pages, page_tokens, axis_dims, pos_min, pos_count,
                 rope_base=10000.0, dtype=torch.bfloat16, layers=1, device="cuda", stream=None, workspace=None):
        self.handle = None
        self.cfg = make_paged_config(kv_heads, q_heads, head_dim, n_pages, page_tokens, axis_dims, pos_min, pos_count,
                                     rope_base, dtype, layers)
        nbytes = kvring_paged_workspace_bytes(self.cfg)
        if nbytes == 0:
            raise KVRingError("invalid kvring_paged configuration")
        self.layers, self.kv_heads, self.q_heads, self.head_dim = int(layers), int(kv_heads), int(q_heads), int(head_dim)
        self.n_pages, self.page_tokens, self.n_axes, self.dtype = int(n_pages), int(page_tokens), len(axis_dims), dtype
        if workspace is None:
            if stream is None:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
            else:
                # memory that no other stream's queued work still uses
                with torch.cuda.stream(_as_stream(stream, device)):
                    workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        elif workspace.dtype != torch.uint8 or workspace.numel() < nbytes or workspace.data_ptr() % 256 \
                or not workspace.is_contiguous() or not workspace.is_cuda:
            raise KVRingError("workspace: a uint8 CUDA tensor of kvring_paged_workspace_bytes, 256-byte aligned")
        self.workspace = workspace
        self.device = workspace.device
        self._index = workspace.get_device()
        lib = _k.load()
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            check(lib.kvring_paged_create(ctypes.byref(self.cfg), workspace.data_ptr(), workspace.numel(),
                                          self._stream(stream), ctypes.byref(h)), "kvring_paged_create")
        self.handle = h
        self._append, self._attend = lib.kvring_paged_append, lib.kvring_paged_attend
        ptrs = [ctypes.c_void_p() for _ in range(5)]
        check(lib.kvring_paged_layout(h, *[ctypes.byref(p) for p in ptrs]), "kvring_paged_layout")
        kc, vc, ks, vs, _ = [p.value - workspace.data_ptr() for p in ptrs]
        L, N, H, P, D = self.layers, self.n_pages, self.kv_heads, self.page_tokens, self.head_dim
        codes = L * N * H * P * D
        self.k_codes = workspace[kc:kc + codes].view(L, N, H, P, D)
        self.v_codes = workspace[vc:vc + codes].view(L, N, H, P, D)
        self.k_scales = workspace[ks:ks + L * N * H * 4].view(torch.float32).view(L, N, H)
        self.v_scales = workspace[vs:vs + L * N * H * 4].view(torch.float32).view(L, N, H)

    def _stream(self, stream):
        if stream is None:
            return _get_stream(self._index)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    # The checks run before every call, beside kernels of a few microseconds:
    # the good case first, the reason only for a bad one.
    def _row_stride(self, t, n, heads, what):
        """Elements between the tokens of [n, heads, head_dim] (q, k and v may be
        slices of one tensor)."""
        dim = self.head_dim
        if t.dtype is self.dtype and t.shape == (n, heads, dim) and t.get_device() == self._index:
            row, head, one = t.stride()
            if n <= 1:
                row = heads * dim              # the only token's stride is not used
            if not n or one == 1 and (head == dim or heads == 1) and row >= heads * dim and row % 8 == 0:
                return row
        raise KVRingError(_bad_heads(t, n, heads, dim, self.dtype, self._index, what))

    def _ints(self, t, shape, what):
        if t.dtype is _I32 and t.shape == shape and t.is_contiguous() and t.get_device() == self._index:
            return t.data_ptr()
        raise KVRingError(_bad_ints(t, shape, self._index, what))

    def _batch(self, layer, n, pos, pos_name, seq_start, kv_len, page_table):
        """The batch's arguments in the library's order."""
        if self.handle is None:
            raise KVRingError("the cache is closed")
        if not 0 <= layer < self.layers:
            raise KVRingError(f"layer: {layer} of {self.layers}")
        shape = page_table.shape
        if len(shape) != 2 or shape[1] < 1:
            raise KVRingError(f"page_table: shape {tuple(shape)}; [sequences, at least 1] is read")
        n_seqs, width = shape
        if n_seqs > _k.KVRING_PAGED_MAX_SEQS:
            raise KVRingError(f"page_table: {n_seqs} sequences; a call takes at most {_k.KVRING_PAGED_MAX_SEQS}")
        if width * self.page_tokens > _k.KVRING_PAGED_MAX_LEN:
            raise KVRingError(f"page_table: {width} pages a row, more than {_k.KVRING_PAGED_MAX_LEN} tokens")
        if page_table.dtype is not _I32 or page_table.get_device() != self._index:
            raise KVRingError(f"page_table: {page_table.dtype} on {page_table.device}; torch.int32 on cuda:{self._index} is read")
        row, one = page_table.stride()
        if (width > 1 and one != 1) or (n_seqs > 1 and row < width):
            raise KVRingError(f"page_table: strides {(row, one)}; a row's entries side by side")
        return (self._ints(pos, (n, self.n_axes), pos_name), self._ints(seq_start, (n_seqs + 1,), "seq_start"),
                self._ints(kv_len, (n_seqs,), "kv_len"), n_seqs, page_table.data_ptr(), max(row, width), width)

    def _call(self, fn, *args):
        """The library's function with the cache's device current."""
        if _get_device() == self._index:
            status = fn(self.handle, *args)
        else:
            with torch.cuda.device(self.device):
                status = fn(self.handle, *args)
        if status:
            check(status, fn.__name__)

    def append(self, k, v, pos, seq_start, kv_len, page_table, layer=0, stream=None):
        """Write the new tokens' keys (rotated at ``pos``) and values.

        k, v: [N, kv_heads, head_dim] in the cache's dtype, tokens any multiple
        of 8 elements apart.  pos: int32 [N, n_axes].  Sequence b's new tokens
        are rows seq_start[b] .. seq_start[b+1]-1; kv_len[b] counts its tokens
        with them; page_table[b] lists its pages in order."""
        n = k.shape[0]
        ks, vs = self._row_stride(k, n, self.kv_heads, "k"), self._row_stride(v, n, self.kv_heads, "v")
        p, start, length, n_seqs, table, ts, width = self._batch(layer, n, pos, "pos", seq_start, kv_len, page_table)
        if n and n_seqs:
            self._call(self._append, layer, k.data_ptr(), ks, v.data_ptr(), vs, p, start, length, n_seqs, n,
                       table, ts, width, self._stream(stream))

    def attend(self, q, q_pos, seq_start, kv_len, page_table, out=None, layer=0, causal=True, window=None, scale=None,
               max_new=None, stream=None):
        """softmax(scale q.k) v of every new token's queries over its sequence's
        cache; [N, q_heads, head_dim].

        window: with causal, the number of cached tokens a query sees at most,
        its own included.  scale: 1 / sqrt(head_dim) unless given.  max_new: the
        most new tokens that a sequence of this call has, where the caller
        knows it (a sequence with more is left out and flagged)."""
        n = q.shape[0]
        qs = self._row_stride(q, n, self.q_heads, "q")
        p, start, length, n_seqs, table, ts, width = self._batch(layer, n, q_pos, "q_pos", seq_start, kv_len, page_table)
        if window is not None and (not causal or window < 1):
            raise KVRingError("window: a positive number of tokens, with causal")
        if scale is not None and not 2.0 ** -100 <= scale <= 2.0 ** 100:
            raise KVRingError(f"scale: {scale}; 2^-100 .. 2^100")
        if max_new is not None and not 1 <= max_new <= max(n, 1):
            raise KVRingError(f"max_new: {max_new}; 1 .. {n}")
        if out is None:
            if stream is None:
                out = torch.empty_like(q, memory_format=torch.contiguous_format)
            else:
                # memory that the allocator knows to be in use on that stream
                with torch.cuda.stream(_as_stream(stream, self.device)):
                    out = torch.empty_like(q, memory_format=torch.contiguous_format)
            os_ = self.q_heads * self.head_dim
        else:
            os_ = self._row_stride(out, n, self.q_heads, "out")
        if n and n_seqs:
            self._call(self._attend, layer, q.data_ptr(), qs, p, start, length, n_seqs, n,
                       n if max_new is None else max_new, table, ts, width, 1 if causal else 0, min(window or 0, _k.KVRING_PAGED_MAX_LEN),
                       scale or 0.0, out.data_ptr(), os_, self._stream(stream))
        return out

    def debug_state(self, stream=None):
        """The device error bits (KVRING_DEVERR_*); waits for the stream."""
        err = ctypes.c_int32()
        with torch.cuda.device(self.device):
            check(_k.load().kvring_paged_debug_state(self.handle, self._stream(stream), ctypes.byref(err)),
                  "kvring_paged_debug_state")
        return int(err.value)

    def close(self):
        if self.handle is not None:
            _k.load().kvring_paged_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
