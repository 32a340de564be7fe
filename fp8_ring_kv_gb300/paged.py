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


def _check_ints(t, shape, device, what):
    """int32, contiguous, on the cache's device, of that shape (None: any size)."""
    if t.dtype is not torch.int32:
        raise KVRingError(f"{what}: {t.dtype}; the kernels read torch.int32")
    got = t.shape
    if len(got) != len(shape) or any(w is not None and w != g for w, g in zip(shape, got)):
        raise KVRingError(f"{what}: shape {tuple(got)}; [{', '.join('*' if w is None else str(w) for w in shape)}] is read")
    if not t.is_contiguous():
        raise KVRingError(f"{what}: not contiguous")
    if t.device != device:
        raise KVRingError(f"{what}: on {t.device}, the cache is on {device}")


def _check_heads(t, n, heads, dim, dtype, device, what):
    """[n, heads, dim] with a token's heads side by side and a token stride
    that is a multiple of 8 elements (q, k, v may be slices of one tensor);
    returns the stride."""
    if t.dtype is not dtype:
        raise KVRingError(f"{what}: {t.dtype}; the cache was made for {dtype}")
    if tuple(t.shape) != (n, heads, dim):
        raise KVRingError(f"{what}: shape {tuple(t.shape)}; [{n}, {heads}, {dim}] is read")
    if t.device != device:
        raise KVRingError(f"{what}: on {t.device}, the cache is on {device}")
    st = t.stride()
    row = st[0] if n > 1 else heads * dim      # the only token's stride is not used
    if n and (st[2] != 1 or (heads > 1 and st[1] != dim) or row < heads * dim or row % 8):
        raise KVRingError(f"{what}: strides {st}; heads side by side and tokens a multiple of 8 elements apart")
    return row


class PagedKV:
    """One paged cache: ``layers`` pools of ``n_pages`` pages of
    ``page_tokens`` tokens.

    ``k_codes``, ``v_codes`` (uint8 [layers, n_pages, kv_heads, page_tokens,
    head_dim], e4m3) and ``k_scales``, ``v_scales`` (fp32 [layers, n_pages,
    kv_heads]) are views of the workspace; a cached value is code * scale."""

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
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        elif workspace.dtype != torch.uint8 or workspace.numel() < nbytes or workspace.data_ptr() % 256 \
                or not workspace.is_contiguous() or not workspace.is_cuda:
            raise KVRingError("workspace: a uint8 CUDA tensor of kvring_paged_workspace_bytes, 256-byte aligned")
        self.workspace = workspace
        self.device = workspace.device
        lib = _k.load()
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            check(lib.kvring_paged_create(ctypes.byref(self.cfg), workspace.data_ptr(), workspace.numel(),
                                          self._stream(stream), ctypes.byref(h)), "kvring_paged_create")
        self.handle = h
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
            stream = torch.cuda.current_stream(self.device)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def _check_batch(self, layer, n, pos, seq_start, kv_len, page_table):
        dev = self.device
        if self.handle is None:
            raise KVRingError("the cache is closed")
        if not 0 <= layer < self.layers:
            raise KVRingError(f"layer: {layer} of {self.layers}")
        n_seqs = kv_len.shape[0] if kv_len.dim() == 1 else -1
        if n_seqs > _k.KVRING_PAGED_MAX_SEQS:
            raise KVRingError(f"kv_len: {n_seqs} sequences; a call takes at most {_k.KVRING_PAGED_MAX_SEQS}")
        _check_ints(kv_len, (None,), dev, "kv_len")
        _check_ints(seq_start, (n_seqs + 1,), dev, "seq_start")
        _check_ints(pos, (n, self.n_axes), dev, "pos")
        if page_table.dim() != 2 or page_table.shape[0] != n_seqs or page_table.shape[1] < 1:
            raise KVRingError(f"page_table: shape {tuple(page_table.shape)}; [{n_seqs}, at least 1] is read")
        if page_table.dtype is not torch.int32 or page_table.device != dev:
            raise KVRingError(f"page_table: {page_table.dtype} on {page_table.device}; torch.int32 on {dev} is read")
        width = page_table.shape[1]
        st = page_table.stride()
        if (width > 1 and st[1] != 1) or (n_seqs > 1 and st[0] < width):
            raise KVRingError(f"page_table: strides {st}; a row's entries side by side")
        if width * self.page_tokens > _k.KVRING_PAGED_MAX_LEN:
            raise KVRingError(f"page_table: {width} pages a row, more than {_k.KVRING_PAGED_MAX_LEN} tokens")
        return n_seqs, max(st[0], width), width

    def append(self, k, v, pos, seq_start, kv_len, page_table, layer=0, stream=None):
        """Write the new tokens' keys (rotated at ``pos``) and values.

        k, v: [N, kv_heads, head_dim] in the cache's dtype, tokens any multiple
        of 8 elements apart.  pos: int32 [N, n_axes].  Sequence b's new tokens
        are rows seq_start[b] .. seq_start[b+1]-1; kv_len[b] counts its tokens
        with them; page_table[b] lists its pages in order."""
        n = k.shape[0]
        ks = _check_heads(k, n, self.kv_heads, self.head_dim, self.dtype, self.device, "k")
        vs = _check_heads(v, n, self.kv_heads, self.head_dim, self.dtype, self.device, "v")
        n_seqs, ts, width = self._check_batch(layer, n, pos, seq_start, kv_len, page_table)
        if n == 0 or n_seqs == 0:
            return
        with torch.cuda.device(self.device):
            check(_k.load().kvring_paged_append(
                self.handle, layer, k.data_ptr(), ks, v.data_ptr(), vs, pos.data_ptr(), seq_start.data_ptr(),
                kv_len.data_ptr(), n_seqs, n, page_table.data_ptr(), ts, width, self._stream(stream)),
                "kvring_paged_append")

    def attend(self, q, q_pos, seq_start, kv_len, page_table, out=None, layer=0, causal=True, window=None, scale=None,
               max_new=None, stream=None):
        """softmax(scale q.k) v of every new token's queries over its sequence's
        cache; [N, q_heads, head_dim].

        window: with causal, the number of cached tokens a query sees at most,
        its own included.  scale: 1 / sqrt(head_dim) unless given.  max_new: the
        most new tokens that a sequence of this call has, where the caller
        knows it (a sequence with more is left out and flagged)."""
        n = q.shape[0]
        qs = _check_heads(q, n, self.q_heads, self.head_dim, self.dtype, self.device, "q")
        n_seqs, ts, width = self._check_batch(layer, n, q_pos, seq_start, kv_len, page_table)
        if window is not None and (not causal or window < 1):
            raise KVRingError("window: a positive number of tokens, with causal")
        if scale is not None and not 0.0 < scale < float("inf"):
            raise KVRingError("scale: positive and finite")
        if max_new is not None and not 1 <= max_new <= max(n, 1):
            raise KVRingError(f"max_new: {max_new}; 1 .. {n}")
        if out is None:
            if stream is None:
                out = torch.empty((n, self.q_heads, self.head_dim), dtype=self.dtype, device=self.device)
            else:
                # memory that the allocator knows to be in use on that stream
                s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), self.device)
                with torch.cuda.stream(s):
                    out = torch.empty((n, self.q_heads, self.head_dim), dtype=self.dtype, device=self.device)
        os_ = _check_heads(out, n, self.q_heads, self.head_dim, self.dtype, self.device, "out")
        if n == 0 or n_seqs == 0:
            return out
        with torch.cuda.device(self.device):
            check(_k.load().kvring_paged_attend(
                self.handle, layer, q.data_ptr(), qs, q_pos.data_ptr(), seq_start.data_ptr(), kv_len.data_ptr(),
                n_seqs, n, n if max_new is None else max_new, page_table.data_ptr(), ts, width, 1 if causal else 0,
                window or 0, scale or 0.0, out.data_ptr(), os_, self._stream(stream)), "kvring_paged_attend")
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
