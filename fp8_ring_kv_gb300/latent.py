"""A paged FP8 cache for latent attention (include/kvring_latent.h).

``LatentKV`` keeps one row per token: a latent vector that every head uses as
key and value, and a rotated key part of 64 numbers that they share.  ``append``
writes rows, ``read`` gives them back, ``attend`` is attention over the cache
with the queries in the latent space (absorbed form), ``attend_expanded``
attention with the keys and values of every head that the caller made from the
rows.  Argument checks only: every step runs in the CUDA kernels of
``libkvring.so``.
"""
import ctypes

import torch

from . import kvring as _k
from .kvring import KVRingError, check, kvring_latent_config
from .paged import _I32, _IN, _as_stream, _bad_ints, _get_device, _get_stream

ROPE, HEAD = _k.KVRING_LATENT_ROPE, _k.KVRING_LATENT_HEAD


def make_latent_config(q_heads, latent_dim, n_pages, page_tokens, axis_dims, pos_min, pos_count, rope_base=10000.0,
                       dtype=torch.bfloat16, layers=1) -> kvring_latent_config:
    if dtype not in _IN:
        raise KVRingError(f"dtype: {dtype}; the kernels read bfloat16 or float16")
    if not 1 <= len(axis_dims) <= 3 or len(pos_min) != len(axis_dims) or len(pos_count) != len(axis_dims):
        raise KVRingError("axis_dims, pos_min and pos_count: one entry for each of 1 to 3 axes")
    c = kvring_latent_config()
    c.layers, c.q_heads, c.latent_dim = int(layers), int(q_heads), int(latent_dim)
    c.page_tokens, c.n_pages, c.in_dtype, c.n_axes = int(page_tokens), int(n_pages), _IN[dtype], len(axis_dims)
    for a in range(len(axis_dims)):
        c.axis_dims[a], c.pos_min[a], c.pos_count[a] = int(axis_dims[a]), int(pos_min[a]), int(pos_count[a])
    c.rope_base = float(rope_base)
    return c


def kvring_latent_workspace_bytes(cfg: kvring_latent_config) -> int:
    return int(_k.load().kvring_latent_workspace_bytes(ctypes.byref(cfg)))


def _apart(token, head, n, heads, width):
    """Whether rows [n, heads, width] with these strides are as the kernels take them."""
    if token % 8 or head % 8 or token < 0 or head < 0:
        return False
    if n <= 1:
        return heads <= 1 or head >= width
    if heads <= 1:
        return token >= width
    return (head >= width and token >= (heads - 1) * head + width) or (token >= width and head >= (n - 1) * token + width)


class LatentKV:
    """One latent cache: ``layers`` pools of ``n_pages`` pages of
    ``page_tokens`` tokens.

    ``codes`` (uint8 [layers, n_pages, page_tokens, latent_dim + 64], e4m3) and
    ``scales`` (fp32 [layers, n_pages, page_tokens]) are views of the workspace;
    a cached value is code * scale.  For inference: nothing here has a gradient.

    A workspace of its own is allocated on ``stream``.  Whoever uses the cache
    on other streams keeps it until their work is done, as with any tensor.
    The attention's scratch belongs to the cache: two attention calls on one
    cache must not run at the same time."""

    def __init__(self, q_heads, latent_dim, n_pages, page_tokens, axis_dims, pos_min, pos_count, rope_base=10000.0,
                 dtype=torch.bfloat16, layers=1, device="cuda", stream=None, workspace=None):
        self.handle = None
        self.cfg = make_latent_config(q_heads, latent_dim, n_pages, page_tokens, axis_dims, pos_min, pos_count, rope_base,
                                      dtype, layers)
        nbytes = kvring_latent_workspace_bytes(self.cfg)
        if nbytes == 0:
            raise KVRingError("invalid kvring_latent configuration")
        self.layers, self.q_heads, self.latent_dim, self.width = int(layers), int(q_heads), int(latent_dim), int(latent_dim) + ROPE
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
            raise KVRingError("workspace: a uint8 CUDA tensor of kvring_latent_workspace_bytes, 256-byte aligned")
        self.workspace = workspace
        self.device = workspace.device
        self._index = workspace.get_device()
        lib = _k.load()
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            check(lib.kvring_latent_create(ctypes.byref(self.cfg), workspace.data_ptr(), workspace.numel(),
                                           self._stream(stream), ctypes.byref(h)), "kvring_latent_create")
        self.handle = h
        self._append, self._read = lib.kvring_latent_append, lib.kvring_latent_read
        self._attend, self._expanded = lib.kvring_latent_attend, lib.kvring_latent_attend_expanded
        ptrs = [ctypes.c_void_p() for _ in range(3)]
        check(lib.kvring_latent_layout(h, *[ctypes.byref(p) for p in ptrs]), "kvring_latent_layout")
        kc, ks, _ = [p.value - workspace.data_ptr() for p in ptrs]
        L, N, P, W = self.layers, self.n_pages, self.page_tokens, self.width
        self.codes = workspace[kc:kc + L * N * P * W].view(L, N, P, W)
        self.scales = workspace[ks:ks + L * N * P * 4].view(torch.float32).view(L, N, P)

    def _stream(self, stream):
        if stream is None:
            return _get_stream(self._index)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    # The checks run before every call, beside kernels of a few microseconds:
    # the good case first, the reason only for a bad one.
    def _rows(self, t, n, width, what):
        """Elements between the rows of [n, width]."""
        if t.dtype is self.dtype and t.shape == (n, width) and t.get_device() == self._index:
            row, one = t.stride()
            if n <= 1:
                row = width                    # the only row's stride is not used
            if not n or one == 1 and row >= width and row % 8 == 0:
                return row
        raise KVRingError(self._bad(t, (n, width), what, "numbers side by side and rows a multiple of 8 elements apart"))

    def _heads(self, t, n, width, what):
        """(token, head) strides of [n, q_heads, width], in any order of the two."""
        heads = self.q_heads
        if t.dtype is self.dtype and t.shape == (n, heads, width) and t.get_device() == self._index:
            token, head, one = t.stride()
            if n <= 1:
                token = 0                      # the only token's stride is not used
            if heads == 1:
                head = 0
            if not n or one == 1 and _apart(token, head, n, heads, width):
                return token, head
        raise KVRingError(self._bad(t, (n, heads, width), what,
                                    "a head's numbers side by side, heads and tokens multiples of 8 elements apart"))

    def _bad(self, t, shape, what, rule):
        if t.dtype is not self.dtype:
            return f"{what}: {t.dtype}; the cache was made for {self.dtype}"
        if tuple(t.shape) != shape:
            return f"{what}: shape {tuple(t.shape)}; {list(shape)} is read"
        if t.get_device() != self._index:
            return f"{what}: on {t.device}, the cache is on cuda:{self._index}"
        return f"{what}: strides {t.stride()}; {rule}"

    def _ints(self, t, shape, what):
        if t.dtype is _I32 and t.shape == shape and t.is_contiguous() and t.get_device() == self._index:
            return t.data_ptr()
        raise KVRingError(_bad_ints(t, shape, self._index, what))

    def _batch(self, layer, seq_start, kv_len, page_table):
        """The batch's arguments in the library's order: (start, len, n_seqs), (table, stride, width)."""
        if self.handle is None:
            raise KVRingError("the cache is closed")
        if not 0 <= layer < self.layers:
            raise KVRingError(f"layer: {layer} of {self.layers}")
        shape = page_table.shape
        if len(shape) != 2 or shape[1] < 1:
            raise KVRingError(f"page_table: shape {tuple(shape)}; [sequences, at least 1] is read")
        n_seqs, width = shape
        if width * self.page_tokens > _k.KVRING_PAGED_MAX_LEN:
            raise KVRingError(f"page_table: {width} pages a row, more than {_k.KVRING_PAGED_MAX_LEN} tokens")
        if page_table.dtype is not _I32 or page_table.get_device() != self._index:
            raise KVRingError(f"page_table: {page_table.dtype} on {page_table.device}; torch.int32 on cuda:{self._index} is read")
        row, one = page_table.stride()
        if (width > 1 and one != 1) or (n_seqs > 1 and row < width):
            raise KVRingError(f"page_table: strides {(row, one)}; a row's entries side by side")
        return self._seqs(n_seqs, seq_start, kv_len), (page_table.data_ptr(), max(row, width), width)

    def _seqs(self, n_seqs, seq_start, kv_len):
        if n_seqs > _k.KVRING_PAGED_MAX_SEQS:
            raise KVRingError(f"{n_seqs} sequences; a call takes at most {_k.KVRING_PAGED_MAX_SEQS}")
        return self._ints(seq_start, (n_seqs + 1,), "seq_start"), self._ints(kv_len, (n_seqs,), "kv_len"), n_seqs

    def _call(self, fn, *args):
        """The library's function with the cache's device current."""
        if _get_device() == self._index:
            status = fn(self.handle, *args)
        else:
            with torch.cuda.device(self.device):
                status = fn(self.handle, *args)
        if status:
            check(status, fn.__name__)

    def _out(self, shape, stream):
        if stream is None:
            return torch.empty(shape, dtype=self.dtype, device=self.device)
        # memory that the allocator knows to be in use on that stream
        with torch.cuda.stream(_as_stream(stream, self.device)):
            return torch.empty(shape, dtype=self.dtype, device=self.device)

    def append(self, latent, k_rope, pos, seq_start, kv_len, page_table, layer=0, stream=None):
        """Write the new tokens' rows: ``latent`` [N, latent_dim] and ``k_rope``
        [N, 64], rotated at ``pos`` (int32 [N, n_axes]); rows any multiple of 8
        elements apart.

        Sequence b's new tokens are rows seq_start[b] .. seq_start[b+1]-1;
        kv_len[b] counts its tokens with them; page_table[b] lists its pages in
        order."""
        n = latent.shape[0]
        ls, rs = self._rows(latent, n, self.latent_dim, "latent"), self._rows(k_rope, n, ROPE, "k_rope")
        (start, length, n_seqs), table = self._batch(layer, seq_start, kv_len, page_table)
        p = self._ints(pos, (n, self.n_axes), "pos")
        if n and n_seqs:
            self._call(self._append, layer, latent.data_ptr(), ls, k_rope.data_ptr(), rs, p, start, length, n_seqs, n,
                       *table, self._stream(stream))

    def read(self, seq_start, kv_len, page_table, n_rows=None, out=None, layer=0, stream=None):
        """Cached rows back, [n_rows, latent_dim + 64] in the cache's type (the
        last 64 rotated, as they were written): row i of n of sequence b is its
        token kv_len[b] - n + i, n = seq_start[b+1] - seq_start[b].  ``n_rows`` or
        ``out`` says how many rows there are; rows of no sequence are not written."""
        (start, length, n_seqs), table = self._batch(layer, seq_start, kv_len, page_table)
        if out is None:
            if n_rows is None or n_rows < 0:
                raise KVRingError("n_rows: the number of rows, where no out is given")
            out = self._out((n_rows, self.width), stream)
        n = out.shape[0]
        if n_rows is not None and n_rows != n:
            raise KVRingError(f"n_rows: {n_rows}; out has {n}")
        row = self._rows(out, n, self.width, "out")
        if n and n_seqs:
            self._call(self._read, layer, start, length, n_seqs, n, *table, out.data_ptr(), row, self._stream(stream))
        return out

    def _mask(self, causal, window, scale, max_new, n):
        """The masks' and the scale's arguments: causal, window, scale."""
        if window is not None and (not causal or window < 1):
            raise KVRingError("window: a positive number of tokens, with causal")
        if not 2.0 ** -100 <= scale <= 2.0 ** 100:
            raise KVRingError(f"scale: {scale}; 2^-100 .. 2^100")
        if max_new is not None and not 1 <= max_new <= max(n, 1):
            raise KVRingError(f"max_new: {max_new}; 1 .. {n}")
        return 1 if causal else 0, min(window or 0, _k.KVRING_PAGED_MAX_LEN), scale

    def attend(self, q_latent, q_rope, q_pos, seq_start, kv_len, page_table, scale, out=None, layer=0, causal=True,
               window=None, max_new=None, stream=None):
        """softmax(scale (q_latent . c + rotated q_rope . r)) c of every new token
        and head over its sequence's cache; [N, q_heads, latent_dim].

        q_latent: [N, q_heads, latent_dim], q_rope: [N, q_heads, 64], out; each
        with token and head strides of its own (slices and transposes of what
        the products leave).  window: with causal, the number of cached tokens a
        query sees at most, its own included.  max_new: the most new tokens that
        a sequence of this call has, where the caller knows it (a sequence with
        more is left out and flagged).  Without it any sequence may have all of
        the call's tokens: single tokens of up to 32 heads then take the kernel of
        64 rows, half of them empty (32 over 1,000 to 4,000, 32 heads: 54 us
        instead of 42)."""
        n = q_latent.shape[0]
        qt, qh = self._heads(q_latent, n, self.latent_dim, "q_latent")
        rt, rh = self._heads(q_rope, n, ROPE, "q_rope")
        seqs, table = self._batch(layer, seq_start, kv_len, page_table)
        p = self._ints(q_pos, (n, self.n_axes), "q_pos")
        mask = self._mask(causal, window, scale, max_new, n)
        if out is None:
            out = self._out((n, self.q_heads, self.latent_dim), stream)
        ot, oh = self._heads(out, n, self.latent_dim, "out")
        start, length, n_seqs = seqs
        if n and n_seqs:
            self._call(self._attend, layer, q_latent.data_ptr(), qt, qh, q_rope.data_ptr(), rt, rh, p, start, length,
                       n_seqs, n, n if max_new is None else max_new, *table, *mask, out.data_ptr(), ot, oh,
                       self._stream(stream))
        return out

    def attend_expanded(self, q, k, k_rope, v, q_pos, seq_start, kv_start, kv_len, out=None, causal=True, window=None,
                        scale=None, max_new=None, stream=None):
        """Attention of the new tokens' queries over keys and values that the
        caller made from the rows (``read``); [N, q_heads, 128].

        q: [N, q_heads, 192], its last 64 rotated here at q_pos.  k, v: [T,
        q_heads, 128].  k_rope: [T, 64], rotated already, as ``read`` gives it.
        Sequence b's keys are rows kv_start[b] .. kv_start[b] + kv_len[b] - 1, in
        order; kv_len counts its new tokens' own.  scale: 1 / sqrt(192) unless
        given; causal, window and max_new as in ``attend``.  q, k, v and out
        have token and head strides of their own."""
        if self.handle is None:
            raise KVRingError("the cache is closed")
        n, t = q.shape[0], k.shape[0]
        if t > 1 << 30:
            raise KVRingError(f"k: {t} rows; at most 2^30 are read")
        qt, qh = self._heads(q, n, HEAD + ROPE, "q")
        kt, kh = self._heads(k, t, HEAD, "k")
        vt, vh = self._heads(v, t, HEAD, "v")
        rt = self._rows(k_rope, t, ROPE, "k_rope")
        if kv_len.dim() != 1:
            raise KVRingError(_bad_ints(kv_len, (None,), self._index, "kv_len"))
        start, length, n_seqs = self._seqs(kv_len.shape[0], seq_start, kv_len)
        first = self._ints(kv_start, (n_seqs,), "kv_start")
        p = self._ints(q_pos, (n, self.n_axes), "q_pos")
        mask = self._mask(causal, window, 1.0 if scale is None else scale, max_new, n)
        if out is None:
            out = self._out((n, self.q_heads, HEAD), stream)
        ot, oh = self._heads(out, n, HEAD, "out")
        if n and n_seqs:
            self._call(self._expanded, q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, k_rope.data_ptr(), rt, v.data_ptr(), vt,
                       vh, t, p, start, first, length, n_seqs, n, n if max_new is None else max_new, mask[0], mask[1],
                       scale or 0.0, out.data_ptr(), ot, oh, self._stream(stream))
        return out

    def debug_state(self, stream=None):
        """The device error bits (KVRING_DEVERR_*); waits for the stream."""
        err = ctypes.c_int32()
        with torch.cuda.device(self.device):
            check(_k.load().kvring_latent_debug_state(self.handle, self._stream(stream), ctypes.byref(err)),
                  "kvring_latent_debug_state")
        return int(err.value)

    def close(self):
        if self.handle is not None:
            _k.load().kvring_latent_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
