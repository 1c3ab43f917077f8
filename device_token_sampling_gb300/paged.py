"""The batch's paged cache: block tables from request lengths, and attention of
single tokens behind a prefix that all requests share.

Argument checks and marshalling for the ``vt_paged_*`` entry points of
``include/vt_sampler.h``, which document the layouts; the work runs in the CUDA
kernels of ``libvt_sampler.so``.
"""
from __future__ import annotations

import ctypes as C

from .sampler import (DTYPE_BF16, DTYPE_F16, VT_OK, P, PagedConfig, VtError, _stream_ptr,
                      load_library)


def _ids(t, name, shape, device, dtype=None):
    """A contiguous int32 (or ``dtype``) tensor of ``shape`` (None: any size) on ``device``."""
    import torch
    dtype = dtype or torch.int32
    if not torch.is_tensor(t) or t.dtype != dtype or t.dim() != len(shape):
        raise ValueError(f"{name} must be a {len(shape)}-D {dtype} tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, need {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return P(t.data_ptr())


def _on_stream(stream, tensors):
    """Outputs made here for another stream than the current one live until it is done."""
    import torch
    if stream is not None and stream != torch.cuda.current_stream(stream.device):
        for t in tensors:
            t.record_stream(stream)


class PagedBatch:
    """One ``vt_paged`` handle: a batch of requests over a paged cache."""

    def __init__(self, max_batch: int, block_size: int, max_blocks: int, q_heads: int = 0,
                 kv_heads: int = 0, head_dim: int = 0, device: int | None = None):
        import torch
        self._h = None
        self._lib = load_library()
        if device is None:
            device = torch.cuda.current_device()
        self.device = int(device)
        self.cfg = PagedConfig(max_batch, block_size, max_blocks, q_heads, kv_heads, head_dim,
                               self.device)
        h = P()
        rc = self._lib.vt_paged_create(C.byref(self.cfg), C.byref(h))
        if rc != VT_OK:
            raise VtError(rc, f"vt_paged_create({max_batch}, {block_size}, {max_blocks}, "
                              f"{q_heads}, {kv_heads}, {head_dim}, device={self.device})")
        self._h = h

    # -- lifetime ------------------------------------------------------------
    def close(self):
        if self._h:
            self._lib.vt_paged_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _check(self, rc: int, what: str):
        if rc != VT_OK:
            msg = self._lib.vt_paged_last_error(self._h)
            raise VtError(rc, f"{what}: {msg.decode() if msg else ''}")

    def check_errors(self):
        """Wait for the last call and raise what its kernels met."""
        self._check(self._lib.vt_paged_check_errors(self._h), "vt_paged_check_errors")

    def _device(self):
        import torch
        return torch.device("cuda", self.device)

    # -- block tables ----------------------------------------------------------
    def build_tables(self, table, seq_lens, query_lens, free_blocks, cursor, held=None,
                     prefix_blocks=None, capacity: int | None = None, out=None, stream=None):
        """vt_paged_tables: give every request of ``seq_lens`` its cache blocks and its
        ``query_lens`` new tokens their slots.

        ``table`` int32 [B, >= max_blocks] is written in place.  Returns ``(held, cursor,
        starts, slots, positions, status)``: int32 [B], [1] and [B + 1], int64 and int32
        [capacity] (default: ``B``, one token a request), int32 [B].  ``out`` gives those six
        tensors; ``held`` and ``cursor`` among them must not be the inputs.  Nothing waits."""
        import torch
        dev = self._device()
        if not torch.is_tensor(seq_lens) or seq_lens.dim() != 1:
            raise ValueError("seq_lens must be a 1-D int32 tensor")
        B = seq_lens.shape[0]
        p_seq = _ids(seq_lens, "seq_lens", (B,), dev)
        p_query = _ids(query_lens, "query_lens", (B,), dev)
        p_free = _ids(free_blocks, "free_blocks", (None,), dev)
        p_cursor = _ids(cursor, "cursor", (1,), dev)
        p_held = None if held is None else _ids(held, "held", (B,), dev)
        p_prefix = None if prefix_blocks is None else _ids(prefix_blocks, "prefix_blocks",
                                                           (None,), dev)
        if (not torch.is_tensor(table) or table.dtype != torch.int32 or table.dim() != 2
                or table.device != dev or table.shape[0] != B
                or table.shape[1] < self.cfg.max_blocks or table.stride(1) != 1):
            raise ValueError(f"table must be an int32 tensor [{B}, >= {self.cfg.max_blocks}] on "
                             f"{dev} with contiguous rows")
        n = B if capacity is None else int(capacity)
        if n < 0:
            raise ValueError(f"capacity={n}")
        if out is None:
            i32 = dict(dtype=torch.int32, device=dev)
            out = (torch.empty(B, **i32), torch.empty(1, **i32), torch.empty(B + 1, **i32),
                   torch.empty(n, dtype=torch.int64, device=dev), torch.empty(n, **i32),
                   torch.empty(B, **i32))
            _on_stream(stream, out)
        names = ("held", "cursor", "starts", "slots", "positions", "status")
        shapes = ((B,), (1,), (B + 1,), (n,), (n,), (B,))
        po = [_ids(t, "out " + nm, sh, dev, torch.int64 if nm == "slots" else None)
              for t, nm, sh in zip(out, names, shapes)]
        rc = self._lib.vt_paged_tables(
            self._h, B, p_seq, p_query, p_held, p_prefix,
            0 if prefix_blocks is None else prefix_blocks.shape[0], p_free, free_blocks.shape[0],
            p_cursor, P(table.data_ptr()), table.stride(0) if B > 1 else table.shape[1], po[0],
            po[1], po[2], po[3], po[4], n, po[5], _stream_ptr(stream))
        self._check(rc, "vt_paged_tables")
        return tuple(out)

    # -- attention ---------------------------------------------------------------
    def attention(self, q, k_cache, v_cache, table, seq_lens, prefix_blocks=None,
                  prefix_len: int = 0, scale: float | None = None, max_seq_len: int = 0,
                  out=None, lse=None, stream=None):
        """vt_paged_attention: one query token a request over its first ``seq_lens`` cached
        tokens, the first ``prefix_len`` of which all requests share.

        ``q`` [B, q_heads, head_dim] and the caches [blocks, block_size, kv_heads, head_dim]
        (of any strides that are multiples of 8 elements, the last 1; a cache stored
        [blocks, kv_heads, block_size, head_dim] goes in transposed) are bf16 or fp16.
        Returns ``(out, lse)``: q's type [B, q_heads, head_dim] and float32 [B, q_heads].
        ``scale`` defaults to head_dim ** -0.5.  Nothing waits."""
        import torch
        dev, c = self._device(), self.cfg
        if c.q_heads == 0:
            raise ValueError("this PagedBatch was made without heads")
        if not torch.is_tensor(q) or q.dim() != 3 or q.device != dev:
            raise ValueError(f"q must be a 3-D tensor on {dev}")
        B = q.shape[0]
        dtype = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}.get(q.dtype)
        if dtype is None:
            raise ValueError(f"unsupported dtype {q.dtype}")
        if tuple(q.shape) != (B, c.q_heads, c.head_dim) or q.stride(2) != 1:
            raise ValueError(f"q must be [B, {c.q_heads}, {c.head_dim}] with contiguous heads")
        want = (k_cache.shape[0], c.block_size, c.kv_heads, c.head_dim)
        for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            if t.dtype != q.dtype or t.device != dev or tuple(t.shape) != want:
                raise ValueError(f"{name} must be a {q.dtype} tensor [blocks, {c.block_size}, "
                                 f"{c.kv_heads}, {c.head_dim}] on {dev}")
            if t.stride(3) != 1 or t.stride() != k_cache.stride():
                raise ValueError("the caches must have equal strides and contiguous heads")
        if (not torch.is_tensor(table) or table.dtype != torch.int32 or table.dim() != 2
                or table.device != dev or table.shape[0] != B or table.stride(1) != 1):
            raise ValueError(f"table must be an int32 tensor [{B}, columns] on {dev} with "
                             "contiguous rows")
        if max_seq_len > table.shape[1] * c.block_size:
            raise ValueError(f"max_seq_len={max_seq_len} is past the table's columns")
        p_seq = _ids(seq_lens, "seq_lens", (B,), dev)
        p_prefix = None
        if prefix_len > 0:
            if prefix_blocks is None:
                raise ValueError("prefix_len without prefix_blocks")
            p_prefix = _ids(prefix_blocks, "prefix_blocks", (None,), dev)
            if prefix_blocks.shape[0] * c.block_size < prefix_len:
                raise ValueError(f"{prefix_blocks.shape[0]} prefix blocks do not hold "
                                 f"{prefix_len} tokens")
        made = []
        if out is None:
            out = torch.empty((B, c.q_heads, c.head_dim), dtype=q.dtype, device=dev)
            made.append(out)
        elif (out.dtype != q.dtype or out.device != dev or not out.is_contiguous()
              or tuple(out.shape) != (B, c.q_heads, c.head_dim)):
            raise ValueError(f"out must be a contiguous {q.dtype} tensor like q")
        if lse is None:
            lse = torch.empty((B, c.q_heads), dtype=torch.float32, device=dev)
            made.append(lse)
        elif (lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous()
              or tuple(lse.shape) != (B, c.q_heads)):
            raise ValueError(f"lse must be a contiguous float32 tensor [{B}, {c.q_heads}]")
        _on_stream(stream, made)
        rc = self._lib.vt_paged_attention(
            self._h, dtype, B, P(q.data_ptr()), q.stride(0), q.stride(1), P(k_cache.data_ptr()),
            P(v_cache.data_ptr()), k_cache.shape[0], k_cache.stride(0), k_cache.stride(1),
            k_cache.stride(2), P(table.data_ptr()), table.stride(0) if B > 1 else table.shape[1],
            p_seq, p_prefix, int(prefix_len), int(max_seq_len),
            c.head_dim ** -0.5 if scale is None else float(scale), P(out.data_ptr()),
            P(lse.data_ptr()), _stream_ptr(stream))
        self._check(rc, "vt_paged_attention")
        return out, lse
