"""The batch's paged cache: block tables from request lengths, attention of single
tokens behind a prefix that all requests share and of chunks of new tokens, and the
blocks' way from row to row and back to the free list.

Argument checks and marshalling for the ``vt_paged_*`` entry points of
``include/vt_sampler.h``, which document the layouts; the work runs in the CUDA
kernels of ``libvt_sampler.so``.
"""
from __future__ import annotations

import ctypes as C

import torch

from .sampler import (DTYPE_BF16, DTYPE_F16, VT_OK, P, PagedConfig, VtError, lend, load_library,
                      make_on, other_stream, raw_stream)

# A decode step makes these calls once a layer or once a token, and at its sizes
# the host's share is the larger one: checks read each attribute once, pointers go
# to ctypes as plain integers.
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


def _ids(t, name, device, size=None, dtype=_I32):
    """The address of a contiguous 1-D tensor of ``size`` elements (None: any) on ``device``."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device
            and t.dim() == 1 and t.is_contiguous() and (size is None or t.shape[0] == size)):
        what = (f"{tuple(t.shape)} {t.dtype} on {t.device}" if isinstance(t, torch.Tensor)
                else type(t).__name__)
        raise ValueError(f"{name} must be a contiguous {dtype} tensor "
                         f"[{'n' if size is None else size}] on cuda:{device}, not {what}")
    return t.data_ptr()


def _outputs(out, names, sizes, place, device, other):
    """int32 outputs of ``sizes`` elements, new ones where ``out`` is None, and their addresses."""
    if out is None:
        empty = torch.empty
        out = make_on(other, lambda: tuple([empty(n, dtype=_I32, device=place) for n in sizes]))
        return out, [t.data_ptr() for t in out]
    return out, [_ids(t, "out " + nm, device, n)
                 for t, nm, n in zip(out, names, sizes, strict=True)]


class PagedBatch:
    """One ``vt_paged`` handle: a batch of requests over a paged cache."""

    def __init__(self, max_batch: int, block_size: int, max_blocks: int, q_heads: int = 0,
                 kv_heads: int = 0, head_dim: int = 0, device: int | None = None):
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
        self._shape = (block_size, q_heads, kv_heads, head_dim)

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

    # -- block tables ----------------------------------------------------------
    def build_tables(self, table, seq_lens, query_lens, free_blocks, cursor, held=None,
                     prefix_blocks=None, capacity: int | None = None, out=None, stream=None):
        """vt_paged_tables: give every request of ``seq_lens`` its cache blocks and its
        ``query_lens`` new tokens their slots.

        ``table`` int32 [B, >= max_blocks] is written in place.  Returns ``(held, cursor,
        starts, slots, positions, status)``: int32 [B], [1] and [B + 1], int64 and int32
        [capacity] (default: ``B``, one token a request), int32 [B].  ``out`` gives those six
        tensors; ``held`` and ``cursor`` among them must not be the inputs.  Nothing waits: on a
        ``stream`` that is not the current one the inputs have to be ready there, and the outputs
        are."""
        dev = self.device
        B = seq_lens.shape[0] if isinstance(seq_lens, torch.Tensor) and seq_lens.dim() else 0
        p_seq = _ids(seq_lens, "seq_lens", dev, B)
        p_query = _ids(query_lens, "query_lens", dev, B)
        p_free = _ids(free_blocks, "free_blocks", dev)
        p_cursor = _ids(cursor, "cursor", dev, 1)
        p_held = None if held is None else _ids(held, "held", dev, B)
        if prefix_blocks is None:
            p_prefix, n_prefix = None, 0
        else:
            p_prefix, n_prefix = _ids(prefix_blocks, "prefix_blocks", dev), prefix_blocks.shape[0]
        p_table, ld = self._table(table, B, self.cfg.max_blocks)
        n = B if capacity is None else int(capacity)
        if n < 0:
            raise ValueError(f"capacity={n}")
        other = other_stream(stream)
        if out is None:
            new, place = torch.empty, seq_lens.device  # (half of new_empty's time)
            out = make_on(other, lambda: (
                new(B, dtype=_I32, device=place), new(1, dtype=_I32, device=place),
                new(B + 1, dtype=_I32, device=place), new(n, dtype=_I64, device=place),
                new(n, dtype=_I32, device=place), new(B, dtype=_I32, device=place)))
            po = [t.data_ptr() for t in out]
        else:
            names = ("held", "cursor", "starts", "slots", "positions", "status")
            sizes = (B, 1, B + 1, n, n, B)
            po = [_ids(t, "out " + nm, dev, k, _I64 if nm == "slots" else _I32)
                  for t, nm, k in zip(out, names, sizes, strict=True)]
        rc = self._lib.vt_paged_tables(
            self._h, B, p_seq, p_query, p_held, p_prefix, n_prefix, p_free, free_blocks.shape[0],
            p_cursor, p_table, ld, po[0], po[1], po[2], po[3], po[4], n, po[5],
            raw_stream(stream, dev))
        if rc != VT_OK:
            self._check(rc, "vt_paged_tables")
        if other is not None:
            lend(other, (table, seq_lens, query_lens, free_blocks, cursor, held, prefix_blocks,
                         *out))
        return out

    def _table(self, table, B, columns, name="table"):
        """Address and row stride of a block table."""
        if not (isinstance(table, torch.Tensor) and table.dtype is _I32 and table.dim() == 2
                and table.get_device() == self.device and table.shape[0] == B
                and table.shape[1] >= columns and table.stride(1) == 1):
            raise ValueError(f"{name} must be an int32 tensor [{B}, >= {columns}] on "
                             f"cuda:{self.device} with contiguous rows")
        return table.data_ptr(), table.stride(0) if B > 1 else table.shape[1]

    # -- attention ---------------------------------------------------------------
    def attention(self, q, k_cache, v_cache, table, seq_lens, prefix_blocks=None,
                  prefix_len: int = 0, scale: float | None = None, max_seq_len: int = 0,
                  out=None, lse=None, stream=None):
        """vt_paged_attention_ex: one query token a request over its first ``seq_lens`` cached
        tokens, the first ``prefix_len`` of which all requests share.

        ``q`` [B, q_heads, head_dim] and the caches [blocks, block_size, kv_heads, head_dim]
        (of any strides that are multiples of 8 elements, the last 1; a cache stored
        [blocks, kv_heads, block_size, head_dim] goes in transposed) are bf16 or fp16.
        Requests longer than the table's columns are cut there.
        Returns ``(out, lse)``: q's type [B, q_heads, head_dim] and float32 [B, q_heads].
        ``scale`` defaults to head_dim ** -0.5.  Nothing waits: on a ``stream`` that is not the
        current one the inputs have to be ready there, and the outputs are."""
        dev = self.device
        block_size, q_heads, kv_heads, d = self._shape
        if q_heads == 0:
            raise ValueError("this PagedBatch was made without heads")
        qt = q.dtype if isinstance(q, torch.Tensor) else None
        dtype = DTYPE_BF16 if qt is torch.bfloat16 else DTYPE_F16 if qt is torch.float16 else None
        if dtype is None:
            raise ValueError(f"unsupported q: {qt or type(q).__name__}")
        B = q.shape[0]
        if q.shape != (B, q_heads, d) or q.get_device() != dev or q.stride(2) != 1:
            raise ValueError(f"q must be [B, {q_heads}, {d}] on cuda:{dev} with contiguous heads, "
                             f"not {tuple(q.shape)} on {q.device}")
        blocks, s_block, s_token, s_head = self._caches(qt, k_cache, v_cache)
        p_table, ld = self._table(table, B, 1)
        if max_seq_len > table.shape[1] * block_size:
            raise ValueError(f"max_seq_len={max_seq_len} is past the table's columns")
        p_seq = _ids(seq_lens, "seq_lens", dev, B)
        p_prefix = None
        if prefix_len > 0:
            p_prefix = _ids(prefix_blocks, "prefix_blocks", dev)
            if prefix_blocks.shape[0] * block_size < prefix_len:
                raise ValueError(f"{prefix_blocks.shape[0]} prefix blocks do not hold "
                                 f"{prefix_len} tokens")
        other = other_stream(stream)
        if out is None:
            out, = make_on(other, lambda: (
                torch.empty((B, q_heads, d), dtype=qt, device=q.device),))
        elif (out.dtype is not qt or out.get_device() != dev or not out.is_contiguous()
              or out.shape != q.shape):
            raise ValueError(f"out must be a contiguous {qt} tensor like q")
        if lse is None:
            lse, = make_on(other, lambda: (
                torch.empty((B, q_heads), dtype=_F32, device=q.device),))
        elif (lse.dtype is not _F32 or lse.get_device() != dev or not lse.is_contiguous()
              or lse.shape != (B, q_heads)):
            raise ValueError(f"lse must be a contiguous float32 tensor [{B}, {q_heads}]")
        rc = self._lib.vt_paged_attention_ex(
            self._h, dtype, B, q.data_ptr(), q.stride(0) if B > 1 else q_heads * d,
            q.stride(1) if q_heads > 1 else d, k_cache.data_ptr(), v_cache.data_ptr(), blocks,
            s_block, s_token, s_head, p_table, ld, table.shape[1], p_seq,
            p_prefix, int(prefix_len), int(max_seq_len), d ** -0.5 if scale is None else scale,
            out.data_ptr(), lse.data_ptr(), raw_stream(stream, dev))
        if rc != VT_OK:
            self._check(rc, "vt_paged_attention")
        if other is not None:
            lend(other, (q, k_cache, v_cache, table, seq_lens,
                         None if p_prefix is None else prefix_blocks, out, lse))
        return out, lse

    def chunk_attention(self, q, starts, k_cache, v_cache, table, seq_lens,
                        scale: float | None = None, out=None, lse=None, stream=None):
        """vt_paged_chunk_attention: several new query tokens a request, each up to its own
        position.

        ``q`` [T, q_heads, head_dim]: rows ``starts[b]`` .. ``starts[b + 1] - 1`` (int32 [B + 1],
        as ``build_tables`` returns it) are the last of request b's ``seq_lens[b]`` tokens, which
        the caches already hold.  Rows behind ``starts[B]`` are left as they are.  The caches,
        ``table``, ``scale`` and what is returned, ``(out, lse)`` of T rows, as in ``attention``.
        Nothing waits: on a ``stream`` that is not the current one the inputs have to be ready
        there, and the outputs are."""
        dev = self.device
        block_size, q_heads, kv_heads, d = self._shape
        if q_heads == 0:
            raise ValueError("this PagedBatch was made without heads")
        qt = q.dtype if isinstance(q, torch.Tensor) else None
        dtype = DTYPE_BF16 if qt is torch.bfloat16 else DTYPE_F16 if qt is torch.float16 else None
        if dtype is None:
            raise ValueError(f"unsupported q: {qt or type(q).__name__}")
        T = q.shape[0]
        if q.shape != (T, q_heads, d) or q.get_device() != dev or q.stride(2) != 1:
            raise ValueError(f"q must be [T, {q_heads}, {d}] on cuda:{dev} with contiguous heads, "
                             f"not {tuple(q.shape)} on {q.device}")
        blocks, s_block, s_token, s_head = self._caches(qt, k_cache, v_cache)
        B = seq_lens.shape[0] if isinstance(seq_lens, torch.Tensor) and seq_lens.dim() else 0
        p_seq = _ids(seq_lens, "seq_lens", dev, B)
        p_starts = _ids(starts, "starts", dev, B + 1)
        p_table, ld = self._table(table, B, 1)
        other = other_stream(stream)
        if out is None:
            out, = make_on(other, lambda: (
                torch.empty((T, q_heads, d), dtype=qt, device=q.device),))
        elif (out.dtype is not qt or out.get_device() != dev or not out.is_contiguous()
              or out.shape != q.shape):
            raise ValueError(f"out must be a contiguous {qt} tensor like q")
        if lse is None:
            lse, = make_on(other, lambda: (
                torch.empty((T, q_heads), dtype=_F32, device=q.device),))
        elif (lse.dtype is not _F32 or lse.get_device() != dev or not lse.is_contiguous()
              or lse.shape != (T, q_heads)):
            raise ValueError(f"lse must be a contiguous float32 tensor [{T}, {q_heads}]")
        rc = self._lib.vt_paged_chunk_attention(
            self._h, dtype, B, T, q.data_ptr(), q.stride(0) if T > 1 else q_heads * d,
            q.stride(1) if q_heads > 1 else d, p_starts, k_cache.data_ptr(), v_cache.data_ptr(),
            blocks, s_block, s_token, s_head, p_table, ld, table.shape[1], p_seq,
            d ** -0.5 if scale is None else scale, out.data_ptr(), lse.data_ptr(),
            raw_stream(stream, dev))
        if rc != VT_OK:
            self._check(rc, "vt_paged_chunk_attention")
        if other is not None:
            lend(other, (q, starts, k_cache, v_cache, table, seq_lens, out, lse))
        return out, lse

    def _caches(self, qt, k_cache, v_cache):
        """Blocks and strides of the two caches, checked."""
        dev = self.device
        block_size, _, kv_heads, d = self._shape
        kv = k_cache.stride()
        for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            shape = t.shape
            if (t.dtype is not qt or t.get_device() != dev or len(shape) != 4
                    or shape != (k_cache.shape[0], block_size, kv_heads, d)):
                raise ValueError(f"{name} must be a {qt} tensor [blocks, {block_size}, "
                                 f"{kv_heads}, {d}] on cuda:{dev}, not {tuple(shape)}")
            if t.stride() != kv or kv[3] != 1:
                raise ValueError("the caches must have equal strides and contiguous heads")
        # (the stride of a dimension of one element may be anything)
        blocks = k_cache.shape[0]
        return (blocks, kv[0] if blocks > 1 else block_size * kv_heads * d,
                kv[1] if block_size > 1 else kv_heads * d, kv[2] if kv_heads > 1 else d)

    # -- the blocks' way -------------------------------------------------------------
    def fork(self, table, held, seq_lens, parents, free_blocks, cursor, out_table, out=None,
             stream=None):
        """vt_paged_fork: rows of a new table that continue rows ``parents`` (int32 [R], -1: an
        empty row) of ``table``.

        ``out_table`` int32 [R, >= max_blocks] (not ``table``) is written.  Returns ``(held,
        seq_lens, cursor, src, dst, status)``, int32 [R] ([1] for the cursor); ``src`` and ``dst``
        go to ``copy_blocks``.  ``out`` gives those six tensors.  Nothing waits: on a ``stream``
        that is not the current one the inputs have to be ready there, and the outputs are."""
        dev = self.device
        B = seq_lens.shape[0] if isinstance(seq_lens, torch.Tensor) and seq_lens.dim() else 0
        p_seq = _ids(seq_lens, "seq_lens", dev, B)
        p_held = _ids(held, "held", dev, B)
        p_parents = _ids(parents, "parents", dev)
        R = parents.shape[0]
        p_free = _ids(free_blocks, "free_blocks", dev)
        p_cursor = _ids(cursor, "cursor", dev, 1)
        p_table, ld = self._table(table, B, self.cfg.max_blocks)
        p_out, ld_out = self._table(out_table, R, self.cfg.max_blocks, "out_table")
        other = other_stream(stream)
        out, po = _outputs(out, ("held", "seq_lens", "cursor", "src", "dst", "status"),
                           (R, R, 1, R, R, R), seq_lens.device, dev, other)
        rc = self._lib.vt_paged_fork(
            self._h, R, p_parents, B, p_table, ld, p_held, p_seq, p_free, free_blocks.shape[0],
            p_cursor, p_out, ld_out, *po, raw_stream(stream, dev))
        if rc != VT_OK:
            self._check(rc, "vt_paged_fork")
        if other is not None:
            lend(other, (table, held, seq_lens, parents, free_blocks, cursor, out_table, *out))
        return out

    def release(self, table, held, seq_lens, num_blocks: int, prefix_blocks=None, out=None,
                stream=None):
        """vt_paged_release: keep the blocks that ``seq_lens`` tokens of each row fill and make
        the free list anew of all others of the cache's ``num_blocks``.

        ``table`` is written in place (-1 past the kept columns).  Returns ``(held, free_blocks,
        cursor)``, int32 [B], [num_blocks] and [1]; ``out`` gives those three.  Nothing waits: on
        a ``stream`` that is not the current one the inputs have to be ready there, and the
        outputs are."""
        args, other, ins = self._reclaim(table, held, seq_lens, num_blocks, prefix_blocks, stream)
        out, po = _outputs(out, ("held", "free_blocks", "cursor"), (args[0], num_blocks, 1),
                           seq_lens.device, self.device, other)
        rc = self._lib.vt_paged_release(self._h, *args, *po, raw_stream(stream, self.device))
        if rc != VT_OK:
            self._check(rc, "vt_paged_release")
        if other is not None:
            lend(other, (*ins, *out))
        return out

    def compact(self, table, held, seq_lens, num_blocks: int, prefix_blocks=None, out_table=None,
                out=None, stream=None):
        """vt_paged_compact: ``release``, and the blocks in use moved to the cache's low end.

        ``out_table`` (default: ``table``, in place) receives the rows with the new ids.  Returns
        ``(held, free_blocks, cursor, src, dst, count, prefix_blocks)``, int32; ``copy_blocks(
        caches, src, dst, count)`` then makes the moves.  ``out`` gives those seven.  Nothing
        waits: on a ``stream`` that is not the current one the inputs have to be ready there, and
        the outputs are."""
        args, other, ins = self._reclaim(table, held, seq_lens, num_blocks, prefix_blocks, stream)
        B = seq_lens.shape[0]
        if out_table is None:
            out_table = table
        p_table, ld_out = self._table(out_table, B, self.cfg.max_blocks, "out_table")
        n_prefix, most = args[6], num_blocks // 2
        out, po = _outputs(
            out, ("held", "free_blocks", "cursor", "src", "dst", "count", "prefix_blocks"),
            (B, num_blocks, 1, most, most, 1, n_prefix), seq_lens.device, self.device, other)
        rc = self._lib.vt_paged_compact(
            self._h, *args, p_table, ld_out, po[0], po[1], po[2], po[6], po[3], po[4], po[5],
            raw_stream(stream, self.device))
        if rc != VT_OK:
            self._check(rc, "vt_paged_compact")
        if other is not None:
            lend(other, (*ins, out_table, *out))
        return out

    def _reclaim(self, table, held, seq_lens, num_blocks, prefix_blocks, stream):
        """The arguments that release and compact share, the other stream, and the inputs."""
        dev = self.device
        B = seq_lens.shape[0] if isinstance(seq_lens, torch.Tensor) and seq_lens.dim() else 0
        p_seq = _ids(seq_lens, "seq_lens", dev, B)
        p_held = _ids(held, "held", dev, B)
        if num_blocks < 1:
            raise ValueError(f"num_blocks={num_blocks}")
        p_prefix, n_prefix = None, 0
        if prefix_blocks is not None:
            p_prefix, n_prefix = _ids(prefix_blocks, "prefix_blocks", dev), prefix_blocks.shape[0]
        p_table, ld = self._table(table, B, self.cfg.max_blocks)
        return ((B, p_table, ld, p_held, p_seq, p_prefix, n_prefix, num_blocks),
                other_stream(stream), (table, held, seq_lens, prefix_blocks))

    def copy_blocks(self, caches, src, dst, count=None, stream=None):
        """vt_paged_copy_blocks: block ``src[i]`` to block ``dst[i]`` (int32 [n], pairs with a
        negative id skipped; ``count`` int32 [1]: only the first of them) in every tensor of
        ``caches``: equal in shape, type and strides, the first dimension the blocks, each block's
        elements without gaps, in any order.  Nothing waits: on a ``stream`` that is not the
        current one the inputs have to be ready there, and the caches are."""
        dev = self.device
        caches = list(caches)
        p_src = _ids(src, "src", dev)
        n = src.shape[0]
        p_dst = _ids(dst, "dst", dev, n)
        p_count = None if count is None else _ids(count, "count", dev, 1)
        if not caches:
            return
        first = caches[0]
        shape, strides, dt = first.shape, first.stride(), first.dtype
        for t in caches:
            if t.shape != shape or t.stride() != strides or t.dtype is not dt:
                raise ValueError("the caches must be equal in shape, strides and type")
            if t.get_device() != dev:
                raise ValueError(f"a cache is on {t.device}, the handle on cuda:{dev}")
        each = 1
        for stride, size in sorted([(st, s) for s, st in zip(shape[1:], strides[1:]) if s != 1]):
            if stride != each:
                raise ValueError(f"the elements of a block have gaps: strides {tuple(strides)}")
            each *= size
        if len(shape) < 2 or each < 1 or shape[0] < 1 or (shape[0] > 1 and strides[0] < each):
            raise ValueError(f"caches of shape {tuple(shape)}, strides {tuple(strides)}")
        size = first.element_size()
        ptrs = (P * len(caches))(*[t.data_ptr() for t in caches])
        rc = self._lib.vt_paged_copy_blocks(
            self._h, ptrs, len(caches), shape[0], (strides[0] if shape[0] > 1 else each) * size,
            each * size, p_src, p_dst, n, p_count, raw_stream(stream, dev))
        if rc != VT_OK:
            self._check(rc, "vt_paged_copy_blocks")
        other = other_stream(stream)
        if other is not None:
            lend(other, (*caches, src, dst, count))
