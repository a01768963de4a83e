"""A KV cache held in 4 bits, on torch tensors: append, read, attention and eviction by accumulated
attention weight (the mbk_kv4_* entry points of include/mbk.h, which documents format, layout and
semantics).

    cache = Kv4Cache(n_layers, n_heads, n_kv_heads, head_dim, num_pages, page_size=64, max_pages=32)
    batch = cache.batch(offsets, rows, tables)           # device int32 tensors; made once, used in every layer
    cache.append(layer, batch, k, v)                     # k, v [n_tokens, n_kv_heads, head_dim], K rotated
    out = cache.attention(layer, batch, q)               # q [n_tokens, n_heads, head_dim]
    rows = cache.evict(rows, tables, next_pos, keep=4096, recent=256)   # track=True

All work goes to torch's current stream of the cache's device.  Nothing here copies, synchronises or
falls back: a tensor of another device, type or layout is refused with ValueError, and a bad argument
that only the library can tell raises MbkError.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import mbk


def _raw_stream(index: int) -> int:
    """The handle of torch's current stream of a device."""
    return torch._C._cuda_getCurrentRawStream(index)  # torch.cuda.current_stream makes an object first: 2 us more


_DTYPES = {torch.float32: mbk.MBK_KV4_FP32, torch.bfloat16: mbk.MBK_KV4_BF16}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


class Kv4Batch:
    """The tokens of a call (mbk_kv4_batch).  It keeps its tensors; their contents may change between
    calls within the bounds that it was made with, their addresses may not.  It serves the cache that made it."""

    def __init__(self, cache: "Kv4Cache", c: mbk.MbkKv4Batch, keep, workspace_bytes: int):
        self.cache = cache  # its bounds and tables are of this cache's shape
        self.c = c
        self.ref = ctypes.byref(c)
        self.keep = keep
        self.n_tokens = c.n_tokens
        self.workspace_bytes = workspace_bytes


class Kv4Cache:
    """A pool of 4-bit pages.  pool: a uint8 tensor of pool_bytes() on the device (made here, zeroed, if
    not given); page tables, row counts and positions stay the caller's."""

    def __init__(self, n_layers: int, n_heads: int, n_kv_heads: int, head_dim: int, num_pages: int, page_size: int = 64,
                 max_pages: int = 1, track: bool = False, pool: Optional[torch.Tensor] = None, device: int = 0):
        if pool is not None:
            device = pool.device.index if pool.device.index is not None else device
        self.cfg = mbk.MbkKv4Config(device, n_layers, n_heads, n_kv_heads, head_dim, num_pages, page_size, max_pages, int(bool(track)))
        self._cfg = ctypes.byref(self.cfg)
        self.lib = mbk.load_library()
        self.bytes = self._size(self.lib.mbk_kv4_pool_bytes(self._cfg), "mbk_kv4_pool_bytes")
        self.index = device
        self.device = torch.device("cuda", device)
        if pool is None:
            pool = torch.zeros(self.bytes, dtype=torch.uint8, device=self.device)
        if pool.dtype != torch.uint8 or not pool.is_contiguous() or pool.numel() != self.bytes or not pool.is_cuda:
            raise ValueError(f"pool: a contiguous uint8 CUDA tensor of {self.bytes} bytes")
        self.pool = pool
        self._evict_bytes = {}  # the last eviction's workspace size, by its arguments
        self._pool = pool.data_ptr()
        # errors that only the kernels see (bits MBK_KV4_BAD_PAGE, MBK_KV4_BAD_BATCH), since the last clear
        self.status_word = torch.zeros(1, dtype=torch.int32, device=self.device)

    @staticmethod
    def _size(n: int, where: str) -> int:
        if n < 0:
            raise mbk.MbkError(int(n), where)
        return int(n)

    def _ints(self, name: str, t, shape) -> None:
        if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != self.device or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous int32 tensor {tuple(shape)} on {self.device}")

    def _rows(self, name: str, t, n: int, heads: int):
        """Data pointer and elements between tokens of a [n, heads, head_dim] tensor."""
        d = self.cfg.head_dim
        if not isinstance(t, torch.Tensor) or t.device != self.device or t.dtype not in _DTYPES or t.shape != (n, heads, d):
            raise ValueError(f"{name}: an fp32 or bf16 tensor {(n, heads, d)} on {self.device}")
        p, ld = t.data_ptr(), heads * d
        if not t.is_contiguous():
            st, unit = t.stride(), 16 // t.element_size()
            if st[2] != 1 or (heads > 1 and st[1] != d) or (n > 1 and (st[0] < ld or st[0] % unit != 0)):
                raise ValueError(f"{name}: heads and elements contiguous, tokens apart by a multiple of 16 bytes")
            ld = st[0] if n > 1 else ld
        if p % 16 != 0:
            raise ValueError(f"{name}: 16-byte aligned")
        return p, ld

    def _own(self, batch: Kv4Batch):
        if batch.cache is not self:
            raise ValueError("batch: of this cache (Kv4Cache.batch)")
        return batch.ref

    def _stream(self) -> int:
        return _raw_stream(self.index)

    def batch(self, offsets, rows, tables, positions=None, n_tokens: Optional[int] = None, max_count: Optional[int] = None,
              max_rows: Optional[int] = None, status: Optional[torch.Tensor] = None) -> Kv4Batch:
        """offsets [n_seq + 1], rows [n_seq], tables [n_seq, max_pages], positions [n_seq] or None: int32 on
        the device.  n_tokens, max_count, max_rows: host bounds; those not given are read from the tensors
        (a synchronising copy) or, max_rows, taken as the tables' reach."""
        n_seq = rows.shape[0] if isinstance(rows, torch.Tensor) and rows.dim() == 1 else 0
        self._ints("rows", rows, (n_seq,))
        self._ints("offsets", offsets, (n_seq + 1,))
        self._ints("tables", tables, (n_seq, self.cfg.max_pages))
        if positions is not None:
            self._ints("positions", positions, (n_seq,))
        if n_tokens is None or max_count is None:
            host = offsets.tolist()
            n_tokens = host[-1] if n_tokens is None else n_tokens
            max_count = max(b - a for a, b in zip(host, host[1:])) if max_count is None else max_count
        if max_rows is None:
            max_rows = self.cfg.max_pages * self.cfg.page_size
        status = self.status_word if status is None else status
        self._ints("status", status, (1,))
        c = mbk.MbkKv4Batch(n_seq, n_tokens, max_count, max_rows, _ptr(offsets), _ptr(rows), _ptr(positions), _ptr(tables), _ptr(status))
        if not (1 <= n_seq <= mbk.MBK_KV4_MAX_SEQS and n_tokens >= 1 and 1 <= max_count <= n_tokens and
                0 <= max_rows <= self.cfg.max_pages * self.cfg.page_size):
            raise mbk.MbkError(mbk.MBK_ERR_INVALID_ARG, "Kv4Cache.batch")
        size = self._size(self.lib.mbk_kv4_attention_workspace(self._cfg, ctypes.byref(c)), "mbk_kv4_attention_workspace")
        return Kv4Batch(self, c, (offsets, rows, tables, positions, status), size)

    def append(self, layer: int, batch: Kv4Batch, k, v) -> None:
        """Store the new tokens' rows (mbk_kv4_append)."""
        kp, ld = self._rows("k", k, batch.n_tokens, self.cfg.n_kv_heads)
        vp, ldv = self._rows("v", v, batch.n_tokens, self.cfg.n_kv_heads)
        if ld != ldv or k.dtype != v.dtype:
            raise ValueError("k and v: one type and one distance between tokens")
        mbk._check(self.lib.mbk_kv4_append(self._cfg, self._pool, layer, self._own(batch), kp, vp, ld, _DTYPES[k.dtype], self._stream()),
                   "mbk_kv4_append")

    def read(self, layer: int, batch: Kv4Batch, dtype=torch.float32):
        """The values of the new tokens' rows (mbk_kv4_read): (k, v), each [n_tokens, n_kv_heads, head_dim]."""
        if dtype not in _DTYPES:
            raise ValueError("dtype: torch.float32 or torch.bfloat16")
        shape = (batch.n_tokens, self.cfg.n_kv_heads, self.cfg.head_dim)
        k = torch.empty(shape, dtype=dtype, device=self.device)
        v = torch.empty(shape, dtype=dtype, device=self.device)
        mbk._check(self.lib.mbk_kv4_read(self._cfg, self._pool, layer, self._own(batch), k.data_ptr(), v.data_ptr(), shape[1] * shape[2],
                                         _DTYPES[dtype], self._stream()), "mbk_kv4_read")
        return k, v

    def attention(self, layer: int, batch: Kv4Batch, q, scale: Optional[float] = None, cap: float = 0.0, slopes=None, window: int = 0,
                  accumulate: bool = False, out=None):
        """Attention of the new tokens (mbk_kv4_attention); scale defaults to head_dim ** -0.5."""
        cfg = self.cfg
        qp, ldq = self._rows("q", q, batch.n_tokens, cfg.n_heads)
        if out is None:
            out = torch.empty((batch.n_tokens, cfg.n_heads, cfg.head_dim), dtype=q.dtype, device=self.device)
            op, ldo = out.data_ptr(), cfg.n_heads * cfg.head_dim
        else:
            op, ldo = self._rows("out", out, batch.n_tokens, cfg.n_heads)
            if out.dtype != q.dtype:
                raise ValueError("out: the type of q")
        if slopes is not None and (slopes.dtype != torch.float32 or slopes.device != self.device or not slopes.is_contiguous() or
                                   slopes.shape != (cfg.n_heads,)):
            raise ValueError(f"slopes: a contiguous fp32 tensor {(cfg.n_heads,)} on {self.device}")
        ws = torch.empty(batch.workspace_bytes, dtype=torch.uint8, device=self.device) if batch.workspace_bytes else None
        rc = self.lib.mbk_kv4_attention(self._cfg, self._pool, layer, self._own(batch), qp, ldq, op, ldo, _DTYPES[q.dtype],
                                        cfg.head_dim ** -0.5 if scale is None else scale, cap, _ptr(slopes), window, int(accumulate),
                                        _ptr(ws), batch.workspace_bytes, _raw_stream(self.index))
        if rc != mbk.MBK_OK:
            raise mbk.MbkError(rc, "mbk_kv4_attention")
        return out

    def evict(self, rows, tables, next_pos, keep: int, recent: int = 0, out_tables=None, layer: int = 0, n_layers: Optional[int] = None,
              max_rows: Optional[int] = None, rows_out=None):
        """Cut each sequence to at most `keep` rows in layers [layer, layer + n_layers) (default: all from
        `layer` on), in place or into the pages of out_tables (mbk_kv4_evict).  Returns the new row counts."""
        cfg = self.cfg
        n_seq = rows.shape[0] if isinstance(rows, torch.Tensor) and rows.dim() == 1 else 0
        self._ints("rows", rows, (n_seq,))
        self._ints("tables", tables, (n_seq, cfg.max_pages))
        self._ints("next_pos", next_pos, (n_seq,))
        out_pages = 0
        if out_tables is not None:
            out_pages = out_tables.shape[1] if isinstance(out_tables, torch.Tensor) and out_tables.dim() == 2 else 0
            self._ints("out_tables", out_tables, (n_seq, out_pages))
        if rows_out is None:
            rows_out = torch.empty_like(rows)
        else:
            self._ints("rows_out", rows_out, (n_seq,))
        n_layers = cfg.n_layers - layer if n_layers is None else n_layers
        max_rows = min(cfg.max_pages * cfg.page_size, mbk.MBK_KV4_MAX_EVICT_ROWS) if max_rows is None else max_rows
        key = (n_layers, n_seq, keep)
        size = self._evict_bytes.get(key)
        if size is None:
            size = self._size(self.lib.mbk_kv4_evict_workspace(self._cfg, n_layers, n_seq, keep), "mbk_kv4_evict_workspace")
            self._evict_bytes = {key: size}
        ws = torch.empty(size, dtype=torch.uint8, device=self.device)
        rc = self.lib.mbk_kv4_evict(self._cfg, self._pool, layer, n_layers, n_seq, max_rows, _ptr(rows), _ptr(tables), _ptr(next_pos), keep,
                                    recent, _ptr(out_tables), out_pages, _ptr(rows_out), _ptr(self.status_word), ws.data_ptr(), size,
                                    self._stream())
        mbk._check(rc, "mbk_kv4_evict")
        return rows_out

    def _field(self, at: int, dtype):
        cfg = self.cfg
        if not cfg.track:
            raise ValueError("the pool is not tracked")
        blocks = self.pool.view(cfg.num_pages, cfg.n_layers, cfg.n_kv_heads, cfg.page_size // 32, -1)
        start = 32 * (cfg.head_dim + cfg.head_dim // 64 * 8) + at
        return blocks[..., start:start + 128].view(dtype)

    @property
    def positions(self):
        """The rows' positions: int32 [num_pages, n_layers, n_kv_heads, page_size / 32, 32], a view of the pool."""
        return self._field(0, torch.int32)

    @property
    def weights(self):
        """The rows' accumulated attention weights: fp32, shape as positions, a view of the pool."""
        return self._field(128, torch.float32)

    def status(self) -> int:
        """The bits MBK_KV4_BAD_PAGE / MBK_KV4_BAD_BATCH that calls have raised since clear_status() (synchronises)."""
        return int(self.status_word.item())

    def clear_status(self) -> None:
        self.status_word.zero_()
