"""Paged key-value cache and the attention over it (C ABI in ``include/qgkv.h``).

Like the rest of the package this only marshals arguments: the cache's tensors
are PyTorch tensors, every step of the work runs in the library's HIP kernels on
the current (or the given) stream, and nothing is copied to the host.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

__all__ = ["KVCache"]

TYPE_F16, TYPE_BF16 = 0, 1
INFO_SHORT, INFO_LONG, INFO_PAIR = 1, 2, 4
MAX_SEQS, MIN_PAGE, MAX_PAGE = 1024, 16, 256


class _KvDesc(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("layers", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("dtype", ctypes.c_int32), ("pool", ctypes.c_void_p),
                ("tables", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("info", ctypes.c_void_p)]


class _KvBatch(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("rows", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("seqs", ctypes.c_void_p), ("row_start", ctypes.c_void_p)]


class _KvRows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


def bind(L) -> None:
    """Argument and result types of the qgkv_* functions."""
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    L.qgkv_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(_KvDesc), vp]
    L.qgkv_destroy.argtypes = [vp]
    L.qgkv_extend.argtypes = [vp, vp, vp]
    L.qgkv_fork.argtypes = [vp, vp, vp, i32, vp]
    L.qgkv_trim.argtypes = [vp, vp, vp, i32, vp]
    L.qgkv_compact.argtypes = [vp, vp]
    L.qgkv_append.argtypes = [vp, i32, ctypes.POINTER(_KvBatch), ctypes.POINTER(_KvRows), ctypes.POINTER(_KvRows), vp]
    L.qgkv_attend.argtypes = [vp, i32, ctypes.POINTER(_KvBatch), ctypes.POINTER(_KvRows), ctypes.POINTER(_KvRows), i32,
                              ctypes.c_float, i32, i32, vp]
    for f in ("create", "destroy", "extend", "fork", "trim", "compact", "append", "attend"):
        getattr(L, "qgkv_" + f).restype = ctypes.c_int


class KVCache:
    """A pool of key-value pages, the page tables of up to ``max_seqs`` sequences
    (slots), and the operations on them.

    ``pool`` [pages][layers][2][kv_heads][page_size][head_dim] (fp16 or bf16),
    ``tables`` int32 [max_seqs][max_pages], ``lens`` int32 [max_seqs], ``refs``
    int32 [pages] and ``info`` int32 [4] are CUDA tensors that the caller may
    read at any time (see include/qgkv.h).  One step of a model:

        kv.extend(n_new)                       # once: room for the new tokens
        for layer in ...:
            kv.append(k, v, layer=layer)       # their keys and values
            out = kv.attend(q, layer=layer)    # attention of the new rows

    Rows of a call: ``seqs`` (int32 [n], default slots 0 .. n - 1) names the
    slots; with ``row_start`` (int32 [n + 1], with ``max_rows`` at least the
    largest count) entry j has rows row_start[j] .. row_start[j + 1] - 1, without
    it each has the same number.  They are the last tokens of their slots.
    Index tensors may also be given as lists (copied to the device).
    """

    def __init__(self, pages: int, page_size: int, kv_heads: int, head_dim: int, *, layers: int = 1, max_seqs: int = 1,
                 max_pages: int = None, dtype=None, device=None, stream=None):
        import torch
        device = torch.device("cuda") if device is None else device
        dtype = torch.float16 if dtype is None else dtype
        with _on(stream):
            pool = torch.empty((pages, layers, 2, kv_heads, page_size, head_dim), dtype=dtype, device=device)
            tables = torch.full((max_seqs, pages if max_pages is None else max_pages), -1, dtype=torch.int32,
                                device=device)
            lens = torch.zeros(max_seqs, dtype=torch.int32, device=device)
            refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self._open(pool, tables, lens, refs, stream)

    @classmethod
    def of(cls, pool, tables, lens, refs, stream=None) -> "KVCache":
        """A cache over tensors that exist: a pool in use with its tables."""
        self = cls.__new__(cls)
        self._open(pool, tables, lens, refs, stream)
        return self

    def _open(self, pool, tables, lens, refs, stream):
        import torch
        from . import _check, _stream, lib
        self._h = None
        types = {torch.float16: TYPE_F16, torch.bfloat16: TYPE_BF16}
        if pool.dim() != 6 or pool.shape[2] != 2:
            raise ValueError("pool must be [pages][layers][2][kv_heads][page_size][head_dim]")
        if pool.dtype not in types:
            raise TypeError(f"pool must be float16 or bfloat16, not {pool.dtype}")
        for name, t, shape in (("tables", tables, (lens.numel(), tables.shape[-1])), ("lens", lens, (lens.numel(),)),
                               ("refs", refs, (pool.shape[0],))):
            if t.dtype != torch.int32 or tuple(t.shape) != shape:
                raise ValueError(f"{name} must be int32 {list(shape)}, not {t.dtype} {list(t.shape)}")
        for name, t in (("pool", pool), ("tables", tables), ("lens", lens), ("refs", refs)):
            if not t.is_cuda or t.device != pool.device or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous on the pool's GPU")
        self.pool, self.tables, self.lens, self.refs = pool, tables, lens, refs
        self.pages, self.layers, _, self.kv_heads, self.page_size, self.head_dim = pool.shape
        self.max_seqs, self.max_pages = tables.shape
        with torch.cuda.device(pool.device), _on(stream):
            self.info = torch.zeros(4, dtype=torch.int32, device=pool.device)
            d = _KvDesc(self.pages, self.layers, self.kv_heads, self.head_dim, self.page_size, self.max_seqs,
                        self.max_pages, types[pool.dtype], pool.data_ptr(), tables.data_ptr(), lens.data_ptr(),
                        refs.data_ptr(), self.info.data_ptr())
            h = ctypes.c_void_p()
            _check(lib().qgkv_create(ctypes.byref(h), ctypes.byref(d), _stream(stream)))
        self._h = h

    @property
    def handle(self):
        return self._h

    def _index(self, name, x, n=None):
        """An int32 tensor on the cache's GPU (lists are copied there)."""
        import torch
        if x is None:
            return None
        if not isinstance(x, torch.Tensor):
            x = torch.tensor(list(x), dtype=torch.int32, device=self.pool.device)
        if x.dtype != torch.int32 or x.dim() != 1 or x.device != self.pool.device or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 1-d int32 tensor on {self.pool.device}")
        if n is not None and x.numel() != n:
            raise ValueError(f"{name} has {x.numel()} entries, not {n}")
        return x

    def _rows(self, name, t, heads=None, rows=None) -> _KvRows:
        if t.dim() != 3 or t.shape[2] != self.head_dim or (heads is not None and t.shape[1] != heads) \
                or (rows is not None and t.shape[0] != rows):
            raise ValueError(f"{name} must be [{'rows' if rows is None else rows}]"
                             f"[{'heads' if heads is None else heads}][{self.head_dim}], not {list(t.shape)}")
        if t.dtype != self.pool.dtype or t.device != self.pool.device:
            raise ValueError(f"{name} must be {self.pool.dtype} on {self.pool.device}")
        if t.stride(2) != 1:
            raise ValueError(f"{name}: the last axis must be contiguous")
        return _KvRows(t.data_ptr(), t.stride(0), t.stride(1))

    def _batch(self, rows, seqs, row_start, max_rows):
        seqs = self._index("seqs", seqs)
        if row_start is not None:
            row_start = self._index("row_start", row_start, None if seqs is None else seqs.numel() + 1)
            n = row_start.numel() - 1
            if max_rows is None:
                raise ValueError("row_start needs max_rows, the largest number of rows of an entry")
        else:
            n = seqs.numel() if seqs is not None else min(rows, self.max_seqs)
        b = _KvBatch(n, rows, 0 if row_start is None else int(max_rows),
                     None if seqs is None else seqs.data_ptr(), None if row_start is None else row_start.data_ptr())
        return b, (seqs, row_start)

    def extend(self, n_new, stream=None) -> None:
        """Room for n_new[s] more tokens in every slot s; lens grow by them."""
        from . import _check, _stream, lib
        with self._at(stream):
            n_new = self._index("n_new", n_new, self.max_seqs)
            _check(lib().qgkv_extend(self._h, n_new.data_ptr(), _stream(stream)))

    def fork(self, src, dst, stream=None) -> None:
        """The empty slots dst become second names of the slots src."""
        from . import _check, _stream, lib
        with self._at(stream):
            src = self._index("src", src)
            dst = self._index("dst", dst, src.numel())
            _check(lib().qgkv_fork(self._h, src.data_ptr(), dst.data_ptr(), src.numel(), _stream(stream)))

    def trim(self, seqs, keep=None, stream=None) -> None:
        """Cut slots to their first ``keep`` tokens (default 0: free them)."""
        from . import _check, _stream, lib
        with self._at(stream):
            seqs = self._index("seqs", seqs)
            keep = self._index("keep", keep, seqs.numel())
            _check(lib().qgkv_trim(self._h, seqs.data_ptr(), None if keep is None else keep.data_ptr(), seqs.numel(),
                                   _stream(stream)))

    def compact(self, stream=None) -> None:
        """Move the live pages to the lowest ids."""
        from . import _check, _stream, lib
        with self._at(stream):
            _check(lib().qgkv_compact(self._h, _stream(stream)))

    def append(self, k, v, *, layer: int = 0, seqs=None, row_start=None, max_rows: int = None, stream=None) -> None:
        """Write the rows' keys and values, [rows][kv_heads][head_dim] each."""
        from . import _check, _stream, lib
        with self._at(stream):
            kr = self._rows("k", k, self.kv_heads)
            vr = self._rows("v", v, self.kv_heads, k.shape[0])
            b, _keep = self._batch(k.shape[0], seqs, row_start, max_rows)
            _check(lib().qgkv_append(self._h, int(layer), ctypes.byref(b), ctypes.byref(kr), ctypes.byref(vr),
                                     _stream(stream)))

    def attend(self, q, *, layer: int = 0, seqs=None, row_start=None, max_rows: int = None, scale: float = None,
               window: int = 0, sinks: int = 0, out=None, stream=None):
        """Attention of q [rows][q_heads][head_dim] over the cached tokens of one
        layer; returns out of the same shape.  scale: default head_dim ** -0.5.
        window: a row sees its last ``window`` tokens (0: all) and the first
        ``sinks`` of its slot."""
        import torch
        from . import _check, _stream, lib
        with self._at(stream):
            qr = self._rows("q", q)
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            o = self._rows("out", out, q.shape[1], q.shape[0])
            b, _keep = self._batch(q.shape[0], seqs, row_start, max_rows)
            sc = 1.0 / math.sqrt(self.head_dim) if scale is None else float(scale)
            _check(lib().qgkv_attend(self._h, int(layer), ctypes.byref(b), ctypes.byref(qr), ctypes.byref(o),
                                     q.shape[1], sc, int(window), int(sinks), _stream(stream)))
        return out

    def check(self) -> None:
        """Raise if a call found something to refuse on the device since the last
        check (waits for the GPU)."""
        from . import QGError, QG_ERR_INVALID_ARG, QG_ERR_OOM
        bits, short = self.info[:2].tolist()
        self.info[:2] = 0
        if bits & INFO_SHORT:
            raise QGError(QG_ERR_OOM, f"extend: {short} free pages short")
        if bits & INFO_LONG:
            raise QGError(QG_ERR_INVALID_ARG, f"extend: a slot longer than {self.max_pages * self.page_size} tokens")
        if bits & INFO_PAIR:
            raise QGError(QG_ERR_INVALID_ARG, "fork / trim: an entry was refused")

    def _at(self, stream):
        """Tensors made inside belong to the stream that the work runs on."""
        if self._h is None:
            raise ValueError("the cache is closed")
        return _on(stream)

    def close(self):
        if getattr(self, "_h", None) is not None:
            from . import lib
            lib().qgkv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _on(stream):
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)
