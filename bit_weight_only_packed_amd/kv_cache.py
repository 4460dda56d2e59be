"""Paged key-value cache and the attention over it (C ABI in ``include/qgkv.h``).

Like the rest of the package this only marshals arguments: the cache's tensors
are PyTorch tensors, every step of the work runs in the library's HIP kernels on
the current (or the given) stream, and nothing is copied to the host.
"""
from __future__ import annotations

import contextlib
import ctypes

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
    L.qgkv_append_rotary.argtypes = [vp, i32, ctypes.POINTER(_KvBatch)] + [ctypes.POINTER(_KvRows)] * 4 + [i32, vp, vp]
    L.qgkv_attend.argtypes = [vp, i32, ctypes.POINTER(_KvBatch), ctypes.POINTER(_KvRows), ctypes.POINTER(_KvRows), i32,
                              ctypes.c_float, i32, i32, vp]
    L.qgkv_attend_shared.argtypes = L.qgkv_attend.argtypes[:-1] + [vp, i32, ctypes.c_int64, vp]
    for f in ("create", "destroy", "extend", "fork", "trim", "compact", "append", "append_rotary", "attend",
              "attend_shared"):
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

    (with rotary positions q = kv.append_rotated(q, k, v, rotary, layer=layer), and
    kv.attend_shared where slots are long forks of one another).

    Rows of a call: ``seqs`` (int32 [n], default slots 0 .. n - 1) names the
    slots; with ``row_start`` (int32 [n + 1], with ``max_rows`` at least the
    largest count) entry j has rows row_start[j] .. row_start[j + 1] - 1, without
    it each has the same number.  They are the last tokens of their slots.
    With neither, n is the smaller of the number of rows and ``max_seqs``: up to
    ``max_seqs`` rows are one new token each of slots 0, 1, ..., more of them are
    rows / max_seqs each of all slots.  So the rows of one slot of several need
    ``seqs=[slot]``.
    Index tensors may also be given as lists (copied to the device).  Calls run on
    the cache's GPU, whichever is the current one.
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
        # what a call needs besides its tensors, made once: the bound functions, the
        # argument blocks (calls on one cache are ordered by the caller), the device
        L = lib()
        self._c = {n: getattr(L, "qgkv_" + n) for n in ("extend", "fork", "trim", "compact", "append", "append_rotary",
                                                         "attend", "attend_shared")}
        self._check = _check
        self._torch = torch
        self._dev = pool.get_device()
        self._dtype = pool.dtype
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._args = (_KvBatch(), _KvRows(), _KvRows())
        self._more = (_KvRows(), _KvRows())
        self._refs = tuple(ctypes.byref(x) for x in self._args)
        self._more_refs = tuple(ctypes.byref(x) for x in self._more)

    @property
    def handle(self):
        return self._h

    def _on(self, stream) -> int:
        """The stream of a call: the given one or the current one of the cache's GPU."""
        if self._h is None:
            raise ValueError("the cache is closed")
        if stream is not None:
            return stream.cuda_stream
        if self._raw_stream is not None:
            return self._raw_stream(self._dev)
        return self._torch.cuda.current_stream(self._dev).cuda_stream

    def _call(self, name, *args) -> None:
        st = self._c[name](self._h, *args)
        if st:
            # the library refuses, before all else, a cache that is not on the current GPU
            cuda = self._torch.cuda
            if cuda.current_device() != self._dev:
                with cuda.device(self._dev):
                    st = self._c[name](self._h, *args)
            self._check(st)

    def _index(self, name, x, n=None, stream=None):
        """An int32 tensor on the cache's GPU (lists are copied there)."""
        torch = self._torch
        if not isinstance(x, torch.Tensor):
            with _on(stream):  # memory made here belongs to the stream that uses it
                x = torch.tensor(list(x), dtype=torch.int32, device=self.pool.device)
        if x.dtype != torch.int32 or x.dim() != 1 or x.get_device() != self._dev or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 1-d int32 tensor on {self.pool.device}")
        if n is not None and x.numel() != n:
            raise ValueError(f"{name} has {x.numel()} entries, not {n}")
        return x

    def _rows(self, into: _KvRows, name, t, heads=None, rows=None) -> tuple:
        """Fill an argument block; the operand's (rows, heads)."""
        size = t.shape
        if len(size) != 3 or size[2] != self.head_dim or (heads is not None and size[1] != heads) \
                or (rows is not None and size[0] != rows):
            raise ValueError(f"{name} must be [{'rows' if rows is None else rows}]"
                             f"[{'heads' if heads is None else heads}][{self.head_dim}], not {list(size)}")
        if t.dtype != self._dtype or t.get_device() != self._dev:
            raise ValueError(f"{name} must be {self._dtype} on {self.pool.device}")
        into.row_stride, into.head_stride, last = t.stride()
        if last != 1:
            raise ValueError(f"{name}: the last axis must be contiguous")
        into.ptr = t.data_ptr()
        return size[0], size[1]

    def _batch(self, rows, seqs, row_start, max_rows, stream):
        """Fill the call's batch; the index tensors, which the caller holds until the call is made."""
        b = self._args[0]
        b.rows = rows
        n = None
        if seqs is not None:
            seqs = self._index("seqs", seqs, None, stream)
            n = seqs.numel()
        if row_start is not None:
            row_start = self._index("row_start", row_start, None if n is None else n + 1, stream)
            if max_rows is None:
                raise ValueError("row_start needs max_rows, the largest number of rows of an entry")
            n = row_start.numel() - 1
            b.max_rows, b.row_start = int(max_rows), row_start.data_ptr()
        else:
            n = min(rows, self.max_seqs) if n is None else n
            b.max_rows, b.row_start = 0, None
        b.n = n
        b.seqs = None if seqs is None else seqs.data_ptr()
        return seqs, row_start

    def extend(self, n_new, stream=None) -> None:
        """Room for n_new[s] more tokens in every slot s; lens grow by them.  Refused
        on the device if pages are short or a slot would be too long: then nothing
        changes, and appends write nothing until an extend is granted or ``check``
        has been called."""
        st = self._on(stream)
        n_new = self._index("n_new", n_new, self.max_seqs, stream)
        self._call("extend", n_new.data_ptr(), st)

    def fork(self, src, dst, stream=None) -> None:
        """The empty slots dst become second names of the slots src."""
        st = self._on(stream)
        src = self._index("src", src, None, stream)
        dst = self._index("dst", dst, src.numel(), stream)
        self._call("fork", src.data_ptr(), dst.data_ptr(), src.numel(), st)

    def trim(self, seqs, keep=None, stream=None) -> None:
        """Cut slots to their first ``keep`` tokens (default 0: free them)."""
        st = self._on(stream)
        seqs = self._index("seqs", seqs, None, stream)
        if keep is not None:
            keep = self._index("keep", keep, seqs.numel(), stream)
        self._call("trim", seqs.data_ptr(), None if keep is None else keep.data_ptr(), seqs.numel(), st)

    def compact(self, stream=None) -> None:
        """Move the live pages to the lowest ids."""
        self._call("compact", self._on(stream))

    def append(self, k, v, *, layer: int = 0, seqs=None, row_start=None, max_rows: int = None, stream=None) -> None:
        """Write the rows' keys and values, [rows][kv_heads][head_dim] each.  Which
        slots: see the class; one slot takes one entry of a call."""
        st = self._on(stream)
        _, ka, va = self._args
        rows, _ = self._rows(ka, "k", k, self.kv_heads)
        self._rows(va, "v", v, self.kv_heads, rows)
        held = self._batch(rows, seqs, row_start, max_rows, stream)
        rb, rk, rv = self._refs
        self._call("append", layer, rb, rk, rv, st)
        del held

    def append_rotated(self, q, k, v, rotary, *, layer: int = 0, seqs=None, row_start=None, max_rows: int = None, out=None,
                       stream=None):
        """``append`` with rotary positions: each row's k is rotated to its position in its
        slot on its way into the page, and its q [rows][q_heads][head_dim] into out, which
        is returned (out may be q; q None: keys and values only).  rotary: a ``Rotary`` on
        the cache's GPU.  out of a row at a position before 0 (an idle slot's) is 0."""
        st = self._on(stream)
        (_, ka, va), (qa, oa) = self._args, self._more
        rows, _ = self._rows(ka, "k", k, self.kv_heads)
        self._rows(va, "v", v, self.kv_heads, rows)
        if rotary.turns.get_device() != self._dev:
            raise ValueError(f"the frequencies are on {rotary.turns.device}, the cache on {self.pool.device}")
        heads = 0
        if q is not None:
            _, heads = self._rows(qa, "q", q, None, rows)
            if out is None:
                with _on(stream):
                    out = self._torch.empty(q.shape, dtype=q.dtype, device=q.device)
            self._rows(oa, "out", out, heads, rows)
        elif out is not None:
            raise ValueError("out without q")
        held = self._batch(rows, seqs, row_start, max_rows, stream)
        (rb, rk, rv), (rq, ro) = self._refs, self._more_refs
        self._call("append_rotary", layer, rb, rk, rv, rq, ro, heads, rotary._ref, st)
        del held
        return out

    def attend(self, q, *, layer: int = 0, seqs=None, row_start=None, max_rows: int = None, scale: float = None,
               window: int = 0, sinks: int = 0, out=None, stream=None):
        """Attention of q [rows][q_heads][head_dim] over the cached tokens of one
        layer; returns out of the same shape.  scale: default head_dim ** -0.5.
        window: a row sees its last ``window`` tokens (0: all) and the first
        ``sinks`` of its slot.  Which slots the rows are of: see the class."""
        st = self._on(stream)
        _, qa, oa = self._args
        rows, heads = self._rows(qa, "q", q)
        if out is None:
            with _on(stream):
                out = self._torch.empty(q.shape, dtype=q.dtype, device=q.device)
        self._rows(oa, "out", out, heads, rows)
        held = self._batch(rows, seqs, row_start, max_rows, stream)
        rb, rq, ro = self._refs
        self._call("attend", layer, rb, rq, ro, heads, self.head_dim ** -0.5 if scale is None else scale, window, sinks, st)
        del held
        return out

    def attend_shared(self, q, *, groups=None, least: int = None, layer: int = 0, seqs=None, row_start=None,
                      max_rows: int = None, scale: float = None, window: int = 0, sinks: int = 0, out=None, stream=None):
        """``attend`` where entries share their first tokens (forked answers to a prompt): the
        pages that all entries of a group name alike are read once for all of them.
        groups: int32 [g + 1], the entries at which groups begin, and n (default: all
        entries are one group).  Nothing else need be told: the tables are looked at on
        the device.  least: bytes of shared tokens, counted for every entry that reads
        them, from which on it is done and not left to ``attend`` (default: where it was
        measured to pay; 0: always)."""
        if groups is None:
            more = (None, 1, -1 if least is None else least)
        else:
            groups = self._index("groups", groups, None, stream)
            if groups.numel() == 0:
                raise ValueError("groups is empty: it holds the entries at which groups begin, and n")
            more = (groups.data_ptr(), groups.numel() - 1, -1 if least is None else least)
        st = self._on(stream)
        _, qa, oa = self._args
        rows, heads = self._rows(qa, "q", q)
        if out is None:
            with _on(stream):
                out = self._torch.empty(q.shape, dtype=q.dtype, device=q.device)
        self._rows(oa, "out", out, heads, rows)
        held = self._batch(rows, seqs, row_start, max_rows, stream)
        rb, rq, ro = self._refs
        self._call("attend_shared", layer, rb, rq, ro, heads, self.head_dim ** -0.5 if scale is None else scale, window, sinks, *more, st)
        del held
        return out

    def check(self, stream=None) -> None:
        """Raise if a call found something to refuse on the device since the last
        check.  Waits for the given stream, or for all work on the cache's GPU, and
        returns after ``info`` has been cleared."""
        from . import QGError, QG_ERR_INVALID_ARG, QG_ERR_OOM
        cuda = self._torch.cuda
        with cuda.device(self._dev), _on(stream):
            (cuda.synchronize if stream is None else stream.synchronize)()
            bits, short = self.info[:2].tolist()
            if bits or short:
                self.info[:2] = 0
                cuda.current_stream().synchronize()
        if bits & INFO_SHORT:
            raise QGError(QG_ERR_OOM, f"extend: {short} free pages short")
        if bits & INFO_LONG:
            raise QGError(QG_ERR_INVALID_ARG, f"extend: a slot longer than {self.max_pages * self.page_size} tokens")
        if bits & INFO_PAIR:
            raise QGError(QG_ERR_INVALID_ARG, "fork / trim: an entry was refused")

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


_HERE = contextlib.nullcontext()


def _on(stream):
    """Tensors made inside belong to the stream that the work runs on."""
    if stream is None:
        return _HERE
    import torch
    return torch.cuda.stream(stream)
