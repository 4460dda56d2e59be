"""What a decode step does with rows between its products (C ABI in ``include/qgstep.h``):
the norm with the residual's addition, rotary positions, and picking tokens.

Like the rest of the package this only marshals arguments; the work runs in the
library's HIP kernels on the current (or the given) stream of the operands' GPU.
"""
from __future__ import annotations

import ctypes
import math

__all__ = ["rms_norm", "Rotary", "sample", "sample_workspace"]

TYPE_F16, TYPE_BF16, TYPE_F32 = 0, 1, 2
CODES_SAME, CODES_INT8, CODES_E4M3 = 0, 1, 2
HALVES, PAIRS = 0, 1
MAX_NORM, MAX_VOCAB = 32768, 1 << 20

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class _Norm(ctypes.Structure):
    _fields_ = [("x", _vp), ("residual", _vp), ("weight", _vp), ("out", _vp), ("scales", _vp), ("x_stride", _i64),
                ("residual_stride", _i64), ("out_stride", _i64), ("rows", _i32), ("n", _i32), ("dtype", _i32),
                ("codes", _i32), ("group", _i32), ("eps", _f32)]


class _Rotary(ctypes.Structure):
    _fields_ = [("turns", _vp), ("dim", _i32), ("layout", _i32), ("size", _f32)]


class _Rows(ctypes.Structure):
    _fields_ = [("x", _vp), ("out", _vp), ("positions", _vp), ("x_row", _i64), ("x_head", _i64), ("out_row", _i64),
                ("out_head", _i64), ("rows", _i32), ("heads", _i32), ("head_dim", _i32), ("dtype", _i32)]


class _Sampling(ctypes.Structure):
    _fields_ = [("logits", _vp), ("stride", _i64), ("rows", _i32), ("vocab", _i32), ("dtype", _i32), ("u", _vp),
                ("temperature", _vp), ("top_k", _vp), ("top_p", _vp), ("min_p", _vp), ("temperature1", _f32),
                ("top_k1", _i32), ("top_p1", _f32), ("min_p1", _f32), ("tokens", _vp), ("probs", _vp)]


def bind(L) -> None:
    """Argument and result types of the qgs_* functions."""
    P = ctypes.POINTER
    L.qgs_rms_norm.argtypes = [P(_Norm), _vp]
    L.qgs_rotate.argtypes = [P(_Rows), P(_Rotary), _vp]
    L.qgs_sample_workspace.argtypes = [_i32, _i32, P(ctypes.c_size_t)]
    L.qgs_sample.argtypes = [P(_Sampling), _vp, ctypes.c_size_t, _vp]
    for f in ("rms_norm", "rotate", "sample_workspace", "sample"):
        getattr(L, "qgs_" + f).restype = ctypes.c_int


_state = None


def _lib():
    """torch, the library's functions and the check of their status: looked up once."""
    global _state
    if _state is None:
        import torch
        from . import _check, lib
        _state = (torch, lib(), _check, {torch.float16: TYPE_F16, torch.bfloat16: TYPE_BF16},
                  getattr(torch._C, "_cuda_getCurrentRawStream", None),
                  getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device))
    return _state


def _call(fn, dev, stream, *args) -> None:
    """One call on a GPU's stream, with that GPU the current one."""
    torch, _, check, _, raw, current = _state
    if stream is not None:
        st = stream.cuda_stream
    elif raw is not None:
        st = raw(dev)
    else:
        st = torch.cuda.current_stream(dev).cuda_stream
    if current() == dev:
        status = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, st)
    if status:
        check(status)


def _empty(shape, dtype, like, stream):
    """Memory that belongs to the stream the work runs on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _state[0].cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _count(name, n) -> None:
    if n > 2 ** 31 - 1:
        raise ValueError(f"{name}: {n} in one call")


def _matrix(name, t, shape, dtype, dev) -> int:
    """The row stride of [rows][n]."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} {list(shape)} on GPU {dev}, not {t.dtype} {list(t.shape)} on {t.device}")
    row, col = t.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return row


def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, quant=None, group: int = 0, out=None, scales=None,
             stream=None):
    """y = h * weight / sqrt(mean(h^2) + eps) of each row of x [rows][n] (fp16 or bf16), with h = x, or with
    ``residual`` h = x + residual, which is stored there (rounded once; the norm is of what is stored).

    quant: torch.int8 or torch.float8_e4m3fn for an output in 8 bits: returns (codes, scales) with y = codes * scale,
    one fp32 scale for each ``group`` elements of a row (32, 64 or 128; 0: the row), max |y| / 127 or / 448.
    ``out`` (and ``scales``, contiguous [rows][groups]) may be given; out may be x.
    """
    torch, L, _, types, *_ = _lib()
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    if len(shape) != 2 or dtype not in types or dev < 0:
        raise ValueError(f"x must be float16 or bfloat16 [rows][n] on a GPU, not {dtype} {list(shape)} on {x.device}")
    rows, n = shape
    _count("rows", rows)
    w = r = s = None
    r_stride = codes = 0
    if weight is not None:
        if weight.shape != (n,) or weight.dtype != dtype or weight.get_device() != dev or not weight.is_contiguous():
            raise ValueError(f"weight must be contiguous {dtype} [{n}] on {x.device}")
        w = weight.data_ptr()
    if residual is not None:
        r_stride = _matrix("residual", residual, shape, dtype, dev)
        r = residual.data_ptr()
    if quant is None:
        kind = dtype
        if scales is not None:
            raise ValueError("scales are an output of quant")
    elif quant in (torch.int8, torch.float8_e4m3fn):
        kind = quant
        codes = CODES_INT8 if quant == torch.int8 else CODES_E4M3
        per = -(-n // group) if group > 0 else 1
        if scales is None:
            scales = _empty((rows, per), torch.float32, x, stream)
        elif scales.shape != (rows, per) or scales.dtype != torch.float32 or scales.get_device() != dev or not scales.is_contiguous():
            raise ValueError(f"scales must be contiguous float32 [{rows}][{per}] on {x.device}")
        s = scales.data_ptr()
    else:
        raise ValueError(f"quant must be None, torch.int8 or torch.float8_e4m3fn, not {quant}")
    x_stride = _matrix("x", x, shape, dtype, dev)
    if out is None:
        out, out_stride = _empty(shape, kind, x, stream), n
    else:
        out_stride = _matrix("out", out, shape, kind, dev)
    d = _Norm(x.data_ptr(), r, w, out.data_ptr(), s, x_stride, r_stride, out_stride, rows, n, types[dtype], codes, group, eps)
    _call(L.qgs_rms_norm, dev, stream, ctypes.byref(d))
    return out if quant is None else (out, scales)


class Rotary:
    """Rotary positions of a model: the frequencies of the pairs of a head's first ``dim`` elements, on one GPU.

    interleaved: pair j is elements 2 j and 2 j + 1 (else j and j + dim / 2).  Its frequency is base ** (-2 j / dim)
    radians per position; scaling changes it for contexts ``factor`` times as long as trained:
      "linear"  all divided by factor
      "ntk"     base * factor ** (dim / (dim - 2)): the fastest pair stays, the slowest is divided by factor
      "yarn"    pairs that turn more than ``fast`` times within ``original`` positions stay, those that turn fewer than
                ``slow`` times are divided by factor, linearly in j between; rotated values times 0.1 ln(factor) + 1
    ``freqs`` (64-bit floats, radians per position) and ``size`` (the factor on rotated values) are attributes;
    Rotary.of(freqs, ...) takes any others.  Positions are exact: the angle of a far one is as good as a near one's.
    """

    def __init__(self, dim: int, base: float = 10000.0, *, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, original: int = 4096, fast: float = 32.0, slow: float = 1.0, device=None):
        if dim < 16 or dim % 16:
            raise ValueError(f"dim = {dim} is not a positive multiple of 16")
        if not (math.isfinite(base) and base > 1.0) or not (math.isfinite(factor) and factor > 0.0):
            raise ValueError(f"base = {base} must be above 1 and factor = {factor} positive")
        size = 1.0
        if scaling == "ntk":
            base = base * factor ** (dim / (dim - 2))
        freqs = [base ** (-2 * j / dim) for j in range(dim // 2)]
        if scaling == "linear":
            freqs = [f / factor for f in freqs]
        elif scaling == "yarn":
            if original < 1 or not fast > slow > 0:
                raise ValueError(f"yarn: original = {original} must be positive, and fast = {fast} above slow = {slow} above 0")
            def pair(turns):  # the pair that turns so often within the original context
                return dim * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), dim - 1)
            for j, f in enumerate(freqs):
                s = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
                freqs[j] = f * (1 - s) + f / factor * s
            size = 0.1 * math.log(factor) + 1
        elif scaling not in ("none", "ntk"):
            raise ValueError(f'scaling = {scaling!r} is not "none", "linear", "ntk" or "yarn"')
        self._open(freqs, size, interleaved, device)

    @classmethod
    def of(cls, freqs, *, size: float = 1.0, interleaved: bool = False, device=None) -> "Rotary":
        """Any frequencies, radians per position, one for each pair."""
        self = cls.__new__(cls)
        freqs = [float(f) for f in freqs]
        if not freqs or len(freqs) % 8 or not all(map(math.isfinite, freqs)):
            raise ValueError("freqs must be finite, a positive multiple of 8 of them")
        self._open(freqs, float(size), interleaved, device)
        return self

    def _open(self, freqs, size, interleaved, device):
        import torch
        if not math.isfinite(size):
            raise ValueError(f"size = {size} is not finite")
        self.freqs, self.size, self.interleaved, self.dim = freqs, size, bool(interleaved), 2 * len(freqs)
        words = []
        for f in freqs:  # turns per position, as a 64-bit fraction of one turn (what is whole turns no matter)
            t = f / (2 * math.pi)
            w = int(round(math.ldexp(t - math.floor(t), 64))) & (2 ** 64 - 1)
            words.append(w - 2 ** 64 if w >= 2 ** 63 else w)
        self.turns = torch.tensor(words, dtype=torch.int64).to(torch.device("cuda") if device is None else device)
        self._c = _Rotary(self.turns.data_ptr(), self.dim, PAIRS if interleaved else HALVES, size)
        self._ref = ctypes.byref(self._c)

    def rotate(self, x, positions, out=None, stream=None):
        """x [rows][heads][head_dim] (fp16 or bf16) with row i turned to positions[i] (int32, on x's GPU); elements
        from ``dim`` on are copied.  Returns out, which may be x."""
        torch, L, _, types, *_ = _lib()
        if x.dim() != 3 or x.dtype not in types or not x.is_cuda:
            raise ValueError(f"x must be float16 or bfloat16 [rows][heads][head_dim] on a GPU, not {x.dtype} {list(x.shape)} on {x.device}")
        rows, heads, d = x.shape
        _count("rows", rows)
        dev = x.get_device()
        if self.turns.get_device() != dev:
            raise ValueError(f"the frequencies are on {self.turns.device}, x on {x.device}")
        if positions.shape != (rows,) or positions.dtype != torch.int32 or positions.get_device() != dev or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous int32 [{rows}] on {x.device}")
        if out is None:
            out = _empty(x.shape, x.dtype, x, stream)
        elif out.shape != x.shape or out.dtype != x.dtype or out.get_device() != dev:
            raise ValueError(f"out must be {x.dtype} {list(x.shape)} on {x.device}")
        xs, os = x.stride(), out.stride()
        if (xs[2] != 1 or os[2] != 1) and d > 1:
            raise ValueError("the last axis must be contiguous")
        a = _Rows(x.data_ptr(), out.data_ptr(), positions.data_ptr(), xs[0], xs[1], os[0], os[1], rows, heads, d, types[x.dtype])
        _call(L.qgs_rotate, dev, stream, ctypes.byref(a), self._ref)
        return out


def sample(logits, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, probs: bool = False, out=None, workspace=None,
           stream=None):
    """A token of each row of logits [rows][vocab] (fp16, bf16 or fp32), picked by the uniform numbers u (fp32 [rows],
    in [0, 1)); int32 [rows], and with ``probs`` also its probability among the kept tokens (fp32 [rows]).

    temperature, top_k, top_p and min_p are numbers for all rows or tensors of one for each (fp32, top_k int32):
    of the tokens in falling order of their logits, equal ones by index, the first top_k are kept (0: all), of these the
    fewest first ones with top_p of their mass (1: all), of these those of at least min_p of the largest's
    probability (0: all); temperature 0 takes the first.  The token is the first, by index, up to which the kept
    tokens' mass passes u times all of it.  NaN counts as -inf; a row of -inf alone gives -1.
    workspace: a uint8 tensor of at least sample_workspace(rows, vocab) bytes (default: made here).
    """
    torch, L, _, types, *_ = _lib()
    kind = types.get(logits.dtype, TYPE_F32 if logits.dtype == torch.float32 else None)
    if logits.dim() != 2 or kind is None or not logits.is_cuda:
        raise ValueError(f"logits must be float16, bfloat16 or float32 [rows][vocab] on a GPU, not {logits.dtype} "
                         f"{list(logits.shape)} on {logits.device}")
    rows, vocab = logits.shape
    _count("rows", rows)
    dev = logits.get_device()
    d = _Sampling()
    d.stride = _matrix("logits", logits, logits.shape, logits.dtype, dev)
    d.logits, d.rows, d.vocab, d.dtype = logits.data_ptr(), rows, vocab, kind

    def each(name, t, dtype):
        if t.shape != (rows,) or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dtype} [{rows}] on {logits.device}")
        return t.data_ptr()

    d.u = each("u", u, torch.float32)
    for name, value, dtype in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                               ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if isinstance(value, torch.Tensor):
            setattr(d, name, each(name, value, dtype))
        else:
            setattr(d, name + "1", min(max(value, 0), 2 ** 31 - 1) if name == "top_k" else value)
    if out is None:
        out = _empty((rows,), torch.int32, logits, stream)
    d.tokens = each("out", out, torch.int32)
    prob = None
    if probs:
        prob = _empty((rows,), torch.float32, logits, stream)
        d.probs = prob.data_ptr()
    if workspace is None:
        workspace = _empty((sample_workspace(rows, vocab),), torch.uint8, logits, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {logits.device}")
    _call(L.qgs_sample, dev, stream, ctypes.byref(d), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return (out, prob) if probs else out


_sizes = {}


def sample_workspace(rows: int, vocab: int) -> int:
    """Bytes of workspace that sample takes for so many rows and tokens."""
    got = _sizes.get((rows, vocab))
    if got is None:
        _, L, check, *_ = _lib()
        n = ctypes.c_size_t()
        check(L.qgs_sample_workspace(rows, vocab, ctypes.byref(n)))
        if len(_sizes) > 256:
            _sizes.clear()
        got = _sizes[rows, vocab] = int(n.value)
    return got
