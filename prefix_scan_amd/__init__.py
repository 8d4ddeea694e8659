"""Python binding of libscan, the MI355X (gfx950) prefix-scan library.

Argument marshalling only: every function here checks tensors, takes their
device pointers and the current HIP stream, and calls the C entry point of the
same name in ``libscan.so`` (declared in ``include/libscan.h``).  All
computation runs in the library's HIP kernels; there is no CPU fallback, and
a missing ``libscan.so`` raises.

PyTorch supplies device memory and streams.  Tensors must be on the current CUDA
(HIP) device, contiguous, with 4-byte elements (torch.int32 or torch.uint32), or
8-byte elements (torch.int64 or torch.uint64) for the *_u64 entry points.
Rows of linear attention, gated recurrences, embeddings and logits are float32,
bfloat16 or float16, with any strides whose last is 1; an output's rows may not
overlap one another.
"""
import ctypes
import functools
import os
import threading

import torch

__all__ = [
    "LibscanError", "lib", "version",
    "scan_exclusive_u32", "scan_inclusive_u32", "scan_u32_ex",
    "scan_op_u32", "reduce_op_u32", "scan_op_u64", "reduce_op_u64",
    "runs_layout_u32", "runs_slots_i32", "runs_owner_u32", "runs_owner_all_u32",
    "segscan_flags_u32",
    "linattn", "linattn_grad", "linattn_step", "sample_logits",
    "gatescan", "gatescan_grad", "gatescan_step",
    "embed_rows", "embed_grad", "penalize_logits",
    "segscan_u32", "compact_flags_u32", "radix_perm_u32", "copy_u32", "scan_u32_noalloc",
    "scan_scratch_bytes", "scan_ex_scratch_bytes", "segscan_scratch_bytes",
    "compact_scratch_bytes", "radix_scratch_bytes",
    "ALGO_AUTO", "ALGO_LOOKBACK", "ALGO_THREEPASS", "ALGO_LOOKBACK_TILE",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libscan.so")

OK = 0
ERR_NULL, ERR_SIZE, ERR_ARG, ERR_SCRATCH, ERR_HIP, ERR_ALIGN = -1, -2, -3, -4, -5, -6
ALGO_AUTO, ALGO_LOOKBACK, ALGO_THREEPASS, ALGO_LOOKBACK_TILE = 0, 1, 2, 3
_ALGOS = {"auto": ALGO_AUTO, "lookback": ALGO_LOOKBACK, "threepass": ALGO_THREEPASS,
          "lookback_tile": ALGO_LOOKBACK_TILE}


class LibscanError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, lib().libscan_strerror(status).decode(),
                                                         status))


LINATTN_MAX_WIDTH = 128
SAMPLE_MAX_VOCAB = 1 << 24
EMBED_MAX_ROWS = 0x7FFFFFFF
_CLEAR_REST = 0x100                     # LINATTN_CLEAR_REST
_FORMS = {"decay": 0, "log": 1, "sigmoid": 2}       # GATESCAN_*
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}     # LIBSCAN_F32 / BF16 / F16


class _Rows(ctypes.Structure):
    """linattn_rows_t"""
    _fields_ = [("data", ctypes.c_void_p), ("seq_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_uint32)]


class _Shape(ctypes.Structure):
    """linattn_shape_t"""
    _fields_ = [("dtype", ctypes.c_int), ("seqs", ctypes.c_uint32), ("heads", ctypes.c_uint32),
                ("key_width", ctypes.c_uint32), ("value_width", ctypes.c_uint32),
                ("tokens", ctypes.c_uint64), ("ends", ctypes.c_void_p),
                ("log_decay", ctypes.c_void_p), ("scale", ctypes.c_float)]


class _GateRows(ctypes.Structure):
    """gatescan_rows_t"""
    _fields_ = [("data", ctypes.c_void_p), ("seq_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class _GateShape(ctypes.Structure):
    """gatescan_shape_t"""
    _fields_ = [("dtype", ctypes.c_int), ("form", ctypes.c_int), ("blend", ctypes.c_int),
                ("clear_rest", ctypes.c_int), ("seqs", ctypes.c_uint32),
                ("tokens", ctypes.c_uint64), ("width", ctypes.c_uint64), ("ends", ctypes.c_void_p)]


class _Embed(ctypes.Structure):
    """embed_shape_t"""
    _fields_ = [("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("id_bytes", ctypes.c_int),
                ("tokens", ctypes.c_uint64), ("rows", ctypes.c_uint64), ("width", ctypes.c_uint64),
                ("scale", ctypes.c_float)]


class _List(ctypes.Structure):
    """penalty_list_t"""
    _fields_ = [("tokens", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("count", ctypes.c_uint64), ("ends", ctypes.c_void_p)]


class _Penalty(ctypes.Structure):
    """penalty_args_t"""
    _fields_ = [("dtype", ctypes.c_int), ("rows", ctypes.c_uint64), ("vocab", ctypes.c_uint64),
                ("logits", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64), ("past", _List),
                ("prompts", ctypes.c_void_p), ("repetition", ctypes.c_float),
                ("presence", ctypes.c_float), ("frequency", ctypes.c_float),
                ("repetitions", ctypes.c_void_p), ("presences", ctypes.c_void_p),
                ("frequencies", ctypes.c_void_p), ("bias", _List),
                ("bias_values", ctypes.c_void_p), ("bias_stride", ctypes.c_int64),
                ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64),
                ("masks", ctypes.c_uint64), ("mask_slots", ctypes.c_void_p)]


class _Sample(ctypes.Structure):
    """sample_args_t"""
    _fields_ = [("dtype", ctypes.c_int), ("rows", ctypes.c_uint64), ("vocab", ctypes.c_uint64),
                ("logits", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("u", ctypes.c_void_p), ("temperature", ctypes.c_float),
                ("top_p", ctypes.c_float), ("min_p", ctypes.c_float), ("top_k", ctypes.c_int32),
                ("temperatures", ctypes.c_void_p), ("top_ps", ctypes.c_void_p),
                ("min_ps", ctypes.c_void_p), ("top_ks", ctypes.c_void_p),
                ("tokens", ctypes.c_void_p), ("logprobs", ctypes.c_void_p),
                ("kept", ctypes.c_void_p)]


_lib = None
_lib_lock = threading.Lock()


def lib():
    """The loaded libscan.so (ctypes.CDLL) with argument types declared."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libscan.so is not built (%s); run `python -m prefix_scan_amd.build`"
                               % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, u64, i32, sz = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int, ctypes.c_size_t
        u32p = ctypes.POINTER(ctypes.c_uint32)
        L.libscan_strerror.argtypes = [i32]
        L.libscan_strerror.restype = ctypes.c_char_p
        L.libscan_version.argtypes = []
        L.libscan_version.restype = ctypes.c_char_p
        L.libscan_scratch_init.argtypes = [vp, sz, vp]
        L.libscan_scratch_init.restype = i32
        L.libscan_scratch_captured.argtypes = [vp, sz]
        L.libscan_scratch_captured.restype = i32
        L.scan_scratch_bytes.argtypes = [u64]
        L.scan_scratch_bytes.restype = sz
        L.scan_ex_scratch_bytes.argtypes = [u64, i32, i32]
        L.scan_ex_scratch_bytes.restype = sz
        for name in ("scan_exclusive_u32", "scan_inclusive_u32"):
            f = getattr(L, name)
            f.argtypes = [vp, u64, u32p, vp, vp, sz, vp]
            f.restype = i32
        L.scan_u32_ex.argtypes = [vp, u64, i32, i32, i32, u32p, vp, vp, sz, vp]
        L.scan_u32_ex.restype = i32
        L.scan_op_u32.argtypes = [vp, u64, i32, i32, u32p, vp, vp, sz, vp]
        L.scan_op_u32.restype = i32
        L.reduce_scratch_bytes.argtypes = [u64]
        L.reduce_scratch_bytes.restype = sz
        L.reduce_op_u32.argtypes = [vp, u64, i32, u32p, vp, vp, sz, vp]
        L.reduce_op_u32.restype = i32
        u64p = ctypes.POINTER(ctypes.c_uint64)
        L.scan_op_u64_scratch_bytes.argtypes = [u64]
        L.scan_op_u64_scratch_bytes.restype = sz
        L.scan_op_u64.argtypes = [vp, u64, i32, i32, u64p, vp, vp, sz, vp]
        L.scan_op_u64.restype = i32
        L.reduce_op_u64.argtypes = [vp, u64, i32, u64p, vp, vp, sz, vp]
        L.reduce_op_u64.restype = i32
        L.segscan_flags_scratch_bytes.argtypes = [u64]
        L.segscan_flags_scratch_bytes.restype = sz
        L.segscan_flags_u32.argtypes = [vp, vp, vp, u64, vp, u32p, vp, vp, sz, vp]
        L.segscan_flags_u32.restype = i32
        L.runs_scratch_bytes.argtypes = [u64, u64]
        L.runs_scratch_bytes.restype = sz
        L.runs_layout_u32.argtypes = [vp, vp, u64, u32p, vp, vp, sz, vp]
        L.runs_layout_u32.restype = i32
        L.runs_slots_i32.argtypes = [vp, u64, vp]
        L.runs_slots_i32.restype = i32
        L.runs_owner_u32.argtypes = [vp, u64, vp, u64, vp, vp, sz, vp]
        L.runs_owner_u32.restype = i32
        L.runs_owner_all_u32.argtypes = [vp, u64, vp, u64, vp, sz, vp]
        L.runs_owner_all_u32.restype = i32
        L.segscan_scratch_bytes.argtypes = [u64, u64]
        L.segscan_scratch_bytes.restype = sz
        L.segscan_u32.argtypes = [vp, vp, u64, u64, vp, vp, sz, vp]
        L.segscan_u32.restype = i32
        L.compact_scratch_bytes.argtypes = [u64]
        L.compact_scratch_bytes.restype = sz
        L.compact_flags_u32.argtypes = [vp, vp, u64, u32p, vp, vp, sz, vp]
        L.compact_flags_u32.restype = i32
        L.radix_scratch_bytes.argtypes = [u64, i32]
        L.radix_scratch_bytes.restype = sz
        L.radix_perm_u32.argtypes = [vp, vp, u64, i32, vp, sz, vp]
        L.radix_perm_u32.restype = i32
        L.copy_scratch_bytes.argtypes = [u64]
        L.copy_scratch_bytes.restype = sz
        L.copy_u32.argtypes = [vp, vp, u64, vp, sz, vp]
        L.copy_u32.restype = i32
        L.scan_u32_noalloc.argtypes = [vp, u64, i32, vp, vp]
        L.scan_u32_noalloc.restype = i32
        shape, rows = ctypes.POINTER(_Shape), ctypes.POINTER(_Rows)
        L.linattn_scratch_bytes.argtypes = [shape]
        L.linattn_scratch_bytes.restype = sz
        L.linattn.argtypes = [shape, rows, rows, rows, vp, rows, vp, vp, sz, vp]
        L.linattn.restype = i32
        L.linattn_grad_scratch_bytes.argtypes = [shape] + [ctypes.c_uint32] * 3
        L.linattn_grad_scratch_bytes.restype = sz
        L.linattn_grad.argtypes = ([shape] + [rows] * 4 + [vp, vp] + [rows] * 3 +
                                   [vp, vp, sz, vp])
        L.linattn_grad.restype = i32
        L.linattn_step.argtypes = [shape, rows, rows, rows, vp, u64, vp, rows, vp, vp]
        L.linattn_step.restype = i32
        gshape, grows = ctypes.POINTER(_GateShape), ctypes.POINTER(_GateRows)
        L.gatescan_scratch_bytes.argtypes = [gshape, i32]
        L.gatescan_scratch_bytes.restype = sz
        L.gatescan.argtypes = [gshape, grows, grows, vp, grows, vp, vp, sz, vp]
        L.gatescan.restype = i32
        L.gatescan_grad.argtypes = [gshape] + [grows] * 4 + [vp, vp, grows, grows, vp, vp, sz, vp]
        L.gatescan_grad.restype = i32
        L.gatescan_step.argtypes = [gshape, grows, grows, vp, u64, vp, grows, vp, vp]
        L.gatescan_step.restype = i32
        eshape, i64 = ctypes.POINTER(_Embed), ctypes.c_int64
        L.embed_rows.argtypes = [eshape, vp, i64, vp, vp, i64, vp]
        L.embed_rows.restype = i32
        L.embed_grad_scratch_bytes.argtypes = [eshape]
        L.embed_grad_scratch_bytes.restype = sz
        L.embed_grad.argtypes = [eshape, vp, i64, vp, vp, i64, i32, vp, sz, vp]
        L.embed_grad.restype = i32
        L.penalize_logits.argtypes = [ctypes.POINTER(_Penalty), vp]
        L.penalize_logits.restype = i32
        L.sample_scratch_bytes.argtypes = [u64, u64]
        L.sample_scratch_bytes.restype = sz
        L.sample_logits.argtypes = [ctypes.POINTER(_Sample), vp, sz, vp]
        L.sample_logits.restype = i32
        _lib = L
    return _lib


def version():
    return lib().libscan_version().decode()


def _check(status, what):
    if status != OK:
        raise LibscanError(status, what)


def _dev_u32(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on a GPU device, got %s" % (name, t.device))
    if t.dtype not in (torch.int32, torch.uint32):
        raise TypeError("%s must be int32 or uint32, got %s" % (name, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _dev_u64(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on a GPU device, got %s" % (name, t.device))
    if t.dtype not in (torch.int64, torch.uint64):
        raise TypeError("%s must be int64 or uint64, got %s" % (name, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _stream_handle(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream), s


def _new(shape, dtype, device, stream, zeros=False):
    """A tensor of the memory of the stream that will write it (None: the current one)."""
    make = torch.zeros if zeros else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


# --------------------------------------------------------------------------
# Scratch: one zero-initialised buffer per (device, stream), grown on demand.
# The library keeps a buffer consistent between calls by itself, so a buffer
# is initialised only when it is created.  A call is a chain of kernels through
# its buffer, and host threads may share a stream: each call holds the buffer
# (`with`) until all of its kernels are enqueued, so that chains follow one
# another on the stream and never mix.
# --------------------------------------------------------------------------
_scratch = {}
_outgrown = []          # kept: buffers that a captured graph may hold
_DOUBLED = 1 << 28      # larger buffers grow to the need, smaller ones to twice their size


class _Scratch:
    """A stream's buffer; its lock is taken by _scratch_at and given back as the `with` ends."""
    __slots__ = ("buf", "lock")

    def __init__(self):
        self.buf, self.lock = None, threading.Lock()

    def __enter__(self):
        return self.buf

    def __exit__(self, *exc):
        self.lock.release()

    def grow(self, device, stream_obj, nbytes):
        size = max(nbytes, 1 << 16)
        if self.buf is not None:
            if size < _DOUBLED:
                size = max(size, 2 * self.buf.numel())
            if lib().libscan_scratch_captured(_ptr(self.buf), self.buf.numel()):
                _outgrown.append(self.buf)
            # The work that is under way in it is ahead, on the stream that it
            # goes back to.
            self.buf = None
        with torch.cuda.stream(stream_obj):
            buf = torch.empty(size, dtype=torch.uint8, device=device)
        _check(lib().libscan_scratch_init(ctypes.c_void_p(buf.data_ptr()), size,
                                          ctypes.c_void_p(stream_obj.cuda_stream)),
               "libscan_scratch_init")
        self.buf = buf


# The current stream's handle, by the short way where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _scratch_at(device, index, handle, stream, nbytes):
    """The buffer of a stream (by its handle) of at least nbytes, held: for a `with`."""
    held = _scratch.get((index, handle))
    if held is None:
        held = _scratch.setdefault((index, handle), _Scratch())
    held.lock.acquire()
    try:
        if held.buf is None or held.buf.numel() < nbytes:
            held.grow(device, stream or torch.cuda.current_stream(device), nbytes)
    except BaseException:
        held.lock.release()
        raise
    return held


def _scratch_for(device, stream_obj, nbytes):
    return _scratch_at(device, device.index, stream_obj.cuda_stream, stream_obj, nbytes)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _total_args(want_total, total_dev):
    host = ctypes.c_uint32(0)
    hp = ctypes.pointer(host) if want_total else ctypes.POINTER(ctypes.c_uint32)()
    if total_dev is not None:
        _dev_u32(total_dev, "total_dev")
    return host, hp


# --------------------------------------------------------------------------
# Entry points
# --------------------------------------------------------------------------

def scan_scratch_bytes(n):
    return lib().scan_scratch_bytes(n)


def scan_ex_scratch_bytes(n, algo=ALGO_AUTO, fork_depth=-1):
    return lib().scan_ex_scratch_bytes(n, _algo(algo), fork_depth)


def _algo(algo):
    return _ALGOS[algo] if isinstance(algo, str) else int(algo)


def scan_u32_ex(data, inclusive=False, algo="auto", fork_depth=-1, want_total=True,
                total_dev=None, stream=None):
    """In-place scan of `data` by the chosen algorithm; returns the total
    (an int, after waiting for the stream) when want_total, else None."""
    _dev_u32(data, "data")
    a = _algo(algo)
    sh, s = _stream_handle(data.device, stream)
    need = lib().scan_ex_scratch_bytes(data.numel(), a, fork_depth)
    with _scratch_for(data.device, s, need) as scr:
        host, hp = _total_args(want_total, total_dev)
        _check(lib().scan_u32_ex(_ptr(data), data.numel(), 1 if inclusive else 0, a, fork_depth, hp,
                                 _ptr(total_dev), _ptr(scr), scr.numel(), sh), "scan_u32_ex")
    return int(host.value) if want_total else None


def _scan(name, data, want_total, total_dev, stream):
    _dev_u32(data, "data")
    sh, s = _stream_handle(data.device, stream)
    with _scratch_for(data.device, s, lib().scan_scratch_bytes(data.numel())) as scr:
        host, hp = _total_args(want_total, total_dev)
        _check(getattr(lib(), name)(_ptr(data), data.numel(), hp, _ptr(total_dev), _ptr(scr),
                                    scr.numel(), sh), name)
    return int(host.value) if want_total else None


# LIBSCAN_OP_* of libscan.h.
OPS = {"add": 0, "mul": 1, "and": 2, "or": 3, "xor": 4, "min": 5, "max": 6, "min_s": 7,
       "max_s": 8}


def _op(op):
    if op not in OPS:
        raise ValueError("op must be one of %s, got %r" % (sorted(OPS), op))
    return OPS[op]


def scan_op_u32(data, op, inclusive=False, want_total=True, total_dev=None, stream=None):
    """In-place scan of `data` under the operator named `op` ("add", "mul",
    "and", "or", "xor", "min", "max", or "min_s" / "max_s" comparing as
    signed); returns the fold of all values (an int, after waiting for the
    stream) when want_total, else None."""
    _dev_u32(data, "data")
    o = _op(op)
    sh, s = _stream_handle(data.device, stream)
    with _scratch_for(data.device, s, lib().scan_scratch_bytes(data.numel())) as scr:
        host, hp = _total_args(want_total, total_dev)
        _check(lib().scan_op_u32(_ptr(data), data.numel(), o, 1 if inclusive else 0, hp,
                                 _ptr(total_dev), _ptr(scr), scr.numel(), sh), "scan_op_u32")
    return int(host.value) if want_total else None


def reduce_op_u32(data, op, want_total=True, total_dev=None, stream=None):
    """The fold of `data` under the operator named `op` (data is only read);
    returns it as an int when want_total, else leaves it in total_dev."""
    _dev_u32(data, "data")
    o = _op(op)
    sh, s = _stream_handle(data.device, stream)
    with _scratch_for(data.device, s, lib().reduce_scratch_bytes(data.numel())) as scr:
        host, hp = _total_args(want_total, total_dev)
        _check(lib().reduce_op_u32(_ptr(data), data.numel(), o, hp, _ptr(total_dev), _ptr(scr),
                                   scr.numel(), sh), "reduce_op_u32")
    return int(host.value) if want_total else None


def _total64_args(want_total, total_dev):
    host = ctypes.c_uint64(0)
    hp = ctypes.pointer(host) if want_total else ctypes.POINTER(ctypes.c_uint64)()
    if total_dev is not None:
        _dev_u64(total_dev, "total_dev")
    return host, hp


def scan_op_u64(data, op, inclusive=False, want_total=True, total_dev=None, stream=None):
    """In-place scan of the 64-bit tensor `data` (int64 or uint64, taken as
    unsigned) under `op`, mod 2^64; returns the fold of all values as an int
    in [0, 2^64) when want_total, else None."""
    _dev_u64(data, "data")
    o = _op(op)
    sh, s = _stream_handle(data.device, stream)
    with _scratch_for(data.device, s, lib().scan_op_u64_scratch_bytes(data.numel())) as scr:
        host, hp = _total64_args(want_total, total_dev)
        _check(lib().scan_op_u64(_ptr(data), data.numel(), o, 1 if inclusive else 0, hp,
                                 _ptr(total_dev), _ptr(scr), scr.numel(), sh), "scan_op_u64")
    return int(host.value) if want_total else None


def reduce_op_u64(data, op, want_total=True, total_dev=None, stream=None):
    """The fold of the 64-bit tensor `data` under `op`, mod 2^64 (data is
    only read)."""
    _dev_u64(data, "data")
    o = _op(op)
    sh, s = _stream_handle(data.device, stream)
    with _scratch_for(data.device, s, lib().reduce_scratch_bytes(data.numel())) as scr:
        host, hp = _total64_args(want_total, total_dev)
        _check(lib().reduce_op_u64(_ptr(data), data.numel(), o, hp, _ptr(total_dev), _ptr(scr),
                                   scr.numel(), sh), "reduce_op_u64")
    return int(host.value) if want_total else None


def scan_exclusive_u32(data, want_total=True, total_dev=None, stream=None):
    """data[j] <- data[0] + .. + data[j-1] in place (mod 2^32); returns the total."""
    return _scan("scan_exclusive_u32", data, want_total, total_dev, stream)


def scan_inclusive_u32(data, want_total=True, total_dev=None, stream=None):
    """data[j] <- data[0] + .. + data[j] in place (mod 2^32); returns the total."""
    return _scan("scan_inclusive_u32", data, want_total, total_dev, stream)


def runs_layout_u32(counts, ends=None, want_entries=True, entries_dev=None, stream=None):
    """ends <- inclusive prefix sum of the per-owner counts (pass ends=counts
    for in place); returns (ends, entries) with entries = max(total, 1) as an
    int when want_entries, else None (then see entries_dev)."""
    _dev_u32(counts, "counts")
    n = counts.numel()
    if ends is None:
        ends = _new(counts.shape, counts.dtype, counts.device, stream)
    _dev_u32(ends, "ends")
    if ends.numel() != n:
        raise ValueError("ends must have as many elements as counts")
    sh, s = _stream_handle(counts.device, stream)
    with _scratch_for(counts.device, s, lib().runs_scratch_bytes(n, 0)) as scr:
        host, hp = _total_args(want_entries, entries_dev)
        _check(lib().runs_layout_u32(_ptr(counts), _ptr(ends), n, hp, _ptr(entries_dev), _ptr(scr),
                                     scr.numel(), sh), "runs_layout_u32")
    return ends, (int(host.value) if want_entries else None)


def runs_slots_i32(slots, stream=None):
    """Every slot of the int32 tensor `slots` set to -1 (the row the runs are
    laid in); returns it."""
    _dev_u32(slots, "slots")
    sh, _ = _stream_handle(slots.device, stream)
    _check(lib().runs_slots_i32(_ptr(slots), slots.numel(), sh), "runs_slots_i32")
    return slots


def runs_owner_u32(ends, entry, owner=None, stream=None):
    """owner[j] = owner(entry[j], ends): the least i with ends[i] > entry[j],
    or -1 when no run holds the entry."""
    _dev_u32(ends, "ends")
    _dev_u32(entry, "entry")
    if owner is None:
        owner = _new(entry.numel(), torch.int32, entry.device, stream)
    _dev_u32(owner, "owner")
    if owner.numel() != entry.numel():
        raise ValueError("owner must have as many elements as entry")
    sh, s = _stream_handle(entry.device, stream)
    with _scratch_for(entry.device, s, lib().runs_scratch_bytes(ends.numel(), 0)) as scr:
        _check(lib().runs_owner_u32(_ptr(ends), ends.numel(), _ptr(entry), entry.numel(), _ptr(owner),
                                    _ptr(scr), scr.numel(), sh), "runs_owner_u32")
    return owner


def runs_owner_all_u32(ends, total, owner=None, stream=None):
    """The owner of every entry 0 .. total-1 (an int32 tensor of `total`)."""
    _dev_u32(ends, "ends")
    if owner is None:
        owner = _new(total, torch.int32, ends.device, stream)
    _dev_u32(owner, "owner")
    if owner.numel() != total:
        raise ValueError("owner must have `total` elements")
    sh, s = _stream_handle(ends.device, stream)
    with _scratch_for(ends.device, s, lib().runs_scratch_bytes(ends.numel(), total)) as scr:
        _check(lib().runs_owner_all_u32(_ptr(ends), ends.numel(), _ptr(owner), total, _ptr(scr),
                                        scr.numel(), sh), "runs_owner_all_u32")
    return owner


def segscan_scratch_bytes(n, seg_len):
    return lib().segscan_scratch_bytes(n, seg_len)


def segscan_u32(inp, seg_len, out=None, seg_sums=True, stream=None):
    """Inclusive scan restarted every seg_len entries, and the segment sums.

    out: output tensor (default: a new one; pass `inp` for in place).
    seg_sums: True for a new sums tensor, a tensor to fill, or None to skip.
    Returns (out, sums)."""
    _dev_u32(inp, "inp")
    n = inp.numel()
    if out is None:
        out = _new(inp.shape, inp.dtype, inp.device, stream)
    _dev_u32(out, "out")
    if out.numel() != n:
        raise ValueError("out must have as many elements as inp")
    if seg_len <= 0:
        raise ValueError("seg_len must be positive")
    if seg_sums is True:
        seg_sums = _new((n + seg_len - 1) // seg_len, inp.dtype, inp.device, stream)
    if seg_sums is not None:
        _dev_u32(seg_sums, "seg_sums")
        if seg_sums.numel() < (n + seg_len - 1) // seg_len:
            raise ValueError("seg_sums needs ceil(n / seg_len) entries")
    sh, s = _stream_handle(inp.device, stream)
    with _scratch_for(inp.device, s, lib().segscan_scratch_bytes(n, seg_len)) as scr:
        _check(lib().segscan_u32(_ptr(inp), _ptr(out), n, seg_len, _ptr(seg_sums), _ptr(scr),
                                 scr.numel(), sh), "segscan_u32")
    return out, seg_sums


def segscan_flags_u32(inp, flags, out=None, seg_sums=True, want_nsegs=True, nsegs_dev=None,
                      stream=None):
    """Inclusive scan restarted at element 0 and wherever flags is non-zero,
    and each segment's total.

    out: output tensor (default: a new one; pass `inp` for in place).
    seg_sums: True for a new tensor of n entries, a tensor with room for
    every segment, or None to skip.  Returns (out, sums, nsegs): when
    want_nsegs, nsegs is the segment count and sums (if made here) is cut to
    it; else nsegs is None and the count goes to nsegs_dev."""
    _dev_u32(inp, "inp")
    _dev_u32(flags, "flags")
    n = inp.numel()
    if flags.numel() != n:
        raise ValueError("flags must have as many elements as inp")
    if out is None:
        out = _new(inp.shape, inp.dtype, inp.device, stream)
    _dev_u32(out, "out")
    if out.numel() != n:
        raise ValueError("out must have as many elements as inp")
    made = seg_sums is True
    if made:
        seg_sums = _new(max(n, 1), inp.dtype, inp.device, stream)
    if seg_sums is not None:
        _dev_u32(seg_sums, "seg_sums")
    sh, s = _stream_handle(inp.device, stream)
    with _scratch_for(inp.device, s, lib().segscan_flags_scratch_bytes(n)) as scr:
        host, hp = _total_args(want_nsegs, nsegs_dev)
        _check(lib().segscan_flags_u32(_ptr(inp), _ptr(flags), _ptr(out), n, _ptr(seg_sums), hp,
                                       _ptr(nsegs_dev), _ptr(scr), scr.numel(), sh),
               "segscan_flags_u32")
    nsegs = int(host.value) if want_nsegs else None
    if made and nsegs is not None:
        seg_sums = seg_sums[:nsegs]
    return out, seg_sums, nsegs


def compact_scratch_bytes(n):
    return lib().compact_scratch_bytes(n)


def compact_flags_u32(flags, out=None, want_count=True, count_dev=None, stream=None):
    """Kept indices (non-zero flags) in order, -1 elsewhere; returns
    (out, count) with count an int when want_count, else None."""
    _dev_u32(flags, "flags")
    n = flags.numel()
    if out is None:
        out = _new(n, torch.int32, flags.device, stream)
    _dev_u32(out, "out")
    if out.numel() != n:
        raise ValueError("out must have as many elements as flags")
    sh, s = _stream_handle(flags.device, stream)
    with _scratch_for(flags.device, s, lib().compact_scratch_bytes(n)) as scr:
        host, hp = _total_args(want_count, count_dev)
        _check(lib().compact_flags_u32(_ptr(flags), _ptr(out), n, hp, _ptr(count_dev), _ptr(scr),
                                       scr.numel(), sh), "compact_flags_u32")
    return out, (int(host.value) if want_count else None)


def radix_scratch_bytes(n, bits_per_pass=1):
    return lib().radix_scratch_bytes(n, bits_per_pass)


def radix_perm_u32(keys, bits_per_pass=1, perm=None, stream=None):
    """Stable LSB-first radix-sort permutation of u32 keys (gather form)."""
    _dev_u32(keys, "keys")
    n = keys.numel()
    if perm is None:
        perm = _new(n, torch.int32, keys.device, stream)
    _dev_u32(perm, "perm")
    if perm.numel() != n:
        raise ValueError("perm must have as many elements as keys")
    sh, s = _stream_handle(keys.device, stream)
    with _scratch_for(keys.device, s, lib().radix_scratch_bytes(n, bits_per_pass)) as scr:
        _check(lib().radix_perm_u32(_ptr(keys), _ptr(perm), n, bits_per_pass, _ptr(scr), scr.numel(),
                                    sh), "radix_perm_u32")
    return perm


# Largest n of scan_u32_noalloc (LIBSCAN_NOALLOC_MAX_N of libscan.h).
NOALLOC_MAX_N = 1 << 32


def scan_u32_noalloc(data, inclusive=False, total_dev=None, stream=None):
    """In-place scan of `data` (as scan_exclusive_u32 / scan_inclusive_u32)
    whose scratch is the library's own static device array: nothing is
    allocated, here or in the library.  The total goes to the device u32
    `total_dev` when given; nothing waits."""
    _dev_u32(data, "data")
    if total_dev is not None:
        _dev_u32(total_dev, "total_dev")
    sh, _ = _stream_handle(data.device, stream)
    _check(lib().scan_u32_noalloc(_ptr(data), data.numel(), 1 if inclusive else 0,
                                  _ptr(total_dev), sh), "scan_u32_noalloc")
    return None


def copy_u32(src, dst, stream=None):
    """dst <- src with the library's streaming copy (dst may be src: an
    in-place pass with the scan's memory traffic and none of its work)."""
    _dev_u32(src, "src")
    _dev_u32(dst, "dst")
    if dst.numel() != src.numel():
        raise ValueError("src and dst differ in size")
    sh, s = _stream_handle(src.device, stream)
    with _scratch_for(src.device, s, lib().copy_scratch_bytes(src.numel())) as scr:
        _check(lib().copy_u32(_ptr(src), _ptr(dst), src.numel(), _ptr(scr), scr.numel(), sh),
               "copy_u32")
    return dst


# --------------------------------------------------------------------------
# Linear attention with a decay for each head, and sampling
# --------------------------------------------------------------------------

def _dev_rows(t, name, dtype=None, dims=None, device=None):
    """A tensor of float rows: any strides, its last dimension contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s" % (
            name, dtype or "float32, bfloat16 or float16", t.dtype))
    if dims is not None and t.dim() != dims:
        raise ValueError("%s must have %d dimensions, got %d" % (name, dims, t.dim()))
    if t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError("%s must be on %s, got %s" % (name, device or "a GPU device", t.device))
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    return t


def _dev_dense(t, name, dtype, shape, device):
    """A contiguous tensor of one type, shape and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


# What the checks of a call's tensors found, by the tensors' layouts: shapes,
# strides, types and devices, never addresses or values.
_plans = {}


def _layout(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _planned(make, *tensors):
    try:
        key = (make, *map(_layout, tensors))
    except AttributeError:              # something is no tensor: the checks say which
        return make(*tensors)
    plan = _plans.get(key)
    if plan is None:
        plan = make(*tensors)
        if len(_plans) >= 1024:
            _plans.clear()
        _plans[key] = plan
    return plan


def _no_gradient(what, *tensors, pair="linattn", back=None):
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise RuntimeError("%s records no gradient: call it under torch.no_grad(), or %s and "
                                   "%s as the forward and backward of a torch.autograd.Function"
                                   % (what, pair, back or pair + "_grad"))


def _rows(t, packed):
    """(strides of sequence, token and head, heads) of a [B, T, H, D] tensor's rows, a packed
    [N, H, D] one's or a step's [B, H, D]."""
    seq, tok = (0, t.stride(0)) if packed else (t.stride(0), t.stride(1) if t.dim() == 4 else 0)
    return seq, tok, t.stride(-2), t.shape[-2]


def _dense_rows(shape, packed):
    """_rows of a new tensor."""
    heads, width = shape[-2:]
    if packed:
        return 0, heads * width, width, heads
    return (heads * width * (shape[1] if len(shape) == 4 else 1),
            heads * width if len(shape) == 4 else 0, width, heads)


def _shape_of(q, k, v, log_decay, ends, dims):
    """The call's _Shape without its pointers and scale."""
    _dev_rows(q, "q", dims=dims)
    device = q.device
    _dev_rows(k, "k", q.dtype, dims, device)
    _dev_rows(v, "v", q.dtype, dims, device)
    if k.shape[:-2] != q.shape[:-2] or v.shape[:-2] != q.shape[:-2]:
        raise ValueError("q, k and v must have the same tokens, got %s, %s and %s" % (
            tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    if k.shape[-1] != q.shape[-1]:
        raise ValueError("q and k must have the same width, got %d and %d" % (
            q.shape[-1], k.shape[-1]))
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not 1 <= t.shape[-1] <= LINATTN_MAX_WIDTH:
            raise ValueError("%s must be 1 to %d wide, got %d" % (
                name, LINATTN_MAX_WIDTH, t.shape[-1]))
    if not isinstance(log_decay, torch.Tensor) or log_decay.dim() != 1:
        raise TypeError("log_decay must be a torch.Tensor of one float for each head")
    heads = log_decay.shape[0]
    _dev_dense(log_decay, "log_decay", torch.float32, (heads,), device)
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.shape[-2] == 0 or heads % t.shape[-2]:
            raise ValueError("the heads of %s (%d) must divide log_decay's %d" % (
                name, t.shape[-2], heads))
    seqs = q.shape[0]
    if ends is not None:
        _dev_u32(ends, "ends")
        if ends.device != device or ends.dim() != 1:
            raise ValueError("ends must be one number for each sequence, on %s" % device)
        seqs = ends.shape[0]
    return _Shape(_DTYPES[q.dtype], seqs, heads, q.shape[-1], v.shape[-1],
                  q.shape[-3] if dims == 4 or ends is not None else 1)


def _states(shape, t, name, device, count=None):
    return None if t is None else _dev_dense(
        t, name, torch.float32,
        (shape.seqs if count is None else count, shape.heads, shape.key_width, shape.value_width),
        device)


def _apart(t, name):
    """Refuses an output (or None) whose rows share elements."""
    if t is None or t.numel() == 0:
        return
    width = covered = t.shape[-1]
    steps = sorted((s, n) for s, n in zip(t.stride()[:-1], t.shape[:-1]) if n > 1)
    for s, n in steps:                  # mostly each steps past all that those before it cover
        if s < covered:
            break
        covered += s * (n - 1)
    else:
        return
    apart = steps[0][0] >= width
    if apart:                           # woven into each other: by where each row starts
        at = torch.zeros(1, dtype=torch.int64)
        for s, n in steps:
            at = (at.unsqueeze(1) + s * torch.arange(n)).flatten()
        apart = bool((at.sort().values.diff() >= width).all())
    if not apart:
        raise ValueError("the rows of %s overlap" % name)


def _out_like(out, name, want, dtype, device):
    """`out`, checked, or None."""
    if out is not None:
        _dev_rows(out, name, dtype, len(want), device)
        if tuple(out.shape) != tuple(want):
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(want), tuple(out.shape)))
        _apart(out, name)
    return out


class _Plan:
    """What a call's layout comes to: the _Shape's fields, and for each tensor of rows its
    strides and the shape that a new one would have."""

    def __init__(self, shape, q, rows, need):
        self.fields = [getattr(shape, n) for n, _ in _Shape._fields_[:6]]
        self.rows = rows
        self.need = need
        self.dtype, self.device, self.index = q.dtype, q.device, q.get_device()
        self.states = (shape.seqs, shape.heads, shape.key_width, shape.value_width)

    def shape(self, ends, log_decay, scale, clear=False):
        sh = _Shape(*self.fields, None if ends is None else ends.data_ptr(), log_decay.data_ptr(), scale)
        if clear:
            sh.dtype |= _CLEAR_REST
        return sh

    def new(self, i, stream, zeros=False):
        return _new(self.rows[i][1], self.dtype, self.device, stream, zeros)

    def new_rows(self, ends, given, stream):
        """The tensors {index: tensor or None} with new ones for None, and whether the call has to
        clear their rows past the last end: it does so for all or for none of them."""
        made = [t is None for t in given.values()]
        rest = ends is not None and any(made)
        clear = rest and all(made) and self.fields[1] != 0
        return [self.new(i, stream, rest and not clear) if t is None else t for i, t in given.items()], clear

    def new_states(self, stream):
        return _new(self.states, torch.float32, self.device, stream)

    def stream(self, stream):
        return _raw_stream(self.index) if stream is None else stream.cuda_stream

    def scratch(self, handle, stream):
        return _scratch_at(self.device, self.index, handle, stream, self.need)

    def at(self, i, t):
        return _Rows(t.data_ptr(), *self.rows[i][0])


def _addr(t):
    return None if t is None else t.data_ptr()


def _row_plan(packed, *pairs):
    """For each (tensor or None, its shape): (strides and heads, shape)."""
    return [(_dense_rows(want, packed) if t is None else _rows(t, packed), tuple(want)) for t, want in pairs]


def _linattn_plan(q, k, v, log_decay, ends, state, out, state_out):
    packed = ends is not None
    shape = _shape_of(q, k, v, log_decay, ends, 3 if packed else 4)
    _states(shape, state, "state", q.device)
    want = q.shape[:-2] + (shape.heads, shape.value_width)
    _out_like(out, "out", want, q.dtype, q.device)
    _states(shape, state_out, "state_out", q.device)
    if packed:                          # no value of ends plays a part in the scratch's size
        shape.ends = ends.data_ptr()
    return _Plan(shape, q, _row_plan(packed, (q, q.shape), (k, k.shape), (v, v.shape), (out, want)),
                 lib().linattn_scratch_bytes(shape))


def linattn(q, k, v, log_decay, scale=1.0, ends=None, state=None, want_state=False, out=None,
            state_out=None, stream=None):
    """Linear attention with a decay for each head, over whole sequences:
    S(t) = exp(log_decay) S(t-1) + k(t) v(t)^T, out(t) = scale S(t)^T q(t).

    q, k [B, T, H, Dk] and v [B, T, H, Dv] (k, v and q may have fewer heads,
    each shared by consecutive ones); with ends (int32 [B], as
    runs_layout_u32 leaves them) [N, H, D], the sequences one after another.
    state: float32 [B, H, Dk, Dv] before the first token (None: zeros).
    Tokens past the last end are in no sequence: there a given out stays as
    it is, and a new one holds zeros.
    Returns (out, state_out), state_out None unless want_state or given.
    Neither carries a gradient (linattn_grad has it, for an autograd.Function;
    examples/recall.py has one): tensors that require one are refused."""
    p = _planned(_linattn_plan, q, k, v, log_decay, ends, state, out, state_out)
    _no_gradient("linattn", q, k, v, log_decay, state)
    (out,), clear = p.new_rows(ends, {3: out}, stream)
    if state_out is None and want_state:
        state_out = p.new_states(stream)
    handle = p.stream(stream)
    with p.scratch(handle, stream) as scr:
        _check(lib().linattn(p.shape(ends, log_decay, scale, clear), p.at(0, q), p.at(1, k), p.at(2, v), _addr(state),
                             p.at(3, out), _addr(state_out), scr.data_ptr(), scr.numel(), handle), "linattn")
    return out, state_out


def _linattn_grad_plan(dout, q, k, v, log_decay, ends, state, dstate_out, dq, dk, dv, dstate):
    packed = ends is not None
    shape = _shape_of(q, k, v, log_decay, ends, 3 if packed else 4)
    _dev_rows(dout, "dout", q.dtype, q.dim(), q.device)
    want = tuple(q.shape[:-2]) + (shape.heads, shape.value_width)
    if tuple(dout.shape) != want:
        raise ValueError("dout must have the shape of linattn's out, got %s" % (tuple(dout.shape),))
    for t, name in ((state, "state"), (dstate_out, "dstate_out"), (dstate, "dstate")):
        _states(shape, t, name, q.device)
    for t, name, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        _out_like(t, name, like.shape, q.dtype, q.device)
    if packed:
        shape.ends = ends.data_ptr()
    return _Plan(shape, q, _row_plan(packed, (dout, want), (q, q.shape), (k, k.shape), (v, v.shape),
                                     (dq, q.shape), (dk, k.shape), (dv, v.shape)),
                 lib().linattn_grad_scratch_bytes(shape, q.shape[-2], k.shape[-2], v.shape[-2]))


def linattn_grad(dout, q, k, v, log_decay, scale=1.0, ends=None, state=None, dstate_out=None,
                 want_dstate=False, dq=None, dk=None, dv=None, dstate=None, stream=None):
    """The gradient of linattn: (dq, dk, dv, dstate) for out's gradient dout
    and state_out's dstate_out (None: zeros); dstate is None unless
    want_dstate or given.  Gradients of shared heads are summed; past the last
    end they are as linattn's out is."""
    p = _planned(_linattn_grad_plan, dout, q, k, v, log_decay, ends, state, dstate_out, dq, dk, dv, dstate)
    _no_gradient("linattn_grad", dout, q, k, v, log_decay, state, dstate_out)
    (dq, dk, dv), clear = p.new_rows(ends, {4: dq, 5: dk, 6: dv}, stream)
    if dstate is None and want_dstate:
        dstate = p.new_states(stream)
    handle = p.stream(stream)
    with p.scratch(handle, stream) as scr:
        _check(lib().linattn_grad(p.shape(ends, log_decay, scale, clear), p.at(0, dout), p.at(1, q), p.at(2, k),
                                  p.at(3, v), _addr(state), _addr(dstate_out), p.at(4, dq), p.at(5, dk),
                                  p.at(6, dv), _addr(dstate), scr.data_ptr(), scr.numel(), handle),
               "linattn_grad")
    return dq, dk, dv, dstate


def _linattn_step_plan(q, k, v, log_decay, state, slots, out, state_out):
    shape = _shape_of(q, k, v, log_decay, None, 3)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise TypeError("state must be a torch.Tensor of [P, H, Dk, Dv]")
    pool = state.shape[0]
    _states(shape, state, "state", q.device, pool)
    _states(shape, state_out, "state_out", q.device, pool)
    if slots is None:
        if pool != shape.seqs:
            raise ValueError("without slots, state must hold one state for each of %d rows, got %d"
                             % (shape.seqs, pool))
    else:
        _dev_dense(slots, "slots", torch.int32, (shape.seqs,), q.device)
    want = (shape.seqs, shape.heads, shape.value_width)
    _out_like(out, "out", want, q.dtype, q.device)
    return _Plan(shape, q, _row_plan(False, (q, q.shape), (k, k.shape), (v, v.shape), (out, want)), 0)


def linattn_step(q, k, v, log_decay, state, scale=1.0, slots=None, out=None, state_out=None,
                 stream=None):
    """One token of each row of linattn's recurrence: q, k [B, H, Dk] and
    v [B, H, Dv]; row r updates state[slots[r]] (state[r] without slots) of
    the float32 pool [P, H, Dk, Dv], in place or into state_out.  A row whose
    slot is outside the pool, as -1, gives zeros and touches nothing; no slot
    may be listed twice.  Returns (out, the pool that was written)."""
    if state_out is None:
        state_out = state
    p = _planned(_linattn_step_plan, q, k, v, log_decay, state, slots, out, state_out)
    _no_gradient("linattn_step", q, k, v, log_decay, state)
    if out is None:
        out = p.new(3, stream)
    _check(lib().linattn_step(p.shape(None, log_decay, scale), p.at(0, q), p.at(1, k), p.at(2, v),
                              state.data_ptr(), state.shape[0], _addr(slots), p.at(3, out),
                              state_out.data_ptr(), p.stream(stream)), "linattn_step")
    return out, state_out


# --------------------------------------------------------------------------
# Gated recurrence of each channel
# --------------------------------------------------------------------------

class _GatePlan:
    """What a call's layout comes to: the _GateShape's fields, and for each tensor of rows its
    strides."""

    def __init__(self, gate, ends, rows, grad):
        packed = ends is not None
        step = grad is None
        tokens = 1 if step else gate.shape[-2]
        self.lead = gate.shape[:-1]
        self.dtype, self.device, self.index = gate.dtype, gate.device, gate.get_device()
        self.fields = (ends.shape[0] if packed else gate.shape[0], tokens, gate.shape[-1])
        self.states = (self.fields[0], gate.shape[-1])
        dense = (0 if packed else tokens * gate.shape[-1], gate.shape[-1])
        self.rows = [dense if t is None else (0 if packed else t.stride(0), 0 if step else t.stride(-2))
                     for t in rows]
        self.shape_of = tuple(gate.shape)
        self.need = 0
        if not step:
            shape = _GateShape(_DTYPES[self.dtype], 0, 0, 0, *self.fields, ends.data_ptr() if packed else None)
            self.need = lib().gatescan_scratch_bytes(shape, int(grad))

    def shape(self, form, blend, ends=None, clear=False):
        return _GateShape(_DTYPES[self.dtype], form, int(bool(blend)), int(clear), *self.fields, _addr(ends))

    def new(self, stream, zeros=False):
        return _new(self.shape_of, self.dtype, self.device, stream, zeros)

    def new_rows(self, ends, given, stream):
        """The tensors with new ones for None, and whether the call has to clear their rows past
        the last end: it does so for all or for none of them."""
        made = [t is None for t in given]
        rest = ends is not None and any(made)
        clear = rest and all(made) and self.fields[0] != 0
        return [self.new(stream, rest and not clear) if t is None else t for t in given], clear

    def new_states(self, stream):
        return _new(self.states, torch.float32, self.device, stream)

    def stream(self, stream):
        return _raw_stream(self.index) if stream is None else stream.cuda_stream

    def scratch(self, handle, stream):
        return _scratch_at(self.device, self.index, handle, stream, self.need)

    def at(self, i, t):
        return _GateRows(_addr(t), *self.rows[i])


def _form(form):
    if form not in _FORMS:
        raise ValueError("form must be one of %s, got %r" % (sorted(_FORMS), form))
    return _FORMS[form]


def _given(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)


def _gate_rows(gate, dims, *named):
    """Checks of a call's rows, all of the gate's shape, type and device."""
    _dev_rows(gate, "gate", dims=dims)
    if gate.shape[-1] == 0:
        raise ValueError("gate must be 1 wide at least")
    for t, name in named:
        if t is not None:
            _dev_rows(t, name, gate.dtype, dims, gate.device)
            if t.shape != gate.shape:
                raise ValueError("%s must have gate's shape %s, got %s" % (
                    name, tuple(gate.shape), tuple(t.shape)))


def _gate_ends(gate, ends):
    if ends is not None:
        _dev_u32(ends, "ends")
        if ends.device != gate.device or ends.dim() != 1:
            raise ValueError("ends must be one number for each sequence, on %s" % gate.device)
    return gate.shape[0] if ends is None else ends.shape[0]


def _gate_states(gate, count, *named):
    for t, name in named:
        if t is not None:
            _dev_dense(t, name, torch.float32, (count, gate.shape[-1]), gate.device)


def _gatescan_plan(gate, x, ends, state, out, state_out):
    _given(x, "x")
    _gate_rows(gate, 3 if ends is None else 2, (x, "x"), (out, "out"))
    _gate_states(gate, _gate_ends(gate, ends), (state, "state"), (state_out, "state_out"))
    _apart(out, "out")
    return _GatePlan(gate, ends, (gate, x, out), False)


def gatescan(gate, x, form="decay", blend=False, ends=None, state=None, want_state=False, out=None,
             state_out=None, stream=None):
    """A gated recurrence of each channel, over whole sequences:
    h(t) = a(t) h(t-1) + b(t), and out = h.

    gate and x are [B, T, D], or with ends (int32 [B], as runs_layout_u32
    leaves them) [N, D], the sequences one after another.  a is the gate
    itself, its exponential (form="log") or its sigmoid (form="sigmoid"), at
    most 1 in size; b is x, or (1 - a) x with blend.  state: float32 [B, D]
    before the first token (None: zeros).  Tokens past the last end are in no
    sequence: there a given out stays as it is, and a new one holds zeros.
    Returns (out, state_out), state_out None unless want_state or given.
    Neither carries a gradient (gatescan_grad has it, for an
    autograd.Function): tensors that require one are refused."""
    form = _form(form)
    p = _planned(_gatescan_plan, gate, x, ends, state, out, state_out)
    _no_gradient("gatescan", gate, x, state, pair="gatescan")
    (out,), clear = p.new_rows(ends, [out], stream)
    if state_out is None and want_state:
        state_out = p.new_states(stream)
    handle = p.stream(stream)
    with p.scratch(handle, stream) as scr:
        _check(lib().gatescan(p.shape(form, blend, ends, clear), p.at(0, gate), p.at(1, x), _addr(state),
                              p.at(2, out), _addr(state_out), scr.data_ptr(), scr.numel(), handle), "gatescan")
    return out, state_out


def _gatescan_grad_plan(dout, gate, x, out, ends, state, dstate_out, dgate, dx, dstate):
    _gate_rows(gate, 3 if ends is None else 2, (dout, "dout"), (x, "x"), (out, "out"), (dgate, "dgate"), (dx, "dx"))
    _gate_states(gate, _gate_ends(gate, ends), (state, "state"), (dstate_out, "dstate_out"), (dstate, "dstate"))
    _apart(dgate, "dgate")
    _apart(dx, "dx")
    return _GatePlan(gate, ends, (dout, gate, x, out, dgate, dx), True)


def gatescan_grad(dout, gate, x, out, form="decay", blend=False, ends=None, state=None, dstate_out=None,
                  want_dstate=False, dgate=None, dx=None, dstate=None, stream=None):
    """The gradient of gatescan: (dgate, dx, dstate) for out's gradient dout
    and state_out's dstate_out (None: zeros); dstate is None unless want_dstate
    or given.  out is what gatescan returned: the gates' gradient is taken from
    it as it is rounded there.  Without blend x is not read and may be None.
    Past the last end the gradients are as gatescan's out is."""
    form = _form(form)
    for t, name in ((dout, "dout"), (out, "out")) + (((x, "x"),) if blend else ()):
        _given(t, name)
    p = _planned(_gatescan_grad_plan, dout, gate, x, out, ends, state, dstate_out, dgate, dx, dstate)
    _no_gradient("gatescan_grad", dout, gate, x, out, state, dstate_out, pair="gatescan")
    (dgate, dx), clear = p.new_rows(ends, [dgate, dx], stream)
    if dstate is None and want_dstate:
        dstate = p.new_states(stream)
    handle = p.stream(stream)
    with p.scratch(handle, stream) as scr:
        _check(lib().gatescan_grad(p.shape(form, blend, ends, clear), p.at(0, dout), p.at(1, gate), p.at(2, x),
                                   p.at(3, out), _addr(state), _addr(dstate_out), p.at(4, dgate), p.at(5, dx),
                                   _addr(dstate), scr.data_ptr(), scr.numel(), handle), "gatescan_grad")
    return dgate, dx, dstate


def _gatescan_step_plan(gate, x, state, slots, out, state_out):
    _given(x, "x")
    _gate_rows(gate, 2, (x, "x"), (out, "out"))
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise TypeError("state must be a torch.Tensor of [P, D]")
    pool = state.shape[0]
    _gate_states(gate, pool, (state, "state"), (state_out, "state_out"))
    if slots is not None:
        _dev_dense(slots, "slots", torch.int32, (gate.shape[0],), gate.device)
    elif pool != gate.shape[0]:
        raise ValueError("without slots, state must hold one state for each of %d rows, got %d"
                         % (gate.shape[0], pool))
    _apart(out, "out")
    return _GatePlan(gate, None, (gate, x, out), None)


def gatescan_step(gate, x, state, form="decay", blend=False, slots=None, out=None, state_out=None, stream=None):
    """One token of each row of gatescan's recurrence: gate, x [B, D]; row r
    updates state[slots[r]] (state[r] without slots) of the float32 pool
    [P, D], in place or into state_out.  A row whose slot is outside the pool,
    as -1, gives zeros and touches nothing; no slot may be listed twice.
    Returns (out, the pool that was written)."""
    form = _form(form)
    if state_out is None:
        state_out = state
    p = _planned(_gatescan_step_plan, gate, x, state, slots, out, state_out)
    _no_gradient("gatescan_step", gate, x, state, pair="gatescan")
    if out is None:
        out = p.new(stream)
    _check(lib().gatescan_step(p.shape(form, blend), p.at(0, gate), p.at(1, x), state.data_ptr(), state.shape[0],
                               _addr(slots), p.at(2, out), state_out.data_ptr(), p.stream(stream)),
           "gatescan_step")
    return out, state_out


# --------------------------------------------------------------------------
# Rows of a table by their ids, and the gradient
# --------------------------------------------------------------------------

def _spaced(t, name):
    """The stride of t's rows, all of its dimensions but the last taken as one."""
    if t.numel() == 0:                  # no rows, and strides that say nothing
        return t.shape[-1]
    stride, count = 0, 1
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if count == 1:
            stride = s
        elif s != stride * count:
            raise ValueError("the rows of %s must be evenly spaced" % name)
        count *= n
    return stride


def _ids(ids, device):
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64, got %s" % ids.dtype)
    if ids.device != device:
        raise ValueError("ids must be on %s, got %s" % (device, ids.device))
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")


def _embed_plan(rows, to, ids, name):
    """What _embed_rows_plan and _embed_grad_plan have alike: rows (weight or dout) and ids."""
    _dev_rows(rows, name)
    if rows.shape[-1] == 0:
        raise ValueError("%s must be 1 wide at least" % name)
    _ids(ids, rows.device)
    if to not in _DTYPES:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % to)
    return (_DTYPES[rows.dtype], _DTYPES[to], ids.element_size(), ids.numel())


def _embed_rows_plan(to, weight, ids, out):
    to = to or (weight.dtype if out is None else out.dtype)
    fields = _embed_plan(weight, to, ids, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must have 2 dimensions, got %d" % weight.dim())
    want = tuple(ids.shape) + (weight.shape[1],)
    _out_like(out, "out", want, to, weight.device)
    return (fields + tuple(weight.shape), weight.stride(0), weight.shape[1] if out is None else _spaced(out, "out"),
            want, to, weight.device, weight.get_device())


def _embed_grad_plan(to, dout, ids, dweight):
    to = to or (dout.dtype if dweight is None else dweight.dtype)
    fields = _embed_plan(dout, to, ids, "dout")
    if dout.shape[:-1] != ids.shape:
        raise ValueError("dout must have a row for each id, got %s for %s" % (tuple(dout.shape), tuple(ids.shape)))
    if dweight is not None:
        _dev_rows(dweight, "dweight", to, 2, dout.device)
        if dweight.shape[1] != dout.shape[-1]:
            raise ValueError("dweight must be %d wide, got %d" % (dout.shape[-1], dweight.shape[1]))
        _apart(dweight, "dweight")
    return (fields, dout.shape[-1], _spaced(dout, "dout"), dout.shape[-1] if dweight is None else dweight.stride(0),
            to, dout.device, dout.get_device())


# By the type asked for, which plans differ by as well.
_embed_rows_plans = {d: functools.partial(_embed_rows_plan, d) for d in (None, *_DTYPES)}
_embed_grad_plans = {d: functools.partial(_embed_grad_plan, d) for d in (None, *_DTYPES)}


def _embed_type(dtype, plans):
    if dtype not in plans:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % (dtype,))
    return plans[dtype]


def embed_rows(weight, ids, scale=1.0, dtype=None, out=None, stream=None):
    """scale * weight[ids]: rows of the table weight [V, D] by ids (int32 or
    int64, of any shape), as dtype (None: weight's, or a given out's).  An id
    outside the table, as -1 for padding, gives zeros.  It carries no
    gradient (embed_grad has it, for an autograd.Function): a weight that
    requires one is refused."""
    fields, stride, out_stride, want, to, device, index = _planned(
        _embed_type(dtype, _embed_rows_plans), weight, ids, out)
    _no_gradient("embed_rows", weight, pair="embed_rows", back="embed_grad")
    if out is None:
        out = _new(want, to, device, stream)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    _check(lib().embed_rows(_Embed(*fields, scale), weight.data_ptr(), stride, ids.data_ptr(), out.data_ptr(),
                            out_stride, handle), "embed_rows")
    return out


def embed_grad(dout, ids, rows, scale=1.0, dtype=None, dweight=None, accumulate=False, stream=None):
    """The gradient of embed_rows for a table of `rows` rows: dweight[v] =
    scale * the sum of dout[i] over all i with ids[i] = v, as dtype (None:
    dout's, or a given dweight's), zeros in rows of no id.  With accumulate
    it is added to the given dweight instead.  The sums' order is the same
    every time."""
    fields, width, stride, to_stride, to, device, index = _planned(
        _embed_type(dtype, _embed_grad_plans), dout, ids, dweight)
    _no_gradient("embed_grad", dout, pair="embed_rows", back="embed_grad")
    rows = int(rows)
    if not 0 <= rows <= EMBED_MAX_ROWS:
        raise ValueError("rows must be 0 to %d, got %d" % (EMBED_MAX_ROWS, rows))
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate needs a dweight to add to")
        dweight = _new((rows, width), to, device, stream)
    elif dweight.shape[0] != rows:
        raise ValueError("dweight must have %d rows, got %d" % (rows, dweight.shape[0]))
    shape = _Embed(*fields, rows, width, scale)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    with _scratch_at(device, index, handle, stream, lib().embed_grad_scratch_bytes(shape)) as scr:
        _check(lib().embed_grad(shape, dout.data_ptr(), stride, ids.data_ptr(), dweight.data_ptr(), to_stride,
                                int(bool(accumulate)), scr.data_ptr(), scr.numel(), handle), "embed_grad")
    return dweight


# --------------------------------------------------------------------------
# Penalties on logits, and sampling
# --------------------------------------------------------------------------

def _lists(tokens, ends, name, rows, device):
    """(stride of a row, elements of a row or in all) of a row's lists, checked."""
    if tokens is None:
        if ends is not None:
            raise ValueError("%s are missing where their ends are given" % name)
        return 0, 0
    if not isinstance(tokens, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if tokens.dtype != torch.int32:
        raise TypeError("%s must be int32, got %s" % (name, tokens.dtype))
    if tokens.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, tokens.device))
    if ends is not None:
        _dev_dense(ends, "the ends of %s" % name, (torch.int32, torch.uint32), (rows,), device)
        _dev_dense(tokens, name, torch.int32, (tokens.numel(),), device)
        return 0, tokens.numel()
    if tokens.dim() != 2 or tokens.shape[0] != rows:
        raise ValueError("%s must be a list for each of %d rows, got %s" % (name, rows, tuple(tokens.shape)))
    if tokens.shape[1] > 1 and tokens.stride(1) != 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    return tokens.stride(0), tokens.shape[1]


def _penalize_plan(logits, tokens, ends, prompt, repetition, presence, frequency, bias_tokens, bias_values,
                   bias_ends, mask, mask_slots, out):
    _dev_rows(logits, "logits", dims=2)
    device, (rows, vocab) = logits.device, logits.shape
    if vocab > SAMPLE_MAX_VOCAB:
        raise ValueError("logits must have at most %d columns, got %d" % (SAMPLE_MAX_VOCAB, vocab))
    _out_like(out, "out", logits.shape, logits.dtype, device)
    past = _lists(tokens, ends, "tokens", rows, device)
    bias = _lists(bias_tokens, bias_ends, "bias_tokens", rows, device)
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values come together")
    values = 0
    if bias_values is not None:
        _dev_rows(bias_values, "bias_values", torch.float32, 2 if bias_ends is None else 1, device)
        if bias_values.shape != bias_tokens.shape:
            raise ValueError("bias_values must have a value for each of bias_tokens, got %s for %s" % (
                tuple(bias_values.shape), tuple(bias_tokens.shape)))
        values = bias_values.stride(0)
    for t, name, dtype in ((prompt, "prompt", torch.int32), (repetition, "repetition", torch.float32),
                           (presence, "presence", torch.float32), (frequency, "frequency", torch.float32),
                           (mask_slots, "mask_slots", torch.int32)):
        if t is not None:
            _dev_dense(t, name, dtype, (rows,), device)
    masks, mask_stride = 0, 0
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.int32, torch.uint32):
            raise TypeError("mask must be a torch.Tensor of int32 or uint32 words")
        if mask.device != device or mask.dim() != 2 or mask.shape[1] != (vocab + 31) // 32:
            raise ValueError("mask must be [masks, %d] on %s, got %s on %s" % (
                (vocab + 31) // 32, device, tuple(mask.shape), mask.device))
        if mask.shape[1] > 1 and mask.stride(1) != 1:
            raise ValueError("the last dimension of mask must be contiguous")
        if mask_slots is None and mask.shape[0] != rows:
            raise ValueError("without mask_slots, mask must have one for each of %d rows, got %d" % (
                rows, mask.shape[0]))
        masks, mask_stride = mask.shape[0], mask.stride(0)
    elif mask_slots is not None:
        raise ValueError("mask_slots need a mask")
    return ((_DTYPES[logits.dtype], rows, vocab), logits.stride(0), vocab if out is None else out.stride(0), past,
            bias, values, mask_stride, masks, logits.dtype, device, logits.get_device())


def penalize_logits(logits, tokens=None, ends=None, prompt=None, repetition=1.0, presence=0.0, frequency=0.0,
                    bias_tokens=None, bias_values=None, bias_ends=None, mask=None, mask_slots=None, out=None,
                    stream=None):
    """Logits [R, V] as sample_logits is to have them.  tokens: what each row
    holds so far, int32 [R, L] (-1 behind shorter ones) or, with ends (int32
    [R], as runs_layout_u32 leaves them), one row's after another's; the first
    prompt[r] of a row (int32 [R]; None: none) are its prompt.

    A token among them is divided by repetition where its logit is above 0 and
    multiplied by it elsewhere; one that came g times after the prompt loses
    presence + frequency * g; each of these is a number or float32 [R].
    bias_values (float32) are added to bias_tokens' logits, listed as tokens
    are (the last value counts where a token is listed twice).  mask: words
    of 32 bits [G, ceil(V / 32)], a set bit for each token that may follow;
    row r has mask[mask_slots[r]] (int32 [R], outside as -1: none), mask[r]
    without slots; what is banned gets -inf.  Returns out, which may be
    logits itself; it carries no gradient, and tensors that require one are
    refused."""
    each = [t if isinstance(t, torch.Tensor) else None for t in (repetition, presence, frequency)]
    fields, stride, out_stride, past, bias, values, mask_stride, masks, dtype, device, index = _planned(
        _penalize_plan, logits, tokens, ends, prompt, *each, bias_tokens, bias_values, bias_ends, mask,
        mask_slots, out)
    if torch.is_grad_enabled():
        for t in (logits, bias_values, *each):
            if t is not None and t.requires_grad:
                raise RuntimeError("penalize_logits records no gradient: call it under torch.no_grad()")
    if out is None:
        out = _new(fields[1:], dtype, device, stream)
    a = _Penalty(*fields, logits.data_ptr(), stride, out.data_ptr(), out_stride,
                 _List(_addr(tokens), *past, _addr(ends)), _addr(prompt),
                 1.0 if each[0] is not None else repetition, 0.0 if each[1] is not None else presence,
                 0.0 if each[2] is not None else frequency, *map(_addr, each),
                 _List(_addr(bias_tokens), *bias, _addr(bias_ends)), _addr(bias_values), values,
                 _addr(mask), mask_stride, masks, _addr(mask_slots))
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    _check(lib().penalize_logits(a, handle), "penalize_logits")
    return out


def _sample_plan(logits, u, temperature, top_k, top_p, min_p, tokens, logprobs, kept):
    _dev_rows(logits, "logits", dims=2)
    device, rows = logits.device, logits.shape[0]
    if logits.shape[1] > SAMPLE_MAX_VOCAB:
        raise ValueError("logits must have at most %d columns, got %d" % (
            SAMPLE_MAX_VOCAB, logits.shape[1]))
    _dev_dense(u, "u", torch.float32, (rows,), device)
    for t, name, dtype in ((temperature, "temperature", torch.float32), (top_k, "top_k", torch.int32),
                           (top_p, "top_p", torch.float32), (min_p, "min_p", torch.float32),
                           (tokens, "tokens", torch.int32), (logprobs, "logprobs", torch.float32),
                           (kept, "kept", torch.int32)):
        if t is not None:
            _dev_dense(t, name, dtype, (rows,), device)
    return (_DTYPES[logits.dtype], rows, logits.shape[1], logits.stride(0), device, logits.get_device(),
            lib().sample_scratch_bytes(rows, logits.shape[1]))


def sample_logits(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None,
                  logprobs=None, kept=None, stream=None):
    """One token from each row of logits [R, V] by the random numbers u
    (float32 [R], in [0, 1)); temperature, top_k, top_p and min_p are numbers
    or tensors with one for each row (float32, and int32 for top_k).

    Of the tokens by falling logit, those with at least min_p of the largest
    one's weight are kept, top_k of them at most, then the fewest whose
    weight is at least top_p; the token is where u of the kept weights, in
    index order, is passed.  temperature 0 is the largest logit.  Returns
    (tokens int32, logprobs float32, kept int32), none of them with a gradient;
    a row with nothing but -inf and NaN gets token -1."""
    each = [t if isinstance(t, torch.Tensor) else None for t in (temperature, top_k, top_p, min_p)]
    code, rows, vocab, stride, device, index, need = _planned(
        _sample_plan, logits, u, *each, tokens, logprobs, kept)
    if tokens is None:
        tokens = _new(rows, torch.int32, device, stream)
    if logprobs is None:
        logprobs = _new(rows, torch.float32, device, stream)
    if kept is None:
        kept = _new(rows, torch.int32, device, stream)
    a = _Sample(code, rows, vocab, logits.data_ptr(), stride, u.data_ptr(),
                1.0 if each[0] is not None else temperature,
                1.0 if each[2] is not None else top_p,
                0.0 if each[3] is not None else min_p,
                0 if each[1] is not None else min(max(int(top_k), 0), 0x7FFFFFFF),
                _addr(each[0]), _addr(each[2]), _addr(each[3]), _addr(each[1]),
                tokens.data_ptr(), logprobs.data_ptr(), kept.data_ptr())
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    with _scratch_at(device, index, handle, stream, need) as scr:
        _check(lib().sample_logits(a, scr.data_ptr(), scr.numel(), handle), "sample_logits")
    return tokens, logprobs, kept
