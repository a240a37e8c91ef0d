"""GB300 exact epsilon self-join: thin Python binding of libhiss.so.

The library (include/hiss.h) computes the Euclidean self-join of RT-HiSS
(Munugala & Gowanlock, "RT-HiSS: Ray Tracing Accelerated High Dimensional
Vector Similarity Searches", Section II-A): every pair of points within eps,
self pairs included.  This module only marshals arguments: every step of the
join runs in the library's CUDA kernels.  PyTorch supplies device memory and
streams.  There is no CPU fallback: importing this module fails if
libhiss.so has not been built (``python exact_dimensional_distance_gb300/build.py``).

Operators that take a model's parameters to the points and a gradient back
(embedding lookup, layer norm, their gradients, clipping by the global gradient
norm) are methods of ``Join`` too; they are asynchronous on its stream.  They
work outside torch's differentiation: a result never requires a gradient, whatever
its inputs do, and the way back is called as such (``layer_norm_grad``, ``embed_grad``).

Functions with the names of the C ABI (``hiss_create``, ``hiss_build``, ...)
are the raw entry points; ``Join`` wraps a context for convenience.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhiss.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libhiss.so is missing: build it with "
                      "`python exact_dimensional_distance_gb300/build.py` (needs nvcc)")

_lib = ctypes.CDLL(LIB_PATH)

HISS_OK = 0
HISS_E_ARG = -1
HISS_E_NOMEM = -2
HISS_E_STATE = -3
HISS_E_BATCH_TOO_SMALL = -4
HISS_E_OVERFLOW = -5
HISS_E_CUDA = -6
HISS_E_CALLBACK = -7
HISS_OUT_CSR = 0
HISS_OUT_MASK = 1
HISS_OPT_ALLOC_LIMIT = 1
HISS_OPT_REFINE = 2
HISS_REFINE_CUDA_CORES = 0
HISS_REFINE_TENSOR_CORES = 1
HISS_MAX_DIM = 256
HISS_F32 = 0
HISS_F16 = 1
HISS_BF16 = 2
HISS_MAX_WIDTH = 65536
HISS_NO_PAD = -(1 << 63)

_i64, _i32, _f32, _p = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p


class hiss_batch(ctypes.Structure):
    _fields_ = [("index", _i64), ("nq", _i64), ("query_ids", _p), ("row_ptr", _p), ("cols", _p),
                ("mask", _p), ("cand", _p), ("query_rows", _p), ("nnz", _i64), ("n_words", _i64),
                ("on_host", _i32), ("mode", _i32)]


HISS_BATCH_FN = ctypes.CFUNCTYPE(ctypes.c_int, _p, ctypes.POINTER(hiss_batch))


class hiss_out(ctypes.Structure):
    _fields_ = [("mode", _i32), ("copy_to_host", _i32), ("on_batch", HISS_BATCH_FN), ("user", _p)]


class hiss_index_view(ctypes.Structure):
    _fields_ = [("n", _i64), ("cells", _i64), ("ids", _p), ("cell_start", _p), ("cell_of_row", _p),
                ("nbr", _p), ("nbr_count", _p), ("cell_bound", _p), ("cell_key", _p),
                ("perm", _i32 * 3), ("sub_bits", _i32), ("cell_width", ctypes.c_double),
                ("origin", ctypes.c_double * 3)]


class hiss_stats(ctypes.Structure):
    _fields_ = [("n", _i64), ("cells", _i64), ("cell_pairs", _i64), ("candidates", _i64), ("pairs", _i64),
                ("batches", _i64), ("query_tiles", _i64), ("refine_units", _i64), ("mask_words_max", _i64),
                ("kernel_launches", _i64), ("d", _i32), ("d_pad", _i32), ("sub_bits", _i32),
                ("key_bits", _i32), ("eps", _f32), ("cell_width", ctypes.c_double),
                ("ms_build", ctypes.c_double), ("ms_index", ctypes.c_double), ("ms_count", ctypes.c_double),
                ("ms_refine", ctypes.c_double), ("ms_compact", ctypes.c_double),
                ("ms_deliver", ctypes.c_double), ("ms_total", ctypes.c_double), ("deliveries", _i64),
                ("candidates_refined", _i64)]


class hiss_tensor(ctypes.Structure):
    _fields_ = [("in_", _p), ("out", _p), ("n", _i64), ("dtype", _i32), ("reserved", _i32)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


hiss_create = _sig("hiss_create", ctypes.c_int, [ctypes.POINTER(_p), _p])
hiss_destroy = _sig("hiss_destroy", None, [_p])
hiss_build = _sig("hiss_build", ctypes.c_int, [_p, _p, _i64, _i32])
hiss_build_host = _sig("hiss_build_host", ctypes.c_int, [_p, _p, _i64, _i32])
hiss_count = _sig("hiss_count", ctypes.c_int, [_p, _f32, _p])
hiss_join = _sig("hiss_join", ctypes.c_int, [_p, _f32, ctypes.c_size_t, ctypes.POINTER(hiss_out)])
hiss_index = _sig("hiss_index", ctypes.c_int, [_p, ctypes.POINTER(hiss_index_view)])
hiss_last_stats = _sig("hiss_last_stats", ctypes.c_int, [_p, ctypes.POINTER(hiss_stats)])
hiss_launch_count = _sig("hiss_launch_count", _i64, [_p])
hiss_strerror = _sig("hiss_strerror", ctypes.c_char_p, [ctypes.c_int])
hiss_last_cuda_error = _sig("hiss_last_cuda_error", ctypes.c_char_p, [_p])
hiss_set_option = _sig("hiss_set_option", ctypes.c_int, [_p, ctypes.c_int, _i64])
hiss_sort_pairs = _sig("hiss_sort_pairs", ctypes.c_int, [_p, _p, _p, _i64, _i32])
hiss_exclusive_scan = _sig("hiss_exclusive_scan", ctypes.c_int, [_p, _p, _p, _i64])
hiss_mask_positions = _sig("hiss_mask_positions", ctypes.c_int, [_p, _p, _i64, _p, ctypes.POINTER(_i64)])
hiss_work_profile = _sig("hiss_work_profile", ctypes.c_int, [_p, _f32, _p])
hiss_join_queries = _sig("hiss_join_queries", ctypes.c_int,
                         [_p, _p, _i64, _f32, ctypes.c_size_t, ctypes.POINTER(hiss_out)])
hiss_count_queries = _sig("hiss_count_queries", ctypes.c_int, [_p, _p, _i64, _f32, _p])
hiss_exclusive_scan_noalloc = _sig("hiss_exclusive_scan_noalloc", ctypes.c_int, [_p, _p, _p, _i64])
hiss_gram_tf32 = _sig("hiss_gram_tf32", ctypes.c_int, [_p, _p, _p, _i32, _p])
hiss_knn = _sig("hiss_knn", ctypes.c_int, [_p, _i32, _f32, _p, _p])
hiss_join_shard = _sig("hiss_join_shard", ctypes.c_int,
                       [_p, _f32, ctypes.c_size_t, ctypes.POINTER(hiss_out), _i32, _i32])
hiss_embed = _sig("hiss_embed", ctypes.c_int,
                  [_p, _p, _i32, _i64, _i32, _i64, _p, _i32, _i64, _i64, _f32, _p, _i32, _i64])
hiss_embed_grad = _sig("hiss_embed_grad", ctypes.c_int,
                       [_p, _p, _i32, _i64, _p, _i32, _i64, _i64, _f32, _i64, _i32, _i32, _p, _i32, _i64])
hiss_layer_norm = _sig("hiss_layer_norm", ctypes.c_int,
                       [_p, _p, _i32, _i64, _i64, _i32, _p, _p, _i32, _f32, _p, _i32, _i64, _p, _p])
hiss_layer_norm_grad = _sig("hiss_layer_norm_grad", ctypes.c_int,
                            [_p, _p, _i32, _i64, _p, _i32, _i64, _p, _p, _p, _i32, _i64, _i32, _p, _i64, _p, _p])
hiss_clip_grads = _sig("hiss_clip_grads", ctypes.c_int, [_p, ctypes.POINTER(hiss_tensor), _i64, _f32, _p])
hiss_finish = _sig("hiss_finish", ctypes.c_int, [_p])

EXPORTED = ["hiss_create", "hiss_destroy", "hiss_build", "hiss_build_host", "hiss_count", "hiss_join",
            "hiss_index", "hiss_last_stats", "hiss_launch_count", "hiss_strerror", "hiss_last_cuda_error",
            "hiss_set_option", "hiss_sort_pairs", "hiss_exclusive_scan", "hiss_mask_positions",
            "hiss_exclusive_scan_noalloc", "hiss_work_profile", "hiss_join_queries", "hiss_count_queries",
            "hiss_gram_tf32", "hiss_knn", "hiss_join_shard", "hiss_embed", "hiss_embed_grad", "hiss_layer_norm",
            "hiss_layer_norm_grad", "hiss_clip_grads", "hiss_finish"]


class HissError(RuntimeError):
    def __init__(self, status, ctx=None, what=""):
        msg = hiss_strerror(status).decode()
        if status == HISS_E_CUDA and ctx:
            msg += " (" + hiss_last_cuda_error(ctx).decode() + ")"
        super().__init__("%s: %s [%d]" % (what, msg, status))
        self.status = status


def _check(rc, ctx=None, what=""):
    if rc != HISS_OK:
        raise HissError(rc, ctx, what)


class DeviceArray:
    """A library-owned device buffer exposed through __cuda_array_interface__
    (wrap with torch.as_tensor(a, device='cuda'))."""

    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (int(ptr or 0), False), "version": 3}


def _host_array(ptr, n, dtype):
    if n == 0:
        return np.zeros(0, dtype=dtype)
    ctype = np.ctypeslib.as_ctypes_type(np.dtype(dtype))
    return np.ctypeslib.as_array(ctypes.cast(ptr, ctypes.POINTER(ctype)), shape=(n,)).copy()


def _device_tensor(ptr, n, typestr):
    import torch
    if n == 0:
        return torch.zeros(0, dtype={"<i8": torch.int64, "<i4": torch.int32, "<u4": torch.int32}[typestr],
                           device="cuda")
    return torch.as_tensor(DeviceArray(ptr, (n,), typestr), device="cuda")


_DTYPES = {}  # hiss_dtype of a torch dtype, filled on first use (torch is imported late)


def _dtype(t):
    """The hiss_dtype of a torch dtype."""
    code = _DTYPES.get(t)
    if code is None:
        import torch
        _DTYPES.update({torch.float32: HISS_F32, torch.float16: HISS_F16, torch.bfloat16: HISS_BF16})
        code = _DTYPES.get(t)
        if code is None:
            raise ValueError("float32, float16 or bfloat16 expected, not %s" % t)
    return code


def _matrix(t, name):
    """t as rows of unit column stride, a copy only where its strides need one:
    (matrix, rows, width, row stride)."""
    if t.dim() != 2:
        if t.dim() < 1:
            raise ValueError("%s: at least one dimension expected" % name)
        t = t.reshape(-1, t.shape[-1]) if t.shape[-1] else t.new_empty((0, 0))
    n, d = t.shape
    if d < 1 or d > HISS_MAX_WIDTH:
        raise ValueError("%s: width %d is outside 1..%d" % (name, d, HISS_MAX_WIDTH))
    row, column = t.stride()
    if column != 1:
        t = t.contiguous()
        row = d
    return t, n, d, row if n > 1 else d


def _pad(pad):
    """The library's pad argument (ctypes would wrap a larger number around to a token)."""
    if pad is None:
        return HISS_NO_PAD
    if not -1 << 63 <= pad < 1 << 63:
        raise ValueError("pad does not fit 64 bits")
    return pad


def _vector(t, width):
    """The address of a contiguous vector of width entries."""
    if t.shape != (width,) or not t.is_contiguous():
        raise ValueError("weight and bias: contiguous vectors of %d entries expected" % width)
    return t.data_ptr()


def _out_matrix(t, name):
    """As _matrix without a copy (t is written)."""
    m = t
    if t.dim() != 2:
        try:
            m = t.view(-1, t.shape[-1])
        except RuntimeError:
            raise ValueError("%s: rows of unit stride expected" % name) from None
    n, d = m.shape
    row, column = m.stride()
    if column != 1 and d > 1:
        raise ValueError("%s: rows of unit stride expected" % name)
    return m, row if n > 1 else d


def _raw_stream(index):
    """cudaStream_t of torch's current stream on a device."""
    import torch
    return torch.cuda.current_stream(index).cuda_stream


class Gradients:
    """Tensors to be clipped together: grads (float32, float16 or bfloat16 CUDA
    tensors) and optionally the tensors of the same shapes and types that receive the
    clipped values (default: in place).  Keeps the list that
    ``Join.clip_grads`` hands to the library, so a step that reuses its gradient
    tensors builds it once.  A tensor that has since got other memory (``t.data = ...``,
    ``t.set_()``) is found by each call, which then builds the list again.  One whose
    size, type or order changed within the memory it had needs a new list: until
    then the old elements are clipped, whose memory the list keeps from being freed.
    Tensors must be dense (contiguous in some order of their dimensions) and must not
    overlap."""

    def __init__(self, grads, out=None):
        grads = list(grads)
        out = grads if out is None else list(out)
        if len(out) != len(grads):
            raise ValueError("as many outputs as gradients expected")
        from torch import Tensor
        self._address, self._storage = Tensor.data_ptr, Tensor.untyped_storage
        self.grads, self.out = grads, out
        self._tensors = grads if out is grads else grads + out
        self._build()

    def _build(self):
        grads, out = self.grads, self.out
        spans = []
        array = (hiss_tensor * max(1, len(grads)))()
        for i, (g, o) in enumerate(zip(grads, out)):
            if not (g.is_cuda and o.is_cuda and g.device == o.device == grads[0].device):
                raise ValueError("gradient %d: CUDA tensors of one device expected" % i)
            if g.dtype != o.dtype or g.shape != o.shape or g.stride() != o.stride():
                raise ValueError("gradient %d: the output's type, shape and strides must be the gradient's" % i)
            if not self._dense(g):
                raise ValueError("gradient %d is not dense" % i)
            n = g.numel()
            array[i] = hiss_tensor(g.data_ptr(), o.data_ptr(), n, _dtype(g.dtype), 0)
            if n:
                spans.append((g.data_ptr(), g.data_ptr() + n * g.element_size()))
                if o.data_ptr() != g.data_ptr():
                    spans.append((o.data_ptr(), o.data_ptr() + n * o.element_size()))
        spans.sort()
        for a, b in zip(spans, spans[1:]):
            if b[0] < a[1]:
                raise ValueError("the tensors overlap")
        self.array, self._seen = array, [*map(self._address, self._tensors)]
        # as long as these are held, an address that is still a tensor's is the same memory
        self._memory = [*map(self._storage, self._tensors)]
        self.all = [t for t in self._tensors if t.numel()]

    def current(self):
        """The list for the tensors where they are now (60 tensors: 3 us)."""
        if [*map(self._address, self._tensors)] != self._seen:
            self._build()
        return self.array

    @staticmethod
    def _dense(t):
        if t.is_contiguous():
            return True
        want = 1
        for size, stride in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n != 1), key=lambda p: p[1]):
            if stride != want:
                return t.numel() == 0
            want *= size
        return True

    def __len__(self):
        return len(self.grads)


class Join:
    """One library context on a torch CUDA stream (default: the current one)."""

    def __init__(self, stream=None):
        import torch
        if not torch.cuda.is_available():
            raise RuntimeError("a CUDA device is required")
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        self._torch = torch
        self._device = self.stream.device
        self._index = self.stream.device_index
        self._raw = self.stream.cuda_stream
        # the same value without building a Stream object, where torch has it
        self._current = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
        self._scalar = None  # a model of clip_grads' result
        h = _p()
        _check(hiss_create(ctypes.byref(h), _p(self.stream.cuda_stream)), None, "hiss_create")
        self._h = h
        self.n = 0
        self.d = 0

    def close(self):
        if getattr(self, "_h", None):
            hiss_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def build(self, points):
        """points: torch CUDA float32 (n, d) tensor, or a numpy float32 (n, d) array."""
        if isinstance(points, np.ndarray):
            x = np.ascontiguousarray(points, dtype=np.float32)
            _check(hiss_build_host(self._h, x.ctypes.data, x.shape[0], x.shape[1]), self._h, "hiss_build_host")
            self.n, self.d = x.shape
            return self
        import torch
        assert points.is_cuda and points.dtype == torch.float32 and points.dim() == 2
        x = points.contiguous()
        _check(hiss_build(self._h, x.data_ptr(), x.shape[0], x.shape[1]), self._h, "hiss_build")
        self.n, self.d = x.shape
        return self

    def count(self, eps, out=None):
        """Count bound B_q of every point (int64 torch CUDA tensor, original order)."""
        import torch
        if out is None:
            out = torch.empty(self.n, dtype=torch.int64, device="cuda")
        _check(hiss_count(self._h, float(eps), out.data_ptr() if out is not False else None), self._h,
               "hiss_count")
        return out

    def join(self, eps, batch_bytes=0, mode=HISS_OUT_CSR, copy_to_host=False, on_batch=None):
        """Run the join; on_batch(hiss_batch) is called once per batch (raw
        struct, pointers valid during the call).  Returns the stats dict."""
        err = []

        def cb(user, bptr):
            try:
                on_batch(bptr.contents)
                return 0
            except BaseException as e:  # surfaced after the join returns
                err.append(e)
                return 1

        out = hiss_out(mode, 1 if copy_to_host else 0,
                       HISS_BATCH_FN(cb) if on_batch is not None else HISS_BATCH_FN(), None)
        rc = hiss_join(self._h, float(eps), int(batch_bytes), ctypes.byref(out))
        if err:
            raise err[0]
        _check(rc, self._h, "hiss_join")
        return self.stats()

    def _run(self, call, on_batch):
        err = []

        def cb(user, bptr):
            try:
                on_batch(bptr.contents)
                return 0
            except BaseException as e:  # surfaced after the call returns
                err.append(e)
                return 1

        fn = HISS_BATCH_FN(cb) if on_batch is not None else HISS_BATCH_FN()
        rc = call(fn)
        if err:
            raise err[0]
        return rc

    def join_shard(self, eps, rank, nranks, batch_bytes=0, mode=HISS_OUT_CSR, copy_to_host=False, on_batch=None):
        """Shard rank of nranks of the self-join (hiss_join_shard); on_batch as
        in ``join``.  Returns the stats dict."""
        def call(fn):
            out = hiss_out(mode, 1 if copy_to_host else 0, fn, None)
            return hiss_join_shard(self._h, float(eps), int(batch_bytes), ctypes.byref(out), int(rank), int(nranks))

        _check(self._run(call, on_batch), self._h, "hiss_join_shard")
        return self.stats()

    def join_shard_sets(self, eps, rank, nranks, batch_bytes=0):
        """Rows of one shard as {query id: numpy array of neighbour ids}."""
        res = {}

        def take(b):
            q = _host_array(b.query_ids, b.nq, np.int64)
            rp = _host_array(b.row_ptr, b.nq + 1, np.int64)
            cols = _host_array(b.cols, b.nnz, np.int32)
            for i in range(b.nq):
                res[int(q[i])] = cols[rp[i]:rp[i + 1]]

        self.join_shard(eps, rank, nranks, batch_bytes, HISS_OUT_CSR, True, take)
        return res

    def join_queries(self, queries, eps, batch_bytes=0, mode=HISS_OUT_CSR, copy_to_host=False, on_batch=None):
        """Semi-join of the query points (torch CUDA float32 (nq, d)) against
        the built dataset; on_batch as in ``join``.  Returns the stats dict."""
        q = queries.contiguous()
        assert q.is_cuda and q.dim() == 2 and q.shape[1] == self.d

        def call(fn):
            out = hiss_out(mode, 1 if copy_to_host else 0, fn, None)
            return hiss_join_queries(self._h, q.data_ptr() if q.numel() else None, q.shape[0], float(eps),
                                     int(batch_bytes), ctypes.byref(out))

        _check(self._run(call, on_batch), self._h, "hiss_join_queries")
        return self.stats()

    def join_queries_sets(self, queries, eps, batch_bytes=0):
        """Semi-join result as {query row: numpy array of data ids}."""
        res = {}

        def take(b):
            q = _host_array(b.query_ids, b.nq, np.int64)
            rp = _host_array(b.row_ptr, b.nq + 1, np.int64)
            cols = _host_array(b.cols, b.nnz, np.int32)
            for i in range(b.nq):
                res[int(q[i])] = cols[rp[i]:rp[i + 1]]

        self.join_queries(queries, eps, batch_bytes, HISS_OUT_CSR, True, take)
        return res

    def count_queries(self, queries, eps):
        import torch
        q = queries.contiguous()
        out = torch.empty(q.shape[0], dtype=torch.int64, device="cuda")
        _check(hiss_count_queries(self._h, q.data_ptr() if q.numel() else None, q.shape[0], float(eps),
                                  out.data_ptr() if q.numel() else None), self._h, "hiss_count_queries")
        return out

    def join_sets(self, eps, batch_bytes=0):
        """Full result as {query id: numpy array of neighbour ids}, through
        host delivery (copy_to_host = 1)."""
        res = {}

        def take(b):
            q = _host_array(b.query_ids, b.nq, np.int64)
            rp = _host_array(b.row_ptr, b.nq + 1, np.int64)
            cols = _host_array(b.cols, b.nnz, np.int32)
            for i in range(b.nq):
                res[int(q[i])] = cols[rp[i]:rp[i + 1]]

        self.join(eps, batch_bytes, HISS_OUT_CSR, True, take)
        return res

    def join_csr(self, eps, batch_bytes=0):
        """Full result as (row_ptr int64[n+1], cols int32[nnz]) in original
        query order, neighbours of each row sorted ascending (host arrays)."""
        rows = self.join_sets(eps, batch_bytes)
        n = self.n
        cnt = np.zeros(n + 1, dtype=np.int64)
        for q, c in rows.items():
            cnt[q + 1] = c.size
        row_ptr = np.cumsum(cnt)
        cols = np.empty(int(row_ptr[-1]), dtype=np.int32)
        for q, c in rows.items():
            cols[row_ptr[q]:row_ptr[q + 1]] = np.sort(c)
        return row_ptr, cols

    def index(self):
        v = hiss_index_view()
        _check(hiss_index(self._h, ctypes.byref(v)), self._h, "hiss_index")
        n, C = v.n, v.cells
        return {"n": n, "cells": C,
                "ids": _device_tensor(v.ids, n, "<i4"),
                "cell_start": _device_tensor(v.cell_start, C + 1, "<i4"),
                "cell_of_row": _device_tensor(v.cell_of_row, n, "<i4"),
                "nbr": _device_tensor(v.nbr, C * 27, "<i4"),
                "nbr_count": _device_tensor(v.nbr_count, C, "<i4"),
                "cell_bound": _device_tensor(v.cell_bound, C, "<i8"),
                "cell_key": _device_tensor(v.cell_key, C, "<i8"),
                "perm": list(v.perm), "sub_bits": v.sub_bits, "cell_width": v.cell_width,
                "origin": list(v.origin)}

    def stats(self):
        s = hiss_stats()
        _check(hiss_last_stats(self._h, ctypes.byref(s)), self._h, "hiss_last_stats")
        return {k: getattr(s, k) for k, _ in hiss_stats._fields_}

    def work_profile(self, eps):
        """(sum of per-pair early-exit dimensions, dimensions the join's
        refinement evaluates) over all candidate pairs for eps."""
        out = (_i64 * 2)()
        _check(hiss_work_profile(self._h, float(eps), out), self._h, "hiss_work_profile")
        return int(out[0]), int(out[1])

    def launches(self):
        return int(hiss_launch_count(self._h))

    def set_alloc_limit(self, nbytes):
        _check(hiss_set_option(self._h, HISS_OPT_ALLOC_LIMIT, int(nbytes)), self._h, "hiss_set_option")

    def knn(self, k, eps0=0.0):
        """Exact k nearest neighbours of every point (hiss_knn): (ids int64
        (n, k), squared distances float32 (n, k)) as torch CUDA tensors."""
        import torch
        ids = torch.empty((self.n, k), dtype=torch.int64, device="cuda")
        d2 = torch.empty((self.n, k), dtype=torch.float32, device="cuda")
        _check(hiss_knn(self._h, int(k), float(eps0), ids.data_ptr(), d2.data_ptr()), self._h, "hiss_knn")
        return ids, d2

    def set_refine(self, tensor_cores):
        """Select the refinement: CUDA cores (default) or the tensor-core
        prefilter with exact recheck (HISS_OPT_REFINE)."""
        mode = HISS_REFINE_TENSOR_CORES if tensor_cores else HISS_REFINE_CUDA_CORES
        _check(hiss_set_option(self._h, HISS_OPT_REFINE, mode), self._h, "hiss_set_option")
        return self

    # building blocks
    def sort_pairs(self, keys, vals, key_bits):
        _check(hiss_sort_pairs(self._h, keys.data_ptr(), vals.data_ptr(), keys.numel(), key_bits), self._h,
               "hiss_sort_pairs")

    def exclusive_scan(self, x, out):
        _check(hiss_exclusive_scan(self._h, x.data_ptr(), out.data_ptr(), x.numel()), self._h,
               "hiss_exclusive_scan")

    def mask_positions(self, words, nbits, pos):
        cnt = _i64()
        _check(hiss_mask_positions(self._h, words.data_ptr(), int(nbits), pos.data_ptr(), ctypes.byref(cnt)),
               self._h, "hiss_mask_positions")
        return int(cnt.value)

    # operators between a model's parameters and the points: asynchronous on
    # the context's stream (``finish`` waits).  Called with another current
    # stream, that stream's earlier work is waited for on the device first and
    # its later work waits for the call.  They can be captured in a graph after
    # a call of the same sizes that was not; the graph is replayed on the context's
    # stream, or ordered with it, while the Join is open.

    def _enqueue(self, fn, args, what, tensors):
        """fn(context, *args): tensors are those that it reads or writes."""
        if self._current(self._index) == self._raw:
            rc = fn(self._h, *args)
            if rc:
                raise HissError(rc, self._h, what)
            return
        cur = self._torch.cuda.current_stream(self._index)
        self.stream.wait_stream(cur)
        rc = fn(self._h, *args)
        for t in tensors:  # keep the allocator from reusing them before the context's stream is done
            if t is not None:
                t.record_stream(self.stream)
        cur.wait_stream(self.stream)
        _check(rc, self._h, what)

    def _here(self, what, *tensors):
        for t in tensors:
            if t is not None and t.get_device() != self._index:
                raise ValueError("%s: CUDA tensors on the context's device expected" % what)

    def _tokens(self, tokens):
        """(contiguous tokens, bits)."""
        if tokens.dtype == self._torch.int64:
            return tokens if tokens.is_contiguous() else tokens.contiguous(), 64
        if tokens.dtype == self._torch.int32:
            return tokens if tokens.is_contiguous() else tokens.contiguous(), 32
        raise ValueError("int32 or int64 tokens expected, not %s" % tokens.dtype)

    def _out(self, out, shape, dtype, default, width, what):
        """(out checked, or a new tensor; its rows; their stride; their hiss_dtype)."""
        if out is None:
            dtype = dtype or default
            code = _dtype(dtype)
            out = self._torch.empty(*shape, dtype=dtype, device=self._device)  # sizes apart: parsed faster than a Size
            return out, out, width, code
        if out.shape != shape or (dtype is not None and out.dtype != dtype):
            raise ValueError("out: shape or type differs from the result's")
        self._here(what, out)
        return (out, *_out_matrix(out, "out"), _dtype(out.dtype))

    def embed(self, tokens, table, scale=1.0, pad=None, dtype=None, out=None):
        """scale * table[tokens] (hiss_embed): tokens int32 or int64 of any
        shape, table (vocab, width); zeros where tokens == pad.  dtype: the result's
        type (default: the table's); out: a tensor of shape
        (*tokens.shape, width) that receives it."""
        t, bits = self._tokens(tokens)
        if table.dim() != 2:
            raise ValueError("table: (vocab, width) expected")
        w, vocab, width, stride = _matrix(table, "table")
        kind = table.dtype
        code = _dtype(kind)
        self._here("hiss_embed", t, w)
        out, o, o_stride, o_code = self._out(out, (*t.shape, width), dtype, kind, width, "hiss_embed")
        self._enqueue(hiss_embed, (w.data_ptr(), code, vocab, width, stride, t.data_ptr(), bits, t.numel(),
                                   _pad(pad), scale, o.data_ptr(), o_code, o_stride),
                      "hiss_embed", (t, w, o))
        return out

    def embed_grad(self, tokens, dy, vocab, scale=1.0, pad=None, dtype=None, out=None, accumulate=False):
        """Gradient of ``embed`` with respect to its table (hiss_embed_grad):
        dy (*tokens.shape, width); returns (vocab, width) of the given dtype
        (default: dy's), or out, to which it is added with accumulate."""
        t, bits = self._tokens(tokens)
        g, n, width, stride = _matrix(dy, "dy")
        if dy.shape[:-1] != t.shape:
            raise ValueError("dy: shape (*tokens.shape, width) expected")
        if out is None and accumulate:
            raise ValueError("accumulate needs out")
        kind = dy.dtype
        code = _dtype(kind)
        self._here("hiss_embed_grad", t, g)
        out, o, o_stride, o_code = self._out(out, (max(vocab, 0), width), dtype, kind, width, "hiss_embed_grad")
        self._enqueue(hiss_embed_grad, (g.data_ptr(), code, stride, t.data_ptr(), bits, n,
                                        _pad(pad), scale, vocab, width,
                                        1 if accumulate else 0, o.data_ptr(), o_code, o_stride),
                      "hiss_embed_grad", (t, g, o))
        return out

    def layer_norm(self, x, weight=None, bias=None, eps=1e-5, dtype=None, out=None):
        """Layer norm over the last dimension (hiss_layer_norm): (y, mean,
        rstd), the statistics float32 of shape x.shape[:-1].  dtype: y's type, x's
        (default) or float32."""
        m, n, width, stride = _matrix(x, "x")
        kind, shape, torch = x.dtype, x.shape, self._torch
        code = _dtype(kind)
        p, w_ptr, b_ptr = self._params(width, weight, bias)
        self._here("hiss_layer_norm", m, weight, bias)
        out, o, o_stride, o_code = self._out(out, shape, dtype, kind, width, "hiss_layer_norm")
        rows = shape[:-1]
        mean = torch.empty(*rows or ((),), dtype=torch.float32, device=self._device)
        rstd = torch.empty_like(mean)
        self._enqueue(hiss_layer_norm, (m.data_ptr(), code, stride, n, width, w_ptr, b_ptr, p, eps, o.data_ptr(),
                                        o_code, o_stride, mean.data_ptr(), rstd.data_ptr()),
                      "hiss_layer_norm", (m, weight, bias, o, mean, rstd))
        return out, mean, rstd

    def layer_norm_grad(self, dy, x, mean, rstd, weight=None, param_dtype=None):
        """Gradient of ``layer_norm`` (hiss_layer_norm_grad): (dx, dweight,
        dbias).  dweight and dbias have the weight's type, or param_dtype
        (default: float32) without a weight."""
        torch, shape, kind = self._torch, x.shape, x.dtype
        m, n, width, stride = _matrix(x, "x")
        g, _, _, g_stride = _matrix(dy, "dy")
        rows = shape[:-1]
        if dy.shape != shape or mean.shape != rows or rstd.shape != rows:
            raise ValueError("dy, mean and rstd do not match x")
        f32 = torch.float32
        if mean.dtype != f32 or rstd.dtype != f32:
            raise ValueError("mean and rstd: float32 expected")
        code, g_code = _dtype(kind), _dtype(dy.dtype)
        p, w_ptr, _ = self._params(width, weight, None)
        pt = weight.dtype if weight is not None else param_dtype or f32
        if weight is None:
            p = _dtype(pt)
        if not mean.is_contiguous():
            mean = mean.contiguous()
        if not rstd.is_contiguous():
            rstd = rstd.contiguous()
        self._here("hiss_layer_norm_grad", g, m, mean, rstd, weight)
        dx = torch.empty(*shape, dtype=kind, device=self._device)
        dw = torch.empty(width, dtype=pt, device=self._device)
        db = torch.empty_like(dw)
        self._enqueue(hiss_layer_norm_grad, (g.data_ptr(), g_code, g_stride, m.data_ptr(), code, stride,
                                             mean.data_ptr(), rstd.data_ptr(), w_ptr, p, n, width, dx.data_ptr(), width,
                                             dw.data_ptr(), db.data_ptr()),
                      "hiss_layer_norm_grad", (g, m, mean, rstd, weight, dx, dw, db))
        return dx, dw, db

    def clip_grads(self, grads, max_norm):
        """Clip by the global norm (hiss_clip_grads): grads is a ``Gradients``
        or a sequence of tensors, clipped in place.  Returns the norm before
        clipping (float32 CUDA scalar)."""
        g = grads if isinstance(grads, Gradients) else Gradients(grads)
        array = g.current() if g is grads else g.array
        self._here("hiss_clip_grads", *g.grads[:1])  # one device for all: checked by Gradients
        if self._scalar is None:
            self._scalar = self._torch.empty((), dtype=self._torch.float32, device=self._device)
        norm = self._torch.empty_like(self._scalar)
        here = self._current(self._index) == self._raw  # then no list of the tensors is needed
        self._enqueue(hiss_clip_grads, (array, len(g.grads), max_norm, norm.data_ptr()), "hiss_clip_grads",
                      () if here else g.all + [norm])
        return norm

    def finish(self):
        """Wait for the context's stream (hiss_finish); raises if a token since
        the last call was neither padding nor in the table."""
        _check(hiss_finish(self._h), self._h, "hiss_finish")

    @staticmethod
    def _params(width, weight, bias):
        """(hiss_dtype, pointer, pointer) of weight and bias."""
        if weight is None:
            if bias is None:
                return HISS_F32, None, None
            return _dtype(bias.dtype), None, _vector(bias, width)
        if bias is None:
            return _dtype(weight.dtype), _vector(weight, width), None
        if weight.dtype != bias.dtype:
            raise ValueError("weight and bias of one type expected")
        return _dtype(weight.dtype), _vector(weight, width), _vector(bias, width)
