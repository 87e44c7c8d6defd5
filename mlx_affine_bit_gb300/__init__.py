"""Python binding of libtfqmm, the MLX-affine quantized row product for GB300, and
of the 8-bit cache, attention and sampling around it, and the pages, positions and
4-bit cache that serving adds.

Argument marshalling only: every step of the product runs in the library's
CUDA kernels (``csrc/``).  The names and arguments follow ``include/tfqmm.h``,
``include/tfdecode.h`` and ``include/tfserve.h``.
Tensors may be passed as torch tensors (their ``data_ptr()`` is used) or as
raw integer addresses; ``KvCache``, ``KvBatch``, ``sample``, ``KvPages``, ``Rope`` and
``Kv4Cache`` take tensors, and check their types, shapes, strides and devices.  ``stream`` is a
``torch.cuda.Stream``, a raw ``cudaStream_t`` integer, or None for torch's current
stream.

The library must be built first (``mlx_affine_bit_gb300.build.build()``);
loading fails loudly when it is missing.  There is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
SO = os.path.join(HERE, "_build", "libtfqmm.so")
SO_DEBUG = os.path.join(HERE, "_build", "libtfqmm_debug.so")   # bounds-checking build (tfqmm_debug.h)
SO_TRACE = os.path.join(HERE, "_build", "libtfqmm_trace.so")   # phase-trace build (tfqmm_trace.h)

TF_OK = 0
STATUS = {
    -1: "TF_EINVAL_BITS", -2: "TF_EINVAL_GROUP", -3: "TF_EINVAL_ROWS", -4: "TF_EINVAL_STRIDE",
    -5: "TF_EINVAL_PTR", -6: "TF_EINVAL_SIZE", -7: "TF_ENARROW", -8: "TF_EGROUP",
    -9: "TF_ESTACK", -10: "TF_ECUDA", -11: "TF_EDEVICE", -12: "TF_EINVAL_FLAGS", -13: "TF_EGATHER",
    -14: "TF_EBOUNDS",
}
SYMBOLS = ("tf_qmm", "tf_qmm_ex", "tf_qmm_prompt", "tf_qmm_gather", "tf_qmm_noalloc", "tf_noalloc_status", "tf_qmm_stack", "tf_widen",
           "tf_widen_host", "tf_common_width", "tf_qmm_bytes", "tf_device_status", "tf_set_launch_mode",
           "tf_inject_stall", "tf_last_error_string", "tf_version",
           "tf_kv_append", "tf_kv_read", "tf_kv_attend", "tf_sample",
           "tf_kv_plan", "tf_rope", "tf_kv4_append", "tf_kv4_read", "tf_kv4_attend")
TF_LAUNCH_PDL, TF_LAUNCH_EARLY_WEIGHTS, TF_LAUNCH_EARLY_X = 1, 2, 4
TF_OUT_BF16, TF_EPI_RELU2 = 1, 2
TF_IN_F32, TF_KV_CAUSAL, TF_IN_BF16 = 4, 8, 16
TF_KV_BY_ROWS, TF_KV_BY_TILES = 64, 128
TF_ROPE_PAIRS, TF_ROPE_BACK = 256, 512


class TfError(RuntimeError):
    def __init__(self, rc: int, msg: str):
        super().__init__("%s (%d): %s" % (STATUS.get(rc, "?"), rc, msg))
        self.rc = rc


class TfRun(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p),
                ("N", ctypes.c_int), ("bits", ctypes.c_int), ("group", ctypes.c_int)]


class TfMember(ctypes.Structure):
    _fields_ = [("run", ctypes.c_int), ("src_col", ctypes.c_int), ("n_cols", ctypes.c_int),
                ("dst_col", ctypes.c_int)]


class TfKv(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "open_k", "open_v", "open_max")] + \
               [(n, ctypes.c_int) for n in ("n_blocks", "n_slots", "kv_heads", "block", "dim", "f32")]


class TfKvBatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n_seqs", "rows", "max_rows", "max_len")] + \
               [(n, ctypes.c_void_p) for n in ("row_start", "kv_len", "table")] + \
               [("table_stride", ctypes.c_int64), ("slots", ctypes.c_void_p)]


class TfKvPages(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64)] + \
               [(n, ctypes.c_void_p) for n in ("kv_len", "free_pages", "n_free")] + \
               [(n, ctypes.c_int) for n in ("n_seqs", "n_blocks", "max_pages", "block")]


class TfKv4(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_affine", "v_affine")] + \
               [(n, ctypes.c_int) for n in ("n_blocks", "kv_heads", "block", "dim")]


_lib = None
_debug_lib = None
_trace_lib = None


def lib():
    """The loaded libtfqmm (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = _load(SO)
    return _lib


def debug_lib():
    """The loaded bounds-checking build, libtfqmm_debug.so (same entry points, plus tf_debug_shrink_y)."""
    global _debug_lib
    if _debug_lib is None:
        _debug_lib = _load(SO_DEBUG)
        _debug_lib.tf_debug_shrink_y.argtypes = [ctypes.c_int]
        _debug_lib.tf_debug_shrink_y.restype = ctypes.c_int
    return _debug_lib


def trace_lib():
    """The loaded phase-trace build, libtfqmm_trace.so (same entry points, plus tf_trace_reset / tf_trace_read)."""
    global _trace_lib
    if _trace_lib is None:
        _trace_lib = _load(SO_TRACE)
        _trace_lib.tf_trace_reset.argtypes = []
        _trace_lib.tf_trace_reset.restype = ctypes.c_int
        _trace_lib.tf_trace_read.argtypes = [ctypes.c_void_p, ctypes.c_int]
        _trace_lib.tf_trace_read.restype = ctypes.c_int
    return _trace_lib


class using:
    """Context manager: the calls of this module go to library L (a build from
    debug_lib() or trace_lib()) inside the block."""

    def __init__(self, L):
        self.L = L

    def __enter__(self):
        global _lib
        self.old, _lib = _lib, self.L
        return self.L

    def __exit__(self, *exc):
        global _lib
        _lib = self.old
        return False


def _load(path):
    """Open one build of the library and declare its entry points' argument types."""
    if not os.path.exists(path):
        raise ImportError("%s is not built; run mlx_affine_bit_gb300.build.build()" % path)
    L = ctypes.CDLL(path)
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    L.tf_qmm.argtypes = [P, i32, i32, P, P, P, i32, i32, i32, P, i64, P]
    L.tf_qmm_noalloc.argtypes = [P, i32, i32, P, P, P, i32, i32, i32, P, i64, P]
    L.tf_qmm_ex.argtypes = [P, i32, i32, P, P, P, i32, i32, i32, P, i64, i32, P]
    L.tf_qmm_prompt.argtypes = [P, i32, i32, P, P, P, i32, i32, i32, P, i64, i32, P]
    L.tf_qmm_gather.argtypes = [P, i32, i32, ctypes.POINTER(TfRun), i32, ctypes.POINTER(ctypes.c_int),
                                ctypes.POINTER(ctypes.c_int), i32, P, i64, i32, P]
    L.tf_qmm_stack.argtypes = [P, i32, i32, ctypes.POINTER(TfRun), i32,
                               ctypes.POINTER(TfMember), i32, P, i64, P]
    L.tf_widen.argtypes = [P, P, P, i32, i32, i32, i32, P, P, P, i32, i32, P]
    L.tf_widen_host.argtypes = [P, P, P, i32, i32, i32, i32, P, P, P, i32, i32]
    L.tf_common_width.argtypes = [P, P, i32, P, P]
    L.tf_qmm_bytes.argtypes = [i32, i32, i32, i32, P, P]
    L.tf_device_status.argtypes = []
    L.tf_noalloc_status.argtypes = []
    L.tf_set_launch_mode.argtypes = [i32]
    L.tf_inject_stall.argtypes = []
    kv, batch = ctypes.POINTER(TfKv), ctypes.POINTER(TfKvBatch)
    L.tf_kv_append.argtypes = [kv, batch, P, i64, P, i64, P]
    L.tf_kv_read.argtypes = [kv, batch, P, i64, P, i64, i32, P]
    L.tf_kv_attend.argtypes = [kv, batch, P, i64, i32, P, i64, ctypes.c_float, i32, i32, P]
    L.tf_sample.argtypes = [P, i32, i32, i64, P, P, P, P, P, P, P, i32, P]
    pages, kv4 = ctypes.POINTER(TfKvPages), ctypes.POINTER(TfKv4)
    L.tf_kv_plan.argtypes = [pages, P, i32, i32, i32, P, P, P, P, P]
    L.tf_rope.argtypes = [P, i32, ctypes.c_float, P, i32, P, i64, P, i64, i32, i32, i32, P]
    L.tf_kv4_append.argtypes = [kv4, P, i32, P, i64, P, i64, i32, P]
    L.tf_kv4_read.argtypes = [kv4, batch, P, i64, P, i64, i32, P]
    L.tf_kv4_attend.argtypes = [kv4, batch, P, i64, i32, P, i64, ctypes.c_float, i32, i32, P]
    L.tf_last_error_string.restype = ctypes.c_char_p
    L.tf_version.restype = ctypes.c_char_p
    for name in ("tf_qmm", "tf_qmm_ex", "tf_qmm_prompt", "tf_qmm_gather", "tf_qmm_noalloc", "tf_qmm_stack", "tf_widen",
                 "tf_widen_host", "tf_common_width", "tf_qmm_bytes", "tf_device_status", "tf_noalloc_status",
                 "tf_set_launch_mode", "tf_inject_stall", "tf_kv_append", "tf_kv_read", "tf_kv_attend", "tf_sample",
                 "tf_kv_plan", "tf_rope", "tf_kv4_append", "tf_kv4_read", "tf_kv4_attend"):
        getattr(L, name).restype = i32
    return L


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = None


def _current_stream() -> int:
    """torch's current stream of the current device.  (Its handle without a Stream object, where torch
    gives it: 0.3 us instead of 3.)"""
    global _raw_stream
    if _raw_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        torch.cuda.current_stream()             # (initializes CUDA)
        if raw is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream   # noqa: E731
        else:
            device = torch._C._cuda_getDevice
            _raw_stream = lambda: raw(device())                             # noqa: E731
    return _raw_stream()


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int) -> None:
    if rc != TF_OK:
        raise TfError(rc, lib().tf_last_error_string().decode())


def tf_qmm(x, rows, K, W, scales, biases, N, bits, group, y, y_stride, stream=None) -> None:
    _check(lib().tf_qmm(_ptr(x), rows, K, _ptr(W), _ptr(scales), _ptr(biases), N, bits, group,
                        _ptr(y), y_stride, _stream(stream)))


def tf_qmm_noalloc(x, rows, K, W, scales, biases, N, bits, group, y, y_stride, stream=None) -> None:
    """tf_qmm with no device allocation (fixed built-in scratch; see include/tfqmm.h)."""
    _check(lib().tf_qmm_noalloc(_ptr(x), rows, K, _ptr(W), _ptr(scales), _ptr(biases), N, bits,
                                group, _ptr(y), y_stride, _stream(stream)))


def tf_qmm_ex(x, rows, K, W, scales, biases, N, bits, group, y, y_stride, flags, stream=None) -> None:
    """tf_qmm with output flags (TF_OUT_BF16: y is bf16; TF_EPI_RELU2: squared ReLU)."""
    _check(lib().tf_qmm_ex(_ptr(x), rows, K, _ptr(W), _ptr(scales), _ptr(biases), N, bits, group,
                           _ptr(y), y_stride, flags, _stream(stream)))


def tf_qmm_prompt(x, rows, K, W, scales, biases, N, bits, group, y, y_stride, flags=0, stream=None) -> None:
    """Many-row product on the tcgen05 tensor cores, weights read once per 64 rows (see include/tfqmm.h)."""
    _check(lib().tf_qmm_prompt(_ptr(x), rows, K, _ptr(W), _ptr(scales), _ptr(biases), N, bits, group,
                               _ptr(y), y_stride, flags, _stream(stream)))


def tf_qmm_gather(x, x_rows, K, experts, slot_expert, slot_row, y, y_stride, flags=0, stream=None) -> None:
    """experts: [(W, scales, biases, N, bits, group)]; slot i: y row i = experts[slot_expert[i]] x row slot_row[i]."""
    ee = (TfRun * len(experts))(*[TfRun(_ptr(W), _ptr(s), _ptr(b), N, bits, g)
                                  for (W, s, b, N, bits, g) in experts])
    n = len(slot_expert)
    se = (ctypes.c_int * n)(*slot_expert)
    sr = (ctypes.c_int * len(slot_row))(*slot_row)
    _check(lib().tf_qmm_gather(_ptr(x), x_rows, K, ee, len(experts), se, sr, n, _ptr(y), y_stride, flags,
                               _stream(stream)))


def tf_qmm_stack(x, rows, K, runs, members, y, y_stride, stream=None) -> None:
    """runs: [(W, scales, biases, N, bits, group)]; members: [(run, src_col, n_cols, dst_col)]."""
    rr = (TfRun * len(runs))(*[TfRun(_ptr(W), _ptr(s), _ptr(b), N, bits, g)
                               for (W, s, b, N, bits, g) in runs])
    mm = (TfMember * len(members))(*[TfMember(*m) for m in members])
    _check(lib().tf_qmm_stack(_ptr(x), rows, K, rr, len(runs), mm, len(members), _ptr(y),
                              y_stride, _stream(stream)))


def tf_widen(W, scales, biases, N, K, bits, group, W_out, s_out, b_out, bits_out, group_out,
             stream=None) -> None:
    _check(lib().tf_widen(_ptr(W), _ptr(scales), _ptr(biases), N, K, bits, group, _ptr(W_out),
                          _ptr(s_out), _ptr(b_out), bits_out, group_out, _stream(stream)))


def tf_widen_host(W, scales, biases, N, K, bits, group, bits_out, group_out):
    """Widen / regroup on host numpy arrays (uint32 W, uint16 scales/biases); returns (W_out, s_out, b_out)."""
    import numpy as np
    W = np.ascontiguousarray(W, dtype=np.uint32)
    s = np.ascontiguousarray(scales, dtype=np.uint16)
    b = np.ascontiguousarray(biases, dtype=np.uint16)
    Wo = np.zeros((N, K * bits_out // 32), dtype=np.uint32)
    so = np.zeros((N, K // group_out), dtype=np.uint16)
    bo = np.zeros((N, K // group_out), dtype=np.uint16)
    _check(lib().tf_widen_host(W.ctypes.data, s.ctypes.data, b.ctypes.data, N, K, bits, group, Wo.ctypes.data,
                               so.ctypes.data, bo.ctypes.data, bits_out, group_out))
    return Wo, so, bo


def tf_common_width(bits_list, groups_list) -> tuple[int, int]:
    n = len(bits_list)
    b = (ctypes.c_int * n)(*bits_list)
    g = (ctypes.c_int * n)(*groups_list)
    bo, go = ctypes.c_int(), ctypes.c_int()
    _check(lib().tf_common_width(b, g, n, ctypes.byref(bo), ctypes.byref(go)))
    return bo.value, go.value


def tf_qmm_bytes(N, K, bits, group) -> tuple[int, int]:
    wb, sb = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().tf_qmm_bytes(N, K, bits, group, ctypes.byref(wb), ctypes.byref(sb)))
    return wb.value, sb.value


def tf_device_status() -> None:
    _check(lib().tf_device_status())


def tf_noalloc_status() -> None:
    """Raise TfError(TF_EDEVICE) if a tf_qmm_noalloc product gave up a bounded wait (clears it)."""
    _check(lib().tf_noalloc_status())


def tf_set_launch_mode(mode: int) -> int:
    """Set the launch mode (TF_LAUNCH_* bits) of later calls; returns the previous mode."""
    rc = lib().tf_set_launch_mode(mode)
    if rc < 0:
        _check(rc)
    return rc


def tf_inject_stall() -> None:
    """Test hook: the next product's first stage is withheld (its bounded wait runs out)."""
    _check(lib().tf_inject_stall())


def tf_kv_append(kv: TfKv, batch: TfKvBatch, k, k_stride, v, v_stride, stream=None) -> None:
    """Quantize new tokens' keys and values into the cache (see include/tfdecode.h)."""
    _check(lib().tf_kv_append(kv, batch, _ptr(k), k_stride, _ptr(v), v_stride, _stream(stream)))


def tf_kv_read(kv: TfKv, batch: TfKvBatch, k_out, k_stride, v_out, v_stride, flags=0, stream=None) -> None:
    """Read the batch's tokens back as fp32 (bf16 with TF_OUT_BF16) rows; either output may be None."""
    _check(lib().tf_kv_read(kv, batch, _ptr(k_out), k_stride, _ptr(v_out), v_stride, flags, _stream(stream)))


def tf_kv_attend(kv: TfKv, batch: TfKvBatch, q, q_stride, heads, out, out_stride, scale, window=0, flags=TF_KV_CAUSAL,
                 stream=None) -> None:
    """Attention of the batch's rows over the cache; out is bf16 (see include/tfdecode.h)."""
    _check(lib().tf_kv_attend(kv, batch, _ptr(q), q_stride, heads, _ptr(out), out_stride, scale, window, flags,
                              _stream(stream)))


def tf_sample(logits, rows, vocab, stride, u, temperature, top_k, top_p, min_p, tokens, probs=None, flags=0,
              stream=None) -> None:
    """One token per row of logits from the random numbers u (see include/tfdecode.h)."""
    _check(lib().tf_sample(_ptr(logits), rows, vocab, stride, _ptr(u), _ptr(temperature), _ptr(top_k), _ptr(top_p),
                           _ptr(min_p), _ptr(tokens), _ptr(probs), flags, _stream(stream)))


def tf_kv_plan(pages: TfKvPages, change, rows, max_rows, max_len, row_start, positions, slots, info, stream=None) -> None:
    """One step of growing and shrinking sequences: their pages, row starts, positions and slots (see include/tfserve.h)."""
    _check(lib().tf_kv_plan(pages, _ptr(change), rows, max_rows, max_len, _ptr(row_start), _ptr(positions), _ptr(slots),
                            _ptr(info), _stream(stream)))


def tf_rope(turns, rot, factor, positions, rows, x, x_stride, out, out_stride, heads, dim, flags=0, stream=None) -> None:
    """Rotary positions of rows of heads (see include/tfserve.h)."""
    _check(lib().tf_rope(_ptr(turns), rot, factor, _ptr(positions), rows, _ptr(x), x_stride, _ptr(out), out_stride, heads,
                         dim, flags, _stream(stream)))


def tf_kv4_append(kv: TfKv4, slots, rows, k, k_stride, v, v_stride, flags=0, stream=None) -> None:
    """Quantize rows of keys and values into their slots of the 4-bit cache (see include/tfserve.h)."""
    _check(lib().tf_kv4_append(kv, _ptr(slots), rows, _ptr(k), k_stride, _ptr(v), v_stride, flags, _stream(stream)))


def tf_kv4_read(kv: TfKv4, batch: TfKvBatch, k_out, k_stride, v_out, v_stride, flags=0, stream=None) -> None:
    """Read the batch's tokens back from the 4-bit cache; either output may be None."""
    _check(lib().tf_kv4_read(kv, batch, _ptr(k_out), k_stride, _ptr(v_out), v_stride, flags, _stream(stream)))


def tf_kv4_attend(kv: TfKv4, batch: TfKvBatch, q, q_stride, heads, out, out_stride, scale, window=0, flags=TF_KV_CAUSAL,
                  stream=None) -> None:
    """Attention of the batch's rows over the 4-bit cache; out is bf16 (see include/tfserve.h)."""
    _check(lib().tf_kv4_attend(kv, batch, _ptr(q), q_stride, heads, _ptr(out), out_stride, scale, window, flags,
                               _stream(stream)))


def tf_version() -> str:
    return lib().tf_version().decode()


def qmm(x, W, scales, biases, bits, group, y=None, y_stride=None, stream=None):
    """Convenience wrapper on torch tensors: x [rows][K] bf16, W [N][K*bits/32] int32.

    Allocates y [rows][N] fp32 when not given, then calls tf_qmm.
    """
    import torch
    rows, K = x.shape
    N = W.shape[0]
    if y is None:
        y = torch.empty((rows, N), dtype=torch.float32, device=x.device)
        y_stride = N
    tf_qmm(x, rows, K, W, scales, biases, N, bits, group, y,
           y_stride if y_stride is not None else y.stride(0), stream)
    return y


def _tensor(t, name, dtypes, shape=None, contiguous=True, device=None):
    """Refuse a tensor that a call could not take: TypeError for its type, ValueError for the rest.
    device: the number of the device that it must be on (get_device())."""
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if shape is not None and t.shape != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device is not None and t.get_device() != device:
        raise ValueError("%s must be on %s, is on %s" % (name, "the host" if device < 0 else "cuda:%d" % device, t.device))
    return t


_get_device = None


def _on_gpu(device, what):
    """Refuse tensors that are not on the current GPU, where the kernels run."""
    global _get_device
    if device < 0:
        raise ValueError("%s must be on a GPU" % what)
    if _get_device is None:
        import torch
        _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    if device != _get_device():
        raise ValueError("%s is on cuda:%d, which is not the current device" % (what, device))


def _rows(t, name, dtypes, rows, width, device):
    """The row stride of a [rows][width] matrix on that device whose rows are contiguous."""
    if t.dtype not in dtypes or t.shape != (rows, width):
        _tensor(t, name, dtypes, (rows, width), contiguous=False)
    stride = t.stride()
    if width > 1 and stride[1] != 1:
        raise ValueError("%s must have contiguous rows" % name)
    if t.get_device() != device:
        _tensor(t, name, dtypes, contiguous=False, device=device)
    return stride[0] if rows > 1 else max(width, stride[0])


class KvBatch:
    """The rows of one call on a KvCache (tf_kv_batch), on torch tensors.

    kv_len [seqs] int32 (the new tokens included), table [seqs][pages] int32,
    max_len a bound of kv_len; row_start [seqs + 1] int32 with rows and
    max_rows, or max_rows (1) rows for each sequence; slots [seqs] int32, or
    None for 0, 1, ...  block: tokens of a page, where the table was made for pages of one size (a cache of
    another is then refused).  The tensors are kept, and read by the device at each call."""

    def __init__(self, kv_len, table, max_len, row_start=None, rows=None, max_rows=1, slots=None, block=None):
        import torch
        i32 = (torch.int32,)
        n = kv_len.shape[0]
        _tensor(kv_len, "kv_len", i32, (n,))
        self.device = kv_len.get_device()
        _tensor(table, "table", i32, (n, table.shape[-1]), contiguous=False, device=self.device)
        if table.shape[1] > 1 and table.stride(1) != 1:
            raise ValueError("table must have contiguous rows")
        if row_start is not None:
            _tensor(row_start, "row_start", i32, (n + 1,), device=self.device)
            if rows is None:
                raise ValueError("row_start needs rows")
        if slots is not None:
            _tensor(slots, "slots", i32, (n,), device=self.device)
        if max_len > table.shape[1] * 128:
            raise ValueError("max_len exceeds the table")
        self.rows = n * max_rows if row_start is None else rows
        self._keep = (kv_len, table, row_start, slots)
        self._pages, self.block = table.shape[1], block
        self.c = TfKvBatch(n, self.rows, max_rows, max_len, _ptr(row_start), _ptr(kv_len), _ptr(table),
                           table.stride(0) if n > 1 else table.shape[1], _ptr(slots))


class KvCache:
    """An 8-bit paged key/value cache (tf_kv) on torch tensors.

    k, v [n_blocks][kv_heads][block][dim] int8 and k_scale, v_scale
    [n_blocks][kv_heads] fp32; for append also open_k, open_v
    [n_slots][kv_heads][2 * block][dim] (bf16 or fp32, the type of the appended
    rows) and open_max [n_slots][2][kv_heads][2 * block] fp32."""

    def __init__(self, k, v, k_scale, v_scale, open_k=None, open_v=None, open_max=None):
        import torch
        if k.dim() != 4:
            raise ValueError("k must be [n_blocks][kv_heads][block][dim]")
        n_blocks, heads, block, dim = k.shape
        _tensor(k, "k", (torch.int8,))
        self.device = device = k.get_device()
        _tensor(v, "v", (torch.int8,), k.shape, device=device)
        _tensor(k_scale, "k_scale", (torch.float32,), (n_blocks, heads), device=device)
        _tensor(v_scale, "v_scale", (torch.float32,), (n_blocks, heads), device=device)
        n_slots = 0
        self.dtype = torch.bfloat16
        if open_k is not None:
            n_slots, self.dtype = open_k.shape[0], open_k.dtype
            _tensor(open_k, "open_k", (torch.bfloat16, torch.float32), (n_slots, heads, 2 * block, dim), device=device)
            _tensor(open_v, "open_v", (self.dtype,), open_k.shape, device=device)
            _tensor(open_max, "open_max", (torch.float32,), (n_slots, 2, heads, 2 * block), device=device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.open_k, self.open_v, self.open_max = open_k, open_v, open_max
        self.kv_heads, self.block, self.dim = heads, block, dim
        self.c = TfKv(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(open_k), _ptr(open_v), _ptr(open_max),
                      n_blocks, n_slots, heads, block, dim, int(self.dtype == torch.float32))

    @classmethod
    def empty(cls, n_blocks, kv_heads, dim, block=64, n_slots=1, dtype=None, device="cuda"):
        """A new cache of n_blocks pages for n_slots sequences that grow at a time."""
        import torch
        dtype = dtype or torch.bfloat16
        code = dict(dtype=torch.int8, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        shape, ring = (n_blocks, kv_heads, block, dim), (n_slots, kv_heads, 2 * block, dim)
        return cls(torch.zeros(shape, **code), torch.zeros(shape, **code), torch.zeros(shape[:2], **f32),
                   torch.zeros(shape[:2], **f32), torch.zeros(ring, dtype=dtype, device=device),
                   torch.zeros(ring, dtype=dtype, device=device),
                   torch.zeros((n_slots, 2, kv_heads, 2 * block), **f32))

    def _batch(self, batch):
        if batch.block is not None and batch.block != self.block:
            raise ValueError("the batch's pages hold %d tokens, the cache's %d" % (batch.block, self.block))
        if batch.c.max_len > batch._pages * self.block:
            raise ValueError("max_len exceeds the table's pages")
        if batch.device != self.device:
            raise ValueError("the batch's tensors must be on the cache's device")
        _on_gpu(self.device, "the cache")
        return batch.c

    def append(self, k, v, batch, stream=None) -> None:
        """Quantize rows k, v [rows][kv_heads * dim] (row stride free) in as the batch's last tokens."""
        width, types = self.kv_heads * self.dim, (self.dtype,)
        ks = _rows(k, "k", types, batch.rows, width, self.device)
        vs = _rows(v, "v", types, batch.rows, width, self.device)
        tf_kv_append(self.c, self._batch(batch), k, ks, v, vs, stream)

    def read(self, batch, dtype=None, k_out=None, v_out=None, stream=None):
        """The batch's tokens as k, v rows [rows][kv_heads * dim] of dtype (by default the type of the output that is
        given, or of the appended rows).  An output that is not given is made."""
        import torch
        given = k_out if k_out is not None else v_out
        dtype = dtype or (self.dtype if given is None else given.dtype)
        width = self.kv_heads * self.dim
        types = (torch.bfloat16, torch.float32)
        if k_out is None and v_out is None:
            k_out = torch.empty((batch.rows, width), dtype=dtype, device=self.k.device)
            v_out = torch.empty_like(k_out)
            ks = vs = width
            if dtype not in types:
                raise TypeError("read gives bf16 or fp32")
        else:
            k_out = torch.empty((batch.rows, width), dtype=dtype, device=self.k.device) if k_out is None else k_out
            v_out = torch.empty((batch.rows, width), dtype=dtype, device=self.k.device) if v_out is None else v_out
            ks = _rows(k_out, "k_out", types, batch.rows, width, self.device)
            vs = _rows(v_out, "v_out", types, batch.rows, width, self.device)
            if k_out.dtype != v_out.dtype:
                raise TypeError("k_out and v_out must have one type")
        tf_kv_read(self.c, self._batch(batch), k_out, ks, v_out, vs,
                   TF_OUT_BF16 if k_out.dtype == torch.bfloat16 else 0, stream)
        return k_out, v_out

    def attend(self, q, batch, out=None, scale=None, causal=True, window=0, stream=None, kernel=0):
        """Attention of q [rows][heads * dim] (bf16 or fp32) over the cache; out is bf16, scale 1/sqrt(dim) by default.

        kernel: 0 (by the call's sizes), TF_KV_BY_ROWS or TF_KV_BY_TILES."""
        import torch
        rows, width = q.shape
        qs = _rows(q, "q", (torch.bfloat16, torch.float32), batch.rows, width, self.device)
        if out is None:
            out = torch.empty((rows, width), dtype=torch.bfloat16, device=q.device)
            os_ = width
        else:
            os_ = _rows(out, "out", (torch.bfloat16,), rows, width, self.device)
        if width % self.dim:
            raise ValueError("q's rows must hold heads * dim values")
        tf_kv_attend(self.c, self._batch(batch), q, qs, width // self.dim, out, os_,
                     self.dim ** -0.5 if scale is None else scale, window,
                     (TF_KV_CAUSAL if causal else 0) | (TF_IN_F32 if q.dtype == torch.float32 else 0) | kernel, stream)
        return out


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, probs=None, stream=None):
    """tf_sample on torch tensors: logits [rows][vocab] fp32 or bf16 (row stride free), u [rows] fp32 random
    numbers, per-row temperature, top_p, min_p (fp32) and top_k (int32) or None.  Returns (tokens, probs)."""
    import torch
    rows, vocab = logits.shape
    device = logits.get_device()
    stride = _rows(logits, "logits", (torch.float32, torch.bfloat16), rows, vocab, device)
    f32, i32 = (torch.float32,), (torch.int32,)
    shape = (rows,)
    for t, name, types in ((u, "u", f32), (temperature, "temperature", f32), (top_k, "top_k", i32), (top_p, "top_p", f32),
                           (min_p, "min_p", f32), (tokens, "tokens", i32), (probs, "probs", f32)):
        if t is not None and (t.dtype not in types or t.shape != shape or not t.is_contiguous() or t.get_device() != device):
            _tensor(t, name, types, shape, device=device)
    _on_gpu(device, "logits")
    if tokens is None:
        tokens = torch.empty(rows, dtype=torch.int32, device=logits.device)
    if probs is None:
        probs = torch.empty(rows, dtype=torch.float32, device=logits.device)
    tf_sample(logits, rows, vocab, stride, u, temperature, top_k, top_p, min_p, tokens, probs,
              TF_IN_BF16 if logits.dtype == torch.bfloat16 else 0, stream)
    return tokens, probs


from .serve import Kv4Cache, KvPages, KvPlan, Rope   # noqa: E402,F401
