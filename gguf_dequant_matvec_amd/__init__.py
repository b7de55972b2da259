"""Python binding of libqmv.so: dequantize-fused GGUF matvec on MI355X.

Argument marshalling only -- every step runs in the HIP kernels of libqmv.so.
Each function has the name and argument order of the C entry point in
include/qmv.h; tensor arguments may be torch tensors (their data pointer is
passed) or raw integer device addresses.  `stream` defaults to torch's
current stream.  A status other than QMV_OK raises QmvError.

Importing works without a GPU (the library only needs the HIP runtime to be
loadable); the library is never replaced by a CPU fallback: if libqmv.so is
missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

Q4_0 = 2
Q4_1 = 3
Q5_0 = 6
Q5_1 = 7
Q8_0 = 8
Q8_1 = 9
Q2_K = 10
Q3_K = 11
Q4_K = 12
Q5_K = 13
Q6_K = 14
TYPES = {"q4_0": Q4_0, "q4_1": Q4_1, "q5_0": Q5_0, "q5_1": Q5_1, "q8_0": Q8_0, "q8_1": Q8_1,
         "q2_k": Q2_K, "q3_k": Q3_K, "q4_k": Q4_K, "q5_k": Q5_K, "q6_k": Q6_K}
BLOCK_WEIGHTS = {Q4_0: 32, Q4_1: 32, Q5_0: 32, Q5_1: 32, Q8_0: 32, Q8_1: 32,
                 Q2_K: 256, Q3_K: 256, Q4_K: 256, Q5_K: 256, Q6_K: 256}
BLOCK_BYTES = {Q4_0: 18, Q4_1: 20, Q5_0: 22, Q5_1: 24, Q8_0: 34, Q8_1: 36,
               Q2_K: 84, Q3_K: 110, Q4_K: 144, Q5_K: 176, Q6_K: 210}

OP_ARGMAX = 1
OP_MOE = 2
OP_GEMM_N = 3
OP_SHORT_CONV = 4
OP_GEMM = 5
# types of a key-value cache (the GGUF ids of F16, I8 and BF16; 4 bits have none)
KV_F16 = 1
KV_I8 = 24
KV_BF16 = 30
KV_Q4 = 104
KV_TYPES = {"f16": KV_F16, "i8": KV_I8, "bf16": KV_BF16, "q4": KV_Q4}
# which columns turn together
ROPE_PAIRS = {"halves": 0, "adjacent": 1}
MAX_ATTN_N = 16
MAX_KV_ROWS = 1 << 27
MAX_K = 32768
MAX_SEGMENTS = 8
MAX_N = 16
MAX_PREFILL_N = 16384

STATUS = {0: "QMV_OK", 1: "QMV_EINVAL", 2: "QMV_ESHAPE", 3: "QMV_EALIGN",
          4: "QMV_EWORKSPACE", 5: "QMV_EHIP"}

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqmv.so")

# every symbol include/qmv.h declares
EXPORTS = ["qmv_q8_0", "qmv_q4_k", "qmv_q6_k", "qmv_q4_0", "qmv_q4_1", "qmv_q5_0", "qmv_q5_1",
           "qmv_q8_1", "qmv_q5_k", "qmv_q2_k", "qmv_q3_k", "qmv_fused_rows", "qmv_fused_rows2",
           "qmv_gate_up_silu", "qmv_short_conv", "qmv_argmax", "qmv_argmax_noalloc", "moe_qmv_topk", "qmv_gemm_n", "qmv_gemm", "qmv_dequant",
           "qmv_quantize", "qmv_row_bytes", "qmv_workspace_bytes", "qmv_last_hip_error",
           "qmv_status_str", "qmv_probe_stream_read", "qmv_time_next_launch",
           "qmv_kv_page_bytes", "qmv_kv_append", "qmv_attn_decode", "qmv_attn_decode_workspace",
           "qmv_attn_prefill", "qmv_attn_prefill_workspace", "qmv_kv_evict", "qmv_kv_read",
           "qmv_qk_norm_rope", "qmv_kv_append_rope", "qmv_kv_reserve", "qmv_kv_release"]


class QmvError(RuntimeError):
    def __init__(self, fn: str, status: int, hip: int = 0):
        self.status = status
        self.status_name = STATUS.get(status, str(status))
        self.hip_error = hip
        msg = f"{fn}: {self.status_name}"
        if status == 5:
            msg += f" (hip error {hip})"
        super().__init__(msg)


_lib = None


def load():
    """Load libqmv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m gguf_dequant_matvec_amd.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, i32, ci, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int,
                           ctypes.c_size_t)
    cf = ctypes.c_float
    sig = {
        "qmv_q8_0": [P, i64, i64, P, P, P],
        "qmv_q4_k": [P, i64, i64, P, P, P],
        "qmv_q6_k": [P, i64, i64, P, P, P],
        "qmv_q4_0": [P, i64, i64, P, P, P],
        "qmv_q4_1": [P, i64, i64, P, P, P],
        "qmv_q5_0": [P, i64, i64, P, P, P],
        "qmv_q5_1": [P, i64, i64, P, P, P],
        "qmv_q8_1": [P, i64, i64, P, P, P],
        "qmv_q5_k": [P, i64, i64, P, P, P],
        "qmv_q2_k": [P, i64, i64, P, P, P],
        "qmv_q3_k": [P, i64, i64, P, P, P],
        "qmv_fused_rows": [ci, P, i64, P, i32, P, P, P],
        "qmv_fused_rows2": [ci, P, i32, P, P, ci, P, i32, P, P, i64, P, P],
        "qmv_gate_up_silu": [ci, P, i64, i64, P, P, P],
        "qmv_short_conv": [ci, P, i64, i64, P, P, P, ci, P, P, P, sz, P],
        "qmv_argmax": [ci, P, i64, i64, P, P, P, P, sz, P],
        "qmv_argmax_noalloc": [ci, P, i64, i64, P, P, P, P],
        "moe_qmv_topk": [P, i64, P, P, i32, i32, ci, P, ci, P, i64, P, P, P, P, sz, P],
        "qmv_gemm_n": [ci, P, i64, i64, i32, P, P, P, sz, P],
        "qmv_gemm": [ci, P, i64, i64, i64, P, P, P, sz, P],
        "qmv_dequant": [ci, P, i64, i64, P, P],
        "qmv_quantize": [ci, P, i64, i64, P, P],
        "qmv_probe_stream_read": [P, sz, P, P],
        "qmv_time_next_launch": [P, P],
        "qmv_kv_append": [P, i64, P, P, i64, P, i64, P],
        "qmv_attn_decode": [P, i32, i32, P, i64, cf, i32, i32, P, i64, P, i64, P, sz, P],
        "qmv_attn_prefill": [P, i64, P, i32, P, i64, cf, i32, i32, P, i64, P, sz, P],
        "qmv_kv_evict": [P, P, i64, i32, i32, i32, P, i64, P, P, i64, P, P],
        "qmv_kv_read": [P, i64, P, P, i64, P, i64, P],
        "qmv_qk_norm_rope": [P, i32, i64, P, i32, P, i64, P, i64, i32, P, i64, P, i64, P],
        "qmv_kv_append_rope": [P, P, i64, P, i32, P, i64, P, i64, P, i64, P, i64, P],
        "qmv_kv_reserve": [P, P, P, P, i64, P, P, P, P, P],
        "qmv_kv_release": [P, P, P, P, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ci
    lib.qmv_row_bytes.argtypes = [ci, i64]
    lib.qmv_row_bytes.restype = sz
    lib.qmv_workspace_bytes.argtypes = [ci, i64, i64, i32, i32]
    lib.qmv_workspace_bytes.restype = sz
    lib.qmv_kv_page_bytes.argtypes = [i32, i32, i32, i32]
    lib.qmv_kv_page_bytes.restype = sz
    lib.qmv_attn_decode_workspace.argtypes = [P, i32, i32, i64, i32, i32, i32]
    lib.qmv_attn_decode_workspace.restype = sz
    lib.qmv_attn_prefill_workspace.argtypes = [P, i64, i32, i64, i32, i32]
    lib.qmv_attn_prefill_workspace.restype = sz
    lib.qmv_last_hip_error.argtypes = []
    lib.qmv_last_hip_error.restype = ci
    lib.qmv_status_str.argtypes = [ci]
    lib.qmv_status_str.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _ptr(a) -> int:
    if a is None:
        return 0
    if isinstance(a, int):
        return a
    return int(a.data_ptr())


_torch_module = None
_raw_stream = None   # () -> address of torch's current stream on the current device
_raw_stream_on = None   # device -> address of torch's current stream there


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _find_raw_stream():
    """torch's current stream without building a Stream object for every call
    (0.6 us instead of 3.5 us of a small call's time); null without a GPU."""
    global _raw_stream, _raw_stream_on
    import torch
    if not torch.cuda.is_available():
        return 0
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if get is None:
        _raw_stream = lambda: int(torch.cuda.current_stream().cuda_stream)  # noqa: E731
    else:
        device = torch.cuda.current_device
        _raw_stream_on = get
        _raw_stream = lambda: get(device())  # noqa: E731
    return _raw_stream()


def _stream(stream) -> int:
    if stream is None:
        return _raw_stream() if _raw_stream is not None else _find_raw_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _cache_stream(cache, stream, *tensors) -> int:
    """The stream of a call over a cache of tensors, all of whose tensors must
    be on the pages' GPU, the current one: a kernel cannot tell, it would fault.
    Raw addresses are taken as they are."""
    return _stream_on(cache.device, "the cache", stream, tensors)


def _rope_stream(rope, stream, *tensors) -> int:
    """The same for rows of queries and keys beside a rotation, which may have no
    tensors itself: then the rows' first one says which GPU it is."""
    on = rope.device
    if on is None:
        on = next((a.get_device() for a in tensors if a is not None and a.__class__ is not int), None)
    return _stream_on(on, "the rotation" if rope.device is not None else "another", stream, tensors)


def _stream_on(on, what, stream, tensors) -> int:
    if on is None:
        return _stream(stream)
    if on < 0:
        raise ValueError("the call's tensors are not on a GPU")
    for a in tensors:
        if a is not None and a.__class__ is not int and a.get_device() != on:
            raise ValueError(f"a tensor on {a.device}, {what} on GPU {on}")
    if _torch().cuda.current_device() != on:
        raise ValueError(f"the call's tensors are on GPU {on}, which is not the current one")
    if stream is not None and not isinstance(stream, int) and stream.device_index != on:
        raise ValueError(f"a stream of GPU {stream.device_index}, the call's tensors on GPU {on}")
    return _raw_stream_on(on) if stream is None and _raw_stream_on is not None else _stream(stream)


def _type(t) -> int:
    return TYPES[t] if isinstance(t, str) else int(t)


def _call(name: str, *args):
    lib = _lib if _lib is not None else load()
    st = getattr(lib, name)(*args)
    if st != 0:
        raise QmvError(name, st, lib.qmv_last_hip_error())


def row_bytes(t, K: int) -> int:
    t = _type(t)
    return (K // BLOCK_WEIGHTS[t]) * BLOCK_BYTES[t]


def qmv_row_bytes(t, K: int) -> int:
    return int(load().qmv_row_bytes(_type(t), K))


def qmv_workspace_bytes(op: int, a: int, b: int = 0, c: int = 0, d: int = 0) -> int:
    return int(load().qmv_workspace_bytes(op, a, b, c, d))


def qmv_q8_0(blocks, M, K, x, y, stream=None):
    _call("qmv_q8_0", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv_q4_k(blocks, M, K, x, y, stream=None):
    _call("qmv_q4_k", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv_q6_k(blocks, M, K, x, y, stream=None):
    _call("qmv_q6_k", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv(t, blocks, M, K, x, y, stream=None):
    """Single-token matvec in format t (any of TYPES)."""
    _call("qmv_" + {v: k for k, v in TYPES.items()}[_type(t)], _ptr(blocks), M, K, _ptr(x), _ptr(y),
          _stream(stream))


def qmv_q4_0(blocks, M, K, x, y, stream=None):
    _call("qmv_q4_0", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv_q4_1(blocks, M, K, x, y, stream=None):
    _call("qmv_q4_1", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv_q5_0(blocks, M, K, x, y, stream=None):
    _call("qmv_q5_0", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv_q5_1(blocks, M, K, x, y, stream=None):
    _call("qmv_q5_1", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv_q8_1(blocks, M, K, x, y, stream=None):
    _call("qmv_q8_1", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv_q5_k(blocks, M, K, x, y, stream=None):
    _call("qmv_q5_k", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv_q2_k(blocks, M, K, x, y, stream=None):
    _call("qmv_q2_k", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def qmv_q3_k(blocks, M, K, x, y, stream=None):
    _call("qmv_q3_k", _ptr(blocks), M, K, _ptr(x), _ptr(y), _stream(stream))


def _check_segments(seg_rows, y_seg):
    # the C entry point reads nseg entries of both host arrays
    if len(seg_rows) != len(y_seg):
        raise ValueError(f"seg_rows has {len(seg_rows)} entries but y_seg has {len(y_seg)}")


def qmv_fused_rows(t, blocks, K, x, seg_rows, y_seg, stream=None):
    _check_segments(seg_rows, y_seg)
    n = len(seg_rows)
    rows = (ctypes.c_int64 * max(n, 1))(*seg_rows)
    ys = (ctypes.c_void_p * max(len(y_seg), 1))(*[_ptr(y) for y in y_seg])
    _call("qmv_fused_rows", _type(t), _ptr(blocks), K, _ptr(x), n,
          ctypes.cast(rows, ctypes.c_void_p), ctypes.cast(ys, ctypes.c_void_p), _stream(stream))


def qmv_fused_rows2(t1, blocks1, seg_rows1, y_seg1, t2, blocks2, seg_rows2, y_seg2, K, x,
                    stream=None):
    def arrays(seg_rows, y_seg):
        _check_segments(seg_rows, y_seg)
        rows = (ctypes.c_int64 * max(len(seg_rows), 1))(*seg_rows)
        ys = (ctypes.c_void_p * max(len(y_seg), 1))(*[_ptr(y) for y in y_seg])
        return rows, ys
    r1, y1 = arrays(seg_rows1, y_seg1)
    r2, y2 = arrays(seg_rows2, y_seg2)
    _call("qmv_fused_rows2", _type(t1), _ptr(blocks1), len(seg_rows1), ctypes.cast(r1, ctypes.c_void_p),
          ctypes.cast(y1, ctypes.c_void_p), _type(t2), _ptr(blocks2), len(seg_rows2),
          ctypes.cast(r2, ctypes.c_void_p), ctypes.cast(y2, ctypes.c_void_p), K, _ptr(x),
          _stream(stream))


def qmv_gate_up_silu(t, blocks, I, K, x, h, stream=None):
    _call("qmv_gate_up_silu", _type(t), _ptr(blocks), I, K, _ptr(x), _ptr(h), _stream(stream))


def qmv_short_conv(in_t, in_proj, D, H, h, w_conv, state, out_t, out_proj, out, workspace,
                   ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call("qmv_short_conv", _type(in_t), _ptr(in_proj), D, H, _ptr(h), _ptr(w_conv), _ptr(state),
          _type(out_t), _ptr(out_proj), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream))


def qmv_argmax(t, blocks, M, K, x, idx_out, max_out, workspace, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call("qmv_argmax", _type(t), _ptr(blocks), M, K, _ptr(x), _ptr(idx_out), _ptr(max_out),
          _ptr(workspace), ws_bytes, _stream(stream))


def qmv_argmax_noalloc(t, blocks, M, K, x, idx_out, max_out, stream=None):
    _call("qmv_argmax_noalloc", _type(t), _ptr(blocks), M, K, _ptr(x), _ptr(idx_out),
          _ptr(max_out), _stream(stream))


def moe_qmv_topk(x, H, router, bias, E, k, gu_t, gate_up, dn_t, down, I, y, topk_idx, topk_w,
                 workspace, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call("moe_qmv_topk", _ptr(x), H, _ptr(router), _ptr(bias), E, k, _type(gu_t),
          _ptr(gate_up), _type(dn_t), _ptr(down), I, _ptr(y), _ptr(topk_idx), _ptr(topk_w),
          _ptr(workspace), ws_bytes, _stream(stream))


def qmv_gemm_n(t, blocks, M, K, n, X, Y, workspace=None, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call("qmv_gemm_n", _type(t), _ptr(blocks), M, K, n, _ptr(X), _ptr(Y), _ptr(workspace),
          ws_bytes, _stream(stream))


def qmv_gemm(t, blocks, M, K, n, X, Y, workspace=None, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _call("qmv_gemm", _type(t), _ptr(blocks), M, K, n, _ptr(X), _ptr(Y), _ptr(workspace),
          ws_bytes, _stream(stream))


def qmv_dequant(t, blocks, M, K, w_out, stream=None):
    _call("qmv_dequant", _type(t), _ptr(blocks), M, K, _ptr(w_out), _stream(stream))


def qmv_quantize(t, w, M, K, blocks_out, stream=None):
    _call("qmv_quantize", _type(t), _ptr(w), M, K, _ptr(blocks_out), _stream(stream))


class _KvCacheStruct(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int64), ("pages", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("table_ld", ctypes.c_int64),
                ("seq_len", ctypes.c_void_p), ("n_seq", ctypes.c_int64)]


class KvCache:
    """A paged key-value cache (qmv_kv_cache): `pages` a byte buffer of whole
    pages, `table` int32 [n_seq][table_ld], `seq_len` int32 [n_seq], all on the
    device.  Tensors are checked and kept alive; with raw addresses the counts
    have to be given.  Lengths and table are read when a call runs, so both
    may be changed in place between calls.  The calls refuse tensors of another
    device, and a cache that is not on the current one."""

    def __init__(self, t, n_kv_heads, head_dim, page_size, pages, table, seq_len, n_pages=None,
                 n_seq=None, table_ld=None):
        t = KV_TYPES[t] if isinstance(t, str) else int(t)
        page_bytes = int(load().qmv_kv_page_bytes(t, n_kv_heads, head_dim, page_size))
        if not isinstance(pages, int):
            if not pages.is_contiguous():
                raise ValueError("pages must be contiguous")
            have = pages.numel() * pages.element_size() // max(page_bytes, 1)
            if n_pages is not None and n_pages > have:
                raise ValueError(f"pages holds {have} pages, not {n_pages}")
            n_pages = have if n_pages is None else n_pages
        if not isinstance(table, int):
            if table.dtype is not _torch().int32 or table.dim() != 2 or \
                    (table.shape[1] > 1 and table.stride(1) != 1):
                raise ValueError("table must be an int32 matrix with contiguous rows")
            if n_seq is not None and n_seq > table.shape[0]:
                raise ValueError(f"table has {table.shape[0]} rows, not {n_seq}")
            n_seq = table.shape[0] if n_seq is None else n_seq
            if table.shape[0] > 1 and table.stride(0) != table.shape[1]:
                raise ValueError("table must be contiguous")
            if table_ld is not None and table_ld != table.shape[1]:
                raise ValueError(f"table rows have {table.shape[1]} entries, not {table_ld}")
            table_ld = table.shape[1]
        if not isinstance(seq_len, int):
            if seq_len.dtype is not _torch().int32 or not seq_len.is_contiguous() or \
                    seq_len.numel() < n_seq:
                raise ValueError("seq_len must be n_seq contiguous int32 values")
        self.device = None if isinstance(pages, int) else pages.get_device()
        for a in (table, seq_len):
            if self.device is not None and not isinstance(a, int) and a.get_device() != self.device:
                raise ValueError(f"pages on {pages.device}, but a tensor on {a.device}")
        self.type, self.n_kv_heads, self.head_dim, self.page_size = t, n_kv_heads, head_dim, page_size
        self.page_bytes, self.n_pages, self.n_seq, self.table_ld = page_bytes, n_pages, n_seq, table_ld
        self.pages, self.table, self.seq_len = pages, table, seq_len
        self._struct = _KvCacheStruct(t, n_kv_heads, head_dim, page_size, n_pages, _ptr(pages),
                                      _ptr(table), table_ld, _ptr(seq_len), n_seq)
        self._address = ctypes.addressof(self._struct)

    def __setattr__(self, name, value):
        if "_address" in self.__dict__:   # the calls go by the addresses taken above
            raise AttributeError("a KvCache stays as it was made: change its tensors in place, or make another")
        object.__setattr__(self, name, value)


def qmv_kv_page_bytes(t, n_kv_heads, head_dim, page_size) -> int:
    t = KV_TYPES[t] if isinstance(t, str) else int(t)
    return int(load().qmv_kv_page_bytes(t, n_kv_heads, head_dim, page_size))


def _f32_rows(name, a, ld, n, width):
    """Leading dimension of n rows of `width` f32 values: what the tensor's shape
    says, or `ld` from its first value on, as far as its storage reaches."""
    if a is None or isinstance(a, int):
        return width if ld is None else ld
    if a.dtype is not _torch().float32:
        raise ValueError(f"{name} must be float32")
    if ld is None and a.dim() == 2:      # the usual rows, without the loop below
        rows, cols = a.shape
        step, inner = a.stride()
        if rows >= n and cols == width and inner == 1:
            return step if n > 1 else width
    if ld is not None:
        have = a.untyped_storage().nbytes() // 4 - a.storage_offset()
        if (n - 1) * ld + width > have:
            raise ValueError(f"{name} holds {have} values, not {n} rows {ld} apart")
    if ld is None:
        shape, stride = a.shape, a.stride()
        inner = 1
        for i in range(len(shape) - 1, 0, -1):    # every dimension but the first is one row
            if shape[i] > 1 and stride[i] != inner:
                raise ValueError(f"the rows of {name} must be contiguous")
            inner *= shape[i]
        if len(shape) < 2 or shape[0] < n or inner != width:
            raise ValueError(f"{name} must be {n} rows of {width} values")
        ld = stride[0] if n > 1 else width
    return ld


def _check_start(cache, start):
    if start is not None and not isinstance(start, int):
        if start.dtype is not _torch().int32 or not start.is_contiguous() or \
                start.numel() < cache.n_seq + 1:
            raise ValueError("start must be n_seq + 1 contiguous int32 values")


def _check_dense(name, a, dtype, numel):
    if a is not None and not isinstance(a, int):
        if a.dtype is not getattr(_torch(), dtype) or not a.is_contiguous() or a.numel() < numel:
            raise ValueError(f"{name} must hold {numel} contiguous {dtype} values")


def _workspace_bytes(workspace, ws_bytes):
    """Bytes of a workspace: what its tensor spans, or fewer if the caller says so."""
    if workspace is None or isinstance(workspace, int):
        return 0 if ws_bytes is None else ws_bytes
    have = workspace.numel() * workspace.element_size()
    if not workspace.is_contiguous() or (ws_bytes is not None and ws_bytes > have):
        raise ValueError(f"workspace must be contiguous and hold {have if ws_bytes is None else ws_bytes} bytes")
    return have if ws_bytes is None else ws_bytes


def qmv_kv_append(cache, n, k, v, start=None, ldk=None, ldv=None, stream=None):
    width = cache.n_kv_heads * cache.head_dim
    ldk, ldv = _f32_rows("k", k, ldk, n, width), _f32_rows("v", v, ldv, n, width)
    _check_start(cache, start)
    _call("qmv_kv_append", cache._address, n, _ptr(start), _ptr(k), ldk, _ptr(v), ldv,
          _cache_stream(cache, stream, start, k, v))


def qmv_kv_read(cache, n, k, v, start=None, ldk=None, ldv=None, stream=None):
    width = cache.n_kv_heads * cache.head_dim
    ldk, ldv = _f32_rows("k", k, ldk, n, width), _f32_rows("v", v, ldv, n, width)
    _check_start(cache, start)
    _call("qmv_kv_read", cache._address, n, _ptr(start), _ptr(k), ldk, _ptr(v), ldv,
          _cache_stream(cache, stream, start, k, v))


class _QkRopeStruct(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("pairs", ctypes.c_int32),
                ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("eps", ctypes.c_float)]


class QkRope:
    """Norms of queries and keys and the rotation (qmv_qk_rope): `freq` float64
    [rot_dim / 2], radians a position; `pairs` "halves" or "adjacent"; `q_norm`,
    `k_norm` float32 [head_dim] or None.  Tensors are checked and kept alive; their
    values are read when a call runs."""

    def __init__(self, freq, rot_dim, pairs="halves", q_norm=None, k_norm=None, eps=1e-5):
        pairs = ROPE_PAIRS[pairs] if isinstance(pairs, str) else int(pairs)
        _check_dense("freq", freq, "float64", max(rot_dim, 0) // 2)
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            _check_dense(name, w, "float32", 0)
        self.freq, self.rot_dim, self.pairs = freq, rot_dim, pairs
        self.q_norm, self.k_norm, self.eps = q_norm, k_norm, eps
        self.device = None
        for a in (freq, q_norm, k_norm):
            if a is not None and not isinstance(a, int):
                if self.device is not None and a.get_device() != self.device:
                    raise ValueError(f"a tensor on {a.device}, another on GPU {self.device}")
                self.device = a.get_device()
        if self.device is not None and self.device < 0:
            raise ValueError("the rotation's tensors are not on a GPU")
        self._struct = _QkRopeStruct(_ptr(freq), rot_dim, pairs, _ptr(q_norm), _ptr(k_norm), eps)
        self._address = ctypes.addressof(self._struct)

    def __setattr__(self, name, value):
        if "_address" in self.__dict__:
            raise AttributeError("a QkRope stays as it was made: change its tensors in place, or make another")
        object.__setattr__(self, name, value)

    def _check_width(self, head_dim):
        for name, w in (("q_norm", self.q_norm), ("k_norm", self.k_norm)):
            if w is not None and not isinstance(w, int) and w.numel() < head_dim:
                raise ValueError(f"{name} must hold {head_dim} values")


def qmv_qk_norm_rope(rope, head_dim, n, pos, n_heads=0, q=None, q_out=None, n_kv_heads=0, k=None, k_out=None,
                     ldq=None, ldqo=None, ldk=None, ldko=None, stream=None):
    rope._check_width(head_dim)
    _check_dense("pos", pos, "int32", n)
    lds = [_f32_rows(name, a, ld, n, heads * head_dim) if heads else 0 for name, a, ld, heads in
           (("q", q, ldq, n_heads), ("q_out", q_out, ldqo, n_heads), ("k", k, ldk, n_kv_heads),
            ("k_out", k_out, ldko, n_kv_heads))]
    _call("qmv_qk_norm_rope", rope._address, head_dim, n, _ptr(pos), n_heads, _ptr(q), lds[0], _ptr(q_out), lds[1],
          n_kv_heads, _ptr(k), lds[2], _ptr(k_out), lds[3], _rope_stream(rope, stream, pos, q, q_out, k, k_out))


def qmv_kv_append_rope(cache, rope, n, n_heads, q, q_out, k, v, start=None, ldq=None, ldqo=None, ldk=None, ldv=None,
                       stream=None):
    rope._check_width(cache.head_dim)
    width = cache.n_kv_heads * cache.head_dim
    ldk, ldv = _f32_rows("k", k, ldk, n, width), _f32_rows("v", v, ldv, n, width)
    ldq = _f32_rows("q", q, ldq, n, n_heads * cache.head_dim)
    ldqo = _f32_rows("q_out", q_out, ldqo, n, n_heads * cache.head_dim)
    _check_start(cache, start)
    if rope.device is not None and cache.device is not None and rope.device != cache.device:
        raise ValueError(f"the rotation on GPU {rope.device}, the cache on GPU {cache.device}")
    _call("qmv_kv_append_rope", cache._address, rope._address, n, _ptr(start), n_heads, _ptr(q), ldq, _ptr(q_out),
          ldqo, _ptr(k), ldk, _ptr(v), ldv, _cache_stream(cache, stream, start, q, q_out, k, v))


def _dense_ptr(name, a, dtype, numel, on):
    """Address of `numel` contiguous values of a torch dtype on GPU `on` (None: any), all checks
    in one pass: these calls are as short as their checks."""
    if a is None:
        return 0
    if a.__class__ is int:
        return a
    if a.dtype is not dtype or a.numel() < numel or not a.is_contiguous():
        raise ValueError(f"{name} must hold {numel} contiguous {dtype} values")
    if on is not None and a.get_device() != on:
        raise ValueError(f"{name} is on {a.device}, the cache on GPU {on}")
    return a.data_ptr()


def qmv_kv_reserve(cache, add, free_pages, free_count, n, granted, start, pos=None, slot=None, stream=None):
    on, n_seq, i32 = cache.device, cache.n_seq, _torch().int32
    _call("qmv_kv_reserve", cache._address, _dense_ptr("add", add, i32, n_seq, on),
          _dense_ptr("free_pages", free_pages, i32, cache.n_pages, on), _dense_ptr("free_count", free_count, i32, 1, on),
          n, _dense_ptr("granted", granted, i32, n_seq, on), _dense_ptr("start", start, i32, n_seq + 1, on),
          _dense_ptr("pos", pos, i32, n, on), _dense_ptr("slot", slot, _torch().int64, n, on), _cache_stream(cache, stream))


def qmv_kv_release(cache, new_len, free_pages, free_count, stream=None):
    on, i32 = cache.device, _torch().int32
    _call("qmv_kv_release", cache._address, _dense_ptr("new_len", new_len, i32, cache.n_seq, on),
          _dense_ptr("free_pages", free_pages, i32, cache.n_pages, on), _dense_ptr("free_count", free_count, i32, 1, on),
          _cache_stream(cache, stream))


def qmv_attn_decode_workspace(cache, n, n_heads, max_len, window=0, sinks=0, with_acc=False) -> int:
    return int(load().qmv_attn_decode_workspace(cache._address, n, n_heads, max_len, window, sinks,
                                                int(bool(with_acc))))


def _head_rows(name, a, ld, cache):
    """Leading dimension of a [n_seq][n_kv_heads][ld] f32 array."""
    if a is None or isinstance(a, int):
        return 0 if ld is None else ld
    if a.dtype is not _torch().float32 or a.dim() != 3 or not a.is_contiguous() or \
            a.shape[0] < cache.n_seq or a.shape[1] != cache.n_kv_heads:
        raise ValueError(f"{name} must be contiguous float32 [n_seq][n_kv_heads][positions]")
    if ld is not None and ld != a.shape[2]:
        raise ValueError(f"the heads of {name} have {a.shape[2]} positions, not {ld}")
    return a.shape[2]


def qmv_attn_decode(cache, n, n_heads, q, scale, out, max_len, window=0, sinks=0, acc=None,
                    workspace=None, ldq=None, ld_acc=None, ws_bytes=None, stream=None):
    ldq = _f32_rows("q", q, ldq, cache.n_seq * n, n_heads * cache.head_dim)
    _check_dense("out", out, "float32", cache.n_seq * n * n_heads * cache.head_dim)
    ld_acc = _head_rows("acc", acc, ld_acc, cache)
    ws_bytes = _workspace_bytes(workspace, ws_bytes)
    _call("qmv_attn_decode", cache._address, n, n_heads, _ptr(q), ldq, scale, window, sinks,
          _ptr(out), max_len, _ptr(acc), ld_acc, _ptr(workspace), ws_bytes,
          _cache_stream(cache, stream, q, out, acc, workspace))


def qmv_attn_prefill_workspace(cache, n, n_heads, max_len, window=0, sinks=0) -> int:
    return int(load().qmv_attn_prefill_workspace(cache._address, n, n_heads, max_len, window, sinks))


def qmv_attn_prefill(cache, n, n_heads, q, scale, out, max_len, start=None, window=0, sinks=0,
                     workspace=None, ldq=None, ws_bytes=None, stream=None):
    ldq = _f32_rows("q", q, ldq, n, n_heads * cache.head_dim)
    _check_dense("out", out, "float32", n * n_heads * cache.head_dim)
    _check_start(cache, start)
    ws_bytes = _workspace_bytes(workspace, ws_bytes)
    _call("qmv_attn_prefill", cache._address, n, _ptr(start), n_heads, _ptr(q), ldq, scale, window,
          sinks, _ptr(out), max_len, _ptr(workspace), ws_bytes,
          _cache_stream(cache, stream, start, q, out, workspace))


def qmv_kv_evict(cache, dst_table, keep, first, recent, acc, kept, acc_out, len_out, dst_ld=None,
                 ld_acc=None, ld_out=None, stream=None):
    if not isinstance(dst_table, int):
        if dst_table is None or dst_table.dim() != 2 or dst_table.shape[0] < cache.n_seq:
            raise ValueError("dst_table must be a matrix with a row per sequence")
        _check_dense("dst_table", dst_table, "int32", 0)
        if dst_ld is not None and dst_ld != dst_table.shape[1]:
            raise ValueError(f"the rows of dst_table have {dst_table.shape[1]} entries, not {dst_ld}")
        dst_ld = dst_table.shape[1]
    ld_acc = _head_rows("acc", acc, ld_acc, cache)
    ld_out = _head_rows("acc_out", acc_out, ld_out, cache)
    _check_dense("kept", kept, "int32", cache.n_seq * cache.n_kv_heads * max(keep, 0))
    _check_dense("len_out", len_out, "int32", cache.n_seq)
    _call("qmv_kv_evict", cache._address, _ptr(dst_table), dst_ld, keep, first, recent, _ptr(acc),
          ld_acc, _ptr(kept), _ptr(acc_out), ld_out, _ptr(len_out),
          _cache_stream(cache, stream, dst_table, acc, kept, acc_out, len_out))


def qmv_probe_stream_read(buf, nbytes, sink, stream=None):
    _call("qmv_probe_stream_read", _ptr(buf), nbytes, _ptr(sink), _stream(stream))


def qmv_time_next_launch(start, stop):
    """Arm the timing hook: the next call's main kernel records its own start
    and end into these events (torch.cuda.Event objects already recorded once,
    or raw hipEvent_t addresses; None disarms)."""
    def h(e):
        if e is None:
            return 0
        return e if isinstance(e, int) else int(e.cuda_event)
    _call("qmv_time_next_launch", h(start), h(stop))
