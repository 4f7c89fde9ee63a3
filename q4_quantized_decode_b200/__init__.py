"""q4_quantized_decode_b200 -- B200-native Q4_0 GEMV for memory-bound decode.

A thin ctypes binding over the C-ABI library ``libq4gemv.so`` (declared in
``include/q4gemv.h``).  The functions below carry the ABI's names and only
marshal arguments: every step of the computation runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams (``Q4Gemv`` accepts
tensors); nothing here computes on the CPU, and there is no fallback: if the
library is missing or fails to load, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4gemv.so")

Q4_OK = 0
Q4_EINVAL = -1
Q4_ESHAPE = -2
Q4_EALIGN = -3
Q4_ENOMEM = -4
Q4_ECUDA = -5
Q4_EUNSUPPORTED = -6
Q4_ETIMEOUT = -7
Q4_EFAULTINJ = -8
Q4_ECONCURRENT = -9
Q4_EINDEX = -10
MAX_M = 256        # vectors per q4gemv_run call
MAX_M_GEMV = 16    # above this, the tensor-core GEMM path
F16, BF16 = 0, 1   # q4gemv_dtype
ROPE_PLAIN, ROPE_LINEAR, ROPE_BY_PARTS = 0, 1, 2
MIX_ATTENTION, MIX_LINEAR = 0, 1


class Q4Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"q4gemv status {status}: {msg}")
        self.status = status


class q4gemv_layer(ctypes.Structure):
    _fields_ = [("qkv", ctypes.c_void_p), ("o", ctypes.c_void_p),
                ("gate_up", ctypes.c_void_p), ("down", ctypes.c_void_p)]


class q4gemv_kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("n_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("table_cols", ctypes.c_int64), ("dtype", ctypes.c_int)]


class q4gemv_rope(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("amp", ctypes.c_float)]


class q4gemv_linattn_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("log_decay", ctypes.c_void_p), ("state_in", ctypes.c_void_p),
                ("state_out", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("decay_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("n_slots", ctypes.c_int64),
                ("qk_heads", ctypes.c_int64), ("v_heads", ctypes.c_int64),
                ("k_dim", ctypes.c_int64), ("v_dim", ctypes.c_int64),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class q4gemv_mixer(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("kv", q4gemv_kv), ("log_decay", ctypes.c_void_p),
                ("state", ctypes.c_void_p)]


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "or `python q4_quantized_decode_b200/build_ext.py`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, ci, dbl = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
    sigs = {
        "q4gemv_version": ([], ci),
        "q4gemv_create": ([ctypes.POINTER(vp), ci], ci),
        "q4gemv_destroy": ([vp], ci),
        "q4gemv_gguf_bytes": ([i64, i64], ctypes.c_size_t),
        "q4gemv_packed_bytes": ([i64, i64], ctypes.c_size_t),
        "q4gemv_validate": ([ci, i64, i64, vp, vp, vp], ci),
        "q4gemv_repack": ([vp, vp, vp, i64, i64, vp], ci),
        "q4gemv_run": ([vp, vp, vp, vp, ci, i64, i64, vp], ci),
        "q4gemv_run_swiglu": ([vp, vp, vp, vp, i64, i64, vp], ci),
        "q4gemv_shard_rows": ([i64, ci, ci, ctypes.POINTER(i64), ctypes.POINTER(i64),
                               ctypes.POINTER(i64)], ci),
        "q4gemv_comm_unique_id": ([ctypes.c_char_p], ci),
        "q4gemv_comm_init": ([vp, ci, ci, ctypes.c_char_p], ci),
        "q4gemv_run_stack_sharded": ([vp, ctypes.POINTER(q4gemv_layer), ci, i64, i64, i64, vp, vp,
                                      vp], ci),
        "q4gemv_peer_layout": ([ci, i64, i64, i64, ctypes.POINTER(i64)], ci),
        "q4gemv_peer_check": ([ctypes.c_char_p, ci], ci),
        "q4gemv_peer_export": ([vp, ci, ci, i64, i64, i64, ctypes.c_char_p], ci),
        "q4gemv_peer_open": ([vp, ctypes.c_char_p], ci),
        "q4gemv_peer_close": ([vp], ci),
        "q4gemv_run_stack": ([vp, ctypes.POINTER(q4gemv_layer), ci, i64, i64, i64,
                              vp, vp, vp, vp, vp], ci),
        "q4gemv_run_stack_gated": ([vp, ctypes.POINTER(q4gemv_layer), ci, i64, i64, i64,
                                    vp, vp, vp], ci),
        "q4gemv_sync_status": ([vp, vp], ci),
        "q4gemv_strerror": ([ci], ctypes.c_char_p),
        "q4gemv_last_error": ([vp], ctypes.c_char_p),
        "q4gemv_set_fault": ([vp, ctypes.c_char_p], ci),
        "q4gemv_run_noalloc": ([vp, vp, vp, ci, i64, i64, vp], ci),
        "q4gemv_q8_0_gguf_bytes": ([i64, i64], ctypes.c_size_t),
        "q4gemv_q8_0_packed_bytes": ([i64, i64], ctypes.c_size_t),
        "q4gemv_q8_0_repack": ([vp, vp, vp, i64, i64, vp], ci),
        "q4gemv_q8_0_validate": ([ci, i64, i64, vp, vp, vp], ci),
        "q4gemv_q8_0_run": ([vp, vp, vp, vp, ci, i64, i64, vp], ci),
        "q4gemv_rope_freqs": ([ci, ci, dbl, dbl, dbl, dbl, dbl, ctypes.POINTER(dbl)], ci),
        "q4gemv_kv_append": ([vp, ctypes.POINTER(q4gemv_kv), i64, i64, vp, vp, vp,
                              ctypes.POINTER(q4gemv_rope), vp, i64, i64, vp, i64, vp, i64, vp, i64,
                              vp], ci),
        "q4gemv_attn_paged": ([vp, ctypes.POINTER(q4gemv_kv), i64, i64, vp, vp, i64, vp, i64, i64, vp,
                               i64, ctypes.c_float, ci, i64, vp], ci),
        "q4gemv_run_stack_mixed": ([vp, ctypes.POINTER(q4gemv_layer), ctypes.POINTER(q4gemv_mixer), ci, i64,
                                    i64, i64, i64, ctypes.POINTER(q4gemv_rope), vp, vp, vp, vp], ci),
        "q4gemv_linattn": ([vp, ctypes.POINTER(q4gemv_linattn_args), i64, i64, vp, i64, vp], ci),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load_library()
lib = _lib


def q4gemv_version() -> int:
    return _lib.q4gemv_version()


def q4gemv_strerror(status: int) -> str:
    return _lib.q4gemv_strerror(status).decode()


def q4gemv_last_error(h) -> str:
    return _lib.q4gemv_last_error(h).decode()


def q4gemv_gguf_bytes(N: int, K: int) -> int:
    return _lib.q4gemv_gguf_bytes(N, K)


def q4gemv_packed_bytes(N: int, K: int) -> int:
    return _lib.q4gemv_packed_bytes(N, K)


def q4gemv_validate(M, N, K, W, x, y) -> int:
    return _lib.q4gemv_validate(M, N, K, W, x, y)


def q4gemv_create(device: int = 0):
    h = ctypes.c_void_p()
    st = _lib.q4gemv_create(ctypes.byref(h), device)
    return st, h


def q4gemv_destroy(h) -> int:
    return _lib.q4gemv_destroy(h)


def q4gemv_repack(h, gguf, packed, N, K, stream) -> int:
    return _lib.q4gemv_repack(h, gguf, packed, N, K, stream)


def q4gemv_run(h, W, x, y, M, N, K, stream) -> int:
    return _lib.q4gemv_run(h, W, x, y, M, N, K, stream)


def q4gemv_run_swiglu(h, W, gate_up, y, N, K, stream) -> int:
    return _lib.q4gemv_run_swiglu(h, W, gate_up, y, N, K, stream)


def q4gemv_run_stack(h, layers, n_layers, hidden, qkv_n, ffn, x_in, x_out,
                     trace_x, trace_y, stream) -> int:
    return _lib.q4gemv_run_stack(h, layers, n_layers, hidden, qkv_n, ffn, x_in, x_out,
                                 trace_x, trace_y, stream)


def q4gemv_run_stack_gated(h, layers, n_layers, hidden, qkv_n, ffn, x_in, x_out, stream) -> int:
    return _lib.q4gemv_run_stack_gated(h, layers, n_layers, hidden, qkv_n, ffn, x_in, x_out, stream)


def q4gemv_sync_status(h, stream) -> int:
    return _lib.q4gemv_sync_status(h, stream)


def q4gemv_set_fault(h, which: str) -> int:
    return _lib.q4gemv_set_fault(h, which.encode())


def q4gemv_shard_rows(N: int, world: int, rank: int):
    """(status, row0, rows, chunk) of rank's row slice of an N-row matrix."""
    r0, n, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    st = _lib.q4gemv_shard_rows(N, world, rank, ctypes.byref(r0), ctypes.byref(n), ctypes.byref(c))
    return st, r0.value, n.value, c.value


def q4gemv_comm_unique_id():
    """(status, 128-byte NCCL unique id)."""
    buf = ctypes.create_string_buffer(128)
    st = _lib.q4gemv_comm_unique_id(buf)
    return st, buf.raw


def q4gemv_comm_init(h, world: int, rank: int, uid: bytes) -> int:
    return _lib.q4gemv_comm_init(h, world, rank, ctypes.create_string_buffer(uid, 128))


PEER_BLOB_BYTES = 128
PEER_MAX_WORLD = 8


def q4gemv_peer_layout(world: int, hidden: int, qkv_n: int, ffn: int):
    """(status, [6 byte offsets]) of the peer exchange buffer (see the header)."""
    off = (ctypes.c_int64 * 6)()
    st = _lib.q4gemv_peer_layout(world, hidden, qkv_n, ffn, off)
    return st, list(off)


def q4gemv_peer_check(blobs: bytes, world: int) -> int:
    return _lib.q4gemv_peer_check(ctypes.create_string_buffer(blobs, len(blobs)), world)


def q4gemv_peer_export(h, world: int, rank: int, hidden: int, qkv_n: int, ffn: int):
    """(status, this rank's 128-byte exchange blob)."""
    buf = ctypes.create_string_buffer(PEER_BLOB_BYTES)
    st = _lib.q4gemv_peer_export(h, world, rank, hidden, qkv_n, ffn, buf)
    return st, buf.raw


def q4gemv_peer_open(h, blobs: bytes) -> int:
    return _lib.q4gemv_peer_open(h, ctypes.create_string_buffer(blobs, len(blobs)))


def q4gemv_peer_close(h) -> int:
    return _lib.q4gemv_peer_close(h)


def q4gemv_run_stack_sharded(h, layers, n_layers, hidden, qkv_n, ffn, x_in, x_out, stream) -> int:
    return _lib.q4gemv_run_stack_sharded(h, layers, n_layers, hidden, qkv_n, ffn, x_in, x_out, stream)


def q4gemv_run_noalloc(W, x, y, M, N, K, stream) -> int:
    """The M <= 2 GEMV without a handle or any allocation (see the header)."""
    return _lib.q4gemv_run_noalloc(W, x, y, M, N, K, stream)


def q4gemv_q8_0_gguf_bytes(N: int, K: int) -> int:
    return _lib.q4gemv_q8_0_gguf_bytes(N, K)


def q4gemv_q8_0_packed_bytes(N: int, K: int) -> int:
    return _lib.q4gemv_q8_0_packed_bytes(N, K)


def q4gemv_q8_0_repack(h, gguf, packed, N, K, stream) -> int:
    return _lib.q4gemv_q8_0_repack(h, gguf, packed, N, K, stream)


def q4gemv_q8_0_validate(M, N, K, W, x, y) -> int:
    return _lib.q4gemv_q8_0_validate(M, N, K, W, x, y)


def q4gemv_q8_0_run(h, W, x, y, M, N, K, stream) -> int:
    return _lib.q4gemv_q8_0_run(h, W, x, y, M, N, K, stream)


def q4gemv_rope_freqs(kind: int, rot: int, base: float, factor: float = 1.0, trained: float = 0.0,
                      lo: float = 0.0, hi: float = 0.0):
    """(status, [rot/2 radians per position]) of a rotation (see the header)."""
    buf = (ctypes.c_double * max(1, rot // 2))()
    st = _lib.q4gemv_rope_freqs(kind, rot, base, factor, trained, lo, hi, buf)
    return st, list(buf[:rot // 2]) if st == Q4_OK else []


def q4gemv_kv_append(h, kv, rows, n_seqs, start, length, pos, rope, q, q_stride, q_heads, k, k_stride,
                     v, v_stride, q_out, q_out_stride, stream) -> int:
    return _lib.q4gemv_kv_append(h, kv, rows, n_seqs, start, length, pos, rope, q, q_stride, q_heads,
                                 k, k_stride, v, v_stride, q_out, q_out_stride, stream)


def q4gemv_attn_paged(h, kv, rows, n_seqs, start, length, max_new, q, q_stride, q_heads, out,
                      out_stride, scale, causal, window, stream) -> int:
    return _lib.q4gemv_attn_paged(h, kv, rows, n_seqs, start, length, max_new, q, q_stride, q_heads,
                                  out, out_stride, scale, causal, window, stream)


def q4gemv_linattn(h, args, rows, n_seqs, start, max_new, stream) -> int:
    return _lib.q4gemv_linattn(h, args, rows, n_seqs, start, max_new, stream)


def q4gemv_run_stack_mixed(h, layers, mixers, n_layers, hidden, ffn, q_heads, kv_heads, rope, length, x_in,
                           x_out, stream) -> int:
    return _lib.q4gemv_run_stack_mixed(h, layers, mixers, n_layers, hidden, ffn, q_heads, kv_heads, rope,
                                       length, x_in, x_out, stream)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


import torch as _torch  # noqa: E402  (after the library: a missing one is reported first)

_raw_stream = _torch._C._cuda_getCurrentRawStream   # current_stream(device).cuda_stream, without the object
_kv_append, _attn_paged, _linattn = _lib.q4gemv_kv_append, _lib.q4gemv_attn_paged, _lib.q4gemv_linattn


def _dtype_code(t) -> int:
    if t.dtype is _torch.float16:
        return F16
    if t.dtype is _torch.bfloat16:
        return BF16
    raise Q4Error(Q4_EINVAL, f"tensor of {t.dtype}: float16 or bfloat16 expected")


def _rows(t, name: str, dtype, device):
    """(rows, heads, dim, row stride) of t [rows][heads][dim], its heads and elements packed in a
    row.  `device`: the CUDA device's index."""
    if t.dtype is not dtype or t.get_device() != device:
        raise Q4Error(Q4_EINVAL, f"{name}: {t.dtype} on {t.device}, {dtype} on cuda:{device} expected")
    if t.dim() != 3:
        raise Q4Error(Q4_ESHAPE, f"{name}: shape {tuple(t.shape)}, [rows][heads][dim] expected")
    n, m, d = t.shape
    rs, hs, es = t.stride()
    if (es != 1 and d != 1) or (hs != d and m != 1):
        raise Q4Error(Q4_ESHAPE, f"{name}: the heads of a row must lie one after the other")
    return n, m, d, rs if n > 1 else m * d          # torch gives a single row any stride


def _want(name: str, got, want):
    raise Q4Error(Q4_ESHAPE, f"{name}: shape {got}, {want} expected")


def _ints(t, name: str, device, n: int):
    if t.dtype is not _torch.int32 or t.get_device() != device:
        raise Q4Error(Q4_EINVAL, f"{name}: {t.dtype} on {t.device}, int32 on cuda:{device} expected")
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise Q4Error(Q4_ESHAPE, f"{name}: {n} contiguous entries expected")
    return t.data_ptr()


class PagedKV:
    """A paged cache of keys and values: k and v [pages][page_size][heads][head_dim] (any strides,
    the same for both, head_dim contiguous; a permuted view of pools laid out [pages][heads][..]
    will do) and the page table, int32 [sequences][pages of a sequence].  Keeps the tensors alive."""

    def __init__(self, k, v, table):
        dt = _dtype_code(k)
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype or v.stride() != k.stride():
            raise Q4Error(Q4_ESHAPE, "k and v: one shape, type and layout [pages][page_size][heads][head_dim]")
        if k.stride(3) != 1 and k.shape[3] != 1:
            raise Q4Error(Q4_ESHAPE, "k and v: head_dim must be contiguous")
        if table.dtype != _torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise Q4Error(Q4_ESHAPE, "table: int32 [sequences][pages of a sequence] expected")
        if not (k.device == v.device == table.device) or k.device.type != "cuda":
            raise Q4Error(Q4_EINVAL, "k, v and table: one CUDA device expected")
        self.k, self.v, self.table = k, v, table
        self.device, self.dtype = k.device, k.dtype
        pages, size, heads, dim = k.shape
        self.index, self.heads, self.dim, self.seqs = k.get_device(), heads, dim, table.shape[0]
        ps, ts, hs, _ = k.stride()
        cols = table.shape[1]
        self.args = q4gemv_kv(k.data_ptr(), v.data_ptr(), table.data_ptr(), pages, size, heads, dim, ps, ts, hs,
                              table.stride(0) if table.shape[0] > 1 else cols, cols, dt)
        self.ref = ctypes.byref(self.args)


class Q4Gemv:
    """Owns one library handle on one device; methods take torch tensors."""

    def __init__(self, device: int = 0):
        st, h = q4gemv_create(device)
        if st != Q4_OK:
            raise Q4Error(st, q4gemv_strerror(st))
        self.h = h
        self.device = device

    def close(self):
        if self.h:
            q4gemv_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, st: int):
        if st != Q4_OK:
            raise Q4Error(st, q4gemv_last_error(self.h) or q4gemv_strerror(st))

    def packed_bytes(self, N: int, K: int) -> int:
        return q4gemv_packed_bytes(N, K)

    def repack(self, gguf, N: int, K: int, out=None, stream=None):
        """gguf: uint8 CUDA tensor of N*(K/32)*18 bytes -> packed uint8 tensor."""
        import torch
        if out is None:
            out = torch.empty(q4gemv_packed_bytes(N, K), dtype=torch.uint8, device=gguf.device)
        self._check(q4gemv_repack(self.h, _ptr(gguf), _ptr(out), N, K, _stream(stream)))
        return out

    def run(self, W_packed, x, N: int, K: int, out=None, stream=None):
        """x: f16 CUDA tensor [M][K] (or [K]) -> y f16 [M][N]."""
        import torch
        x2 = x.reshape(-1, K)
        M = x2.shape[0]
        if out is None:
            out = torch.empty((M, N), dtype=torch.float16, device=x.device)
        self._check(q4gemv_run(self.h, _ptr(W_packed), _ptr(x2), _ptr(out), M, N, K,
                               _stream(stream)))
        return out

    def run_swiglu(self, W_packed, gate_up, N: int, K: int, out=None, stream=None):
        """gate_up: f16 CUDA tensor [2K] ([gate | up]) -> y f16 [N] = W (SiLU(gate) * up)."""
        import torch
        if out is None:
            out = torch.empty(N, dtype=torch.float16, device=gate_up.device)
        self._check(q4gemv_run_swiglu(self.h, _ptr(W_packed), _ptr(gate_up), _ptr(out), N, K,
                                      _stream(stream)))
        return out

    def repack_q8_0(self, gguf, N: int, K: int, out=None, stream=None):
        """gguf: uint8 CUDA tensor of N*(K/32)*34 bytes -> packed Q8_0 tensor."""
        import torch
        if out is None:
            out = torch.empty(q4gemv_q8_0_packed_bytes(N, K), dtype=torch.uint8, device=gguf.device)
        self._check(q4gemv_q8_0_repack(self.h, _ptr(gguf), _ptr(out), N, K, _stream(stream)))
        return out

    def run_q8_0(self, W_packed, x, N: int, K: int, out=None, stream=None):
        """x: f16 CUDA tensor [M][K] (M <= 256) -> y f16 [M][N] for a packed Q8_0 W."""
        import torch
        x2 = x.reshape(-1, K)
        M = x2.shape[0]
        if out is None:
            out = torch.empty((M, N), dtype=torch.float16, device=x.device)
        self._check(q4gemv_q8_0_run(self.h, _ptr(W_packed), _ptr(x2), _ptr(out), M, N, K,
                                    _stream(stream)))
        return out

    def run_stack(self, layers, x_in, hidden: int, qkv_n: int, ffn: int, x_out=None,
                  trace_x=None, trace_y=None, stream=None):
        """layers: list of (qkv, o, gate_up, down) packed tensors."""
        import torch
        if x_out is None:
            x_out = torch.empty(hidden, dtype=torch.float16, device=x_in.device)
        arr = (q4gemv_layer * len(layers))()
        for i, (a, b, c, d) in enumerate(layers):
            arr[i] = q4gemv_layer(_ptr(a), _ptr(b), _ptr(c), _ptr(d))
        self._check(q4gemv_run_stack(self.h, arr, len(layers), hidden, qkv_n, ffn, _ptr(x_in),
                                     _ptr(x_out), _ptr(trace_x), _ptr(trace_y), _stream(stream)))
        return x_out

    def run_stack_gated(self, layers, x_in, hidden: int, qkv_n: int, ffn: int, x_out=None, stream=None):
        """The step with each down GEMV fed SiLU(gate) * up (see the header)."""
        import torch
        if x_out is None:
            x_out = torch.empty(hidden, dtype=torch.float16, device=x_in.device)
        arr = (q4gemv_layer * len(layers))()
        for i, (a, b, c, d) in enumerate(layers):
            arr[i] = q4gemv_layer(_ptr(a), _ptr(b), _ptr(c), _ptr(d))
        self._check(q4gemv_run_stack_gated(self.h, arr, len(layers), hidden, qkv_n, ffn, _ptr(x_in),
                                           _ptr(x_out), _stream(stream)))
        return x_out

    def init_comm(self, world: int, rank: int, uid: bytes):
        """Joins the `world`-GPU communicator of the row-sharded step as `rank`."""
        self._check(q4gemv_comm_init(self.h, world, rank, uid))

    def peer_export(self, world: int, rank: int, hidden: int, qkv_n: int, ffn: int) -> bytes:
        """Allocates this rank's exchange buffer for the peer-memory sharded step
        and returns the blob every rank must receive (e.g. all_gather_object)."""
        st, blob = q4gemv_peer_export(self.h, world, rank, hidden, qkv_n, ffn)
        self._check(st)
        return blob

    def peer_open(self, blobs):
        """Maps every rank's exchange buffer; `blobs`: the world's blobs in rank order.
        run_stack_sharded then gathers over peer memory for these shapes."""
        self._check(q4gemv_peer_open(self.h, b"".join(blobs)))

    def peer_close(self):
        self._check(q4gemv_peer_close(self.h))

    def run_stack_sharded(self, layers_local, x_in, hidden: int, qkv_n: int, ffn: int, x_out=None,
                          stream=None):
        """layers_local: this rank's (qkv, o, gate_up, down) row slices (packed tensors, or
        None for a slice of 0 rows)."""
        import torch
        if x_out is None:
            x_out = torch.empty(hidden, dtype=torch.float16, device=x_in.device)
        arr = (q4gemv_layer * len(layers_local))()
        for i, (a, b, c, d) in enumerate(layers_local):
            arr[i] = q4gemv_layer(_ptr(a), _ptr(b), _ptr(c), _ptr(d))
        self._check(q4gemv_run_stack_sharded(self.h, arr, len(layers_local), hidden, qkv_n, ffn,
                                             _ptr(x_in), _ptr(x_out), _stream(stream)))
        return x_out

    # ---- token mixing: start int32 [sequences + 1] (rows of each sequence), length int32
    # [sequences] (its tokens in the cache, the new ones counted), all on the handle's device ----

    def _on_device(self, index):
        if index != self.device:
            raise Q4Error(Q4_EINVAL, f"tensors on device {index}, the handle is on cuda:{self.device}")

    def _stream_of(self, stream) -> int:
        if stream is None:
            return _raw_stream(self.device)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def _new(self, like, shape, stream):
        """An output of the type and device of `like`, from the pool of the stream that writes it."""
        if stream is None:
            return like.new_empty(shape)
        if not hasattr(stream, "cuda_stream"):
            stream = _torch.cuda.ExternalStream(int(stream), device=self.device)
        with _torch.cuda.stream(stream):
            return like.new_empty(shape)

    def rope_freqs(self, rot: int, base: float = 10000.0, kind: int = ROPE_PLAIN, factor: float = 1.0,
                   trained: float = 0.0, lo: float = 1.0, hi: float = 32.0):
        """float64 [rot/2] on the handle's device: radians per position of each pair."""
        st, f = q4gemv_rope_freqs(kind, rot, base, factor, trained, lo, hi)
        if st != Q4_OK:
            raise Q4Error(st, f"rope_freqs: {q4gemv_strerror(st)}")
        return _torch.tensor(f, dtype=_torch.float64, device=f"cuda:{self.device}")

    def kv_append(self, cache, start, length, k, v, q=None, q_out=None, freqs=None,
                  interleaved: bool = False, amp: float = 1.0, pos=None, stream=None):
        """Appends k, v [rows][heads][head_dim] to the cache, k rotated; returns q
        [rows][q_heads][head_dim] rotated (None without q).  freqs: float64 [rot/2] or None (no
        rotation); pos: int32 [rows] rotation positions, by default the places in the cache."""
        dev, dt, heads, dim = cache.index, cache.dtype, cache.heads, cache.dim
        self._on_device(dev)
        n_seqs = length.numel()
        if cache.seqs < n_seqs:
            raise Q4Error(Q4_ESHAPE, "fewer page-table rows than sequences")
        rows, m, d, ks = _rows(k, "k", dt, dev)
        if m != heads or d != dim:
            _want("k", (rows, m, d), (rows, heads, dim))
        n, m, d, vs = _rows(v, "v", dt, dev)
        if n != rows or m != heads or d != dim:
            _want("v", (n, m, d), (rows, heads, dim))
        qs = qos = hq = 0
        qp = qop = None
        if q is not None:
            n, hq, d, qs = _rows(q, "q", dt, dev)
            if n != rows or d != dim:
                _want("q", (n, hq, d), (rows, hq, dim))
            if q_out is None:
                q_out = self._new(q, q.shape, stream)
            n, m, d, qos = _rows(q_out, "q_out", dt, dev)
            if n != rows or m != hq or d != dim:
                _want("q_out", (n, m, d), (rows, hq, dim))
            qp, qop = q.data_ptr(), q_out.data_ptr()
        rope = None
        if freqs is not None:
            if freqs.dtype is not _torch.float64 or freqs.get_device() != dev or not freqs.is_contiguous():
                raise Q4Error(Q4_EINVAL, "freqs: contiguous float64 on the cache's device expected")
            rope = q4gemv_rope(freqs.data_ptr(), 2 * freqs.numel(), interleaved, amp)
        self._check(_kv_append(
            self.h, cache.ref, rows, n_seqs, _ints(start, "start", dev, n_seqs + 1),
            _ints(length, "length", dev, n_seqs), None if pos is None else _ints(pos, "pos", dev, rows), rope,
            qp, qs, hq, k.data_ptr(), ks, v.data_ptr(), vs, qop, qos, self._stream_of(stream)))
        return q_out if q is not None else None

    def attn_paged(self, cache, start, length, q, out=None, scale: float | None = None,
                   causal: bool = True, window: int = 0, max_new: int | None = None, stream=None):
        """Attention of q [rows][q_heads][head_dim] over the cache (default scale
        1/sqrt(head_dim)); max_new: the most new tokens of a sequence, where known."""
        dev, dt, dim = cache.index, cache.dtype, cache.dim
        self._on_device(dev)
        n_seqs = length.numel()
        if cache.seqs < n_seqs:
            raise Q4Error(Q4_ESHAPE, "fewer page-table rows than sequences")
        rows, hq, d, qs = _rows(q, "q", dt, dev)
        if d != dim:
            _want("q", (rows, hq, d), (rows, hq, dim))
        if out is None:
            out = self._new(q, q.shape, stream)
        n, m, d, os_ = _rows(out, "out", dt, dev)
        if n != rows or m != hq or d != dim:
            _want("out", (n, m, d), (rows, hq, dim))
        self._check(_attn_paged(
            self.h, cache.ref, rows, n_seqs, _ints(start, "start", dev, n_seqs + 1),
            _ints(length, "length", dev, n_seqs), (rows or 1) if max_new is None else max_new,
            q.data_ptr(), qs, hq, out.data_ptr(), os_, dim ** -0.5 if scale is None else scale,
            causal, window, self._stream_of(stream)))
        return out

    def linattn(self, q, k, v, log_decay, start, state, state_out=None, slots=None, scale: float = 1.0,
                out=None, max_new: int | None = None, stream=None):
        """Linear attention with decay: q, k [rows][qk_heads][k_dim], v [rows][v_heads][v_dim],
        log_decay float32 [rows][v_heads] (an expanded row: fixed decays), state float32
        [slots][v_heads][k_dim][v_dim] (updated in place unless state_out is given; None: from
        zeros into state_out).  Returns (out, state_out)."""
        if state_out is None:
            state_out = state
        if state_out is None:
            raise Q4Error(Q4_EINVAL, "linattn: neither state nor state_out")
        dev = state_out.get_device()
        self._on_device(dev)
        n_seqs = start.numel() - 1
        dt, code = q.dtype, _dtype_code(q)
        rows, hk, dk, qs = _rows(q, "q", dt, dev)
        n, m, d, ks = _rows(k, "k", dt, dev)
        if n != rows or m != hk or d != dk:
            _want("k", (n, m, d), (rows, hk, dk))
        n, hv, dv, vs = _rows(v, "v", dt, dev)
        if n != rows:
            _want("v", (n, hv, dv), (rows, hv, dv))
        if out is None:
            out = self._new(q, (rows, hv, dv), stream)
        n, m, d, os_ = _rows(out, "out", dt, dev)
        if n != rows or m != hv or d != dv:
            _want("out", (n, m, d), (rows, hv, dv))
        if log_decay.dtype is not _torch.float32 or log_decay.get_device() != dev or \
                log_decay.shape != (rows, hv) or (hv > 1 and log_decay.stride(1) != 1):
            raise Q4Error(Q4_ESHAPE, f"log_decay: float32 [{rows}][{hv}] on cuda:{dev} expected")
        shape = state_out.shape
        if len(shape) != 4 or shape[1:] != (hv, dk, dv) or state_out.dtype is not _torch.float32 or \
                not state_out.is_contiguous() or \
                (state is not None and state is not state_out and
                 (state.shape != shape or state.dtype is not _torch.float32 or state.get_device() != dev or
                  not state.is_contiguous())):
            raise Q4Error(Q4_ESHAPE, f"state: contiguous float32 [slots][{hv}][{dk}][{dv}] on cuda:{dev} expected, "
                          "the same for state_out")
        a = q4gemv_linattn_args(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(state), state_out.data_ptr(),
            None if slots is None else _ints(slots, "slots", dev, n_seqs), out.data_ptr(), qs, ks, vs,
            log_decay.stride(0) if rows > 1 else hv, os_, shape[0], hk, hv, dk, dv, scale, code)
        self._check(_linattn(self.h, a, rows, n_seqs, _ints(start, "start", dev, n_seqs + 1),
                             (rows or 1) if max_new is None else max_new, self._stream_of(stream)))
        return out, state_out

    def run_stack_mixed(self, layers, mixers, x_in, hidden: int, ffn: int, q_heads: int, kv_heads: int,
                        length, freqs=None, interleaved: bool = False, amp: float = 1.0, x_out=None,
                        stream=None):
        """One token's decode step with a token mixer in every layer.  layers: (qkv, o, gate_up,
        down) packed tensors; mixers: for each layer a PagedKV (attention) or a pair (log_decay
        float32 [q_heads], state float32 [q_heads][D][D]) (linear attention), D = hidden/q_heads;
        length: int32 [1], the sequence's tokens with this one."""
        d = hidden // q_heads
        if len(mixers) != len(layers):
            raise Q4Error(Q4_ESHAPE, "run_stack_mixed: one mixer a layer expected")
        if x_in.dtype is not _torch.float16 or x_in.numel() != hidden or not x_in.is_contiguous():
            raise Q4Error(Q4_ESHAPE, f"x_in: contiguous float16 [{hidden}] expected")
        self._on_device(x_in.get_device())
        la = (q4gemv_layer * len(layers))(*[q4gemv_layer(*(t.data_ptr() for t in row)) for row in layers])
        ma = (q4gemv_mixer * len(layers))()
        for i, m in enumerate(mixers):
            if isinstance(m, PagedKV):
                self._on_device(m.index)
                ma[i] = q4gemv_mixer(MIX_ATTENTION, m.args, None, None)
                continue
            g, s = m
            for t, shape in ((g, (q_heads,)), (s, (q_heads, d, d))):
                if t.dtype is not _torch.float32 or t.shape != shape or not t.is_contiguous():
                    raise Q4Error(Q4_ESHAPE, f"mixer {i}: contiguous float32 {shape} expected")
                self._on_device(t.get_device())
            ma[i] = q4gemv_mixer(MIX_LINEAR, q4gemv_kv(), g.data_ptr(), s.data_ptr())
        rope = None
        if freqs is not None:
            if freqs.dtype is not _torch.float64 or not freqs.is_contiguous():
                raise Q4Error(Q4_EINVAL, "freqs: contiguous float64 expected")
            self._on_device(freqs.get_device())
            rope = q4gemv_rope(freqs.data_ptr(), 2 * freqs.numel(), interleaved, amp)
        if x_out is None:
            x_out = self._new(x_in, (hidden,), stream)
        elif x_out.dtype is not _torch.float16 or x_out.numel() != hidden or not x_out.is_contiguous():
            raise Q4Error(Q4_ESHAPE, f"x_out: contiguous float16 [{hidden}] expected")
        self._on_device(x_out.get_device())
        self._check(_lib.q4gemv_run_stack_mixed(
            self.h, la, ma, len(layers), hidden, ffn, q_heads, kv_heads, rope,
            _ints(length, "length", self.device, 1), x_in.data_ptr(), x_out.data_ptr(), self._stream_of(stream)))
        return x_out

    def sync_status(self, stream=None) -> int:
        return q4gemv_sync_status(self.h, _stream(stream))

    def set_fault(self, which: str):
        self._check(q4gemv_set_fault(self.h, which))


def stack_trace_dims(hidden: int, qkv_n: int, ffn: int):
    """Row strides of the trace_x / trace_y buffers of q4gemv_run_stack."""
    return max(hidden, ffn), max(qkv_n, hidden, 2 * ffn)
