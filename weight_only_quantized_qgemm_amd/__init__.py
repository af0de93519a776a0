"""Python binding of the qgemm C ABI (include/qgemm.h, qgemm_attention.h, qgemm_w8a8.h): argument marshalling only.

Every step of the GEMM runs in the HIP library ``libqgemm.so`` built next to this file;
torch serves only for device memory and the current stream.  Importing this package
fails loudly when the library has not been built.

Quick use::

    import weight_only_quantized_qgemm_amd as q
    p = q.problem(M, N, K, "int4", group_size=128)
    codes, scales, alpha = q.quantize(p, w_nk)          # host, numpy
    wpk, spk = q.pack(p, codes, scales)                  # host, numpy
    ... upload with torch, then q.run(p, A, wpk_dev, spk_dev, alpha_dev, out, ws)
"""
import ctypes
import importlib
import os
import threading

import numpy as np
# torch first: it loads its HIP runtime (soname libamdhip64.so.7), and the library below then
# binds to that same runtime instance, so torch's pointers and streams are valid in it.  Loading
# the library first would bring in a second runtime that cannot share the device with torch's.
import torch  # noqa: F401

_PKG = os.path.dirname(os.path.abspath(__file__))
# QGEMM_LIB_PATH selects another build of the same library (the CPU tests load the
# host-sanitizer build this way); by default the in-tree libqgemm.so.
LIB_PATH = os.environ.get("QGEMM_LIB_PATH") or os.path.join(_PKG, "libqgemm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m weight_only_quantized_qgemm_amd._build` (hipcc, gfx950)")
_lib = ctypes.CDLL(LIB_PATH)

# ----------------------------------------------------------------------------- enums
OK, ERR_INVALID_ARGUMENT, ERR_UNSUPPORTED, ERR_MISALIGNED, ERR_WORKSPACE_TOO_SMALL, ERR_HIP = range(6)
DT_F16, DT_BF16, DT_F32, DT_INT4, DT_FP8_E4M3, DT_FP4_E2M1, DT_INT2, DT_NF4 = range(8)
SCALE_GROUP_F16, SCALE_TENSOR_F32, SCALE_BLOCK16_E4M3, SCALE_GROUP_F16_LUT16 = range(4)
KERNEL_AUTO, KERNEL_DECODE, KERNEL_PREFILL, KERNEL_PREFILL_STREAMK, KERNEL_PREFILL_TRANSFORM = range(5)


ATTENTION_AUTO, ATTENTION_ROWS, ATTENTION_TILES = range(3)
GATE_NONE, GATE_SILU, GATE_GELU_TANH = range(3)
W8A8_AUTO, W8A8_ROWS, W8A8_TILES = range(3)
W8A8_SUMS_AUTO, W8A8_SUMS_WHOLE = range(2)


class Problem(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("a_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("scale_layout", ctypes.c_int32),
                ("kernel_hint", ctypes.c_int32), ("split_k_hint", ctypes.c_int32),
                ("tile_hint", ctypes.c_int32)]


assert ctypes.sizeof(Problem) == 56


class NormRope(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("max_pos", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class Cache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("group_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Attention(ctypes.Structure):
    _fields_ = [("cache", Cache), ("total_q", ctypes.c_int64), ("batch", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("max_q_len", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("window", ctypes.c_int32), ("scale", ctypes.c_float), ("kernel_hint", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 2)]


class AddNorm(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class W8A8(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("out_dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("kernel_hint", ctypes.c_int32), ("split_hint", ctypes.c_int32),
                ("tile_hint", ctypes.c_int32), ("sums", ctypes.c_int32)]


assert (ctypes.sizeof(NormRope), ctypes.sizeof(Cache), ctypes.sizeof(Attention)) == (48, 32, 80)
assert (ctypes.sizeof(AddNorm), ctypes.sizeof(W8A8)) == (32, 48)

_P = ctypes.POINTER(Problem)
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_lib.qgemm_quantize.argtypes = [_P, _vp, _vp, _vp, ctypes.POINTER(ctypes.c_float)]
_lib.qgemm_pack.argtypes = [_P, _vp, _vp, _vp, ctypes.POINTER(_sz), _vp, ctypes.POINTER(_sz)]
_lib.qgemm_workspace_bytes.argtypes = [_P, ctypes.POINTER(_sz)]
_lib.qgemm_run.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.qgemm_run_bias.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.qgemm_run_no_alloc.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.qgemm_plan_describe.argtypes = [_P, ctypes.c_char_p, _sz]
_lib.qgemm_status_string.argtypes = [ctypes.c_int]
_lib.qgemm_status_string.restype = ctypes.c_char_p
_lib.qgemm_last_error.argtypes = []
_lib.qgemm_last_error.restype = ctypes.c_char_p
_lib.qgemm_version.restype = ctypes.c_int32
_i64 = ctypes.c_int64
_NRP, _CP, _AP = ctypes.POINTER(NormRope), ctypes.POINTER(Cache), ctypes.POINTER(Attention)
_lib.qgemm_qk_norm_rope.argtypes = [_NRP, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp]
_lib.qgemm_cache_bytes.argtypes = [_CP, ctypes.POINTER(_sz)]
_lib.qgemm_cache_write.argtypes = [_CP, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
_lib.qgemm_cache_read.argtypes = [_CP, _vp, _vp, _i64, _vp, _vp, _vp]
_lib.qgemm_attention_workspace_bytes.argtypes = [_AP, ctypes.POINTER(_sz)]
_lib.qgemm_attention.argtypes = [_AP, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _sz, _vp]
_lib.qgemm_attention_describe.argtypes = [_AP, ctypes.c_char_p, _sz]
_ANP, _W8P = ctypes.POINTER(AddNorm), ctypes.POINTER(W8A8)
_lib.qgemm_add_norm.argtypes = [_ANP, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp]
_lib.qgemm_w8a8_quantize.argtypes = [_W8P, _vp, _vp, _vp]
_lib.qgemm_w8a8_workspace_bytes.argtypes = [_W8P, ctypes.POINTER(_sz)]
_lib.qgemm_w8a8_run.argtypes = [_W8P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.qgemm_w8a8_describe.argtypes = [_W8P, ctypes.c_char_p, _sz]
NO_ALLOC_SCRATCH_BYTES = (32 << 20) + (64 << 10)    # QGEMM_NO_ALLOC_SCRATCH_BYTES of include/qgemm.h
for _f in ("qgemm_quantize", "qgemm_pack", "qgemm_workspace_bytes", "qgemm_run", "qgemm_run_bias",
           "qgemm_run_no_alloc", "qgemm_plan_describe", "qgemm_qk_norm_rope", "qgemm_cache_bytes", "qgemm_cache_write",
           "qgemm_cache_read", "qgemm_attention_workspace_bytes", "qgemm_attention", "qgemm_attention_describe",
           "qgemm_add_norm", "qgemm_w8a8_quantize", "qgemm_w8a8_workspace_bytes", "qgemm_w8a8_run", "qgemm_w8a8_describe"):
    getattr(_lib, _f).restype = ctypes.c_int

lib = _lib


class QgemmError(RuntimeError):
    def __init__(self, status, detail):
        self.status = status
        self.detail = detail
        super().__init__(f"{_lib.qgemm_status_string(status).decode()}: {detail}")


def _check(status):
    if status != OK:
        raise QgemmError(status, _lib.qgemm_last_error().decode())


# ----------------------------------------------------------------------------- problems
_FORMATS = {
    "int4": (DT_F16, DT_INT4, SCALE_GROUP_F16, DT_F16),
    "fp8": (DT_BF16, DT_FP8_E4M3, SCALE_TENSOR_F32, DT_BF16),
    "fp8h": (DT_F16, DT_FP8_E4M3, SCALE_TENSOR_F32, DT_F16),      # FP8 weights, fp16 activations
    "fp4": (DT_BF16, DT_FP4_E2M1, SCALE_BLOCK16_E4M3, DT_BF16),
    "int2": (DT_F16, DT_INT2, SCALE_GROUP_F16, DT_F16),             # W2A16
    "nf4": (DT_F16, DT_NF4, SCALE_GROUP_F16_LUT16, DT_F16),         # 4-bit code-book index
}
GROUP_SCALED = ("int4", "int2", "nf4")


def problem(M, N, K, fmt, group_size=None, out_dtype=None, kernel_hint=KERNEL_AUTO, split_k_hint=0,
            tile_hint=0):
    """Problem descriptor for one of the formats 'int4', 'int2', 'nf4', 'fp8' (bf16
    activations), 'fp8h' (fp16 activations), 'fp4'."""
    a, w, sl, o = _FORMATS[fmt]
    if group_size is None:
        group_size = {"int4": 128, "int2": 128, "nf4": 128, "fp8": 0, "fp8h": 0, "fp4": 16}[fmt]
    if out_dtype is not None:
        o = out_dtype
    return Problem(M, N, K, a, w, o, group_size, sl, kernel_hint, split_k_hint, tile_hint)


def fmt_of(p):
    if p.w_dtype == DT_FP8_E4M3:
        return "fp8h" if p.a_dtype == DT_F16 else "fp8"
    return {DT_INT4: "int4", DT_INT2: "int2", DT_NF4: "nf4", DT_FP4_E2M1: "fp4"}[p.w_dtype]


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    return x.data_ptr()          # torch tensor


# ----------------------------------------------------------------------------- host calls
def quantize(p, w_nk):
    """fp32 [N, K] weights -> (canonical codes uint8, canonical scales or None, alpha).

    NF4 scales are one flat fp16 (uint16) array: the 16 code-book entries, then [K/G][N]."""
    w = np.ascontiguousarray(w_nk, dtype=np.float32)
    N, K = int(p.N), int(p.K)
    assert w.shape == (N, K)
    f = fmt_of(p)
    codes = np.empty((N, K) if f in ("fp8", "fp8h") else (N, K // 4) if f == "int2" else (N, K // 2), np.uint8)
    scales = None
    if f in ("int4", "int2"):
        scales = np.empty((K // p.group_size, N), np.uint16)
    elif f == "nf4":
        scales = np.empty(16 + (K // p.group_size) * N, np.uint16)
    elif f == "fp4":
        scales = np.empty((N, K // 16), np.uint8)
    alpha = ctypes.c_float(0.0)
    _check(_lib.qgemm_quantize(ctypes.byref(p), w.ctypes.data, codes.ctypes.data,
                               None if scales is None else scales.ctypes.data, ctypes.byref(alpha)))
    return codes, scales, float(alpha.value)


def packed_sizes(p):
    wb, sb = _sz(0), _sz(0)
    _check(_lib.qgemm_pack(ctypes.byref(p), None, None, None, ctypes.byref(wb), None, ctypes.byref(sb)))
    return wb.value, sb.value


def pack(p, codes, scales):
    """Canonical codes / scales (host) -> packed device-layout bytes (host numpy uint8)."""
    wsz, ssz = packed_sizes(p)
    codes = np.ascontiguousarray(codes)
    wpk = np.empty(wsz, np.uint8)
    spk = np.empty(max(ssz, 0), np.uint8)
    if scales is not None:
        scales = np.ascontiguousarray(scales)
    wb, sb = _sz(wsz), _sz(ssz)
    _check(_lib.qgemm_pack(ctypes.byref(p), codes.ctypes.data,
                           None if scales is None else scales.ctypes.data,
                           wpk.ctypes.data, ctypes.byref(wb),
                           spk.ctypes.data if ssz else None, ctypes.byref(sb)))
    return wpk, (spk if ssz else None)


def workspace_bytes(p):
    n = _sz(0)
    _check(_lib.qgemm_workspace_bytes(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def plan_describe(p):
    """The launch qgemm_run would make for this problem, as one line of text."""
    buf = ctypes.create_string_buffer(512)
    _check(_lib.qgemm_plan_describe(ctypes.byref(p), buf, 512))
    return buf.value.decode()


def plan_fields(p):
    """plan_describe as a dict: {"kernel": ..., key: value, ...} (values as text)."""
    head, *rest = plan_describe(p).split()
    return {"kernel": head, **dict(f.split("=", 1) for f in rest)}


# ----------------------------------------------------------------------------- device calls
def alloc_workspace(p, device="cuda"):
    """A zero-filled workspace of the size qgemm_workspace_bytes reports (or None)."""
    import torch
    n = workspace_bytes(p)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device)


def run(p, A, w_packed, s_packed, alpha, out, workspace=None, stream=None, bias=None):
    """Enqueue out = A . dequant(W) (* alpha) (+ bias) on `stream` (default: torch's current
    stream); qgemm_run, or qgemm_run_bias when a bias is given."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if bias is None:
        _check(_lib.qgemm_run(ctypes.byref(p), _ptr(A), _ptr(w_packed), _ptr(s_packed), _ptr(alpha),
                              _ptr(out), _ptr(workspace), ws_bytes, stream))
    else:
        _check(_lib.qgemm_run_bias(ctypes.byref(p), _ptr(A), _ptr(w_packed), _ptr(s_packed), _ptr(alpha),
                                   _ptr(bias), _ptr(out), _ptr(workspace), ws_bytes, stream))


def run_no_alloc(p, A, w_packed, s_packed, alpha, out, stream=None, bias=None):
    """qgemm_run_no_alloc: as run(), with the library's static per-GPU scratch as the split-K
    workspace (no workspace argument; nothing is allocated).  Calls that overlap in time on
    one GPU race."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    _check(_lib.qgemm_run_no_alloc(ctypes.byref(p), _ptr(A), _ptr(w_packed), _ptr(s_packed), _ptr(alpha),
                                   _ptr(bias), _ptr(out), stream))


def run_raw(p, A, w_packed, s_packed, alpha, out, workspace, workspace_bytes_, stream):
    """qgemm_run on raw integer addresses; returns the status (no exception)."""
    return _lib.qgemm_run(ctypes.byref(p), A, w_packed, s_packed, alpha, out, workspace,
                          workspace_bytes_, stream)


def run_bias_raw(p, A, w_packed, s_packed, alpha, bias, out, workspace, workspace_bytes_, stream):
    """qgemm_run_bias on raw integer addresses; returns the status (no exception)."""
    return _lib.qgemm_run_bias(ctypes.byref(p), A, w_packed, s_packed, alpha, bias, out, workspace,
                               workspace_bytes_, stream)


def last_error():
    return _lib.qgemm_last_error().decode()


def status_string(st):
    return _lib.qgemm_status_string(st).decode()


def version():
    return int(_lib.qgemm_version())


# ----------------------------------------------------------------------------- attention operators
# The device calls below, those of the 8-bit operators too, are made once per layer and token: their tensors are checked, and the C function
# called, in csrc/qgemm_calls.cpp.  A tensor of the wrong type, shape or strides, or that is not on the call's GPU,
# raises ValueError.
def _stream(stream, x):
    """The handle of `stream`; by default that of torch's current stream."""
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


class _Calls:
    """Stands for the compiled module until the first call loads it: programs that call the products only need not have it."""
    _lock = threading.Lock()

    def __getattr__(self, name):
        global _calls_ready
        with self._lock:
            if _calls_ready is self:
                try:
                    module = importlib.import_module("._calls", __name__)
                except ImportError as e:
                    raise ImportError("the _calls module is missing or of another Python: build it with "
                                      "`python -m weight_only_quantized_qgemm_amd._build`") from e
                module.setup(*(ctypes.cast(f, _vp).value for f in (_lib.qgemm_qk_norm_rope, _lib.qgemm_cache_write,
                                                                   _lib.qgemm_cache_read, _lib.qgemm_attention,
                                                                   _lib.qgemm_add_norm, _lib.qgemm_w8a8_run)),
                             torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8,
                             torch.float8_e4m3fn,
                             # the raw stream handle of a device, without building a Stream object for it
                             getattr(torch._C, "_cuda_getCurrentRawStream", None), _stream)
                _calls_ready = module
        return getattr(_calls_ready, name)


# the calls go through _calls_ready, which becomes the module once it is set up (importing it binds _calls before)
_calls = _calls_ready = _Calls()


def norm_rope_problem(tokens, q_heads, kv_heads, head_dim, dtype=DT_F16, rot_dim=None, max_pos=0, interleaved=False,
                      norm=True, eps=1e-6):
    """Descriptor of qk_norm_rope; rot_dim defaults to the whole head, 0 turns nothing."""
    return NormRope(tokens, q_heads, kv_heads, head_dim, head_dim if rot_dim is None else rot_dim, max_pos, dtype,
                    int(interleaved), int(norm), eps, 0)


def qk_norm_rope(p, q, k, q_weight, k_weight, positions, cos_sin, q_out, k_out, stream=None):
    """Enqueue the norm and rotation of the heads of q and k (qgemm_qk_norm_rope).  The tensors are
    [tokens, heads, head_dim], each with its own token stride; outputs may be the inputs."""
    st = _calls_ready.qk_norm_rope(p, q, k, q_weight, k_weight, positions, cos_sin, q_out, k_out, stream)
    if st:
        _check(st)


def cache(num_pages, page_size, kv_heads, head_dim, dtype=DT_F16, group_size=None):
    """Descriptor of a 4-bit paged key/value cache; group_size defaults to the whole head."""
    return Cache(num_pages, page_size, kv_heads, head_dim, head_dim if group_size is None else group_size, dtype, 0)


def cache_bytes(c):
    n = _sz(0)
    _check(_lib.qgemm_cache_bytes(ctypes.byref(c), ctypes.byref(n)))
    return n.value


def alloc_cache(c, device="cuda"):
    """A zero-filled cache buffer (every slot reads as zeros)."""
    return torch.zeros(cache_bytes(c), dtype=torch.uint8, device=device)


def cache_write(c, data, k, v, slots, stream=None):
    """Enqueue the quantization of k, v [tokens, kv_heads, head_dim] into the int64 slots."""
    st = _calls_ready.cache_write(c, data, k, v, slots, stream)
    if st:
        _check(st)


def cache_read(c, data, slots, k_out, v_out, stream=None):
    """Enqueue the values of the slots into k_out, v_out [tokens, kv_heads, head_dim], contiguous."""
    st = _calls_ready.cache_read(c, data, slots, k_out, v_out, stream)
    if st:
        _check(st)


def attention_problem(c, batch, total_q, q_heads, max_q_len, max_pages, causal=True, window=0, scale=None,
                      kernel_hint=ATTENTION_AUTO):
    """Descriptor of attention over the cache `c`; scale defaults to head_dim ** -0.5."""
    return Attention(c, total_q, batch, q_heads, max_q_len, max_pages, int(causal), window,
                     c.head_dim ** -0.5 if scale is None else scale, kernel_hint, (0, 0))


def attention_workspace_bytes(p):
    n = _sz(0)
    _check(_lib.qgemm_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def alloc_attention_workspace(p, device="cuda"):
    """A zero-filled workspace of the size qgemm_attention_workspace_bytes reports (or None)."""
    n = attention_workspace_bytes(p)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def attention_describe(p):
    """The launch qgemm_attention would make for this problem, as one line of text."""
    buf = ctypes.create_string_buffer(512)
    _check(_lib.qgemm_attention_describe(ctypes.byref(p), buf, 512))
    return buf.value.decode()


def attention(p, q, data, page_table, seq_lens, q_start, out, workspace=None, stream=None):
    """Enqueue attention of q [total_q, q_heads, head_dim] over the cache into out (qgemm_attention)."""
    st = _calls_ready.attention(p, q, data, page_table, seq_lens, q_start, out, workspace, stream)
    if st:
        _check(st)


# ----------------------------------------------------------------------------- 8-bit operators
# Values in 8 bits are torch.float8_e4m3fn codes and fp32 scales: of activations [K / 128, tokens], of weights
# [row blocks, K / 128].
def add_norm_problem(tokens, dim, dtype=DT_F16, out_dtype=None, norm=True, eps=1e-6):
    """Descriptor of add_norm; out_dtype is DT_FP8_E4M3 or, by default, dtype."""
    return AddNorm(tokens, dim, dtype, dtype if out_dtype is None else out_dtype, int(norm), eps, 0)


def add_norm(p, x, residual, weight, sum_out, y, y_scales=None, stream=None):
    """Enqueue y = norm(x + residual) * weight and sum_out = x + residual (qgemm_add_norm).  x, residual and
    sum_out are [tokens, dim], each with its own token stride; residual, weight and sum_out may be None."""
    st = _calls_ready.add_norm(p, x, residual, weight, sum_out, y, y_scales, stream)
    if st:
        _check(st)


def w8a8_problem(M, N, K, out_dtype=DT_BF16, gate=GATE_NONE, kernel_hint=W8A8_AUTO, split_hint=0, tile_hint=0,
                 sums=W8A8_SUMS_AUTO):
    """Descriptor of a product of 8-bit activations and weights, or with a gate of a pair of them.  W8A8_SUMS_WHOLE has every
    product enter its sum whole where the default leaves 16-bit outputs to the faster e4m3 matrix instruction."""
    return W8A8(M, N, K, out_dtype, gate, kernel_hint, split_hint, tile_hint, sums)


def w8a8_quantize(p, w):
    """fp32 [rows, K] weights (rows = N, or 2 N with a gate) -> (codes uint8 [rows, K], scales fp32
    [row blocks, K / 128]), host numpy.  On the GPU the codes are viewed as torch.float8_e4m3fn."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    parts = 1 if p.gate == GATE_NONE else 2
    if w.shape != (parts * p.N, p.K):
        raise ValueError(f"w must be [{parts * p.N}, {p.K}], got {list(w.shape)}")
    codes = np.empty(w.shape, np.uint8)
    scales = np.empty((parts * -(-int(p.N) // 128), p.K // 128), np.float32)
    _check(_lib.qgemm_w8a8_quantize(ctypes.byref(p), w.ctypes.data, codes.ctypes.data, scales.ctypes.data))
    return codes, scales


def w8a8_workspace_bytes(p):
    """Bytes of workspace of one problem.  They do not grow with M: a program that runs several M needs the largest of theirs."""
    n = _sz(0)
    _check(_lib.qgemm_w8a8_workspace_bytes(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def alloc_w8a8_workspace(p, device="cuda"):
    """A zero-filled workspace of the size qgemm_w8a8_workspace_bytes reports (or None); of several problems, one that serves them all."""
    n = w8a8_workspace_bytes(p) if isinstance(p, W8A8) else max(map(w8a8_workspace_bytes, p), default=0)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def w8a8_describe(p):
    """The launch qgemm_w8a8_run would make for this problem, as one line of text."""
    buf = ctypes.create_string_buffer(512)
    _check(_lib.qgemm_w8a8_describe(ctypes.byref(p), buf, 512))
    return buf.value.decode()


def w8a8_run(p, A, a_scales, W, w_scales, out, out_scales=None, workspace=None, stream=None):
    """Enqueue the product, or with a gate the gated pair, of A [M, K] and W (qgemm_w8a8_run)."""
    st = _calls_ready.w8a8_run(p, A, a_scales, W, w_scales, out, out_scales, workspace, stream)
    if st:
        _check(st)
