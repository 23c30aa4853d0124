"""Python binding of libfp4 -- FP4 (E2M1) block-scaled quantisation and GEMM
for AMD Instinct MI355X (gfx950).

The C ABI (include/fp4.h) is exposed under the same names (``fp4_quantize``,
``fp4_dequantize``, ``fp4_gemm``, ``fp4_gemm_ex``, ``fp4_gemm_grouped``, ``fp4_gemm_w4a8``, ``fp4_scale_bytes``,
``fp4_workspace_size``, ``fp4_status_string``; the decode step's ``fp4_kv_append``, ``fp4_attn_decode``,
``fp4_kv_evict``, ``fp4_logprobs``, ``fp4_logprobs_backward``), taking raw device pointers as
integers.  The tensor helpers below only allocate outputs with torch and
marshal ``data_ptr()`` / the current stream into those calls: every step of the
computation runs in the HIP kernels of libfp4.so.  There is no fallback -- if
the library is not built, or no GPU is present, the calls fail loudly.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
# FP4_LIB_PATH selects another build of the same library (the tests use it
# for the host-sanitized build); the default is the in-tree libfp4.so.
LIB_PATH = os.environ.get("FP4_LIB_PATH") or os.path.join(HERE, "libfp4.so")

# enum fp4_fmt / fp4_dtype / fp4_op, flags
MXFP4, NVFP4, MXFP4_OCP, MXFP8, MXFP8_OCP = 0, 1, 2, 3, 4
F32, BF16 = 0, 1
OP_QUANTIZE, OP_GEMM, OP_GEMM_GROUPED = 0, 1, 2
TS_GIVEN = 1
Q_SR, Q_2D = 2, 4
# enum fp4_out / fp4_act (fp4_gemm_ex)
OUT_F32, OUT_BF16, OUT_MXFP4, OUT_MXFP4_OCP, OUT_NVFP4 = 0, 1, 2, 3, 4
ACT_NONE, ACT_RELU = 0, 1
# enum fp4_kv_fmt (cache rows)
KV_BF16, KV_MXFP8, KV_MXFP4 = 0, 1, 2

FUNCTIONS = ("fp4_scale_bytes", "fp4_workspace_size", "fp4_quantize", "fp4_quantize_noalloc", "fp4_quantize_sr",
             "fp4_quantize_ex",
             "fp4_hadamard16", "fp4_dequantize", "fp4_gemm", "fp4_gemm_ex",
             "fp4_gemm_grouped", "fp4_gemm_nvfp4_act", "fp4_gemm_nvfp4_act_supported", "fp4_gemm_w4a8",
             "fp4_status_string", "fp4_set_debug", "fp4_kv_append", "fp4_attn_decode_workspace", "fp4_attn_decode",
             "fp4_kv_evict_workspace", "fp4_kv_evict", "fp4_logprobs_workspace", "fp4_logprobs",
             "fp4_logprobs_backward")


class KVCacheStruct(ctypes.Structure):
    """struct fp4_kv_cache of include/fp4.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("fmt", ctypes.c_int32)]


class Fp4Error(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, fp4_status_string(status), status))


_lib = None


def lib():
    """Load libfp4.so (built in-tree by block_scaled_fp4_03_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfp4.so is not built (run python -m block_scaled_fp4_03_amd.build)")
        # torch first: its HIP runtime then satisfies the library's
        # libamdhip64.so.7, so both share one runtime (streams, allocations).
        # Loaded the other way round, torch loads a second copy of the
        # runtime under another name, and the library's own HIP calls do not
        # see torch's device.
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, U32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
        F32C, CACHE = ctypes.c_float, ctypes.POINTER(KVCacheStruct)
        sig = {
            "fp4_scale_bytes": (I64, [I32, I64, I64]),
            "fp4_workspace_size": (SZ, [I32, I32, I64, I64, I64, I32]),
            "fp4_quantize": (I32, [P, I32, P, P, P, I64, I64, I32, U32, P, SZ, P]),
            "fp4_quantize_noalloc": (I32, [P, I32, P, P, P, I64, I64, I32, U32, P]),
            "fp4_quantize_sr": (I32, [P, I32, P, P, P, I64, I64, I32, U32, ctypes.c_uint64, P, SZ, P]),
            "fp4_quantize_ex": (I32, [P, I32, P, P, P, I64, I64, I32, U32, ctypes.c_uint64, P, SZ, P]),
            "fp4_hadamard16": (I32, [P, I32, P, I32, I64, I64, ctypes.c_uint64, P]),
            "fp4_dequantize": (I32, [P, P, P, I32, P, I32, I64, I64, P]),
            "fp4_gemm": (I32, [P, P, P, P, P, P, P, I64, I64, I64, I32, I32, P, SZ, P]),
            "fp4_gemm_ex": (I32, [P, P, P, P, P, P, P, I32, P, P, P, I64, I64, I64, I32, I32, P]),
            "fp4_gemm_grouped": (I32, [P, P, I64, P, P, I32, P, P, P, P, P, I64, I64, I64, I32, I32, P, SZ, P]),
            "fp4_gemm_nvfp4_act": (I32, [P, I32, P, U32, P, P, P, P, I64, I64, I64, I32, P]),
            "fp4_gemm_nvfp4_act_supported": (I32, [I64, I64, I64, I32]),
            "fp4_gemm_w4a8": (I32, [P, P, P, P, P, I32, P, I64, I64, I64, I32, P]),
            "fp4_status_string": (ctypes.c_char_p, [I32]),
            "fp4_set_debug": (I32, [I32]),
            "fp4_kv_append": (I32, [CACHE, P, P, I32, I64, I64, P, I64, I64, P, P, I64, P]),
            "fp4_attn_decode_workspace": (SZ, [CACHE, I64, I64, I64, I32]),
            "fp4_attn_decode": (I32, [CACHE, P, I32, I64, P, I64, P, I64, I64, I64, I64, F32C, P, I32, P, P, P, I64,
                                      P, SZ, P]),
            "fp4_kv_evict_workspace": (SZ, [CACHE, I64, I64, I64]),
            "fp4_kv_evict": (I32, [CACHE, P, I64, P, P, I64, CACHE, P, I64, P, P, I64, P, I64, I64, I64, I64, P, SZ,
                                   P]),
            "fp4_logprobs_workspace": (SZ, [I64, I64, I32]),
            "fp4_logprobs": (I32, [P, I32, I64, I64, I64, F32C, P, I32, P, P, P, I32, P, P, P, SZ, P]),
            "fp4_logprobs_backward": (I32, [P, I32, I64, I64, I64, F32C, P, I32, P, P, P, P, P, I64, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


# ---- raw C-ABI calls (integers for pointers) --------------------------------
def fp4_set_debug(on):
    """Debug mode on (1) or off (0); returns the previous setting."""
    return lib().fp4_set_debug(1 if on else 0)


def fp4_status_string(status):
    return lib().fp4_status_string(int(status)).decode()


def fp4_scale_bytes(fmt, rows, K):
    return lib().fp4_scale_bytes(fmt, rows, K)


def fp4_workspace_size(op, fmt, M, N, K, E=0):
    return lib().fp4_workspace_size(op, fmt, M, N, K, E)


def fp4_quantize(x, fmt, codes, block_scales, tensor_scale, rows, K, in_dtype, flags, workspace, workspace_bytes,
                 stream):
    return lib().fp4_quantize(x, fmt, codes, block_scales, tensor_scale, rows, K, in_dtype, flags, workspace,
                              workspace_bytes, stream)


def fp4_quantize_noalloc(x, fmt, codes, block_scales, tensor_scale, rows, K, in_dtype, flags, stream):
    return lib().fp4_quantize_noalloc(x, fmt, codes, block_scales, tensor_scale, rows, K, in_dtype, flags, stream)


def fp4_quantize_sr(x, fmt, codes, block_scales, tensor_scale, rows, K, in_dtype, flags, seed, workspace,
                    workspace_bytes, stream):
    return lib().fp4_quantize_sr(x, fmt, codes, block_scales, tensor_scale, rows, K, in_dtype, flags,
                                 int(seed) & 0xFFFFFFFFFFFFFFFF, workspace, workspace_bytes, stream)


def fp4_quantize_ex(x, fmt, codes, block_scales, tensor_scale, rows, K, in_dtype, flags, seed, workspace,
                    workspace_bytes, stream):
    return lib().fp4_quantize_ex(x, fmt, codes, block_scales, tensor_scale, rows, K, in_dtype, flags,
                                 int(seed) & 0xFFFFFFFFFFFFFFFF, workspace, workspace_bytes, stream)


def fp4_hadamard16(x, in_dtype, y, out_dtype, rows, K, seed, stream):
    return lib().fp4_hadamard16(x, in_dtype, y, out_dtype, rows, K, int(seed) & 0xFFFFFFFFFFFFFFFF, stream)


def fp4_dequantize(codes, block_scales, tensor_scale, fmt, out, out_dtype, rows, K, stream):
    return lib().fp4_dequantize(codes, block_scales, tensor_scale, fmt, out, out_dtype, rows, K, stream)


def fp4_gemm(A, sA, B, sB, tsA, tsB, C, M, N, K, fmt, out_dtype, workspace, workspace_bytes, stream):
    return lib().fp4_gemm(A, sA, B, sB, tsA, tsB, C, M, N, K, fmt, out_dtype, workspace, workspace_bytes, stream)


def fp4_gemm_ex(A, sA, B, sB, tsA, tsB, bias, act, C, C_scales, C_tensor_scale, M, N, K, fmt, out, stream):
    return lib().fp4_gemm_ex(A, sA, B, sB, tsA, tsB, bias, act, C, C_scales, C_tensor_scale, M, N, K, fmt, out,
                             stream)


def fp4_gemm_grouped(A, sA, A_rows, row_idx, group_off, E, B, sB, tsA, tsB, C, total_rows, N, K, fmt, out_dtype,
                     workspace, workspace_bytes, stream):
    return lib().fp4_gemm_grouped(A, sA, A_rows, row_idx, group_off, E, B, sB, tsA, tsB, C, total_rows, N, K, fmt,
                                  out_dtype, workspace, workspace_bytes, stream)


def fp4_gemm_nvfp4_act(X, x_dtype, x_tensor_scale, flags, W, sW, tsW, C, M, N, K, out_dtype, stream):
    return lib().fp4_gemm_nvfp4_act(X, x_dtype, x_tensor_scale, flags, W, sW, tsW, C, M, N, K, out_dtype, stream)


def fp4_gemm_nvfp4_act_supported(M, N, K, x_dtype):
    return lib().fp4_gemm_nvfp4_act_supported(M, N, K, x_dtype)


def fp4_gemm_w4a8(A, sA, B, sB, bias, act, C, M, N, K, out_dtype, stream):
    return lib().fp4_gemm_w4a8(A, sA, B, sB, bias, act, C, M, N, K, out_dtype, stream)


def fp4_kv_append(cache, k, v, in_dtype, k_stride, v_stride, page_table, table_width, seqs, seq, pos, rows, stream):
    return lib().fp4_kv_append(cache, k, v, in_dtype, k_stride, v_stride, page_table, table_width, seqs, seq, pos,
                               rows, stream)


def fp4_attn_decode_workspace(cache, B, q_heads, max_len, weights):
    return lib().fp4_attn_decode_workspace(cache, B, q_heads, max_len, weights)


def fp4_attn_decode(cache, q, q_dtype, q_stride, page_table, table_width, lens, B, q_heads, max_len, window, scale,
                    out, out_dtype, lse, weights_in, weights_out, weights_stride, workspace, workspace_bytes, stream):
    return lib().fp4_attn_decode(cache, q, q_dtype, q_stride, page_table, table_width, lens, B, q_heads, max_len,
                                 window, scale, out, out_dtype, lse, weights_in, weights_out, weights_stride,
                                 workspace, workspace_bytes, stream)


def fp4_kv_evict_workspace(cache, B, max_len, budget):
    return lib().fp4_kv_evict_workspace(cache, B, max_len, budget)


def fp4_kv_evict(src, src_table, src_width, lens, weights, weights_stride, dst, dst_table, dst_width, out_lens,
                 out_weights, out_stride, kept, B, max_len, budget, recent, workspace, workspace_bytes, stream):
    return lib().fp4_kv_evict(src, src_table, src_width, lens, weights, weights_stride, dst, dst_table, dst_width,
                              out_lens, out_weights, out_stride, kept, B, max_len, budget, recent, workspace,
                              workspace_bytes, stream)


def fp4_logprobs_workspace(N, V, top_k):
    return lib().fp4_logprobs_workspace(N, V, top_k)


def fp4_logprobs(x, dtype, stride_, N, V, scale, tokens, M, logp, entropy, lse, top_k, top_logp, top_index, workspace,
                 workspace_bytes, stream):
    return lib().fp4_logprobs(x, dtype, stride_, N, V, scale, tokens, M, logp, entropy, lse, top_k, top_logp,
                              top_index, workspace, workspace_bytes, stream)


def fp4_logprobs_backward(x, dtype, stride_, N, V, scale, tokens, M, lse, entropy, g_logp, g_entropy, dx, dx_stride,
                          stream):
    return lib().fp4_logprobs_backward(x, dtype, stride_, N, V, scale, tokens, M, lse, entropy, g_logp, g_entropy, dx,
                                       dx_stride, stream)


# ---- torch helpers: allocation + pointer/stream marshalling only -------------
def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(rc, where):
    if rc != 0:
        raise Fp4Error(rc, where)


def _need(t, name, dtypes=None, numel=None, device=None, ndim=None):
    """Reject, before any library call, an argument the C ABI would misread:
    not a tensor, not on a GPU, not contiguous (the kernels take a raw
    pointer and assume the documented dense layout), of another dtype (an
    int64 index read as int32 halves), too small, or on another device than
    the call's first operand.  Returns t."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor, got %s" % (name, type(t).__name__))
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dimensions, got shape %s" % (name, ndim, tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if numel is not None and t.numel() < numel:
        raise ValueError("%s holds %d elements, %d needed" % (name, t.numel(), numel))
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor, got device %s" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the call's operands on %s" % (name, t.device, device))
    return t


def _need_q(q, name, device=None):
    """Check a Quantized operand: codes, scales (and the NVFP4 tensor scale)
    contiguous uint8 / float32 GPU tensors of the sizes its format needs."""
    if not isinstance(q, Quantized):
        raise TypeError("%s must be a Quantized, got %s" % (name, type(q).__name__))
    torch = _torch()
    if q.fmt == NVFP4 and q.tensor_scale is None:
        raise ValueError("%s: an NVFP4 operand needs its tensor scale" % name)
    ncodes = q.rows * (q.K if is_fp8(q.fmt) else q.K // 2)
    _need(q.codes, name + ".codes", (torch.uint8,), ncodes, device)
    nbytes = fp4_scale_bytes(q.fmt, q.rows, q.K)
    if nbytes < 0:
        raise Fp4Error(int(nbytes), "fp4_scale_bytes")
    _need(q.scales, name + ".scales", (torch.uint8,), nbytes, device)
    if q.tensor_scale is not None:
        _need(q.tensor_scale, name + ".tensor_scale", (torch.float32,), 1, device)
    return q


def _need_out(t, name, shape, dtypes, device):
    _need(t, name, dtypes, None, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("expected float32 or bfloat16, got %s" % t.dtype)


def workspace(op, fmt, M, N, K, E=0, device="cuda"):
    """A zero-filled workspace tensor of the size the operation needs (or None)."""
    torch = _torch()
    n = fp4_workspace_size(op, fmt, M, N, K, E)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def is_fp8(fmt):
    """MXFP8 formats hold one E4M3 byte per element (the FP4 ones two codes per byte)."""
    return fmt in (MXFP8, MXFP8_OCP)


class Quantized:
    """codes (rows x K/2 uint8; MXFP8 rows x K), scales (tiled uint8), tensor_scale (1 float32 or None)."""

    def __init__(self, codes, scales, tensor_scale, fmt, rows, K):
        self.codes, self.scales, self.tensor_scale = codes, scales, tensor_scale
        self.fmt, self.rows, self.K = fmt, rows, K


def quantize(x, fmt, tensor_scale=None, ws=None, out=None, stream=None, sr_seed=None, two_d=False):
    """Quantise a 2-D float32/bfloat16 CUDA tensor along its last dimension.

    NVFP4: pass `tensor_scale` (a 1-element float32 tensor) to use a given
    scale; otherwise one is computed and returned in the result.  MXFP8 /
    MXFP8_OCP: E4M3 codes, one byte per element.  sr_seed:
    round the elements stochastically with that seed (fp4_quantize_sr).
    two_d: NVFP4 scales per 16 x 16 patch (fp4_quantize_ex, FP4_Q_2D)."""
    torch = _torch()
    _need(x, "x", (torch.float32, torch.bfloat16), ndim=2)
    rows, K = x.shape
    dev = x.device
    if tensor_scale is not None:
        _need(tensor_scale, "tensor_scale", (torch.float32,), 1, dev)
    if ws is not None:
        _need(ws, "ws", (torch.uint8,), None, dev)
    if out is not None:
        if (out.rows, out.K, out.fmt) != (rows, K, fmt):
            raise ValueError("out is a %d x %d matrix of format %d, x needs %d x %d of format %d"
                             % (out.rows, out.K, out.fmt, rows, K, fmt))
        if fmt == NVFP4 and out.tensor_scale is None:
            raise ValueError("out: an NVFP4 result needs a tensor-scale tensor")
        _need_q(out, "out", dev)
    if out is None:
        codes = torch.empty((rows, K if is_fp8(fmt) else K // 2), dtype=torch.uint8, device=dev)
        nbytes = fp4_scale_bytes(fmt, rows, K)
        if nbytes < 0:
            raise Fp4Error(int(nbytes), "fp4_scale_bytes")
        scales = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ts = None
        if fmt == NVFP4:
            ts = tensor_scale if tensor_scale is not None else torch.empty(1, dtype=torch.float32, device=dev)
        out = Quantized(codes, scales, ts, fmt, rows, K)
    flags = TS_GIVEN if (fmt == NVFP4 and tensor_scale is not None) else 0
    if fmt == NVFP4 and not flags and ws is None:
        ws = workspace(OP_QUANTIZE, fmt, rows, 0, K, device=dev)
    if two_d:
        rc = fp4_quantize_ex(_ptr(x), fmt, _ptr(out.codes), _ptr(out.scales), _ptr(out.tensor_scale), rows, K,
                             _dtype_code(x), flags | Q_2D | (Q_SR if sr_seed is not None else 0),
                             0 if sr_seed is None else sr_seed, _ptr(ws), 0 if ws is None else ws.numel(),
                             _stream(stream))
    elif sr_seed is None:
        rc = fp4_quantize(_ptr(x), fmt, _ptr(out.codes), _ptr(out.scales), _ptr(out.tensor_scale), rows, K,
                          _dtype_code(x), flags, _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
    else:
        rc = fp4_quantize_sr(_ptr(x), fmt, _ptr(out.codes), _ptr(out.scales), _ptr(out.tensor_scale), rows, K,
                             _dtype_code(x), flags, sr_seed, _ptr(ws), 0 if ws is None else ws.numel(),
                             _stream(stream))
    _check(rc, "fp4_quantize_sr" if sr_seed is not None else "fp4_quantize")
    return out


def hadamard16(x, seed, out_dtype=None, out=None, stream=None):
    """Random Hadamard transform of a 2-D float32/bfloat16 CUDA tensor on
    16-value blocks along its last dimension (fp4_hadamard16)."""
    torch = _torch()
    _need(x, "x", (torch.float32, torch.bfloat16), ndim=2)
    rows, K = x.shape
    if out is None:
        out = torch.empty((rows, K), dtype=x.dtype if out_dtype is None else out_dtype, device=x.device)
    _need_out(out, "out", (rows, K), (torch.float32, torch.bfloat16), x.device)
    rc = fp4_hadamard16(_ptr(x), _dtype_code(x), _ptr(out), _dtype_code(out), rows, K, seed, _stream(stream))
    _check(rc, "fp4_hadamard16")
    return out


def dequantize(q, out_dtype=None, stream=None):
    torch = _torch()
    _need_q(q, "q")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    out = torch.empty((q.rows, q.K), dtype=out_dtype, device=q.codes.device)
    rc = fp4_dequantize(_ptr(q.codes), _ptr(q.scales), _ptr(q.tensor_scale), q.fmt, _ptr(out), _dtype_code(out),
                        q.rows, q.K, _stream(stream))
    _check(rc, "fp4_dequantize")
    return out


def gemm(a, b, out_dtype=None, out=None, ws=None, stream=None):
    """C = A . B^T for quantised A (M x K) and B (N x K) of the same format."""
    torch = _torch()
    dev = _need_q(a, "a").codes.device
    _need_q(b, "b", dev)
    M, N, K = a.rows, b.rows, a.K
    if b.K != K or a.fmt != b.fmt:
        raise ValueError("operands disagree on K or format")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16 if out_dtype is None else out_dtype, device=dev)
    _need_out(out, "out", (M, N), (torch.float32, torch.bfloat16), dev)
    if ws is None:
        ws = workspace(OP_GEMM, a.fmt, M, N, K, device=dev)
    else:
        _need(ws, "ws", (torch.uint8,), None, dev)
    rc = fp4_gemm(_ptr(a.codes), _ptr(a.scales), _ptr(b.codes), _ptr(b.scales), _ptr(a.tensor_scale),
                  _ptr(b.tensor_scale), _ptr(out), M, N, K, a.fmt, _dtype_code(out), _ptr(ws),
                  0 if ws is None else ws.numel(), _stream(stream))
    _check(rc, "fp4_gemm")
    return out


def gemm_ex(a, b, bias=None, act=ACT_NONE, out=OUT_BF16, C=None, c_tensor_scale=None, stream=None):
    """C = act((A . B^T) * tsA * tsB + bias) in one kernel (see fp4_gemm_ex in
    include/fp4.h).  out: OUT_F32 / OUT_BF16 -> an M x N tensor; OUT_MXFP4 /
    OUT_MXFP4_OCP -> a Quantized M x N MXFP4 matrix (the next GEMM's A);
    OUT_NVFP4 -> a Quantized M x N NVFP4 matrix under c_tensor_scale (a
    1-element float32 CUDA tensor, required).  bias: N float32 CUDA tensor or
    None.  C: optional preallocated output (tensor, or Quantized for FP4
    output)."""
    torch = _torch()
    dev = _need_q(a, "a").codes.device
    _need_q(b, "b", dev)
    M, N, K = a.rows, b.rows, a.K
    if b.K != K or a.fmt != b.fmt:
        raise ValueError("operands disagree on K or format")
    if bias is not None:
        _need(bias, "bias", (torch.float32,), N, dev)
    fp4_out = out in (OUT_MXFP4, OUT_MXFP4_OCP, OUT_NVFP4)
    ofmt = {OUT_MXFP4: MXFP4, OUT_MXFP4_OCP: MXFP4_OCP, OUT_NVFP4: NVFP4}.get(out)
    if out == OUT_NVFP4:
        if c_tensor_scale is None:
            raise ValueError("OUT_NVFP4 needs c_tensor_scale (1-element float32 CUDA tensor)")
        _need(c_tensor_scale, "c_tensor_scale", (torch.float32,), 1, dev)
    if C is None:
        if fp4_out:
            nbytes = fp4_scale_bytes(ofmt, M, N)
            if nbytes < 0:
                raise Fp4Error(int(nbytes), "fp4_scale_bytes")
            C = Quantized(torch.empty((M, N // 2), dtype=torch.uint8, device=dev),
                          torch.empty(nbytes, dtype=torch.uint8, device=dev),
                          c_tensor_scale if out == OUT_NVFP4 else None, ofmt, M, N)
        else:
            C = torch.empty((M, N), dtype=torch.float32 if out == OUT_F32 else torch.bfloat16, device=dev)
    if fp4_out:
        if (C.rows, C.K) != (M, N):
            raise ValueError("C is a %d x %d matrix, the product %d x %d" % (C.rows, C.K, M, N))
        _need(C.codes, "C.codes", (torch.uint8,), M * (N // 2), dev)
        _need(C.scales, "C.scales", (torch.uint8,), max(0, fp4_scale_bytes(ofmt, M, N)), dev)
    else:
        _need_out(C, "C", (M, N), (torch.float32 if out == OUT_F32 else torch.bfloat16,), dev)
    cptr, sptr = (_ptr(C.codes), _ptr(C.scales)) if fp4_out else (_ptr(C), None)
    tsc = _ptr(c_tensor_scale) if out == OUT_NVFP4 else None
    rc = fp4_gemm_ex(_ptr(a.codes), _ptr(a.scales), _ptr(b.codes), _ptr(b.scales), _ptr(a.tensor_scale),
                     _ptr(b.tensor_scale), _ptr(bias), act, cptr, sptr, tsc, M, N, K, a.fmt, out, _stream(stream))
    _check(rc, "fp4_gemm_ex")
    return C


def gemm_w4a8(a, b, bias=None, act=ACT_NONE, out_dtype=None, out=None, stream=None):
    """C = act(A . B^T + bias) for MXFP8 activations A (M x K) and MXFP4
    weights B (N x K), FP32 accumulation (see fp4_gemm_w4a8 in include/fp4.h)."""
    torch = _torch()
    dev = _need_q(a, "a").codes.device
    _need_q(b, "b", dev)
    M, N, K = a.rows, b.rows, a.K
    if b.K != K or not is_fp8(a.fmt) or b.fmt not in (MXFP4, MXFP4_OCP):
        raise ValueError("A must be MXFP8 and B MXFP4 with the same K")
    if bias is not None:
        _need(bias, "bias", (torch.float32,), N, dev)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16 if out_dtype is None else out_dtype, device=dev)
    _need_out(out, "out", (M, N), (torch.float32, torch.bfloat16), dev)
    rc = fp4_gemm_w4a8(_ptr(a.codes), _ptr(a.scales), _ptr(b.codes), _ptr(b.scales), _ptr(bias), act, _ptr(out),
                       M, N, K, _dtype_code(out), _stream(stream))
    _check(rc, "fp4_gemm_w4a8")
    return out


def gemm_grouped(a, row_idx, group_off, b_codes, b_scales, N, K, fmt, b_tensor_scale=None, out_dtype=None,
                 out=None, ws=None, stream=None, pregather=True):
    """Grouped (mixture-of-experts) GEMM; see fp4_gemm_grouped in include/fp4.h.
    NVFP4: b_tensor_scale holds one float32 per expert.  pregather: pass a
    workspace (ws, or one allocated here) so that the call first copies the
    token rows into expert order; False runs the GEMM on the gathered rows."""
    torch = _torch()
    dev = _need_q(a, "a").codes.device
    if a.K != K or a.fmt != fmt:
        raise ValueError("a is %d x %d of format %d, the call K = %d, format %d" % (a.rows, a.K, a.fmt, K, fmt))
    # int32 indices: torch's default int64 (cumsum, argsort) would be read as
    # pairs of int32 halves.
    _need(row_idx, "row_idx", (torch.int32,), None, dev, ndim=1)
    _need(group_off, "group_off", (torch.int32,), 1, dev, ndim=1)
    E = group_off.numel() - 1
    total = row_idx.numel()
    nscale = fp4_scale_bytes(fmt, N, K)
    if nscale < 0:
        raise Fp4Error(int(nscale), "fp4_scale_bytes")
    _need(b_codes, "b_codes", (torch.uint8,), E * N * (K // 2), dev)
    _need(b_scales, "b_scales", (torch.uint8,), E * nscale, dev)
    if fmt == NVFP4 and (a.tensor_scale is None or b_tensor_scale is None):
        raise ValueError("NVFP4 needs a's tensor scale and b_tensor_scale (one float32 per expert)")
    if b_tensor_scale is not None:
        _need(b_tensor_scale, "b_tensor_scale", (torch.float32,), E if fmt == NVFP4 else 1, dev)
    if out is None:
        out = torch.empty((total, N), dtype=torch.bfloat16 if out_dtype is None else out_dtype, device=dev)
    _need_out(out, "out", (total, N), (torch.float32, torch.bfloat16), dev)
    if not pregather:
        ws = None
    elif ws is None:
        n = fp4_workspace_size(OP_GEMM_GROUPED, fmt, total, N, K, E)
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None   # no control words: not zeroed
    else:
        _need(ws, "ws", (torch.uint8,), None, dev)
    rc = fp4_gemm_grouped(_ptr(a.codes), _ptr(a.scales), a.rows, _ptr(row_idx), _ptr(group_off), E, _ptr(b_codes),
                          _ptr(b_scales), _ptr(a.tensor_scale), _ptr(b_tensor_scale), _ptr(out), total, N, K, fmt,
                          _dtype_code(out), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
    _check(rc, "fp4_gemm_grouped")
    return out


def gemm_nvfp4_act(x, w, tensor_scale=None, ts_out=None, out_dtype=None, out=None, stream=None):
    """C = quantise_nvfp4(x) . w^T in one call (see fp4_gemm_nvfp4_act in
    include/fp4.h).  x: M x K float32/bfloat16 CUDA tensor; w: NVFP4 Quantized.
    tensor_scale: given activation tensor scale (1-element float32 tensor), or
    None to compute it; ts_out: optional 1-element tensor receiving it."""
    torch = _torch()
    _need(x, "x", (torch.float32, torch.bfloat16), ndim=2)
    _need_q(w, "w", x.device)
    M, K = x.shape
    N = w.rows
    if w.K != K or w.fmt != NVFP4:
        raise ValueError("weights must be NVFP4 with the same K")
    for t, name in ((tensor_scale, "tensor_scale"), (ts_out, "ts_out")):
        if t is not None:
            _need(t, name, (torch.float32,), 1, x.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16 if out_dtype is None else out_dtype, device=x.device)
    _need_out(out, "out", (M, N), (torch.float32, torch.bfloat16), x.device)
    flags = TS_GIVEN if tensor_scale is not None else 0
    ts = tensor_scale if tensor_scale is not None else ts_out
    rc = fp4_gemm_nvfp4_act(_ptr(x), _dtype_code(x), _ptr(ts), flags, _ptr(w.codes), _ptr(w.scales),
                            _ptr(w.tensor_scale), _ptr(out), M, N, K, _dtype_code(out), _stream(stream))
    _check(rc, "fp4_gemm_nvfp4_act")
    return out


# ---- decode-step operators: cache, attention, eviction, log probabilities ------
# These calls take microseconds on the GPU, so their wrappers are kept short:
# one test for a well-formed tensor, with _need naming the fault of any other.
def _want(t, name, dtype, ndim, device, numel=None):
    """_need for one dtype and dimension count, quickly."""
    try:
        if (t.dtype is dtype and t.ndim == ndim and t.device == device and t.is_contiguous()
                and (numel is None or t.numel() >= numel)):
            return
    except AttributeError:
        pass
    _need(t, name, (dtype,), numel, device, ndim)


def _want_rows(t, name, ndim, device=None, like=None):
    """Check a float32 or bfloat16 tensor (with `like`: of its dtype and shape)
    whose dimensions after the first are dense and whose first may have any
    stride (columns of a wider matrix).  Returns its fp4_dtype and that
    stride."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor, got %s" % (name, type(t).__name__))
    code = F32 if t.dtype is torch.float32 else BF16 if t.dtype is torch.bfloat16 else None
    if code is None or (like is not None and t.dtype is not like.dtype):
        raise TypeError("%s must be %s, got %s"
                        % (name, "float32 or bfloat16" if like is None else like.dtype, t.dtype))
    sizes, strides = t.shape, t.stride()
    if len(sizes) != ndim:
        raise ValueError("%s must have %d dimensions, got shape %s" % (name, ndim, tuple(sizes)))
    if like is not None and sizes != like.shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(like.shape), tuple(sizes)))
    width = 1
    for i in range(ndim - 1, 0, -1):
        if strides[i] != width and sizes[i] != 1:
            raise ValueError("%s must be dense but for its first dimension, got strides %s" % (name, strides))
        width *= sizes[i]
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor, got device %s" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the call's operands on %s" % (name, t.device, device))
    if sizes[0] <= 1:
        return code, width
    if strides[0] < width:
        raise ValueError("%s has overlapping rows (strides %s)" % (name, strides))
    return code, strides[0]


def _run_on(stream, device):
    """The raw handle of the stream a call runs on: the given one, or the
    device's current one."""
    return stream.cuda_stream if stream is not None else _torch()._C._cuda_getCurrentRawStream(device.index)


def _alloc(stream, make, *args, **kw):
    """make(*args, **kw), a call's output or workspace, for the stream it runs
    on: from that stream's memory, so that what the current stream still does
    with memory freed there cannot meet the call's writes, and marked as used
    on the current stream too, where the caller goes on with it."""
    if stream is None:
        return make(*args, **kw)
    torch = _torch()
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    if t is not None:
        t.record_stream(torch.cuda.current_stream())
    return t


class KVCache:
    """A pool of key-value cache pages (struct fp4_kv_cache of include/fp4.h).

    k, v: the pool tensors, pages x kv_heads x page_size x row, where a row is
    head_dim bfloat16 values (format KV_BF16), head_dim uint8 E4M3 codes
    (KV_MXFP8) or head_dim / 2 uint8 bytes of E2M1 codes (KV_MXFP4); the MX
    formats also take k_scales, v_scales, uint8, pages x kv_heads x page_size x
    head_dim / 32.  The tensors are checked once, here; the object holds them.
    KVCache.empty allocates a pool."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        torch = _torch()
        _need(k, "k", (torch.bfloat16, torch.uint8), ndim=4)
        dev = k.device
        _need_out(v, "v", k.shape, (k.dtype,), dev)
        pages, heads, page_size, row = k.shape
        if k.dtype == torch.bfloat16:
            if k_scales is not None or v_scales is not None:
                raise ValueError("a bfloat16 cache has no scales")
            fmt, dim = KV_BF16, row
        else:
            for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
                _need(t, name, (torch.uint8,), None, dev, ndim=4)
            blocks = k_scales.shape[3]
            if blocks * 32 == row:
                fmt, dim = KV_MXFP8, row
            elif blocks * 16 == row:
                fmt, dim = KV_MXFP4, 2 * row
            else:
                raise ValueError("rows of %d bytes and %d scales are neither MXFP8 nor MXFP4" % (row, blocks))
            for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
                _need_out(t, name, (pages, heads, page_size, blocks), (torch.uint8,), dev)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.fmt, self.pages, self.kv_heads, self.page_size, self.head_dim = fmt, pages, heads, page_size, dim
        self.device = dev
        self.struct = KVCacheStruct(_ptr(k), _ptr(v), _ptr(k_scales), _ptr(v_scales), pages, page_size, heads, dim,
                                    fmt)
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, pages, page_size, kv_heads, head_dim, fmt=KV_BF16, device="cuda"):
        """A pool of uninitialised pages."""
        torch = _torch()
        if fmt not in (KV_BF16, KV_MXFP8, KV_MXFP4):
            raise ValueError("unknown cache format %r" % (fmt,))
        lead = (pages, kv_heads, page_size)
        if fmt == KV_BF16:
            return cls(*(torch.empty(lead + (head_dim,), dtype=torch.bfloat16, device=device) for _ in range(2)))
        row = head_dim if fmt == KV_MXFP8 else head_dim // 2
        return cls(*(torch.empty(lead + (w,), dtype=torch.uint8, device=device)
                     for w in (row, row, head_dim // 32, head_dim // 32)))


def _need_cache(cache, name="cache"):
    if not isinstance(cache, KVCache):
        raise TypeError("%s must be a KVCache, got %s" % (name, type(cache).__name__))
    return cache.device


def kv_append(cache, k, v, table, seq, pos, stream=None):
    """Write new keys and values (n x kv_heads x head_dim float32/bfloat16, any
    row stride) into the cache: row i becomes token pos[i] of sequence seq[i]
    of the page table (int32, sequences x pages); seq -1 skips a row.  See
    fp4_kv_append in include/fp4.h."""
    torch = _torch()
    dev = _need_cache(cache)
    code, ks = _want_rows(k, "k", 3, dev)
    shape = k.shape
    n = shape[0]
    if shape[1] != cache.kv_heads or shape[2] != cache.head_dim:
        raise ValueError("k must have shape %s, got %s" % ((n, cache.kv_heads, cache.head_dim), tuple(shape)))
    vs = _want_rows(v, "v", 3, dev, k)[1]
    i32 = torch.int32
    _want(table, "table", i32, 2, dev)
    _want(seq, "seq", i32, 1, dev, n)
    _want(pos, "pos", i32, 1, dev, n)
    seqs, width = table.shape
    rc = lib().fp4_kv_append(cache.ref, k.data_ptr(), v.data_ptr(), code, ks, vs, table.data_ptr(), width, seqs,
                             seq.data_ptr(), pos.data_ptr(), n, _run_on(stream, dev))
    if rc != 0:
        _check(rc, "fp4_kv_append")
    return cache


def attention_workspace(cache, batch, q_heads, max_len, weights=False):
    """A zero-filled workspace tensor for decode_attention (or None)."""
    torch = _torch()
    dev = _need_cache(cache)
    n = fp4_attn_decode_workspace(cache.struct, batch, q_heads, max_len, 1 if weights else 0)
    return torch.zeros(n, dtype=torch.uint8, device=dev) if n else None


def decode_attention(q, cache, table, lens, max_len=None, window=0, scale=None, out=None, out_dtype=None, lse=None,
                     weights=None, weights_out=None, ws=None, stream=None):
    """Attention of one new token per sequence over the paged cache; see
    fp4_attn_decode in include/fp4.h.

    q: batch x q_heads x head_dim float32/bfloat16 (any row stride); table:
    int32 batch x pages; lens: int32 batch.  max_len bounds lens (default: what
    the table holds).  scale: default 1 / sqrt(head_dim).  lse: optional
    float32 batch x q_heads output.  weights_out: optional float32 batch x
    kv_heads x (>= max_len) output of weights (or 0) plus every token's
    attention weight; it may be weights itself.  ws: attention_workspace's
    tensor, kept by the caller from call to call (one is allocated here if
    None).  Returns out (dtype of q, or out_dtype)."""
    torch = _torch()
    dev = _need_cache(cache)
    code, qs = _want_rows(q, "q", 3, dev)
    shape = q.shape
    B, heads, dim = shape
    if dim != cache.head_dim:
        raise ValueError("q has head_dim %d, the cache %d" % (dim, cache.head_dim))
    _want(table, "table", torch.int32, 2, dev)
    _want(lens, "lens", torch.int32, 1, dev, B)
    rows, width = table.shape
    if rows != B:
        raise ValueError("table has %d rows, q %d" % (rows, B))
    if max_len is None:
        max_len = width * cache.page_size
    if out is None:
        out = _alloc(stream, torch.empty, shape, dtype=q.dtype if out_dtype is None else out_dtype, device=dev)
        _dtype_code(out)
    else:
        _need_out(out, "out", shape, (torch.float32, torch.bfloat16), dev)
    if lse is not None:
        _need_out(lse, "lse", (B, heads), (torch.float32,), dev)
    stride = 0
    if weights_out is not None:
        _want(weights_out, "weights_out", torch.float32, 3, dev)
        stride = weights_out.shape[2]
        _need_out(weights_out, "weights_out", (B, cache.kv_heads, stride), (torch.float32,), dev)
        if weights is not None:
            _need_out(weights, "weights", (B, cache.kv_heads, stride), (torch.float32,), dev)
    elif weights is not None:
        raise ValueError("weights needs weights_out")
    if ws is None:
        ws = _alloc(stream, attention_workspace, cache, B, heads, max_len, weights_out is not None)
    else:
        _want(ws, "ws", torch.uint8, 1, dev)
    rc = lib().fp4_attn_decode(cache.ref, q.data_ptr(), code, qs, table.data_ptr(), width,
                               lens.data_ptr(), B, heads, max_len, window, dim ** -0.5 if scale is None else scale,
                               out.data_ptr(), code if out.dtype is q.dtype else 1 - code, _ptr(lse), _ptr(weights),
                               _ptr(weights_out), stride,
                               _ptr(ws), 0 if ws is None else ws.numel(), _run_on(stream, dev))
    if rc != 0:
        _check(rc, "fp4_attn_decode")
    return out


def evict_workspace(cache, batch, max_len, budget):
    """A zero-filled workspace tensor for kv_evict (or None)."""
    torch = _torch()
    dev = _need_cache(cache)
    n = fp4_kv_evict_workspace(cache.struct, batch, max_len, budget)
    return torch.zeros(n, dtype=torch.uint8, device=dev) if n else None


def kv_evict(cache, table, lens, weights, budget, recent, out_table, out_cache=None, ws=None, stream=None):
    """Keep `budget` tokens of every longer (sequence, kv head): the last
    `recent` and the largest accumulated attention weights; see fp4_kv_evict
    in include/fp4.h.

    weights: float32 batch x kv_heads x (>= what the table holds).  The kept
    tokens move, in order, to out_table's pages (of out_cache; default the
    same pool), which must not be pages that table reads.  ws:
    evict_workspace's tensor (one is allocated here if None).  Returns (lens
    int32 batch, weights float32 batch x kv_heads x what out_table holds, kept
    int32 batch x kv_heads x budget: old token numbers, then -1)."""
    torch = _torch()
    dev = _need_cache(cache)
    if out_cache is None:
        out_cache = cache
    elif _need_cache(out_cache, "out_cache") != dev:
        raise ValueError("out_cache is on %s, the call's operands on %s" % (out_cache.device, dev))
    _want(table, "table", torch.int32, 2, dev)
    B, width = table.shape
    _want(lens, "lens", torch.int32, 1, dev, B)
    _want(out_table, "out_table", torch.int32, 2, dev)
    if out_table.shape[0] != B:
        raise ValueError("out_table has %d rows, table %d" % (out_table.shape[0], B))
    if budget < 0:
        raise ValueError("budget is negative")
    cap, heads = width * cache.page_size, cache.kv_heads
    _want(weights, "weights", torch.float32, 3, dev)
    if weights.shape[0] != B or weights.shape[1] != heads or weights.shape[2] < cap:
        raise ValueError("weights must have shape (%d, %d, >= %d), got %s" % (B, heads, cap, tuple(weights.shape)))
    out_width = out_table.shape[1]
    room = max(out_width * cache.page_size, budget)
    out_lens = _alloc(stream, torch.empty, B, dtype=torch.int32, device=dev)
    out_weights = _alloc(stream, torch.empty, (B, heads, room), dtype=torch.float32, device=dev)
    kept = _alloc(stream, torch.empty, (B, heads, budget), dtype=torch.int32, device=dev)
    if ws is None:
        ws = _alloc(stream, evict_workspace, cache, B, cap, budget)
    else:
        _want(ws, "ws", torch.uint8, 1, dev)
    rc = lib().fp4_kv_evict(cache.ref, table.data_ptr(), width, lens.data_ptr(), weights.data_ptr(),
                            weights.shape[2], out_cache.ref, out_table.data_ptr(), out_width, out_lens.data_ptr(),
                            out_weights.data_ptr(), room, kept.data_ptr(), B, cap, budget, recent, _ptr(ws),
                            0 if ws is None else ws.numel(), _run_on(stream, dev))
    if rc != 0:
        _check(rc, "fp4_kv_evict")
    return out_lens, out_weights, kept


class LogProbs:
    """logprobs' results: logp (N x M), entropy, lse (N), top_logp, top_index (N x top_k, or None)."""

    def __init__(self, logp, entropy, lse, top_logp, top_index):
        self.logp, self.entropy, self.lse = logp, entropy, lse
        self.top_logp, self.top_index = top_logp, top_index


def logprobs_workspace(n, vocab, top_k=0, device="cuda"):
    """A zero-filled workspace tensor for logprobs (or None)."""
    torch = _torch()
    b = fp4_logprobs_workspace(n, vocab, top_k)
    return torch.zeros(b, dtype=torch.uint8, device=device) if b else None


def logprobs(x, tokens, top_k=0, scale=1.0, ws=None, stream=None):
    """Log probabilities of the given tokens (int32 N x M; outside [0, V):
    padding, 0) under softmax(scale * x), x: N x V float32/bfloat16 logits
    (any row stride), with the entropy, the log-sum-exp and the top_k <= 32
    largest alternatives; see fp4_logprobs in include/fp4.h.  ws:
    logprobs_workspace's tensor (one is allocated here if None).  The results
    carry no autograd history, also where x requires a gradient:
    logprobs_backward gives that of logp and the entropy."""
    torch = _torch()
    code, xs = _want_rows(x, "x", 2)
    dev = x.device
    N, V = x.shape
    _want(tokens, "tokens", torch.int32, 2, dev)
    rows, M = tokens.shape
    if rows != N:
        raise ValueError("tokens has %d rows, x %d" % (rows, N))
    f32 = torch.float32
    logp = _alloc(stream, torch.empty, (N, M), dtype=f32, device=dev)
    entropy = _alloc(stream, torch.empty, N, dtype=f32, device=dev)
    lse = _alloc(stream, torch.empty, N, dtype=f32, device=dev)
    top = index = None
    if top_k > 0:
        top = _alloc(stream, torch.empty, (N, top_k), dtype=f32, device=dev)
        index = _alloc(stream, torch.empty, (N, top_k), dtype=torch.int32, device=dev)
    if ws is None:
        ws = _alloc(stream, logprobs_workspace, N, V, top_k, dev)
    else:
        _want(ws, "ws", torch.uint8, 1, dev)
    rc = lib().fp4_logprobs(x.data_ptr(), code, xs, N, V, scale, tokens.data_ptr(), M, logp.data_ptr(),
                            entropy.data_ptr(), lse.data_ptr(), top_k, _ptr(top), _ptr(index), _ptr(ws),
                            0 if ws is None else ws.numel(), _run_on(stream, dev))
    if rc != 0:
        _check(rc, "fp4_logprobs")
    return LogProbs(logp, entropy, lse, top, index)


def logprobs_backward(x, tokens, lse, g_logp, entropy=None, g_entropy=None, scale=1.0, out=None, stream=None):
    """Gradient of logprobs with respect to x from the gradients of logp
    (N x M) and, if given, of the entropy (N; then entropy too); lse and
    entropy as logprobs returned them; see fp4_logprobs_backward in
    include/fp4.h.  Returns dx of x's dtype."""
    torch = _torch()
    code, xs = _want_rows(x, "x", 2)
    dev = x.device
    N, V = x.shape
    _want(tokens, "tokens", torch.int32, 2, dev)
    rows, M = tokens.shape
    if rows != N:
        raise ValueError("tokens has %d rows, x %d" % (rows, N))
    f32 = torch.float32
    _want(g_logp, "g_logp", f32, 2, dev)
    if g_logp.shape != tokens.shape:
        raise ValueError("g_logp must have shape %s, got %s" % (tuple(tokens.shape), tuple(g_logp.shape)))
    _want(lse, "lse", f32, 1, dev, N)
    if g_entropy is not None:
        if entropy is None:
            raise ValueError("g_entropy needs entropy")
        _want(g_entropy, "g_entropy", f32, 1, dev, N)
        _want(entropy, "entropy", f32, 1, dev, N)
    if out is None:
        out = _alloc(stream, torch.empty, (N, V), dtype=x.dtype, device=dev)
        os_ = V
    else:
        os_ = _want_rows(out, "out", 2, dev, x)[1]
    rc = lib().fp4_logprobs_backward(x.data_ptr(), code, xs, N, V, scale, tokens.data_ptr(), M,
                                     lse.data_ptr(), _ptr(entropy), g_logp.data_ptr(), _ptr(g_entropy),
                                     out.data_ptr(), os_, _run_on(stream, dev))
    if rc != 0:
        _check(rc, "fp4_logprobs_backward")
    return out
