"""Python binding of libfp8fg.so: fine-grained FP8 quantization and block-scaled
FP8 GEMM for AMD MI355X (gfx950).

The functions below carry the names of the C entry points declared in
include/fp8fg.h and only marshal arguments: they take torch tensors that live
on the GPU, check dtypes and shapes, pass raw device pointers and the current
HIP stream to the library, and raise Fp8fgError on a non-zero status.  Every
step of the computation runs in the library's HIP kernels; there is no other
implementation behind these names.  Outputs are allocated here with torch
unless the caller passes them in (``out=``/``q=``/``s=``).
"""
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8fg.so")

BSCALE_128x128 = 0
BSCALE_1x128 = 1
OUT_BF16 = 0
OUT_FP32 = 1
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1

ABI_VERSION = 16
EXPORTS = ("fp8_quant_act_1x128", "fp8_quant_weight_128x128", "fp8_gemm_blockscaled",
           "fp8_grouped_gemm_contiguous", "fp8_grouped_gemm_masked",
           "fp8_quant_act_1x128_bf16", "fp8_quant_weight_128x128_bf16", "fp8_requant_act_tokenwise",
           "fp8_quant_mx_1x32", "fp8_gemm_mx", "fp8_gemm_blockscaled_fp8out", "fp8_quant_fprop_operands",
           "fp8_tile_weights_decode", "fp8_grouped_gemm_masked_tiled", "fp8_gemm_blockscaled_fp8mfma",
           "fp8_grouped_gemm_contiguous_fp8out", "fp8_grouped_gemm_contiguous_mx", "fp8_grouped_gemm_masked_mx",
           "fp8_quant_mx_1x32_transposed", "fp8_grouped_gemm_masked_tiled_fp8out",
           "fp8_grouped_gemm_masked_tiled_mx", "moe_route", "moe_route_backward", "fp8_moe_dispatch_contiguous",
           "fp8_moe_dispatch_masked", "moe_combine", "fp8_moe_combine_backward", "fp8_swiglu", "fp8_swiglu_backward",
           "fp8_grouped_gemm_wgrad", "kv_assign_pages", "kv_release_pages", "rope", "fp8_kv_append",
           "fp8_kv_attention_workspace", "fp8_kv_attention", "fp8fg_status_string", "fp8fg_abi_version")
_COMPUTE = EXPORTS[:-2]


class Fp8fgError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")


_lib = None


def load_library(path=LIB_PATH):
    """Load (once) and return the ctypes handle of libfp8fg.so; raise if missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
                          "or `python fp8_fine_grained_amd/build.py`")
    lib = ctypes.CDLL(path)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.fp8_quant_act_1x128.argtypes = [vp, i64, i64, i32, vp, vp, vp]
    lib.fp8_quant_weight_128x128.argtypes = [vp, i64, i64, i32, vp, vp, vp]
    lib.fp8_gemm_blockscaled.argtypes = [vp, vp, vp, vp, i32, vp, i32, i64, i64, i64, vp]
    lib.fp8_gemm_blockscaled_fp8mfma.argtypes = [vp, vp, vp, vp, i32, vp, i32, i64, i64, i64, vp]
    lib.fp8_grouped_gemm_contiguous.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    lib.fp8_grouped_gemm_masked.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    lib.fp8_quant_act_1x128_bf16.argtypes = [vp, i64, i64, i32, vp, vp, vp]
    lib.fp8_quant_weight_128x128_bf16.argtypes = [vp, i64, i64, i32, vp, vp, vp]
    lib.fp8_requant_act_tokenwise.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    lib.fp8_quant_mx_1x32.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.fp8_quant_mx_1x32_transposed.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.fp8_gemm_mx.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    lib.fp8_gemm_blockscaled_fp8out.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    lib.fp8_quant_fprop_operands.argtypes = [vp, i32, i64, vp, i32, i64, i64, vp, vp, vp, vp, vp]
    lib.fp8_tile_weights_decode.argtypes = [vp, i64, i64, i64, vp, vp]
    lib.fp8_grouped_gemm_masked_tiled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    lib.fp8_grouped_gemm_contiguous_fp8out.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, vp]
    lib.fp8_grouped_gemm_masked_tiled_fp8out.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, vp]
    lib.fp8_grouped_gemm_masked_tiled_mx.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    lib.fp8_grouped_gemm_contiguous_mx.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    lib.fp8_grouped_gemm_masked_mx.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    f32 = ctypes.c_float
    lib.moe_route.argtypes = [vp, i32, i64, vp, i64, i64, i64, i64, i64, i32, i32, i32, f32, vp, vp, vp]
    lib.moe_route_backward.argtypes = [vp, i32, i64, vp, vp, i64, i64, i64, i32, i32, f32, vp, vp]
    lib.fp8_moe_dispatch_contiguous.argtypes = [vp, i32, i64, i64, vp, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp]
    lib.fp8_moe_dispatch_masked.argtypes = [vp, i32, i64, i64, vp, i64, i64, i64, i64, vp, vp, vp, vp, vp]
    lib.moe_combine.argtypes = [vp, i32, i64, i64, vp, vp, i64, i64, vp, i32, vp]
    lib.fp8_moe_combine_backward.argtypes = [vp, i32, i64, i64, vp, i32, i64, vp, vp, i64, vp, vp, i64, vp, vp, vp, vp]
    lib.fp8_swiglu.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, vp]
    lib.fp8_swiglu_backward.argtypes = [vp, vp, vp, i32, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.fp8_grouped_gemm_wgrad.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    lib.kv_assign_pages.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, vp, vp]
    lib.kv_release_pages.argtypes = [vp, vp, vp, i64, i64, i64, vp, i64, vp, vp, vp, vp]
    lib.rope.argtypes = [vp, i64, vp, i64, i64, vp, i64, vp, i64, i64, i32, vp, vp, i64, i64, i64, i32, f32, i32, vp]
    lib.fp8_kv_append.argtypes = [vp, i64, vp, i64, i32, vp, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp]
    lib.fp8_kv_attention_workspace.argtypes = [i64, i64, i64, i64, i64, i64, i64, ctypes.POINTER(i64)]
    lib.fp8_kv_attention.argtypes = [vp, i64, vp, vp, vp, vp, i64, i64, vp, i64, vp, vp, i64, i64, i64, i64, i64, f32, vp, vp, vp, i64, vp]
    for name in _COMPUTE:
        getattr(lib, name).restype = ctypes.c_int
    lib.fp8fg_status_string.argtypes = [ctypes.c_int]
    lib.fp8fg_status_string.restype = ctypes.c_char_p
    lib.fp8fg_abi_version.argtypes = []
    lib.fp8fg_abi_version.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status):
    return load_library().fp8fg_status_string(int(status)).decode()


def abi_version():
    return load_library().fp8fg_abi_version()


def _ptr(t):
    return t.data_ptr() if t is not None else None


# The current stream's handle on t's device.  torch.cuda.current_stream builds a
# Stream object around the same handle, 2 us of host time per call; it serves where
# torch has no entry for the handle alone.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t):
    if _raw_stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return _raw_stream(t.get_device())


def _check(fn, status):
    if status != 0:
        raise Fp8fgError(fn, status)


def _need(t, dtype, shape, name):
    if t.is_cuda and t.dtype == dtype and t.shape == shape and t.is_contiguous():
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _nb(n):
    """Number of 128-wide groups along an axis of length n (a last partial group counts)."""
    return (n + 127) // 128


def _empty(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


def _quant_act(fn, x, dtype, transpose_out, q, s):
    M, K = x.shape
    _need(x, dtype, (M, K), "x")
    qs = (K, M) if transpose_out else (M, K)
    ss = (_nb(M), K) if transpose_out else (_nb(K), M)
    q = _empty(qs, torch.uint8, x) if q is None else q
    s = _empty(ss, torch.float32, x) if s is None else s
    _need(q, torch.uint8, qs, "q")
    _need(s, torch.float32, ss, "s")
    _check(fn, getattr(load_library(), fn)(_ptr(x), M, K, int(bool(transpose_out)), _ptr(q), _ptr(s), _stream(x)))
    return q, s


def _quant_weight(fn, w, dtype, transpose_out, q, s):
    N, K = w.shape
    _need(w, dtype, (N, K), "w")
    qs = (K, N) if transpose_out else (N, K)
    ss = (_nb(K), _nb(N)) if transpose_out else (_nb(N), _nb(K))
    q = _empty(qs, torch.uint8, w) if q is None else q
    s = _empty(ss, torch.float32, w) if s is None else s
    _need(q, torch.uint8, qs, "q")
    _need(s, torch.float32, ss, "s")
    _check(fn, getattr(load_library(), fn)(_ptr(w), N, K, int(bool(transpose_out)), _ptr(q), _ptr(s), _stream(w)))
    return q, s


def fp8_quant_act_1x128(x, transpose_out=False, q=None, s=None):
    """1x128 activation quantization of x f32 [M][K].
    transpose_out=False -> (q u8 [M][K], s f32 [K/128][M]);
    transpose_out=True  -> (q u8 [K][M], s f32 [M/128][K]) (tiles along M)."""
    return _quant_act("fp8_quant_act_1x128", x, torch.float32, transpose_out, q, s)


def fp8_quant_act_1x128_bf16(x, transpose_out=False, q=None, s=None):
    """fp8_quant_act_1x128 for x bf16 [M][K] (quantizes the exactly widened values)."""
    return _quant_act("fp8_quant_act_1x128_bf16", x, torch.bfloat16, transpose_out, q, s)


def fp8_quant_weight_128x128(w, transpose_out=False, q=None, s=None):
    """128x128 weight quantization of w f32 [N][K] -> (q u8 [N][K], s f32 [N/128][K/128]),
    or the transposed codes and scales when transpose_out=True."""
    return _quant_weight("fp8_quant_weight_128x128", w, torch.float32, transpose_out, q, s)


def fp8_quant_weight_128x128_bf16(w, transpose_out=False, q=None, s=None):
    """fp8_quant_weight_128x128 for w bf16 [N][K] (quantizes the exactly widened values)."""
    return _quant_weight("fp8_quant_weight_128x128_bf16", w, torch.bfloat16, transpose_out, q, s)


def fp8_quant_fprop_operands(x, w, qa=None, sa=None, qb=None, sb=None):
    """Both Fprop operands in one launch: x f32 or bf16 [M][K], w f32 or bf16
    [N][K] -> (qa u8 [M][K], sa f32 [K/128][M], qb u8 [N][K], sb f32
    [N/128][K/128]), exactly fp8_quant_act_1x128(x) and
    fp8_quant_weight_128x128(w) (or their bf16 forms)."""
    M, K = x.shape
    N = w.shape[0]
    if x.dtype not in (torch.float32, torch.bfloat16) or w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("x and w must be float32 or bfloat16")
    _need(x, x.dtype, (M, K), "x")
    _need(w, w.dtype, (N, K), "w")
    qa = _empty((M, K), torch.uint8, x) if qa is None else qa
    sa = _empty((_nb(K), M), torch.float32, x) if sa is None else sa
    qb = _empty((N, K), torch.uint8, w) if qb is None else qb
    sb = _empty((_nb(N), _nb(K)), torch.float32, w) if sb is None else sb
    _need(qa, torch.uint8, (M, K), "qa")
    _need(sa, torch.float32, (_nb(K), M), "sa")
    _need(qb, torch.uint8, (N, K), "qb")
    _need(sb, torch.float32, (_nb(N), _nb(K)), "sb")
    _check("fp8_quant_fprop_operands", load_library().fp8_quant_fprop_operands(
        _ptr(x), int(x.dtype == torch.bfloat16), M, _ptr(w), int(w.dtype == torch.bfloat16), N, K,
        _ptr(qa), _ptr(sa), _ptr(qb), _ptr(sb), _stream(x)))
    return qa, sa, qb, sb


def fp8_requant_act_tokenwise(q, s, qt=None, st=None):
    """Rowwise FP8 cache (q u8 [M][K], s f32 [K/128][M]) -> the token-wise
    operand (qt u8 [K][M], st f32 [M/128][K]) of RN32(decode(q) * s)."""
    M, K = q.shape
    _need(q, torch.uint8, (M, K), "q")
    _need(s, torch.float32, (_nb(K), M), "s")
    qt = _empty((K, M), torch.uint8, q) if qt is None else qt
    st = _empty((_nb(M), K), torch.float32, q) if st is None else st
    _need(qt, torch.uint8, (K, M), "qt")
    _need(st, torch.float32, (_nb(M), K), "st")
    _check("fp8_requant_act_tokenwise",
           load_library().fp8_requant_act_tokenwise(_ptr(q), _ptr(s), M, K, _ptr(qt), _ptr(st), _stream(q)))
    return qt, st


def fp8_quant_mx_1x32(x, q=None, e=None):
    """MX quantization of x f32 [R][K]: (codes u8 [R][K], E8M0 scale bytes u8 [K/32][R])."""
    R, K = x.shape
    _need(x, torch.float32, (R, K), "x")
    q = _empty((R, K), torch.uint8, x) if q is None else q
    e = _empty((K // 32, R), torch.uint8, x) if e is None else e
    _need(q, torch.uint8, (R, K), "q")
    _need(e, torch.uint8, (K // 32, R), "e")
    _check("fp8_quant_mx_1x32", load_library().fp8_quant_mx_1x32(_ptr(x), R, K, _ptr(q), _ptr(e), _stream(x)))
    return q, e


def fp8_quant_mx_1x32_transposed(x, q=None, e=None):
    """MX quantization of x f32 [M][K] in blocks of 32 rows, transposed:
    (codes u8 [K][M], E8M0 scale bytes u8 [M/32][K]) = fp8_quant_mx_1x32(x^T)."""
    M, K = x.shape
    _need(x, torch.float32, (M, K), "x")
    q = _empty((K, M), torch.uint8, x) if q is None else q
    e = _empty((M // 32, K), torch.uint8, x) if e is None else e
    _need(q, torch.uint8, (K, M), "q")
    _need(e, torch.uint8, (M // 32, K), "e")
    _check("fp8_quant_mx_1x32_transposed", load_library().fp8_quant_mx_1x32_transposed(
        _ptr(x), M, K, _ptr(q), _ptr(e), _stream(x)))
    return q, e


def fp8_gemm_mx(a, ea, b, eb, out_dtype=torch.bfloat16, out=None):
    """C = A . B^T of MX operands: a u8 [M][K] / ea u8 [K/32][M], b u8 [N][K] / eb u8 [K/32][N]."""
    M, K = a.shape
    N = b.shape[0]
    _need(a, torch.uint8, (M, K), "a")
    _need(ea, torch.uint8, (K // 32, M), "ea")
    _need(b, torch.uint8, (N, K), "b")
    _need(eb, torch.uint8, (K // 32, N), "eb")
    out = _empty((M, N), out_dtype, a) if out is None else out
    _need(out, out_dtype, (M, N), "out")
    _check("fp8_gemm_mx", load_library().fp8_gemm_mx(_ptr(a), _ptr(ea), _ptr(b), _ptr(eb), _ptr(out),
                                                      _out_dtype(out_dtype), M, N, K, _stream(a)))
    return out


def fp8_grouped_gemm_contiguous_mx(a, ea, b, eb, group_offsets, out_dtype=torch.bfloat16, out=None):
    """fp8_grouped_gemm_contiguous on MX operands: a u8 [M_total][K] / ea u8
    [K/32][M_total], b u8 [G][N][K] / eb u8 [G][K/32][N]; off device int32 [G+1]."""
    M_total, K = a.shape
    G, N, _ = b.shape
    _need(a, torch.uint8, (M_total, K), "a")
    _need(ea, torch.uint8, (K // 32, M_total), "ea")
    _need(b, torch.uint8, (G, N, K), "b")
    _need(eb, torch.uint8, (G, K // 32, N), "eb")
    _need(group_offsets, torch.int32, (G + 1,), "group_offsets")
    out = _empty((M_total, N), out_dtype, a) if out is None else out
    _need(out, out_dtype, (M_total, N), "out")
    _check("fp8_grouped_gemm_contiguous_mx", load_library().fp8_grouped_gemm_contiguous_mx(
        _ptr(a), _ptr(ea), _ptr(b), _ptr(eb), _ptr(group_offsets), G, M_total, N, K, _ptr(out),
        _out_dtype(out_dtype), _stream(a)))
    return out


def fp8_grouped_gemm_masked_mx(a, ea, b, eb, masked_m, out_dtype=torch.bfloat16, out=None):
    """fp8_grouped_gemm_masked on MX operands: a u8 [G][M_max][K] / ea u8
    [G][K/32][M_max], b u8 [G][N][K] / eb u8 [G][K/32][N]; rows >= masked_m[g]
    of out are not written."""
    G, M_max, K = a.shape
    N = b.shape[1]
    _need(a, torch.uint8, (G, M_max, K), "a")
    _need(ea, torch.uint8, (G, K // 32, M_max), "ea")
    _need(b, torch.uint8, (G, N, K), "b")
    _need(eb, torch.uint8, (G, K // 32, N), "eb")
    _need(masked_m, torch.int32, (G,), "masked_m")
    out = _empty((G, M_max, N), out_dtype, a) if out is None else out
    _need(out, out_dtype, (G, M_max, N), "out")
    _check("fp8_grouped_gemm_masked_mx", load_library().fp8_grouped_gemm_masked_mx(
        _ptr(a), _ptr(ea), _ptr(b), _ptr(eb), _ptr(masked_m), G, M_max, N, K, _ptr(out),
        _out_dtype(out_dtype), _stream(a)))
    return out


def _out_dtype(out_dtype):
    return {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32}[out_dtype]


def _gemm_dense(fn, a, sa, b, sb, bscale_kind, out_dtype, out):
    M, K = a.shape
    N = b.shape[0]
    _need(a, torch.uint8, (M, K), "a")
    _need(sa, torch.float32, (_nb(K), M), "sa")
    _need(b, torch.uint8, (N, K), "b")
    _need(sb, torch.float32, (_nb(N), _nb(K)) if bscale_kind == BSCALE_128x128 else (_nb(K), N), "sb")
    out = _empty((M, N), out_dtype, a) if out is None else out
    _need(out, out_dtype, (M, N), "out")
    _check(fn, getattr(load_library(), fn)(
        _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), int(bscale_kind), _ptr(out), _out_dtype(out_dtype),
        M, N, K, _stream(a)))
    return out


def fp8_gemm_blockscaled(a, sa, b, sb, bscale_kind=BSCALE_128x128, out_dtype=torch.bfloat16, out=None):
    """C[M][N] = A[M][K] . B[N][K]^T with 1x128 A scales and 128x128 (or 1x128) B scales."""
    return _gemm_dense("fp8_gemm_blockscaled", a, sa, b, sb, bscale_kind, out_dtype, out)


def fp8_gemm_blockscaled_fp8mfma(a, sa, b, sb, bscale_kind=BSCALE_128x128, out_dtype=torch.bfloat16, out=None):
    """fp8_gemm_blockscaled on the FP8 matrix cores: same operands and layouts,
    accuracy contract 2^-9 * sum|a b| instead of 2^-14 (see fp8fg.h)."""
    return _gemm_dense("fp8_gemm_blockscaled_fp8mfma", a, sa, b, sb, bscale_kind, out_dtype, out)


def fp8_gemm_blockscaled_fp8out(a, sa, b, sb, q=None, s=None):
    """C = A . B^T (128x128 B scales) quantized 1x128 along N in the epilogue:
    returns (q u8 [M][N], s f32 [N/128][M]) -- the next layer's A operand."""
    M, K = a.shape
    N = b.shape[0]
    _need(a, torch.uint8, (M, K), "a")
    _need(sa, torch.float32, (_nb(K), M), "sa")
    _need(b, torch.uint8, (N, K), "b")
    _need(sb, torch.float32, (N // 128, _nb(K)), "sb")
    q = _empty((M, N), torch.uint8, a) if q is None else q
    s = _empty((N // 128, M), torch.float32, a) if s is None else s
    _need(q, torch.uint8, (M, N), "q")
    _need(s, torch.float32, (N // 128, M), "s")
    _check("fp8_gemm_blockscaled_fp8out", load_library().fp8_gemm_blockscaled_fp8out(
        _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(q), _ptr(s), M, N, K, _stream(a)))
    return q, s


def fp8_grouped_gemm_contiguous_fp8out(a, sa, b, sb, group_offsets, q=None, s=None):
    """Contiguous MoE layout with the output quantized 1x128 along N in the
    epilogue: returns (q u8 [M_total][N], s f32 [N/128][M_total]); rows in no
    expert's range are left as they were (zeros when q, s are allocated here)."""
    M_total, K = a.shape
    G, N, _ = b.shape
    _need(a, torch.uint8, (M_total, K), "a")
    _need(sa, torch.float32, (_nb(K), M_total), "sa")
    _need(b, torch.uint8, (G, N, K), "b")
    _need(sb, torch.float32, (G, _nb(N), _nb(K)), "sb")
    _need(group_offsets, torch.int32, (G + 1,), "group_offsets")
    q = torch.zeros((M_total, N), dtype=torch.uint8, device=a.device) if q is None else q
    s = torch.zeros((N // 128, M_total), dtype=torch.float32, device=a.device) if s is None else s
    _need(q, torch.uint8, (M_total, N), "q")
    _need(s, torch.float32, (N // 128, M_total), "s")
    _check("fp8_grouped_gemm_contiguous_fp8out", load_library().fp8_grouped_gemm_contiguous_fp8out(
        _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(group_offsets), G, M_total, N, K, _ptr(q), _ptr(s), _stream(a)))
    return q, s


def fp8_grouped_gemm_contiguous(a, sa, b, sb, group_offsets, out_dtype=torch.bfloat16, out=None):
    """Contiguous MoE layout: expert g owns rows [off[g], off[g+1]) of a; off is device int32 [G+1]."""
    M_total, K = a.shape
    G, N, _ = b.shape
    _need(a, torch.uint8, (M_total, K), "a")
    _need(sa, torch.float32, (_nb(K), M_total), "sa")
    _need(b, torch.uint8, (G, N, K), "b")
    _need(sb, torch.float32, (G, _nb(N), _nb(K)), "sb")
    _need(group_offsets, torch.int32, (G + 1,), "group_offsets")
    out = _empty((M_total, N), out_dtype, a) if out is None else out
    _need(out, out_dtype, (M_total, N), "out")
    _check("fp8_grouped_gemm_contiguous", load_library().fp8_grouped_gemm_contiguous(
        _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(group_offsets), G, M_total, N, K, _ptr(out),
        _out_dtype(out_dtype), _stream(a)))
    return out


def fp8_grouped_gemm_masked(a, sa, b, sb, masked_m, out_dtype=torch.bfloat16, out=None):
    """Masked MoE layout: a u8 [G][M_max][K]; rows >= masked_m[g] of out are not written."""
    G, M_max, K = a.shape
    N = b.shape[1]
    _need(a, torch.uint8, (G, M_max, K), "a")
    _need(sa, torch.float32, (G, _nb(K), M_max), "sa")
    _need(b, torch.uint8, (G, N, K), "b")
    _need(sb, torch.float32, (G, _nb(N), _nb(K)), "sb")
    _need(masked_m, torch.int32, (G,), "masked_m")
    out = _empty((G, M_max, N), out_dtype, a) if out is None else out
    _need(out, out_dtype, (G, M_max, N), "out")
    _check("fp8_grouped_gemm_masked", load_library().fp8_grouped_gemm_masked(
        _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(masked_m), G, M_max, N, K, _ptr(out),
        _out_dtype(out_dtype), _stream(a)))
    return out


def fp8_grouped_gemm_masked_tiled_mx(a, ea, b_tiled, eb, masked_m, out_dtype=torch.bfloat16, out=None):
    """fp8_grouped_gemm_masked_mx with the experts' codes in the decode-tiled
    layout (b_tiled u8 [G][N/256][K/64][16384], from fp8_tile_weights_decode)."""
    G, M_max, K = a.shape
    N = b_tiled.shape[1] * 256
    _need(a, torch.uint8, (G, M_max, K), "a")
    _need(ea, torch.uint8, (G, K // 32, M_max), "ea")
    _need(b_tiled, torch.uint8, (G, N // 256, K // 64, 16384), "b_tiled")
    _need(eb, torch.uint8, (G, K // 32, N), "eb")
    _need(masked_m, torch.int32, (G,), "masked_m")
    out = _empty((G, M_max, N), out_dtype, a) if out is None else out
    _need(out, out_dtype, (G, M_max, N), "out")
    _check("fp8_grouped_gemm_masked_tiled_mx", load_library().fp8_grouped_gemm_masked_tiled_mx(
        _ptr(a), _ptr(ea), _ptr(b_tiled), _ptr(eb), _ptr(masked_m), G, M_max, N, K, _ptr(out),
        _out_dtype(out_dtype), _stream(a)))
    return out


def fp8_grouped_gemm_masked_tiled_fp8out(a, sa, b_tiled, sb, masked_m, q=None, s=None):
    """fp8_grouped_gemm_masked_tiled with the output quantized 1x128 along N in
    the epilogue: returns (q u8 [G][M_max][N], s f32 [G][N/128][M_max]); rows
    past masked_m[g] are left as they were (zeros when q, s are allocated here)."""
    G, M_max, K = a.shape
    N = b_tiled.shape[1] * 256
    _need(a, torch.uint8, (G, M_max, K), "a")
    _need(sa, torch.float32, (G, _nb(K), M_max), "sa")
    _need(b_tiled, torch.uint8, (G, N // 256, K // 64, 16384), "b_tiled")
    _need(sb, torch.float32, (G, _nb(N), _nb(K)), "sb")
    _need(masked_m, torch.int32, (G,), "masked_m")
    q = torch.zeros((G, M_max, N), dtype=torch.uint8, device=a.device) if q is None else q
    s = torch.zeros((G, N // 128, M_max), dtype=torch.float32, device=a.device) if s is None else s
    _need(q, torch.uint8, (G, M_max, N), "q")
    _need(s, torch.float32, (G, N // 128, M_max), "s")
    _check("fp8_grouped_gemm_masked_tiled_fp8out", load_library().fp8_grouped_gemm_masked_tiled_fp8out(
        _ptr(a), _ptr(sa), _ptr(b_tiled), _ptr(sb), _ptr(masked_m), G, M_max, N, K, _ptr(q), _ptr(s), _stream(a)))
    return q, s


def fp8_tile_weights_decode(q, out=None):
    """Experts' codes u8 [G][N][K] -> the decode-tiled layout, returned as u8
    [G][N/256][K/64][16384]: one 16 KB block per (expert, 256-row n-tile,
    64-byte K piece), in the order fp8fg.h defines."""
    G, N, K = q.shape
    _need(q, torch.uint8, (G, N, K), "q")
    shape = (G, N // 256, K // 64, 16384)
    out = _empty(shape, torch.uint8, q) if out is None else out
    _need(out, torch.uint8, shape, "out")
    _check("fp8_tile_weights_decode", load_library().fp8_tile_weights_decode(
        _ptr(q), G, N, K, _ptr(out), _stream(q)))
    return out


def fp8_grouped_gemm_masked_tiled(a, sa, b_tiled, sb, masked_m, out_dtype=torch.bfloat16, out=None):
    """fp8_grouped_gemm_masked with the experts' codes in the decode-tiled
    layout (b_tiled u8 [G][N/256][K/64][16384], from fp8_tile_weights_decode)."""
    G, M_max, K = a.shape
    N = b_tiled.shape[1] * 256
    _need(a, torch.uint8, (G, M_max, K), "a")
    _need(sa, torch.float32, (G, _nb(K), M_max), "sa")
    _need(b_tiled, torch.uint8, (G, N // 256, K // 64, 16384), "b_tiled")
    _need(sb, torch.float32, (G, _nb(N), _nb(K)), "sb")
    _need(masked_m, torch.int32, (G,), "masked_m")
    out = _empty((G, M_max, N), out_dtype, a) if out is None else out
    _need(out, out_dtype, (G, M_max, N), "out")
    _check("fp8_grouped_gemm_masked_tiled", load_library().fp8_grouped_gemm_masked_tiled(
        _ptr(a), _ptr(sa), _ptr(b_tiled), _ptr(sb), _ptr(masked_m), G, M_max, N, K, _ptr(out),
        _out_dtype(out_dtype), _stream(a)))
    return out


# The operators around the grouped GEMMs of a mixture-of-experts layer.

def _out(t, shape, dtype, like, name):
    """An output: the caller's tensor once checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _need(t, dtype, shape, name)
    return t


def _f32_or_bf16(t, name):
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return int(t.dtype == torch.bfloat16)


def _logits(x):
    if not x.is_cuda:
        raise ValueError("logits must be a GPU tensor")
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < x.shape[1]):
        raise ValueError("logits must have shape [T][E] with contiguous rows")
    return _f32_or_bf16(x, "logits"), (x.stride(0) if x.shape[0] > 1 else x.shape[1])


def moe_route(logits, topk, bias=None, n_groups=1, topk_groups=1, group_top=1, score=SCORE_SIGMOID, renormalize=True,
              scale=1.0, idx=None, w=None):
    """Experts of each token: logits f32 or bf16 [T][E] (rows may be strided) ->
    (idx int32 [T][topk], w f32 [T][topk]).  score SCORE_SOFTMAX or SCORE_SIGMOID;
    bias f32 [E] is added for the choice only; of n_groups groups the
    topk_groups best (by the sum of their group_top largest scores) stay in.
    Logits of -inf are never chosen; missing choices are -1 with weight 0."""
    bf16, ld = _logits(logits)
    T, E = logits.shape
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    idx = _out(idx, (T, topk), torch.int32, logits, "idx")
    w = _out(w, (T, topk), torch.float32, logits, "w")
    _check("moe_route", load_library().moe_route(
        _ptr(logits), bf16, ld, _ptr(bias), T, E, topk, n_groups, topk_groups, group_top, score, int(bool(renormalize)),
        scale, _ptr(idx), _ptr(w), _stream(logits)))
    return idx, w


def moe_route_backward(logits, idx, dw, score=SCORE_SIGMOID, renormalize=True, scale=1.0, out=None):
    """The gradient of moe_route's logits from dw f32 [T][topk], for the choice
    idx: [T][E] in the logits' type."""
    bf16, ld = _logits(logits)
    T, E = logits.shape
    topk = idx.shape[1]
    _need(idx, torch.int32, (T, topk), "idx")
    _need(dw, torch.float32, (T, topk), "dw")
    out = _out(out, (T, E), logits.dtype, logits, "out")
    _check("moe_route_backward", load_library().moe_route_backward(
        _ptr(logits), bf16, ld, _ptr(idx), _ptr(dw), T, E, topk, score, int(bool(renormalize)), scale, _ptr(out),
        _stream(logits)))
    return out


def moe_rows_bound(T, topk, n_experts):
    """Rows of the contiguous layout that hold any choice of topk experts for T
    tokens among n_experts local ones (every expert's rows padded to 128)."""
    n = T * topk if n_experts else 0
    return (n + 127 * min(n_experts, n)) // 128 * 128


def _row_of(idx, n_experts):
    """The entries' rows, for the call to write; all -1 where no expert is local, for which it writes nothing."""
    return torch.empty_like(idx) if n_experts else torch.full_like(idx, -1)


def fp8_moe_dispatch_contiguous(x, idx, n_experts, first=0, M_total=None, q=None, s=None):
    """Tokens x f32 or bf16 [T][H] into the rows of their experts (idx int32
    [T][topk]; local experts first .. first + n_experts - 1), quantized 1x128:
    (q u8 [M_total][H], s f32 [H/128][M_total], row_of int32 [T][topk],
    group_offsets int32 [G+1], counts int32 [G]).  M_total defaults to
    moe_rows_bound; rows from group_offsets[G] on are not written."""
    T, H = x.shape
    topk = idx.shape[1]
    _need(x, x.dtype, (T, H), "x")
    _need(idx, torch.int32, (T, topk), "idx")
    if M_total is None:
        M_total = moe_rows_bound(T, topk, n_experts) if q is None else q.shape[0]
    q = _out(q, (M_total, H), torch.uint8, x, "q")
    s = _out(s, (_nb(H), M_total), torch.float32, x, "s")
    row_of = _row_of(idx, n_experts)
    offsets = _empty((n_experts + 1,), torch.int32, x) if n_experts else torch.zeros(1, dtype=torch.int32, device=x.device)
    counts = _empty((n_experts,), torch.int32, x)
    _check("fp8_moe_dispatch_contiguous", load_library().fp8_moe_dispatch_contiguous(
        _ptr(x), _f32_or_bf16(x, "x"), T, H, _ptr(idx), topk, first, n_experts, M_total, _ptr(q), _ptr(s), _ptr(row_of),
        _ptr(offsets), _ptr(counts), _stream(x)))
    return q, s, row_of, offsets, counts


def fp8_moe_dispatch_masked(x, idx, n_experts, M_max, first=0, q=None, s=None):
    """fp8_moe_dispatch_contiguous in the masked layout (decode): (q u8
    [G][M_max][H], s f32 [G][H/128][M_max], row_of int32 [T][topk] (g * M_max +
    row), masked_m int32 [G]); rows past masked_m[g] are not written."""
    T, H = x.shape
    topk = idx.shape[1]
    _need(x, x.dtype, (T, H), "x")
    _need(idx, torch.int32, (T, topk), "idx")
    q = _out(q, (n_experts, M_max, H), torch.uint8, x, "q")
    s = _out(s, (n_experts, _nb(H), M_max), torch.float32, x, "s")
    row_of = _row_of(idx, n_experts)
    masked_m = _empty((n_experts,), torch.int32, x)
    _check("fp8_moe_dispatch_masked", load_library().fp8_moe_dispatch_masked(
        _ptr(x), _f32_or_bf16(x, "x"), T, H, _ptr(idx), topk, first, n_experts, M_max, _ptr(q), _ptr(s), _ptr(row_of),
        _ptr(masked_m), _stream(x)))
    return q, s, row_of, masked_m


def moe_combine(y, row_of, w=None, out_dtype=torch.bfloat16, out=None):
    """out[t] = sum_j w[t][j] * y[row_of[t][j]] over the entries that have a row:
    y f32 or bf16 [R][H] (or the masked [G][M_max][H]), row_of int32 [T][topk],
    w f32 [T][topk] or None (weights of 1) -> [T][H]."""
    T, topk = row_of.shape
    H = y.shape[-1]
    R = y.numel() // H if H else 0
    _need(y, y.dtype, y.shape, "y")
    _need(row_of, torch.int32, (T, topk), "row_of")
    if w is not None:
        _need(w, torch.float32, (T, topk), "w")
    out = _out(out, (T, H), out_dtype, y, "out")
    _check("moe_combine", load_library().moe_combine(
        _ptr(y), _f32_or_bf16(y, "y"), R, H, _ptr(row_of), _ptr(w), T, topk, _ptr(out), _out_dtype(out_dtype), _stream(y)))
    return out


def fp8_moe_combine_backward(dout, y, row_of, w, group_offsets, counts, q=None, s=None, dw=None):
    """The backward pass of moe_combine in the contiguous layout: dout [T][H],
    y [R][H] -> (q u8 [R][H], s f32 [H/128][R]: the rows' gradient
    w[t][j] * dout[t] as a grouped GEMM's A operand; dw f32 [T][topk])."""
    T, H = dout.shape
    R = y.shape[0]
    topk = row_of.shape[1]
    G = counts.shape[0]
    _need(dout, dout.dtype, (T, H), "dout")
    _need(y, y.dtype, (R, H), "y")
    _need(row_of, torch.int32, (T, topk), "row_of")
    _need(w, torch.float32, (T, topk), "w")
    _need(group_offsets, torch.int32, (G + 1,), "group_offsets")
    _need(counts, torch.int32, (G,), "counts")
    q = _out(q, (R, H), torch.uint8, y, "q")
    s = _out(s, (_nb(H), R), torch.float32, y, "s")
    dw = _out(dw, (T, topk), torch.float32, y, "dw")
    _check("fp8_moe_combine_backward", load_library().fp8_moe_combine_backward(
        _ptr(dout), _f32_or_bf16(dout, "dout"), T, H, _ptr(y), _f32_or_bf16(y, "y"), R, _ptr(row_of), _ptr(w), topk,
        _ptr(group_offsets), _ptr(counts), G, _ptr(q), _ptr(s), _ptr(dw), _stream(y)))
    return q, s, dw


def _need_rows(rows, G):
    if rows is not None:
        _need(rows, torch.int32, (G,), "rows")


def fp8_swiglu(gu, rows=None, checkpoint=False, q=None, s=None, qc=None, sc=None):
    """The gate h = g * sigmoid(g) * u of gu f32 or bf16 [M][2 I] (or the masked
    [G][M_max][2 I]; g the first I columns, u the others), quantized 1x128:
    (q u8 [M][I], s f32 [I/128][M]), and with checkpoint=True also the 1x128
    quantization of gu (qc u8 [M][2 I], sc f32 [2 I/128][M]) for the backward
    pass; a masked gu adds a leading [G] to each.  rows: int32 [1] (group_offsets[G:])
    or int32 [G] (masked_m): the rows in use; the others are neither read nor written."""
    lead, I = tuple(gu.shape[:-1]), gu.shape[-1] // 2
    if gu.dim() not in (2, 3) or gu.shape[-1] % 2:
        raise ValueError("gu must have shape [M][2 I] or [G][M_max][2 I]")
    G, M = (1, lead[0]) if len(lead) == 1 else lead
    _need(gu, gu.dtype, gu.shape, "gu")
    _need_rows(rows, G)
    ss = lead[:-1] + (_nb(I), M)
    q = _out(q, lead + (I,), torch.uint8, gu, "q")
    s = _out(s, ss, torch.float32, gu, "s")
    if checkpoint:
        cs = lead[:-1] + (2 * _nb(I), M)
        qc = _out(qc, gu.shape, torch.uint8, gu, "qc")
        sc = _out(sc, cs, torch.float32, gu, "sc")
    elif qc is not None or sc is not None:
        raise ValueError("qc and sc are written with checkpoint=True only")
    _check("fp8_swiglu", load_library().fp8_swiglu(
        _ptr(gu), _f32_or_bf16(gu, "gu"), G, M, I, _ptr(rows), _ptr(q), _ptr(s), _ptr(qc), _ptr(sc), _stream(gu)))
    return (q, s, qc, sc) if checkpoint else (q, s)


def fp8_swiglu_backward(qc, sc, dh, rows=None, out=None):
    """The backward pass of fp8_swiglu from its checkpoint (qc u8 [M][2 I], sc f32
    [2 I/128][M]) and dh f32 or bf16 [M][I]: (q u8 [M][2 I], s f32 [2 I/128][M],
    qt u8 [2 I][M], st f32 [M/128][2 I], qh u8 [I][M], sh f32 [M/128][I]) -- the
    gradient of gu along its channels and along its rows, and h along its rows.
    out: the six buffers to write."""
    M, I = dh.shape
    _need(qc, torch.uint8, (M, 2 * I), "qc")
    _need(sc, torch.float32, (2 * _nb(I), M), "sc")
    _need(dh, dh.dtype, (M, I), "dh")
    _need_rows(rows, 1)
    shapes = ((torch.uint8, (M, 2 * I), "q"), (torch.float32, (2 * _nb(I), M), "s"), (torch.uint8, (2 * I, M), "qt"),
              (torch.float32, (_nb(M), 2 * I), "st"), (torch.uint8, (I, M), "qh"), (torch.float32, (_nb(M), I), "sh"))
    out = (None,) * 6 if out is None else tuple(out)
    if len(out) != 6:
        raise ValueError("out must hold six tensors")
    out = tuple(_out(t, shape, dtype, dh, name) for t, (dtype, shape, name) in zip(out, shapes))
    _check("fp8_swiglu_backward", load_library().fp8_swiglu_backward(
        _ptr(qc), _ptr(sc), _ptr(dh), _f32_or_bf16(dh, "dh"), M, I, _ptr(rows), *(_ptr(t) for t in out), _stream(dh)))
    return out


def fp8_grouped_gemm_wgrad(a, sa, b, sb, group_offsets, out=None, accumulate=False):
    """The experts' weight gradients out[g] = sum over expert g's rows r of
    a[:, r] b[:, r]^T (FP32 [G][M][N]): a u8 [M][R] / sa f32 [R/128][M], b u8
    [N][R] / sb f32 [R/128][N] (1x128 along the rows), group_offsets device int32
    [G+1].  accumulate=True adds to out."""
    M, R = a.shape
    N = b.shape[0]
    G = group_offsets.shape[0] - 1
    _need(a, torch.uint8, (M, R), "a")
    _need(sa, torch.float32, (_nb(R), M), "sa")
    _need(b, torch.uint8, (N, R), "b")
    _need(sb, torch.float32, (_nb(R), N), "sb")
    _need(group_offsets, torch.int32, (G + 1,), "group_offsets")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    out = _out(out, (G, M, N), torch.float32, a, "out")
    _check("fp8_grouped_gemm_wgrad", load_library().fp8_grouped_gemm_wgrad(
        _ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(group_offsets), G, M, N, R, _ptr(out), int(bool(accumulate)),
        _stream(a)))
    return out


# Attention over a key/value cache held in 8 bits, in pages.

_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())


def _run(fn, index, like, *args):
    """The call fn on the device `index` of like and its current stream."""
    call = getattr(load_library(), fn)
    if index == _current_device():
        status = call(*args, _stream(like))
    else:
        with torch.cuda.device(index):
            status = call(*args, _stream(like))
    if status != 0:
        raise Fp8fgError(fn, status)


def _device_of(t, name):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return index


def _need_at(index, t, dtype, shape, name):
    """_need, and that t lies on the device `index`."""
    if t.get_device() == index and t.dtype == dtype and t.shape == shape and t.is_contiguous():
        return
    _need(t, dtype, shape, name)
    raise ValueError(f"{name} must be on device {index}, got {t.device}")


def _out_at(index, t, shape, dtype, like, name):
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _need_at(index, t, dtype, shape, name)
    return t


def kv_cache(n_pages, heads, page, dim, device="cuda"):
    """An empty cache of one layer: (k_cache u8 [n_pages][heads][page][dim], k_scale f32
    [n_pages][heads], v_cache u8 [n_pages][heads][dim][page], v_scale f32 [n_pages][heads])."""
    def zeros(*shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype, device=device)

    return (zeros(n_pages, heads, page, dim), zeros(n_pages, heads, dtype=torch.float32),
            zeros(n_pages, heads, dim, page), zeros(n_pages, heads, dtype=torch.float32))


def kv_assign_pages(have, add, table, free_pages, n_free, page, T, out=None):
    """A step's pages, slots and positions.  have, add int32 [B]: tokens that the
    cache holds of each request, and new ones; table int32 [B][width], to which the new pages are
    added; free_pages int32 [F], of which the first n_free (int32 [1]) are free; T rows
    -> (lens int32 [B], cu int32 [B+1], positions int32 [T], slots int32 [T], left int32
    [2]: pages left free, pages missing).  out: the five buffers to write, none of them an input."""
    B, width = table.shape
    F = free_pages.shape[0]
    at = _device_of(table, "table")
    _need_at(at, table, torch.int32, (B, width), "table")
    _need_at(at, have, torch.int32, (B,), "have")
    _need_at(at, add, torch.int32, (B,), "add")
    _need_at(at, free_pages, torch.int32, (F,), "free_pages")
    _need_at(at, n_free, torch.int32, (1,), "n_free")
    lens, cu, positions, slots, left = (None,) * 5 if out is None else out
    lens = _out_at(at, lens, (B,), torch.int32, table, "lens")
    cu = _out_at(at, cu, (B + 1,), torch.int32, table, "cu")
    positions = _out_at(at, positions, (T,), torch.int32, table, "positions")
    slots = _out_at(at, slots, (T,), torch.int32, table, "slots")
    left = _out_at(at, left, (2,), torch.int32, table, "left")
    _run("kv_assign_pages", at, table,
         _ptr(have), _ptr(add), B, _ptr(free_pages), _ptr(n_free), F, page, _ptr(table), width, T, _ptr(lens), _ptr(cu),
         _ptr(positions), _ptr(slots), _ptr(left))
    return lens, cu, positions, slots, left


def kv_release_pages(done, lens, table, free_pages, n_free, page, out=None):
    """The pages of the requests that are done (int32 [B], 0 or not) back to the free
    list, which is extended in place -> (lens int32 [B], 0 where done; left int32 [1],
    the pages that are free now).  out: the two buffers to write, neither of them an input."""
    B, width = table.shape
    F = free_pages.shape[0]
    at = _device_of(table, "table")
    _need_at(at, table, torch.int32, (B, width), "table")
    _need_at(at, done, torch.int32, (B,), "done")
    _need_at(at, lens, torch.int32, (B,), "lens")
    _need_at(at, free_pages, torch.int32, (F,), "free_pages")
    _need_at(at, n_free, torch.int32, (1,), "n_free")
    lens_out, left = (None, None) if out is None else out
    lens_out = _out_at(at, lens_out, (B,), torch.int32, table, "lens")
    left = _out_at(at, left, (1,), torch.int32, table, "left")
    _run("kv_release_pages", at, table,
         _ptr(done), _ptr(lens), _ptr(table), B, width, page, _ptr(free_pages), F, _ptr(n_free), _ptr(lens_out), _ptr(left))
    return lens_out, left


def _heads(index, t, dtype, shape, name):
    """The distance of the rows of t [T][H][D], whose heads are contiguous."""
    T, H, D = shape
    if t.get_device() != index:
        raise ValueError(f"{name} must be on device {index}, got {t.device}" if t.is_cuda else f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    ld, step, one = t.stride()
    if (D > 1 and one != 1) or (H > 1 and step != D) or (T > 1 and ld < H * D):
        raise ValueError(f"{name} must have contiguous heads")
    return ld if T > 1 else H * D


def rope_frequencies(rot, base=10000.0, factor=1.0, original=4096, fast=32.0, slow=1.0, device="cuda"):
    """Frequencies f32 [rot/2] for rope, base^(-2 i / rot), and the scale that goes
    with them.  factor > 1 stretches a context of `original` tokens: frequencies that turn
    fewer than `slow` times in it are divided by factor, those that turn more than `fast`
    times are kept, with a ramp between that is linear in the turns (models whose ramp is linear in the channel's
    number between two rounded ones bring frequencies of their own), and the scale is 0.1 ln(factor) + 1."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor > 1.0:
        turns = f * (original / 6.283185307179586)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    scale = 0.1 * float(torch.log(torch.tensor(factor, dtype=torch.float64))) + 1.0 if factor > 1.0 else 1.0
    return f.float().to(device), scale


def rope(q, k, positions, freqs, interleaved=False, scale=1.0, inverse=False, q_out=None, k_out=None):
    """Rotary positions: q [T][Hq][D] and k [T][Hkv][D] (or None), f32 or bf16, rows may
    be strided, turned by positions int32 [T] * freqs f32 [rot/2] and times scale ->
    (q_out, k_out).  Pairs (i, i + rot/2), or (2 i, 2 i + 1) when interleaved; channels from
    rot on are copied; rows with a negative position are not written.  inverse=True: the
    gradient of q and k from that of the outputs.  q_out=q, k_out=k turns in place."""
    T, Hq, D = q.shape
    at = _device_of(q, "q")
    ldq = _heads(at, q, q.dtype, (T, Hq, D), "q")
    bf16 = _f32_or_bf16(q, "q")
    _need_at(at, positions, torch.int32, (T,), "positions")
    _need_at(at, freqs, torch.float32, (freqs.shape[0],), "freqs")
    ldqo = Hq * D
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        ldqo = _heads(at, q_out, q.dtype, (T, Hq, D), "q_out")
    Hkv = ldk = ldko = 0
    if k is not None:
        Hkv = k.shape[1]
        ldk = _heads(at, k, q.dtype, (T, Hkv, D), "k")
        ldko = Hkv * D
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        else:
            ldko = _heads(at, k_out, q.dtype, (T, Hkv, D), "k_out")
    elif k_out is not None:
        raise ValueError("k_out needs k")
    _run("rope", at, q,
         _ptr(q), ldq, _ptr(q_out), ldqo, Hq, _ptr(k), ldk, _ptr(k_out), ldko, Hkv, bf16, _ptr(positions), _ptr(freqs), T, D,
         2 * freqs.shape[0], int(bool(interleaved)), scale, int(bool(inverse)))
    return q_out, k_out


def _need_cache(k_cache, k_scale, v_cache, v_scale):
    """The cache's device and sizes, once its tensors fit together."""
    n, H, page, D = k_cache.shape
    at = _device_of(k_cache, "k_cache")
    _need_at(at, k_cache, torch.uint8, (n, H, page, D), "k_cache")
    _need_at(at, v_cache, torch.uint8, (n, H, D, page), "v_cache")
    _need_at(at, k_scale, torch.float32, (n, H), "k_scale")
    _need_at(at, v_scale, torch.float32, (n, H), "v_scale")
    return at, n, H, page, D


def fp8_kv_append(k, v, slots, k_cache, k_scale, v_cache, v_scale):
    """New keys and values k, v f32 or bf16 [T][H][D] (rows may be strided) into their
    slots int32 [T] of the cache (see kv_cache), in place: E4M3 codes under one power of
    two per page and head.  Rows with a slot outside the cache are skipped; the rows of
    a page are consecutive, with consecutive slots."""
    at, n, H, page, D = _need_cache(k_cache, k_scale, v_cache, v_scale)
    T = k.shape[0]
    ldk, ldv = _heads(at, k, k.dtype, (T, H, D), "k"), _heads(at, v, k.dtype, (T, H, D), "v")
    _need_at(at, slots, torch.int32, (T,), "slots")
    _run("fp8_kv_append", at, k,
         _ptr(k), ldk, _ptr(v), ldv, _f32_or_bf16(k, "k"), _ptr(slots), T, H, D, page, n, _ptr(k_cache), _ptr(k_scale),
         _ptr(v_cache), _ptr(v_scale))


@functools.lru_cache(maxsize=4096)
def fp8_kv_attention_workspace(T, B, Hq, Hkv, D, page, width):
    """Bytes of workspace of a call of fp8_kv_attention with these sizes."""
    got = ctypes.c_int64(0)
    _check("fp8_kv_attention_workspace", load_library().fp8_kv_attention_workspace(T, B, Hq, Hkv, D, page, width, ctypes.byref(got)))
    return got.value


def fp8_kv_attention(q, k_cache, k_scale, v_cache, v_scale, table, cu, lens, scale=None, out=None, lse=None, workspace=None):
    """Causal attention of the new tokens q bf16 [T][Hq][D] (rows may be strided) over
    the cache, which holds them already: request b's rows cu[b] .. cu[b+1] - 1 (int32
    [B+1]), its lens[b] tokens (int32 [B]) in the pages table[b] (int32 [B][width]).
    scale defaults to D^-0.5.  Returns out bf16 [T][Hq][D], or (out, lse) where lse f32 [T][Hq] is given to be
    written.  Rows from cu[B] on are not written.  workspace: a uint8 tensor of at least
    fp8_kv_attention_workspace bytes, used by one call at a time."""
    at, n, Hkv, page, D = _need_cache(k_cache, k_scale, v_cache, v_scale)
    T, Hq, _ = q.shape
    B, width = table.shape
    ldq = _heads(at, q, torch.bfloat16, (T, Hq, D), "q")
    _need_at(at, table, torch.int32, (B, width), "table")
    _need_at(at, cu, torch.int32, (B + 1,), "cu")
    _need_at(at, lens, torch.int32, (B,), "lens")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _need_at(at, out, torch.bfloat16, (T, Hq, D), "out")
    if lse is not None:
        _need_at(at, lse, torch.float32, (T, Hq), "lse")
    if workspace is None:
        need = fp8_kv_attention_workspace(T, B, Hq, Hkv, D, page, width)
        workspace = q.new_empty(need, dtype=torch.uint8) if need else None
    else:
        need = workspace.numel()
        _need_at(at, workspace, torch.uint8, (need,), "workspace")
    _run("fp8_kv_attention", at, q,
         _ptr(q), ldq, _ptr(k_cache), _ptr(k_scale), _ptr(v_cache), _ptr(v_scale), n, page, _ptr(table), width, _ptr(cu),
         _ptr(lens), B, T, Hq, Hkv, D, D ** -0.5 if scale is None else scale, _ptr(out), _ptr(lse), _ptr(workspace), need)
    return out if lse is None else (out, lse)
