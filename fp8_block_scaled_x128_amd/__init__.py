"""MI355X (gfx950) FP8 GEMM with fine-grained block scaling: Python binding of libfp8gemm.so.

Argument marshalling only -- every step of the computation runs in the HIP kernels behind the
C ABI declared in include/fp8gemm.h.  torch supplies device memory and the current stream.

    D = gemm_nt(A, sa, B, sb)                              # dense NT, bf16 out
    D = gemm_nt_specialized(A, sa, B, sb)                  # the same, kernel built at run time for N, K
    D = grouped_contiguous(A, sa, B, sb, m_indices)        # MoE, groups concatenated along M
    D = grouped_masked(A, sa, B, sb, masked_m, expected_m) # MoE, fixed per-group capacity
    D = fp8fp4_grouped_masked(A, sa, B4, sb4, masked_m, expected_m)  # the same, B in E2M1 + E8M0
    A, sa = quantize_1x128(X)                              # bf16 activations -> codes + scales
    A, sa = quantize_1x128_masked(X, masked_m)             # the same, masked layout
    H, sh = swiglu_quantize_1x128(Y)                       # silu(gate) * up -> codes + scales
    out = moe_expert_masked(A, sa, W1, s1, W2, s2, masked_m, expected_m)  # one MoE expert layer
    ids, w = route_topk(logits, k, bias, score="sigmoid", ...)   # the router's experts and weights
    dlogits = route_topk_backward(logits, ids, dw, ...)          # and their gradient
    A, sa, masked_m, rows = moe_dispatch_masked(X, ids, G, M_max)      # tokens -> masked rows, quantised
    A, sa, m_indices, rows = moe_dispatch_contiguous(X, ids, G)        # the same, contiguous layout
    out = moe_combine(Y, w, rows)                                # expert rows -> tokens, weighted
    dY, dw = moe_combine_backward(dout, Y, w, rows)              # and its gradients
    Y = w4_gemv(X, W4, scales, zeros)                            # few rows times 4-bit weights
    Y = w4_gemv_experts(X, W4, scales, ids, zeros, swiglu=True)  # the same, by the router's ids

A and B are E4M3 codes (torch.float8_e4m3fn or uint8), sa one fp32 scale per 1x128 block of a
row of A stored K-block-major (sa[kb, m], shape [K/128, M]), sb one per 128x128 block of B (page "DeepSeek開源第三彈：V3/R1訓練推理關鍵秘籍，核心代碼僅
300行", sections 深入了解DeepGEMM and 如何使用？).  There is no CPU fallback: without the built
library every call raises.
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["gemm_nt", "gemm_nt_noalloc", "gemm_nt_specialized", "specialize_nt", "specialized_code_object", "specialized_count",
           "grouped_contiguous", "grouped_masked", "quantize_1x128",
           "quantize_1x128_masked", "fp8fp4_grouped_masked", "swiglu_quantize_1x128", "swiglu_quantize_1x128_masked",
           "moe_expert_masked", "route_topk", "route_topk_backward", "moe_dispatch_masked",
           "moe_dispatch_contiguous", "moe_combine", "moe_combine_backward", "w4_gemv", "w4_gemv_experts", "init", "prepare_stream", "set_num_cus",
           "last_config", "read_device_error", "status_string", "lib", "library_path",
           "Fp8GemmError", "STATUS", "DEVERR_BAD_INDEX", "DEVERR_BAD_COUNT"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libfp8gemm.so")
_lib = None

STATUS = {0: "FP8GEMM_OK", 1: "FP8GEMM_ERR_NULL_PTR", 2: "FP8GEMM_ERR_BAD_SHAPE",
          3: "FP8GEMM_ERR_MISALIGNED", 4: "FP8GEMM_ERR_UNSUPPORTED", 5: "FP8GEMM_ERR_LAUNCH",
          6: "FP8GEMM_ERR_HIP"}
DEVERR_BAD_INDEX = 1
DEVERR_BAD_COUNT = 2

#: exported C symbols and their ctypes signatures (restype, argtypes)
_P, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
SIGNATURES = {
    "fp8gemm_nt": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "fp8gemm_nt_noalloc": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "fp8gemm_nt_specialized": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "fp8gemm_specialize_nt": (ctypes.c_int, [_I64, _I64, _I64, ctypes.POINTER(ctypes.c_double)]),
    "fp8gemm_specialized_code_object": (ctypes.c_int, [ctypes.c_int] * 6 + [_I64, _I64, _P,
                                                       ctypes.POINTER(ctypes.c_size_t), ctypes.c_char_p,
                                                       ctypes.c_int]),
    "fp8gemm_specialized_count": (ctypes.c_int, []),
    "fp8gemm_grouped_contiguous": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P]),
    "fp8gemm_grouped_masked": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _I64, _P]),
    "fp8gemm_quantize_1x128": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _P]),
    "fp8gemm_quantize_1x128_masked": (ctypes.c_int, [_P, _P, _P, _P, _I32, _I64, _I64, _P]),
    "fp8gemm_fp8fp4_grouped_masked": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _I64, _P]),
    "fp8gemm_swiglu_quantize_1x128": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _P]),
    "fp8gemm_swiglu_quantize_1x128_masked": (ctypes.c_int, [_P, _P, _P, _P, _I32, _I64, _I64, _P]),
    "fp8gemm_moe_expert_masked": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                                 _I32, _I64, _I64, _I64, _I64, _P]),
    "fp8gemm_route_topk": (ctypes.c_int, [_P, _P, _P, _P, _I64] + [_I32] * 8 + [_F32, _P]),
    "fp8gemm_route_topk_backward": (ctypes.c_int, [_P, _P, _P, _P, _I64] + [_I32] * 5 + [_F32, _P]),
    "fp8gemm_moe_dispatch_masked": (ctypes.c_int, [_P] * 6 + [_I64, _I64, _I32, _I32, _I64, _I32, _P]),
    "fp8gemm_moe_dispatch_contiguous": (ctypes.c_int, [_P] * 6 + [_I64, _I64, _I32, _I32, _I64, _I32, _P]),
    "fp8gemm_moe_combine": (ctypes.c_int, [_P] * 4 + [_I64, _I64, _I32, _I64, _P]),
    "fp8gemm_moe_combine_backward": (ctypes.c_int, [_P] * 6 + [_I64, _I64, _I32, _I64, _P]),
    "fp8gemm_w4_gemv": (ctypes.c_int, [_P] * 5 + [_I64, _I64, _I64, _I32, _I32, _P]),
    "fp8gemm_w4_gemv_experts": (ctypes.c_int, [_P] * 6 + [_I64, _I32, _I32, _I64, _I64] + [_I32] * 5 + [_P]),
    "fp8gemm_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fp8gemm_init": (ctypes.c_int, []),
    "fp8gemm_prepare_stream": (ctypes.c_int, [_P]),
    "fp8gemm_set_num_cus": (ctypes.c_int, [ctypes.c_int]),
    "fp8gemm_last_config": (ctypes.c_int, [ctypes.c_char_p, ctypes.c_int]),
    "fp8gemm_read_device_error": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32)]),
}


class Fp8GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, status_string(status), STATUS.get(status, status)))


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libfp8gemm.so is not built (python -m fp8_block_scaled_x128_amd.build)")
        l = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def status_string(status: int) -> str:
    return lib().fp8gemm_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != 0:
        raise Fp8GemmError(status, where)


def init() -> None:
    _check(lib().fp8gemm_init(), "fp8gemm_init")


def prepare_stream(stream=None) -> None:
    """Create the split-K workspace of `stream` (default: torch's current stream) now, so that
    later calls on it -- HIP graph capture included -- allocate nothing."""
    torch = _torch()
    _check(lib().fp8gemm_prepare_stream(_stream(stream, torch.cuda.current_device())), "fp8gemm_prepare_stream")


def set_num_cus(n: int) -> None:
    _check(lib().fp8gemm_set_num_cus(int(n)), "fp8gemm_set_num_cus")


def last_config() -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib().fp8gemm_last_config(buf, 256), "fp8gemm_last_config")
    return buf.value.decode()


# ---- tensor front end -------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _stream(stream, device):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def read_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    torch = _torch()
    dev = torch.cuda.current_device()
    v = ctypes.c_int32(0)
    _check(lib().fp8gemm_read_device_error(_stream(stream, dev), ctypes.byref(v)),
           "fp8gemm_read_device_error")
    return v.value


def _codes(t, name):
    torch = _torch()
    if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError("%s must be float8_e4m3fn or uint8 codes, got %s" % (name, t.dtype))
    return _dev_contig(t, name)


def _dev_contig(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _f32(t, name):
    torch = _torch()
    if t.dtype != torch.float32:
        raise TypeError("%s must be float32, got %s" % (name, t.dtype))
    return _dev_contig(t, name)


def _i32(t, name):
    torch = _torch()
    if t.dtype != torch.int32:
        raise TypeError("%s must be int32, got %s" % (name, t.dtype))
    return _dev_contig(t, name)


def _out(out, shape, device):
    torch = _torch()
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != tuple(shape):
        raise ValueError("out must be bfloat16 of shape %s" % (tuple(shape),))
    return _dev_contig(out, "out")


def _shape_check(cond, msg):
    if not cond:
        raise ValueError(msg)


def gemm_nt(A, sa, B, sb, out=None, stream=None):
    """D[M,N] (bf16) = A[M,K] . B[N,K]^T with sa [K/128, M] and sb [ceil(N/128), K/128]."""
    return _dense("fp8gemm_nt", A, sa, B, sb, out, stream)


def gemm_nt_noalloc(A, sa, B, sb, out=None, stream=None):
    """gemm_nt with its split-K partials in the library's static device scratch: the library
    allocates nothing (pass `out`, so that this wrapper does not allocate either).  Calls that
    overlap in time on one GPU race on the scratch."""
    return _dense("fp8gemm_nt_noalloc", A, sa, B, sb, out, stream)


def gemm_nt_specialized(A, sa, B, sb, out=None, stream=None):
    """gemm_nt with the tiled kernel compiled at run time for this N and K (cached per device);
    the same results, bit for bit."""
    return _dense("fp8gemm_nt_specialized", A, sa, B, sb, out, stream)


def specialize_nt(M: int, N: int, K: int) -> float:
    """Build (or find cached) the kernel gemm_nt_specialized runs for (M, N, K) on the current
    device; returns the compile + load time in ms (0.0 when it was cached)."""
    ms = ctypes.c_double(0.0)
    _check(lib().fp8gemm_specialize_nt(int(M), int(N), int(K), ctypes.byref(ms)), "fp8gemm_specialize_nt")
    return ms.value


def specialized_code_object(layout: int, bm: int, bn: int, waves_m: int, waves_n: int, stages: int,
                            N: int, K: int):
    """(code object bytes, kernel symbol) of a tiled table entry specialised to (N, K); no GPU."""
    size = ctypes.c_size_t(0)
    log = ctypes.create_string_buffer(65536)
    args = [int(layout), int(bm), int(bn), int(waves_m), int(waves_n), int(stages), int(N), int(K)]
    _check(lib().fp8gemm_specialized_code_object(*args, None, ctypes.byref(size), log, len(log)),
           "fp8gemm_specialized_code_object: " + log.value.decode(errors="replace")[:2000])
    buf = ctypes.create_string_buffer(size.value)
    _check(lib().fp8gemm_specialized_code_object(*args, buf, ctypes.byref(size), log, len(log)),
           "fp8gemm_specialized_code_object")
    return buf.raw[:size.value], log.value.decode()


def specialized_count() -> int:
    """Number of run-time specialised kernels cached in this process."""
    return int(lib().fp8gemm_specialized_count())


def _dense(fn, A, sa, B, sb, out, stream):
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sa, sb = _f32(sa, "sa"), _f32(sb, "sb")
    _shape_check(A.dim() == 2 and B.dim() == 2 and A.shape[1] == B.shape[1], "A [M,K] and B [N,K]")
    M, K = A.shape
    N = B.shape[0]
    _shape_check(tuple(sa.shape) == (K // 128, M) and tuple(sb.shape) == ((N + 127) // 128, K // 128),
                 "sa [K/128,M], sb [ceil(N/128),K/128]")
    D = _out(out, (M, N), A.device)
    with torch.cuda.device(A.device):
        st = getattr(lib(), fn)(A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(), D.data_ptr(),
                                M, N, K, _stream(stream, A.device))
    _check(st, fn)
    return D


def grouped_contiguous(A, sa, B, sb, m_indices, out=None, stream=None):
    """MoE contiguous layout: A [M_total,K], sa [K/128,M_total], B [G,N,K], m_indices int32 [M_total]
    (-1 = padding).
    Padding rows of ``out`` are left untouched (zeros when ``out`` is allocated here)."""
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sa, sb = _f32(sa, "sa"), _f32(sb, "sb")
    m_indices = _i32(m_indices, "m_indices")
    _shape_check(A.dim() == 2 and B.dim() == 3 and A.shape[1] == B.shape[2], "A [M,K] and B [G,N,K]")
    M, K = A.shape
    G, N = B.shape[0], B.shape[1]
    _shape_check(tuple(sa.shape) == (K // 128, M) and tuple(sb.shape) == (G, (N + 127) // 128, K // 128)
                 and tuple(m_indices.shape) == (M,), "sa [K/128,M], sb [G,ceil(N/128),K/128], m_indices [M]")
    if out is None:
        out = torch.zeros((M, N), dtype=torch.bfloat16, device=A.device)
    D = _out(out, (M, N), A.device)
    with torch.cuda.device(A.device):
        st = lib().fp8gemm_grouped_contiguous(A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(),
                                              m_indices.data_ptr(), D.data_ptr(), M, N, K, G,
                                              _stream(stream, A.device))
    _check(st, "fp8gemm_grouped_contiguous")
    return D


def grouped_masked(A, sa, B, sb, masked_m, expected_m: int, out=None, stream=None):
    """MoE masked layout: A [G,M_max,K], sa [G,K/128,M_max], B [G,N,K], masked_m int32 [G]; rows past masked_m[g] of
    ``out`` are left untouched (zeros when ``out`` is allocated here)."""
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sa, sb = _f32(sa, "sa"), _f32(sb, "sb")
    masked_m = _i32(masked_m, "masked_m")
    _shape_check(A.dim() == 3 and B.dim() == 3 and A.shape[0] == B.shape[0] and A.shape[2] == B.shape[2],
                 "A [G,M_max,K] and B [G,N,K]")
    G, M_max, K = A.shape
    N = B.shape[1]
    _shape_check(tuple(sa.shape) == (G, K // 128, M_max) and tuple(sb.shape) == (G, (N + 127) // 128, K // 128)
                 and tuple(masked_m.shape) == (G,), "sa [G,K/128,M_max], sb [G,ceil(N/128),K/128], masked_m [G]")
    if out is None:
        out = torch.zeros((G, M_max, N), dtype=torch.bfloat16, device=A.device)
    D = _out(out, (G, M_max, N), A.device)
    with torch.cuda.device(A.device):
        st = lib().fp8gemm_grouped_masked(A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(),
                                          masked_m.data_ptr(), D.data_ptr(), G, M_max, N, K,
                                          int(expected_m), _stream(stream, A.device))
    _check(st, "fp8gemm_grouped_masked")
    return D


def _u8(t, name):
    torch = _torch()
    if t.dtype != torch.uint8:
        raise TypeError("%s must be uint8, got %s" % (name, t.dtype))
    return _dev_contig(t, name)


def fp8fp4_grouped_masked(A, sa, B, sb, masked_m, expected_m: int, out=None, stream=None):
    """Masked layout with B in E2M1: A [G,M_max,K] e4m3 codes, sa [G,K/128,M_max], B uint8
    [G,N,K/2] (two E2M1 codes per byte, even element in the low nibble), sb uint8 [G,N,K/32]
    (E8M0 scales per 32 K), masked_m int32 [G].  Rows past masked_m[g] of ``out`` are left
    untouched (zeros when ``out`` is allocated here)."""
    torch = _torch()
    A = _codes(A, "A")
    B, sb = _u8(B, "B"), _u8(sb, "sb")
    sa = _f32(sa, "sa")
    masked_m = _i32(masked_m, "masked_m")
    _shape_check(A.dim() == 3 and B.dim() == 3 and A.shape[0] == B.shape[0] and 2 * B.shape[2] == A.shape[2],
                 "A [G,M_max,K] and B [G,N,K/2]")
    G, M_max, K = A.shape
    N = B.shape[1]
    _shape_check(tuple(sa.shape) == (G, K // 128, M_max) and tuple(sb.shape) == (G, N, K // 32)
                 and tuple(masked_m.shape) == (G,), "sa [G,K/128,M_max], sb [G,N,K/32], masked_m [G]")
    if out is None:
        out = torch.zeros((G, M_max, N), dtype=torch.bfloat16, device=A.device)
    D = _out(out, (G, M_max, N), A.device)
    with torch.cuda.device(A.device):
        st = lib().fp8gemm_fp8fp4_grouped_masked(A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(),
                                                 masked_m.data_ptr(), D.data_ptr(), G, M_max, N, K,
                                                 int(expected_m), _stream(stream, A.device))
    _check(st, "fp8gemm_fp8fp4_grouped_masked")
    return D


def _bf16(t, name):
    torch = _torch()
    if t.dtype != torch.bfloat16:
        raise TypeError("%s must be bfloat16, got %s" % (name, t.dtype))
    return _dev_contig(t, name)


def _quant_outputs(codes, scales, codes_shape, scales_shape, device):
    torch = _torch()
    if codes is None:
        codes = torch.empty(codes_shape, dtype=torch.float8_e4m3fn, device=device)
    if scales is None:
        scales = torch.empty(scales_shape, dtype=torch.float32, device=device)
    codes, scales = _codes(codes, "codes"), _f32(scales, "scales")
    _shape_check(tuple(codes.shape) == tuple(codes_shape) and tuple(scales.shape) == tuple(scales_shape),
                 "codes %s, scales %s" % (tuple(codes_shape), tuple(scales_shape)))
    return codes, scales


def quantize_1x128(X, codes=None, scales=None, stream=None):
    """Activations X bf16 [M,K] -> (E4M3 codes [M,K], scales fp32 [K/128,M]), one scale per 1x128
    block of a row, in the layout gemm_nt and grouped_contiguous take as A and sa."""
    torch = _torch()
    X = _bf16(X, "X")
    _shape_check(X.dim() == 2, "X [M,K]")
    M, K = X.shape
    codes, scales = _quant_outputs(codes, scales, (M, K), (K // 128, M), X.device)
    with torch.cuda.device(X.device):
        st = lib().fp8gemm_quantize_1x128(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), M, K,
                                          _stream(stream, X.device))
    _check(st, "fp8gemm_quantize_1x128")
    return codes, scales


def quantize_1x128_masked(X, masked_m, codes=None, scales=None, stream=None):
    """Masked layout: X bf16 [G,M_max,K] -> (codes [G,M_max,K], scales [G,K/128,M_max]); rows at or
    past masked_m[g] are not written (zeros when the outputs are allocated here)."""
    torch = _torch()
    X = _bf16(X, "X")
    masked_m = _i32(masked_m, "masked_m")
    _shape_check(X.dim() == 3 and tuple(masked_m.shape) == (X.shape[0],), "X [G,M_max,K], masked_m [G]")
    G, M_max, K = X.shape
    if codes is None:
        codes = torch.zeros((G, M_max, K), dtype=torch.uint8, device=X.device).view(torch.float8_e4m3fn)
    if scales is None:
        scales = torch.zeros((G, K // 128, M_max), dtype=torch.float32, device=X.device)
    codes, scales = _quant_outputs(codes, scales, (G, M_max, K), (G, K // 128, M_max), X.device)
    with torch.cuda.device(X.device):
        st = lib().fp8gemm_quantize_1x128_masked(X.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                                 masked_m.data_ptr(), G, M_max, K,
                                                 _stream(stream, X.device))
    _check(st, "fp8gemm_quantize_1x128_masked")
    return codes, scales


def swiglu_quantize_1x128(Y, codes=None, scales=None, stream=None):
    """SwiGLU + requantisation: Y bf16 [M,2I] (gate | up) -> (codes [M,I], scales fp32 [I/128,M]) of
    h = silu(gate) * up, one scale per 1x128 block (the second expert layer's A and sa)."""
    torch = _torch()
    Y = _bf16(Y, "Y")
    _shape_check(Y.dim() == 2 and Y.shape[1] % 2 == 0, "Y [M,2I]")
    M, I = Y.shape[0], Y.shape[1] // 2
    codes, scales = _quant_outputs(codes, scales, (M, I), (I // 128, M), Y.device)
    with torch.cuda.device(Y.device):
        st = lib().fp8gemm_swiglu_quantize_1x128(Y.data_ptr(), codes.data_ptr(), scales.data_ptr(), M, I,
                                                 _stream(stream, Y.device))
    _check(st, "fp8gemm_swiglu_quantize_1x128")
    return codes, scales


def swiglu_quantize_1x128_masked(Y, masked_m, codes=None, scales=None, stream=None):
    """Masked layout: Y bf16 [G,M_max,2I] -> (codes [G,M_max,I], scales [G,I/128,M_max]); rows at or
    past masked_m[g] are not written (zeros when the outputs are allocated here)."""
    torch = _torch()
    Y = _bf16(Y, "Y")
    masked_m = _i32(masked_m, "masked_m")
    _shape_check(Y.dim() == 3 and Y.shape[2] % 2 == 0 and tuple(masked_m.shape) == (Y.shape[0],),
                 "Y [G,M_max,2I], masked_m [G]")
    G, M_max, I = Y.shape[0], Y.shape[1], Y.shape[2] // 2
    if codes is None:
        codes = torch.zeros((G, M_max, I), dtype=torch.uint8, device=Y.device).view(torch.float8_e4m3fn)
    if scales is None:
        scales = torch.zeros((G, I // 128, M_max), dtype=torch.float32, device=Y.device)
    codes, scales = _quant_outputs(codes, scales, (G, M_max, I), (G, I // 128, M_max), Y.device)
    with torch.cuda.device(Y.device):
        st = lib().fp8gemm_swiglu_quantize_1x128_masked(Y.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                                        masked_m.data_ptr(), G, M_max, I,
                                                        _stream(stream, Y.device))
    _check(st, "fp8gemm_swiglu_quantize_1x128_masked")
    return codes, scales


def moe_expert_masked(A, sa, W1, s1, W2, s2, masked_m, expected_m: int, out=None, workspace=None,
                      stream=None):
    """One MoE expert layer per group, masked layout: out = (swiglu(A . W1^T) requantised) . W2^T.
    A [G,M_max,H] codes, sa [G,H/128,M_max], W1 [G,2I,H], s1 [G,2I/128,H/128], W2 [G,H,I],
    s2 [G,H/128,I/128], masked_m int32 [G].  ``workspace``: optional (Y1 bf16 [G,M_max,2I],
    Hq codes [G,M_max,I], sh fp32 [G,I/128,M_max]), allocated here when None.  Returns out bf16
    [G,M_max,H] (rows past masked_m[g] untouched: zeros when allocated here)."""
    torch = _torch()
    A, W1, W2 = _codes(A, "A"), _codes(W1, "W1"), _codes(W2, "W2")
    sa, s1, s2 = _f32(sa, "sa"), _f32(s1, "s1"), _f32(s2, "s2")
    masked_m = _i32(masked_m, "masked_m")
    _shape_check(A.dim() == 3 and W1.dim() == 3 and W2.dim() == 3, "A [G,M_max,H], W1 [G,2I,H], W2 [G,H,I]")
    G, M_max, H = A.shape
    I = W2.shape[2]
    _shape_check(tuple(W1.shape) == (G, 2 * I, H) and tuple(W2.shape) == (G, H, I)
                 and tuple(sa.shape) == (G, H // 128, M_max)
                 and tuple(s1.shape) == (G, (2 * I + 127) // 128, H // 128)
                 and tuple(s2.shape) == (G, (H + 127) // 128, I // 128) and tuple(masked_m.shape) == (G,),
                 "A [G,M_max,H], sa [G,H/128,M_max], W1 [G,2I,H], s1 [G,2I/128,H/128], W2 [G,H,I], "
                 "s2 [G,H/128,I/128], masked_m [G]")
    if workspace is None:
        workspace = (torch.empty((G, M_max, 2 * I), dtype=torch.bfloat16, device=A.device),
                     torch.empty((G, M_max, I), dtype=torch.float8_e4m3fn, device=A.device),
                     torch.empty((G, I // 128, M_max), dtype=torch.float32, device=A.device))
    Y1, Hq, sh = workspace
    Y1, Hq, sh = _bf16(Y1, "Y1"), _codes(Hq, "Hq"), _f32(sh, "sh")
    _shape_check(tuple(Y1.shape) == (G, M_max, 2 * I) and tuple(Hq.shape) == (G, M_max, I)
                 and tuple(sh.shape) == (G, I // 128, M_max), "workspace shapes")
    if out is None:
        out = torch.zeros((G, M_max, H), dtype=torch.bfloat16, device=A.device)
    D = _out(out, (G, M_max, H), A.device)
    with torch.cuda.device(A.device):
        st = lib().fp8gemm_moe_expert_masked(A.data_ptr(), sa.data_ptr(), W1.data_ptr(), s1.data_ptr(),
                                             W2.data_ptr(), s2.data_ptr(), masked_m.data_ptr(),
                                             Y1.data_ptr(), Hq.data_ptr(), sh.data_ptr(), D.data_ptr(),
                                             G, M_max, H, I, int(expected_m), _stream(stream, A.device))
    _check(st, "fp8gemm_moe_expert_masked")
    return D


# ---- expert routing, token permutation, 4-bit matrix-vector products ---------------------------

_SCORES = {"softmax": 0, "sigmoid": 1}


def _call(fn, device, stream, *args):
    """One C call on torch's current stream of `device` (or `stream`)."""
    c = _cuda()
    if stream is None:
        s = c._cuda_getCurrentRawStream(device)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    f = getattr(_lib or lib(), fn)
    if device == c._cuda_getDevice():
        st = f(*args, s)
    else:
        with _torch().cuda.device(device):
            st = f(*args, s)
    if st != 0:
        raise Fp8GemmError(st, fn)


def _cuda():
    """torch's C module (the current stream and device without the Python layers above it)."""
    global _torch_c
    if _torch_c is None:
        _torch_c = _torch()._C
    return _torch_c


_torch_c = None


def _take(t, dtype, shape, device, name):
    """Address of a contiguous device tensor of this type and shape."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != device:
        raise ValueError("%s must be a tensor of device %d" % (name, device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _device_of(t, dims, name):
    d = t.get_device()
    if d < 0:
        raise ValueError("%s must be a device tensor" % name)
    if t.dim() != dims:
        raise ValueError("%s must have %d dimensions" % (name, dims))
    return d


def _logits(logits, device):
    torch = _torch()
    if logits.dtype is torch.float32:
        return _take(logits, torch.float32, logits.shape, device, "logits"), 0
    return _take(logits, torch.bfloat16, logits.shape, device, "logits"), 1


def _score(score):
    if score not in _SCORES:
        raise ValueError('score must be "softmax" or "sigmoid"')
    return _SCORES[score]


def route_topk(logits, k: int, bias=None, score="softmax", n_group: int = 1, topk_group: int = 1, group_top: int = 1,
               renorm: bool = True, scale: float = 1.0, ids=None, weights=None, stream=None):
    """The k experts of each token and their weights: logits fp32 or bf16 [T,E] -> (ids int32 [T,k],
    weights fp32 [T,k]).  ``bias`` fp32 [E] enters the choice, not the weights; with ``n_group`` > 1
    only the experts of the ``topk_group`` best groups (by the sum of their ``group_top`` largest
    choice values) can be chosen; ``renorm`` divides a token's weights by their sum.  Ties go to the
    lower index; where fewer than k experts can be chosen the rest are id -1, weight 0."""
    torch = _torch()
    dev = _device_of(logits, 2, "logits")
    p, dtype = _logits(logits, dev)
    T, E = logits.shape
    pb = None if bias is None else _take(bias, torch.float32, (E,), dev, "bias")
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if weights is None:
        weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _call("fp8gemm_route_topk", dev, stream, p, pb, _take(ids, torch.int32, (T, k), dev, "ids"),
          _take(weights, torch.float32, (T, k), dev, "weights"), T, E, k, dtype, _score(score), n_group, topk_group,
          group_top, int(renorm), scale)
    return ids, weights


def route_topk_backward(logits, ids, dweights, score="softmax", renorm: bool = True, scale: float = 1.0, dlogits=None,
                        stream=None):
    """Gradient of route_topk's weights: dweights fp32 [T,k] -> dlogits [T,E] of the logits' type."""
    torch = _torch()
    dev = _device_of(logits, 2, "logits")
    p, dtype = _logits(logits, dev)
    T, E = logits.shape
    _device_of(ids, 2, "ids")
    k = ids.shape[1]
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    _call("fp8gemm_route_topk_backward", dev, stream, p, _take(ids, torch.int32, (T, k), dev, "ids"),
          _take(dweights, torch.float32, (T, k), dev, "dweights"), _take(dlogits, logits.dtype, (T, E), dev, "dlogits"),
          T, E, k, dtype, _score(score), int(renorm), scale)
    return dlogits


def _code_ptr(t, shape, device, name):
    torch = _torch()
    return _take(t, torch.uint8 if t.dtype is torch.uint8 else torch.float8_e4m3fn, shape, device, name)


def moe_dispatch_masked(X, ids, G: int, M_max: int, first_expert: int = 0, codes=None, scales=None, masked_m=None,
                        row_map=None, stream=None):
    """Token rows into the masked layout, quantised: X bf16 [T,H], ids int32 [T,k] -> (codes
    [G,M_max,H], scales fp32 [G,H/128,M_max], masked_m int32 [G], row_map int32 [T,k]).  A pair goes
    to expert ids - first_expert if that is one of the G; its row is g * M_max + rank, or -1 (another
    rank's expert, or past M_max).  Rows that no pair goes to are left untouched (zeros when the
    outputs are allocated here)."""
    torch = _torch()
    dev = _device_of(X, 2, "X")
    T, H = X.shape
    _device_of(ids, 2, "ids")
    k = ids.shape[1]
    if codes is None:
        codes = torch.zeros((G, M_max, H), dtype=torch.uint8, device=X.device).view(torch.float8_e4m3fn)
    if scales is None:
        scales = torch.zeros((G, H // 128, M_max), dtype=torch.float32, device=X.device)
    if masked_m is None:
        masked_m = torch.empty((G,), dtype=torch.int32, device=X.device)
    if row_map is None:
        row_map = torch.empty((T, k), dtype=torch.int32, device=X.device)
    _call("fp8gemm_moe_dispatch_masked", dev, stream, _take(X, torch.bfloat16, (T, H), dev, "X"),
          _take(ids, torch.int32, (T, k), dev, "ids"), _code_ptr(codes, (G, M_max, H), dev, "codes"),
          _take(scales, torch.float32, (G, H // 128, M_max), dev, "scales"),
          _take(masked_m, torch.int32, (G,), dev, "masked_m"), _take(row_map, torch.int32, (T, k), dev, "row_map"),
          T, H, k, G, M_max, first_expert)
    return codes, scales, masked_m, row_map


def moe_dispatch_contiguous(X, ids, G: int, M_total: int = None, first_expert: int = 0, codes=None, scales=None,
                            m_indices=None, row_map=None, stream=None):
    """Token rows into the contiguous layout, quantised: X bf16 [T,H], ids int32 [T,k] -> (codes
    [M_total,H], scales fp32 [H/128,M_total], m_indices int32 [M_total], row_map int32 [T,k]).  Each
    expert's rows are padded to a multiple of 128.  M_total None: the rows of ``codes`` or
    ``m_indices`` if given, else room for every pair."""
    torch = _torch()
    dev = _device_of(X, 2, "X")
    T, H = X.shape
    _device_of(ids, 2, "ids")
    k = ids.shape[1]
    if M_total is None:
        if codes is not None:
            M_total = codes.shape[0]
        elif m_indices is not None:
            M_total = m_indices.shape[0]
        else:
            M_total = -(-(T * k + 127 * min(G, T * k)) // 128) * 128
    if codes is None:
        codes = torch.zeros((M_total, H), dtype=torch.uint8, device=X.device).view(torch.float8_e4m3fn)
    if scales is None:
        scales = torch.zeros((H // 128, M_total), dtype=torch.float32, device=X.device)
    if m_indices is None:
        m_indices = torch.empty((M_total,), dtype=torch.int32, device=X.device)
    if row_map is None:
        row_map = torch.empty((T, k), dtype=torch.int32, device=X.device)
    _call("fp8gemm_moe_dispatch_contiguous", dev, stream, _take(X, torch.bfloat16, (T, H), dev, "X"),
          _take(ids, torch.int32, (T, k), dev, "ids"), _code_ptr(codes, (M_total, H), dev, "codes"),
          _take(scales, torch.float32, (H // 128, M_total), dev, "scales"),
          _take(m_indices, torch.int32, (M_total,), dev, "m_indices"),
          _take(row_map, torch.int32, (T, k), dev, "row_map"), T, H, k, G, M_total, first_expert)
    return codes, scales, m_indices, row_map


def _combine_shapes(Y, weights, row_map, T):
    """(k, rows of Y) of a combine; Y [R,H] or [G,M_max,H]."""
    pairs = weights if weights is not None else row_map
    if pairs is None:
        raise ValueError("weights or row_map must be given")
    if pairs.dim() != 2:
        raise ValueError("weights and row_map must be [T,k]")
    if T is not None and pairs.shape[0] != T:
        raise ValueError("weights and row_map must have a row per token")
    R = None
    if Y is not None:
        if Y.dim() not in (2, 3):
            raise ValueError("Y must be [R,H] or [G,M_max,H]")
        R = Y.shape[0] if Y.dim() == 2 else Y.shape[0] * Y.shape[1]
    return pairs.shape[0], pairs.shape[1], R


def moe_combine(Y, weights=None, row_map=None, out=None, stream=None):
    """out[t] = sum_j weights[t,j] * Y[row_map[t,j]]: Y bf16 [R,H] (or [G,M_max,H]), weights fp32
    [T,k] (None: ones), row_map int32 [T,k] with -1 left out (None: row t * k + j) -> bf16 [T,H]."""
    torch = _torch()
    T, k, R = _combine_shapes(Y, weights, row_map, None)
    dev, H = Y.get_device(), Y.shape[-1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=Y.device)
    _call("fp8gemm_moe_combine", dev, stream, _take(Y, torch.bfloat16, Y.shape, dev, "Y"),
          None if weights is None else _take(weights, torch.float32, (T, k), dev, "weights"),
          None if row_map is None else _take(row_map, torch.int32, (T, k), dev, "row_map"),
          _take(out, torch.bfloat16, (T, H), dev, "out"), T, H, k, R)
    return out


def moe_combine_backward(dout, Y, weights=None, row_map=None, dY=None, dweights=None, stream=None):
    """Gradients of moe_combine: dout bf16 [T,H], Y bf16 [R,H] (or [G,M_max,H]) -> (dY of Y's shape,
    dweights fp32 [T,k]).  Rows of dY that no pair names are left untouched (zeros when allocated
    here)."""
    torch = _torch()
    dev = _device_of(dout, 2, "dout")
    T, H = dout.shape
    T, k, R = _combine_shapes(Y, weights, row_map, T)
    if Y.shape[-1] != H:
        raise ValueError("Y must have dout's columns")
    if dY is None:
        dY = torch.zeros_like(Y)
    if dweights is None:
        dweights = torch.empty((T, k), dtype=torch.float32, device=dout.device)
    _call("fp8gemm_moe_combine_backward", dev, stream, _take(dout, torch.bfloat16, (T, H), dev, "dout"),
          _take(Y, torch.bfloat16, Y.shape, dev, "Y"),
          None if weights is None else _take(weights, torch.float32, (T, k), dev, "weights"),
          None if row_map is None else _take(row_map, torch.int32, (T, k), dev, "row_map"),
          _take(dY, torch.bfloat16, Y.shape, dev, "dY"), _take(dweights, torch.float32, (T, k), dev, "dweights"),
          T, H, k, R)
    return dY, dweights


def _w4_format(W, scales, zeros, lead, N, K, device):
    """(addresses of W, scales, zeros, format, group): E8M0 scales (uint8) are MXFP4, bf16 ones INT4."""
    torch = _torch()
    if scales.dim() != len(lead) + 2 or scales.shape[-1] == 0 or K % scales.shape[-1] != 0:
        raise ValueError("scales must have one value per group of K")
    groups = scales.shape[-1]
    shape = (*lead, N, groups)
    pw = _take(W, torch.uint8, W.shape, device, "W")
    if scales.dtype is torch.uint8:
        if zeros is not None:
            raise ValueError("MXFP4 weights have no zeros")
        return pw, _take(scales, torch.uint8, shape, device, "scales"), None, 0, K // groups
    ps = _take(scales, torch.bfloat16, shape, device, "scales")
    return pw, ps, None if zeros is None else _take(zeros, torch.uint8, shape, device, "zeros"), 1, K // groups


def w4_gemv(X, W, scales, zeros=None, out=None, stream=None):
    """Y = X . V^T for few rows: X bf16 [M,K], W uint8 [N,K/2] (two codes a byte, the even element in
    the low nibble) -> bf16 [M,N].  ``scales`` uint8 [N,K/32]: MXFP4 (E2M1 codes, E8M0 scales);
    bf16 [N,K/group], group 32, 64 or 128: INT4, V = (code - zero) * scale with ``zeros`` uint8
    [N,K/group] (None: 8)."""
    torch = _torch()
    dev = _device_of(X, 2, "X")
    M, K = X.shape
    if W.dim() != 2 or 2 * W.shape[1] != K:
        raise ValueError("W must be [N,K/2]")
    N = W.shape[0]
    pw, ps, pz, fmt, group = _w4_format(W, scales, zeros, (), N, K, dev)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _call("fp8gemm_w4_gemv", dev, stream, _take(X, torch.bfloat16, (M, K), dev, "X"), pw, ps, pz,
          _take(out, torch.bfloat16, (M, N), dev, "out"), M, N, K, fmt, group)
    return out


def w4_gemv_experts(X, W, scales, ids, zeros=None, first_expert: int = 0, swiglu: bool = False, out=None, stream=None):
    """w4_gemv with the matrix of each pair's expert: W uint8 [E,N,K/2], scales (and zeros)
    [E,N,K/group], ids int32 [T,k] -> bf16 [T*k,N].  X bf16 [T,K], or [T*k,K] with a row per pair.
    ``swiglu``: silu(rows [0,N/2)) * rows [N/2,N) -> [T*k,N/2].  Pairs without an expert among the E
    (id - first_expert) get zeros."""
    torch = _torch()
    dev = _device_of(X, 2, "X")
    _device_of(ids, 2, "ids")
    T, k = ids.shape
    rows, K = X.shape
    if rows != T and rows != T * k:
        raise ValueError("X must have a row per token or per pair")
    if W.dim() != 3 or 2 * W.shape[2] != K:
        raise ValueError("W must be [E,N,K/2]")
    E, N = W.shape[0], W.shape[1]
    if swiglu and N % 2:
        raise ValueError("swiglu needs gate and up rows")
    pw, ps, pz, fmt, group = _w4_format(W, scales, zeros, (E,), N, K, dev)
    nout = N // 2 if swiglu else N
    if out is None:
        out = torch.empty((T * k, nout), dtype=torch.bfloat16, device=X.device)
    _call("fp8gemm_w4_gemv_experts", dev, stream, _take(X, torch.bfloat16, (rows, K), dev, "X"), pw, ps, pz,
          _take(ids, torch.int32, (T, k), dev, "ids"), _take(out, torch.bfloat16, (T * k, nout), dev, "out"),
          T, k, E, N, K, fmt, group, first_expert, int(rows != T), int(swiglu))
    return out
