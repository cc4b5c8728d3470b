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
#
# These calls take a few microseconds, so their tensors go to the C ABI through the compiled module
# `_native`, which checks them as it reads them.  A refusal there (-1) is put into words here.

_SCORES = {"softmax": 0, "sigmoid": 1}
_native_module = None


def _calls():
    global _native_module
    if _native_module is None:
        import torch  # noqa: F401  (the module needs torch's libraries in the process)
        if not os.path.exists(os.path.join(_HERE, "_native.so")):
            raise RuntimeError("_native.so is not built (python -m fp8_block_scaled_x128_amd.build)")
        from . import _native as module
        _native_module = module
    return _native_module


def _handle(stream):
    """None (the current stream) or a stream's address."""
    if stream is None:
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(shape, dtype, like, stream, zero=False):
    """A new tensor on `like`'s device, allocated (and filled) on the stream that is to write it."""
    torch = _torch()
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=like.device)


def _require(t, name, dtypes, shape, device):
    """Raise what is wrong with an argument."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor, got %s" % (name, type(t).__name__))
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if len(t.shape) != len(shape) or any(s is not None and s != n for s, n in zip(shape, t.shape)):
        raise ValueError("%s must have shape [%s], got %s" % (name, ",".join("*" if s is None else str(s) for s in shape),
                                                              list(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _refuse(fn, status, *arguments):
    """Raise for a call that did not succeed: the first argument (tensor, name, types, shape) that is not
    as the call takes it, or the C call's status.  None stands for any size, and for a tensor left out."""
    if status > 0:
        raise Fp8GemmError(status, fn)
    device = None
    for t, name, dtypes, shape in arguments:
        if t is None:
            continue
        if device is None:
            device = getattr(t, "device", None)
        _require(t, name, dtypes, shape, device)
    raise ValueError("%s: arguments out of range" % fn)


def _dims(t, n, name):
    """The shape of a tensor of n dimensions."""
    shape = t.shape
    if len(shape) != n:
        raise ValueError("%s must have %d dimensions" % (name, n))
    return shape


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
    if ids is None or weights is None:
        torch = _torch()
        T, _ = _dims(logits, 2, "logits")
        if ids is None:
            ids = _new((T, k), torch.int32, logits, stream)
        if weights is None:
            weights = _new((T, k), torch.float32, logits, stream)
    st = _calls().route_topk(logits, bias, ids, weights, k, _score(score), n_group, topk_group, group_top, renorm, scale,
                              _handle(stream))
    if st != 0:
        torch = _torch()
        T, E = _dims(logits, 2, "logits")
        _refuse("fp8gemm_route_topk", st, (logits, "logits", (torch.float32, torch.bfloat16), (T, E)),
                (bias, "bias", (torch.float32,), (E,)), (ids, "ids", (torch.int32,), (T, k)),
                (weights, "weights", (torch.float32,), (T, k)))
    return ids, weights


def route_topk_backward(logits, ids, dweights, score="softmax", renorm: bool = True, scale: float = 1.0, dlogits=None,
                        stream=None):
    """Gradient of route_topk's weights: dweights fp32 [T,k] -> dlogits [T,E] of the logits' type."""
    if dlogits is None:
        dlogits = _new(_dims(logits, 2, "logits"), logits.dtype, logits, stream)
    st = _calls().route_topk_backward(logits, ids, dweights, dlogits, _score(score), renorm, scale, _handle(stream))
    if st != 0:
        torch = _torch()
        T, E = _dims(logits, 2, "logits")
        k = _dims(ids, 2, "ids")[1]
        _refuse("fp8gemm_route_topk_backward", st, (logits, "logits", (torch.float32, torch.bfloat16), (T, E)),
                (ids, "ids", (torch.int32,), (T, k)), (dweights, "dweights", (torch.float32,), (T, k)),
                (dlogits, "dlogits", (logits.dtype,), (T, E)))
    return dlogits


def _code_types():
    torch = _torch()
    return (torch.float8_e4m3fn, torch.uint8)


def moe_dispatch_masked(X, ids, G: int, M_max: int, first_expert: int = 0, codes=None, scales=None, masked_m=None,
                        row_map=None, stream=None):
    """Token rows into the masked layout, quantised: X bf16 [T,H], ids int32 [T,k] -> (codes
    [G,M_max,H], scales fp32 [G,H/128,M_max], masked_m int32 [G], row_map int32 [T,k]).  A pair goes
    to expert ids - first_expert if that is one of the G; its row is g * M_max + rank, or -1 (another
    rank's expert, or past M_max).  Rows that no pair goes to are left untouched (zeros when the
    outputs are allocated here)."""
    torch = _torch()
    if codes is None or scales is None or masked_m is None or row_map is None:
        H = _dims(X, 2, "X")[1]
        if codes is None:
            codes = _new((G, M_max, H), torch.uint8, X, stream, zero=True).view(torch.float8_e4m3fn)
        if scales is None:
            scales = _new((G, H // 128, M_max), torch.float32, X, stream, zero=True)
        if masked_m is None:
            masked_m = _new((G,), torch.int32, X, stream)
        if row_map is None:
            row_map = _new(_dims(ids, 2, "ids"), torch.int32, X, stream)
    st = _calls().moe_dispatch(X, ids, codes, scales, masked_m, row_map, G, M_max, first_expert, True, _handle(stream))
    if st != 0:
        T, H = _dims(X, 2, "X")
        k = _dims(ids, 2, "ids")[1]
        _refuse("fp8gemm_moe_dispatch_masked", st, (X, "X", (torch.bfloat16,), (T, H)), (ids, "ids", (torch.int32,), (T, k)),
                (codes, "codes", _code_types(), (G, M_max, H)), (scales, "scales", (torch.float32,), (G, H // 128, M_max)),
                (masked_m, "masked_m", (torch.int32,), (G,)), (row_map, "row_map", (torch.int32,), (T, k)))
    return codes, scales, masked_m, row_map


def moe_dispatch_contiguous(X, ids, G: int, M_total: int = None, first_expert: int = 0, codes=None, scales=None,
                            m_indices=None, row_map=None, stream=None):
    """Token rows into the contiguous layout, quantised: X bf16 [T,H], ids int32 [T,k] -> (codes
    [M_total,H], scales fp32 [H/128,M_total], m_indices int32 [M_total], row_map int32 [T,k]).  Each
    expert's rows are padded to a multiple of 128.  M_total None: the rows of ``codes`` or
    ``m_indices`` if given, else room for every pair."""
    torch = _torch()
    if M_total is None:
        if codes is not None:
            M_total = _dims(codes, 2, "codes")[0]
        elif m_indices is not None:
            M_total = _dims(m_indices, 1, "m_indices")[0]
        else:
            T, k = _dims(ids, 2, "ids")
            M_total = -(-(T * k + 127 * min(G, T * k)) // 128) * 128
    if codes is None or scales is None or m_indices is None or row_map is None:
        H = _dims(X, 2, "X")[1]
        if codes is None:
            codes = _new((M_total, H), torch.uint8, X, stream, zero=True).view(torch.float8_e4m3fn)
        if scales is None:
            scales = _new((H // 128, M_total), torch.float32, X, stream, zero=True)
        if m_indices is None:
            m_indices = _new((M_total,), torch.int32, X, stream)
        if row_map is None:
            row_map = _new(_dims(ids, 2, "ids"), torch.int32, X, stream)
    st = _calls().moe_dispatch(X, ids, codes, scales, m_indices, row_map, G, M_total, first_expert, False,
                               _handle(stream))
    if st != 0:
        T, H = _dims(X, 2, "X")
        k = _dims(ids, 2, "ids")[1]
        _refuse("fp8gemm_moe_dispatch_contiguous", st, (X, "X", (torch.bfloat16,), (T, H)), (ids, "ids", (torch.int32,), (T, k)),
                (codes, "codes", _code_types(), (M_total, H)), (scales, "scales", (torch.float32,), (H // 128, M_total)),
                (m_indices, "m_indices", (torch.int32,), (M_total,)), (row_map, "row_map", (torch.int32,), (T, k)))
    return codes, scales, m_indices, row_map


def _pairs(weights, row_map):
    """[T,k] of a combine."""
    if weights is None and row_map is None:
        raise ValueError("weights or row_map must be given")
    return _dims(row_map if weights is None else weights, 2, "row_map" if weights is None else "weights")


def _rows_shape(Y):
    if len(Y.shape) not in (2, 3):
        raise ValueError("Y must be [R,H] or [G,M_max,H]")
    return Y.shape


def moe_combine(Y, weights=None, row_map=None, out=None, stream=None):
    """out[t] = sum_j weights[t,j] * Y[row_map[t,j]]: Y bf16 [R,H] (or [G,M_max,H]), weights fp32
    [T,k] (None: ones), row_map int32 [T,k] with -1 left out (None: row t * k + j) -> bf16 [T,H]."""
    if out is None:
        out = _new((_pairs(weights, row_map)[0], _rows_shape(Y)[-1]), _torch().bfloat16, Y, stream)
    st = _calls().moe_combine(Y, weights, row_map, out, _handle(stream))
    if st != 0:
        torch = _torch()
        T, k = _pairs(weights, row_map)
        _refuse("fp8gemm_moe_combine", st, (Y, "Y", (torch.bfloat16,), _rows_shape(Y)),
                (weights, "weights", (torch.float32,), (T, k)), (row_map, "row_map", (torch.int32,), (T, k)),
                (out, "out", (torch.bfloat16,), (T, Y.shape[-1])))
    return out


def moe_combine_backward(dout, Y, weights=None, row_map=None, dY=None, dweights=None, stream=None):
    """Gradients of moe_combine: dout bf16 [T,H], Y bf16 [R,H] (or [G,M_max,H]) -> (dY of Y's shape,
    dweights fp32 [T,k]).  Rows of dY that no pair names are left untouched (zeros when allocated
    here)."""
    if dY is None:
        dY = _new(_rows_shape(Y), Y.dtype, Y, stream, zero=True)
    if dweights is None:
        dweights = _new(_pairs(weights, row_map), _torch().float32, Y, stream)
    st = _calls().moe_combine_backward(dout, Y, weights, row_map, dY, dweights, _handle(stream))
    if st != 0:
        torch = _torch()
        T, k = _pairs(weights, row_map)
        H = _rows_shape(Y)[-1]
        _refuse("fp8gemm_moe_combine_backward", st, (dout, "dout", (torch.bfloat16,), (T, H)),
                (Y, "Y", (torch.bfloat16,), Y.shape), (weights, "weights", (torch.float32,), (T, k)),
                (row_map, "row_map", (torch.int32,), (T, k)), (dY, "dY", (torch.bfloat16,), Y.shape),
                (dweights, "dweights", (torch.float32,), (T, k)))
    return dY, dweights


def _w4_weights(W, scales, zeros, lead, N, K):
    """What _refuse looks for in 4-bit weights [*lead,N,K/2] with their scales and zeros."""
    torch = _torch()
    if zeros is not None and scales.dtype is torch.uint8:
        raise ValueError("MXFP4 weights have no zeros")
    return ((W, "W", (torch.uint8,), (*lead, N, K // 2)), (scales, "scales", (torch.uint8, torch.bfloat16), (*lead, N, None)),
            (zeros, "zeros", (torch.uint8,), scales.shape))


def w4_gemv(X, W, scales, zeros=None, out=None, stream=None):
    """Y = X . V^T for few rows: X bf16 [M,K], W uint8 [N,K/2] (two codes a byte, the even element in
    the low nibble) -> bf16 [M,N].  ``scales`` uint8 [N,K/32]: MXFP4 (E2M1 codes, E8M0 scales);
    bf16 [N,K/group], group 32, 64 or 128: INT4, V = (code - zero) * scale with ``zeros`` uint8
    [N,K/group] (None: 8)."""
    if out is None:
        out = _new((_dims(X, 2, "X")[0], _dims(W, 2, "W")[0]), _torch().bfloat16, X, stream)
    st = _calls().w4_gemv(X, W, scales, zeros, out, _handle(stream))
    if st != 0:
        torch = _torch()
        M, K = _dims(X, 2, "X")
        N = _dims(W, 2, "W")[0]
        _refuse("fp8gemm_w4_gemv", st, (X, "X", (torch.bfloat16,), (M, K)), *_w4_weights(W, scales, zeros, (), N, K),
                (out, "out", (torch.bfloat16,), (M, N)))
    return out


def w4_gemv_experts(X, W, scales, ids, zeros=None, first_expert: int = 0, swiglu: bool = False, out=None, stream=None):
    """w4_gemv with the matrix of each pair's expert: W uint8 [E,N,K/2], scales (and zeros)
    [E,N,K/group], ids int32 [T,k] -> bf16 [T*k,N].  X bf16 [T,K], or [T*k,K] with a row per pair.
    ``swiglu``: silu(rows [0,N/2)) * rows [N/2,N) -> [T*k,N/2].  Pairs without an expert among the E
    (id - first_expert) get zeros."""
    if out is None:
        T, k = _dims(ids, 2, "ids")
        N = _dims(W, 3, "W")[1]
        out = _new((T * k, N // 2 if swiglu else N), _torch().bfloat16, X, stream)
    st = _calls().w4_gemv_experts(X, W, scales, zeros, ids, out, first_expert, swiglu, _handle(stream))
    if st != 0:
        torch = _torch()
        T, k = _dims(ids, 2, "ids")
        E, N, _ = _dims(W, 3, "W")
        rows, K = _dims(X, 2, "X")
        if st < 0 and rows not in (T, T * k):
            raise ValueError("X must have a row per token or per pair")
        if st < 0 and swiglu and N % 2:
            raise ValueError("swiglu needs gate and up rows")
        _refuse("fp8gemm_w4_gemv_experts", st, (X, "X", (torch.bfloat16,), (rows, K)),
                *_w4_weights(W, scales, zeros, (E,), N, K), (ids, "ids", (torch.int32,), (T, k)),
                (out, "out", (torch.bfloat16,), (T * k, N // 2 if swiglu else N)))
    return out
