// moe_device.h -- device helpers of the routing, permutation and 4-bit product kernels: sums and
// maxima over the 16 lanes of a DPP row, and the exponential the score functions use.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8gemm {

// A value of the lane that `CTRL` (a DPP control of a 16-lane row) names.
template <int CTRL>
__device__ __forceinline__ int dpp16(int v) {
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp16f(float v) {
    return __int_as_float(dpp16<CTRL>(__float_as_int(v)));
}

// quad_perm [1,0,3,2], quad_perm [2,3,0,1], row_half_mirror, row_mirror: four steps after which
// every lane of a 16-lane row holds the row's result, the same bits in each (every step adds or
// compares the same two values in both partners).
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

__device__ __forceinline__ float row16_max_f(float v) {
    v = fmaxf(v, dpp16f<kDppXor1>(v));
    v = fmaxf(v, dpp16f<kDppXor2>(v));
    v = fmaxf(v, dpp16f<kDppHalfMirror>(v));
    v = fmaxf(v, dpp16f<kDppMirror>(v));
    return v;
}
__device__ __forceinline__ float row16_sum_f(float v) {
    v += dpp16f<kDppXor1>(v);
    v += dpp16f<kDppXor2>(v);
    v += dpp16f<kDppHalfMirror>(v);
    v += dpp16f<kDppMirror>(v);
    return v;
}

// LDS traffic between the lanes of one wave: its LDS operations execute in order, so only the
// compiler has to keep them so.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// e^x within 2 units in the last place, subnormal results included: x log2(e) = n + f with n a
// whole number and f formed with the low part of log2(e), then 2^f by the hardware and n by ldexp.
// Outside [-120, 100] the result is 0 or infinity all the same; NaN is taken as -120.
__device__ __forceinline__ float exp_f32(float x) {
    x = __builtin_amdgcn_fmed3f(x, -120.0f, 100.0f);
    const float n = __builtin_rintf(x * 1.44269504088896341f);
    const float f = __builtin_fmaf(x, 1.92596299112661746e-8f, __builtin_fmaf(x, 1.44269502162933350f, -n));
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
    const __bf16 b = (__bf16)f;   // round to nearest even
    uint16_t u;
    __builtin_memcpy(&u, &b, 2);
    return u;
}

}  // namespace fp8gemm
