// w4_kernels.hip -- gfx950 matrix-vector products with 4-bit weights and group scales: Y = X . V^T
// for few rows of X, V decoded from MXFP4 (E2M1 codes, one E8M0 scale per 32) or INT4 (unsigned
// codes, a bf16 scale and an optional zero point per 32, 64 or 128), and the same with the matrix
// of each of a token's experts.  The mathematics is stated in include/fp8gemm.h.
//
// Bound: the weights are read once, N K / 2 bytes for 2 M N K operations, so the kernel streams.
// At the HBM rate a CU receives about 16 weights per cycle and has 64 lane operations per cycle
// to decode them, 4 a weight; the products run on the matrix cores (16x16x32 bf16, X's rows as one
// operand's 16 rows and 16 weight rows as the other's), where up to 16 rows of X cost the same.
//
// One workgroup of 8 waves owns 16 RN rows of V and all of K; wave w takes the steps (128 values
// of K) w, w + 8, ..., so the workgroup reads each row in runs of 512 bytes, and a ring of PD
// steps keeps that many loads in flight.  The waves' fp32 sums meet in LDS and are added in wave
// order.  In a step lane (n, j) = (lane % 16, lane / 16) loads 16 bytes of row n: its chunk j of
// 32 values.
//   MXFP4: the lane decodes its chunk with the chunk's scale in the conversion instruction (two
//   values each, exact in bf16); matrix-core step i takes the values 8 i .. 8 i + 7 of all four
//   chunks.
//   INT4: the sums of different groups have to stay apart until they are scaled.  Two lane swaps
//   transpose the four chunks' words across the four lanes of a row, so that matrix-core step i
//   takes chunk i alone.  Codes become the bf16 values 16 + q by inserting them below the
//   exponent of 16 (exact); the group's sum is then (sum - (16 + z) sum_k x) * scale in fp32, with
//   sum_k x from one more matrix-core step against ones.

#include "fp8gemm_device.h"
#include "moe_device.h"
#include "moe_internal.h"

namespace fp8gemm {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8, kW4Threads = kWaves * 64;
constexpr int kStep = 128;                 // K values per wave and step: four chunks of 32

enum Mode { kOne = 0, kExperts = 1, kExpertsSwiglu = 2 };

__device__ __forceinline__ v4f mfma_bf16(const v4u& x, const v4u& w, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, w), c, 0, 0, 0);
}

// 8 E2M1 codes of a word times `scale` (a power of two), as bf16.
__device__ __forceinline__ v4u decode_e2m1(uint32_t w, float scale) {
    v4u o;
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    return o;
}

// 8 unsigned codes q of a word as bf16 16 + q, in the order 0 4 1 5 2 6 3 7 (pairs share a mask).
__device__ __forceinline__ v4u decode_u4(uint32_t w) {
    v4u o;
    o[0] = ((w << 3) & 0x00780078u) | 0x41804180u;
    o[1] = ((w >> 1) & 0x00780078u) | 0x41804180u;
    o[2] = ((w >> 5) & 0x00780078u) | 0x41804180u;
    o[3] = ((w >> 9) & 0x00780078u) | 0x41804180u;
    return o;
}
// 8 bf16 values brought into the same order.
__device__ __forceinline__ v4u order_u4(const v4u& x) {
    v4u o;
    o[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);   // 0 4
    o[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);   // 1 5
    o[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);   // 2 6
    o[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);   // 3 7
    return o;
}

// The 4 words of the lanes (n, 0..3) transposed: word i of lane j becomes word j of lane i.
__device__ __forceinline__ void transpose4(v4u& w) {
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w[0] = c[0];
    w[1] = c[1];
    w[2] = d[0];
    w[3] = d[1];
}

// One operand's rows as a bounded buffer: reads past `bytes` give 0.
struct Rows {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t bytes;
    __device__ __forceinline__ Rows(const void* p, int64_t n)
        : rsrc(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)n, kBufferFlags)), bytes((uint32_t)n) {}
};

// GROUP: values per scale; MX: MXFP4; WIDE: a step's scales are adjacent and aligned (K a multiple
// of 128), one load; RN: 16-row tiles of V, MT: 16-row tiles of X; MODE: see Mode (with SwiGLU
// tile 0 holds gate rows and tile 1 the matching up rows).
template <int GROUP, bool MX, bool WIDE, bool ZEROS, int RN, int MT, int PD, int MODE>
__global__ __launch_bounds__(kW4Threads) void w4_kernel(W4Args a) {
    constexpr int PER = kStep / GROUP;             // scales per step
    constexpr int SB = MX ? 1 : 2;                 // bytes per scale
    constexpr bool SWIGLU = MODE == kExpertsSwiglu;
    constexpr int kBatch = RN * MT < 4 ? RN * MT : 4;   // output tiles reduced at a time
    __shared__ v4f red[kWaves][kBatch][64];
    __shared__ int cols[MODE == kOne ? 1 : kW4MaxPairsBySlot];
    __shared__ int count, early;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ln = lane & 15, j = lane >> 4;
    const int tile_rows = SWIGLU ? 16 : 16 * RN;
    const int n0 = blockIdx.x * tile_rows;
    const int n_end = SWIGLU ? a.half : a.N;

    int expert = 0;
    int window = 0;                                // experts: first pair of the scanned window
    do {
        int ncols = 0;
        if constexpr (MODE == kOne) {
            ncols = 1;
        } else {
            // the pairs of this workgroup's expert; their order changes no result
            const int slot = blockIdx.y;
            const int last = min(a.pairs - window, kW4MaxPairsBySlot);
            const int id = a.by_slot ? a.ids[slot] : slot + a.first;
            const bool none = a.by_slot ? (id < a.first || (int64_t)id - a.first >= a.E) : slot == a.E;
            if (tid == 0) count = early = 0;
            __syncthreads();
            if (a.by_slot && none) {
                if (tid == 0) { cols[0] = slot; count = 1; }
            } else {
                for (int p = tid; p < last; p += kW4Threads) {
                    const int o = a.ids[window + p];
                    const bool outside = o < a.first || (int64_t)o - a.first >= a.E;
                    if (none ? outside : o == id && !outside) {
                        cols[atomicAdd(&count, 1)] = window + p;
                        if (a.by_slot && p < slot) early = 1;
                    }
                }
            }
            __syncthreads();
            ncols = a.by_slot && early ? 0 : count;
            expert = none ? -1 : id - a.first;
            if (expert < 0) {                      // pairs without an expert here: zero rows
                for (int i = tid; i < ncols * tile_rows; i += kW4Threads) {
                    const int n = n0 + i % tile_rows;
                    if (n < a.nout) a.Y[(int64_t)cols[i / tile_rows] * a.nout + n] = 0;
                }
                ncols = 0;
            }
        }
        const int64_t matrix = (int64_t)expert * a.N;
        const int row_bytes = a.K / 2, rows = min(n_end - n0, tile_rows);
        const int chunks = a.K / 32, steps = (chunks + 3) / 4;
        const int group_row = a.groups * SB;
        // buffers of this workgroup's rows; with SwiGLU one for the gate rows and one for the up rows
        constexpr int kParts = SWIGLU ? 2 : 1;
        const int64_t first_row[2] = {matrix + n0, matrix + a.half + n0};
        auto part = [&](int r) { return SWIGLU ? r : 0; };

        for (int m0 = MODE == kOne ? blockIdx.y * 16 * MT : 0; MODE == kOne ? m0 >= 0 : m0 < ncols; m0 += 16 * MT) {
            const Rows w0(a.W + first_row[0] * row_bytes, (int64_t)rows * row_bytes);
            const Rows w1(a.W + first_row[kParts - 1] * row_bytes, (int64_t)rows * row_bytes);
            const uint8_t* sp = static_cast<const uint8_t*>(a.scales);
            const Rows s0(sp + first_row[0] * group_row, (int64_t)rows * group_row);
            const Rows s1(sp + first_row[kParts - 1] * group_row, (int64_t)rows * group_row);
            const Rows z0(ZEROS ? a.zeros + first_row[0] * a.groups : nullptr, ZEROS ? (int64_t)rows * a.groups : 0);
            const Rows z1(ZEROS ? a.zeros + first_row[kParts - 1] * a.groups : nullptr, ZEROS ? (int64_t)rows * a.groups : 0);
            const int64_t xrows = MODE == kOne ? min(a.M - m0, (int64_t)16 * MT) : 0;
            const Rows x(MODE == kOne ? a.X + (int64_t)m0 * a.K : a.X,
                         MODE == kOne ? xrows * a.K * 2
                                      : (int64_t)(a.per_pair ? a.pairs : a.pairs / (int)a.div_k.d) * a.K * 2);
            uint32_t xoff[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int m = t * 16 + ln;
                if constexpr (MODE == kOne) {
                    xoff[t] = (uint32_t)m * a.K * 2;                     // rows past the end lie past the buffer
                    if (m >= xrows) xoff[t] = x.bytes;
                } else {
                    xoff[t] = x.bytes;
                    if (m0 + m < ncols) {
                        const int p = cols[m0 + m];
                        xoff[t] = (uint32_t)(a.per_pair ? p : (int)fast_div(p, a.div_k)) * a.K * 2;
                    }
                }
            }

            struct Slot {
                v4u w[RN];
                uint32_t s[RN][WIDE || MX ? (PER * SB + 3) / 4 : 4];
                uint32_t z[RN][WIDE ? 1 : 4];
                v4u x[MT][4];
            };
            Slot ring[PD];
            v4f acc[MT][RN];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int r = 0; r < RN; ++r) acc[t][r] = v4f{0.f, 0.f, 0.f, 0.f};

            auto load = [&](Slot& b, int step) {
                const int c0 = step * 4, cj = c0 + j;
#pragma unroll
                for (int r = 0; r < RN; ++r) {
                    const Rows& w = part(r) ? w1 : w0;
                    const uint32_t n = (uint32_t)((SWIGLU ? 0 : r * 16) + ln);
                    b.w[r] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
                        w.rsrc, cj < chunks ? (int)(n * row_bytes + cj * 16) : (int)w.bytes, 0, 0));
                }
#pragma unroll
                for (int r = 0; r < RN; ++r) {
                    const Rows& s = part(r) ? s1 : s0;
                    const Rows& z = part(r) ? z1 : z0;
                    const uint32_t n = (uint32_t)((SWIGLU ? 0 : r * 16) + ln);
                    if constexpr (WIDE) {
                        const bool in = c0 < chunks;
                        const int o = in ? (int)(n * group_row + step * PER * SB) : (int)s.bytes;
                        if constexpr (PER * SB == 8) {
                            const auto v = __builtin_amdgcn_raw_buffer_load_b64(s.rsrc, o, 0, 0);
                            b.s[r][0] = v[0];
                            b.s[r][1] = v[1];
                        } else if constexpr (PER * SB == 4) {
                            b.s[r][0] = __builtin_amdgcn_raw_buffer_load_b32(s.rsrc, o, 0, 0);
                        } else {
                            b.s[r][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(s.rsrc, o, 0, 0);
                        }
                        if constexpr (ZEROS) {
                            const int oz = in ? (int)(n * a.groups + step * PER) : (int)z.bytes;
                            if constexpr (PER == 4) b.z[r][0] = __builtin_amdgcn_raw_buffer_load_b32(z.rsrc, oz, 0, 0);
                            else if constexpr (PER == 2) b.z[r][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(z.rsrc, oz, 0, 0);
                            else b.z[r][0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(z.rsrc, oz, 0, 0);
                        }
                    } else if constexpr (MX) {
                        b.s[r][0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                            s.rsrc, cj < chunks ? (int)(n * group_row + cj) : (int)s.bytes, 0, 0);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool in = c0 + i < chunks;
                            const int gi = (c0 + i) / (GROUP / 32);
                            b.s[r][i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                                s.rsrc, in ? (int)(n * group_row + gi * SB) : (int)s.bytes, 0, 0);
                            if constexpr (ZEROS)
                                b.z[r][i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                                    z.rsrc, in ? (int)(n * a.groups + gi) : (int)z.bytes, 0, 0);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // values 8 i .. of chunk j (MXFP4), values 8 j .. of chunk i (INT4)
                        const int c = MX ? cj : c0 + i;
                        const int within = MX ? i * 16 : j * 16;
                        const bool in = c < chunks && xoff[t] < x.bytes;
                        b.x[t][i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
                            x.rsrc, in ? (int)(xoff[t] + c * 64 + within) : (int)x.bytes, 0, 0));
                    }
            };
            auto compute = [&](Slot& b) {
                if constexpr (MX) {
#pragma unroll
                    for (int r = 0; r < RN; ++r) {
                        const uint32_t s = WIDE ? (b.s[r][0] >> (8 * j)) & 0xFFu : b.s[r][0];
                        const float scale = __uint_as_float(s << 23);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const v4u w = decode_e2m1(b.w[r][i], scale);
#pragma unroll
                            for (int t = 0; t < MT; ++t) acc[t][r] = mfma_bf16(b.x[t][i], w, acc[t][r]);
                        }
                    }
                } else {
                    const v4u ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
                    const v4f none = {0.f, 0.f, 0.f, 0.f};
                    constexpr int CPG = GROUP / 32;    // chunks per group
                    v4f sum[MT][PER];
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            b.x[t][i] = order_u4(b.x[t][i]);
                            sum[t][i / CPG] = mfma_bf16(b.x[t][i], ones, i % CPG ? sum[t][i / CPG] : none);
                        }
#pragma unroll
                    for (int r = 0; r < RN; ++r) {
                        transpose4(b.w[r]);
                        v4f g[MT];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const v4u w = decode_u4(b.w[r][i]);
#pragma unroll
                            for (int t = 0; t < MT; ++t) g[t] = mfma_bf16(b.x[t][i], w, i % CPG ? g[t] : none);
                            if (i % CPG != CPG - 1) continue;
                            const int gi = i / CPG;
                            uint32_t s, z = 8;
                            if constexpr (WIDE) {
                                s = gi % 2 ? b.s[r][gi / 2] & 0xFFFF0000u : b.s[r][gi / 2] << 16;
                                if constexpr (ZEROS) z = (b.z[r][0] >> (8 * gi)) & 0xFFu;
                            } else {
                                s = b.s[r][i] << 16;
                                if constexpr (ZEROS) z = b.z[r][i];
                            }
                            const float scale = __uint_as_float(s), shift = -(16.0f + (float)z);
#pragma unroll
                            for (int t = 0; t < MT; ++t)
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    acc[t][r][q] = __builtin_fmaf(scale, __builtin_fmaf(shift, sum[t][gi][q], g[t][q]), acc[t][r][q]);
                        }
                    }
                }
            };

            // steps past the end read zeros (a step's loads are past the buffers), so the ring
            // needs no other end than the count
            const int mine = (steps - wave + kWaves - 1) / kWaves;
#pragma unroll
            for (int u = 0; u < PD; ++u) load(ring[u], wave + u * kWaves);
            for (int i = 0; i < mine; i += PD) {
#pragma unroll
                for (int u = 0; u < PD; ++u) {
                    compute(ring[u]);
                    load(ring[u], wave + (i + u + PD) * kWaves);
                    // keep the slots apart: interleaving them costs the registers that waves need
                    __builtin_amdgcn_sched_barrier(0);
                }
            }

            // the waves' sums, added in wave order
#pragma unroll
            for (int b0 = 0; b0 < RN * MT; b0 += kBatch) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b) red[wave][b][lane] = acc[(b0 + b) / RN][(b0 + b) % RN];
                __syncthreads();
                for (int o = tid; o < (SWIGLU ? 256 : kBatch * 256); o += kW4Threads) {
                    const int b = o >> 8, n = o & 15, m = (o >> 4) & 15;
                    auto total = [&](int tile) {
                        float v = 0.0f;
#pragma unroll
                        for (int w = 0; w < kWaves; ++w) v += red[w][tile][(m >> 2) * 16 + n][m & 3];
                        return v;
                    };
                    float v;
                    if constexpr (SWIGLU) {
                        const float gate = total(0), up = total(kBatch - 1);
                        v = gate * __builtin_amdgcn_rcpf(1.0f + exp_f32(-gate)) * up;
                    } else {
                        v = total(b);
                    }
                    const int t = (b0 + b) / RN, r = SWIGLU ? 0 : (b0 + b) % RN;
                    const int nn = n0 + r * 16 + n, mm = m0 + t * 16 + m;
                    if (nn < n_end && (MODE == kOne ? mm < a.M : mm < ncols)) {
                        const int64_t row = MODE == kOne ? mm : cols[mm];
                        a.Y[row * a.nout + nn] = f32_to_bf16(v);
                    }
                }
                __syncthreads();
            }
            if constexpr (MODE == kOne) break;
        }
        if constexpr (MODE != kOne) __syncthreads();   // the next window resets the list
        window += kW4MaxPairsBySlot;
    } while (MODE != kOne && !a.by_slot && window < a.pairs);
}

template <int RN, int MT, int PD, int MODE, bool Z>
void launch_int4(const W4Args& a, int group, bool wide, dim3 grid, hipStream_t s) {
    const dim3 block(kW4Threads);
    if (group == 32 && wide) hipLaunchKernelGGL((w4_kernel<32, false, true, Z, RN, MT, PD, MODE>), grid, block, 0, s, a);
    else if (group == 32) hipLaunchKernelGGL((w4_kernel<32, false, false, Z, RN, MT, PD, MODE>), grid, block, 0, s, a);
    else if (group == 64 && wide) hipLaunchKernelGGL((w4_kernel<64, false, true, Z, RN, MT, PD, MODE>), grid, block, 0, s, a);
    else if (group == 64) hipLaunchKernelGGL((w4_kernel<64, false, false, Z, RN, MT, PD, MODE>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((w4_kernel<128, false, true, Z, RN, MT, PD, MODE>), grid, block, 0, s, a);
}

template <int RN, int MT, int PD, int MODE>
void launch_mode(const W4Args& a, int group, bool mxfp4, dim3 grid, hipStream_t s) {
    const dim3 block(kW4Threads);
    const bool wide = a.K % kStep == 0;
    if (mxfp4 && wide) hipLaunchKernelGGL((w4_kernel<32, true, true, false, RN, MT, PD, MODE>), grid, block, 0, s, a);
    else if (mxfp4) hipLaunchKernelGGL((w4_kernel<32, true, false, false, RN, MT, PD, MODE>), grid, block, 0, s, a);
    else if (a.zeros) launch_int4<RN, MT, PD, MODE, true>(a, group, wide, grid, s);
    else launch_int4<RN, MT, PD, MODE, false>(a, group, wide, grid, s);
}

}  // namespace

void launch_w4(const W4Args& a, int group, bool mxfp4, int, hipStream_t s) {
    auto grid = [&](int rn, int mt) {
        return dim3((unsigned)((a.N + 16 * rn - 1) / (16 * rn)), (unsigned)((a.M + 16 * mt - 1) / (16 * mt)));
    };
    if (a.M <= 16) launch_mode<1, 1, 4, kOne>(a, group, mxfp4, grid(1, 1), s);
    else launch_mode<2, 2, 2, kOne>(a, group, mxfp4, grid(2, 2), s);
}

void launch_w4_experts(const W4Args& a, int group, bool mxfp4, bool swiglu, int, hipStream_t s) {
    const unsigned slots = a.by_slot ? a.pairs : a.E + 1;
    if (swiglu) launch_mode<2, 1, 2, kExpertsSwiglu>(a, group, mxfp4, dim3((unsigned)((a.half + 15) / 16), slots), s);
    else launch_mode<1, 1, 4, kExperts>(a, group, mxfp4, dim3((unsigned)((a.N + 15) / 16), slots), s);
}

}  // namespace fp8gemm
