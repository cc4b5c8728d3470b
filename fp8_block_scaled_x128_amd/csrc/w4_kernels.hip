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
// A workgroup owns 16 RN rows of V and all of K.  Its waves take pairs of steps (a step is 128
// values of K, 64 bytes of a row; a pair is one 128-byte line) in turn, each with all RN row
// tiles, and keep PP pairs in registers on their way, up to 64 KB per workgroup of 8 waves.  X's
// values stand in LDS, all of them or by chunks: read from the caches step by step by the lanes that
// need them they cost 27.8 us for 13 x 7168 x 16384 (MXFP4), from LDS 22.  The waves' fp32 sums
// meet in LDS and are added in wave order.  Splitting K over workgroups was measured and dropped:
// the exchange of sums costs 2 us, more than the idle CUs of a small matrix do.
//
// 1 x 32768 x 7168 MXFP4 24 us, 5.2 TB/s; 1 x 4096 x 7168 INT4 in 128s 7.6 us, a launch, the way of X into
// LDS and the exchange of sums around 3.1 us of weights; 13 x 7168 x 16384 MXFP4 22 us: 224 workgroups on
// 256 CUs, and 98 MB of X through L2 into their LDS beside 66 from HBM; 8 experts' 4096 x 7168 for a token,
// MXFP4 with SwiGLU, 28 us, 4.5 TB/s; 128 pairs of 7168 x 2048 on 64 experts, INT4 in 64s with zero points,
// 107 us, 4.2 TB/s, its decoding 5 lane operations a weight.
//
// In a step lane (n, j) = (lane % 16, lane / 16) loads 16 bytes of row n: its chunk j of 32 values.
//   MXFP4: the lane decodes its 32 values with their scale in the conversion instruction (two
//   values each, exact in bf16); matrix-core step i takes the values 8 i .. 8 i + 7 of all four
//   lanes.
//   INT4: the sums of different groups have to stay apart until they are scaled.  Two lane swaps
//   transpose the words across the four lanes of a row, so that matrix-core step i takes 32
//   consecutive values.  Codes become the bf16 values 16 + q by inserting them below the
//   exponent of 16 (exact); the group's sum is then (sum - (16 + z) sum_k x) * scale in fp32, with
//   sum_k x from one more matrix-core step against ones.  An infinite x, or |x| near the end of the type, makes
//   the two sums cancel to NaN or pass fp32's range where sum x (q - z) does not: an output that is not finite
//   is formed once more, from q - z (a test of each output; nothing else where all are finite: 13 x 7168 x
//   16384 in 128s takes 25 us, 233 with an infinity in one row, 886 with NaN throughout).

#include <algorithm>
#include <type_traits>

#include "fp8gemm_device.h"
#include "fp8gemm_internal.h"
#include "moe_device.h"
#include "moe_internal.h"

namespace fp8gemm {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kStep = 128;                 // K values per wave and step: four runs of 32

// X past this many bytes stands in LDS by chunks of kXSteps steps x rows (256 bytes each).  64 KB chunks leave
// room for a second workgroup on the CU, which hides the chunk's change; INT4 in groups of 32 and 64 has too
// few registers for that beside X's values on their way, and takes 128 KB.  Measured, 64 and 128 KB, us:
// MXFP4 12 x 16384 x 4096 12.1 and 16.3, 16 x 32768 x 7168 38.4 and 42.5, 13 x 7168 x 16384 22.8 and 23.6;
// INT4 in 128s 12 x 16384 x 4096 13.8 and 19.2, but in 32s 20.1 and 11.4 for 16 x 7168 x 4096 (spills).
template <int GROUP, bool MX>
constexpr int kXSteps = MX || GROUP == 128 ? 256 : 512;
template <int GROUP, bool MX>
constexpr int kXBytes = MX || GROUP == 128 ? 76 * 1024 : 130 * 1024;

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
// A row of X times a row of codes as the definition has it, q - z first, by a wave: a lane's groups are
// `lane`, lane + 64, ..., and the lanes' sums are added.
template <int GROUP, bool ZEROS>
__device__ __forceinline__ float dot_u4(const uint16_t* x, const uint8_t* w, const uint16_t* scales, const uint8_t* zeros,
                                        int groups, int lane) {
    float acc = 0.0f;
#pragma unroll 1
    for (int g = lane; g < groups; g += 64) {
        const float z = ZEROS ? (float)zeros[g] : 8.0f;
        float sum = 0.0f;
#pragma unroll 1
        for (int k = g * GROUP; k < (g + 1) * GROUP; k += 8) {
            const uint32_t q = *reinterpret_cast<const uint32_t*>(w + k / 2);
            const v4u v = *reinterpret_cast<const v4u*>(x + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum = __builtin_fmaf(__uint_as_float(v[i] << 16), (float)((q >> (8 * i)) & 15u) - z, sum);
                sum = __builtin_fmaf(__uint_as_float(v[i] & 0xFFFF0000u), (float)((q >> (8 * i + 4)) & 15u) - z, sum);
            }
        }
        acc = __builtin_fmaf(bf16_to_f32(scales[g]), sum, acc);
    }
    acc = row16_sum_f(acc);
    acc += __shfl_xor(acc, 16, 64);
    return acc + __shfl_xor(acc, 32, 64);
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

// `bytes` bytes at p, a buffer: reads past them give 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, kBufferFlags);
}

// Workgroup barrier that orders LDS traffic only: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// GROUP: values per scale; MX: MXFP4; PAIR: a pair's scales (and zero points) are adjacent and aligned, one
// load each, else each lane loads its own (MXFP4) or a part for the lanes of its row (INT4; in K with whole
// pairs that takes 36 us for 1 x 32768 x 7168 in groups of 64, against 33); RN: 16-row tiles of V; PP: pairs of
// steps in flight per wave; ALONE: a wave has all of K of its tiles, else the workgroup's waves share a tile's K;
// MULTI: X stands in LDS by chunks; MODE: see Mode (with SwiGLU tile 0 holds gate rows and tile 1 the matching
// up rows).
template <int GROUP, bool MX, bool PAIR, bool ZEROS, int RN, int PP, bool ALONE, bool MULTI, int MODE>
__global__ __launch_bounds__(kThreads, (MULTI && kXSteps<GROUP, MX> == 512 ? 2 : 4)) void w4_kernel(W4Args a) {
    constexpr int PER = kStep / GROUP;             // scales per step
    constexpr int SBYTES = 2 * PER * (MX ? 1 : 2); // bytes of a pair's scales
    constexpr bool SWIGLU = MODE == kExpertsSwiglu;
    constexpr int SHARE = ALONE ? 1 : kWaves;      // waves that share a tile's K
    constexpr int CS = SHARE * PP * 2;             // steps per round of the ring
    static_assert(!(ALONE && MULTI), "waves of their own pass over X at their own pace");
    // X's rows [cols][xstride], then the waves' sums
    extern __shared__ v4u lds[];
    v4f(*red)[RN][64] = reinterpret_cast<v4f(*)[RN][64]>(lds);
    __shared__ int cols[MODE == kOne ? 1 : kW4MaxPairsBySlot];
    __shared__ int count, early;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ln = lane & 15, j = lane >> 4;
    constexpr int kTileRows = SWIGLU ? 16 : 16 * RN;
    const int n_end = SWIGLU ? a.half : a.N;
    // tiles of this workgroup
    const int per_wg = ALONE ? kWaves * a.tiles_per_wave : 1;
    const int tile0 = blockIdx.x * per_wg, tile_end = min(tile0 + per_wg, (n_end + kTileRows - 1) / kTileRows);

    int expert = 0;
    int window = 0;                                // experts: first pair of the scanned window
    do {
        int ncols = 0;
        if constexpr (MODE == kOne) {
            ncols = (int)min(a.M - (int64_t)blockIdx.y * 16, (int64_t)16);
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
                for (int p = tid; p < last; p += kThreads) {
                    const int o = a.ids[window + p];
                    const bool outside = o < a.first || (int64_t)o - a.first >= a.E;
                    if (none ? outside : o == id && !outside) {
                        cols[atomicAdd(&count, 1)] = window + p;
                        if (a.by_slot && p < slot) early = 1;   // an earlier pair's workgroup has them all
                    }
                }
            }
            __syncthreads();
            ncols = __builtin_amdgcn_readfirstlane(a.by_slot && early ? 0 : count);
            expert = __builtin_amdgcn_readfirstlane(none ? -1 : id - a.first);
            if (expert < 0) {                      // pairs without an expert here: zero rows
                const int width = min(tile_end * kTileRows, a.nout) - tile0 * kTileRows;
                for (int i = tid; i < ncols * width; i += kThreads)
                    a.Y[(int64_t)cols[i / width] * a.nout + tile0 * kTileRows + i % width] = 0;
                ncols = 0;
            }
        }
        const int row_bytes = a.K / 2;
        const int units32 = a.K / 32, steps = (units32 + 3) / 4;
        const int group_row = a.groups * (MX ? 1 : 2);
        // a row tile is a buffer of weights, one of scales and one of zero points (with SwiGLU tile 0 holds
        // the gate rows, tile 1 the up rows); a lane's offsets in them
        const int64_t matrix = (int64_t)max(expert, 0) * a.N;
        const int vw = ln * row_bytes + j * 16, vs = ln * group_row, vz = ln * a.groups;
        auto tile_row = [&](int n0, int r) { return matrix + n0 + (SWIGLU ? r * a.half : r * 16); };
        auto tile_rows = [&](int n0, int r) { return max(0, min(16, n_end - n0 - (SWIGLU ? 0 : r * 16))); };

        for (int m0 = 0; m0 < ncols; m0 += a.cols) {     // kOne: once
            const int here = min(ncols - m0, a.cols);

            // registers of a pair's scales; without PAIR INT4's are spread over the four lanes of a row, lane j
            // having group j of the pair (of a step in groups of 32, group j % 2 in groups of 128)
            constexpr int SREGS = PAIR ? (SBYTES + 3) / 4 : MX || GROUP == 32 ? 2 : 1;
            constexpr int ZREGS = !ZEROS ? 1 : PAIR ? (2 * PER + 3) / 4 : SREGS;
            struct Slot {
                v4u w[2][RN];
                uint32_t s[RN][SREGS], z[RN][ZREGS];
            };
            Slot ring[PP];
            v4f acc[RN];

            // Loads of the pair of steps from `step` (even) of the tile from row n0.  A step past the end, or a
            // tile past the last row, reads an empty buffer; a step's offset is uniform and stays inside a row.
            auto load = [&](Slot& b, int step, int n0) {
#pragma unroll
                for (int r = 0; r < RN; ++r) {
                    const int n = step < steps ? tile_rows(n0, r) : 0, n1 = step + 1 < steps ? tile_rows(n0, r) : 0;
                    const uint8_t* w = a.W + tile_row(n0, r) * row_bytes;
                    b.w[0][r] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
                        buffer(w, n * row_bytes), vw, n ? step * 64 : 0, 0));
                    b.w[1][r] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
                        buffer(w, n1 * row_bytes), vw, n1 ? step * 64 + 64 : 0, 0));
                }
#pragma unroll
                for (int r = 0; r < RN; ++r) {
                    const int n = step < steps ? tile_rows(n0, r) : 0;
                    const uint8_t* sp = static_cast<const uint8_t*>(a.scales) + tile_row(n0, r) * group_row;
                    const uint8_t* zp = ZEROS ? a.zeros + tile_row(n0, r) * a.groups : nullptr;
                    if constexpr (PAIR) {
                        const auto s = buffer(sp, n * group_row);
                        const int so = n ? step / 2 * SBYTES : 0, zo = n ? step * PER : 0;
                        if constexpr (SBYTES == 16) {
                            const auto v = __builtin_amdgcn_raw_buffer_load_b128(s, vs, so, 0);
#pragma unroll
                            for (int i = 0; i < 4; ++i) b.s[r][i] = v[i];
                        } else if constexpr (SBYTES == 8) {
                            const auto v = __builtin_amdgcn_raw_buffer_load_b64(s, vs, so, 0);
                            b.s[r][0] = v[0];
                            b.s[r][1] = v[1];
                        } else {
                            b.s[r][0] = __builtin_amdgcn_raw_buffer_load_b32(s, vs, so, 0);
                        }
                        if constexpr (ZEROS) {
                            const auto z = buffer(zp, n * a.groups);
                            if constexpr (PER == 4) {
                                const auto v = __builtin_amdgcn_raw_buffer_load_b64(z, vz, zo, 0);
                                b.z[r][0] = v[0];
                                b.z[r][1] = v[1];
                            } else if constexpr (PER == 2) {
                                b.z[r][0] = __builtin_amdgcn_raw_buffer_load_b32(z, vz, zo, 0);
                            } else {
                                b.z[r][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(z, vz, zo, 0);
                            }
                        }
                    } else if constexpr (MX) {
                        // a lane's own scale; past the end of the row (where the next row's stand) 0
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int g = (step + i) * 4 + j;
                            b.s[r][i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                                buffer(sp, n * group_row), g < units32 ? vs + g : n * group_row, 0, 0);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < SREGS; ++i) {
                            // past the end of the row (where the next row's stand) 0
                            const int g = step * PER + i * 4, mine = GROUP == 128 ? j & 1 : j;
                            const bool in = mine < a.groups - g;
                            b.s[r][i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                                buffer(sp, n * group_row), in ? vs + mine * 2 : n * group_row, n ? g * 2 : 0, 0);
                            if constexpr (ZEROS)
                                b.z[r][i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                                    buffer(zp, n * a.groups), in ? vz + mine : n * a.groups, n ? g : 0, 0);
                        }
                    }
                }
            };

            // X's values of a chunk of steps in LDS, 16 bytes a thread and unit, zeros past K; INT4 keeps them
            // in the order of the decoded codes
            const int chunk = a.xsteps;                  // whole rounds of the ring
            const int row_units = chunk * (kStep / 8), xrow = a.xstride / 16;
            const auto xbuf = buffer(MODE == kOne ? a.X + (int64_t)blockIdx.y * 16 * a.K : a.X,
                                     MODE == kOne ? ncols * a.K * 2 : a.xrows * a.K * 2);
            constexpr int XU = MULTI ? kXSteps<GROUP, MX> * 16 / kThreads : 2;   // units a thread moves at a time (MULTI: the chunk)
            v4u xv[XU];
            auto fetch = [&](int first_step, int u0) {
#pragma unroll
                for (int i = 0; i < XU; ++i) {
                    const int u = u0 + i * kThreads, c = (int)fast_div(u, a.div_units), q = u - c * row_units;
                    const int k = first_step * kStep + q * 8;
                    int o = -16;                         // past the buffer (unsigned)
                    if (c < here && k < a.K) {
                        int row = c;
                        if constexpr (MODE != kOne) {
                            const int p = cols[m0 + c];
                            row = a.per_pair ? p : (int)fast_div(p, a.div_k);
                        }
                        o = (row * a.K + k) * 2;
                    }
                    xv[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(xbuf, o, 0, 0));
                }
            };
            auto stage = [&](int u0) {
#pragma unroll
                for (int i = 0; i < XU; ++i) {
                    const int u = u0 + i * kThreads, c = (int)fast_div(u, a.div_units), q = u - c * row_units;
                    if (c < here) lds[c * xrow + q] = MX ? xv[i] : order_u4(xv[i]);
                }
            };
            // (opaque: nothing derived from it is worth registers across the products)
            auto thread = [&]() {
                int u = tid;
                asm volatile("" : "+v"(u));
                return u;
            };

            // a lane's values of its row of X (rows past the last repeat it: their results are not used)
            const int xl = min(ln, here - 1) * xrow + (MX ? j * 4 : j);
            // step `sl` of the chunk, the h-th of the slot's pair
            auto compute = [&](Slot& b, int h, int sl) {
                v4u x[4];
#pragma unroll
                // values 8 i .. of lane j's 32 (MXFP4), values 8 j .. of the i-th 32 (INT4)
                for (int i = 0; i < 4; ++i) x[i] = lds[xl + sl * 16 + (MX ? i : i * 4)];
                if constexpr (MX) {
#pragma unroll
                    for (int r = 0; r < RN; ++r) {
                        const uint32_t s = PAIR ? (b.s[r][h] >> (8 * j)) & 0xFFu : b.s[r][h];
                        const float scale = __uint_as_float(s << 23);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[r] = mfma_bf16(x[i], decode_e2m1(b.w[h][r][i], scale), acc[r]);
                    }
                } else {
                    const v4u ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
                    const v4f none = {0.f, 0.f, 0.f, 0.f};
                    constexpr int CPG = GROUP / 32;    // matrix-core steps per group
                    v4f sum[PER];
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i / CPG] = mfma_bf16(x[i], ones, i % CPG ? sum[i / CPG] : none);
#pragma unroll
                    for (int r = 0; r < RN; ++r) {
                        v4u wt = b.w[h][r];
                        transpose4(wt);
                        // the step's scales (and zero points below them) from the lanes that hold them
                        uint32_t sz[4];
                        if constexpr (!PAIR) {
                            const uint32_t mine = b.s[r][SREGS == 2 ? h : 0] << 16 | (ZEROS ? b.z[r][SREGS == 2 ? h : 0] : 8u);
                            auto low = [](uint32_t v, uint32_t* o) {     // of lanes j = 0 and 1, or of 2 and 3
                                auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
                                o[0] = p[0];
                                o[1] = p[1];
                            };
                            if constexpr (GROUP == 128) {
                                low(mine, sz);                           // the pair's two groups
                                sz[0] = sz[h];
                            } else {
                                auto p = __builtin_amdgcn_permlane32_swap(mine, mine, false, false);
                                if constexpr (GROUP == 64) low(p[h], sz);
                                else low(p[0], sz), low(p[1], sz + 2);
                            }
                        }
                        v4f g;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            g = mfma_bf16(x[i], decode_u4(wt[i]), i % CPG ? g : none);
                            if (i % CPG != CPG - 1) continue;
                            const int gi = h * PER + i / CPG;      // group within the pair
                            uint32_t s, z = 8;
                            if constexpr (PAIR) {
                                s = gi % 2 ? b.s[r][gi / 2] & 0xFFFF0000u : b.s[r][gi / 2] << 16;
                                if constexpr (ZEROS) z = (b.z[r][gi / 4] >> (8 * (gi % 4))) & 0xFFu;
                            } else {
                                s = sz[i / CPG] & 0xFFFF0000u;
                                if constexpr (ZEROS) z = sz[i / CPG] & 0xFFu;
                            }
                            const float scale = __uint_as_float(s), shift = -(16.0f + (float)z);
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                acc[r][q] = __builtin_fmaf(scale, __builtin_fmaf(shift, sum[i / CPG][q], g[q]), acc[r][q]);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);       // interleaving steps costs registers that waves need
            };

            // Rounds of the ring: it is refilled pair by pair for the next round, or the wave's next tile.
            // Where X takes several chunks, the next one's values are asked for ahead of the last refills of
            // the present one, so that waiting for them does not empty the ring.
            auto pair_step = [&](int u) { return (ALONE ? u : u * kWaves + wave) * 2; };
            int tile = ALONE ? tile0 + wave : tile0;
            int u0 = thread();
            fetch(0, u0);
#pragma unroll
            for (int u = 0; u < PP; ++u) load(ring[u], pair_step(u), min(tile, tile_end) * kTileRows);
            stage(u0);
            if constexpr (!MULTI)
                for (u0 += XU * kThreads; u0 < here * row_units; u0 += XU * kThreads) {
                    fetch(0, u0);
                    stage(u0);
                }
            lds_barrier();
            int first = 0;                               // step of the chunk in LDS
            for (; tile < tile_end; tile += kWaves) {
                const int n0 = tile * kTileRows;
#pragma unroll
                for (int r = 0; r < RN; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
                // (whole rounds, a chunk's last and the tile's last stand apart, each free of the others' conditions:
                // fewer registers, and waits for no more loads than are needed)
                int base = 0;
                auto whole_round = [&]() {
#pragma unroll
                    for (int u = 0; u < PP; ++u) {
                        const int step = base + pair_step(u);
                        compute(ring[u], 0, step - first);
                        compute(ring[u], 1, step + 1 - first);
                        load(ring[u], step + CS, n0);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                };
                if constexpr (MULTI) {
                    for (; first + chunk < steps; first = base) {
                        for (; base + CS < first + chunk; base += CS) whole_round();
                        fetch(base + CS, thread());
                        __builtin_amdgcn_sched_barrier(0);
                        whole_round();
                        base += CS;
                        lds_barrier();                   // the chunk has been read
                        stage(thread());
                        lds_barrier();
                    }
                }
                for (; base + CS < steps; base += CS) whole_round();
                auto last_round = [&](auto refill) {
#pragma unroll
                    for (int u = 0; u < PP; ++u) {
                        const int step = base + pair_step(u);
                        if (step < steps) compute(ring[u], 0, step - first);
                        if (step + 1 < steps) compute(ring[u], 1, step + 1 - first);
                        if constexpr (refill.value) {
                            load(ring[u], pair_step(u), n0 + kWaves * kTileRows);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                };
                if (ALONE && tile + kWaves < tile_end) last_round(std::true_type());
                else last_round(std::false_type());

                // output (m, n) of this lane, if it has one (called by whole waves)
                auto finish = [&](bool there, int m, int n, float v, float up) {
                    if constexpr (!MX) {
                        auto wild = [](float f) { return !(__builtin_fabsf(f) < __builtin_inff()); };
                        for (uint64_t b = __ballot(there && (wild(v) || (SWIGLU && wild(up)))); b; b &= b - 1) {
                            const int from = __builtin_ctzll(b), mf = __builtin_amdgcn_readlane(m, from);
                            int64_t row = (int64_t)blockIdx.y * 16 + mf;
                            if constexpr (MODE != kOne) {
                                const int p = cols[m0 + mf];
                                row = a.per_pair ? p : (int)fast_div(p, a.div_k);
                            }
#pragma unroll 1
                            for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
                                const int64_t at = matrix + n0 + __builtin_amdgcn_readlane(n, from) + h * a.half;
                                const float d = dot_u4<GROUP, ZEROS>(a.X + row * a.K, a.W + at * row_bytes,
                                                                     static_cast<const uint16_t*>(a.scales) + at * a.groups,
                                                                     ZEROS ? a.zeros + at * a.groups : nullptr, a.groups, lane);
                                if (lane == from) (h ? up : v) = d;
                            }
                        }
                    }
                    if (!there) return;
                    if constexpr (SWIGLU) v = v * __builtin_amdgcn_rcpf(1.0f + exp_f32(-v)) * up;
                    const int64_t row = MODE == kOne ? (int64_t)blockIdx.y * 16 + m : cols[m0 + m];
                    a.Y[row * a.nout + n0 + n] = f32_to_bf16(v);
                };
                if constexpr (ALONE) {
#pragma unroll
                    for (int r = 0; r < (SWIGLU ? 1 : RN); ++r)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            finish(j * 4 + q < here && n0 + r * 16 + ln < n_end, j * 4 + q, r * 16 + ln, acc[r][q],
                                   acc[RN - 1][q]);
                } else {
                    // the waves' sums, added in wave order
                    lds_barrier();
#pragma unroll
                    for (int r = 0; r < RN; ++r)
                        if (j * 4 < here) red[wave][r][lane] = acc[r];
                    lds_barrier();
                    for (int o = thread(); o < kTileRows * 16; o += kThreads) {
                        const int n = o % kTileRows, m = o / kTileRows;
                        const bool there = n0 + n < n_end && m < here;
                        auto total = [&](int r) {
                            float v = 0.0f;
                            if (!there) return v;
#pragma unroll
                            for (int w = 0; w < kWaves; ++w) v += red[w][r][(m >> 2) * 16 + (n & 15)][m & 3];
                            return v;
                        };
                        finish(there, m, n, total(SWIGLU ? 0 : n >> 4), SWIGLU ? total(1) : 0.0f);
                    }
                    break;                               // one tile
                }
            }
            if constexpr (MODE == kOne) break;
            __syncthreads();                             // LDS and the list are used again
        }
        if constexpr (MODE != kOne) __syncthreads();
        window += kW4MaxPairsBySlot;
    } while (MODE != kOne && !a.by_slot && window < a.pairs);
}

// Workgroups over tiles of V and rows of X (or pairs, or experts).
template <int GROUP, bool MX, bool PAIR, bool Z, int RN, int PP, bool ALONE, int MODE>
void launch_one(W4Args a, unsigned y, hipStream_t s) {
    constexpr int tile_rows = MODE == kExpertsSwiglu ? 16 : 16 * RN;
    const int steps = (a.K + kStep - 1) / kStep;
    const int tiles = (a.nout + tile_rows - 1) / tile_rows, per_wg = ALONE ? kWaves * a.tiles_per_wave : 1;
    const dim3 grid((unsigned)((tiles + per_wg - 1) / per_wg), y), block(kThreads);
    const size_t red = ALONE ? 0 : (size_t)kWaves * RN * 64 * sizeof(v4f);
    auto lds = [&](int xsteps) {
        a.xsteps = xsteps;
        a.xstride = xsteps * kStep * 2 + 16;         // rows 16 bytes apart in the banks
        a.div_units = make_fastdiv((uint32_t)(xsteps * (kStep / 8)));
        return std::max((size_t)a.cols * a.xstride, red);
    };
    if constexpr (!ALONE) {
        if (a.cols * (steps * kStep * 2 + 16) > kXBytes<GROUP, MX>) {
            // pairs in flight: what registers hold beside X's values on their way, and a chunk of 16 rows holds
            constexpr int X = kXSteps<GROUP, MX>, FEW = MX ? PP : (PP + 1) / 2, MANY = std::min(PP, X / 256);
            auto go = [&](auto pm) {
                constexpr int round = kWaves * pm.value * 2;
                const size_t bytes = lds(X / a.cols / round * round);
                hipLaunchKernelGGL((w4_kernel<GROUP, MX, PAIR, Z, RN, pm.value, ALONE, true, MODE>), grid, block, bytes, s, a);
            };
            static_assert(X / 4 >= kWaves * FEW * 2 && X / 16 >= kWaves * MANY * 2, "X's chunk has room for a round");
            if constexpr (RN == 1) {
                if (a.cols <= 4) {
                    go(std::integral_constant<int, FEW>());
                    return;
                }
            }
            go(std::integral_constant<int, MANY>());
            return;
        }
    }
    const size_t bytes = lds(steps);
    hipLaunchKernelGGL((w4_kernel<GROUP, MX, PAIR, Z, RN, PP, ALONE, false, MODE>), grid, block, bytes, s, a);
}

// The scales of groups of 32 take more registers, which leaves room for fewer pairs in flight.
template <int RN, int PP, bool ALONE, int MODE, bool Z>
void launch_int4(const W4Args& a, int group, unsigned y, hipStream_t s) {
    constexpr int PH = (PP + 1) / 2;
    // a pair's scales are 16, 8 or 4 bytes, its zero points 8, 4 or 2, at that many bytes' alignment (at most 4)
    const bool pair = a.K % (group == 32 || (group == 64 && !Z) ? 128 : 256) == 0;
    if (group == 32 && pair) launch_one<32, false, true, Z, RN, PH, ALONE, MODE>(a, y, s);
    else if (group == 32) launch_one<32, false, false, Z, RN, (PP == 4 ? 3 : 1), ALONE, MODE>(a, y, s);
    else if (group == 64 && pair) launch_one<64, false, true, Z, RN, PP, ALONE, MODE>(a, y, s);
    else if (group == 64) launch_one<64, false, false, Z, RN, PP, ALONE, MODE>(a, y, s);
    else if (pair) launch_one<128, false, true, Z, RN, PP, ALONE, MODE>(a, y, s);
    else launch_one<128, false, false, Z, RN, PP, ALONE, MODE>(a, y, s);
}

// PP: pairs in flight of MXFP4, PI of INT4.
template <int RN, int PP, int PI, bool ALONE, int MODE>
void launch_mode(const W4Args& a, int group, bool mxfp4, unsigned y, hipStream_t s) {
    if (mxfp4 && a.K % kStep == 0) launch_one<32, true, true, false, RN, PP, ALONE, MODE>(a, y, s);
    else if (mxfp4) launch_one<32, true, false, false, RN, PP, ALONE, MODE>(a, y, s);
    else if (a.zeros) launch_int4<RN, PI, ALONE, MODE, true>(a, group, y, s);
    else launch_int4<RN, PI, ALONE, MODE, false>(a, group, y, s);
}

}  // namespace

void launch_w4(const W4Args& a, int rn, int group, bool mxfp4, hipStream_t s) {
    const unsigned y = (unsigned)((a.M + 15) / 16);
    if (a.tiles_per_wave > 0) launch_mode<1, 4, 4, true, kOne>(a, group, mxfp4, y, s);
    else if (rn == 1) launch_mode<1, 4, 4, false, kOne>(a, group, mxfp4, y, s);
    else launch_mode<2, 2, 2, false, kOne>(a, group, mxfp4, y, s);
}

// (INT4 with the experts' bookkeeping has registers for one pair in flight and two workgroups per CU: us, 8
// pairs of 4096 x 7168 with SwiGLU, groups of 64 with zero points, one pair 30.6, two 33.8)
void launch_w4_experts(const W4Args& a, int rn, int group, bool mxfp4, bool swiglu, hipStream_t s) {
    const unsigned y = a.by_slot ? a.pairs : a.E + 1;
    if (swiglu && a.tiles_per_wave > 0) launch_mode<2, 2, 2, true, kExpertsSwiglu>(a, group, mxfp4, y, s);
    else if (swiglu) launch_mode<2, 2, 1, false, kExpertsSwiglu>(a, group, mxfp4, y, s);
    else if (a.tiles_per_wave > 0) launch_mode<1, 4, 4, true, kExperts>(a, group, mxfp4, y, s);
    else if (rn == 1) launch_mode<1, 3, 2, false, kExperts>(a, group, mxfp4, y, s);
    else launch_mode<2, 2, 1, false, kExperts>(a, group, mxfp4, y, s);
}

}  // namespace fp8gemm
