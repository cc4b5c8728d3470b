// permute_kernels.hip -- gfx950 kernels that move rows between token order and expert order: the
// dispatch (each token's row, quantised to E4M3 with 1x128 scales, into the rows of its experts),
// the weighted combine back, and the combine's gradients.  The mathematics is stated in
// include/fp8gemm.h.
//
// The rank of a pair (token t, pick j) among its expert's rows is the number of earlier pairs, in
// (t, j) order, with the same expert, so the layout does not depend on timing.  Small batches
// recompute the ranks in every workgroup of the one copying launch; large ones count chunks of
// pairs, scan the counts and then copy, in three launches.

#include "fp8gemm_device.h"
#include "moe_device.h"
#include "moe_internal.h"

namespace fp8gemm {
namespace {

// Workgroup size and elements per thread of every row pass: 16 lanes own a 128-value block, as
// 16 bytes of bf16 per lane, so a wave's load is 1 KB of consecutive memory.
constexpr int kThreads = 256;
constexpr int kSpan = kThreads * 8;      // elements of a row one workgroup handles per pass

// Correctly rounded x / s for one E4M3 conversion: with r = RN(1/s) and q = RN(x r), one
// residual step gives RN(x / s) (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34(1), 1990); the sign is x's, so that -0 stays -0.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = x * r;
    return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, x), r, q), x);
}

// The 1x128 quantiser on 8 bf16 values of a lane (16 lanes a block): 8 codes and the scale.
__device__ __forceinline__ uint2 quantize8(const v4u& c, float* scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(c[i] & 0x7FFFu, (c[i] >> 16) & 0x7FFFu));
    // bit patterns of |x| order like the values
    m = max(m, (uint32_t)dpp16<kDppXor1>((int)m));
    m = max(m, (uint32_t)dpp16<kDppXor2>((int)m));
    m = max(m, (uint32_t)dpp16<kDppHalfMirror>((int)m));
    m = max(m, (uint32_t)dpp16<kDppMirror>((int)m));
    const float s = fmaxf(__uint_as_float(m << 16), 1e-4f) / 448.0f;
    const float r = 1.0f / s;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __builtin_amdgcn_fmed3f(quotient(__uint_as_float(c[i] << 16), s, r), -448.0f, 448.0f);
        v[2 * i + 1] = __builtin_amdgcn_fmed3f(quotient(__uint_as_float(c[i] & 0xFFFF0000u), s, r), -448.0f, 448.0f);
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    *scale = s;
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Local expert of a pair, or -1 (no pick, or another rank's expert).
__device__ __forceinline__ int local_expert(const DispatchArgs& a, int pair) {
    const int64_t id = (int64_t)a.ids[pair] - a.first;   // any int32 id and first stay in range
    return a.ids[pair] >= 0 && id >= 0 && id < a.G ? (int)id : -1;
}

__device__ __forceinline__ int padded(int n) { return (n + 127) & ~127; }

// Row of local expert e's rank-th pair, or -1 past the capacity; `first` is the expert's first
// row in the contiguous layout.
__device__ __forceinline__ int place(const DispatchArgs& a, int e, int rank, int64_t first) {
    const int64_t row = a.contiguous ? first + rank : (int64_t)e * a.cap + rank;
    return rank < a.cap && (!a.contiguous || row < a.cap) ? (int)row : -1;
}

// A thread's 8 values of span `s` of token t's row (asked for before the rows are known).
__device__ __forceinline__ v4u load_span(const DispatchArgs& a, int64_t t, int s) {
    const int col = s * kSpan + threadIdx.x * 8;
    return *reinterpret_cast<const v4u*>(a.X + t * a.H + min(col, a.H - 8));
}

// Quantise them and store them in the rows[0..k) that are not -1.
__device__ __forceinline__ void store_span(const DispatchArgs& a, int s, const v4u& c, const int* rows) {
    const int col = s * kSpan + threadIdx.x * 8;
    if (col >= a.H) return;              // the 16 lanes of a 128-value block leave together
    float scale;
    const uint2 q = quantize8(c, &scale);
    const int kb = col >> 7;
    for (int j = 0; j < a.k; ++j) {
        const int row = rows[j];
        if (row < 0) continue;
        *reinterpret_cast<uint2*>(a.A + (int64_t)row * a.H + col) = q;
        if ((threadIdx.x & 15) == 0) {
            const int e = a.contiguous ? 0 : row / a.cap;
            a.sa[((int64_t)e * a.nkb + kb) * a.cap + (row - (int64_t)e * a.cap)] = scale;
        }
    }
}

// m_indices of this token's share of the contiguous layout's rows: the expert whose rows [first,
// first + count) hold the row, or -1.
template <typename First, typename Count>
__device__ __forceinline__ void fill_indices(const DispatchArgs& a, int64_t t, First first, Count count) {
    const int64_t per = (a.cap + a.T - 1) / a.T;
    const int64_t end = min((t + 1) * per, (int64_t)a.cap);
    for (int64_t r = t * per + threadIdx.x; r < end; r += kThreads) {
        int lo = 0, hi = a.G;            // the last expert whose first row is not past r
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first(mid) <= r) lo = mid;
            else hi = mid;
        }
        a.where[r] = r - first(lo) < count(lo) ? lo : -1;
    }
}

// One launch: workgroup (t, s) counts every pair's expert, and those before token t, in LDS.
__global__ __launch_bounds__(kThreads) void dispatch_small_kernel(DispatchArgs a, int spans) {
    __shared__ int all[kDispatchMaxGroups], before[kDispatchMaxGroups];
    __shared__ int first[kDispatchMaxGroups + 1];
    __shared__ int rows[kDispatchMaxTopk], mine[kDispatchMaxTopk];
    const int64_t t = blockIdx.x / spans;
    const int s = blockIdx.x - (int)t * spans;
    const v4u c = load_span(a, t, s);
    for (int e = threadIdx.x; e < a.G; e += kThreads) all[e] = before[e] = 0;
    __syncthreads();
    const int p0 = (int)t * a.k;
    for (int p = threadIdx.x; p < a.pairs; p += kThreads) {
        const int e = local_expert(a, p);
        if (e >= 0) {
            atomicAdd(&all[e], 1);
            if (p < p0) atomicAdd(&before[e], 1);
        }
    }
    if (threadIdx.x < a.k) mine[threadIdx.x] = local_expert(a, p0 + threadIdx.x);
    __syncthreads();
    if (a.contiguous && threadIdx.x < 64) {   // first rows: a running sum over 64 experts at a time
        int carry = 0;
        for (int e0 = 0; e0 < a.G; e0 += 64) {
            const int e = e0 + threadIdx.x;
            const int n = e < a.G ? padded(all[e]) : 0;
            int sum = n;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(sum, o, 64);
                if ((int)threadIdx.x >= o) sum += up;
            }
            if (e < a.G) first[e] = carry + sum - n;
            carry += __shfl(sum, 63, 64);
        }
    }
    __syncthreads();
    if (threadIdx.x < a.k) {
        const int e = mine[threadIdx.x];
        int row = -1;
        if (e >= 0) {
            int rank = before[e];
            for (int j = 0; j < (int)threadIdx.x; ++j) rank += mine[j] == e;
            row = place(a, e, rank, a.contiguous ? first[e] : 0);
            if (row < 0 && s == 0) atomicOr(a.err, (int32_t)kDevErrBadCount);
        }
        rows[threadIdx.x] = row;
        if (s == 0) a.row_map[p0 + threadIdx.x] = row;
    }
    if (s == 0) {
        if (a.contiguous) {
            fill_indices(a, t, [&](int e) { return first[e]; }, [&](int e) { return all[e]; });
        } else if (t == 0) {
            for (int e = threadIdx.x; e < a.G; e += kThreads) a.where[e] = min(all[e], a.cap);
        }
    }
    __syncthreads();
    store_span(a, s, c, rows);
}

// Scratch of the large path, in words.
struct Scratch {
    int32_t* counts;   // [G][chunks]: pairs per chunk, then their exclusive sums over chunks
    int32_t* first;    // [G]: first row (contiguous)
    int32_t* total;    // [G]
    int32_t* local;    // [pairs]: rank within the chunk
};
__device__ __forceinline__ Scratch scratch_of(const DispatchArgs& a) {
    Scratch s;
    s.counts = a.scratch;
    s.first = s.counts + (int64_t)a.G * a.chunks;
    s.total = s.first + a.G;
    s.local = s.total + a.G;
    return s;
}

// Ranks within a chunk of kDispatchChunk pairs: each of the four waves takes 64 consecutive pairs
// at a time; lanes with the same expert find each other by one ballot per bit of the index.
__global__ __launch_bounds__(kThreads) void dispatch_count_kernel(DispatchArgs a) {
    constexpr int kWaves = kThreads / 64, kPerWave = kDispatchChunk / kWaves, kSteps = kPerWave / 64;
    __shared__ int hist[kWaves][kDispatchMaxGroups];
    const Scratch sc = scratch_of(a);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < a.G; e += kThreads)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) hist[w][e] = 0;
    __syncthreads();
    const int p0 = blockIdx.x * kDispatchChunk + wave * kPerWave + lane;
    const uint64_t below = (1ull << lane) - 1;
    int expert[kSteps], rank[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int p = p0 + i * 64;
        expert[i] = p < a.pairs ? local_expert(a, p) : -1;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int e = expert[i];
        uint64_t same = __ballot(e >= 0);
        for (int b = 1; b < a.G; b <<= 1) {
            const uint64_t set = __ballot((e & b) != 0);
            same &= (e & b) ? set : ~set;
        }
        rank[i] = 0;
        int had = 0;
        if (e >= 0) had = hist[wave][e];
        wave_sync();
        if (e >= 0) {
            rank[i] = had + __popcll(same & below);
            if ((same >> lane) == 1) hist[wave][e] = had + __popcll(same);   // the last lane of the expert
        }
        wave_sync();
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if (expert[i] < 0) continue;
        for (int w = 0; w < wave; ++w) rank[i] += hist[w][expert[i]];
        sc.local[p0 + i * 64] = rank[i];
    }
    for (int e = threadIdx.x; e < a.G; e += kThreads) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) n += hist[w][e];
        sc.counts[(int64_t)e * a.chunks + blockIdx.x] = n;
    }
}

// Exclusive sums of each expert's counts over the chunks, the experts' totals and first rows.
__global__ __launch_bounds__(1024) void dispatch_scan_kernel(DispatchArgs a) {
    __shared__ int total[kDispatchMaxGroups];
    const Scratch sc = scratch_of(a);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = wave; e < a.G; e += 16) {
        int carry = 0;
        int32_t* row = sc.counts + (int64_t)e * a.chunks;
        for (int c0 = 0; c0 < a.chunks; c0 += 64) {
            const int c = c0 + lane;
            const int n = c < a.chunks ? row[c] : 0;
            int sum = n;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(sum, o, 64);
                if (lane >= o) sum += up;
            }
            if (c < a.chunks) row[c] = carry + sum - n;
            carry += __shfl(sum, 63, 64);
        }
        if (lane == 0) total[e] = carry;
    }
    __syncthreads();
    if (wave == 0) {
        int64_t carry = 0;
        for (int e0 = 0; e0 < a.G; e0 += 64) {
            const int e = e0 + lane;
            const int n = e < a.G ? total[e] : 0;
            int sum = padded(n);
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(sum, o, 64);
                if (lane >= o) sum += up;
            }
            if (e < a.G) {
                // 2^31 rows and more lie past every capacity
                sc.first[e] = (int32_t)min(carry + sum - padded(n), (int64_t)0x7FFFFFFF);
                sc.total[e] = n;
                if (!a.contiguous) {
                    a.where[e] = min(n, a.cap);
                    if (n > a.cap) atomicOr(a.err, (int32_t)kDevErrBadCount);
                }
            }
            carry += __shfl(sum, 63, 64);
        }
    }
}

// No tokens: every expert has no rows, every row is padding.
__global__ __launch_bounds__(kThreads) void dispatch_empty_kernel(int32_t* where, int n, int32_t value) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i < n) where[i] = value;
}

__global__ __launch_bounds__(kThreads) void dispatch_copy_kernel(DispatchArgs a, int spans) {
    __shared__ int rows[kDispatchMaxTopk];
    const Scratch sc = scratch_of(a);
    const int64_t t = blockIdx.x / spans;
    const int s = (int)(blockIdx.x - t * spans);
    const v4u c = load_span(a, t, s);
    if (threadIdx.x < a.k) {
        const int p = (int)(t * a.k) + threadIdx.x;
        const int e = local_expert(a, p);
        int row = -1;
        if (e >= 0) {
            const int rank = sc.counts[(int64_t)e * a.chunks + p / kDispatchChunk] + sc.local[p];
            row = place(a, e, rank, sc.first[e]);
            if (row < 0 && s == 0) atomicOr(a.err, (int32_t)kDevErrBadCount);
        }
        rows[threadIdx.x] = row;
        if (s == 0) a.row_map[p] = row;
    }
    __syncthreads();
    if (s == 0 && a.contiguous)
        fill_indices(a, t, [&](int e) { return sc.first[e]; }, [&](int e) { return sc.total[e]; });
    store_span(a, s, c, rows);
}

// ---- combine ----

// Row of pair (t, j) in Y, or -1.
__device__ __forceinline__ int64_t pair_row(const CombineArgs& a, int64_t t, int j) {
    if (!a.row_map) return t * a.k + j;
    const int r = a.row_map[t * a.k + j];
    return r >= 0 && r < a.R ? r : -1;
}

// out[t] = sum_j w[t][j] Y[row(t, j)], in fp32 in the order of j.  Memory bound: each thread owns
// 16 bytes of the output and keeps the loads of several rows in flight.
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineArgs a, int spans) {
    const int64_t t = blockIdx.x / spans;
    const int s = (int)(blockIdx.x - t * spans);
    const int col = s * kSpan + threadIdx.x * 8;
    if (s == 0 && threadIdx.x < a.k && a.row_map && a.row_map[t * a.k + threadIdx.x] >= a.R)
        atomicOr(a.err, (int32_t)kDevErrBadIndex);
    if (col >= a.H) return;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    constexpr int kDeep = 4;
    for (int j0 = 0; j0 < a.k; j0 += kDeep) {
        v4u y[kDeep];
        float w[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            y[i] = v4u{0, 0, 0, 0};
            w[i] = 0.0f;
            if (j0 + i < a.k) {
                const int64_t r = pair_row(a, t, j0 + i);
                if (r >= 0) {
                    y[i] = *reinterpret_cast<const v4u*>(a.Y + r * a.H + col);
                    w[i] = a.weights ? a.weights[t * a.k + j0 + i] : 1.0f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                acc[2 * q] = __builtin_fmaf(w[i], __uint_as_float(y[i][q] << 16), acc[2 * q]);
                acc[2 * q + 1] = __builtin_fmaf(w[i], __uint_as_float(y[i][q] & 0xFFFF0000u), acc[2 * q + 1]);
            }
    }
    v4u o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(acc[2 * q], acc[2 * q + 1]);
    *reinterpret_cast<v4u*>(a.out + t * a.H + col) = o;
}

// dY[row(t, j)] = w[t][j] dout[t] and dw[t][j] = <dout[t], Y[row(t, j)]>: one workgroup per token
// passes over the row once for each kDeep picks, with the products' sums in registers.
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(CombineArgs a) {
    constexpr int kDeep = 8;
    __shared__ float part[kThreads / 64][kDeep];
    const int64_t t = blockIdx.x;
    if (threadIdx.x < a.k && a.row_map && a.row_map[t * a.k + threadIdx.x] >= a.R)
        atomicOr(a.err, (int32_t)kDevErrBadIndex);
    for (int j0 = 0; j0 < a.k; j0 += kDeep) {
        int64_t row[kDeep];
        float w[kDeep], dot[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            row[i] = j0 + i < a.k ? pair_row(a, t, j0 + i) : -1;
            w[i] = row[i] >= 0 && a.weights ? a.weights[t * a.k + j0 + i] : 1.0f;
            dot[i] = 0.0f;
        }
        for (int col = threadIdx.x * 8; col < a.H; col += kSpan) {
            const v4u d = *reinterpret_cast<const v4u*>(a.dout + t * a.H + col);
            v4u y[kDeep];
#pragma unroll
            for (int i = 0; i < kDeep; ++i)
                y[i] = a.dweights && row[i] >= 0 ? *reinterpret_cast<const v4u*>(a.Y + row[i] * a.H + col) : v4u{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                if (row[i] < 0) continue;
                v4u o;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float lo = __uint_as_float(d[q] << 16), hi = __uint_as_float(d[q] & 0xFFFF0000u);
                    o[q] = pack_bf16x2(w[i] * lo, w[i] * hi);
                    dot[i] = __builtin_fmaf(lo, __uint_as_float(y[i][q] << 16), dot[i]);
                    dot[i] = __builtin_fmaf(hi, __uint_as_float(y[i][q] & 0xFFFF0000u), dot[i]);
                }
                *reinterpret_cast<v4u*>(a.dY + row[i] * a.H + col) = o;
            }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            float v = row16_sum_f(dot[i]);
            v += __shfl_xor(v, 16, 64);
            v += __shfl_xor(v, 32, 64);
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][i] = v;
        }
        __syncthreads();
        if (threadIdx.x < kDeep && j0 + (int)threadIdx.x < a.k) {
            float v = 0.0f;
#pragma unroll
            for (int w2 = 0; w2 < kThreads / 64; ++w2) v += part[w2][threadIdx.x];
            a.dweights[t * a.k + j0 + threadIdx.x] = v;
        }
        __syncthreads();
    }
}

int spans_of(int H) { return (H + kSpan - 1) / kSpan; }

}  // namespace

void launch_dispatch(const DispatchArgs& a, bool large, hipStream_t s) {
    const int spans = spans_of(a.H);
    const dim3 grid((unsigned)(a.T * spans));
    if (a.T == 0) {
        const int n = a.contiguous ? a.cap : a.G;
        if (n > 0)
            hipLaunchKernelGGL(dispatch_empty_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                               a.where, n, a.contiguous ? -1 : 0);
        return;
    }
    if (!large) {
        hipLaunchKernelGGL(dispatch_small_kernel, grid, dim3(kThreads), 0, s, a, spans);
        return;
    }
    hipLaunchKernelGGL(dispatch_count_kernel, dim3((unsigned)a.chunks), dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(dispatch_scan_kernel, dim3(1), dim3(1024), 0, s, a);
    hipLaunchKernelGGL(dispatch_copy_kernel, grid, dim3(kThreads), 0, s, a, spans);
}

void launch_combine(const CombineArgs& a, hipStream_t s) {
    const int spans = spans_of(a.H);
    hipLaunchKernelGGL(combine_kernel, dim3((unsigned)(a.T * spans)), dim3(kThreads), 0, s, a, spans);
}

void launch_combine_backward(const CombineArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(combine_backward_kernel, dim3((unsigned)a.T), dim3(kThreads), 0, s, a);
}

}  // namespace fp8gemm
