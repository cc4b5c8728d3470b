// permute_kernels.hip -- gfx950 kernels that move rows between token order and expert order: the
// dispatch (each token's row, quantised to E4M3 with 1x128 scales, into the rows of its experts),
// the weighted combine back, and the combine's gradients.  The mathematics is stated in
// include/fp8gemm.h.
//
// The rank of a pair (token t, pick j) among its expert's rows is the number of earlier pairs, in
// (t, j) order, with the same expert, so the layout does not depend on timing.  Small batches
// recompute the ranks in every workgroup of the one copying launch; large ones count chunks of
// pairs, scan the counts, copy, and put the scales in place, in four launches.
//
// Bound: memory, with next to no arithmetic (the quantiser's is hidden).  4095 x 8 x 7168 on 64 experts
// 66 to 71 us, 4.2 to 4.6 TB/s (count 5, scan 5, copy 53, scales 6); 128 x 8 x 7168 on 16 experts 5.1 us, a
// launch and the pass over the picks; combine 4096 x 8 x 7168 102.4 us, 5.15 TB/s, and 128 x 8 x 7168 6.8 us
// with Y's rows in the memory-side cache; its gradient 1000 x 6 x 2048 11.6 us, 4.6 TB/s.

#include <algorithm>

#include "fp8gemm_device.h"
#include "moe_device.h"
#include "moe_internal.h"

namespace fp8gemm {
namespace {

// Workgroup size of the row passes with 16 bytes of bf16 per thread: 16 lanes own a 128-value block, and
// a wave's load is 1 KB of consecutive memory.
constexpr int kThreads = kRowThreads;
constexpr int64_t kCacheBytes = 256 << 20;   // the memory-side cache
constexpr int kSpan = kRowSpan;          // elements of a row one workgroup handles per pass

// Correctly rounded x / s for one E4M3 conversion: with r = RN(1/s) and q = RN(x r), one
// residual step gives RN(x / s) (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34(1), 1990); the sign is x's, so that -0 stays -0.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = x * r;
    return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, x), r, q), x);
}

// The 1x128 quantiser on 8 C bf16 values of a lane (16 / C lanes a block): codes and the scale.
template <int C>
struct Codes {
    typedef uint32_t Words __attribute__((ext_vector_type(2 * C)));
    Words w;
    float scale;
};
template <int C>
__device__ __forceinline__ Codes<C> quantize(const v4u (&x)[C]) {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < C; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(x[h][i] & 0x7FFFu, (x[h][i] >> 16) & 0x7FFFu));
    // bit patterns of |x| order like the values
    m = max(m, (uint32_t)dpp16<kDppXor1>((int)m));
    m = max(m, (uint32_t)dpp16<kDppXor2>((int)m));
    m = max(m, (uint32_t)dpp16<kDppHalfMirror>((int)m));
    if constexpr (C == 1) m = max(m, (uint32_t)dpp16<kDppMirror>((int)m));
    const float s = fmaxf(__uint_as_float(m << 16), 1e-4f) / 448.0f;
    const float r = 1.0f / s;
    Codes<C> o;
#pragma unroll
    for (int h = 0; h < C; ++h) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __builtin_amdgcn_fmed3f(quotient(__uint_as_float(x[h][i] << 16), s, r), -448.0f, 448.0f);
            v[2 * i + 1] = __builtin_amdgcn_fmed3f(quotient(__uint_as_float(x[h][i] & 0xFFFF0000u), s, r), -448.0f, 448.0f);
        }
        int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
        int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
        o.w[2 * h] = (uint32_t)lo;
        o.w[2 * h + 1] = (uint32_t)hi;
    }
    o.scale = s;
    return o;
}

// Local expert of a pick, or -1 (no pick, or another rank's expert).
__device__ __forceinline__ int expert_of(const DispatchArgs& a, int pick) {
    const int64_t id = (int64_t)pick - a.first;          // any int32 pick and first stay in range
    return pick >= 0 && id >= 0 && id < a.G ? (int)id : -1;
}
__device__ __forceinline__ int local_expert(const DispatchArgs& a, int pair) { return expert_of(a, a.ids[pair]); }

__device__ __forceinline__ int padded(int n) { return (n + 127) & ~127; }

// Row of local expert e's rank-th pair, or -1 past the capacity; `first` is the expert's first
// row in the contiguous layout.
__device__ __forceinline__ int place(const DispatchArgs& a, int e, int rank, int64_t first) {
    const int64_t row = a.contiguous ? first + rank : (int64_t)e * a.cap + rank;
    return (uint32_t)rank < (uint32_t)a.cap && (!a.contiguous || row < a.cap) ? (int)row : -1;
}

// Store a lane's codes at column `col` of the rows[0..k) that are not -1, past the caches (nothing reads
// them before the next product).
template <int C>
__device__ __forceinline__ void store_codes(const DispatchArgs& a, int col, const Codes<C>& q, const int* rows) {
    for (int j = 0; j < a.k; ++j) {
        const int row = rows[j];
        if (row >= 0)
            __builtin_nontemporal_store(q.w, reinterpret_cast<typename Codes<C>::Words*>(a.A + (int64_t)row * a.H + col));
    }
}

// Address of the scale of row `row`, K block kb (K-block-major per group).
__device__ __forceinline__ float* scale_at(const DispatchArgs& a, int row, int kb) {
    const int e = a.contiguous ? 0 : row / a.cap;
    return a.sa + ((int64_t)e * a.nkb + kb) * a.cap + (row - (int64_t)e * a.cap);
}

// Scales of K blocks kb0 .. kb0 + blocks from LDS to the rows, a lane each.
__device__ __forceinline__ void store_scales(const DispatchArgs& a, int kb0, int blocks, const int* rows, const float* scales) {
    for (int i = threadIdx.x; i < blocks * a.k; i += blockDim.x) {
        const int kb = (int)fast_div(i, a.div_k), pick = i - kb * a.k;
        if (rows[pick] >= 0) *scale_at(a, rows[pick], kb0 + kb) = scales[kb];
    }
}

// m_indices of this workgroup's share of the contiguous layout's rows: the expert whose rows [first,
// first + count) hold the row, or -1.
template <typename First, typename Count>
__device__ __forceinline__ void fill_indices(const DispatchArgs& a, First first, Count count) {
    const int64_t per = (a.cap + gridDim.x - 1) / gridDim.x;
    const int64_t end = min((blockIdx.x + 1) * per, (int64_t)a.cap);
    for (int64_t r = blockIdx.x * per + threadIdx.x; r < end; r += blockDim.x) {
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
    __shared__ int first[kDispatchMaxGroups], wave_total[kThreads / 64];
    __shared__ int rows[kDispatchMaxTopk], mine[kDispatchMaxTopk];
    __shared__ float scales[kSpan / 128];
    const int64_t t = blockIdx.x / spans;
    const int s = blockIdx.x - (int)t * spans;
    // a thread's 8 values are asked for before their rows are known
    const int col = s * kSpan + threadIdx.x * 8;
    const v4u x[1] = {*reinterpret_cast<const v4u*>(a.X + t * a.H + min(col, a.H - 8))};
    for (int e = threadIdx.x; e < a.G; e += kThreads) all[e] = before[e] = 0;
    __syncthreads();
    const int p0 = (int)t * a.k;
    constexpr int kDeep = 8;             // picks a thread has on their way
    for (int p1 = threadIdx.x; p1 < a.pairs; p1 += kThreads * kDeep) {
        int pick[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) pick[i] = p1 + i * kThreads < a.pairs ? a.ids[p1 + i * kThreads] : -1;
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int e = expert_of(a, pick[i]);
            if (e >= 0) {
                atomicAdd(&all[e], 1);
                if (p1 + i * kThreads < p0) atomicAdd(&before[e], 1);
            }
        }
    }
    if (threadIdx.x < a.k) mine[threadIdx.x] = local_expert(a, p0 + threadIdx.x);
    __syncthreads();
    if (a.contiguous) {                  // first rows: a running sum over 256 experts at a time, 64 a wave
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        int carry = 0;
        for (int e0 = 0; e0 < a.G; e0 += kThreads) {
            const int e = e0 + threadIdx.x;
            const int n = e < a.G ? padded(all[e]) : 0;
            int sum = n;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(sum, o, 64);
                if (lane >= o) sum += up;
            }
            int row = carry + sum - n;
            if (a.G > 64) {
                if (lane == 63) wave_total[wave] = sum;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kThreads / 64; ++w) {
                    row += w < wave ? wave_total[w] : 0;
                    carry += wave_total[w];
                }
                if (e0 + kThreads < a.G) __syncthreads();
            }
            if (e < a.G) first[e] = row;
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
    if (a.contiguous) {
        fill_indices(a, [&](int e) { return first[e]; }, [&](int e) { return all[e]; });
    } else if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < a.G; e += kThreads) a.where[e] = min(all[e], a.cap);
    }
    __syncthreads();
    const Codes<1> q = quantize(x);
    if (col < a.H) {                     // the 16 lanes of a 128-value block are in or out together
        store_codes(a, col, q, rows);
        if ((threadIdx.x & 15) == 0) scales[threadIdx.x >> 4] = q.scale;
    }
    __syncthreads();
    store_scales(a, s * (kSpan / 128), min(kSpan / 128, a.nkb - s * (kSpan / 128)), rows, scales);
}

// Scratch of the large path, in words.
struct Scratch {
    int32_t* counts;   // [G][chunks]: pairs per chunk, then their exclusive sums over chunks
    int32_t* first;    // [G]: first row (contiguous)
    int32_t* total;    // [G]
    int32_t* local;    // [pairs]: rank within the chunk
    float* scales;     // by_row: [T][nkb]
    int32_t* token;    // by_row: the token of each row of the layout that has one
};
__device__ __forceinline__ Scratch scratch_of(const DispatchArgs& a) {
    Scratch s;
    s.counts = a.scratch;
    s.first = s.counts + (int64_t)a.G * a.chunks;
    s.total = s.first + a.G;
    s.local = s.total + a.G;
    s.scales = reinterpret_cast<float*>(s.local + a.pairs);
    s.token = s.local + a.pairs + a.T * a.nkb;
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
    constexpr int kBatch = 4;            // experts a wave scans side by side, their loads in flight together
    for (int e0 = wave * kBatch; e0 < a.G; e0 += 16 * kBatch) {
        int carry[kBatch] = {0, 0, 0, 0};
        for (int c0 = 0; c0 < a.chunks; c0 += 64) {
            const int c = c0 + lane;
            int n[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                n[i] = e0 + i < a.G && c < a.chunks ? sc.counts[(int64_t)(e0 + i) * a.chunks + c] : 0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                int sum = n[i];
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) {
                    const int up = __shfl_up(sum, o, 64);
                    if (lane >= o) sum += up;
                }
                if (e0 + i < a.G && c < a.chunks) sc.counts[(int64_t)(e0 + i) * a.chunks + c] = carry[i] + sum - n[i];
                carry[i] += __shfl(sum, 63, 64);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (lane == 0 && e0 + i < a.G) total[e0 + i] = carry[i];
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

// A workgroup per token, 16 values a thread.  A token's scattered scales (4 bytes each, a row apart) would
// cost as much as a third of its codes, so with by_row they are kept token by token, for
// dispatch_scales_kernel to turn round.
__global__ __launch_bounds__(1024) void dispatch_copy_kernel(DispatchArgs a) {
    __shared__ int rows[kDispatchMaxTopk];
    __shared__ float scales[128];
    const Scratch sc = scratch_of(a);
    const int64_t t = blockIdx.x;
    v4u x[2];
    auto load = [&](int col) {
        const v4u* p = reinterpret_cast<const v4u*>(a.X + t * a.H + min(col, a.H - 16));
        x[0] = p[0];
        x[1] = p[1];
    };
    int col = threadIdx.x * 16;
    load(col);                           // before the rows are known
    if (threadIdx.x < a.k) {
        const int p = (int)(t * a.k) + threadIdx.x;
        const int e = local_expert(a, p);
        int row = -1;
        if (e >= 0) {
            const int rank = sc.counts[(int64_t)e * a.chunks + p / kDispatchChunk] + sc.local[p];
            row = place(a, e, rank, sc.first[e]);
            if (row < 0) atomicOr(a.err, (int32_t)kDevErrBadCount);
        }
        rows[threadIdx.x] = row;
        a.row_map[p] = row;
        if (a.by_row && row >= 0) sc.token[row] = (int32_t)t;
    }
    __syncthreads();
    if (a.contiguous) fill_indices(a, [&](int e) { return sc.first[e]; }, [&](int e) { return sc.total[e]; });
    for (int col0 = 0; col0 < a.H; col0 += blockDim.x * 16, col += blockDim.x * 16) {
        if (col0) load(col);
        const Codes<2> q = quantize(x);
        const int kb0 = col0 / 128;
        float* keep = a.by_row ? sc.scales + t * a.nkb + kb0 : scales;
        if (col < a.H) {                 // the 8 lanes of a 128-value block are in or out together
            store_codes(a, col, q, rows);
            if ((threadIdx.x & 7) == 0) keep[threadIdx.x >> 3] = q.scale;
        }
        if (!a.by_row) {
            __syncthreads();
            store_scales(a, kb0, min((int)blockDim.x / 8, a.nkb - kb0), rows, scales);
            __syncthreads();
        }
    }
}

// Scales of 64 rows of the layout and 32 K blocks: read token by token, turned round in LDS, written
// K block by K block.
constexpr int kTurnRows = 64, kTurnBlocks = 32;
__global__ __launch_bounds__(kThreads) void dispatch_scales_kernel(DispatchArgs a) {
    __shared__ float tile[kTurnRows][kTurnBlocks + 1];
    const Scratch sc = scratch_of(a);
    const int tiles = (a.cap + kTurnRows - 1) / kTurnRows;       // per group of the masked layout
    const int e = a.contiguous ? 0 : blockIdx.x / tiles;
    const int r0 = (blockIdx.x - e * tiles) * kTurnRows, kb0 = blockIdx.y * kTurnBlocks;
    const int valid = a.contiguous ? a.cap : a.where[e];
    if (r0 >= valid) return;
    auto there = [&](int r) { return r < valid && (!a.contiguous || a.where[r] >= 0); };
    constexpr int kPass = kThreads / kTurnBlocks, kRows = kTurnRows / kPass;
    const int kb = threadIdx.x % kTurnBlocks, r1 = threadIdx.x / kTurnBlocks;
    int token[kRows];                                            // the loads of a step are in flight together
    float v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = r0 + r1 + i * kPass;
        token[i] = there(r) ? sc.token[(int64_t)e * a.cap + r] : -1;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        v[i] = (uint32_t)token[i] < (uint32_t)a.T && kb0 + kb < a.nkb ? sc.scales[(int64_t)token[i] * a.nkb + kb0 + kb] : 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) tile[r1 + i * kPass][kb] = v[i];
    __syncthreads();
    const int r = threadIdx.x % kTurnRows;
    if (!there(r0 + r)) return;
#pragma unroll
    for (int b = threadIdx.x / kTurnRows; b < kTurnBlocks; b += kThreads / kTurnRows)
        if (kb0 + b < a.nkb) a.sa[((int64_t)e * a.nkb + kb0 + b) * a.cap + r0 + r] = tile[r][b];
}

// ---- combine ----

// Row of pair (t, j) in Y, or -1.
__device__ __forceinline__ int64_t pair_row(const CombineArgs& a, int64_t t, int j) {
    if (!a.row_map) return t * a.k + j;
    const int r = a.row_map[t * a.k + j];
    return r >= 0 && r < a.R ? r : -1;
}

// out[t] = sum_j w[t][j] Y[row(t, j)], in fp32 in the order of j.  Memory bound: each thread owns
// 16 bytes of the output and keeps the loads of 8 rows in flight.  STREAM: Y is larger than the
// memory-side cache and is read past the caches (us, with and without: 4096 x 8 x 7168, 470 MB, 104 and 111,
// 5.05 and 4.75 TB/s; 128 x 8 x 7168 with Y in the cache 8.3 and 6.8).
template <bool STREAM>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineArgs a, int spans) {
    const int64_t t = blockIdx.x / spans;
    const int s = (int)(blockIdx.x - t * spans);
    const int col = s * kSpan + threadIdx.x * 8;
    if (s == 0 && threadIdx.x < a.k && a.row_map && a.row_map[t * a.k + threadIdx.x] >= a.R)
        atomicOr(a.err, (int32_t)kDevErrBadIndex);
    if (col >= a.H) return;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    constexpr int kDeep = 8;
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
                    const v4u* p = reinterpret_cast<const v4u*>(a.Y + r * a.H + col);
                    if constexpr (STREAM) y[i] = __builtin_nontemporal_load(p);
                    else y[i] = *p;
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
template <int THREADS>
__global__ __launch_bounds__(THREADS) void combine_backward_kernel(CombineArgs a) {
    constexpr int kDeep = 8;
    __shared__ float part[THREADS / 64][kDeep];
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
        for (int col = threadIdx.x * 8; col < a.H; col += THREADS * 8) {
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
            for (int w2 = 0; w2 < THREADS / 64; ++w2) v += part[w2][threadIdx.x];
            a.dweights[t * a.k + j0 + threadIdx.x] = v;
        }
        __syncthreads();
    }
}

}  // namespace

void launch_dispatch(const DispatchArgs& a, bool large, hipStream_t s) {
    const int spans = (int)row_spans(a.H);
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
    hipLaunchKernelGGL(dispatch_copy_kernel, dim3((unsigned)a.T), dim3((unsigned)dispatch_copy_threads(a.H)), 0, s, a);
    if (a.by_row) {
        const int64_t tiles = (int64_t)(a.contiguous ? 1 : a.G) * ((a.cap + kTurnRows - 1) / kTurnRows);
        const dim3 turn((unsigned)tiles, (unsigned)((a.nkb + kTurnBlocks - 1) / kTurnBlocks));
        if (tiles > 0) hipLaunchKernelGGL(dispatch_scales_kernel, turn, dim3(kThreads), 0, s, a);
    }
}

void launch_combine(const CombineArgs& a, hipStream_t s) {
    const int spans = (int)row_spans(a.H);
    const dim3 grid((unsigned)(a.T * spans));
    if (2 * a.T * a.k * a.H > kCacheBytes) hipLaunchKernelGGL(combine_kernel<true>, grid, dim3(kThreads), 0, s, a, spans);
    else hipLaunchKernelGGL(combine_kernel<false>, grid, dim3(kThreads), 0, s, a, spans);
}

// 512 threads where a token's row is more than one pass of 256 and every CU has a token's workgroup to
// itself.  Measured, 256 and 512, us, 7 picks: 11 x 7168 7.7 and 6.7, 256 x 2944 7.3 and 6.9; but 512 x 2944 10.2
// and 10.3, 1000 x 2944 17.0 and 18.0, 256 x 2048 5.7 and 5.8.
void launch_combine_backward(const CombineArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.T);
    if (a.H > kSpan && a.T <= 256) hipLaunchKernelGGL(combine_backward_kernel<512>, grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL(combine_backward_kernel<256>, grid, dim3(256), 0, s, a);
}

}  // namespace fp8gemm
