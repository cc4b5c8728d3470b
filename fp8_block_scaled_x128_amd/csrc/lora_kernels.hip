// lora_kernels.hip -- gfx950 kernels of low-rank adapters of many requests beside a shared projection:
//   out[t] = bf16(Y[t] + s[a] * B[a] (A[a] x[t])),  a = ids[t] the adapter of row t, or none.
// Three forms, by the rows' number and the adapters' size (the host's rules have both sides measured):
//   a workgroup a row, both products in one launch: small adapters in small batches.  Bound by the launch and by what
//     one CU reads: 45 rows, R = 8, 1544 to 2112, 5.0 us.
//   two launches, 1 to 16 places a workgroup: the rank-R products A x, in fp32 through the workspace, then B's product,
//     the sum and the store.  Bound by two launches, then the adapters' bytes: 1 row 6.9 us, 256 rows of 64 adapters,
//     R = 16, 7168 to 4096, 15.0 us.
//   two launches, 64 places a workgroup, operands through LDS: prefill.  Bound by HBM: 8192 rows of 8 adapters, R = 32,
//     7168 to 4096, 61 us, 4.2 TB/s; with large ranks by A's and B's way through L2: 2000 rows, R = 128, 2048 to 7168, 37 us.
//
// Places are rows, or positions in the order the caller gives.  A tile of them goes through the adapters that its rows
// have, one after the other; matrix-core columns of rows with another adapter are left out of the results.  So any mix
// of rows is right, and one whose neighbours share an adapter reads each of its matrices once per tile.  A x stays in
// 32 bits until the second product, which takes it as two bf16 halves: one rounding of the result, as in the formula.

#include <type_traits>

#include "ffn_internal.h"
#include "fp8gemm_device.h"
#include "moe_device.h"

namespace fp8gemm {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4, kThreads = kWaves * 64;

__device__ __forceinline__ v4f mfma_bf16(const v4u& x, const v4u& y, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y), c, 0, 0, 0);
}

// Row and adapter of a place, both -1 where there is none (past the last place; the order or the id out of range).
struct Place {
    int64_t row;
    int id;
};
__device__ __forceinline__ Place place_of(const LoraArgs& a, int p, bool report) {
    Place o{-1, -1};
    if (p >= a.places) return o;
    const int64_t at = a.first + p;
    const int64_t row = a.order ? a.order[at] : at;
    bool bad = row < 0 || row >= a.T;
    if (!bad) {
        o.row = row;
        const int id = a.ids[row];
        bad = id >= a.L;
        o.id = id < 0 || bad ? -1 : id;
    }
    if (bad && report) atomicOr(a.err, kDevErrBadIndex);
    return o;
}

__device__ __forceinline__ float scale_of(const LoraArgs& a, int id) { return a.scales && id >= 0 ? a.scales[id] : 1.0f; }

// Workgroup barrier for LDS alone: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Four values as bf16 halves: a value's first 8 bits, and what they leave of it, rounded, together within 2^-16 of it.
// The first is cut off, not rounded, so that both have the value's sign, and the second is 2^-133, the least bf16, where
// nothing is left: B's infinities then give the same infinity with both, as with the value, and zero times infinity is
// left to zeros (and to values below 2^-133).  Of an infinity nothing is left either (fmed3 of NaN and two numbers is the
// smaller number); NaN, as sums give it, keeps its first bits.
__device__ __forceinline__ void halves_of(const v4f& v, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
    float rest[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float first = __uint_as_float(__float_as_uint(v[e]) & 0xFFFF0000u);
        rest[e] = __builtin_copysignf(__builtin_amdgcn_fmed3f(__builtin_fabsf(v[e] - first), 0x1p-133f, __builtin_fabsf(first)), v[e]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        hi[e] = __float_as_uint(v[2 * e]) >> 16 | (__float_as_uint(v[2 * e + 1]) & 0xFFFF0000u);
        lo[e] = pack_bf16x2(rest[2 * e], rest[2 * e + 1]);
    }
}

// A lane's copy of what lane `from` holds.
__device__ __forceinline__ int64_t row_of(int64_t row, int from) {
    const int lo = __shfl((int)(uint32_t)row, from, 64), hi = __shfl((int)(row >> 32), from, 64);
    return ((int64_t)hi << 32) | (uint32_t)lo;
}

constexpr int kDownWaves = 8;

// A x for 16 places a workgroup, or fewer, and 16 RT of the rank; AHEAD: loads of 32 values of K on their way.  The
// waves share the split's steps of 64 values of K, and their sums meet in LDS and are added in wave order; where the
// places have three adapters or more, each wave has adapters of its own and all of the steps, and adds the eight
// waves' sums in the same order.
template <int RT, int AHEAD>
__global__ __launch_bounds__(kDownWaves * 64, 2) void lora_down_kernel(const LoraArgs a) {
    __shared__ v4f red[kDownWaves][RT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row16 = lane & 15, grp = lane >> 4;
    const int p0 = blockIdx.y * a.tile;
    const int split = blockIdx.x, r0 = blockIdx.z * (16 * RT);
    const int step0 = split * a.per_split, step1 = min(a.steps, step0 + a.per_split);
    const int rounds = (a.per_split + kDownWaves - 1) / kDownWaves;  // steps of a wave, the last ones past the end perhaps

    // lane l knows place p0 + l
    const Place mine = lane < a.tile ? place_of(a, p0 + lane, split == 0 && r0 == 0 && wave == 0) : Place{-1, -1};
    const uint64_t all = __builtin_amdgcn_ballot_w64(mine.id >= 0);
    uint64_t left = all;
    auto next = [&](uint64_t* has) {                         // the first adapter left, and its places
        const int adapter = __builtin_amdgcn_readlane(mine.id, __builtin_ctzll(left));
        *has = __builtin_amdgcn_ballot_w64(mine.id == adapter);
        left &= ~*has;
        return adapter;
    };
    int adapters = 0;
    for (uint64_t has; left && adapters < 3; ++adapters) next(&has);
    const bool apart = adapters >= 3;
    left = all;

    for (int turn = 0; left; ++turn) {
        uint64_t has;
        const int adapter = next(&has);
        if (apart && (turn & (kDownWaves - 1)) != wave) continue;
        const int first = __builtin_ctzll(has);
        // the row of this lane's matrix-core column; a column of another adapter repeats the first row (and is left out)
        const uint16_t* xp = a.X + row_of(mine.row, (has >> row16) & 1 ? row16 : first) * a.ldx;
        const uint16_t* ap = uniform_ptr(a.A + (int64_t)adapter * a.R * a.K);
        uint32_t arow[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) arow[r] = (uint32_t)min(r0 + 16 * r + row16, a.R - 1) * (uint32_t)a.K;
        v4f acc[RT], total[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = (v4f){0.f, 0.f, 0.f, 0.f};
        // half h of a step: lane group grp has 8 of its 16 values
        struct Half {
            v4u w[RT], x;
        };
        Half ring[AHEAD];
        // the u-th half of this wave: steps 8 apart, for each of the eight waves in turn where the wave has all of them
        const int halves = 2 * rounds * (apart ? kDownWaves : 1);
        auto load = [&](Half& f, int u) {
            if (u >= halves) return;
            const int q = u >> 1;
            const int step = step0 + (apart ? q % rounds * kDownWaves + q / rounds : q * kDownWaves + wave);
            const int k = step * 64 + grp * 16 + (u & 1) * 8;
            const bool in = step < step1 && k < a.K;          // else zeros, in both operands
            const uint32_t ko = in ? (uint32_t)k : 0u;
#pragma unroll
            for (int r = 0; r < RT; ++r) f.w[r] = *reinterpret_cast<const v4u*>(ap + (arow[r] + ko));
            f.x = *reinterpret_cast<const v4u*>(xp + ko);
            if (!in) {
                f.x = (v4u){0, 0, 0, 0};
#pragma unroll
                for (int r = 0; r < RT; ++r) f.w[r] = (v4u){0, 0, 0, 0};
            }
        };
        static_assert(AHEAD % 2 == 0, "whole steps");
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) load(ring[p], p);
        for (int u0 = 0; u0 < halves; u0 += AHEAD) {
#pragma unroll
            for (int p = 0; p < AHEAD; ++p) {
                const int u = u0 + p;
                if (u >= halves) break;
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[r] = mfma_bf16(ring[p].w[r], ring[p].x, acc[r]);
                load(ring[p], u + AHEAD);
                // the end of a wave's steps, taken by this one
                if ((p & 1) && apart && (u + 1) / 2 % rounds == 0) {
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        total[r] = u + 1 == 2 * rounds ? acc[r] : total[r] + acc[r];
                        acc[r] = (v4f){0.f, 0.f, 0.f, 0.f};
                    }
                }
            }
        }
        // tile r: a lane holds values 16 r + 4 grp .. + 3 of its column's row
        auto store = [&](int r, const v4f& v) {
            if (r0 + 16 * r < a.rank && (has >> row16) & 1)
                *reinterpret_cast<v4f*>(a.low + ((int64_t)split * a.places + p0 + row16) * a.rank + r0 + 16 * r + 4 * grp) = v;
        };
        if (apart) {
#pragma unroll
            for (int r = 0; r < RT; ++r) store(r, total[r]);
            continue;
        }
        lds_barrier();                                       // the sums of the adapter before are read
#pragma unroll
        for (int r = 0; r < RT; ++r) red[wave][r][lane] = acc[r];
        lds_barrier();
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if (wave != r) continue;
            v4f v = red[0][r][lane];
#pragma unroll
            for (int w = 1; w < kDownWaves; ++w) v += red[w][r][lane];
            store(r, v);
        }
    }
}

// Sum over groups of 1 << shift lanes, at most 16.
__device__ __forceinline__ float sum_of_lanes(float d, int shift) {
    auto moved = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    if (shift > 0) d += moved(d, std::integral_constant<int, 0xB1>{});      // lane ^ 1
    if (shift > 1) d += moved(d, std::integral_constant<int, 0x4E>{});      // lane ^ 2
    if (shift > 2) d += moved(d, std::integral_constant<int, 0x141>{});     // 7 - lane of 8: the other four
    if (shift > 3) d += moved(d, std::integral_constant<int, 0x140>{});     // 15 - lane of 16: the other eight
    return d;
}

// Both products of a row by one workgroup, for small adapters: its waves take the steps of K in turn, their sums meet in
// LDS, and lanes form the columns of the result from A x in fp32.  One CU brings the adapter's two matrices in, so this
// pays while they are small (the choice, with both sides measured, is the host's): 64 rows, R = 8, 2048 to 1024, 4.6 us.
template <int RT>
__global__ __launch_bounds__(kDownWaves * 64, 2) void lora_row_kernel(const LoraArgs a) {
    constexpr int kRowThreads = kDownWaves * 64;
    __shared__ v4f red[kDownWaves][RT][4];
    __shared__ v4f low[4 * RT];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row16 = lane & 15, grp = lane >> 4;
    const Place mine = place_of(a, blockIdx.x, tid == 0);
    if (mine.row < 0) return;
    const uint16_t* y = a.Y + mine.row * a.ldy;
    uint16_t* out = a.out + mine.row * a.ldo;
    if (mine.id < 0) {
        if (a.Y != a.out)
            for (int n = tid * 8; n < a.N; n += kRowThreads * 8) *reinterpret_cast<v4u*>(out + n) = *reinterpret_cast<const v4u*>(y + n);
        return;
    }
    const uint16_t* xp = a.X + mine.row * a.ldx;
    const uint16_t* ap[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) ap[r] = a.A + ((int64_t)mine.id * a.R + min(16 * r + row16, a.R - 1)) * a.K;
    v4f acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = (v4f){0.f, 0.f, 0.f, 0.f};
    constexpr int AHEAD = RT < 4 ? 4 / RT : 1;                           // steps whose loads go out together
    for (int s0 = wave; s0 < a.steps; s0 += AHEAD * kDownWaves) {
        v4u w[AHEAD][2][RT], x[AHEAD][2];
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (s0 + p * kDownWaves) * 64 + grp * 16 + h * 8;
                const bool in = k < a.K;                     // else zeros, in both operands
                const int ko = in ? k : 0;
                x[p][h] = *reinterpret_cast<const v4u*>(xp + ko);
#pragma unroll
                for (int r = 0; r < RT; ++r) w[p][h][r] = *reinterpret_cast<const v4u*>(ap[r] + ko);
                if (!in) {
                    x[p][h] = (v4u){0, 0, 0, 0};
#pragma unroll
                    for (int r = 0; r < RT; ++r) w[p][h][r] = (v4u){0, 0, 0, 0};
                }
            }
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[r] = mfma_bf16(w[p][h][r], x[p][h], acc[r]);
    }
    // every matrix-core column is the row; lane group grp has values 16 r + 4 grp .. + 3
    if (row16 == 0) {
#pragma unroll
        for (int r = 0; r < RT; ++r) red[wave][r][grp] = acc[r];
    }
    __syncthreads();
    if (tid < 4 * RT) {
        v4f v = red[0][tid >> 2][tid & 3];
#pragma unroll
        for (int w = 1; w < kDownWaves; ++w) v += red[w][tid >> 2][tid & 3];
        low[tid] = v;
    }
    // a column's row of B, and the sums with A x, are shared by as many lanes as it has 16-byte pieces (a power of two)
    const float scale = scale_of(a, mine.id);
    const int units = a.R / 8;
    const int shift = RT == 1 ? units - 1 : 32 - __builtin_clz(units - 1);
    const int u = tid & ((1 << shift) - 1), col = tid >> shift, cols = kRowThreads >> shift;
    const uint16_t* bp = a.B + (int64_t)mine.id * a.N * a.R + 8 * min(u, units - 1);
    constexpr int COLS = RT == 1 ? 4 : 8;                    // columns of a lane at a time
    v4f v[2];
    for (int n0 = 0; n0 < a.N; n0 += COLS * cols) {
        v4u b[COLS];
        uint16_t yv[COLS];
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            const int n = min(n0 + c * cols + col, a.N - 1);
            b[c] = *reinterpret_cast<const v4u*>(bp + (int64_t)n * a.R);
            yv[c] = y[n];
        }
        if (n0 == 0) {
            __syncthreads();                                 // A x is there
            v[0] = low[2 * min(u, units - 1)];
            v[1] = low[2 * min(u, units - 1) + 1];
        }
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            float d = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d = __builtin_fmaf(__uint_as_float(b[c][e] << 16), v[e >> 1][2 * (e & 1)], d);
                d = __builtin_fmaf(__uint_as_float(b[c][e] & 0xFFFF0000u), v[e >> 1][2 * (e & 1) + 1], d);
            }
            d = sum_of_lanes(u < units ? d : 0.f, shift);
            const int n = n0 + c * cols + col;
            if (u == 0 && n < a.N) out[n] = f32_to_bf16(__builtin_fmaf(d, scale, bf16_to_f32(yv[c])));
        }
    }
}

// A x for 64 places a workgroup, for batches whose places mostly share an adapter with their neighbours.  Slices of
// 64 values of K of the 64 rows of X and the adapter's rows of A pass through a ring in LDS, 128-byte rows with
// 16-byte chunk c of row r at c ^ swz(r) (as in the FP8 kernel); a wave has 16 places and all of the rank.
// A tile of several adapters is shared by two workgroups (apart = 1), that have them in turn: else it would take as many
// times as long as the others.  The second ones come first in the grid, where most of them end at once.  The last of a
// tile's splits to arrive adds their sums in split order and leaves A x as two bf16 halves, whose sum is within 2^-16
// of it (partials are written and read past the L2s of the XCDs, with agent-coherent accesses).
__device__ __forceinline__ int swz(int row) { return ((row >> 1) & 3) | ((((row >> 2) ^ (row >> 3)) & 1) << 2); }
__device__ __forceinline__ void dma_far(uint32_t lds_base, const void* p) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(lds_base), "v"(p) : "memory");
}

template <int RT, int STAGES>
__global__ __launch_bounds__(kThreads, 2) void lora_down64_kernel(const LoraArgs a) {
    constexpr int X_LOADS = 2, A_LOADS = RT < 2 ? 1 : RT / 2, NDMA = X_LOADS + A_LOADS;     // 1 KB loads of a wave and slice
    constexpr int A_OFF = 64 * 128, STAGE = A_OFF + RT * 2048;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * STAGE];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row16 = lane & 15, grp = lane >> 4;
    const int split = blockIdx.x, tiles = (a.places + 63) / 64;
    const int turn = a.apart && (int)blockIdx.y < tiles, tile = (int)blockIdx.y - (a.apart && !turn ? tiles : 0), p0 = tile * 64;
    const int s0 = split * a.per_split, nks = min(a.per_split, a.steps - s0);
    const uint32_t base = lds_addr(smem);
    const int tail = a.K - (a.steps - 1) * 64, tail_at = tail < 64 ? a.steps - 1 - s0 : -1;
    const int frag[2] = {((2 * grp) ^ swz(row16)) << 4, ((2 * grp + 1) ^ swz(row16)) << 4};

    const Place mine = place_of(a, p0 + lane, split == 0 && !turn && wave == 0);
    const __amdgpu_buffer_rsrc_t parts = __builtin_amdgcn_make_buffer_rsrc(
        uniform_ptr(a.low), 0, (int)((int64_t)a.splits * a.places * a.rank * 4), kBufferFlags);
    uint64_t left = __builtin_amdgcn_ballot_w64(mine.id >= 0), own = 0;
    for (int n = 0; left; ++n) {
        const int first = __builtin_ctzll(left);
        const int adapter = __builtin_amdgcn_readlane(mine.id, first);
        const uint64_t has = __builtin_amdgcn_ballot_w64(mine.id == adapter);
        left &= ~has;
        if ((n & a.apart) != turn) continue;
        own |= has;
        // a lane's rows of the loads: place 8 (2 wave + q) + lane / 8 (the first of the adapter, where it is another's)
        const int c8 = lane & 7;
        const uint16_t* xp[X_LOADS];
        int xc[X_LOADS], ac[A_LOADS];
        uint32_t aoff[A_LOADS];
#pragma unroll
        for (int q = 0; q < X_LOADS; ++q) {
            const int r = 8 * (X_LOADS * wave + q) + (lane >> 3);
            xc[q] = (c8 ^ swz(r)) * 8;
            xp[q] = a.X + row_of(mine.row, (has >> r) & 1 ? r : first) * a.ldx + (int64_t)s0 * 64;
        }
        auto a_row = [&](int q) { return RT < 2 ? 8 * (wave & 1) : 8 * (A_LOADS * wave + q); };
        const uint16_t* ap = uniform_ptr(a.A + (int64_t)adapter * a.R * a.K + (int64_t)s0 * 64);
#pragma unroll
        for (int q = 0; q < A_LOADS; ++q) {
            const int r = a_row(q) + (lane >> 3);
            ac[q] = (c8 ^ swz(r)) * 8;
            aoff[q] = (uint32_t)min(r, a.R - 1) * (uint32_t)a.K;
        }
        auto issue = [&](int i) {
            const uint32_t st = base + (uint32_t)((i % STAGES) * STAGE);
            const int valid = i == tail_at ? tail - 8 : 56;  // the last chunk that is there
#pragma unroll
            for (int q = 0; q < X_LOADS; ++q) dma_far(st + (X_LOADS * wave + q) * 1024, xp[q] + i * 64 + min(xc[q], valid));
#pragma unroll
            for (int q = 0; q < A_LOADS; ++q)
                dma_x4(st + A_OFF + a_row(q) * 128, uniform_ptr(ap + i * 64), 2 * (aoff[q] + (uint32_t)min(ac[q], valid)));
        };
        v4f acc[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i)
            if (i < nks) issue(i);
        for (int i = 0; i < nks; ++i) {
            wait_slices<NDMA, STAGES - 2, 0>(min(STAGES - 2, nks - 1 - i));
            __syncthreads();
            if (i + STAGES - 1 < nks) issue(i + STAGES - 1);
            uint8_t* st = smem + (i % STAGES) * STAGE;
            if (i == tail_at) {                              // zeros past K, in both operands
                for (int x = tid; x < (64 + RT * 16) * 8; x += kThreads)
                    if ((x & 7) * 8 >= tail)
                        *reinterpret_cast<v4u*>(st + (x >> 3) * 128 + (((x & 7) ^ swz(x >> 3)) << 4)) = (v4u){0, 0, 0, 0};
                __syncthreads();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4u x = *reinterpret_cast<const v4u*>(st + (16 * wave + row16) * 128 + frag[h]);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    acc[r] = mfma_bf16(*reinterpret_cast<const v4u*>(st + A_OFF + (16 * r + row16) * 128 + frag[h]), x, acc[r]);
            }
        }
        if ((has >> (16 * wave + row16)) & 1) {
            const int at = ((split * a.places + p0 + 16 * wave + row16) * a.rank + 4 * grp) * 4;
#pragma unroll
            for (int r = 0; r < RT; ++r)
                if (16 * r < a.rank) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, acc[r]), parts, at + 64 * r, 0, kSc1);
        }
        // the stores count among the loads that the next adapter waits for; its loads go where others may still read
        wait_vmcnt<0>();
        __syncthreads();
    }
    if (!own) return;                                        // (in all splits alike)
    if (a.splits > 1) {
        int32_t* counter = a.counters + 2 * tile + turn;
        if (tid == 0) {
            const int old = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            s_last = old == a.splits - 1;
            if (s_last) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!s_last) return;
    }
    // a thread has RT float4 of places; the reads of all of them, of some splits, are on their way together
    constexpr int SPLITS = RT <= 2 ? 8 : 16 / RT;
    const int per = a.rank / 4, step = a.places * a.rank * 4;
    int at[RT];
    v4f v[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int x = i * kThreads + tid, p = x / per, c = x - p * per;
        at[i] = p < 64 && ((own >> p) & 1) ? ((p0 + p) * a.rank + 4 * c) * 4 : -1;
        v[i] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    for (int s = 0; s < a.splits; s += SPLITS) {
        v4u t[SPLITS][RT];
#pragma unroll
        for (int e = 0; e < SPLITS; ++e)
#pragma unroll
            for (int i = 0; i < RT; ++i)
                t[e][i] = __builtin_amdgcn_raw_buffer_load_b128(parts, max(at[i], 0) + min(s + e, a.splits - 1) * step, 0, kSc1);
#pragma unroll
        for (int e = 0; e < SPLITS; ++e)
#pragma unroll
            for (int i = 0; i < RT; ++i)
                if (s + e < a.splits) v[i] += __builtin_bit_cast(v4f, t[e][i]);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        if (at[i] < 0) continue;
        const int x = i * kThreads + tid, p = x / per, c = x - p * per;
        if (4 * c >= a.R) v[i] = (v4f){0.f, 0.f, 0.f, 0.f};  // (a rank that is padded)
        uint32_t hi[2], lo[2];
        halves_of(v[i], hi, lo);
        uint32_t* d = reinterpret_cast<uint32_t*>(a.halves + ((int64_t)(p0 + p) * 2) * a.rank + 4 * c);
        *reinterpret_cast<uint2*>(d) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(d + a.rank / 2) = make_uint2(lo[0], lo[1]);
    }
}

// The results of 16 rows and 64 columns, in LDS, onto Y's: lane l has rows l / 8 and 8 + l / 8, 8 columns.
__device__ __forceinline__ void add_lines(const LoraArgs& a, const float* line, int lane, int n0, const int64_t (&row)[2],
                                          const bool (&has)[2], const v4u (&y)[2]) {
    const int n = n0 + (lane & 7) * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (row[h] < 0 || n >= a.N || (!has[h] && a.Y == a.out)) continue;
        v4u o = y[h];
        if (has[h]) {
            const float* l = line + (8 * h + (lane >> 3)) * 68 + (lane & 7) * 8;
            const v4f d0 = *reinterpret_cast<const v4f*>(l), d1 = *reinterpret_cast<const v4f*>(l + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = e < 2 ? d0[2 * (e & 1)] : d1[2 * (e & 1)], x1 = e < 2 ? d0[2 * (e & 1) + 1] : d1[2 * (e & 1) + 1];
                o[e] = pack_bf16x2(__uint_as_float(o[e] << 16) + x0, __uint_as_float(o[e] & 0xFFFF0000u) + x1);
            }
        }
        *reinterpret_cast<v4u*>(a.out + row[h] * a.ldo + n) = o;
    }
}

// The second product for 16 places a workgroup, or fewer.  RS: matrix-core steps of the rank.  A workgroup takes
// `chunks` runs of 256 columns, a wave 64 of each; its results become 128-byte lines of rows through LDS.
// A x enters as two bf16 halves, whose sum is within 2^-16 of it, formed in LDS from the splits' sums.  RS = 0: a
// rank of 16 at most in one step, the high halves in the step's first 16 values and the low ones in its last, against
// the same 16 values of B.  Else steps of 32 values of the rank, twice, with the high halves and with the low ones.
template <int RS>
__global__ __launch_bounds__(kThreads, 2) void lora_up_kernel(const LoraArgs a) {
    constexpr int STEPS = RS == 0 ? 1 : RS;
    constexpr int PITCH = RS == 0 ? 3 : 4 * RS + 1;          // 16-byte units of a place
    constexpr int LINE = 68;                                 // floats of a row of the results in LDS
    __shared__ v4u low[2][16][PITCH];                   // [half]
    __shared__ v4f lines[kWaves][16 * LINE / 4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row16 = lane & 15, grp = lane >> 4;
    const int p0 = blockIdx.y * a.tile;
    const Place mine = lane < a.tile ? place_of(a, p0 + lane, false) : Place{-1, -1};
    const uint64_t all = __builtin_amdgcn_ballot_w64(mine.id >= 0);
    float* const line = reinterpret_cast<float*>(lines[wave]);

    // rows and columns that this lane reads of Y and writes: rows lane / 8 and 8 + lane / 8 of a tile, 8 columns
    int64_t row[2];
    bool has[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int from = 8 * h + (lane >> 3);
        row[h] = row_of(mine.row, from);
        has[h] = (all >> from) & 1;
    }
    const float scale = scale_of(a, __shfl(mine.id, row16, 64));     // of this lane's matrix-core column
    int n0 = blockIdx.x * a.chunks * kLoraSpan + wave * 64;
    v4u y[2];
    auto fetch_y = [&]() {
        const int n = n0 + (lane & 7) * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (row[h] >= 0 && n < a.N) y[h] = *reinterpret_cast<const v4u*>(a.Y + row[h] * a.ldy + n);
    };
    // an adapter's part of B
    struct Part {
        v4u b[STEPS][4];
        int adapter, n0;
    };
    auto fetch = [&](Part& f, int adapter) {
        f.adapter = adapter;
        f.n0 = n0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = min(n0 + 16 * j + row16, a.N - 1);
            const uint16_t* bp = a.B + ((int64_t)adapter * a.N + n) * a.R;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int r = RS == 0 ? (grp & 1) * 8 : 32 * s + grp * 8;
                f.b[s][j] = (v4u){0, 0, 0, 0};               // zeros past the rank (in both operands)
                if (r < a.R) f.b[s][j] = *reinterpret_cast<const v4u*>(bp + r);
            }
        }
    };
    Part part;
    part.adapter = -1;
    // on their way ahead of what they meet
    if (n0 < a.N) {
        fetch_y();
        if (all) fetch(part, __builtin_amdgcn_readlane(mine.id, __builtin_ctzll(all)));
    }

    {
        // sums of the splits' parts: four threads share a float4 of a place, each with every fourth split; a thread
        // has ITEMS of them, of U splits at a time
        constexpr int PER = RS == 0 ? 4 : 8 * RS;            // float4s of a place in LDS
        constexpr int ITEMS = 64 * PER / kThreads, U = ITEMS < 4 ? 4 / ITEMS : 1;
        const int g = tid & 3;
        const int64_t ls = (int64_t)a.places * a.rank;
        v4f v[ITEMS];
        const float* lp[ITEMS];
        bool in[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int x = (i * kThreads + tid) >> 2, p = x / PER, c = x % PER;
            in[i] = ((all >> p) & 1) && 4 * c < a.R;
            lp[i] = a.low + (in[i] ? ((int64_t)p0 + p) * a.rank + 4 * c : 0);
            v[i] = (v4f){0.f, 0.f, 0.f, 0.f};
        }
        for (int s = g; s < a.splits; s += 4 * U) {
            v4f t[U][ITEMS];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) t[u][i] = *reinterpret_cast<const v4f*>(lp[i] + min(s + 4 * u, a.splits - 1) * ls);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
                    if (in[i] && s + 4 * u < a.splits) v[i] += t[u][i];
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int x = (i * kThreads + tid) >> 2, p = x / PER, c = x % PER;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[i][e] += dpp16f<kDppXor1>(v[i][e]);
                v[i][e] += dpp16f<kDppXor2>(v[i][e]);
            }
            uint32_t hi[2], lo[2];
            halves_of(v[i], hi, lo);
            if (g == 0) {
                *reinterpret_cast<uint2*>(reinterpret_cast<uint32_t*>(&low[0][p][0]) + 2 * c) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(reinterpret_cast<uint32_t*>(&low[1][p][0]) + 2 * c) = make_uint2(lo[0], lo[1]);
            }
        }
    }
    lds_barrier();

    for (int chunk = 0; chunk < a.chunks && n0 < a.N; ++chunk) {
        // this tile's adapters in turn; a column takes the sums of its own
        v4f acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = (v4f){0.f, 0.f, 0.f, 0.f};
        uint64_t left = all;
        while (left) {
            const int adapter = __builtin_amdgcn_readlane(mine.id, __builtin_ctzll(left));
            const uint64_t its = __builtin_amdgcn_ballot_w64(mine.id == adapter);
            left &= ~its;
            if (part.adapter != adapter || part.n0 != n0) fetch(part, adapter);
            v4f p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if constexpr (RS == 0) {
                    const v4u v = low[grp >> 1][row16][grp & 1];
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = mfma_bf16(part.b[s][j], v, p[j]);
                } else {
                    const v4u vh = low[0][row16][4 * s + grp], vl = low[1][row16][4 * s + grp];
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = mfma_bf16(part.b[s][j], vl, p[j]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = mfma_bf16(part.b[s][j], vh, p[j]);
                }
            }
            const bool here = (its >> row16) & 1;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = here ? p[j][e] * scale : acc[j][e];
        }
        wave_sync();                                     // the tile before is read
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<v4f*>(line + row16 * LINE + 16 * j + 4 * grp) = acc[j];
        wave_sync();
        add_lines(a, line, lane, n0, row, has, y);
        n0 += kLoraSpan;
        if (chunk + 1 < a.chunks && n0 < a.N) {
            fetch_y();
            if (all) fetch(part, part.adapter);
        }
    }
}

// The second product for 64 places a workgroup, 16 a wave, which holds their halves of A x in registers.  Runs of 64
// columns of B, 128 R bytes in one piece, and of Y's rows pass through LDS, one on its way during the products of the
// other; where the places have several adapters, a run of each in turn.  16-byte unit c of column r of B stands at
// c ^ r / (16 / (R / 8)), where R / 8 is a power of two, so that a fragment's 16 columns lie in different banks; else
// at c.  Chunk c of row r of Y stands at c ^ r % 8; the result takes its place, and leaves in 128-byte lines of rows.
// RS as above, one step for each 32 of the rank.
template <int RS>
__global__ __launch_bounds__(kThreads, 2) void lora_up64_kernel(const LoraArgs a) {
    constexpr int STEPS = RS == 0 ? 1 : RS;
    constexpr int LOADS = RS == 0 ? 1 : RS;                  // 1 KB loads of B, of a wave and run
    constexpr int RUN = LOADS * 4096;                        // LDS bytes of a run, at most
    __shared__ __attribute__((aligned(1024))) uint8_t ring[2 * RUN];
    __shared__ __attribute__((aligned(1024))) uint8_t rows[2][kWaves][2048];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row16 = lane & 15, grp = lane >> 4;
    const int p0 = blockIdx.y * 64, mine16 = 16 * wave;
    const uint32_t base = lds_addr(ring), ybase = lds_addr(rows) + wave * 2048;
    const Place mine = place_of(a, p0 + lane, false);
    const uint64_t all = __builtin_amdgcn_ballot_w64(mine.id >= 0);
    const int units = a.R / 8, mask = (units & (units - 1)) == 0 ? units - 1 : 0, shift = mask ? __builtin_ctz(16 / units) : 0;

    // A x and the scale of this lane's place, as the matrix core takes them
    v4u v[STEPS][2];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v[s][h] = (v4u){0, 0, 0, 0};
            const int u = RS == 0 ? grp & 1 : 4 * s + grp, half = RS == 0 ? grp >> 1 : h;
            if (((all >> (mine16 + row16)) & 1) && u < units)
                v[s][h] = *reinterpret_cast<const v4u*>(a.halves + ((int64_t)(p0 + mine16 + row16) * 2 + half) * a.rank + 8 * u);
        }
    const float scale = scale_of(a, __shfl(mine.id, mine16 + row16, 64));
    const bool adds = (all >> (mine16 + row16)) & 1;
    // rows that this lane moves: 8 h + lane / 8 of the wave's, chunk lane % 8 in LDS
    const uint16_t* yp[2];
    uint16_t* op[2];
    bool stores[2];
    bool whole = true;                                       // every lane stores both, in a whole run
    const int chunk = ((lane & 7) ^ ((lane >> 3) & 7)) * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int from = mine16 + 8 * h + (lane >> 3);
        const int64_t row = row_of(mine.row, from);
        stores[h] = row >= 0 && (((all >> from) & 1) || a.Y != a.out);
        whole = whole && __builtin_amdgcn_ballot_w64(stores[h]) == ~uint64_t(0);
        yp[h] = a.Y + max(row, (int64_t)0) * a.ldy;
        op[h] = a.out + max(row, (int64_t)0) * a.ldo;
    }
    // the run of columns from n0 of an adapter into place `at` of the ring, and of Y's rows; past the last column the
    // last unit again
    int off[LOADS];
#pragma unroll
    for (int q = 0; q < LOADS; ++q) {
        const int x = min(wave * LOADS + q, units - 1) * 64 + lane, r = x / units, c = x - r * units;
        off[q] = r * units + (c ^ ((r >> shift) & mask));
    }
    auto issue = [&](int adapter, int n0, int at) {
        const uint16_t* bp = uniform_ptr(a.B + ((int64_t)adapter * a.N + n0) * a.R);
        const int last = min(64, a.N - n0) * units - 1;
#pragma unroll
        for (int q = 0; q < LOADS; ++q)                      // (spare ones repeat the last)
            dma_x4(base + at * RUN + min(wave * LOADS + q, units - 1) * 1024, bp, 16u * (uint32_t)min(off[q], last));
    };
    auto issue_y = [&](int n0, int at) {
#pragma unroll
        for (int h = 0; h < 2; ++h) dma_far(ybase + at * (kWaves * 2048) + h * 1024, yp[h] + min(n0 + chunk, a.N - 8));
    };
    uint64_t left = all;
    auto next = [&](uint64_t* its) {                         // the first adapter left, and its places
        const int adapter = __builtin_amdgcn_readlane(mine.id, __builtin_ctzll(left));
        *its = __builtin_amdgcn_ballot_w64(mine.id == adapter);
        left &= ~*its;
        return adapter;
    };
    int n0 = blockIdx.x * a.chunks * 64, at = 0, aty = 0;
    const int end_n = min(a.N, n0 + a.chunks * 64);
    uint64_t its = 0;
    if (all) issue(next(&its), n0, 0);
    issue_y(n0, 0);
    v4f acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = (v4f){0.f, 0.f, 0.f, 0.f};
    bool stored = false;                                     // the wave's last two memory operations are its stores
    while (n0 < end_n) {
        if (stored) wait_vmcnt<2>();
        else wait_vmcnt<0>();
        __syncthreads();
        // what comes after: this run's next adapter, or the first one's next run
        const bool same = left != 0;
        const int n1 = same ? n0 : n0 + 64;
        uint64_t its1 = 0;
        if (all) {
            if (!same) left = all;
            const int adapter1 = next(&its1);
            if (n1 < end_n) issue(adapter1, n1, at ^ 1);
        }
        if (!same && n1 < end_n) issue_y(n1, aty ^ 1);
        if ((its >> mine16) & 0xFFFF) {
            const uint8_t* st = ring + at * RUN;
            v4f p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int u = RS == 0 ? grp & 1 : 4 * s + grp, c = min(u, units - 1);
                v4u b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 16 * j + row16;
                    b[j] = *reinterpret_cast<const v4u*>(st + (r * units + (c ^ ((r >> shift) & mask))) * 16);
                    if (u >= units) b[j] = (v4u){0, 0, 0, 0};    // past the rank, in both operands
                }
#pragma unroll
                for (int h = RS == 0 ? 0 : 1; h >= 0; --h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = mfma_bf16(b[j], v[s][h], p[j]);
            }
            const bool here = (its >> (mine16 + row16)) & 1;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = here ? p[j][e] * scale : acc[j][e];
        }
        stored = false;
        if (!same) {
            uint8_t* yt = rows[aty][wave];
            // a lane has columns 16 j + 4 grp .. + 3 of row row16; rows without an adapter stay as they are
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint2* at2 = reinterpret_cast<uint2*>(yt + row16 * 128 + (((2 * j + (grp >> 1)) ^ (row16 & 7)) << 4) + (grp & 1) * 8);
                const uint2 y = *at2;
                if (adds)
                    *at2 = make_uint2(pack_bf16x2(__uint_as_float(y.x << 16) + acc[j][0], __uint_as_float(y.x & 0xFFFF0000u) + acc[j][1]),
                                      pack_bf16x2(__uint_as_float(y.y << 16) + acc[j][2], __uint_as_float(y.y & 0xFFFF0000u) + acc[j][3]));
                acc[j] = (v4f){0.f, 0.f, 0.f, 0.f};
            }
            wave_sync();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4u o = *reinterpret_cast<const v4u*>(yt + h * 1024 + lane * 16);
                if (stores[h] && n0 + chunk < a.N) *reinterpret_cast<v4u*>(op[h] + n0 + chunk) = o;
            }
            stored = whole && n0 + 64 <= a.N;
            aty ^= 1;
        }
        n0 = n1;
        at ^= 1;
        its = its1;
    }
}

template <int RT>
void launch_down64(const LoraArgs& a, hipStream_t s) {
    lora_down64_kernel<RT, RT <= 4 ? 4 : 3><<<dim3((uint32_t)a.splits, (uint32_t)((a.places + 63) / 64) << a.apart), kThreads, 0, s>>>(a);
}

template <int RS>
void launch_up(const LoraArgs& a, hipStream_t s) {
    const int span = (a.tile <= 16 ? kLoraSpan : 64) * a.chunks;
    const dim3 grid((uint32_t)((a.N + span - 1) / span), (uint32_t)((a.places + a.tile - 1) / a.tile));
    if (a.tile <= 16) lora_up_kernel<RS><<<grid, kThreads, 0, s>>>(a);
    else lora_up64_kernel<RS><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

void launch_lora_rows(const LoraArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)a.places);
    if (a.rank <= 16) lora_row_kernel<1><<<grid, kDownWaves * 64, 0, s>>>(a);
    else if (a.rank <= 32) lora_row_kernel<2><<<grid, kDownWaves * 64, 0, s>>>(a);
    else if (a.rank <= 64) lora_row_kernel<4><<<grid, kDownWaves * 64, 0, s>>>(a);
    else lora_row_kernel<8><<<grid, kDownWaves * 64, 0, s>>>(a);
}

void launch_lora_down(const LoraArgs& a, hipStream_t s) {
    if (a.tile <= 16) {
        const dim3 grid((uint32_t)a.splits, (uint32_t)((a.places + a.tile - 1) / a.tile), (uint32_t)((a.rank + 31) / 32));
        if (a.rank <= 16) lora_down_kernel<1, 4><<<grid, kDownWaves * 64, 0, s>>>(a);
        else lora_down_kernel<2, 4><<<grid, kDownWaves * 64, 0, s>>>(a);
    } else if (a.rank <= 16) {
        launch_down64<1>(a, s);
    } else if (a.rank <= 32) {
        launch_down64<2>(a, s);
    } else if (a.rank <= 64) {
        launch_down64<4>(a, s);
    } else {
        launch_down64<8>(a, s);
    }
}

void launch_lora_up(const LoraArgs& a, hipStream_t s) {
    if (a.rank <= 16) launch_up<0>(a, s);
    else if (a.rank <= 32) launch_up<1>(a, s);
    else if (a.rank <= 64) launch_up<2>(a, s);
    else launch_up<4>(a, s);
}

}  // namespace fp8gemm
