// gated_kernels.hip -- gfx950 kernels of the gated feed-forward block in bf16 and of its gradients:
//   H = act(X Wg^T) * (X Wu^T)          W [2I,K] = gate rows, then up rows
//   dg = dH u act'(g), du = dH act(g);  dX = [dg|du] W;  dW = [dg|du]^T X
// The mathematics and the limits are stated in include/fp8gemm.h.
//
// Four products with one body (product() below): the two with W's rows pair each gate row with its up row in one lane, so
// that the activation, or its gradient, is an epilogue; the other two read operands whose contraction runs along rows of
// memory with LDS's transposing reads, so nothing is transposed in memory.  dg and du are rounded to bf16 once, between
// the products, since the matrix cores take them so: dX and dW are off by 0.0024 of their norm with it, 0.0017 (their own
// rounding) without, and two halves of each value would double the operations of both products.  g and u, formed again,
// and all sums stay in fp32.
//
// What bounds them: large sizes the matrix cores and what feeds them.  H of 4096 rows, I = 2048, K = 7168 takes 180 us,
// 1.34 PFLOP/s (a library's plain product of the same matrices, in turn with it, 158 us; the matrix instructions alone, on
// the same data from registers, 143 us); its gradients 410 us, 1.17 PFLOP/s (a library's two products 425 us).  Middle
// sizes: how the tiles fill 256 CUs, and a tile's start and end (3 to 8 us); few rows: W's bytes, 1 row 10.7 us, 5.5 TB/s of
// them from HBM and the memory-side cache.

#include <algorithm>
#include <type_traits>

#include "ffn_internal.h"
#include "fp8gemm_device.h"
#include "moe_device.h"

namespace fp8gemm {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v4f mfma_bf16(const v4u& x, const v4u& y, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y), c, 0, 0, 0);
}

// Both activations are x times a logistic function of z(x): z = x (silu), or z = 2 sqrt(2/pi) (x + 0.044715 x^3)
// (gelu's tanh form, since 0.5 (1 + tanh(z / 2)) = 1 / (1 + e^-z)).  1 / (1 + e^-z) within 3 units in the last
// place: the exponential's error and the reciprocal's; below 2^-126 (z below -87) the reciprocal gives zero.
constexpr float kGeluA = 1.5957691216057308f, kGeluB = 0.044715f;

__device__ __forceinline__ float logistic(float x, bool gelu) {
    const float z = gelu ? kGeluA * __builtin_fmaf(kGeluB * x * x, x, x) : x;
    return __builtin_amdgcn_rcpf(1.0f + exp_f32(-z));
}
__device__ __forceinline__ float activation(float x, bool gelu) { return x * logistic(x, gelu); }
// act(x) and act'(x) = s + x s (1 - s) z'(x).  The second term vanishes long before |x| = 64; taken at the
// bounded x it cannot overflow.  Both bounds, this one and the exponential's, turn NaN into a number: act(x) has it
// again from its factor x, act'(x) is given it back.
__device__ __forceinline__ float activation_grad(float x, bool gelu, float* value) {
    const float s = logistic(x, gelu);
    const float xb = __builtin_amdgcn_fmed3f(x, -64.0f, 64.0f);
    const float dz = gelu ? kGeluA * __builtin_fmaf(3.0f * kGeluB * xb, xb, 1.0f) : 1.0f;
    *value = x * s;
    return __builtin_isnan(x) ? x : __builtin_fmaf(xb * s * (1.0f - s), dz, s);
}

__device__ __forceinline__ v2u pack4(const v4f& v) { return (v2u){pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)}; }
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Chunk permutation of a 128-byte LDS row, as in the FP8 kernel: 16-byte chunk c of row r stands at c ^ swz(r).
__device__ __forceinline__ int swz(int row) { return ((row >> 1) & 3) | ((((row >> 2) ^ (row >> 3)) & 1) << 2); }
// Permutation of the 32-byte runs (16 columns) of a turned row k of LDS: run u stands at u ^ turn(k).  A turned
// fragment read takes, in a half-wave, four consecutive rows at k and four at k + 16: eight different runs
// (four, in an operand of 64 columns).
template <int ROWS>
__device__ __forceinline__ int turn(int k) {
    static_assert(ROWS == 64 || ROWS % 128 == 0, "runs of a row: four, or a multiple of eight");
    return ((k & 3) | (((k >> 4) & 1) << 2)) & (ROWS / 16 - 1);
}

// One operand of a tile in LDS: ROWS rows (columns, if turned) of a slice of 64 values of k, ROWS * 128 bytes.
//   straight: row r holds its 64 values, 128 bytes, chunks permuted by swz(r)
//   turned:   row k holds ROWS values, runs permuted by turn(k)
// Lane l's fragment of 16 rows, matrix-core step s of 2: row l % 16, the 8 values of k from 16 (l / 16) + 8 s.
template <int ROWS, int NW, bool TURNED>
struct Operand {
    static constexpr int BYTES = ROWS * 128;
    static constexpr int LOADS = BYTES / 1024 / NW;          // 1 KB loads of a wave and slice
    static_assert(BYTES % (1024 * NW) == 0, "every wave loads the same number of KB");
    static constexpr int ROW_BYTES = TURNED ? ROWS * 2 : 128;
    static constexpr int PER_LOAD = 1024 / ROW_BYTES;        // rows of LDS in a load

    // Row of LDS and 16-byte chunk of the source that lane `lane` moves in load q of wave `wave`.
    static __device__ __forceinline__ int row(int wave, int q, int lane) {
        return (wave * LOADS + q) * PER_LOAD + lane / (ROW_BYTES / 16);
    }
    static __device__ __forceinline__ int chunk(int r, int lane) {
        const int p = lane % (ROW_BYTES / 16);
        return TURNED ? p ^ (turn<ROWS>(r) << 1) : p ^ swz(r);
    }
};

// LAG: a straight operand's rows do not start at 128-byte lines (product() below).
template <int BM_, int BN_, int WMW_, int WNW_, int STAGES_, int KIND_, bool LAG_>
struct Tile {
    static constexpr bool LAG = LAG_;
    static constexpr int BM = BM_, BN = BN_, WMW = WMW_, WNW = WNW_, STAGES = STAGES_, KIND = KIND_;
    static constexpr bool PT = KIND == kTurned, QT = KIND == kTimesW || KIND == kTurned;
    static constexpr bool GATED = KIND == kGated || KIND == kGatedBack;
    static constexpr int NW = WMW * WNW, NT = 64 * NW;
    static constexpr int WM = BM / WMW, WN = BN / WNW;
    static constexpr int JM = WM / 16, IN = WN / 16;
    using OpP = Operand<BM, NW, PT>;
    using OpQ = Operand<BN, NW, QT>;
    static constexpr int P_OFF = OpQ::BYTES;
    static constexpr int STAGE_BYTES = OpQ::BYTES + OpP::BYTES;
    static constexpr int NDMA = OpQ::LOADS + OpP::LOADS;
    static_assert(NDMA * (STAGES - 1) < 64, "vmcnt range");
    static_assert(!LAG || (STAGES >= 4 && !(PT && QT)), "a place of the ring to spare, and rows to use it");
    static constexpr int OUT_COLS = GATED ? BN / 2 : BN;     // columns of the output that a tile covers
    // epilogue: a wave's rows in an LDS region of its own, an odd number of 16-byte units apart
    static constexpr int W_COLS = OUT_COLS / WNW;
    static constexpr int CPR = W_COLS / 8;
    static constexpr int PITCH = 2 * W_COLS + (CPR % 2 == 0 ? 16 : 0);
    static constexpr int STG = WM * PITCH;
    static constexpr int SMEM = STAGES * STAGE_BYTES > NW * STG ? STAGES * STAGE_BYTES : NW * STG;
    static_assert(SMEM < 160 * 1024, "LDS budget");
    static constexpr int WAVES_PER_SIMD = NW / 4 * (SMEM < 40 * 1024 ? 4 : SMEM < 80 * 1024 ? 2 : 1);   // as LDS allows
};

// Unit `block` of the `blocks` of a product; smem: T::SMEM bytes.
template <class T>
__device__ __forceinline__ void product(const ProductArgs& a, int block, int blocks, uint8_t* smem, int& s_flag) {
    constexpr int BM = T::BM, BN = T::BN, WMW = T::WMW, STAGES = T::STAGES, KIND = T::KIND;
    using OpP = typename T::OpP;
    using OpQ = typename T::OpQ;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WMW, wn = wave / WMW;
    const int row16 = lane & 15, grp = lane >> 4;
    const uint32_t smem_base = lds_addr(smem);

    // Workgroups are dealt to the 8 XCDs in turn: those of one XCD take consecutive units, which share operands
    // in its L2.
    const int xcd = block & 7;
    const int unit = xcd * (blocks >> 3) + min(xcd, blocks & 7) + (block >> 3);
    // split fastest, then the M tile within a band of group_m of them, then the N tile
    const uint32_t tile = fast_div((uint32_t)unit, a.div_splits);
    const int split = unit - (int)tile * a.splits;
    const uint32_t band = fast_div(tile, a.div_band_units);
    const uint32_t inb = tile - band * a.div_band_units.d;
    const int band_m0 = (int)band * a.group_m;
    const FastDiv& bh = band_m0 + a.group_m <= a.tiles_m ? a.div_band_h : a.div_band_h_last;
    const uint32_t tq = fast_div(inb, bh);
    const int m0 = (band_m0 + (int)(inb - tq * bh.d)) * BM;
    const int n0 = (int)tq * T::OUT_COLS;                    // first output column
    const int s0 = split * a.per_split, nks = min(a.per_split, a.slices - s0);

    // LAG: a slice's 128 bytes of a row lie in two lines.  Those chunks of it that are in the second are loaded a slice
    // later, with the rest of their line, so that no line is loaded twice: place i of the ring holds line i of each
    // row, and slice i is read from places i and i + 1, in which every chunk stands where it would in a place of its own.
    // Measured, us, without and with, beside whole lines: H of 1001 rows, I = 1416, K = 3400 38, 28.9 and 26.2 (128 x 128),
    // 49, 38.8 and 32 (64 x 64).  A place less for loads on their way costs where few are: 128 rows, K = 3400, 64 x 64 tiles
    // 11.9 and 14.2.
    constexpr int lag = T::LAG;
    const int lines = nks + lag;
    const int tail = a.K - (a.slices - 1) * 64;              // values of the last slice
    const int tail_at = tail < 64 ? a.slices - 1 - s0 : -1;  // this unit's slice that is not whole
    // whether chunk c of row r comes with the next slice (tiles, and a tile's 16 rows, start at multiples of 8)
    auto late = [](const uint16_t* p, int ld, int r, int c) {
        return c + (int)(((uint32_t)(reinterpret_cast<uintptr_t>(p) >> 4) + (uint32_t)r * (uint32_t)(ld >> 3)) & 7) >= 8;
    };
    auto late_p = [&](int r, int c) { return T::LAG && !T::PT && late(a.P, a.ldp, r, c); };
    auto late_q = [&](int r, int c) { return T::LAG && !T::QT && late(a.Q, a.ldq, r, c); };

    // ---- what each lane loads: byte offsets from a line's bases ----------------------------------------------
    // rows and columns past the end repeat the last (their results are not stored), and so do slices and values
    auto values = [&](int slice) { return slice == tail_at ? tail : 64; };
    auto k_off = [&](int line, bool late, int c) {
        if constexpr (!T::LAG) return (uint32_t)(2 * min(8 * c, values(line) - 8));
        const int slice = min(max(line - (int)late, 0), nks - 1);
        return (uint32_t)(128 * (slice - line + lag) + 2 * min(8 * c, values(slice) - 8));
    };
    auto p_off = [&](int q, int line) -> uint32_t {
        const int r = OpP::row(wave, q, lane), c = OpP::chunk(r, lane);
        if constexpr (T::PT) return (uint32_t)min(r, values(line) - 1) * (uint32_t)(2 * a.ldp) + (uint32_t)(2 * min(m0 + 8 * c, a.rows - 8));
        else return (uint32_t)min(r, a.rows - 1 - m0) * (uint32_t)(2 * a.ldp) + k_off(line, late_p(r, c), c);
    };
    auto q_off = [&](int q, int line) -> uint32_t {
        const int r = OpQ::row(wave, q, lane), c = OpQ::chunk(r, lane);
        if constexpr (T::QT) {
            const int there = values(T::LAG ? min(line, nks - 1) : line);
            return (uint32_t)min(r, there - 1) * (uint32_t)(2 * a.ldq) + (uint32_t)(2 * min(n0 + 8 * c, a.cols - 8));
        } else {
            // gate and up rows in turn, 16 each, so that a lane ends with a pair of them (up: qs below)
            const int n = min(((r >> 5) << 4) + (r & 15), a.cols - 1 - n0);
            return (uint32_t)n * (uint32_t)(2 * a.ldq) + k_off(line, late_q(r, c), c);
        }
    };
    uint32_t poff[OpP::LOADS], qoff[OpQ::LOADS];
#pragma unroll
    for (int q = 0; q < OpP::LOADS; ++q) poff[q] = p_off(q, -1);
#pragma unroll
    for (int q = 0; q < OpQ::LOADS; ++q) qoff[q] = q_off(q, -1);
    const uint16_t* pbase = a.P + (T::PT ? (int64_t)s0 * 64 * a.ldp : (int64_t)m0 * a.ldp + ((int64_t)s0 - lag) * 64);
    const uint16_t* qbase = a.Q + (T::QT ? (int64_t)s0 * 64 * a.ldq : (int64_t)n0 * a.ldq + ((int64_t)s0 - lag) * 64);
    const int64_t pstep = T::PT ? (int64_t)64 * a.ldp : 64, qstep = T::QT ? (int64_t)64 * a.ldq : 64;
    const int64_t up = (int64_t)a.cols * a.ldq;              // gated: from a gate row to its up row

    // load x of line i (of a wave's NDMA: Q's, then P's)
    auto issue = [&](int i, int x) {
        const uint32_t st = smem_base + (uint32_t)((i % STAGES) * T::STAGE_BYTES);
        if (x < OpQ::LOADS) {
            const int l = wave * OpQ::LOADS + x;
            const uint16_t* from = qbase + (T::LAG && T::QT ? min(i, nks - 1) : i) * qstep + (T::GATED && (l >> 1 & 1) ? up : 0);
            dma_x4(st + l * 1024, uniform_ptr(from), qoff[x]);
        } else {
            const int l = wave * OpP::LOADS + x - OpQ::LOADS;
            dma_x4(st + T::P_OFF + l * 1024, uniform_ptr(pbase + i * pstep), poff[x - OpQ::LOADS]);
        }
    };
    // before the loads of line i, in order: the first and the last are not like the others
    const int special = tail_at >= 0 ? min(tail_at, nks) : nks;
    auto aim = [&](int i) {
        if (T::LAG ? i > 1 && i < special : i != tail_at) return;
#pragma unroll
        for (int q = 0; q < OpP::LOADS; ++q) poff[q] = p_off(q, i);
#pragma unroll
        for (int q = 0; q < OpQ::LOADS; ++q) qoff[q] = q_off(q, i);
    };
    // zeros in both operands for the values of k that the last slice does not have
    auto clear_tail = [&](int i) {
        const int here = (i % STAGES) * T::STAGE_BYTES, next = ((i + lag) % STAGES) * T::STAGE_BYTES;
        auto clear = [&](int part, int rows, bool turned, int row_bytes, auto comes_late) {
            if (turned) {
                for (int o = tail * row_bytes + tid * 16; o < 64 * row_bytes; o += T::NT * 16)
                    *reinterpret_cast<v4u*>(smem + here + part + o) = (v4u){0, 0, 0, 0};
            } else {
                for (int x = tid; x < rows * 8; x += T::NT) {
                    const int r = x >> 3, c = x & 7;
                    uint8_t* at = smem + (comes_late(r, c) ? next : here) + part + r * 128 + ((c ^ swz(r)) << 4);
                    if (c * 8 >= tail) *reinterpret_cast<v4u*>(at) = (v4u){0, 0, 0, 0};
                }
            }
        };
        clear(0, BN, T::QT, OpQ::ROW_BYTES, late_q);
        clear(T::P_OFF, BM, T::PT, OpP::ROW_BYTES, late_p);
        __syncthreads();
    };

    v4f acc[T::IN][T::JM];
#pragma unroll
    for (int i = 0; i < T::IN; ++i)
#pragma unroll
        for (int j = 0; j < T::JM; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

    const int straight[2] = {((2 * grp) ^ swz(row16)) << 4, ((2 * grp + 1) ^ swz(row16)) << 4};
    const int tk = 16 * grp + (row16 >> 2);                   // a turned read's row of LDS
    const int turned_lane = (lane & 3) * 8, tp = turn<BM>(tk) << 5, tqr = turn<BN>(tk) << 5;   // and its permutations
    const bool plate[2] = {late_p(row16, 2 * grp), late_p(row16, 2 * grp + 1)}, qlate[2] = {late_q(row16, 2 * grp), late_q(row16, 2 * grp + 1)};
    auto fragment = [&](const uint8_t* part, int row0, int s, bool turned, int row_bytes, int tx) -> v4u {
        if (!turned) return *reinterpret_cast<const v4u*>(part + (row0 + row16) * 128 + straight[s]);
        const uint8_t* p = part + ((row0 << 1) ^ tx) + (tk + 8 * s) * row_bytes + turned_lane;
        typedef __attribute__((address_space(3))) v4s* lds_v4s;
        const v2u lo = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p)));
        const v2u hi = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + 4 * row_bytes)));
        return (v4u){lo.x, lo.y, hi.x, hi.y};
    };
    // Fragments of a matrix-core step, P's first
    struct Step {
        v4u f[T::JM + T::IN];
    };
    auto fragment_p = [&](int i, int x, int s, int xp) {
        const uint8_t *here = smem + (i % STAGES) * T::STAGE_BYTES, *next = smem + ((i + lag) % STAGES) * T::STAGE_BYTES;
        return fragment((T::LAG && plate[s] ? next : here) + T::P_OFF, wm * T::WM + 16 * x, s, T::PT, OpP::ROW_BYTES, xp);
    };
    auto fragment_q = [&](int i, int x, int s, int xq) {
        const uint8_t *here = smem + (i % STAGES) * T::STAGE_BYTES, *next = smem + ((i + lag) % STAGES) * T::STAGE_BYTES;
        return fragment(T::LAG && qlate[s] ? next : here, wn * T::WN + 16 * x, s, T::QT, OpQ::ROW_BYTES, xq);
    };
    // The products of the fragments in `from` and, in groups between them, reads of the fragments of step s of slice
    // i and the loads of slice i2 (load 1: if there is one, 2: there is): the matrix core, LDS and the loads' issue work side by side.
    auto products = [&](const Step& from, Step& to, int i, int s, auto load, int i2) {
        constexpr bool LOAD = decltype(load)::value != 0, CERTAIN = decltype(load)::value == 2;
        constexpr int READS = T::JM + T::IN, MFMAS = T::JM * T::IN, GROUPS = LOAD && T::NDMA > 4 ? T::NDMA : 4;
        // (opaque: an address for each fragment, formed ahead of the loop, costs registers that spill)
        int xp = tp, xq = tqr;
        if constexpr (T::PT) asm volatile("" : "+v"(xp));
        if constexpr (T::QT) asm volatile("" : "+v"(xq));
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
#pragma unroll
            for (int x = READS * g / GROUPS; x < READS * (g + 1) / GROUPS; ++x)
                to.f[x] = x < T::JM ? fragment_p(i, x, s, xp) : fragment_q(i, x - T::JM, s, xq);
            if constexpr (LOAD) {
#pragma unroll
                for (int x = T::NDMA * g / GROUPS; x < T::NDMA * (g + 1) / GROUPS; ++x)
                    if (CERTAIN || i2 < lines) issue(i2, x);
            }
#pragma unroll
            for (int x = MFMAS * g / GROUPS; x < MFMAS * (g + 1) / GROUPS; ++x)
                acc[x / T::JM][x % T::JM] = mfma_bf16(from.f[T::JM + x / T::JM], from.f[x % T::JM], acc[x / T::JM][x % T::JM]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // Slices (their lines) stand in a ring of STAGES.  The second step's fragments of a slice are read during the products of
    // its first, then the slice's place is free for slice i + STAGES, and the next slice's first step is read
    // during the products of the second: a wave's matrix core works across the barrier.
    Step f0, f1;
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
        if (i >= lines) continue;
        aim(i);
#pragma unroll
        for (int x = 0; x < T::NDMA; ++x) issue(i, x);
    }
    wait_slices<T::NDMA, STAGES - 1, 0>(min(STAGES - 1 - lag, nks - 1));
    __syncthreads();
    if (tail_at == 0) clear_tail(0);
#pragma unroll
    for (int x = 0; x < T::JM + T::IN; ++x)
        f0.f[x] = x < T::JM ? fragment_p(0, x, 0, tp) : fragment_q(0, x - T::JM, 0, tqr);
    using load = std::integral_constant<int, 1>;
    using load_surely = std::integral_constant<int, 2>;
    using none = std::integral_constant<int, 0>;
    int i = 0;
    // slices with a whole line to load, without a branch
    const int steady = special - STAGES;
    for (; i < steady; ++i) {
        products(f0, f1, i, 1, none{}, 0);
        wait_vmcnt<T::NDMA * (STAGES - 2 - lag)>();
        __syncthreads();
        products(f1, f0, i + 1, 0, load_surely{}, i + STAGES);
    }
    for (; i < nks; ++i) {
        products(f0, f1, i, 1, none{}, 0);
        if (i + 1 < nks) {
            wait_slices<T::NDMA, STAGES - 2, 0>(min(STAGES - 2 - lag, nks - 2 - i));
            __syncthreads();
            aim(i + STAGES);
            if (i + 1 == tail_at) clear_tail(i + 1);
        }
        products(f1, f0, min(i + 1, nks - 1), 0, load{}, i + STAGES);
    }

    // ---- K splits: the last workgroup of a tile to arrive sums the partials in split order -------------------
    // (written and read past the L2s of the XCDs, with agent-coherent accesses; the counter goes back to zero)
    if (a.splits > 1) {
        const __amdgpu_buffer_rsrc_t ws = __builtin_amdgcn_make_buffer_rsrc(
            uniform_ptr(a.ws + (int64_t)tile * a.splits * (BM * BN)), 0, a.splits * BM * BN * 4, kBufferFlags);
        const int own = (wave * (T::WM * T::WN) + lane * 4) * 4;
#pragma unroll
        for (int i2 = 0; i2 < T::IN; ++i2)
#pragma unroll
            for (int j = 0; j < T::JM; ++j)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, acc[i2][j]), ws,
                                                       own + (split * BM * BN + (i2 * T::JM + j) * 256) * 4, 0, kSc1);
        wait_vmcnt<0>();
        __syncthreads();
        if (tid == 0) {
            const int old = __hip_atomic_fetch_add(a.counters + tile * (uint32_t)a.spread, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            s_flag = old == a.splits - 1;
            if (old == a.splits - 1)
                __hip_atomic_store(a.counters + tile * (uint32_t)a.spread, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!s_flag) return;
        for (int s = 0; s < a.splits; ++s) {
#pragma unroll
            for (int i2 = 0; i2 < T::IN; ++i2) {
                v4f x[T::JM];
#pragma unroll
                for (int j = 0; j < T::JM; ++j)
                    x[j] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(
                        ws, own + (s * BM * BN + (i2 * T::JM + j) * 256) * 4, 0, kSc1));
#pragma unroll
                for (int j = 0; j < T::JM; ++j) acc[i2][j] = s == 0 ? x[j] : acc[i2][j] + x[j];
            }
        }
    }

    // ---- epilogue -------------------------------------------------------------------------------------------
    // a lane holds 4 consecutive columns of row 16 j + row16 of its wave's rows, for each of its 16-column tiles
    uint8_t* stg = smem + wave * T::STG;
    const int wrow0 = m0 + wm * T::WM, wcol0 = n0 + wn * T::W_COLS;
    // whole 16-byte chunks of rows from the wave's region (its own LDS operations run in order)
    auto store = [&](uint16_t* dst, int64_t ld, int shift) {
        wave_sync();
#pragma unroll
        for (int x0 = 0; x0 < T::WM * T::CPR; x0 += 64) {
            const int x = x0 + lane, r = x / T::CPR, c = x % T::CPR;
            if (r < T::WM && wrow0 + r < a.rows && wcol0 + 8 * c < a.cols)
                *reinterpret_cast<v4u*>(dst + (int64_t)(wrow0 + r) * ld + shift + wcol0 + 8 * c) =
                    *reinterpret_cast<const v4u*>(stg + r * T::PITCH + c * 16);
        }
        wave_sync();
    };
    auto put = [&](int i, int j, const v4f& v) {
        *reinterpret_cast<v2u*>(stg + (16 * j + row16) * T::PITCH + (16 * i + 4 * grp) * 2) = pack4(v);
    };
    __syncthreads();                                         // every wave is past its last slice
    if constexpr (!T::GATED) {
#pragma unroll
        for (int i = 0; i < T::IN; ++i)
#pragma unroll
            for (int j = 0; j < T::JM; ++j) put(i, j, acc[i][j]);
        store(a.out, a.cols, 0);
    } else if constexpr (KIND == kGated) {
        if (a.pre) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int i = 0; i < T::IN / 2; ++i)
#pragma unroll
                    for (int j = 0; j < T::JM; ++j) put(i, j, acc[2 * i + half][j]);
                store(a.pre, 2 * (int64_t)a.cols, half * a.cols);
            }
        }
#pragma unroll
        for (int i = 0; i < T::IN / 2; ++i)
#pragma unroll
            for (int j = 0; j < T::JM; ++j) {
                v4f h;
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = activation(acc[2 * i][j][e], a.gelu) * acc[2 * i + 1][j][e];
                put(i, j, h);
            }
        store(a.out, a.cols, 0);
    } else {
        // dg in the place of the gate's sums, du in the up's
#pragma unroll
        for (int i = 0; i < T::IN / 2; ++i)
#pragma unroll
            for (int j = 0; j < T::JM; ++j) {
                const int r = wrow0 + 16 * j + row16, n = wcol0 + 16 * i + 4 * grp;
                v2u d = {0, 0};
                if (r < a.rows && n < a.cols) d = *reinterpret_cast<const v2u*>(a.dH + (int64_t)r * a.cols + n);
                const float dh[4] = {low_bf16(d.x), high_bf16(d.x), low_bf16(d.y), high_bf16(d.y)};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float act;
                    const float der = activation_grad(acc[2 * i][j][e], a.gelu, &act);
                    acc[2 * i][j][e] = dh[e] * acc[2 * i + 1][j][e] * der;
                    acc[2 * i + 1][j][e] = dh[e] * act;
                }
            }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int i = 0; i < T::IN / 2; ++i)
#pragma unroll
                for (int j = 0; j < T::JM; ++j) put(i, j, acc[2 * i + half][j]);
            store(a.pre, 2 * (int64_t)a.cols, half * a.cols);
        }
    }
}

template <class T>
__global__ __launch_bounds__(T::NT, T::WAVES_PER_SIMD) void product_kernel(const ProductArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::SMEM];
    __shared__ int s_flag;
    product<T>(a, blockIdx.x, gridDim.x, smem, s_flag);
}

// Two products that need nothing of each other, as one launch: the second's workgroups fill the CUs that the first's
// last ones leave.
template <class T, class T2>
__global__ __launch_bounds__(T::NT, T::WAVES_PER_SIMD) void product_pair_kernel(const ProductArgs a, const ProductArgs b) {
    static_assert(T::NT == T2::NT && T::SMEM == T2::SMEM, "one shape");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::SMEM];
    __shared__ int s_flag;
    const int first = a.tiles_m * a.tiles_n * a.splits;
    if ((int)blockIdx.x < first) product<T>(a, blockIdx.x, first, smem, s_flag);
    else product<T2>(b, blockIdx.x - first, gridDim.x - first, smem, s_flag);
}

// ---- the block for few rows -----------------------------------------------------------------------------
// A workgroup has 8 output columns, whose 8 gate rows and 8 up rows of W are the 16 rows of one matrix-core
// operand; X's rows are the other's.  Its 8 waves take the steps of K (64 values, a 128-byte line of a row) in turn, two on
// their way each; their sums meet in LDS and are added in wave order.  With dH the sums' gradients go to `pre`.
// Bound by W's bytes: I = 2048, K = 7168, us, 1 row 10.6, 8 rows 13.0.
constexpr int kRowsWaves = 8, kRowsAhead = 2;

__global__ __launch_bounds__(kRowsWaves * 64, 2) void gated_rows_kernel(const GatedRowsArgs a) {
    __shared__ v4f red[kRowsWaves][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row16 = lane & 15, grp = lane >> 4;
    const int n0 = blockIdx.x * 8, here = min(8, a.I - n0);
    const int K2 = a.K * 2, steps = (a.K + 63) / 64;

    // gate rows n0.. and up rows I + n0..: one buffer from the first gate row to the last up row
    const __amdgpu_buffer_rsrc_t wb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(uniform_ptr(a.W + (int64_t)n0 * a.K)), 0, (a.I + here) * K2, kBufferFlags);
    const __amdgpu_buffer_rsrc_t xb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(a.X), 0, a.M * K2, kBufferFlags);
    const int wrow = (min(row16 & 7, here - 1) + (row16 >> 3) * a.I) * K2 + grp * 32;
    const int xrow = min(row16, a.M - 1) * K2 + grp * 32;

    v4f acc = {0.f, 0.f, 0.f, 0.f};
    // a step's 64 values of k: lane group grp has 16 of them, in halves for two matrix-core steps
    struct Slot {
        v4u w[2], x[2];
    };
    Slot ring[kRowsAhead];
    auto load = [&](Slot& s, int step) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = step * 128 + h * 16;
            const bool in = k + grp * 32 < K2;               // else past the buffer, which reads as zeros
            s.w[h] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(wb, in ? wrow + k : -16, 0, 0));
            s.x[h] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(xb, in ? xrow + k : -16, 0, 0));
        }
    };
#pragma unroll
    for (int p = 0; p < kRowsAhead; ++p) load(ring[p], wave + p * kRowsWaves);
    for (int s0 = wave; s0 < steps; s0 += kRowsWaves * kRowsAhead) {
#pragma unroll
        for (int p = 0; p < kRowsAhead; ++p) {
#pragma unroll
            for (int h = 0; h < 2; ++h) acc = mfma_bf16(ring[p].w[h], ring[p].x[h], acc);
            load(ring[p], s0 + (p + kRowsAhead) * kRowsWaves);
        }
    }
    red[wave][lane] = acc;
    __syncthreads();
    // output (row m, column n0 + c): gate sum in lane 16 (c / 4) + m, element c % 4; up sum 32 lanes on
    for (int x = tid; x < 8 * a.M; x += kRowsWaves * 64) {
        const int c = x & 7, m = x >> 3;
        if (c >= here) continue;
        const int from = 16 * (c >> 2) + m;
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < kRowsWaves; ++w) {
            g += red[w][from][c & 3];
            u += red[w][from + 32][c & 3];
        }
        if (a.dH) {
            const float d = bf16_to_f32(a.dH[(int64_t)m * a.I + n0 + c]);
            float act;
            const float der = activation_grad(g, a.gelu, &act);
            g = d * u * der;
            u = d * act;
        } else {
            a.out[(int64_t)m * a.I + n0 + c] = f32_to_bf16(activation(g, a.gelu) * u);
        }
        if (a.pre) {
            a.pre[(int64_t)m * 2 * a.I + n0 + c] = f32_to_bf16(g);
            a.pre[(int64_t)m * 2 * a.I + a.I + n0 + c] = f32_to_bf16(u);
        }
    }
}

// ---- gradients of kept products: 8 values of a row a thread, a pass at the rate of a copy ----------------
__global__ __launch_bounds__(256) void gated_grad_kernel(const GatedGradArgs a) {
    const int64_t unit = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (unit >= a.units) return;
    const uint32_t per_row = (uint32_t)a.I / 8;
    const int64_t row = unit < (int64_t(1) << 31) ? (int64_t)fast_div((uint32_t)unit, a.div_row) : unit / per_row;
    const int n = (int)(unit - row * per_row) * 8;
    const uint16_t* pre = a.pre + row * 2 * a.I + n;
    const v4u g4 = *reinterpret_cast<const v4u*>(pre), u4 = *reinterpret_cast<const v4u*>(pre + a.I);
    const v4u d4 = *reinterpret_cast<const v4u*>(a.dH + row * a.I + n);
    v4u og, ou;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float act0, act1;
        const float der0 = activation_grad(low_bf16(g4[i]), a.gelu, &act0);
        const float der1 = activation_grad(high_bf16(g4[i]), a.gelu, &act1);
        og[i] = pack_bf16x2(low_bf16(d4[i]) * low_bf16(u4[i]) * der0, high_bf16(d4[i]) * high_bf16(u4[i]) * der1);
        ou[i] = pack_bf16x2(low_bf16(d4[i]) * act0, high_bf16(d4[i]) * act1);
    }
    uint16_t* dp = a.dpre + row * 2 * a.I + n;
    *reinterpret_cast<v4u*>(dp) = og;
    *reinterpret_cast<v4u*>(dp + a.I) = ou;
}

__global__ __launch_bounds__(256) void fill_zero_kernel(v4u* p, int64_t units) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < units; i += (int64_t)gridDim.x * 256) p[i] = (v4u){0, 0, 0, 0};
}

// A wave's part is 128 x 64 of the largest tile, 64 x 64 or 64 x 32 of the next, 32 x 32 of the smallest.  Larger tiles
// bring less into LDS for a product; their rings are as long as LDS allows.  Measured, us a slice of 64 of K: kTiles.
template <int KIND, bool LAG>
using Tile256 = Tile<256, 256, 2, 4, 2, KIND, false>;
template <int KIND, bool LAG>
using Tile128x256 = Tile<128, 256, 2, 4, 3, KIND, false>;
template <int KIND, bool LAG>
using Tile128 = Tile<128, 128, 2, 4, 4, KIND, LAG && KIND != kTurned>;
template <int KIND, bool LAG>
using Tile64 = Tile<64, 64, 2, 2, 4, KIND, LAG && KIND != kTurned>;

template <int KIND>
using Tile64Short = Tile<64, 64, 2, 2, 2, KIND, false>;

uint32_t units(const ProductArgs& a) { return (uint32_t)(a.tiles_m * a.tiles_n * a.splits); }

template <class T>
void launch_one(const ProductArgs& a, hipStream_t s) {
    product_kernel<T><<<dim3(units(a)), T::NT, 0, s>>>(a);
}

template <int KIND>
void launch_kind(const ProductArgs& a, int shape, hipStream_t s) {
    if (shape == 0) launch_one<Tile256<KIND, false>>(a, s);
    else if (shape == 1) launch_one<Tile128x256<KIND, false>>(a, s);
    else if (shape == 2 && a.lag) launch_one<Tile128<KIND, true>>(a, s);
    else if (shape == 2) launch_one<Tile128<KIND, false>>(a, s);
    else if (shape == 3 && a.lag) launch_one<Tile64<KIND, true>>(a, s);
    else if (shape == 3) launch_one<Tile64<KIND, false>>(a, s);
    else if constexpr (KIND == kTimesW || KIND == kTurned) launch_one<Tile64Short<KIND>>(a, s);
}

// the longer units first
template <class TX, class TW>
void launch_two(const ProductArgs& x, const ProductArgs& w, hipStream_t s) {
    const dim3 grid(units(x) + units(w));
    if (x.per_split >= w.per_split) product_pair_kernel<TX, TW><<<grid, TW::NT, 0, s>>>(x, w);
    else product_pair_kernel<TW, TX><<<grid, TW::NT, 0, s>>>(w, x);
}

}  // namespace

void launch_product(const ProductArgs& a, Product kind, int shape, hipStream_t s) {
    switch (kind) {
        case kGated: return launch_kind<kGated>(a, shape, s);
        case kGatedBack: return launch_kind<kGatedBack>(a, shape, s);
        case kTimesW: return launch_kind<kTimesW>(a, shape, s);
        case kTurned: return launch_kind<kTurned>(a, shape, s);
    }
}

void launch_gradients(const ProductArgs& x, const ProductArgs& w, int shape, hipStream_t s) {
    if (shape == 0) launch_two<Tile256<kTimesW, false>, Tile256<kTurned, false>>(x, w, s);
    else if (shape == 1) launch_two<Tile128x256<kTimesW, false>, Tile128x256<kTurned, false>>(x, w, s);
    else if (shape == 2 && x.lag) launch_two<Tile128<kTimesW, true>, Tile128<kTurned, false>>(x, w, s);
    else if (shape == 2) launch_two<Tile128<kTimesW, false>, Tile128<kTurned, false>>(x, w, s);
    else if (shape == 3 && x.lag) launch_two<Tile64<kTimesW, true>, Tile64<kTurned, false>>(x, w, s);
    else if (shape == 3) launch_two<Tile64<kTimesW, false>, Tile64<kTurned, false>>(x, w, s);
    else launch_two<Tile64Short<kTimesW>, Tile64Short<kTurned>>(x, w, s);
}

void launch_gated_rows(const GatedRowsArgs& a, hipStream_t s) {
    gated_rows_kernel<<<dim3((uint32_t)((a.I + 7) / 8)), kRowsWaves * 64, 0, s>>>(a);
}

void launch_gated_grad(const GatedGradArgs& a, hipStream_t s) {
    gated_grad_kernel<<<dim3((uint32_t)((a.units + 255) / 256)), 256, 0, s>>>(a);
}

void launch_fill_zero(void* p, int64_t bytes, hipStream_t s) {
    const int64_t units = bytes / 16;
    fill_zero_kernel<<<dim3((uint32_t)std::min<int64_t>((units + 255) / 256, 2048)), 256, 0, s>>>(static_cast<v4u*>(p), units);
}

}  // namespace fp8gemm
