// lora_kernels.hip -- gfx950 kernels of low-rank adapters of many requests beside a shared projection:
//   out[t] = bf16(Y[t] + s[a] * B[a] (A[a] x[t])),  a = ids[t] the adapter of row t, or none.
// Two launches: the rank-R products A x, in fp32 through the workspace, then B's product, the sum and the store.
//
// Both take the rows by tiles of 16 places (places are rows, or positions in the order the caller gives) and go
// through the adapters that a tile's rows have, one after the other; matrix-core columns of rows with another
// adapter are left out of the results.  So any mix of rows is right, and one whose neighbours share an adapter
// reads each of its matrices once per tile.

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

// RT: 16-row tiles of A (rank / 16, rounded up to a power of two); MT: 16-place tiles of a workgroup.
// Its waves share the split's steps of 64 values of K; their sums meet in LDS and are added in wave order.
template <int RT, int MT>
__global__ __launch_bounds__(kThreads) void lora_down_kernel(const LoraArgs a) {
    __shared__ v4f red[kWaves][RT * MT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row16 = lane & 15, grp = lane >> 4;
    const int p0 = blockIdx.y * (16 * MT);
    const int split = blockIdx.x;
    const int step0 = split * a.per_split, step1 = min(a.steps, step0 + a.per_split);

    // lane l knows place p0 + l
    const Place mine = lane < 16 * MT ? place_of(a, p0 + lane, split == 0 && wave == 0) : Place{-1, -1};
    // rows of this lane's matrix-core columns (any row where there is none: the column is left out)
    const uint16_t* xp[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int from = 16 * m + row16;
        const int lo = __shfl((int)(uint32_t)mine.row, from, 64), hi = __shfl((int)(mine.row >> 32), from, 64);
        const int64_t row = max(((int64_t)hi << 32) | (uint32_t)lo, (int64_t)0);
        xp[m] = a.X + row * a.ldx + grp * 16;
    }
    uint64_t left = __builtin_amdgcn_ballot_w64(mine.id >= 0);
    while (left) {
        const int first = __builtin_ctzll(left);
        const int adapter = __builtin_amdgcn_readlane(mine.id, first);
        const uint64_t has = __builtin_amdgcn_ballot_w64(mine.id == adapter);
        left &= ~has;
        const uint16_t* ap[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            ap[r] = a.A + ((int64_t)adapter * a.R + min(16 * r + row16, a.R - 1)) * a.K + grp * 16;
        v4f acc[RT][MT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[r][m] = (v4f){0.f, 0.f, 0.f, 0.f};
        for (int step = step0 + wave; step < step1; step += kWaves) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = step * 64 + h * 8;
                const bool in = k + grp * 16 < a.K;              // else zeros in both operands
                const int ko = in ? k : 0;
                v4u af[RT], xf[MT];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    af[r] = (v4u){0, 0, 0, 0};
                    if (in) af[r] = *reinterpret_cast<const v4u*>(ap[r] + ko);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    xf[m] = (v4u){0, 0, 0, 0};
                    if (in && ((has >> (16 * m)) & 0xFFFF)) xf[m] = *reinterpret_cast<const v4u*>(xp[m] + ko);
                }
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int m = 0; m < MT; ++m) acc[r][m] = mfma_bf16(af[r], xf[m], acc[r][m]);
            }
        }
        __syncthreads();                                     // the sums of the adapter before are read
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int m = 0; m < MT; ++m) red[wave][r * MT + m][lane] = acc[r][m];
        __syncthreads();
        // tile x of RT * MT: lane holds values 16 r + 4 grp .. + 3 of its column's row
#pragma unroll
        for (int x0 = 0; x0 < RT * MT; x0 += kWaves) {
            const int x = x0 + wave;
            if (x >= RT * MT) break;
            const int r = x / MT, m = x % MT;
            if (16 * r >= a.rank || !((has >> (16 * m + row16)) & 1)) continue;
            v4f v = red[0][x][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += red[w][x][lane];
            *reinterpret_cast<v4f*>(a.low + ((int64_t)split * a.places + p0 + 16 * m + row16) * a.rank + 16 * r + 4 * grp) = v;
        }
    }
}

// MT: 16-place tiles of a workgroup.  A wave has 64 columns: matrix-core row m of tile j is column
// 16 (m / 4) + 4 j + m % 4 of them, so that a lane ends with 16 neighbours of one row.
// A x stands in LDS as two bf16 halves, whose sum is within 2^-17 of it: the matrix core takes 16 values of the
// rank a step, the high halves in lanes 0 to 31, the low ones in lanes 32 to 63, against the same values of B.
template <int MT>
__global__ __launch_bounds__(kThreads) void lora_up_kernel(const LoraArgs a) {
    extern __shared__ v4u low[];                             // [half][16 MT places][rank + 8]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row16 = lane & 15, grp = lane >> 4;
    const int p0 = blockIdx.y * (16 * MT);
    const int n0 = blockIdx.x * kLoraSpan + wave * 64;
    const int pitch = a.rank / 8 + 1;                        // 16-byte units of a place
    const Place mine = lane < 16 * MT ? place_of(a, p0 + lane, false) : Place{-1, -1};

    // sums of the splits' parts: four threads take a float4 of a place, every fourth split each
    {
        const int per_place = a.rank / 4;
        for (int x = tid >> 2; x < 16 * MT * per_place; x += kThreads / 4) {
            const int p = x / per_place, c = x - p * per_place;
            const int pid = __shfl(mine.id, p, 64);
            v4f v = {0.f, 0.f, 0.f, 0.f};
            if (pid >= 0)
                for (int s = tid & 3; s < a.splits; s += 4)
                    v += *reinterpret_cast<const v4f*>(a.low + ((int64_t)s * a.places + p0 + p) * a.rank + 4 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] += dpp16f<kDppXor1>(v[e]);
                v[e] += dpp16f<kDppXor2>(v[e]);
            }
            if ((tid & 3) == 0) {
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    hi[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
                    lo[e] = pack_bf16x2(v[2 * e] - __uint_as_float(hi[e] << 16), v[2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u));
                }
                uint32_t* d = reinterpret_cast<uint32_t*>(low + p * pitch) + 2 * c;
                d[0] = hi[0];
                d[1] = hi[1];
                d += 16 * MT * pitch * 4;
                d[0] = lo[0];
                d[1] = lo[1];
            }
        }
    }
    __syncthreads();
    if (n0 >= a.N) return;

    v4f acc[4][MT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = (v4f){0.f, 0.f, 0.f, 0.f};
    int id[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) id[m] = __shfl(mine.id, 16 * m + row16, 64);
    uint64_t left = __builtin_amdgcn_ballot_w64(mine.id >= 0);
    while (left) {
        const int first = __builtin_ctzll(left);
        const int adapter = __builtin_amdgcn_readlane(mine.id, first);
        left &= ~__builtin_amdgcn_ballot_w64(mine.id == adapter);
        const float scale = a.scales ? a.scales[adapter] : 1.0f;
        v4f part[4][MT];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m) part[j][m] = (v4f){0.f, 0.f, 0.f, 0.f};
        const uint16_t* bp[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = min(n0 + 16 * (row16 >> 2) + 4 * j + (row16 & 3), a.N - 1);
            bp[j] = a.B + ((int64_t)adapter * a.N + n) * a.R + (grp & 1) * 8;
        }
        for (int r = 0; r < a.rank; r += 16) {
            const bool in = r + (grp & 1) * 8 < a.R;         // else zeros in both operands
            v4u bf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bf[j] = (v4u){0, 0, 0, 0};
                if (in) bf[j] = *reinterpret_cast<const v4u*>(bp[j] + r);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const v4u v = low[((grp >> 1) * 16 * MT + 16 * m + row16) * pitch + r / 8 + (grp & 1)];
                const v4u vf = in ? v : (v4u){0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 4; ++j) part[j][m] = mfma_bf16(bf[j], vf, part[j][m]);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (id[m] == adapter)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j][m] = part[j][m] * scale;
    }
    // 16 columns of a row a lane
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int from = 16 * m + row16;
        const int lo = __shfl((int)(uint32_t)mine.row, from, 64), hi = __shfl((int)(mine.row >> 32), from, 64);
        const int64_t row = ((int64_t)hi << 32) | (uint32_t)lo;
        if (row < 0 || (id[m] < 0 && a.Y == a.out)) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = n0 + 16 * grp + 8 * h;
            if (n >= a.N) continue;
            v4u y = *reinterpret_cast<const v4u*>(a.Y + row * a.ldy + n);
            if (id[m] >= 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const v4f& d = acc[2 * h + (e >> 1)][m];
                    y[e] = pack_bf16x2(__uint_as_float(y[e] << 16) + d[2 * (e & 1)], __uint_as_float(y[e] & 0xFFFF0000u) + d[2 * (e & 1) + 1]);
                }
            }
            *reinterpret_cast<v4u*>(a.out + row * a.ldo + n) = y;
        }
    }
}

template <int RT>
void launch_down(const LoraArgs& a, int tiles, hipStream_t s) {
    const dim3 grid((uint32_t)a.splits, (uint32_t)((a.places + 16 * tiles - 1) / (16 * tiles)));
    if (tiles == 1) lora_down_kernel<RT, 1><<<grid, kThreads, 0, s>>>(a);
    else if (tiles == 2) lora_down_kernel<RT, 2><<<grid, kThreads, 0, s>>>(a);
    else if constexpr (RT <= 4) lora_down_kernel<RT, 4><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

void launch_lora_down(const LoraArgs& a, int tiles, hipStream_t s) {
    if (a.rank <= 16) launch_down<1>(a, tiles, s);
    else if (a.rank <= 32) launch_down<2>(a, tiles, s);
    else if (a.rank <= 64) launch_down<4>(a, tiles, s);
    else launch_down<8>(a, tiles, s);
}

void launch_lora_up(const LoraArgs& a, int tiles, hipStream_t s) {
    const dim3 grid((uint32_t)((a.N + kLoraSpan - 1) / kLoraSpan), (uint32_t)((a.places + 16 * tiles - 1) / (16 * tiles)));
    const size_t lds = (size_t)2 * 16 * tiles * (a.rank / 8 + 1) * 16;
    if (tiles == 1) lora_up_kernel<1><<<grid, kThreads, lds, s>>>(a);
    else if (tiles == 2) lora_up_kernel<2><<<grid, kThreads, lds, s>>>(a);
    else lora_up_kernel<4><<<grid, kThreads, lds, s>>>(a);
}

}  // namespace fp8gemm
