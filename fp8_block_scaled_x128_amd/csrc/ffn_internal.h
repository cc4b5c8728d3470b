// ffn_internal.h -- types shared by the kernels of the gated feed-forward block and the low-rank adapters
// and their host code (ffn_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8gemm_args.h"

namespace fp8gemm {

// ---- tiled bf16 products ----
// out[i][j] = sum_k P(i, k) Q(j, k); each operand either has k contiguous (rows of P are rows of memory) or is
// "turned" (rows of memory are values of k).
enum Product {
    kGated = 0,        // P = X [M,K], Q = W [2I,K]: act(gate) * up, and the products themselves if `pre`
    kGatedBack = 1,    // the same products, then their gradients from dH into `pre`
    kTimesW = 2,       // P = dpre [M,2I], Q = W [2I,K] turned: dX
    kTurned = 3,       // P = dpre [M,2I] turned, Q = X [M,K] turned: dW
};

struct ProductArgs {
    const uint16_t* P;
    const uint16_t* Q;
    const uint16_t* dH;         // kGatedBack: [rows][cols]
    uint16_t* out;              // [rows][cols]
    uint16_t* pre;              // kGated: [rows][2 cols] or null; kGatedBack: [rows][2 cols]
    float* ws;                  // K splits: partial tiles [tile][split][BM * BN]
    int32_t* counters;          // K splits: arrivals by tile, `spread` from one to the next, zero between launches
    int32_t spread;
    int32_t rows, cols;         // of out (kGated, kGatedBack: cols = I)
    int32_t K;                  // contraction
    int32_t ldp, ldq;           // values from one row of memory to the next
    int32_t slices;             // ceil(K / 64)
    int32_t tiles_m, tiles_n;
    int32_t splits, per_split;  // slices of a split
    int32_t group_m;            // M tiles of a band of the tile order
    int32_t gelu;               // activation: silu, or gelu by its tanh form
    int32_t lag;                // tiles of 128 x 128 and 64 x 64: loads by whole lines of rows off the lines
    FastDiv div_splits, div_band_units, div_band_h, div_band_h_last;
};

// Whether rows of a straight operand start beside 128-byte lines, so that a slice of a row lies in two of them: where it
// stands in memory (that is how it is loaded), or anywhere, for its rows' length alone (that is what tiles and K splits
// are chosen by, and with them the order of the sums).
inline bool off_the_lines(const ProductArgs& a, Product kind, bool anywhere) {
    const auto off = [=](const void* p, int32_t ld) { return (((anywhere ? 0 : reinterpret_cast<uintptr_t>(p)) | 2 * (uintptr_t)ld) & 127) != 0; };
    return (kind != kTurned && off(a.P, a.ldp)) || ((kind == kGated || kind == kGatedBack) && off(a.Q, a.ldq));
}

// Tiles of a workgroup: bm rows of P, bn rows of Q, a ring of `ring` slices.  Times in us, measured: a slice where the
// workgroup has a CU to itself, and where `per_cu` share it (for all of them); how much longer it takes with Q turned, with
// both operands, and with rows off the lines; its start and end, in slices; a K split's exchange (constant, and by split).
// The last shape is for gradients: its starts and ends, most of the time of short sums, go on beside those of three others.
struct TileShape {
    int bm, bn, ring, per_cu;
    double alone, shared, turned, both_turned, off, ends, exchange, exchange_split;
};
constexpr TileShape kTiles[] = {{256, 256, 2, 1, 1.48, 1.48, 1.00, 1.05, 1.15, 5.3, 20.0, 2.7},
                                {128, 256, 3, 1, 0.83, 0.83, 1.05, 1.15, 1.30, 6.0, 8.0, 1.5},
                                {128, 128, 4, 1, 0.47, 0.47, 1.15, 1.30, 1.10, 8.0, 6.0, 0.7},
                                {64, 64, 4, 2, 0.25, 0.46, 1.05, 1.10, 1.20, 5.3, 1.0, 0.3},
                                {64, 64, 2, 4, 0.42, 0.85, 1.05, 1.10, 1.25, 2.5, 1.5, 0.6}};
constexpr int kTileShapes = 5, kGatedShapes = 4;
constexpr int kSliceK = 64;

void launch_product(const ProductArgs& a, Product kind, int shape, hipStream_t s);

// kTimesW and kTurned with tiles of one shape, as one launch
void launch_gradients(const ProductArgs& x, const ProductArgs& w, int shape, hipStream_t s);

// ---- the block for few rows ----
struct GatedRowsArgs {
    const uint16_t* X;          // [M][K]
    const uint16_t* W;          // [2I][K]
    const uint16_t* dH;         // [M][I], for gradients, or null
    uint16_t* out;              // [M][I]; none with dH
    uint16_t* pre;              // [M][2I] or null; the gradients with dH
    int32_t M, I, K;
    int32_t gelu;
};
constexpr int kGatedRowsMax = 16;   // rows of X that the kernel takes

void launch_gated_rows(const GatedRowsArgs& a, hipStream_t s);

// ---- gradients of the products from kept ones ----
struct GatedGradArgs {
    const uint16_t* pre;        // [M][2I]
    const uint16_t* dH;         // [M][I]
    uint16_t* dpre;             // [M][2I]
    int64_t units;              // M * I / 8
    int32_t I;
    int32_t gelu;
    FastDiv div_row;            // by I / 8
};
void launch_gated_grad(const GatedGradArgs& a, hipStream_t s);

// ---- low-rank adapters ----
constexpr int kLoraMaxRank = 128;
constexpr int kLoraSpan = 256;      // columns of the result that a workgroup of at most 16 places takes at a time

struct LoraArgs {
    const uint16_t* X;          // [T][ldx]
    const uint16_t* A;          // [L][R][K]
    const uint16_t* B;          // [L][N][R]
    const uint16_t* Y;          // [T][ldy]
    uint16_t* out;              // [T][ldo]
    const int32_t* ids;         // [T]
    const int32_t* order;       // [T] or null
    const float* scales;        // [L] or null
    float* low;                 // A x, partial sums: [splits][places][rank], rank padded to 16
    uint16_t* halves;           // tiles of 64 places: A x as two bf16 halves, [places][2][rank]
    int32_t* counters;          // tiles of 64 places: arrivals, zero between launches
    int32_t* err;
    int64_t ldx, ldy, ldo;
    int64_t T;
    int64_t first;              // first place (row, or position in order) of this pass
    int32_t places;             // of this pass
    int32_t tile;               // places of a workgroup: 64, or at most 16
    int32_t L, R, K, N;
    int32_t rank;               // R rounded up to 16
    int32_t steps;              // ceil(K / 64)
    int32_t splits, per_split;  // steps of a split
    int32_t apart;              // tiles of 64 places: 0, or 1: two workgroups have their adapters in turn
    int32_t chunks;             // runs of columns that a workgroup takes: of kLoraSpan, or of 64 with tiles of 64 places
};

void launch_lora_rows(const LoraArgs& a, hipStream_t s);      // both products, a workgroup a row
void launch_lora_down(const LoraArgs& a, hipStream_t s);
void launch_lora_up(const LoraArgs& a, hipStream_t s);

// 16-byte units set to zero (a gradient over no rows).
void launch_fill_zero(void* p, int64_t bytes, hipStream_t s);

}  // namespace fp8gemm
