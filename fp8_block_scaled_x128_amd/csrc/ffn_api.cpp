// ffn_api.cpp -- C ABI of the gated feed-forward block in bf16, its gradients, and low-rank adapters.  Argument validation,
// launch-shape choice and launch (host code); meaning and layouts: include/fp8gemm.h.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <mutex>
#include <utility>

#include "ffn_internal.h"
#include "fp8gemm.h"
#include "fp8gemm_internal.h"
#include "moe_internal.h"

using namespace fp8gemm;

namespace {

constexpr int64_t kMaxBytes = int64_t(1) << 40;
constexpr int64_t kMaxWidth = int64_t(1) << 20;         // values of a row of X, W or dpre: a tile stays below 2^31 bytes
constexpr size_t kCounters = 4096;                      // of a stream's workspace
constexpr int64_t kMaxUnits = int64_t(1) << 22;         // workgroups of a launch: below 2^32 threads

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int launched() { return hipGetLastError() == hipSuccess ? FP8GEMM_OK : FP8GEMM_ERR_LAUNCH; }

struct Choice {
    int shape, splits;
    double us;                  // of its slices and exchange
};

// FP8GEMM_FORCE_CONFIG=product:BMxBN:SPLIT or product:BMxBNxRING:SPLIT
bool forced(Choice* c, bool gated) {
    const char* s = std::getenv("FP8GEMM_FORCE_CONFIG");
    int bm, bn, split, ring = 0;
    if (!s || (std::sscanf(s, "product:%dx%d:%d", &bm, &bn, &split) != 3 &&
               std::sscanf(s, "product:%dx%dx%d:%d", &bm, &bn, &ring, &split) != 4))
        return false;
    for (int i = 0; i < (gated ? kGatedShapes : kTileShapes); ++i)
        if (kTiles[i].bm == bm && kTiles[i].bn == bn && (ring == 0 || kTiles[i].ring == ring)) {
            *c = {i, std::max(1, split), 0.0};
            return true;
        }
    return false;
}

// Time of a slice where the CUs have up to `units` workgroups together.
double slice_us(const TileShape& t, int64_t units, int cus) {
    const int64_t most = std::min<int64_t>((units + cus - 1) / cus, t.per_cu);
    return most <= 1 ? t.alone : t.alone + (t.shared - t.alone) * (double)(most - 1) / (double)(t.per_cu - 1);
}

// `off`: rows off the lines (of one operand of kTimesW)
double slower(const TileShape& t, Product kind, bool off) {
    const double r = kind == kTimesW ? t.turned : kind == kTurned ? t.both_turned : 1.0;
    return !off ? r : kind == kTimesW ? r * 0.5 * (1.0 + t.off) : r * t.off;
}

// Whether the loads of rows off the lines make a difference, by all that the tiles load: H, us, tiles of 128 x 128 with loads
// by slices and by lines: 51 MB 10.7 and 11.9, 102 MB 12.7 and 12.7, 122 MB 34.5 and 24.4; of 64 x 64: 79 MB 11.9 and 14.2,
// 100 MB 10.5 and 10.0, 159 MB 18.7 and 16.7.  dX, with one such operand, gains or stays (9 to 216 tiles).
bool loads_count(int64_t tiles, const TileShape& t, int64_t slices) { return tiles * slices * (t.bm + t.bn) * 128 >= 96000000; }

// Tile and K splits of a product with `rows` x `cols` results (gated: cols pairs) and `slices` slices of 64 of K:
// the least of the times that the measured slices (kTiles) give for the rounds of workgroups that a CU takes, where
// those take longer than reading both operands and writing the result.  Over 25 sizes of H and of dX (17 to 4096 rows,
// I 64 to 2048, K 128 to 7168) the choice is within 5% of the best of all tiles with 1 to 16 splits.
Choice choose(int64_t rows, int64_t cols, int64_t slices, Product kind, int cus, bool off) {
    const bool gated = kind == kGated || kind == kGatedBack;
    Choice best{0, 1, 1e30};
    if (forced(&best, gated)) return best;
    const double bytes = (128e-6 * (double)slices * (double)(rows + (gated ? 2 : 1) * cols) + 2e-6 * (double)rows * (double)cols) / 5.2;
    for (int i = 0; i < (gated ? kGatedShapes : kTileShapes); ++i) {
        const TileShape& t = kTiles[i];
        const int64_t width = gated ? t.bn / 2 : t.bn;
        const int64_t tiles = ((rows + t.bm - 1) / t.bm) * ((cols + width - 1) / width);
        if (tiles > kMaxUnits) continue;
        const int64_t slots = (int64_t)cus * t.per_cu;
        const double slow = slower(t, kind, off && loads_count(tiles, t, slices));
        for (int64_t s = 1; s <= 16 && (s == 1 || (s * 2 <= slices && tiles * s <= slots)); ++s) {
            const int64_t per = (slices + s - 1) / s;
            if (s > 1 && (slices + per - 1) / per != s) continue;
            const int64_t units = tiles * s, last = units % slots;
            const double rounds = (double)(units / slots) * t.shared + (last == 0 ? 0.0 : slice_us(t, last, cus));
            const double cost = std::max(((double)per + t.ends) * rounds * slow, bytes) +
                                (s > 1 ? t.exchange + t.exchange_split * (double)s : 0.0);
            if (cost < best.us) best = {i, (int)s, cost};
        }
    }
    return best;
}

// Whether the kernel for few rows takes the block.  It brings X to every 8 columns' workgroup, so its time is
// that of the weights and of X's copies, or of a wave's steps one after the other; tiles start and end slower.
// Measured, rows and tiles, us: I = 2048, K = 7168: 1 row 11.2 and 14.2, 8 rows 13.0 and 14.2, 16 rows 15.3 and
// 14.2; 4096 and 4096: 4 rows 14.3 and 15.1, 16 rows 18.1 and 15.1; 256 and 7168: 16 rows 14.9 and 10.1;
// 1416 and 2056: 16 rows 5.8 and 8.7.
bool few_rows(int64_t M, int64_t I, int64_t K, int cus) {
    if (M > kGatedRowsMax || (I + 8) * K * 2 >= (int64_t(1) << 31)) return false;
    const double rounds = (double)((K + 511) / 512);                             // steps of a wave
    const double bytes = 4e-6 * (double)I * (double)K / 5.2 + 2e-6 * (double)M * (double)K * (double)((I + 7) / 8) / 12.0;
    return 2.5 + std::max(rounds * (0.55 + 0.02 * (double)M), bytes) < 3.5 + choose(M, I, (K + kSliceK - 1) / kSliceK, kGated, cus, false).us;
}

// Time, in slices, until n units of L slices and then n2 of L2 are done on `slots` places that take the next unit as
// they get free: half way between the mean load and what units that all take the same time would need.
double rounds_of(int64_t n, double L, int64_t n2, double L2, int64_t slots) {
    const int64_t late = n % slots;
    const double a = (double)(n / slots) * L, b = late ? a + L : a;
    // every place has time for at least (mean - a) / L2 of the second, rounded down
    const double mean = ((double)n * L + (double)n2 * L2) / (double)slots;
    for (int64_t k = std::max<int64_t>(1, (int64_t)((mean - a) / L2));; ++k) {
        const double t = a + (double)k * L2;                  // the early places' k-th ends; the late ones' last until then
        const int64_t j = t > b ? (int64_t)((t - b) / L2) : 0;
        const double tj = b + (double)j * L2;
        if (j > 0 && tj > t - L2 && (slots - late) * (k - 1) + late * j >= n2) return std::max(L, 0.5 * (mean + tj));
        if ((slots - late) * k + late * j >= n2) return std::max(L, 0.5 * (mean + std::max(t, b)));
    }
}

// dX and dW as one launch, if that is quicker than one after the other (the second's units fill the CUs that the
// first's last ones leave, but L2 serves both): a shape for both, and the splits of each.  Measured, one after the
// other and together, us: M = 1023, I = 1416, K = 2056 55 and 47; 1024, 2048, 7168 138 and 120; 905, 336, 456 17.8 and
// 13.1; 77, 512, 1536 12.7 and 11.4; but 256, 2048, 7168 62 and 73, 4096, 2048, 7168 417 and 420.  Over 35 sizes the
// choice is 2% from the best of one shape for both on average, 17% at most (64, 2048, 7168 from cold memory).
bool choose_pair(const ProductArgs& x, const ProductArgs& w, int cus, Choice* cx, Choice* cw) {
    if (forced(cx, false)) {
        *cw = *cx;
        return true;
    }
    const int64_t sx = (x.K + kSliceK - 1) / kSliceK, sw = (w.K + kSliceK - 1) / kSliceK;
    const double bytes = (128e-6 * ((double)sx * (double)(x.rows + x.cols) + (double)sw * (double)(w.rows + w.cols)) +
                          2e-6 * ((double)x.rows * (double)x.cols + (double)w.rows * (double)w.cols)) / 5.2;
    const bool off = off_the_lines(x, kTimesW, true);
    double least = cx->us + cw->us + 3.5;
    bool pair = false;
    for (int i = 0; i < kTileShapes; ++i) {
        const TileShape& t = kTiles[i];
        auto tiles = [&](const ProductArgs& a) { return (((int64_t)a.rows + t.bm - 1) / t.bm) * (((int64_t)a.cols + t.bn - 1) / t.bn); };
        const int64_t tx = tiles(x), tw = tiles(w), slots = (int64_t)cus * t.per_cu;
        if (tx + tw > kMaxUnits) continue;
        for (int64_t px = 1; px <= 8 && (px == 1 || (px * 2 <= sx && px * tx <= slots)); px *= 2)
            for (int64_t pw = 1; pw <= 8 && (pw == 1 || (pw * 2 <= sw && pw * tw <= slots)); pw *= 2) {
                const double lx = ((double)((sx + px - 1) / px) + t.ends) * slower(t, kTimesW, off);
                const double lw = ((double)((sw + pw - 1) / pw) + t.ends) * t.both_turned;
                const int64_t nx = tx * px, nw = tw * pw;
                const double rounds = lx >= lw ? rounds_of(nx, lx, nw, lw, slots) : rounds_of(nw, lw, nx, lx, slots);
                const int64_t most = std::max(px > 1 ? px : 0, pw > 1 ? pw : 0);
                const double us = 1.03 * std::max(rounds * slice_us(t, nx + nw, cus), bytes) +
                                  (most ? t.exchange + t.exchange_split * (double)most : 0.0);
                if (us >= least) continue;
                least = us;
                pair = true;
                *cx = {i, (int)px, us};
                *cw = {i, (int)pw, us};
            }
    }
    return pair;
}

// Sizes and order of the tiles of a product.
int arrange(ProductArgs* a, Choice* c, Product kind) {
    const bool gated = kind == kGated || kind == kGatedBack;
    a->slices = (a->K + kSliceK - 1) / kSliceK;
    const TileShape& t = kTiles[c->shape];
    const int width = gated ? t.bn / 2 : t.bn;
    const int64_t tm = ((int64_t)a->rows + t.bm - 1) / t.bm, tn = ((int64_t)a->cols + width - 1) / width;
    a->per_split = (a->slices + c->splits - 1) / c->splits;
    a->splits = c->splits = (a->slices + a->per_split - 1) / a->per_split;       // none without a slice
    if (tm > kMaxUnits / tn || tm * tn > kMaxUnits / a->splits) return FP8GEMM_ERR_UNSUPPORTED;
    a->lag = t.ring >= 4 && off_the_lines(*a, kind, false) && (kind == kTimesW || loads_count(tm * tn, t, a->slices));
    a->tiles_m = (int32_t)tm;
    a->tiles_n = (int32_t)tn;
    a->group_m = (int32_t)std::min<int64_t>(tm, 8);
    a->div_splits = make_fastdiv((uint32_t)a->splits);
    a->div_band_units = make_fastdiv((uint32_t)(a->group_m * tn));
    a->div_band_h = make_fastdiv((uint32_t)a->group_m);
    a->div_band_h_last = make_fastdiv((uint32_t)(tm - (tm - 1) / a->group_m * a->group_m));
    return FP8GEMM_OK;
}

// The stream's workspace for the K splits of products that may run at the same time, one part after the other; `hold`
// keeps it until the launches are enqueued.
int share_workspace(std::initializer_list<std::pair<ProductArgs*, Choice>> products, hipStream_t stream, std::unique_lock<std::mutex>* hold) {
    size_t floats = 0, tiles = 0;
    for (const auto& p : products) {
        if (p.first->splits <= 1) continue;
        const size_t n = (size_t)p.first->tiles_m * p.first->tiles_n;
        tiles += n;
        floats += n * p.first->splits * kTiles[p.second.shape].bm * kTiles[p.second.shape].bn;
    }
    if (tiles == 0) return FP8GEMM_OK;
    float* ws = nullptr;
    int32_t* counters = nullptr;
    const size_t spread = std::max<size_t>(1, std::min<size_t>(32, kCounters / tiles));
    const int st = host_stream_workspace(stream, floats * sizeof(float), tiles * spread, &ws, &counters,
                                         hold->owns_lock() ? nullptr : hold);
    if (st != FP8GEMM_OK) return st;
    for (const auto& p : products) {
        if (p.first->splits <= 1) continue;
        const size_t n = (size_t)p.first->tiles_m * p.first->tiles_n;
        p.first->ws = ws;
        p.first->counters = counters;
        p.first->spread = (int32_t)spread;
        counters += n * spread;
        ws += n * p.first->splits * kTiles[p.second.shape].bm * kTiles[p.second.shape].bn;
    }
    return FP8GEMM_OK;
}

// Whether adapters are added by a workgroup a row, one launch and no workspace.  One CU reads a row's two matrices, so they
// have to be small; two rounds of workgroups take twice as long, and the two launches take longer the more rows with
// different adapters stand together, which the host does not know.  Measured, two launches (rows in any order, by adapter)
// and this, us, by R (K + N): 8 rows 32768 6.8 and 5.3, 65536 7.4 and 5.9, 81920 6.8 and 7.5; 40 rows 104448 10.6, 10.5 and
// 9.3, 144000 15.5, 12.0 and 12.4; 100 rows 104448 19.3, 12.9 and 9.4, 166400 17, 10.6 and 10.8; 200 rows 110336 16, 9.8 and
// 9.7; 400 rows 51968 17.6, 10.2 and 9.0, 104448 29, 11.0 and 16; 1000 rows 8192 12.7 and 10.6.  By R, 1 row (8 rows
// are like it; of 20 and 31 rows the two launches take up to 13 and 18 with R above 64): 72000 R = 16 6.6 and 6.7, R = 64 7.7 and 6.5;
// 85000 6.7 and 7.8, 7.7 and 6.8; 99000 R = 72 8.6 and 9.0, R = 96 8.8 and 8.7, R = 128 9.6 and 8.2; 129000 9.1 and
// 12.6, 8.8 and 9.3, 9.2 and 7.5.  A wave takes K's steps of 4096 values one after the other: R = 8, N = 1024, 1 row,
// K = 4096 6.6 and 5.9, 5120 6.5 and 7.4; 45 rows 8.0 and 6.1, 8.1 and 7.7.
bool by_row(int64_t T, int64_t R, int64_t K, int64_t N) {
    const int64_t most = T < 32 ? (R > 64 ? 100000 : 72000) : T < 64 ? 110000 : T <= 256 ? 150000 : T <= 512 ? 72000 : T <= 1024 ? 16384 : 0;
    return K <= 4096 && R * (K + N) <= most;
}

int check_gated(int64_t M, int64_t I, int64_t K, int32_t act) {
    if (M < 0 || I <= 0 || K <= 0 || I % 8 != 0 || K % 8 != 0) return FP8GEMM_ERR_BAD_SHAPE;
    if (act != FP8GEMM_ACT_SILU && act != FP8GEMM_ACT_GELU_TANH) return FP8GEMM_ERR_BAD_SHAPE;
    if (K > kMaxWidth || I > kMaxWidth / 2 || M >= (int64_t(1) << 31) - 64 || 2 * M * K >= kMaxBytes || 4 * M * I >= kMaxBytes)
        return FP8GEMM_ERR_UNSUPPORTED;
    return FP8GEMM_OK;
}

}  // namespace

extern "C" {

int fp8gemm_gated_ffn(const void* X, const void* W, void* H, void* pre, int64_t M, int64_t I, int64_t K, int32_t act,
                      void* stream) {
    int st = check_gated(M, I, K, act);
    if (st != FP8GEMM_OK) return st;
    if (M == 0) return FP8GEMM_OK;
    if (!X || !W || !H) return FP8GEMM_ERR_NULL_PTR;
    if (!aligned(X, 16) || !aligned(W, 16) || !aligned(H, 16) || !aligned(pre, 16)) return FP8GEMM_ERR_MISALIGNED;
    HostDevice d;
    st = host_device(&d);
    if (st != FP8GEMM_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    Choice c;
    if (!forced(&c, true) && few_rows(M, I, K, d.cus)) {
        GatedRowsArgs a{};
        a.X = static_cast<const uint16_t*>(X);
        a.W = static_cast<const uint16_t*>(W);
        a.out = static_cast<uint16_t*>(H);
        a.pre = static_cast<uint16_t*>(pre);
        a.M = (int32_t)M;
        a.I = (int32_t)I;
        a.K = (int32_t)K;
        a.gelu = act == FP8GEMM_ACT_GELU_TANH;
        host_set_config("gated_ffn M=%lld I=%lld K=%lld rows", {M, I, K});
        launch_gated_rows(a, s);
        return launched();
    }
    ProductArgs a{};
    a.P = static_cast<const uint16_t*>(X);
    a.Q = static_cast<const uint16_t*>(W);
    a.out = static_cast<uint16_t*>(H);
    a.pre = static_cast<uint16_t*>(pre);
    a.rows = (int32_t)M;
    a.cols = (int32_t)I;
    a.K = a.ldp = a.ldq = (int32_t)K;
    a.gelu = act == FP8GEMM_ACT_GELU_TANH;
    c = choose(M, I, (K + kSliceK - 1) / kSliceK, kGated, d.cus, off_the_lines(a, kGated, true));
    st = arrange(&a, &c, kGated);
    if (st != FP8GEMM_OK) return st;
    std::unique_lock<std::mutex> hold;
    st = share_workspace({{&a, c}}, s, &hold);
    if (st != FP8GEMM_OK) return st;
    host_set_config("gated_ffn M=%lld I=%lld K=%lld tile=%lldx%lld split=%lld lines=%lld",
                    {M, I, K, kTiles[c.shape].bm, kTiles[c.shape].bn, c.splits, a.lag});
    launch_product(a, kGated, c.shape, s);
    return launched();
}

int fp8gemm_gated_ffn_backward(const void* dH, const void* X, const void* W, const void* pre, void* dpre, void* dX, void* dW,
                               int64_t M, int64_t I, int64_t K, int32_t act, void* stream) {
    int st = check_gated(M, I, K, act);
    if (st != FP8GEMM_OK) return st;
    if (M > 0 && (!dH || !dpre || (!X && (!pre || dW)) || (!W && (!pre || dX)))) return FP8GEMM_ERR_NULL_PTR;
    for (const void* p : {dH, X, W, pre, static_cast<const void*>(dpre), static_cast<const void*>(dX), static_cast<const void*>(dW)})
        if (!aligned(p, 16)) return FP8GEMM_ERR_MISALIGNED;
    if ((M * I / 8 + 255) / 256 > kMaxUnits * 4 - 1) return FP8GEMM_ERR_UNSUPPORTED;
    if (M == 0 && !dW) return FP8GEMM_OK;
    HostDevice d;
    st = host_device(&d);
    if (st != FP8GEMM_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (M == 0) {
        launch_fill_zero(dW, 4 * I * K, s);
        return launched();
    }
    // every choice and the workspace before the first launch
    Choice cp{0, 1, 0}, cx{0, 1, 0}, cw{0, 1, 0}, any;
    ProductArgs ap{}, ax{}, aw{};
    GatedRowsArgs ar{};
    const bool rows = !pre && !forced(&any, true) && few_rows(M, I, K, d.cus);
    auto slices = [](int64_t k) { return (k + kSliceK - 1) / kSliceK; };
    if (rows) {
        ar.X = static_cast<const uint16_t*>(X);
        ar.W = static_cast<const uint16_t*>(W);
        ar.dH = static_cast<const uint16_t*>(dH);
        ar.pre = static_cast<uint16_t*>(dpre);
        ar.M = (int32_t)M;
        ar.I = (int32_t)I;
        ar.K = (int32_t)K;
        ar.gelu = act == FP8GEMM_ACT_GELU_TANH;
    } else if (!pre) {
        ap.P = static_cast<const uint16_t*>(X);
        ap.Q = static_cast<const uint16_t*>(W);
        ap.dH = static_cast<const uint16_t*>(dH);
        ap.pre = static_cast<uint16_t*>(dpre);
        ap.rows = (int32_t)M;
        ap.cols = (int32_t)I;
        ap.K = ap.ldp = ap.ldq = (int32_t)K;
        ap.gelu = act == FP8GEMM_ACT_GELU_TANH;
        cp = choose(M, I, slices(K), kGatedBack, d.cus, off_the_lines(ap, kGatedBack, true));
        st = arrange(&ap, &cp, kGatedBack);
        if (st != FP8GEMM_OK) return st;
    }
    if (dX) {
        ax.P = static_cast<const uint16_t*>(dpre);
        ax.Q = static_cast<const uint16_t*>(W);
        ax.out = static_cast<uint16_t*>(dX);
        ax.rows = (int32_t)M;
        ax.cols = ax.ldq = (int32_t)K;
        ax.K = ax.ldp = (int32_t)(2 * I);
        cx = choose(M, K, slices(2 * I), kTimesW, d.cus, off_the_lines(ax, kTimesW, true));
    }
    if (dW) {
        aw.P = static_cast<const uint16_t*>(dpre);
        aw.Q = static_cast<const uint16_t*>(X);
        aw.out = static_cast<uint16_t*>(dW);
        aw.rows = aw.ldp = (int32_t)(2 * I);
        aw.cols = aw.ldq = (int32_t)K;
        aw.K = (int32_t)M;
        cw = choose(2 * I, K, slices(M), kTurned, d.cus, false);
    }
    const bool pair = dX && dW && choose_pair(ax, aw, d.cus, &cx, &cw);
    if (dX && (st = arrange(&ax, &cx, kTimesW)) != FP8GEMM_OK) return st;
    if (dW && (st = arrange(&aw, &cw, kTurned)) != FP8GEMM_OK) return st;
    if (pair && (int64_t)ax.tiles_m * ax.tiles_n * ax.splits + (int64_t)aw.tiles_m * aw.tiles_n * aw.splits > kMaxUnits)
        return FP8GEMM_ERR_UNSUPPORTED;
    // (dX and dW, which follow, take the first product's part again)
    std::unique_lock<std::mutex> hold;
    st = share_workspace({{&ap, cp}}, s, &hold);
    if (st == FP8GEMM_OK) st = share_workspace({{&ax, cx}, {&aw, cw}}, s, &hold);
    if (st != FP8GEMM_OK) return st;
    // (zeros for a product that is not formed)
    const TileShape none{}, &tp = ap.splits ? kTiles[cp.shape] : none, &tx = dX ? kTiles[cx.shape] : none, &tw = dW ? kTiles[cw.shape] : none;
    const char* words = pre    ? "gated_ffn_backward M=%lld I=%lld K=%lld kept together=%lld dX tile=%lldx%lldx%lld split=%lld lines=%lld dW tile=%lldx%lldx%lld split=%lld"
                        : rows ? "gated_ffn_backward M=%lld I=%lld K=%lld rows together=%lld dX tile=%lldx%lldx%lld split=%lld lines=%lld dW tile=%lldx%lldx%lld split=%lld"
                               : "gated_ffn_backward M=%lld I=%lld K=%lld together=%lld dX tile=%lldx%lldx%lld split=%lld lines=%lld dW tile=%lldx%lldx%lld split=%lld "
                                 "products tile=%lldx%lldx%lld split=%lld lines=%lld";
    host_set_config(words, {M, I, K, pair, tx.bm, tx.bn, tx.ring, ax.splits, ax.lag, tw.bm, tw.bn, tw.ring, aw.splits, tp.bm, tp.bn, tp.ring,
                            ap.splits, ap.lag});
    if (pre) {
        GatedGradArgs g{};
        g.pre = static_cast<const uint16_t*>(pre);
        g.dH = static_cast<const uint16_t*>(dH);
        g.dpre = static_cast<uint16_t*>(dpre);
        g.units = M * (I / 8);
        g.I = (int32_t)I;
        g.gelu = act == FP8GEMM_ACT_GELU_TANH;
        g.div_row = make_fastdiv((uint32_t)(I / 8));
        launch_gated_grad(g, s);
    } else if (rows) {
        launch_gated_rows(ar, s);
    } else {
        launch_product(ap, kGatedBack, cp.shape, s);
    }
    st = launched();
    if (st == FP8GEMM_OK && pair) {
        launch_gradients(ax, aw, cx.shape, s);
        return launched();
    }
    if (st == FP8GEMM_OK && dX) {
        launch_product(ax, kTimesW, cx.shape, s);
        st = launched();
    }
    if (st == FP8GEMM_OK && dW) {
        launch_product(aw, kTurned, cw.shape, s);
        st = launched();
    }
    return st;
}

int fp8gemm_lora_add(const void* Y, const void* X, const void* A, const void* B, const int32_t* ids, const int32_t* order,
                     const float* scales, void* out, int64_t T, int32_t L, int32_t R, int64_t K, int64_t N, int64_t ldx,
                     int64_t ldy, int64_t ldo, void* stream) {
    if (T < 0 || L <= 0 || R <= 0 || R % 8 != 0 || K <= 0 || K % 8 != 0 || N < 0 || N % 8 != 0) return FP8GEMM_ERR_BAD_SHAPE;
    if (T > 1 && (ldx < K || ldy < N || ldo < N || ldx % 8 != 0 || ldy % 8 != 0 || ldo % 8 != 0)) return FP8GEMM_ERR_BAD_SHAPE;
    if (R > kLoraMaxRank || K > kMaxWidth || N > kMaxWidth || T >= (int64_t(1) << 31) - 64) return FP8GEMM_ERR_UNSUPPORTED;
    if (T > 1 && std::max(ldx, std::max(ldy, ldo)) > kMaxBytes / 2 / T) return FP8GEMM_ERR_UNSUPPORTED;
    if ((int64_t)L * R > kMaxBytes / 2 / std::max<int64_t>(std::max(K, N), 1)) return FP8GEMM_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return FP8GEMM_OK;
    if (!Y || !X || !A || !B || !ids || !out) return FP8GEMM_ERR_NULL_PTR;
    if (T > 1 && Y == out && ldy != ldo) return FP8GEMM_ERR_BAD_SHAPE;
    if (!aligned(Y, 16) || !aligned(X, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(out, 16) || !aligned(ids, 4) ||
        !aligned(order, 4) || !aligned(scales, 4))
        return FP8GEMM_ERR_MISALIGNED;
    HostDevice d;
    int st = host_device(&d);
    if (st != FP8GEMM_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    LoraArgs a{};
    a.X = static_cast<const uint16_t*>(X);
    a.A = static_cast<const uint16_t*>(A);
    a.B = static_cast<const uint16_t*>(B);
    a.Y = static_cast<const uint16_t*>(Y);
    a.out = static_cast<uint16_t*>(out);
    a.ids = ids;
    a.order = order;
    a.scales = scales;
    a.err = d.err;
    a.ldx = ldx;
    a.ldy = ldy;
    a.ldo = ldo;
    a.T = T;
    a.L = L;
    a.R = R;
    a.K = (int32_t)K;
    a.N = (int32_t)N;
    a.rank = (R + 15) / 16 * 16;
    a.steps = (int32_t)((K + 63) / 64);
    if (by_row(T, R, K, N)) {
        a.places = (int32_t)T;
        host_set_config("lora_add T=%lld R=%lld K=%lld N=%lld by row", {T, R, K, N});
        launch_lora_rows(a, s);
        return launched();
    }
    // Rows of a workgroup.  64, where there are many and an adapter has 16 of them or more on average: measured, 64
    // and 16 rows, us: 8192 rows of 8 adapters, R = 32, 7168 to 4096, 64 and 117; 1000 of 4, R = 64, 22.5 and 26.0,
    // but R = 16 15.2 and 14.0; 4096 of 64, R = 16, 38 and 42; 2048 of 128, R = 8, 32 and 25.  Else so few that the
    // workgroups go through few adapters each and many of them have rows, more the more an adapter's matrices hold: 1, 2,
    // 4, 8 and 16 rows, us, rows in any order and by adapter: 64 adapters, R = 16, 7168 to 4096: 48 rows 10.0, 9.9, 10.4,
    // 13.2, 20.4 and 10.0, 9.7, 10.2, 13.2, 19.2; 270 rows 31, 25, 21, 22, 23 and 31, 25, 18, 14.7, 14.5; 512 rows 38,
    // 33, 34, 32, 32 and 39, 31, 23, 18, 15.5.  3 adapters, R = 104, 2496 to 952: 128 rows 28, 23, 21, 17, 16 and 29, 18,
    // 16, 13.7, 14.0.
    if (T >= 16 * (int64_t)L && T > (R > 32 ? 512 : 1024)) a.tile = 64;
    else for (a.tile = 1; a.tile < 16 && a.tile * 40 < T * ((R + 31) / 32);) a.tile *= 2;
    const int64_t row_tiles = (T + a.tile - 1) / a.tile;
    // Splits of K, of 8 steps at least.  Few rows: such that the CUs have two workgroups each; 4, 8 and 16 steps, us: 1
    // row 7.5, 6.9 and 7.4, 256 rows of 64 adapters 19.8, 16.3 and 20.1.  Tiles of 64 rows: a power of two, so that
    // each CU has a workgroup, beside those for the tiles' second adapters: 1, 2, 4 and 8 splits, us: 8192 rows of 8
    // adapters, R = 32, 7168 to 4096, 61, 53, 57 and 57; 5963 of 4, R = 128, 3640 to 80, 39, 38, 31 and 39; 2000 of 3,
    // R = 128, 4096 to 7168, 55, 42, 36.3 and 36.6.  Without the second workgroups these took 57, 35 and 39 at best.
    int64_t want = std::max<int64_t>(1, 2 * d.cus / row_tiles);
    if (a.tile == 64) {
        a.apart = L > 1;
        for (want = 1; want * row_tiles < d.cus;) want *= 2;
    }
    const int64_t splits = std::min<int64_t>(want, (a.steps + 7) / 8);
    a.per_split = (int32_t)((a.steps + splits - 1) / splits);
    a.splits = (a.steps + a.per_split - 1) / a.per_split;
    // runs of columns that a workgroup takes one after the other, so that there are six for each CU where the rows
    // allow it: 1, 6 and 16 for each CU, us: 8192 rows, R = 32 85, 64 and 65; 2000 rows, R = 128 50, 38 and 43
    const int64_t spans = a.tile <= 16 ? (N + kLoraSpan - 1) / kLoraSpan : (N + 63) / 64;
    a.chunks = (int32_t)std::max<int64_t>(1, std::min<int64_t>(spans, spans * row_tiles / (6 * d.cus)));
    // rows of a pass: the splits' sums of A x and its halves fit the workspace, the tiles the grid's second
    // dimension and the counters
    const int64_t row_bytes = (int64_t)a.rank * 4 * (a.splits + 1);
    const int64_t room = (int64_t)d.all_cus * 512 * 1024 / row_bytes / 64 * 64;
    const int64_t pass = std::min(T, std::min<int64_t>(room, (int64_t)(a.tile == 64 ? 2048 : 4096) * a.tile));
    std::unique_lock<std::mutex> hold;
    st = host_stream_workspace(s, (size_t)(pass * row_bytes), a.tile == 64 ? (size_t)((pass + 63) / 64) * 2 : 0, &a.low, &a.counters, &hold);
    if (st != FP8GEMM_OK) return st;
    a.halves = reinterpret_cast<uint16_t*>(a.low + pass * a.splits * a.rank);
    host_set_config("lora_add T=%lld R=%lld K=%lld N=%lld rows=%lld split=%lld", {T, R, K, N, a.tile, a.splits});
    for (a.first = 0; a.first < T; a.first += pass) {
        a.places = (int32_t)std::min(pass, T - a.first);
        launch_lora_down(a, s);
        launch_lora_up(a, s);
        st = launched();
        if (st != FP8GEMM_OK) return st;
    }
    return FP8GEMM_OK;
}

}  // extern "C"
