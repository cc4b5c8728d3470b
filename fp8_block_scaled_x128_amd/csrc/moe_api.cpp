// moe_api.cpp -- C ABI of the operators around the grouped products: expert routing, token
// permutation (dispatch and combine) and 4-bit matrix-vector products.  Argument validation,
// launch-shape choice and launch (host code); meaning and layouts: include/fp8gemm.h.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fp8gemm.h"
#include "fp8gemm_internal.h"
#include "moe_internal.h"

using namespace fp8gemm;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxBytes = int64_t(1) << 40;
constexpr int64_t kMaxPairs = int64_t(1) << 30;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;   // of a launch, in one dimension
constexpr int64_t kMaxK4 = int64_t(1) << 22;      // 64 rows of a matrix stay below 2^31 bytes

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int launched() { return hipGetLastError() == hipSuccess ? FP8GEMM_OK : FP8GEMM_ERR_LAUNCH; }

// Shared checks of the two routing calls.
int check_route(int64_t T, int32_t E, int32_t k, int32_t dtype, int32_t score, float scale) {
    if (T < 0 || E <= 0 || k <= 0 || k > E) return FP8GEMM_ERR_BAD_SHAPE;
    if ((dtype != FP8GEMM_F32 && dtype != FP8GEMM_BF16) ||
        (score != FP8GEMM_SCORE_SOFTMAX && score != FP8GEMM_SCORE_SIGMOID) || !std::isfinite(scale))
        return FP8GEMM_ERR_BAD_SHAPE;
    if (E > kRouteMaxExperts || k > kRouteMaxTopk || T > kMaxThreads / 16 - 16) return FP8GEMM_ERR_UNSUPPORTED;
    return FP8GEMM_OK;
}

// Batches of at most this many pairs are ranked inside the copying launch, where every workgroup counts
// all pairs; larger ones take four launches, whose time grows with the experts.  Measured, one launch and
// four, us, k = 8: masked, 64 experts, H = 7168: 1024 pairs 5.1 and 14.2, 8192 24.7 and 28.5, 16384 68 and 42;
// H = 2048: 8192 10.7 and 17.1, 16384 23.9 and 21.4; contiguous, 256 experts, H = 7168: 8192 27.2 and 34.4,
// 16384 71 and 48.
constexpr int64_t kSmallPairs = 8192;

int check_dispatch(int64_t T, int64_t H, int32_t k, int32_t G, int64_t cap) {
    if (T < 0 || k <= 0 || G <= 0 || cap < 0 || H <= 0 || H % 128 != 0) return FP8GEMM_ERR_BAD_SHAPE;
    if (k > kDispatchMaxTopk || G > kDispatchMaxGroups || T >= kMaxPairs / k ||
        H > (int64_t(1) << 24) || 2 * T * H >= kMaxBytes)
        return FP8GEMM_ERR_UNSUPPORTED;
    const int64_t threads = T * k <= kSmallPairs ? row_spans((int)H) * kRowThreads : dispatch_copy_threads((int)H);
    return T * threads > kMaxThreads ? FP8GEMM_ERR_UNSUPPORTED : FP8GEMM_OK;
}

int dispatch(DispatchArgs a, hipStream_t stream) {
    HostDevice d;
    int st = host_device(&d);
    if (st != FP8GEMM_OK) return st;
    a.err = d.err;
    a.nkb = a.H / 128;
    a.pairs = (int32_t)(a.T * a.k);
    a.div_k = make_fastdiv((uint32_t)a.k);
    const bool large = a.pairs > kSmallPairs;
    std::unique_lock<std::mutex> hold;       // counts, ranks and scales go from launch to launch in the workspace
    if (large) {
        a.chunks = (a.pairs + kDispatchChunk - 1) / kDispatchChunk;
        const size_t words = (size_t)a.G * a.chunks + 2 * (size_t)a.G + (size_t)a.pairs;
        const size_t rows = (size_t)(a.contiguous ? 1 : a.G) * a.cap;
        void* p = nullptr;
        // the turned scales where their scratch fits the workspace
        a.by_row = host_stream_scratch(stream, (words + (size_t)a.T * a.nkb + rows) * sizeof(int32_t), &p, &hold) == FP8GEMM_OK;
        if (!a.by_row) st = host_stream_scratch(stream, words * sizeof(int32_t), &p, &hold);
        if (st != FP8GEMM_OK) return st;
        a.scratch = static_cast<int32_t*>(p);
    }
    host_set_config(a.contiguous ? (large ? "moe_dispatch_contiguous pairs=%lld experts=%lld count+scan+copy"
                                          : "moe_dispatch_contiguous pairs=%lld experts=%lld one launch")
                                 : (large ? "moe_dispatch_masked pairs=%lld experts=%lld count+scan+copy"
                                          : "moe_dispatch_masked pairs=%lld experts=%lld one launch"),
                    {a.pairs, a.G});
    launch_dispatch(a, large, stream);
    return launched();
}

int check_combine(int64_t T, int64_t H, int32_t k, int64_t R, const int32_t* row_map, bool backward) {
    if (T < 0 || k <= 0 || R < 0 || H <= 0 || H % 8 != 0) return FP8GEMM_ERR_BAD_SHAPE;
    if (k > kCombineMaxTopk || T > kMaxRows / k || R > kMaxRows || H > (int64_t(1) << 24) || 2 * T * H >= kMaxBytes ||
        2 * R * H >= kMaxBytes || T * (backward ? 1 : row_spans((int)H)) * kRowThreads > kMaxThreads)
        return FP8GEMM_ERR_UNSUPPORTED;
    if (!row_map && R < T * k) return FP8GEMM_ERR_BAD_SHAPE;
    return FP8GEMM_OK;
}

// Shared checks of the two 4-bit products; G matrices [N][K].
int check_w4(int64_t rows, int64_t G, int64_t N, int64_t K, int32_t format, int32_t group, const uint8_t* zeros) {
    if (rows < 0 || N < 0 || K <= 0) return FP8GEMM_ERR_BAD_SHAPE;
    if (format == FP8GEMM_W4_MXFP4) {
        if (group != 32 || zeros) return FP8GEMM_ERR_BAD_SHAPE;
    } else if (format != FP8GEMM_W4_INT4 || (group != 32 && group != 64 && group != 128)) {
        return FP8GEMM_ERR_BAD_SHAPE;
    }
    if (K % group != 0) return FP8GEMM_ERR_BAD_SHAPE;
    if (K > kMaxK4 || N > (int64_t(1) << 24) || rows > kMaxRows || G * N * (K / 2) >= kMaxBytes || rows * K * 2 >= kMaxBytes ||
        rows * N * 2 >= kMaxBytes)
        return FP8GEMM_ERR_UNSUPPORTED;
    return FP8GEMM_OK;
}

int check_w4_ptrs(const void* X, const void* W, const void* scales, const uint8_t* zeros, const void* Y) {
    if (!X || !W || !scales || !Y) return FP8GEMM_ERR_NULL_PTR;
    if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(scales, 4) || !aligned(zeros, 4))
        return FP8GEMM_ERR_MISALIGNED;
    return FP8GEMM_OK;
}

// Tiles of 16 rows that a wave takes one after the other, each with all of K, or 0: a workgroup's 8
// waves share a tile's K.  `busy` workgroup columns (row blocks of X, pairs or experts) have work.  A
// wave of its own needs no exchange of sums but 6 waves per CU to fill it, and all of X in LDS (64 KB, so
// that two workgroups share a CU).  Measured, shared K and own, us, MXFP4: 1 x 24576 x 1536 8.4 and 7.1,
// 1 x 32768 x 512 6.7 and 4.7, 16 x 24576 x 1536 10.7 and 8.6, 128 pairs of 7168 x 2048 on 64 experts 156
// and 88; but 1 x 16384 x 2048 7.2 and 7.9, 1 x 7168 x 2048 4.9 and 6.9, 1 x 32768 x 7168 23.9 and 27.3.
// Two tiles keep the loads going from one to the next where there are that many.
int w4_tiles_per_wave(int64_t nout, int64_t K, int cols, int64_t busy, int cus) {
    const int64_t tiles = (nout + 15) / 16 * busy, slots = 16 * (int64_t)cus;
    if (tiles < 6 * (int64_t)cus || K > 4096 || cols * K * 2 > 65536) return 0;
    return tiles >= 2 * slots ? 2 : 1;
}

// Tiles of 16 rows that a workgroup takes at a time.  One, where that gives every CU no more than one
// workgroup, or for few rows of X and rows of 6144 values and more of a single matrix (`lone`); two share X's
// LDS traffic and the exchange of sums.  Measured, one and two, us, MXFP4: 16 x 2048 x 2048 5.0 and 5.7,
// 1 x 4096 x 7168 6.2 and 7.7, 1 x 7168 x 16384 16.7 and 19.1, 1 x 32768 x 7168 23.9 and 26.5; but
// 16 x 7168 x 2048 6.8 and 6.1, 1 x 14336 x 4096 10.9 and 10.0, a token's 8 experts of 2048 x 7168 18.3 and 13.5.
int w4_row_tiles(int64_t nout, int64_t K, int cols, int64_t busy, bool lone, int cus) {
    return (nout + 15) / 16 * busy <= cus || (lone && cols <= 4 && K >= 6144) ? 1 : 2;
}

// Rows of X that a pass over an expert's matrix takes; a more crowded expert takes more passes.  A token's
// picks are distinct as a rule, so an expert has at most T pairs, and pairs / E on average.  Rows that LDS
// has no room for beside a second workgroup (76 KB), or a wave of its own (64 KB), cost more than a few
// experts' second passes, as long as two deviations above the average fit.  Measured, all rows that 4 + 2
// averages allow and fewer, us: MXFP4 with SwiGLU, 16 tokens, 8 of 32 experts of 4096 x 4096, 12 rows 116, 9
// rows 82, 8 rows (waves of their own) 65; INT4, 13 tokens, 7 of 20 experts of 1360 x 3456, 13 rows 27.1, 11
// rows 19.3; but 11 tokens, 4 of 6 experts of 488 x 2880, 11 rows 8.1, 9 rows 11.5.
int w4_expert_rows(int64_t T, int64_t pairs, int64_t E, int64_t K) {
    const double mean = (double)pairs / (double)E;
    const int64_t most = std::min<int64_t>(std::min<int64_t>(T, 16), 4 + 2 * ((pairs + E - 1) / E));
    const int64_t least = (int64_t)std::ceil(mean + 2.0 * std::sqrt(mean));
    for (const int64_t room : {int64_t(65536) / (2 * K), int64_t(76 * 1024) / (2 * ((K + 127) / 128 * 128) + 16)})
        if (room >= least) return (int)std::min(most, room);
    return (int)most;
}

}  // namespace

extern "C" {

int fp8gemm_route_topk(const void* logits, const float* bias, int32_t* ids, float* weights, int64_t T, int32_t E,
                       int32_t k, int32_t dtype, int32_t score, int32_t n_group, int32_t topk_group, int32_t group_top,
                       int32_t renorm, float scale, void* stream) {
    int st = check_route(T, E, k, dtype, score, scale);
    if (st != FP8GEMM_OK) return st;
    if (n_group <= 0 || E % n_group != 0 || topk_group <= 0 || topk_group > n_group) return FP8GEMM_ERR_BAD_SHAPE;
    const int32_t size = E / n_group;
    if (k > topk_group * size || (n_group > 1 && (group_top < 1 || group_top > 2 || group_top > size)))
        return FP8GEMM_ERR_BAD_SHAPE;
    if (n_group > kRouteMaxGroups) return FP8GEMM_ERR_UNSUPPORTED;
    if (T == 0) return FP8GEMM_OK;
    if (!logits || !ids || !weights) return FP8GEMM_ERR_NULL_PTR;
    if (!aligned(logits, dtype == FP8GEMM_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return FP8GEMM_ERR_MISALIGNED;
    RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.T = T;
    a.E = E;
    a.k = k;
    a.n_group = topk_group == n_group ? 1 : n_group;   // every group stays: no choice between them
    a.topk_group = topk_group;
    a.group_top = group_top;
    a.group_size = size;
    a.renorm = renorm != 0;
    a.scale = scale;
    host_set_config("route_topk T=%lld E=%lld k=%lld groups=%lld/%lld", {T, E, k, topk_group, n_group});
    launch_route_topk(a, dtype == FP8GEMM_BF16, score == FP8GEMM_SCORE_SIGMOID, static_cast<hipStream_t>(stream));
    return launched();
}

int fp8gemm_route_topk_backward(const void* logits, const int32_t* ids, const float* dweights, void* dlogits, int64_t T,
                                int32_t E, int32_t k, int32_t dtype, int32_t score, int32_t renorm, float scale,
                                void* stream) {
    const int st = check_route(T, E, k, dtype, score, scale);
    if (st != FP8GEMM_OK) return st;
    if (T == 0) return FP8GEMM_OK;
    if (!logits || !ids || !dweights || !dlogits) return FP8GEMM_ERR_NULL_PTR;
    const uintptr_t al = dtype == FP8GEMM_F32 ? 4 : 2;
    if (!aligned(logits, al) || !aligned(dlogits, al) || !aligned(ids, 4) || !aligned(dweights, 4))
        return FP8GEMM_ERR_MISALIGNED;
    RouteBackwardArgs a{};
    a.logits = logits;
    a.ids = ids;
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.T = T;
    a.E = E;
    a.k = k;
    a.renorm = renorm != 0;
    a.scale = scale;
    host_set_config("route_topk_backward T=%lld E=%lld k=%lld", {T, E, k});
    launch_route_backward(a, dtype == FP8GEMM_BF16, score == FP8GEMM_SCORE_SIGMOID, static_cast<hipStream_t>(stream));
    return launched();
}

int fp8gemm_moe_dispatch_masked(const void* X, const int32_t* ids, void* A, float* sa, int32_t* masked_m,
                                int32_t* row_map, int64_t T, int64_t H, int32_t k, int32_t G, int64_t M_max,
                                int32_t first_expert, void* stream) {
    int st = check_dispatch(T, H, k, G, M_max);
    if (st != FP8GEMM_OK) return st;
    if (first_expert < 0) return FP8GEMM_ERR_BAD_SHAPE;
    if (M_max > kMaxRows / G || (int64_t)G * M_max * H >= kMaxBytes) return FP8GEMM_ERR_UNSUPPORTED;
    if (!masked_m || (T > 0 && (!X || !ids || !row_map || (M_max > 0 && (!A || !sa))))) return FP8GEMM_ERR_NULL_PTR;
    if (!aligned(X, 16) || !aligned(A, 16) || !aligned(sa, 4) || !aligned(ids, 4) || !aligned(masked_m, 4) ||
        !aligned(row_map, 4))
        return FP8GEMM_ERR_MISALIGNED;
    DispatchArgs a{};
    a.X = static_cast<const uint16_t*>(X);
    a.ids = ids;
    a.A = static_cast<uint8_t*>(A);
    a.sa = sa;
    a.where = masked_m;
    a.row_map = row_map;
    a.T = T;
    a.H = (int32_t)H;
    a.k = k;
    a.G = G;
    a.first = first_expert;
    a.cap = (int32_t)M_max;
    return dispatch(a, static_cast<hipStream_t>(stream));
}

int fp8gemm_moe_dispatch_contiguous(const void* X, const int32_t* ids, void* A, float* sa, int32_t* m_indices,
                                    int32_t* row_map, int64_t T, int64_t H, int32_t k, int32_t G, int64_t M_total,
                                    int32_t first_expert, void* stream) {
    int st = check_dispatch(T, H, k, G, M_total);
    if (st != FP8GEMM_OK) return st;
    if (first_expert < 0) return FP8GEMM_ERR_BAD_SHAPE;
    if (M_total > kMaxRows || M_total * H >= kMaxBytes) return FP8GEMM_ERR_UNSUPPORTED;
    if ((M_total > 0 && !m_indices) || (T > 0 && (!X || !ids || !row_map || (M_total > 0 && (!A || !sa)))))
        return FP8GEMM_ERR_NULL_PTR;
    if (!aligned(X, 16) || !aligned(A, 16) || !aligned(sa, 4) || !aligned(ids, 4) || !aligned(m_indices, 4) ||
        !aligned(row_map, 4))
        return FP8GEMM_ERR_MISALIGNED;
    DispatchArgs a{};
    a.X = static_cast<const uint16_t*>(X);
    a.ids = ids;
    a.A = static_cast<uint8_t*>(A);
    a.sa = sa;
    a.where = m_indices;
    a.row_map = row_map;
    a.T = T;
    a.H = (int32_t)H;
    a.k = k;
    a.G = G;
    a.first = first_expert;
    a.cap = (int32_t)M_total;
    a.contiguous = 1;
    return dispatch(a, static_cast<hipStream_t>(stream));
}

int fp8gemm_moe_combine(const void* Y, const float* weights, const int32_t* row_map, void* out, int64_t T, int64_t H,
                        int32_t k, int64_t R, void* stream) {
    int st = check_combine(T, H, k, R, row_map, false);
    if (st != FP8GEMM_OK) return st;
    if (T == 0) return FP8GEMM_OK;
    if (!out || (R > 0 && !Y)) return FP8GEMM_ERR_NULL_PTR;
    if (!aligned(Y, 16) || !aligned(out, 16) || !aligned(weights, 4) || !aligned(row_map, 4)) return FP8GEMM_ERR_MISALIGNED;
    HostDevice d;
    st = host_device(&d);
    if (st != FP8GEMM_OK) return st;
    CombineArgs a{};
    a.Y = static_cast<const uint16_t*>(Y);
    a.weights = weights;
    a.row_map = row_map;
    a.out = static_cast<uint16_t*>(out);
    a.T = T;
    a.R = R;
    a.H = (int32_t)H;
    a.k = k;
    a.err = d.err;
    host_set_config("moe_combine T=%lld k=%lld H=%lld", {T, k, H});
    launch_combine(a, static_cast<hipStream_t>(stream));
    return launched();
}

int fp8gemm_moe_combine_backward(const void* dout, const void* Y, const float* weights, const int32_t* row_map, void* dY,
                                 float* dweights, int64_t T, int64_t H, int32_t k, int64_t R, void* stream) {
    int st = check_combine(T, H, k, R, row_map, true);
    if (st != FP8GEMM_OK) return st;
    if (T == 0) return FP8GEMM_OK;
    if (!dout || (R > 0 && (!dY || (dweights && !Y)))) return FP8GEMM_ERR_NULL_PTR;
    if (!aligned(dout, 16) || !aligned(Y, 16) || !aligned(dY, 16) || !aligned(weights, 4) || !aligned(row_map, 4) ||
        !aligned(dweights, 4))
        return FP8GEMM_ERR_MISALIGNED;
    HostDevice d;
    st = host_device(&d);
    if (st != FP8GEMM_OK) return st;
    CombineArgs a{};
    a.Y = static_cast<const uint16_t*>(Y);
    a.weights = weights;
    a.row_map = row_map;
    a.dout = static_cast<const uint16_t*>(dout);
    a.dY = static_cast<uint16_t*>(dY);
    a.dweights = dweights;
    a.T = T;
    a.R = R;
    a.H = (int32_t)H;
    a.k = k;
    a.err = d.err;
    host_set_config("moe_combine_backward T=%lld k=%lld H=%lld", {T, k, H});
    launch_combine_backward(a, static_cast<hipStream_t>(stream));
    return launched();
}

int fp8gemm_w4_gemv(const void* X, const void* W, const void* scales, const uint8_t* zeros, void* Y, int64_t M, int64_t N,
                    int64_t K, int32_t format, int32_t group, void* stream) {
    int st = check_w4(M, 1, N, K, format, group, zeros);
    if (st != FP8GEMM_OK) return st;
    if (M > (int64_t(1) << 20)) return FP8GEMM_ERR_UNSUPPORTED;   // the grid's second dimension
    if (M == 0 || N == 0) return FP8GEMM_OK;
    st = check_w4_ptrs(X, W, scales, zeros, Y);
    if (st != FP8GEMM_OK) return st;
    W4Args a{};
    a.X = static_cast<const uint16_t*>(X);
    a.W = static_cast<const uint8_t*>(W);
    a.scales = scales;
    a.zeros = zeros;
    a.Y = static_cast<uint16_t*>(Y);
    a.M = M;
    a.N = a.nout = (int32_t)N;
    a.K = (int32_t)K;
    a.groups = (int32_t)(K / group);
    a.div_k = make_fastdiv(1);
    HostDevice d;
    st = host_device(&d);
    if (st != FP8GEMM_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    a.cols = (int32_t)std::min<int64_t>(M, 16);
    const int rn = w4_row_tiles(N, K, a.cols, (M + 15) / 16, true, d.cus);
    a.tiles_per_wave = w4_tiles_per_wave(N, K, a.cols, (M + 15) / 16, d.cus);
    host_set_config(format == FP8GEMM_W4_MXFP4 ? "w4_gemv mxfp4 group=%lld M=%lld N=%lld K=%lld rn=%lld tiles_per_wave=%lld"
                                               : "w4_gemv int4 group=%lld M=%lld N=%lld K=%lld rn=%lld tiles_per_wave=%lld",
                    {group, M, N, K, rn, a.tiles_per_wave});
    launch_w4(a, rn, group, format == FP8GEMM_W4_MXFP4, s);
    return launched();
}

int fp8gemm_w4_gemv_experts(const void* X, const void* W, const void* scales, const uint8_t* zeros, const int32_t* ids,
                            void* Y, int64_t T, int32_t k, int32_t E, int64_t N, int64_t K, int32_t format, int32_t group,
                            int32_t first_expert, int32_t x_per_pair, int32_t swiglu, void* stream) {
    if (T < 0 || k <= 0 || E <= 0 || first_expert < 0) return FP8GEMM_ERR_BAD_SHAPE;
    int st = check_w4(T, E, N, K, format, group, zeros);
    if (st != FP8GEMM_OK) return st;
    if (swiglu && N % 2 != 0) return FP8GEMM_ERR_BAD_SHAPE;
    if (T > kMaxPairs / k || E > 65534 || T * k * N * 2 >= kMaxBytes || (x_per_pair ? T * k : T) * K * 2 >= (int64_t(1) << 31))
        return FP8GEMM_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return FP8GEMM_OK;
    st = check_w4_ptrs(X, W, scales, zeros, Y);
    if (st != FP8GEMM_OK) return st;
    if (!ids) return FP8GEMM_ERR_NULL_PTR;
    if (!aligned(ids, 4)) return FP8GEMM_ERR_MISALIGNED;
    W4Args a{};
    a.X = static_cast<const uint16_t*>(X);
    a.W = static_cast<const uint8_t*>(W);
    a.scales = scales;
    a.zeros = zeros;
    a.Y = static_cast<uint16_t*>(Y);
    a.ids = ids;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.half = swiglu ? (int32_t)(N / 2) : 0;
    a.nout = swiglu ? a.half : a.N;
    a.groups = (int32_t)(K / group);
    a.pairs = (int32_t)(T * k);
    a.E = E;
    a.first = first_expert;
    a.by_slot = a.pairs <= std::min(E, kW4MaxPairsBySlot);
    a.per_pair = x_per_pair != 0;
    a.xrows = (int32_t)(x_per_pair ? T * k : T);
    a.div_k = make_fastdiv((uint32_t)k);
    HostDevice d;
    st = host_device(&d);
    if (st != FP8GEMM_OK) return st;
    const int64_t busy = std::min<int64_t>(a.pairs, E);
    a.cols = w4_expert_rows(T, a.pairs, E, K);
    a.tiles_per_wave = w4_tiles_per_wave(a.nout, K, a.cols, busy, d.cus);
    const int rn = swiglu ? 2 : w4_row_tiles(a.nout, K, a.cols, busy, false, d.cus);
    host_set_config(format == FP8GEMM_W4_MXFP4
                        ? "w4_gemv_experts mxfp4 group=%lld pairs=%lld N=%lld K=%lld rn=%lld tiles_per_wave=%lld by_pair=%lld"
                        : "w4_gemv_experts int4 group=%lld pairs=%lld N=%lld K=%lld rn=%lld tiles_per_wave=%lld by_pair=%lld",
                    {group, a.pairs, N, K, rn, a.tiles_per_wave, a.by_slot});
    launch_w4_experts(a, rn, group, format == FP8GEMM_W4_MXFP4, swiglu != 0, static_cast<hipStream_t>(stream));
    return launched();
}

}  // extern "C"
