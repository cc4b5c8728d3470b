// route_kernels.hip -- gfx950 kernels of the expert router: for each token the k experts with the
// best scores and their weights (route_topk), and the gradient of those weights with respect to
// the logits (route_topk_backward).  The mathematics is stated in include/fp8gemm.h.
//
// Sixteen lanes, one DPP row, own one token: reductions over a token are four cross-lane steps
// without LDS, four tokens advance together in every instruction of a wave, and no work is
// shared between waves.  The choice values of a token stand in LDS as 16 chunks of V consecutive
// experts.  A pick is a two-level tournament: the best chunk maximum (one per lane), then the V
// values of that chunk (one or a few per lane); both levels find the lowest index that equals
// the maximum with a ballot, so ties go to the lowest index.

#include "moe_device.h"
#include "moe_internal.h"

namespace fp8gemm {
namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr float kBig = 3.402823466e38f;

// NaN counts as -infinity, +infinity as the largest finite value.
__device__ __forceinline__ float clean(float x) { return x != x ? kNegInf : fminf(x, kBig); }

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (BF16) return clean(bf16_to_f32(static_cast<const uint16_t*>(p)[i]));
    else return clean(static_cast<const float*>(p)[i]);
}

__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x)); }

// Lowest set bit of the 16 bits of `ballot` that belong to DPP row `row` (16 if none).
__device__ __forceinline__ int first_in_row(uint64_t ballot, int row) {
    return __builtin_ctz(((uint32_t)(ballot >> (row * 16)) & 0xFFFFu) | 0x10000u);
}

// V: values per lane and chunk length (E <= 16 V); WAVES * 4 tokens per workgroup.
template <bool BF16, bool SIGMOID, int V, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void route_topk_kernel(RouteArgs a) {
    // chunk stride in floats: 16-byte aligned, and 16 lanes reading their chunks 16 bytes at a
    // time touch every bank group once
    constexpr int CS = V < 4 ? V : V + 4;
    __shared__ float lds_c[WAVES * 4][16 * CS];
    __shared__ float lds_g[WAVES * 4][kRouteMaxGroups];
    const int lane = threadIdx.x & 63, row = lane >> 4, l = lane & 15;
    const int slot = (threadIdx.x >> 6) * 4 + row;
    const int64_t token = (int64_t)blockIdx.x * (WAVES * 4) + slot;
    const bool live = token < a.T;
    const int64_t tok = live ? token : a.T - 1;   // rows past the end repeat the last token and store nothing
    const int64_t base = tok * a.E;
    float* c = lds_c[slot];
    auto at = [](int e) { return (e / V) * CS + (e & (V - 1)); };

    // scores and choice values, lane-strided so that a row's loads are consecutive
    float s[V];
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 16 + l;
        s[i] = e < a.E ? load_logit<BF16>(a.logits, base + e) : kNegInf;
        m = fmaxf(m, s[i]);
    }
    // scores: sigmoid(x), or exp(x - m) * inv with m and inv = 1 / sum of the token's softmax; the sum
    // is formed only where scores are used as such (a renormalised weight cancels it)
    float inv = 1.0f;
    if constexpr (!SIGMOID) {
        m = row16_max_f(m);
        if (m == kNegInf) m = 0.0f;   // a row with no finite logit: every score is 0
        if (!a.renorm || a.bias || (a.n_group > 1 && a.group_top == 2)) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += s[i] == kNegInf ? 0.0f : exp_f32(s[i] - m);
            sum = row16_sum_f(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        }
    }
    auto score = [&](float x) { return SIGMOID ? sigmoid_f32(x) : exp_f32(x - m) * inv; };
    // choice values: score + bias; without a bias the logits, which order as the scores do and stay
    // apart where scores round to the same value
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 16 + l;
        float v = s[i];
        if (a.bias && e < a.E && v != kNegInf) v = score(v) + clean(a.bias[e]);
        c[at(e)] = v;
    }
    wave_sync();

    // groups: the sum of each one's best (or best two) choice values, kept if fewer than
    // topk_group others are better (or as good with a lower index)
    uint64_t keep = ~0ull;
    if (a.n_group > 1) {
        float* gs = lds_g[slot];
        for (int g = l; g < a.n_group; g += 16) {
            float m1 = kNegInf, m2 = kNegInf;
            for (int q = 0; q < a.group_size; ++q) {
                const float v = c[at(g * a.group_size + q)];
                m2 = fmaxf(m2, fminf(m1, v));
                m1 = fmaxf(m1, v);
            }
            // (without a bias the sum is of scores; a single largest one orders as its logit)
            gs[g] = a.group_top == 1 ? m1 : m2 == kNegInf ? kNegInf : a.bias ? m1 + m2 : score(m1) + score(m2);
        }
        wave_sync();
        keep = 0;
        for (int g0 = 0; g0 < a.n_group; g0 += 16) {
            const int g = g0 + l;
            const float mine = g < a.n_group ? gs[g] : kNegInf;
            int better = 0;
            for (int h = 0; h < a.n_group; ++h) {
                const float o = gs[h];
                better += (o > mine || (o == mine && h < g)) ? 1 : 0;
            }
            const uint64_t b = __ballot(g < a.n_group && better < a.topk_group);
            keep |= ((b >> (row * 16)) & 0xFFFFull) << g0;
        }
    }

    // chunk maxima, with the groups that were not kept struck out
    float cm = kNegInf;
    {
        int g = a.n_group > 1 ? l * V / a.group_size : 0;
        int left = a.n_group > 1 ? a.group_size - (l * V - g * a.group_size) : 1 << 30;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v = c[l * CS + i];
            if (a.n_group > 1) {
                if (left == 0) { ++g; left = a.group_size; }
                --left;
                if (g < a.n_group && !((keep >> g) & 1)) {
                    v = kNegInf;
                    c[l * CS + i] = v;
                }
            }
            cm = fmaxf(cm, v);
        }
    }
    wave_sync();

    // k picks; lane j keeps pick j, and pick 16 + j
    int pick0 = -1, pick1 = -1;
    for (int j = 0; j < a.k; ++j) {
        const float best = row16_max_f(cm);
        const int w = first_in_row(__ballot(cm == best), row);
        int found = V;
        float next = kNegInf;
#pragma unroll
        for (int q = 0; q < (V + 15) / 16; ++q) {
            const int i = q * 16 + l;
            float v = (V >= 16 || i < V) ? c[w * CS + i] : kNegInf;
            const int f = first_in_row(__ballot((V >= 16 || i < V) && v == best), row);
            if (found == V && f < 16) {
                found = q * 16 + f;
                if (l == f) {
                    c[w * CS + i] = kNegInf;
                    v = kNegInf;
                }
            }
            next = fmaxf(next, v);
        }
        next = row16_max_f(next);
        if (l == w) cm = next;
        if (l == (j & 15)) {
            const int e = best > kNegInf ? w * V + found : -1;
            if (j < 16) pick0 = e;
            else pick1 = e;
        }
        wave_sync();
    }

    // weights: the picked experts' scores without the bias
    float w0 = 0.0f, w1 = 0.0f;
    if (l < a.k && pick0 >= 0) w0 = score(load_logit<BF16>(a.logits, base + pick0));
    if (16 + l < a.k && pick1 >= 0) w1 = score(load_logit<BF16>(a.logits, base + pick1));
    float f = a.scale;
    if (a.renorm) {
        const float sum = row16_sum_f(w0 + w1);
        f = sum > 0.0f ? a.scale / sum : 0.0f;
    }
    if (live) {
        if (l < a.k) {
            a.ids[token * a.k + l] = pick0;
            a.weights[token * a.k + l] = w0 * f;
        }
        if (16 + l < a.k) {
            a.ids[token * a.k + 16 + l] = pick1;
            a.weights[token * a.k + 16 + l] = w1 * f;
        }
    }
}

// Gradient of the weights with respect to the logits.  Renormalised weights, and sigmoid scores,
// depend on the picked experts' logits alone; softmax scores as they are depend on every logit.
template <bool BF16, bool SIGMOID, int V, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void route_backward_kernel(RouteBackwardArgs a) {
    __shared__ float lds_d[WAVES * 4][16 * V];
    const int lane = threadIdx.x & 63, row = lane >> 4, l = lane & 15;
    const int slot = (threadIdx.x >> 6) * 4 + row;
    const int64_t token = (int64_t)blockIdx.x * (WAVES * 4) + slot;
    const bool live = token < a.T;
    const int64_t tok = live ? token : a.T - 1;
    const int64_t base = tok * a.E;
    const bool dense = !SIGMOID && !a.renorm;
    float* d = lds_d[slot];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i * 16 + l] = 0.0f;

    // this lane's picks (l and 16 + l): index, logit and incoming gradient
    int id[2];
    float x[2], g[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int j = q * 16 + l;
        id[q] = j < a.k ? a.ids[tok * a.k + j] : -1;
        if (id[q] >= a.E) id[q] = -1;
        x[q] = id[q] >= 0 ? load_logit<BF16>(a.logits, base + id[q]) : kNegInf;
        g[q] = id[q] >= 0 ? a.scale * a.dweights[tok * a.k + j] : 0.0f;
    }
    float s[V];
    float m, sum = 0.0f;
    if (dense) {
        m = kNegInf;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = i * 16 + l;
            s[i] = e < a.E ? load_logit<BF16>(a.logits, base + e) : kNegInf;
            m = fmaxf(m, s[i]);
        }
        m = row16_max_f(m);
        if (m == kNegInf) m = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = s[i] == kNegInf ? 0.0f : exp_f32(s[i] - m);
            sum += s[i];
        }
        sum = row16_sum_f(sum);
    } else {
        m = row16_max_f(fmaxf(x[0], x[1]));   // a softmax over the picks is all that renormalised scores need
        if (m == kNegInf) m = 0.0f;
    }
    float p[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        p[q] = x[q] == kNegInf ? 0.0f : (SIGMOID ? sigmoid_f32(x[q]) : exp_f32(x[q] - m));
    if (a.renorm) {
        const float total = row16_sum_f(p[0] + p[1]);
        const float r = total > 0.0f ? 1.0f / total : 0.0f;
        const float mean = row16_sum_f(g[0] * (p[0] * r) + g[1] * (p[1] * r));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            // sigmoid: ds = (g - mean) / total, dx = ds s (1 - s); softmax: dx = (g - mean) s / total
            float v = (g[q] - mean) * (p[q] * r);
            if constexpr (SIGMOID) v *= sigmoid_f32(-x[q]);
            if (id[q] >= 0) d[id[q]] = x[q] == kNegInf ? 0.0f : v;
        }
    } else if constexpr (SIGMOID) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (id[q] >= 0) d[id[q]] = g[q] * p[q] * sigmoid_f32(-x[q]);
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (id[q] >= 0) d[id[q]] = g[q];
    }
    wave_sync();
    float mean = 0.0f, r = 1.0f;
    if (dense) {
        r = sum > 0.0f ? 1.0f / sum : 0.0f;
        mean = row16_sum_f(g[0] * (p[0] * r) + g[1] * (p[1] * r));
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 16 + l;
        if (e < a.E) {
            float v = d[e];
            if (dense) v = (v - mean) * (s[i] * r);
            if constexpr (BF16) static_cast<uint16_t*>(a.dlogits)[base + e] = f32_to_bf16(v);
            else static_cast<float*>(a.dlogits)[base + e] = v;
        }
    }
}

template <int V, int WAVES>
void launch_forward(const RouteArgs& a, bool bf16, bool sigmoid, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + WAVES * 4 - 1) / (WAVES * 4))), block(WAVES * 64);
    if (bf16 && sigmoid) hipLaunchKernelGGL((route_topk_kernel<true, true, V, WAVES>), grid, block, 0, s, a);
    else if (bf16) hipLaunchKernelGGL((route_topk_kernel<true, false, V, WAVES>), grid, block, 0, s, a);
    else if (sigmoid) hipLaunchKernelGGL((route_topk_kernel<false, true, V, WAVES>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((route_topk_kernel<false, false, V, WAVES>), grid, block, 0, s, a);
}

template <int V, int WAVES>
void launch_back(const RouteBackwardArgs& a, bool bf16, bool sigmoid, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + WAVES * 4 - 1) / (WAVES * 4))), block(WAVES * 64);
    if (bf16 && sigmoid) hipLaunchKernelGGL((route_backward_kernel<true, true, V, WAVES>), grid, block, 0, s, a);
    else if (bf16) hipLaunchKernelGGL((route_backward_kernel<true, false, V, WAVES>), grid, block, 0, s, a);
    else if (sigmoid) hipLaunchKernelGGL((route_backward_kernel<false, true, V, WAVES>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((route_backward_kernel<false, false, V, WAVES>), grid, block, 0, s, a);
}

}  // namespace

// The chunk length is the smallest power of two that holds E experts in 16 chunks; 64-value
// chunks take one wave per workgroup to stay within static LDS.
void launch_route_topk(const RouteArgs& a, bool bf16, bool sigmoid, hipStream_t s) {
    if (a.E <= 64) launch_forward<4, 4>(a, bf16, sigmoid, s);
    else if (a.E <= 128) launch_forward<8, 4>(a, bf16, sigmoid, s);
    else if (a.E <= 256) launch_forward<16, 4>(a, bf16, sigmoid, s);
    else if (a.E <= 512) launch_forward<32, 4>(a, bf16, sigmoid, s);
    else launch_forward<64, 1>(a, bf16, sigmoid, s);
}

void launch_route_backward(const RouteBackwardArgs& a, bool bf16, bool sigmoid, hipStream_t s) {
    if (a.E <= 64) launch_back<4, 4>(a, bf16, sigmoid, s);
    else if (a.E <= 128) launch_back<8, 4>(a, bf16, sigmoid, s);
    else if (a.E <= 256) launch_back<16, 4>(a, bf16, sigmoid, s);
    else if (a.E <= 512) launch_back<32, 4>(a, bf16, sigmoid, s);
    else launch_back<64, 1>(a, bf16, sigmoid, s);
}

}  // namespace fp8gemm
