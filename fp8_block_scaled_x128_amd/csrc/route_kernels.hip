// route_kernels.hip -- gfx950 kernels of the expert router: for each token the k experts with the
// best scores and their weights (route_topk), and the gradient of those weights with respect to
// the logits (route_topk_backward).  The mathematics is stated in include/fp8gemm.h.
//
// Sixteen lanes, one DPP row, own one token: reductions over a token are four cross-lane steps
// without LDS, four tokens advance together in every instruction of a wave, and no work is
// shared between waves.  The choice values of a token stand in LDS as 16 chunks of V consecutive
// experts, chunk l read back by lane l.  A pick is a two-level tournament: the best chunk maximum
// (one per lane), then the V values of that chunk (one or a few per lane); both levels find the
// lowest index that equals the maximum with a ballot, so ties go to the lowest index.  Groups of
// whole chunks take their scores from the chunks' two best values, merged across the group's
// lanes, and strike out whole chunk maxima.  Where 16 lanes divided by the groups (rounded up to a
// power of two) hold a group, it is given those lanes' chunks to itself, with places left free after
// it (32768 x 160 bf16 softmax, bias, 3 of 8 groups, 6 picks: 14.4 us, against 16.9 with groups scanned in
// LDS by a lane each, which stays for the others).
//
// Bound: instructions, then memory: 32768 x 256 fp32, sigmoid, bias, 4 of 8 groups, 8 picks: 13.2 us,
// 2.7 TB/s, 850 vector instructions a wave of 4 tokens, about 30 of them for each pick and the rest for a
// lane's 16 experts' scores, keys and places; a single token 4.4 us, its picks' chain of dependent steps past
// a launch's 2.8 us; gradient 8191 x 160 bf16, 6 picks: 4.1 us.

#include "fp8gemm_device.h"
#include "fp8gemm_internal.h"
#include "moe_device.h"
#include "moe_internal.h"

namespace fp8gemm {
namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr float kBig = 3.402823466e38f;

// NaN counts as -infinity, +infinity as the largest finite value (the maximum of NaN and a number
// is the number).
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, kNegInf), kBig); }

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (BF16) return clean(bf16_to_f32(static_cast<const uint16_t*>(p)[i]));
    else return clean(static_cast<const float*>(p)[i]);
}

// e^x within 2 units in the last place where it is above 2^-126, which it may replace by 0 below: the
// hardware's 2^h, h = x log2(e) rounded, times 1 + r with r = x - h log(2) what the rounding left out.
__device__ __forceinline__ float exp_normal_f32(float x) {
    x = __builtin_amdgcn_fmed3f(x, -88.0f, 88.0f);
    const float h = x * 1.44269504088896341f;
    const float r = __builtin_fmaf(h, 1.90465429995776804e-9f, __builtin_fmaf(h, -0.693147182464599609f, x));
    const float e = __builtin_amdgcn_exp2f(h);
    return __builtin_fmaf(e, r, e);
}

// 1 / (1 + e^-x) with e^-|x| alone, so that scores below 2^-126 are not lost in the reciprocal.
__device__ __forceinline__ float sigmoid_f32(float x) {
    const float e = exp_f32(-__builtin_fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e);
    return x < 0.0f ? e * r : r;
}

// The score of a pick with logit x up to a factor common to a token's picks, of which `most` is the largest
// logit.  Renormalised weights are shares: taken from these values, of which the largest is 1/2 at least, they
// are finite and exact to rounding where the scores themselves come near the end of the type.
template <bool SIGMOID>
__device__ __forceinline__ float share_f32(float x, float most) {
    if constexpr (!SIGMOID) return exp_f32(x - most);
    const float e = exp_f32(-__builtin_fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e);
    return x < 0.0f ? exp_f32(x - fminf(most, 0.0f)) * r : r;
}
constexpr float kNoScore = -104.0f;   // e^x rounds to 0 in 32 bits from here on

// Choice values (not -0) as integers that order as they do: the cross-lane steps of integer maxima
// are single instructions.
constexpr int kLowest = (int)0x807FFFFFu;   // of -infinity
__device__ __forceinline__ int key_of(float x) {
    const int b = __float_as_int(x);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int key) { return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF)); }

__device__ __forceinline__ int row16_max_i(int v) {
    v = max(v, dpp16<kDppXor1>(v));
    v = max(v, dpp16<kDppXor2>(v));
    v = max(v, dpp16<kDppHalfMirror>(v));
    v = max(v, dpp16<kDppMirror>(v));
    return v;
}

// Lowest lane of DPP row `row` whose bit of the ballot is set (16 if none).
__device__ __forceinline__ int first_in_row(uint64_t ballot, int row) {
    const uint32_t half = row & 2 ? (uint32_t)(ballot >> 32) : (uint32_t)ballot;
    return __builtin_ctz((half >> (row & 1) * 16) | 0x10000u);
}

// (m1, m2), the two largest of this lane's and its partner's two largest values.
template <int CTRL>
__device__ __forceinline__ void merge_top2(int& m1, int& m2) {
    const int o1 = dpp16<CTRL>(m1), o2 = dpp16<CTRL>(m2);
    m2 = max(max(min(m1, o1), m2), o2);
    m1 = max(m1, o1);
}

// A lane's share of a row of E values: V values in runs of P consecutive ones (P = 1 without
// vector loads), run i at (16 i + l) P, so that a row's 16 lanes read consecutive memory.
template <int V, int P>
__device__ __forceinline__ int element(int i, int l) { return (i / P * 16 + l) * P + i % P; }

// The lane's values of a row of logits, -infinity past E.
template <bool BF16, int V, int P>
__device__ __forceinline__ void load_row(const void* logits, int64_t base, int E, int l, float (&s)[V]) {
    // (loaded and cleaned without branches: past the end a run repeats the last, and then gives way)
#pragma unroll
    for (int i = 0; i < V; i += P) {
        const int in = min(element<V, P>(i, l), E - P);   // a run is in or out as a whole
        if constexpr (BF16) {
            uint16_t x[P];
            __builtin_memcpy(x, __builtin_assume_aligned(static_cast<const uint16_t*>(logits) + base + in, 2 * P), 2 * P);
#pragma unroll
            for (int q = 0; q < P; ++q) s[i + q] = clean(bf16_to_f32(x[q]));
        } else {
            float x[P];
            __builtin_memcpy(x, __builtin_assume_aligned(static_cast<const float*>(logits) + base + in, 4 * P), 4 * P);
#pragma unroll
            for (int q = 0; q < P; ++q) s[i + q] = clean(x[q]);
        }
    }
    if (E < 16 * V) {
#pragma unroll
        for (int i = 0; i < V; i += P) {
            const bool out = element<V, P>(i, l) >= E;
#pragma unroll
            for (int q = 0; q < P; ++q) s[i + q] = out ? kNegInf : s[i + q];
        }
    }
}

// V: values per lane and chunk length (E <= 16 V); P: values per load (E a multiple of it, rows
// aligned to a run); PAD: places are left free after each group; WAVES * 4 tokens per workgroup.
template <bool BF16, bool SIGMOID, int V, int P, bool PAD, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void route_topk_kernel(RouteArgs a) {
    // chunk stride in floats: 16-byte aligned, and 16 lanes reading their chunks 16 bytes at a
    // time touch every bank group once; tokens a quarter of the banks apart
    constexpr int CS = V + 4, ROW = 16 * CS + 16;
    __shared__ __align__(16) int lds_c[WAVES * 4][ROW];
    __shared__ float lds_g[WAVES * 4][kRouteMaxGroups];
    const int lane = threadIdx.x & 63, row = lane >> 4, l = lane & 15;
    const int slot = (threadIdx.x >> 6) * 4 + row;
    const int64_t token = (int64_t)blockIdx.x * (WAVES * 4) + slot;
    const bool live = token < a.T;
    const int64_t tok = live ? token : a.T - 1;   // rows past the end repeat the last token and store nothing
    const int64_t base = tok * a.E;
    int* c = lds_c[slot];
    auto at = [](int e) { return (e / V) * CS + (e & (V - 1)); };

    float bias[V];   // (asked for first: the same for every token, from the caches)
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < V; i += P)
            __builtin_memcpy(bias + i, __builtin_assume_aligned(a.bias + min(element<V, P>(i, l), a.E - P), 4 * P), 4 * P);
    }
    float s[V];
    load_row<BF16, V, P>(a.logits, base, a.E, l, s);

    // scores: sigmoid(x), or exp(x - m) * inv with m and inv = 1 / sum of the token's softmax; the sum
    // is formed only where scores are used as such (a renormalised weight cancels it).  Any m serves that keeps
    // the powers in range: 0 where the largest logit is 0 to 60, as x - m loses up to |x - m| 2^-24 of a score.
    float m = 0.0f, top = 0.0f, inv = 1.0f;
    if constexpr (!SIGMOID) {
        m = kNegInf;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, s[i]);
        m = row16_max_f(m);
        if (m == kNegInf) m = 0.0f;   // a row with no finite logit: every score is 0
        top = m;
        if (m >= 0.0f && m <= 60.0f) m = 0.0f;
        if (!a.renorm || a.bias || (a.n_group > 1 && a.group_top == 2)) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += exp_f32(s[i] - m);   // e^-infinity is 0
            sum = row16_sum_f(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        }
    }
    auto score = [&](float x) { return SIGMOID ? sigmoid_f32(x) : exp_f32(x - m) * inv; };
    // choice values: score + bias; without a bias the logits, which order as the scores do and stay
    // apart where scores round to the same value.  The scores in them are as exact as the weights', except
    // that those below 2^-126 may count as 0 (a bias of any use is far above): scores by the weights' functions,
    // which keep those apart, cost 14.3 us for 32768 x 256 instead of 13.2.
    auto choice_score = [&](float x) {
        if constexpr (SIGMOID) return __builtin_amdgcn_rcpf(1.0f + exp_normal_f32(-x));
        else return exp_normal_f32(x - m) * inv;
    };
    int key[V];
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i)   // (0 times a logit of -infinity makes the sum NaN, and that -infinity; never -0)
            key[i] = key_of(clean(__builtin_fmaf(s[i], 0.0f, choice_score(s[i]) + bias[i])));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key_of(s[i] + 0.0f);   // -0 as 0
    }
    constexpr int PW = P < 4 ? P : 4;   // values per LDS store
    if constexpr (PAD) {
        auto place = [&](int e) { return at(e + (int)fast_div(e, a.div_group) * a.group_pad); };
#pragma unroll
        for (int i = 0; i < V; ++i) c[l * CS + i] = kLowest;
        wave_sync();
        if (a.group_size % PW == 0) {
#pragma unroll
            for (int i = 0; i < V; i += PW) {
                const int e = element<V, P>(i, l);
                if (e < a.E) __builtin_memcpy(__builtin_assume_aligned(c + place(e), 4 * PW), key + i, 4 * PW);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = element<V, P>(i, l);
                if (e < a.E) c[place(e)] = key[i];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i += PW)
            __builtin_memcpy(__builtin_assume_aligned(c + at(element<V, P>(i, l)), 4 * PW), key + i, 4 * PW);
    }
    wave_sync();

    // this lane's chunk: its two largest values
    int m1 = kLowest, m2 = kLowest;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = c[l * CS + i];
        m2 = max(m2, min(m1, v));
        m1 = max(m1, v);
    }
    int cm = m1;   // the best of the chunk that can be picked

    if (a.n_group > 1) {
        // groups: the sum of each one's best (or best two) choice values, kept if fewer than topk_group
        // others are better (or as good with a lower index)
        float* gs = lds_g[slot];
        auto group_score = [&](int k1, int k2) {
            // (without a bias the sum is of scores; a single largest one orders as its logit)
            const float b1 = value_of(k1), b2 = value_of(k2);
            return a.group_top == 1 ? b1 : k2 == kLowest ? kNegInf : a.bias ? b1 + b2 : score(b1) + score(b2);
        };
        const int lanes = a.group_lanes;
        if (lanes) {
            if (lanes > 1) merge_top2<kDppXor1>(m1, m2);
            if (lanes > 2) merge_top2<kDppXor2>(m1, m2);
            if (lanes > 4) merge_top2<kDppHalfMirror>(m1, m2);
            if (l % lanes == 0 && l / lanes < a.n_group) gs[l / lanes] = group_score(m1, m2);
        } else {
            for (int g = l; g < a.n_group; g += 16) {
                int b1 = kLowest, b2 = kLowest;
#pragma unroll 8
                for (int q = 0; q < a.group_size; ++q) {
                    const int v = c[at(g * a.group_size + q)];
                    b2 = max(b2, min(b1, v));
                    b1 = max(b1, v);
                }
                gs[g] = group_score(b1, b2);
            }
        }
        wave_sync();
        uint64_t keep = 0;
        for (int g0 = 0; g0 < a.n_group; g0 += 16) {
            const int g = g0 + l;
            const float mine = g < a.n_group ? gs[g] : kNegInf;
            int better = 0;
#pragma unroll 8
            for (int h = 0; h < a.n_group; ++h) {
                const float o = gs[h];
                better += (int)(o > mine) | ((int)(o == mine) & (int)(h < g));
            }
            const uint64_t b = __ballot(g < a.n_group && better < a.topk_group);
            keep |= ((b >> (row * 16)) & 0xFFFFull) << g0;
        }
        if (lanes) {
            if (!((keep >> (l / lanes)) & 1)) cm = kLowest;
        } else {
            cm = kLowest;
            int g = l * V / a.group_size, left = a.group_size - (l * V - g * a.group_size);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (left == 0) { ++g; left = a.group_size; }
                --left;
                // (past the last group the shift wraps: those values are the lowest anyway)
                const int v = (keep >> (g & 63)) & 1 ? c[l * CS + i] : kLowest;
                c[l * CS + i] = v;
                cm = max(cm, v);
            }
            wave_sync();
        }
    }

    // k picks; lane j keeps pick j (index and choice value), and pick 16 + j
    int pick0 = -1, pick1 = -1, key0 = kLowest, key1 = kLowest;
    auto pick_next = [&](int j, int& pick, int& key) {
        const int best = row16_max_i(cm);
        const int w = first_in_row(__ballot(cm == best), row);
        int found = 0, next = kLowest;
        bool open = true;
#pragma unroll
        for (int q = 0; q < (V + 15) / 16; ++q) {
            const int i = V >= 16 ? q * 16 + l : l & (V - 1);    // (short chunks: copies of the values, the lowest lane wins)
            int v = c[w * CS + i];
            const int f = first_in_row(__ballot(v == best), row);
            if constexpr (V <= 16) {
                found = f;
                v = (l & (V - 1)) == f ? kLowest : v;
            } else {
                const bool hit = open && f < 16;
                found = hit ? q * 16 + f : found;
                v = hit && l == f ? kLowest : v;
                open = open && !hit;
            }
            c[w * CS + i] = v;
            next = max(next, v);
        }
        next = row16_max_i(next);
        // (with nothing left to pick, w is some chunk, perhaps of a group that was struck out: it stays out)
        cm = l == w && best != kLowest ? next : cm;
        const bool keep_it = l == j;
        pick = keep_it ? w * V + found : pick;
        key = keep_it ? best : key;
        wave_sync();
    };
    for (int j = 0; j < min(a.k, 16); ++j) pick_next(j, pick0, key0);
    for (int j = 16; j < a.k; ++j) pick_next(j - 16, pick1, key1);
    if constexpr (PAD) {                  // places to experts
        pick0 -= (pick0 >> a.group_shift) * a.group_pad;
        pick1 -= (pick1 >> a.group_shift) * a.group_pad;
    }
    if (key0 == kLowest) pick0 = -1;      // nothing left to choose
    if (key1 == kLowest) pick1 = -1;

    // weights: the picked experts' scores without the bias, or their shares
    auto logit = [&](int pick, int key) {
        if (pick < 0) return kNegInf;
        return a.bias ? load_logit<BF16>(a.logits, base + pick) : value_of(key);
    };
    const float x0 = logit(pick0, key0), x1 = a.k > 16 ? logit(pick1, key1) : kNegInf;
    float w0, w1 = 0.0f;
    if (a.renorm) {
        const float most = row16_max_f(fmaxf(x0, x1));
        const bool none = most - top < kNoScore;         // no pick, or every one's score is 0 (top is 0 for sigmoid)
        w0 = share_f32<SIGMOID>(x0, most);
        if (a.k > 16) w1 = share_f32<SIGMOID>(x1, most);
        const float sum = row16_sum_f(w0 + w1);
        w0 = none ? 0.0f : w0 / sum;                     // (not times scale / sum, which may pass the type's range)
        if (a.k > 16) w1 = none ? 0.0f : w1 / sum;
    } else {
        w0 = pick0 < 0 ? 0.0f : score(x0);
        if (a.k > 16) w1 = pick1 < 0 ? 0.0f : score(x1);
    }
    if (live) {
        if (l < a.k) {
            a.ids[token * a.k + l] = pick0;
            a.weights[token * a.k + l] = w0 * a.scale;
        }
        if (16 + l < a.k) {
            a.ids[token * a.k + 16 + l] = pick1;
            a.weights[token * a.k + 16 + l] = w1 * a.scale;
        }
    }
}

// Gradient of the weights with respect to the logits.  Renormalised weights, and sigmoid scores,
// depend on the picked experts' logits alone; softmax scores as they are depend on every logit.
template <bool BF16, bool SIGMOID, int V, int P, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void route_backward_kernel(RouteBackwardArgs a) {
    __shared__ __align__(16) float lds_d[WAVES * 4][16 * V];
    const int lane = threadIdx.x & 63, row = lane >> 4, l = lane & 15;
    const int slot = (threadIdx.x >> 6) * 4 + row;
    const int64_t token = (int64_t)blockIdx.x * (WAVES * 4) + slot;
    const bool live = token < a.T;
    const int64_t tok = live ? token : a.T - 1;
    const int64_t base = tok * a.E;
    const bool dense = !SIGMOID && !a.renorm;
    float* d = lds_d[slot];
#pragma unroll
    for (int i = 0; i < V; ++i) d[element<V, P>(i, l)] = 0.0f;

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
        load_row<BF16, V, P>(a.logits, base, a.E, l, s);
        m = kNegInf;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, s[i]);
        m = row16_max_f(m);
        if (m == kNegInf) m = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = exp_f32(s[i] - m);   // e^-infinity is 0
            sum += s[i];
        }
        sum = row16_sum_f(sum);
    } else {
        m = row16_max_f(fmaxf(x[0], x[1]));   // renormalised scores need the picks alone
        if (m == kNegInf) m = 0.0f;
    }
    float p[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        p[q] = x[q] == kNegInf ? 0.0f : SIGMOID && !a.renorm ? sigmoid_f32(x[q]) : share_f32<SIGMOID>(x[q], m);
    if (SIGMOID && a.renorm && m < kNoScore) p[0] = p[1] = 0.0f;   // the weights are 0 there
    if (a.renorm) {
        const float total = row16_sum_f(p[0] + p[1]);
        // (quotients, not products with 1 / total: a pick alone has a share of exactly 1, and no gradient)
        const float share[2] = {total > 0.0f ? p[0] / total : 0.0f, total > 0.0f ? p[1] / total : 0.0f};
        const float mean = row16_sum_f(g[0] * share[0] + g[1] * share[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            // sigmoid: ds = (g - mean) / total, dx = ds s (1 - s); softmax: dx = (g - mean) s / total
            float v = (g[q] - mean) * share[q];
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
    for (int i = 0; i < V; i += P) {
        const int e = element<V, P>(i, l);
        if (e >= a.E) continue;
        float v[P];
#pragma unroll
        for (int q = 0; q < P; ++q) {
            v[q] = d[e + q];
            if (dense) v[q] = (v[q] - mean) * (s[i + q] * r);
        }
        if constexpr (BF16) {
            uint16_t* out = static_cast<uint16_t*>(a.dlogits) + base + e;
            if constexpr (P == 1) {
                *out = f32_to_bf16(v[0]);
            } else {
                typedef uint32_t Words __attribute__((ext_vector_type(P / 2)));
                Words w;
#pragma unroll
                for (int q = 0; q < P / 2; ++q) w[q] = pack_bf16x2(v[2 * q], v[2 * q + 1]);
                *reinterpret_cast<Words*>(out) = w;
            }
        } else {
            typedef float Words __attribute__((ext_vector_type(P)));
            Words w;
#pragma unroll
            for (int q = 0; q < P; ++q) w[q] = v[q];
            *reinterpret_cast<Words*>(static_cast<float*>(a.dlogits) + base + e) = w;
        }
    }
}

template <int V, int WAVES, bool BF16, int P>
void launch_forward(const RouteArgs& a, bool sigmoid, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + WAVES * 4 - 1) / (WAVES * 4))), block(WAVES * 64);
    const bool pad = a.group_pad > 0;
    if (sigmoid && pad) hipLaunchKernelGGL((route_topk_kernel<BF16, true, V, P, true, WAVES>), grid, block, 0, s, a);
    else if (sigmoid) hipLaunchKernelGGL((route_topk_kernel<BF16, true, V, P, false, WAVES>), grid, block, 0, s, a);
    else if (pad) hipLaunchKernelGGL((route_topk_kernel<BF16, false, V, P, true, WAVES>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((route_topk_kernel<BF16, false, V, P, false, WAVES>), grid, block, 0, s, a);
}

template <int V, int WAVES, bool BF16, int P>
void launch_back(const RouteBackwardArgs& a, bool sigmoid, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + WAVES * 4 - 1) / (WAVES * 4))), block(WAVES * 64);
    if (sigmoid) hipLaunchKernelGGL((route_backward_kernel<BF16, true, V, P, WAVES>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((route_backward_kernel<BF16, false, V, P, WAVES>), grid, block, 0, s, a);
}

// Vector loads (16 bytes, 8 for 64 bf16 experts) where every row is aligned to them.
template <int V, int WAVES>
void launch_forward(RouteArgs a, bool bf16, bool sigmoid, hipStream_t s) {
    constexpr int PB = V < 8 ? V : 8;
    if (a.n_group > 1) {
        int lanes = a.group_size / V;
        if (a.group_size % V != 0 || lanes > 8 || (lanes & (lanes - 1))) {
            lanes = 8;
            while (lanes && lanes * a.n_group > 16) lanes /= 2;
            if (lanes * V < a.group_size) lanes = 0;
            if (lanes) {
                a.group_pad = lanes * V - a.group_size;
                a.group_shift = __builtin_ctz((unsigned)(lanes * V));
                a.div_group = make_fastdiv((uint32_t)a.group_size);
            }
        }
        a.group_lanes = lanes;
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.bias);
    if (bf16 && a.E % PB == 0 && at % 16 == 0) launch_forward<V, WAVES, true, PB>(a, sigmoid, s);
    else if (bf16) launch_forward<V, WAVES, true, 1>(a, sigmoid, s);
    else if (a.E % 4 == 0 && at % 16 == 0) launch_forward<V, WAVES, false, 4>(a, sigmoid, s);
    else launch_forward<V, WAVES, false, 1>(a, sigmoid, s);
}

template <int V, int WAVES>
void launch_back(const RouteBackwardArgs& a, bool bf16, bool sigmoid, hipStream_t s) {
    constexpr int PB = V < 8 ? V : 8;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits);
    if (bf16 && a.E % PB == 0 && at % (2 * PB) == 0) launch_back<V, WAVES, true, PB>(a, sigmoid, s);
    else if (bf16) launch_back<V, WAVES, true, 1>(a, sigmoid, s);
    else if (a.E % 4 == 0 && at % 16 == 0) launch_back<V, WAVES, false, 4>(a, sigmoid, s);
    else launch_back<V, WAVES, false, 1>(a, sigmoid, s);
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
