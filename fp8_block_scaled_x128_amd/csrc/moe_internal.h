// moe_internal.h -- types shared by the kernels around the grouped products (expert routing, token
// permutation, 4-bit matrix-vector products) and their host code, and the services of
// fp8gemm_api.cpp (device set-up, per-stream workspace, last configuration) that code uses.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <mutex>

#include "fp8gemm_args.h"

namespace fp8gemm {

// ---- services of fp8gemm_api.cpp ----
struct HostDevice {
    int cus = 0;
    int32_t* err = nullptr;     // device error word
};
int host_device(HostDevice* out);                                       // status code
// The stream's library-owned workspace (see fp8gemm.h): `bytes` of scratch, status code.  `hold` keeps
// other threads' calls off it and is kept until the last launch that uses it is enqueued.
int host_stream_scratch(hipStream_t stream, size_t bytes, void** scratch, std::unique_lock<std::mutex>* hold);
// The calling thread's last configuration: a static format of %lld fields and at most 8 values.
void host_set_config(const char* fmt, std::initializer_list<long long> values);

// ---- routing ----
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 32;
constexpr int kRouteMaxGroups = 64;

struct RouteArgs {
    const void* logits;         // [T][E] fp32 or bf16
    const float* bias;          // [E] or null
    int32_t* ids;               // [T][k]
    float* weights;             // [T][k]
    int64_t T;
    int32_t E, k;
    int32_t n_group, topk_group, group_top, group_size;
    int32_t group_lanes;        // lanes (1, 2, 4 or 8) whose chunks hold a group, 0 if groups do not fit so
    int32_t group_pad;          // places left free after each group's experts in its lanes' chunks
    int32_t group_shift;        // log2 of a group's places (with group_pad)
    FastDiv div_group;          // by group_size (with group_pad)
    int32_t renorm;
    float scale;
};

struct RouteBackwardArgs {
    const void* logits;         // [T][E] fp32 or bf16
    const int32_t* ids;         // [T][k]
    const float* dweights;      // [T][k]
    void* dlogits;              // [T][E], the type of logits
    int64_t T;
    int32_t E, k;
    int32_t renorm;
    float scale;
};

void launch_route_topk(const RouteArgs& a, bool bf16, bool sigmoid, hipStream_t s);
void launch_route_backward(const RouteBackwardArgs& a, bool bf16, bool sigmoid, hipStream_t s);

// ---- token permutation ----
// The row passes: a workgroup of kRowThreads takes kRowSpan bf16 values of a row, 16 bytes a thread.
constexpr int kRowThreads = 256, kRowSpan = kRowThreads * 8;
inline int64_t row_spans(int H) { return (H + kRowSpan - 1) / kRowSpan; }
// Threads of the large dispatch's workgroup per token: 16 values each, in whole waves.
inline int dispatch_copy_threads(int H) { return H >= 16384 ? 1024 : (H / 16 + 63) / 64 * 64; }
constexpr int kDispatchMaxGroups = 1024;
constexpr int kDispatchMaxTopk = 32;

struct DispatchArgs {
    const uint16_t* X;          // [T][H] bf16 bits
    const int32_t* ids;         // [T][k]
    uint8_t* A;                 // masked [G][cap][H], contiguous [cap][H]
    float* sa;                  // masked [G][nkb][cap], contiguous [nkb][cap]
    int32_t* where;             // masked: masked_m [G]; contiguous: m_indices [cap]
    int32_t* row_map;           // [T][k]
    int32_t* scratch;           // large batches: counts and local ranks
    int32_t* err;
    int64_t T;
    int32_t H, nkb, k, G, first, cap;
    int32_t contiguous;
    int32_t pairs;              // T * k
    int32_t chunks;             // large batches: ceil(pairs / kDispatchChunk)
    int32_t by_row;             // large batches: scales by token in scratch, turned round by a pass of their own
    FastDiv div_k;
};

constexpr int kDispatchChunk = 1024;   // pairs ranked by one workgroup of the counting pass

void launch_dispatch(const DispatchArgs& a, bool large, hipStream_t s);

struct CombineArgs {
    const uint16_t* Y;          // [R][H] bf16 bits
    const float* weights;       // [T][k] or null (ones)
    const int32_t* row_map;     // [T][k] or null (row t * k + j)
    uint16_t* out;              // [T][H]
    const uint16_t* dout;       // backward: [T][H]
    uint16_t* dY;               // backward: [R][H]
    float* dweights;            // backward: [T][k]
    int64_t T, R;
    int32_t H, k;
    int32_t* err;
};

constexpr int kCombineMaxTopk = 32;

void launch_combine(const CombineArgs& a, hipStream_t s);
void launch_combine_backward(const CombineArgs& a, hipStream_t s);

// ---- 4-bit matrix-vector products ----
constexpr int kW4MaxPairsBySlot = 1024;

struct W4Args {
    const uint16_t* X;          // [rows][K] bf16 bits
    const uint8_t* W;           // [(E)][N][K/2]
    const void* scales;         // [(E)][N][K/group]: E8M0 bytes or bf16
    const uint8_t* zeros;       // [(E)][N][K/group] or null
    uint16_t* Y;                // [M][N] (or [pairs][N/2] with SwiGLU)
    const int32_t* ids;         // experts: [pairs]
    int64_t M;                  // rows of X (dense)
    int32_t N, K;               // N: rows of one matrix
    int32_t nout;               // columns of Y
    int32_t groups;             // K / group
    int32_t half;               // SwiGLU: N / 2 (row offset of the up rows)
    int32_t pairs, E, first;    // experts
    int32_t by_slot;            // experts: grid.y counts pairs (else experts)
    int32_t per_pair;           // experts: X has a row per pair (else per token)
    FastDiv div_k;              // pair -> token
    int32_t xrows;              // experts: rows of X
    int32_t tiles_per_wave;     // 0: a workgroup's waves share the K of one tile
    int32_t cols;               // rows of X a pass takes (at most 16)
    int32_t xsteps, xstride;    // X in LDS: steps of 128 values, bytes of a row
    FastDiv div_units;          // 16-byte units of a row
};

// rn: 16-row tiles of V per workgroup where its waves share K.
void launch_w4(const W4Args& a, int rn, int group, bool mxfp4, hipStream_t s);
void launch_w4_experts(const W4Args& a, int rn, int group, bool mxfp4, bool swiglu, hipStream_t s);

}  // namespace fp8gemm
