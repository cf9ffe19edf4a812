// Internal interfaces of the quantized linear operator (linear.cu, linear_gemm.cu,
// linear_stream.cu).
#pragma once
#include <type_traits>

#include "../../include/e4b.h"
#include "e4b_internal.h"

namespace e4b {

// act(z) and act'(z).  SiLU and the tanh form of GELU are both z s with s the logistic
// function of u: u = z, and u = 2 sqrt(2/pi) (z + 0.044715 z^3) (tanh(v) = 2 s(2v) - 1).
// u is taken at z clamped to +-88, so that z^3 stays finite.  y and act' leave in bf16: the fast
// exponential's error (2 + 1.17 |u| units in the last place, a relative 1e-5 at u = -88) is far
// below their half step, and s comes out 0 below u = -87.3, where it is under 2^-125.
template <int ACT>
__device__ __forceinline__ void linear_act(float z, float& y, float& d) {
    if (ACT == E4B_LINEAR_ACT_NONE) {
        y = z;
        d = 1.0f;
        return;
    }
    if (ACT == E4B_LINEAR_ACT_RELU) {
        y = z > 0.0f ? z : (z != z ? z : 0.0f);
        d = z > 0.0f ? 1.0f : 0.0f;
        return;
    }
    const float zc = fminf(fmaxf(z, -88.0f), 88.0f);
    float u = zc, du = 1.0f;
    if (ACT == E4B_LINEAR_ACT_GELU_TANH) {
        const float c = 1.5957691216057308f, q = zc * zc;
        u = c * zc * fmaf(0.044715f, q, 1.0f);
        du = c * fmaf(0.134145f, q, 1.0f);
    }
    const float s = __fdividef(1.0f, 1.0f + __expf(-u));
    y = z * s;
    d = z == z ? fmaf(zc * s * (1.0f - s), du, s) : z;
}

// f(integral_constant ACT): the branch on the kind stays outside the caller's loops, which
// keeps the elements' chains independent (inside them it serialised the epilogue).
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case E4B_LINEAR_ACT_RELU: f(std::integral_constant<int, E4B_LINEAR_ACT_RELU>()); break;
        case E4B_LINEAR_ACT_SILU: f(std::integral_constant<int, E4B_LINEAR_ACT_SILU>()); break;
        case E4B_LINEAR_ACT_GELU_TANH: f(std::integral_constant<int, E4B_LINEAR_ACT_GELU_TANH>()); break;
        default: f(std::integral_constant<int, E4B_LINEAR_ACT_NONE>());
    }
}

// One product over rows grouped by expert, on the tensor cores.
struct LinearGemm {
    int E, K, N, n_tiles;
    const int* tile_prefix;     // [E+1] and [m-tiles]: the m-tile schedule; null: one expert, P rows
    const int4* sched;
    int64_t P;
    const uint8_t* packed;      // 4-bit stacks: [b_rows_total, row bytes]
    const float* absmax;
    const uint8_t* mx_scales;
    int64_t mx_stride;
    const __nv_bfloat16* bf16_b;
    int64_t b_rows_total;
    int b_rows_per_expert, b_blocks_per_row;
    const void* a;              // bf16 [P, K]
    __nv_bfloat16* out;         // [P, N] or null
    __nv_bfloat16* saved;       // [P, N] or null: act'
    const __nv_bfloat16* residual;   // [P, N] or null
    const float* bias;          // [E, N] or null
    int act;
    int splits;                 // > 1: fp32 partial sums over parts of K, added by the finishing kernel
    float* partial;             // [splits, P, N]
    uint32_t* status;
};

// forward: D = A W^T (W [N, K] as stored); else D = A W (W [K, N] as stored), no epilogue.
// codebook: 0 NF4, 1 FP4, 2 MXFP4, 3 bf16.
cudaError_t launch_linear_gemm(bool forward, int codebook, const LinearGemm& p, int max_m_tiles, cudaStream_t st);
// Parts of K for a dense product that has too few tiles to fill the GPU (1: no split).
int linear_splits(int64_t P, int N, int K);
int linear_tile_rows();

// The m-tile schedule of rows grouped by offsets [E+1] (clamped to ascending values in
// [0, P]; null: one expert, P rows).
cudaError_t launch_linear_schedule(const int32_t* offsets, int E, int64_t P, int tile_rows, int* tile_prefix, int4* sched,
                                   cudaStream_t st);

// The weight-streaming form for few rows.
struct LinearStream {
    int E, K, N;
    int P;
    const int32_t* offsets;     // [E+1] or null
    const uint8_t* packed;
    const float* absmax;
    const uint8_t* mx_scales;
    int64_t mx_stride;
    const __nv_bfloat16* x;     // [P, K]
    __nv_bfloat16* out;         // [P, N] or null
    __nv_bfloat16* saved;
    const __nv_bfloat16* residual;
    const float* bias;
    int act;
};
constexpr int kStreamGroupedRows = 1024;
// Whether a forward of P rows streams its weights: dense, up to 8 rows, or 16 that fit in shared
// memory; grouped, up to 4 rows per expert on average (both sides' times are at its definition).
bool linear_streams(bool grouped, int E, int64_t P, int K);
cudaError_t launch_linear_stream(int codebook, const LinearStream& p, cudaStream_t st);

}  // namespace e4b
