// Shared pieces of the block norm kernels (block_norm.cu, block_ring.cu, block_ring_backward.cu).
#pragma once
#include <type_traits>

#include "../../include/e4b.h"
#include "rowops.cuh"

namespace e4b {

constexpr int kMaxRow = 8192;

struct BlockArgs {
    const void *f, *rows, *h, *gate;
    const int32_t* inv_perm;
    const float *topk_w, *post_w, *pre_w;
    void *f_out, *o, *n;
    const void *grad_o, *grad_n;
    void *grad_h, *grad_f, *grad_gate;
    float* partials;                   // [parts][3][H]: post_w, pre_w, channel gate
    int want_post, want_pre, want_cgate;
    int64_t T;
    int H, nvec, k, gate_kind, gate_sigmoid;
    float eps, offset, scale;
    uint32_t* status;                  // device status word (the ring kernels' bounded waits)
};

// Sums N <= 3 values over a row's tx threads; all of them get the sums.  The first step of a
// warp's tree halves the values along with the lanes (each half goes on with other values), so
// 2 values cost the 5 shuffles of one and 3 cost 6.  tx = 32: one warp; else the block's warps
// leave their sums in s_red, warp i adds those of value i, and every thread reads the totals
// behind a second barrier.  (Every warp adding all of them instead, by 16-byte reads, keeps the
// shared-memory pipe busier and was slower.)
// Two reductions through the same buffer need no barrier between them.
template <int N>
struct __align__(16) RowSums {
    float part[N][32];
    float total[4];
};

template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tx, RowSums<N>& s_red) {
    const int lane = threadIdx.x & 31;
    const bool b4 = lane & 16, b3 = lane & 8;
    float a;
    if (N == 1) {
        a = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
        a += __shfl_xor_sync(0xffffffffu, a, 8);
    } else {
        a = b4 ? v[N > 1] : v[0];
        a += __shfl_xor_sync(0xffffffffu, b4 ? v[0] : v[N > 1], 16);
        if (N == 2) {
            a += __shfl_xor_sync(0xffffffffu, a, 8);
        } else {
            float c = b4 ? 0.0f : v[N - 1];
            c += __shfl_xor_sync(0xffffffffu, b4 ? v[N - 1] : 0.0f, 16);
            const float send = b3 ? a : c;
            a = (b3 ? c : a) + __shfl_xor_sync(0xffffffffu, send, 8);
        }
    }
    a += __shfl_xor_sync(0xffffffffu, a, 4);
    a += __shfl_xor_sync(0xffffffffu, a, 2);
    a += __shfl_xor_sync(0xffffffffu, a, 1);
    // value 0 is in lane 0, value 1 in lane 16, value 2 in lane 8
    if (tx == 32) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, a, i == 0 ? 0 : i == 1 ? 16 : 8);
        return;
    }
    const int warp = threadIdx.x >> 5, nw = tx >> 5;
    const int mine = lane == 0 ? 0 : lane == 16 ? 1 : lane == 8 ? 2 : N;
    if (mine < N) s_red.part[mine][warp] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (warp == i % nw) {
            float x = lane < nw ? s_red.part[i][lane] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == 0) s_red.total[i] = x;
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = s_red.total[i];
}

// The logistic function g(x) and its slope g (1 - g): the smaller of g and 1 - g is e / (1 + e),
// e = exp(-|x|), so that no difference costs relative accuracy, over the whole range.  The quotient's
// divisor lies in [1, 2], where the fast one is off by 2 units in the last place; with expf's 2 and
// two roundings that is 5 units.  FAST: by the fast exponential (2 + 1.17 |x| units, a relative 1e-5
// at |x| = 88), for element gates in bf16, whose half step of 2^-8 covers it.
template <bool FAST>
__device__ __forceinline__ void logistic(float x, float& g, float& slope) {
    const float e = FAST ? __expf(-fabsf(x)) : expf(-fabsf(x));
    const float q = __fdividef(1.0f, 1.0f + e), s = e * q;
    g = x < 0.0f ? s : q;
    slope = s * q;
}
template <bool FAST>
__device__ __forceinline__ float sigmoid(float x) {
    float g, slope;
    logistic<FAST>(x, g, slope);
    return g;
}
template <typename E> constexpr bool kFastGate = !std::is_same<E, float>::value;   // of an element gate

template <int V, int NV>
__device__ __forceinline__ void load_channels(const float* w, float add, int tx, int x, int nvec, float (&out)[NV][V]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = i * tx + x;
            out[i][j] = w && v < nvec ? __ldcg(w + v * V + j) + add : 1.0f;
        }
}


// The shared-memory ring forms (block_ring*.cu): runs of rows whose tensors start on 16-byte
// boundaries.  False where the rows do not fit or are too few to fill the rings.
bool block_ring_forward(e4b_dtype dt, bool dense, const BlockArgs& a, cudaStream_t st, cudaError_t* err);
bool block_ring_backward(e4b_dtype dt, bool branch, const BlockArgs& a, int* parts, cudaStream_t st, cudaError_t* err);
int64_t block_ring_parts(int H, int64_t T);   // partials that the ring backward may leave

}  // namespace e4b
