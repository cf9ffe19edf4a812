// e4b_linear_*: argument checks, workspace and launches of the quantized linear, and the
// elementwise part of its backward:
//   dz = grad_y * act'(z),  grad_bias_e = sum over expert e's rows of dz
// (HBM-bound: grad_y and act' are read once, dz written once in bf16; the bias sums take dz before
// that rounding.  16384 x 14336: 228 us, 6.2 TB/s).
//
// dz is rounded to bf16 because it is the tensor cores' operand next to bf16 weights.  It moves an
// element of grad_x by at most 2^-8 sum |dz| |W|: over 16384 x 14336 by 4096 its error in the 2-norm
// is 0.0023, with dz unrounded 0.0017 (the rounding of grad_x alone); against the product of the
// rounded dz the kernel is off by 0.0003.  dz as a sum of two bf16 would be exact at twice the
// product's time.
#include "linear.h"
#include "rowops.cuh"

namespace e4b {
namespace {

// A block takes 256 columns (32 threads of 8) and one part of one expert's rows, 8 rows at a
// time; the 8 row lanes are added in order at the end.  sums: [parts][E][N], or the gradient
// itself when there is one part.
template <bool ACT>
__global__ void __launch_bounds__(256) linear_dz_kernel(const __nv_bfloat16* __restrict__ gy,
                                                        const __nv_bfloat16* __restrict__ saved,
                                                        const int32_t* __restrict__ offsets, int64_t P, int N,
                                                        __nv_bfloat16* __restrict__ dz, float* __restrict__ sums) {
    __shared__ float s_sum[8][256];
    __shared__ int s_top[8];
    const int tid = threadIdx.x, x = tid & 31, y = tid >> 5, e = blockIdx.z;
    pdl_release();
    pdl_wait();
    int64_t begin = 0, end = P;
    if (offsets) {   // the running maximum of the offsets inside [0, P], as in the schedule
        int v = tid <= e ? (int)min(max((int64_t)__ldcg(offsets + tid), (int64_t)0), P) : 0;
        v = __reduce_max_sync(0xffffffffu, v);
        if (x == 0) s_top[y] = v;
        __syncthreads();
        int top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, s_top[i]);
        begin = top;
        end = max(begin, min(max((int64_t)__ldcg(offsets + e + 1), (int64_t)0), P));
    }
    const int64_t per = (end - begin + gridDim.y - 1) / gridDim.y;
    const int64_t r0 = begin + blockIdx.y * per, r1 = min(end, r0 + per);
    const int col = blockIdx.x * 256 + 8 * x;
    const bool in = col < N;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
#pragma unroll 4
        for (int64_t r = r0 + y; r < r1; r += 8) {
            const int64_t at = (r * N + col) / 8;
            float v[8];
            unpack<__nv_bfloat16, 8>(ld_once<uint4>(gy, at), v);
            if (ACT) {
                float d[8];
                unpack<__nv_bfloat16, 8>(ld_once<uint4>(saved, at), d);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= d[j];
                if (dz) reinterpret_cast<uint4*>(dz)[at] = pack<__nv_bfloat16, 8>(v);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += v[j];
        }
    }
    if (!sums) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) s_sum[y][8 * x + j] = acc[j];
    __syncthreads();
    const int c = blockIdx.x * 256 + tid;
    if (c >= N) return;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += s_sum[i][tid];
    sums[((int64_t)blockIdx.y * gridDim.z + e) * N + c] = s;
}

__global__ void __launch_bounds__(256) linear_bias_sum_kernel(const float* __restrict__ sums, int parts, int64_t n,
                                                              float* __restrict__ out) {
    pdl_release();
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.0f;
#pragma unroll 8
    for (int q = 0; q < parts; ++q) s += __ldcg(sums + q * n + i);
    out[i] = s;
}

// Parts of each expert's rows: about four blocks per SM, at least 64 rows each on average.
int dz_parts(int E, int64_t P, int N) {
    const int64_t cols = (N + 255) / 256;
    const int64_t want = (4LL * num_sms() + cols * E - 1) / (cols * E);
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, (P / E + 63) / 64));
}

struct Layout {
    size_t tile_prefix, sched, dz, saved, sums, wbf16, partial, total;
};
size_t align_up(size_t v) { return (v + 255) & ~size_t(255); }

int max_tiles(const e4b_linear_desc* d, int64_t P) {
    const int64_t full = (P + linear_tile_rows() - 1) / linear_tile_rows();
    return (int)(d->E == 1 ? full : full + std::min<int64_t>(d->E, P));
}
bool eight_bit(const e4b_linear_desc* d) {
    return d->codebook == E4B_CODEBOOK_INT8 || d->codebook == E4B_CODEBOOK_FP8;
}
int gemm_format(const e4b_linear_desc* d) { return d->codebook <= E4B_CODEBOOK_MXFP4 ? d->codebook : 3; }

// Bytes of the partial sums of P rows by N outputs, or (any: a workspace's size) the most that P or
// fewer rows need: the parts are fewer for more tiles, so each number of m-tiles has its own most.
size_t partial_bytes(int64_t P, int N, int K, bool any) {
    size_t most = 0;
    for (int64_t rows = any ? std::min<int64_t>(P, linear_tile_rows()) : P;;
         rows = std::min<int64_t>(P, rows + linear_tile_rows())) {
        const int splits = linear_splits(rows, N, K);
        if (splits <= 1) break;
        most = std::max(most, (size_t)splits * rows * N * 4);
        if (rows == P) break;
    }
    return most;
}

// What a call of P rows takes of the workspace.  backward: the forward alone needs no dz, derivative
// or bias sums.  any: room for every call of up to P rows.
Layout layout(const e4b_linear_desc* d, int64_t P, bool backward, bool any = false) {
    Layout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off = align_up(off + bytes); return o; };
    L.tile_prefix = take((size_t)(d->E + 1) * 4);
    L.sched = take((size_t)max_tiles(d, P) * 16);
    const bool act = backward && d->activation != E4B_LINEAR_ACT_NONE;
    L.dz = take(act ? (size_t)P * d->n_out * 2 : 0);
    L.saved = take(act ? (size_t)P * d->n_out * 2 : 0);
    L.sums = take(backward ? (size_t)dz_parts(d->E, P, d->n_out) * d->E * d->n_out * 4 : 0);
    L.wbf16 = take(eight_bit(d) ? (size_t)d->E * d->n_in * d->n_out * 2 : 0);
    if (d->E == 1)
        L.partial = take(std::max(partial_bytes(P, d->n_out, d->n_in, any),
                                  backward ? partial_bytes(P, d->n_in, d->n_out, any) : 0));
    L.total = off;
    return L;
}

e4b_status check_desc(const e4b_linear_desc* d) {
    if (!d) return E4B_ERR_INVALID_ARG;
    if (d->codebook < E4B_CODEBOOK_NF4 || d->codebook > E4B_CODEBOOK_BF16) return E4B_ERR_INVALID_ARG;
    if (d->blocksize != (d->codebook == E4B_CODEBOOK_MXFP4 ? 32 : 64)) return E4B_ERR_BLOCKSIZE;
    if (d->E < 1 || d->E > 256 || d->n_in < 1 || d->n_out < 1) return E4B_ERR_INVALID_ARG;
    if (d->n_in % 64 || d->n_out % 64) return E4B_ERR_BLOCKSIZE;
    if ((int64_t)d->E * std::max(d->n_in, d->n_out) > (int64_t)INT32_MAX) return E4B_ERR_UNSUPPORTED;
    if (d->activation < E4B_LINEAR_ACT_NONE || d->activation > E4B_LINEAR_ACT_GELU_TANH) return E4B_ERR_INVALID_ARG;
    return E4B_OK;
}

e4b_status check_weights(const e4b_linear_desc* d, const e4b_linear_weights* w) {
    if (!w || !w->weight) return E4B_ERR_INVALID_ARG;
    if (d->codebook == E4B_CODEBOOK_MXFP4 ? !w->scales : d->codebook == E4B_CODEBOOK_BF16 ? false : !w->absmax)
        return E4B_ERR_INVALID_ARG;
    return E4B_OK;
}

const __nv_bfloat16* bf(const void* p) { return static_cast<const __nv_bfloat16*>(p); }

// The weight in the GEMM's format: bf16 storage as it is, 8-bit storage dequantized into the
// workspace (the whole stack: its one rounding is the format's own).
cudaError_t bf16_weights(const e4b_linear_desc* d, const e4b_linear_weights* w, uint8_t* ws, const Layout& L,
                         cudaStream_t st, const __nv_bfloat16** out) {
    *out = nullptr;
    if (d->codebook == E4B_CODEBOOK_BF16) {
        *out = bf(w->weight);
    } else if (eight_bit(d)) {
        *out = bf(ws + L.wbf16);
        return launch_dequantize8(static_cast<const uint8_t*>(w->weight), w->absmax, (int64_t)d->E * d->n_in * d->n_out,
                                  d->codebook, 1, ws + L.wbf16, st);
    }
    return cudaSuccess;
}

cudaError_t schedule(const e4b_linear_desc* d, const int32_t* offsets, int64_t P, uint8_t* ws, const Layout& L,
                     cudaStream_t st) {
    if (!offsets) return cudaSuccess;
    return launch_linear_schedule(offsets, d->E, P, linear_tile_rows(), reinterpret_cast<int*>(ws + L.tile_prefix),
                                  reinterpret_cast<int4*>(ws + L.sched), st);
}

LinearGemm gemm_args(const e4b_linear_desc* d, const e4b_linear_weights* w, const int32_t* offsets, int64_t P,
                     uint8_t* ws, const Layout& L, const __nv_bfloat16* wbf16) {
    LinearGemm g{};
    g.E = d->E;
    if (offsets) {
        g.tile_prefix = reinterpret_cast<const int*>(ws + L.tile_prefix);
        g.sched = reinterpret_cast<const int4*>(ws + L.sched);
    }
    g.P = P;
    g.packed = static_cast<const uint8_t*>(w->weight);
    g.absmax = w->absmax;
    g.mx_scales = w->scales;
    g.mx_stride = mxfp4_scale_stride(d->n_in);
    g.bf16_b = wbf16;
    g.b_rows_total = (int64_t)d->E * d->n_out;
    g.b_rows_per_expert = d->n_out;
    g.b_blocks_per_row = d->n_in / 64;
    g.splits = 1;
    g.status = device_status_ptr();
    return g;
}

// y (or null) and saved (or null) from x; scheduled: the m-tile schedule is in the workspace.
cudaError_t run_forward(const e4b_linear_desc* d, const e4b_linear_weights* w, const void* x, int64_t P,
                        const int32_t* offsets, const void* residual, void* y, void* saved, uint8_t* ws, const Layout& L,
                        const __nv_bfloat16* wbf16, bool scheduled, cudaStream_t st) {
    const int fmt = gemm_format(d);
    if (linear_streams(offsets != nullptr, d->E, P, d->n_in)) {
        LinearStream s{};
        s.E = d->E;
        s.K = d->n_in;
        s.N = d->n_out;
        s.P = (int)P;
        s.offsets = offsets;
        s.packed = wbf16 ? reinterpret_cast<const uint8_t*>(wbf16) : static_cast<const uint8_t*>(w->weight);
        s.absmax = w->absmax;
        s.mx_scales = w->scales;
        s.mx_stride = mxfp4_scale_stride(d->n_in);
        s.x = bf(x);
        s.out = static_cast<__nv_bfloat16*>(y);
        s.saved = static_cast<__nv_bfloat16*>(saved);
        s.residual = bf(residual);
        s.bias = w->bias;
        s.act = d->activation;
        return launch_linear_stream(fmt, s, st);
    }
    cudaError_t err = scheduled ? cudaSuccess : schedule(d, offsets, P, ws, L, st);
    if (err != cudaSuccess) return err;
    LinearGemm g = gemm_args(d, w, offsets, P, ws, L, wbf16);
    g.K = d->n_in;
    g.N = d->n_out;
    g.n_tiles = (d->n_out + 255) / 256;
    g.a = x;
    g.out = static_cast<__nv_bfloat16*>(y);
    g.saved = static_cast<__nv_bfloat16*>(saved);
    g.residual = bf(residual);
    g.bias = w->bias;
    g.act = d->activation;
    if (!offsets) {
        g.splits = linear_splits(P, g.N, g.K);
        g.partial = reinterpret_cast<float*>(ws + L.partial);
    }
    return launch_linear_gemm(true, fmt, g, max_tiles(d, P), st);
}

}  // namespace
}  // namespace e4b

using namespace e4b;

#define E4B_TRY(expr)                                  \
    do {                                               \
        if ((expr) != cudaSuccess) return E4B_ERR_CUDA; \
    } while (0)

extern "C" {

size_t e4b_linear_workspace_size(const e4b_linear_desc* d, int64_t P) {
    if (check_desc(d) != E4B_OK || P < 0 || P > (int64_t)INT32_MAX - 256) return 0;
    return layout(d, P, true, true).total;
}

size_t e4b_linear_forward_workspace_size(const e4b_linear_desc* d, int64_t P) {
    if (check_desc(d) != E4B_OK || P < 0 || P > (int64_t)INT32_MAX - 256) return 0;
    return layout(d, P, false, true).total;
}

e4b_status e4b_linear_forward(const e4b_linear_desc* d, const e4b_linear_weights* w, const void* x, int64_t P,
                              const int32_t* offsets, const void* residual, void* y, void* saved_d, void* workspace,
                              size_t ws_bytes, void* stream) {
    NvtxScope nvtx_scope("e4b_linear_forward");
    e4b_status s = check_desc(d);
    if (s != E4B_OK) return s;
    if ((s = check_weights(d, w)) != E4B_OK) return s;
    if (P < 0 || P > (int64_t)INT32_MAX - 256) return E4B_ERR_INVALID_ARG;
    if (P == 0) return E4B_OK;
    if (!x || !y || (d->E > 1 && !offsets)) return E4B_ERR_INVALID_ARG;
    if (off_boundary(16, {x, residual, y, saved_d, w->weight, w->absmax, w->scales, w->bias}) || off_boundary(4, {offsets}))
        return E4B_ERR_INVALID_ARG;
    const Layout L = layout(d, P, false);
    if (!workspace || ws_bytes < L.total) return E4B_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (off_boundary(16, {ws})) return E4B_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const __nv_bfloat16* wb;
    E4B_TRY(bf16_weights(d, w, ws, L, st, &wb));
    E4B_TRY(run_forward(d, w, x, P, offsets, residual, y, saved_d, ws, L, wb, false, st));
    return E4B_OK;
}

e4b_status e4b_linear_backward(const e4b_linear_desc* d, const e4b_linear_weights* w, const void* x, int64_t P,
                               const int32_t* offsets, const void* grad_y, const void* saved_d, void* grad_x,
                               float* grad_bias, void* workspace, size_t ws_bytes, void* stream) {
    NvtxScope nvtx_scope("e4b_linear_backward");
    e4b_status s = check_desc(d);
    if (s != E4B_OK) return s;
    if ((s = check_weights(d, w)) != E4B_OK) return s;
    if (P < 0 || P > (int64_t)INT32_MAX - 256) return E4B_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t nb = (int64_t)d->E * d->n_out;
    if (P == 0) {   // no rows: the bias gradient is zero
        if (grad_bias) E4B_TRY(cudaMemsetAsync(grad_bias, 0, nb * 4, st));
        return E4B_OK;
    }
    const bool act = d->activation != E4B_LINEAR_ACT_NONE;
    if (!grad_y || (!grad_x && !grad_bias) || (d->E > 1 && !offsets) || (act && !saved_d && !x))
        return E4B_ERR_INVALID_ARG;
    if (off_boundary(16, {x, grad_y, saved_d, grad_x, w->weight, w->absmax, w->scales, w->bias}) ||
        off_boundary(4, {offsets, grad_bias}))
        return E4B_ERR_INVALID_ARG;
    const Layout L = layout(d, P, true);
    if (!workspace || ws_bytes < L.total) return E4B_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (off_boundary(16, {ws})) return E4B_ERR_INVALID_ARG;
    const bool recompute = act && !saved_d;
    const __nv_bfloat16* wb = nullptr;
    if (grad_x || recompute) E4B_TRY(bf16_weights(d, w, ws, L, st, &wb));
    if (grad_x || recompute) E4B_TRY(schedule(d, offsets, P, ws, L, st));
    if (recompute) {
        E4B_TRY(run_forward(d, w, x, P, offsets, nullptr, nullptr, ws + L.saved, ws, L, wb, true, st));
        saved_d = ws + L.saved;
    }
    const void* dz = grad_y;
    if (act || grad_bias) {
        const int parts = dz_parts(d->E, P, d->n_out);
        float* sums = !grad_bias ? nullptr : parts == 1 ? grad_bias : reinterpret_cast<float*>(ws + L.sums);
        const dim3 grid((d->n_out + 255) / 256, parts, d->E);
        __nv_bfloat16* out = act && grad_x ? reinterpret_cast<__nv_bfloat16*>(ws + L.dz) : nullptr;
        if (act)
            E4B_TRY(launch_pdl(linear_dz_kernel<true>, grid, dim3(256), 0, st, bf(grad_y), bf(saved_d), offsets, P,
                               d->n_out, out, sums));
        else
            E4B_TRY(launch_pdl(linear_dz_kernel<false>, grid, dim3(256), 0, st, bf(grad_y), bf(nullptr), offsets, P,
                               d->n_out, out, sums));
        if (grad_bias && parts > 1)
            E4B_TRY(launch_pdl(linear_bias_sum_kernel, dim3((unsigned)((nb + 255) / 256)), dim3(256), 0, st,
                               (const float*)sums, parts, nb, grad_bias));
        if (act) dz = ws + L.dz;
    }
    if (!grad_x) return E4B_OK;
    LinearGemm g = gemm_args(d, w, offsets, P, ws, L, wb);
    g.K = d->n_out;
    g.N = d->n_in;
    g.n_tiles = (d->n_in + 255) / 256;
    g.a = dz;
    g.out = static_cast<__nv_bfloat16*>(grad_x);
    if (!offsets) {
        g.splits = linear_splits(P, g.N, g.K);
        g.partial = reinterpret_cast<float*>(ws + L.partial);
    }
    E4B_TRY(launch_linear_gemm(false, gemm_format(d), g, max_tiles(d, P), st));
    return E4B_OK;
}

}  // extern "C"
