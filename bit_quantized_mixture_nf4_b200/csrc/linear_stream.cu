// The quantized linear for few rows (decode, short verification batches): a stream of the
// weights, bound by HBM at a few rows, so every weight byte is read once per group of rows.
//
//   z = X_e W_e^T + b_e,  y = residual + act(z),  saved = act'(z)
//
// A block of 8 warps takes 16 outputs of one expert; its warps take every eighth step of
// 256 inputs and are added in warp order at the end (the same bits every time).  Weights go
// from global memory straight into registers, two steps ahead.  mma.sync m16n8k16 with the
// 16 weight rows as A and up to 8 rows of X as B: K is permuted alike on both operands so
// that a lane owns one whole 64-element block of a row (one scale, 32 contiguous bytes) and
// the matching 128 bytes of X.  (At 8 columns tcgen05 has nothing to win: the tensor work
// is a few percent of the time.)
//
// A weight is bf16_rn(code * absmax), the value the tensor-core path uses: a table in shared
// memory turns a byte into its two fp32 code values (one copy of the 256 entries for each of
// the 16 lanes of a half-warp, so the 8-byte loads have no bank conflicts), then two fp32
// products and one conversion make the pair.
#include <mutex>

#include "linear.h"
#include "rowops.cuh"

namespace e4b {
namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int TOK_STRIDE = 20;   // floats per row of X in the warps' sums: 16 outputs, no bank conflicts
constexpr int LUT_BYTES = 256 * 16 * 8;

struct Slot { int e, row0, rows; };

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's 64 weights of its two rows at one step.
template <int CB> struct Weights {
    uint4 c[2][CB == 3 ? 8 : 2];
    float s[2];   // absmax; MXFP4: the two scale bytes
};

// Two codes of byte b as a bf16 pair (high nibble first), scaled.  lane16 = 16 * (lane & 15).
__device__ __forceinline__ uint32_t pair(const uint8_t* lut, uint32_t off, float s) {
    const float2 v = *reinterpret_cast<const float2*>(lut + off);
    return pack_bf16x2(__fmul_rn(v.x, s), __fmul_rn(v.y, s));
}
__device__ __forceinline__ void decode8(const uint8_t* lut, uint32_t w, uint32_t lane16, float s, uint32_t (&o)[4]) {
    const uint32_t d01 = prmt(w, lane16, 0x1404u), d23 = prmt(w, lane16, 0x3424u);   // [lane16, byte] pairs
    o[0] = pair(lut, (d01 >> 1) & 0x7fffu, s);
    o[1] = pair(lut, d01 >> 17, s);
    o[2] = pair(lut, (d23 >> 1) & 0x7fffu, s);
    o[3] = pair(lut, d23 >> 17, s);
}

template <int CB, int NT>
__global__ void __launch_bounds__(THREADS, 2) linear_stream_kernel(const LinearStream p) {
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ Slot slots[kStreamRows];
    __shared__ int s_nslots;
    __shared__ float cv[16];
    uint8_t* lut = dsm;
    float* red = reinterpret_cast<float*>(dsm + (CB == 3 ? 0 : LUT_BYTES));   // [warp][8 NT][TOK_STRIDE]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;

    if (CB != 3) {
        if (tid < 16) cv[tid] = c_code[CB < 3 ? CB : 0][tid];
        __syncthreads();
        for (int i = tid; i < 256 * 8; i += THREADS) {
            const int v = i >> 3;
            reinterpret_cast<float4*>(lut)[i] = make_float4(cv[v >> 4], cv[v & 15], cv[v >> 4], cv[v & 15]);
        }
    }
    pdl_release();
    pdl_wait();
    // the experts that have rows (offsets as their running maximum inside [0, P])
    if (!p.offsets) {
        if (tid == 0) {
            slots[0] = Slot{0, 0, p.P};
            s_nslots = 1;
        }
    } else if (warp == 0) {
        int top = min(max(__ldcg(p.offsets), 0), p.P), n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int end = e < p.E ? min(max(__ldcg(p.offsets + e + 1), 0), p.P) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end = max(end, u);
            }
            end = max(end, top);
            int begin = __shfl_up_sync(0xffffffffu, end, 1);
            if (lane == 0) begin = top;
            const bool live = e < p.E && end > begin;
            const uint32_t m = __ballot_sync(0xffffffffu, live);
            if (live) slots[n + __popc(m & ((1u << lane) - 1u))] = Slot{e, begin, end - begin};
            n += __popc(m);
            top = __shfl_sync(0xffffffffu, end, 31);
        }
        if (lane == 0) s_nslots = n;
    }
    __syncthreads();

    const int tiles = p.N / 16, units = s_nslots * tiles, KB = p.K / 64, steps = (KB + 3) / 4;
    const uint32_t lane16 = 16u * (lane & 15);
    // unit u: slot u / tiles, outputs 16 (u % tiles) ...; this warp's steps: warp, warp + 8, ...
    auto load = [&](int u, int st, Weights<CB>& w) {
        const int kb = 4 * st + c, sl = u / tiles;
        const bool in = u < units && kb < KB;
        const int64_t r0 = in ? (int64_t)slots[sl].e * p.N + (u - sl * tiles) * 16 + g : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = r0 + 8 * h;
            constexpr int NV = CB == 3 ? 8 : 2;
            const uint4* src = reinterpret_cast<const uint4*>(p.packed + (CB == 3 ? (row * p.K + kb * 64) * 2
                                                                                  : (row * p.K >> 1) + kb * 32));
#pragma unroll
            for (int i = 0; i < NV; ++i) w.c[h][i] = in ? __ldcs(src + i) : make_uint4(0u, 0u, 0u, 0u);
            w.s[h] = 0.0f;
            if (CB == 2)
                w.s[h] = __uint_as_float(
                    in ? (uint32_t)*reinterpret_cast<const uint16_t*>(p.mx_scales + row * p.mx_stride + 2 * kb) : 0u);
            else if (CB < 2 && in)
                w.s[h] = p.absmax[row * KB + kb];
        }
    };
    float acc[NT][2][4];
    auto compute = [&](int u, int st, const Weights<CB>& w) {
        const int kb = 4 * st + c, sl = u / tiles;
        const Slot slot = slots[sl];
        const uint4* xs[NT];
        bool in[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int n = 8 * nt + g;
            in[nt] = n < slot.rows && kb < KB;
            xs[nt] = reinterpret_cast<const uint4*>(p.x + (int64_t)(slot.row0 + (in[nt] ? n : 0)) * p.K + kb * 64);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t lo[4], hi[4];
            if (CB == 3) {
                const uint4 a = w.c[0][CB == 3 ? j : 0], b = w.c[1][CB == 3 ? j : 0];
                lo[0] = a.x; lo[1] = a.y; lo[2] = a.z; lo[3] = a.w;
                hi[0] = b.x; hi[1] = b.y; hi[2] = b.z; hi[3] = b.w;
            } else {
                float s0 = w.s[0], s1 = w.s[1];
                if (CB == 2) {
                    s0 = mx_scale((__float_as_uint(s0) >> (j < 4 ? 0 : 8)) & 0xFFu);
                    s1 = mx_scale((__float_as_uint(s1) >> (j < 4 ? 0 : 8)) & 0xFFu);
                }
                const uint4 a = w.c[0][j >> 2], b = w.c[1][j >> 2];
                const uint32_t wa = (j & 3) == 0 ? a.x : (j & 3) == 1 ? a.y : (j & 3) == 2 ? a.z : a.w;
                const uint32_t wb = (j & 3) == 0 ? b.x : (j & 3) == 1 ? b.y : (j & 3) == 2 ? b.z : b.w;
                decode8(lut, wa, lane16, s0, lo);
                decode8(lut, wb, lane16, s1, hi);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (NT > 1 && 8 * nt >= slot.rows) continue;   // the same for the whole block
                const uint4 xv = in[nt] ? xs[nt][j] : make_uint4(0u, 0u, 0u, 0u);
                mma_16816(acc[nt][0], lo[0], hi[0], lo[1], hi[1], xv.x, xv.y);
                mma_16816(acc[nt][1], lo[2], hi[2], lo[3], hi[3], xv.z, xv.w);
            }
        }
    };

    constexpr int D = CB == 3 ? 1 : 2;   // steps in flight ahead of the one computed
    Weights<CB> w[D];
    const int first = warp < steps ? blockIdx.x : units;   // a warp without steps only joins the sums
    int lu = first, ls = warp;                             // load cursor
    auto advance = [&]() {
        ls += WARPS;
        if (ls >= steps) {
            ls = warp;
            lu += gridDim.x;
        }
    };
#pragma unroll
    for (int i = 0; i < D; ++i) {
        load(lu, ls, w[i]);
        advance();
    }
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][0][i] = acc[nt][1][i] = 0.0f;
        for (int st = warp; st < steps; st += WARPS) {
            const Weights<CB> cur = w[0];
#pragma unroll
            for (int i = 0; i + 1 < D; ++i) w[i] = w[i + 1];
            load(lu, ls, w[D - 1]);
            advance();
            compute(u, st, cur);
        }
        // D fragment: rows g, g + 8 (outputs), columns 2c, 2c + 1 (rows of X)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float* r = red + (warp * 8 * NT + 8 * nt + 2 * c) * TOK_STRIDE + g;
            r[0] = acc[nt][0][0] + acc[nt][1][0];
            r[TOK_STRIDE] = acc[nt][0][1] + acc[nt][1][1];
            r[8] = acc[nt][0][2] + acc[nt][1][2];
            r[TOK_STRIDE + 8] = acc[nt][0][3] + acc[nt][1][3];
        }
        __syncthreads();
        const int sl = u / tiles;
        const Slot slot = slots[sl];
        const int n0 = (u - sl * tiles) * 16;
        for (int i = tid; i < 16 * slot.rows; i += THREADS) {
            const int r = i & 15, t = i >> 4;
            float z = 0.0f;
#pragma unroll
            for (int q = 0; q < WARPS; ++q) z += red[(q * 8 * NT + t) * TOK_STRIDE + r];
            if (p.bias) z += p.bias[(int64_t)slot.e * p.N + n0 + r];
            float y, d;
            with_act(p.act, [&](auto kind) { linear_act<decltype(kind)::value>(z, y, d); });
            const int64_t at = (int64_t)(slot.row0 + t) * p.N + n0 + r;
            if (p.residual) y += __bfloat162float(p.residual[at]);
            if (p.out) p.out[at] = __float2bfloat16_rn(y);
            if (p.saved) p.saved[at] = __float2bfloat16_rn(d);
        }
        __syncthreads();
    }
}

template <int CB, int NT>
cudaError_t launch_nt(const LinearStream& p, cudaStream_t st) {
    constexpr int smem = (CB == 3 ? 0 : LUT_BYTES) + WARPS * 8 * NT * TOK_STRIDE * 4;
    auto kern = linear_stream_kernel<CB, NT>;
    {
        static std::mutex mu;
        static bool set[64] = {false};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        if (!set[dev]) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            set[dev] = true;
        }
    }
    const int units = std::min(p.E, p.P) * (p.N / 16);
    return launch_pdl(kern, dim3(std::min(units, 2 * num_sms())), dim3(THREADS), smem, st, p);
}

template <int CB>
cudaError_t launch_cb(const LinearStream& p, cudaStream_t st) {
    if (p.P <= 8) return launch_nt<CB, 1>(p, st);
    if (p.P <= 16) return launch_nt<CB, 2>(p, st);
    return launch_nt<CB, 4>(p, st);
}

}  // namespace

bool linear_streams(int codebook, int64_t P) {
    (void)codebook;
    return P <= kStreamRows;
}

cudaError_t launch_linear_stream(int codebook, const LinearStream& p, cudaStream_t st) {
    switch (codebook) {
        case 0: return launch_cb<0>(p, st);
        case 1: return launch_cb<1>(p, st);
        case 2: return launch_cb<2>(p, st);
        default: return launch_cb<3>(p, st);
    }
}

}  // namespace e4b
