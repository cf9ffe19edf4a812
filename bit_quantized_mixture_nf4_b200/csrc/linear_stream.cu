// The quantized linear for few rows (decode, short verification batches): a stream of the
// weights, so a weight byte is read once per 16 rows of X (once per 8 of an expert's in a grouped call).
//
//   z = X_e W_e^T + b_e,  y = residual + act(z),  saved = act'(z)
//
// A unit is 16 outputs of one expert for up to 16 of its rows.  One block of 16 warps per SM
// takes every 148th unit; the steps (256 inputs) of all its units form one list that its warps
// split evenly, so a warp may end one unit and begin another: each leaves one partial sum per
// unit in shared memory, and they are added in warp order behind one barrier (the same bits
// every time).  Splitting every unit's K over the warps instead cost two barriers a unit and
// left a third of the last round empty (4096 by 14336 in bf16, 1 row: 49 us before this list, X
// in shared memory and the packed decoding, 23 with them).  Weights go from global
// memory straight into registers, two steps ahead; the rows of X of a dense product wait in
// shared memory (placed without bank conflicts for the fragments) where they fit.
//
// mma.sync m16n8k16 with the 16 weight rows as A and 8 rows of X as B: K is permuted alike on
// both operands so that a lane owns a whole 64-element block of a weight row (one scale, 32
// contiguous bytes) and the matching 128 bytes of X.  (At 8 columns tcgen05 has nothing to
// win: the tensor work is a small part of the time.)
//
// A weight is bf16_rn(code * absmax), the value the tensor-core path uses: a table in shared
// memory turns a byte into its two fp32 code values (one copy of the 256 entries for each lane:
// no bank conflicts, and a byte permute makes the whole offset), then one packed fp32 product
// and one conversion make the pair.
//
// Measured, 4096 by 14336: bf16 23 us at 1 row (5.2 TB/s, 79% of a copy's rate), 24 at 8; NF4
// 20 us at 1 row (1.7 TB/s), 21 at 8: the shared-memory pipe is 44% busy there, mostly with the
// table.  About 5 us are fixed: 2048 by 2048 in bf16, 1.3 us at a copy's rate, takes 7.0.
#include <mutex>

#include "linear.h"
#include "rowops.cuh"

namespace e4b {
namespace {

constexpr int WARPS = 16, THREADS = 32 * WARPS;
constexpr int OUTS = 16;                 // outputs of a unit
constexpr int ROUND = 16;                // units of a block between two barriers
constexpr int SEGMENTS = ROUND / WARPS + 2;   // units that a warp's part of the list can meet
constexpr int TOK_STRIDE = 20;           // floats per row of X in a partial sum: no bank conflicts
constexpr int LUT_BYTES = 256 * 32 * 8;
constexpr int MAX_SMEM = 220 * 1024;
constexpr int MAX_SLOTS = 256 + kStreamGroupedRows / 8;

struct Slot { int e, row0, rows; };

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's 64 weights of each of its two rows at one step.
template <int CB> struct Weights {
    uint4 c[2][CB == 3 ? 8 : 2];
    float s[2];   // absmax; MXFP4: the two scale bytes
};

// Two codes of the table entry at `off` (high nibble first) as a bf16 pair, scaled.
__device__ __forceinline__ uint32_t pair(const uint8_t* lut, uint32_t off, uint64_t s2) {
    const uint64_t v = *reinterpret_cast<const uint64_t*>(lut + off);
    uint64_t w;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(w) : "l"(v), "l"(s2));
    return pack_bf16x2(__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32)));
}
// The 8 weights of a word.  lane8 = 8 * lane: byte b's entry is at 256 b + lane8.
__device__ __forceinline__ void decode8(const uint8_t* lut, uint32_t w, uint32_t lane8, uint64_t s2, uint32_t (&o)[4]) {
    o[0] = pair(lut, prmt(w, lane8, 0x5504u), s2);   // bytes [lane8, b, 0, 0]
    o[1] = pair(lut, prmt(w, lane8, 0x5514u), s2);
    o[2] = pair(lut, prmt(w, lane8, 0x5524u), s2);
    o[3] = pair(lut, prmt(w, lane8, 0x5534u), s2);
}
// First item of warp w's part of a list of n.
__device__ __forceinline__ int part(int w, int n) { return (int)((int64_t)w * n / WARPS); }
__device__ __forceinline__ uint64_t twice(float s) {
    const uint64_t u = __float_as_uint(s);
    return u << 32 | u;
}
// v = *p where `in`; else v keeps its zeros.
__device__ __forceinline__ void load_if(uint4& v, const uint4* p, bool in) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"((int)in));
}
__device__ __forceinline__ void load_if_shared(uint4& v, uint32_t at, bool in) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "r"(at), "r"((int)in));
}

// NT: groups of 8 rows of X.  XS: X in shared memory (one expert).
template <int CB, int NT, bool XS>
__global__ void __launch_bounds__(THREADS, 1) linear_stream_kernel(const LinearStream p) {
    extern __shared__ __align__(128) uint8_t dsm[];
    uint8_t* lut = dsm;
    float* red = reinterpret_cast<float*>(dsm + LUT_BYTES);   // [warp][segment][8 NT][TOK_STRIDE]
    constexpr int SEG = 8 * NT * TOK_STRIDE;
    uint8_t* xs = reinterpret_cast<uint8_t*>(red + WARPS * SEGMENTS * SEG);   // [rows][x_stride]
    __shared__ Slot slots[MAX_SLOTS];
    __shared__ int s_nslots;
    __shared__ float cv[16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;

    if (CB != 3 && tid < 16) cv[tid] = c_code[CB < 3 ? CB : 0][tid];
    pdl_release();
    pdl_wait();
    // slots: up to 8 NT rows each of the experts that have rows (offsets as their running maximum
    // inside [0, P])
    if (!p.offsets) {
        if (tid == 0) {
            slots[0] = Slot{0, 0, p.P};
            s_nslots = 1;
        }
    } else if (warp == 0) {
        constexpr int ROWS = 8 * NT;
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
            const int mine = e < p.E ? (end - begin + ROWS - 1) / ROWS : 0;
            int x = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += u;
            }
            for (int i = 0; i < mine; ++i)
                slots[n + x - mine + i] = Slot{e, begin + ROWS * i, min(ROWS, end - begin - ROWS * i)};
            n += __shfl_sync(0xffffffffu, x, 31);
            top = __shfl_sync(0xffffffffu, end, 31);
        }
        if (lane == 0) s_nslots = n;
    }
    __syncthreads();

    const int tiles = p.N / OUTS, units = s_nslots * tiles, KB = p.K / 64, steps = (KB + 3) / 4;
    const int x_stride = XS ? p.K * 2 + 64 : 0;   // the odd rows' shift keeps 8-lane phases off each other's banks
    const uint32_t lane8 = 8u * lane;
    // The load cursor: this lane's rows g, g + 8 of a unit's weights, and the step.  A lane's share
    // of a step is block 4 st + c; of bf16 weights, every fourth 16-byte piece from c on (64
    // contiguous bytes of a row per load).
    const uint8_t* wrow[2];
    const float* arow[2];
    const uint8_t* srow[2];
    int ls = 0, left = 0;   // step, steps not yet requested
    auto seek = [&](int u) {
        const int sl = XS ? 0 : u / tiles;
        const int64_t r0 = (int64_t)slots[sl].e * p.N + (u - sl * tiles) * OUTS + g;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = r0 + 8 * h;
            wrow[h] = p.packed + (CB == 3 ? row * p.K * 2 + 16 * c : (row * p.K >> 1) + 32 * c);
            if (CB == 2) srow[h] = p.mx_scales + row * p.mx_stride + 2 * c;
            else if (CB < 2) arow[h] = p.absmax + row * KB + c;
        }
    };
    auto load = [&](Weights<CB>& w) {
        const int kb = CB == 3 ? 4 * ls : 4 * ls + c;
        const bool in = left > 0 && kb < KB;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (CB == 3) {
                const uint4* src = reinterpret_cast<const uint4*>(wrow[h] + (int64_t)ls * 512);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w.c[h][CB == 3 ? i : 0] = left > 0 && kb + (i >> 1) < KB ? __ldcs(src + 4 * i) : make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            const uint4* src = reinterpret_cast<const uint4*>(wrow[h] + (int64_t)ls * 128);
#pragma unroll
            for (int i = 0; i < 2; ++i) w.c[h][i] = in ? __ldcs(src + i) : make_uint4(0u, 0u, 0u, 0u);
            w.s[h] = 0.0f;
            if (CB == 2)
                w.s[h] = __uint_as_float(in ? (uint32_t)*reinterpret_cast<const uint16_t*>(srow[h] + 8 * ls) : 0u);
            else if (in)
                w.s[h] = arow[h][4 * ls];
        }
    };
    float acc[NT][2][4];
    uint4 x[NT];   // the B operand's 16 bytes; rows outside the slot stay zero
    auto compute = [&](const Slot& slot, int st, const Weights<CB>& w) {
        const int kb = CB == 3 ? 4 * st : 4 * st + c;
        const uint8_t* at[NT];
        bool in[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int n = 8 * nt + g;
            in[nt] = n < slot.rows && kb < KB;
            const int row = in[nt] ? n : 0, k = in[nt] ? kb : 0;
            at[nt] = XS ? xs + row * x_stride + k * 128
                        : reinterpret_cast<const uint8_t*>(p.x + (int64_t)(slot.row0 + row) * p.K) + (int64_t)k * 128;
        }
        const uint64_t s0 = CB == 2 ? 0 : twice(w.s[0]), s1 = CB == 2 ? 0 : twice(w.s[1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {   // piece j: 8 inputs
                if (CB == 3) {   // behind the end of K the weights are zero, and so must this be (0 inf is NaN)
                    const uint4* q = reinterpret_cast<const uint4*>(at[nt]) + 4 * j + c;
                    x[nt] = in[nt] && kb + (j >> 1) < KB ? *q : make_uint4(0u, 0u, 0u, 0u);
                } else if (XS) {
                    load_if_shared(x[nt], smem_u32(at[nt]) + 16 * (j ^ c), in[nt]);
                } else {
                    load_if(x[nt], reinterpret_cast<const uint4*>(at[nt]) + j, in[nt]);
                }
            }
            uint32_t lo[4], hi[4];
            if (CB == 3) {
                const uint4 q = w.c[0][CB == 3 ? j : 0], r = w.c[1][CB == 3 ? j : 0];
                lo[0] = q.x; lo[1] = q.y; lo[2] = q.z; lo[3] = q.w;
                hi[0] = r.x; hi[1] = r.y; hi[2] = r.z; hi[3] = r.w;
            } else {
                const uint4 q = w.c[0][j >> 2], r = w.c[1][j >> 2];
                const uint32_t wl = (j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w;
                const uint32_t wh = (j & 3) == 0 ? r.x : (j & 3) == 1 ? r.y : (j & 3) == 2 ? r.z : r.w;
                const int sh = j < 4 ? 0 : 8;
                const uint64_t sl = CB == 2 ? twice(mx_scale((__float_as_uint(w.s[0]) >> sh) & 0xFFu)) : s0;
                const uint64_t sr = CB == 2 ? twice(mx_scale((__float_as_uint(w.s[1]) >> sh) & 0xFFu)) : s1;
                decode8(lut, wl, lane8, sl, lo);
                decode8(lut, wh, lane8, sr, hi);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_16816(acc[nt][0], lo[0], hi[0], lo[1], hi[1], x[nt].x, x[nt].y);
                mma_16816(acc[nt][1], lo[2], hi[2], lo[3], hi[3], x[nt].z, x[nt].w);
            }
        }
    };

    const int grid = gridDim.x, all = units > (int)blockIdx.x ? (units - blockIdx.x + grid - 1) / grid : 0;
    bool ready = false;
    for (int i0 = 0; i0 < all; i0 += ROUND) {   // rounds of this block's units i0 ... : blockIdx.x + grid * i
        const int nu = min(ROUND, all - i0), n = nu * steps;
        const int lo = part(warp, n), hi = part(warp + 1, n), first = lo / steps;
        int li = first, unit = first, st = lo - first * steps;   // units of the round: loaded, computed
        ls = st;
        left = hi - lo;
        if (left > 0) seek(blockIdx.x + grid * (i0 + li));
        auto next = [&](Weights<CB>& into) {
            load(into);
            if (--left > 0 && ++ls == steps) {
                ls = 0;
                ++li;
                seek(blockIdx.x + grid * (i0 + li));
            }
        };
        Weights<CB> wa, wb;   // two steps in flight (bf16 weights: one, for the registers)
        next(wa);
        if (CB != 3) next(wb);
        if (!ready) {   // the table and X, behind the first weights' requests
            if (CB != 3)
                for (int i = tid; i < 256 * 16; i += THREADS) {
                    const int v = i >> 4;
                    reinterpret_cast<float4*>(lut)[i] = make_float4(cv[v >> 4], cv[v & 15], cv[v >> 4], cv[v & 15]);
                }
            const int cpr = p.K / 8;
            for (int i = tid; XS && i < p.P * cpr; i += THREADS) {
                const int t = i / cpr, q = i - t * cpr;
                const int at = CB == 3 ? q : (q & ~7) | ((q ^ (q >> 3)) & 3) | (q & 4);
                *reinterpret_cast<uint4*>(xs + t * x_stride + at * 16) =
                    __ldcg(reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.K) + q);
            }
            __syncthreads();
            ready = true;
        }
        Slot slot = left < hi - lo ? slots[XS ? 0 : (blockIdx.x + grid * (i0 + unit)) / tiles] : Slot{0, 0, 0};
        auto clear = [&]() {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                x[nt] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[nt][0][i] = acc[nt][1][i] = 0.0f;
            }
        };
        clear();
        int k = lo;
        auto one = [&](Weights<CB>& w) {   // a step: its products, the next request, the unit's end
            // behind the end of K a lane's weights are zero, and so must be what they multiply
            if (CB != 3 && 4 * st + c >= KB) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x[nt] = make_uint4(0u, 0u, 0u, 0u);
            }
            compute(slot, st, w);
            next(w);
            ++k;
            if (++st == steps || k == hi) {
                // D fragment: outputs g, g + 8, rows of X 2c, 2c + 1
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float* r = red + (warp * SEGMENTS + unit - first) * SEG + (8 * nt + 2 * c) * TOK_STRIDE + g;
                    r[0] = acc[nt][0][0] + acc[nt][1][0];
                    r[TOK_STRIDE] = acc[nt][0][1] + acc[nt][1][1];
                    r[8] = acc[nt][0][2] + acc[nt][1][2];
                    r[TOK_STRIDE + 8] = acc[nt][0][3] + acc[nt][1][3];
                }
                st = 0;
                ++unit;
                if (k < hi) {
                    if (!XS) slot = slots[(blockIdx.x + grid * (i0 + unit)) / tiles];
                    clear();
                }
            }
        };
        while (k < hi) {
            one(wa);
            if (CB != 3 && k < hi) one(wb);
        }
        __syncthreads();
        for (int o = tid; o < nu * 8 * NT * OUTS; o += THREADS) {
            const int i = o / (8 * NT * OUTS), t = (o >> 4) & (8 * NT - 1), r = o & 15;
            const int u = blockIdx.x + grid * (i0 + i), sl = u / tiles;
            const Slot slot = slots[sl];
            if (t >= slot.rows) continue;
            // the warps whose part of the list meets [i steps, (i + 1) steps)
            const int k0 = i * steps, k1 = k0 + steps;
            float z = 0.0f;
            for (int q = (int)((int64_t)k0 * WARPS / n); q < WARPS && part(q, n) < k1; ++q) {
                const int a = part(q, n), e = part(q + 1, n);
                if (e > k0 && e > a) z += red[(q * SEGMENTS + i - a / steps) * SEG + t * TOK_STRIDE + r];
            }
            const int col = (u - sl * tiles) * OUTS + r;
            if (p.bias) z += p.bias[(int64_t)slot.e * p.N + col];
            float y, d;
            with_act(p.act, [&](auto kind) { linear_act<decltype(kind)::value>(z, y, d); });
            const int64_t at = (int64_t)(slot.row0 + t) * p.N + col;
            if (p.residual) y += __bfloat162float(p.residual[at]);
            if (p.out) p.out[at] = __float2bfloat16_rn(y);
            if (p.saved) p.saved[at] = __float2bfloat16_rn(d);
        }
        __syncthreads();
    }
}

template <int CB, int NT, bool XS>
cudaError_t launch_one(const LinearStream& p, int smem, cudaStream_t st) {
    auto kern = linear_stream_kernel<CB, NT, XS>;
    {
        static std::mutex mu;
        static bool set[64] = {false};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        if (!set[dev]) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
            if (e != cudaSuccess) return e;
            set[dev] = true;
        }
    }
    const int slots = p.E == 1 ? 1 : std::min(p.E, p.P) + p.P / (8 * NT);
    return launch_pdl(kern, dim3(std::min(slots * (p.N / OUTS), num_sms())), dim3(THREADS), smem, st, p);
}

int base_smem(int NT) { return LUT_BYTES + WARPS * SEGMENTS * 8 * NT * TOK_STRIDE * 4; }
int64_t x_smem(int64_t P, int K) { return P * (K * 2LL + 64); }

template <int CB, int NT>
cudaError_t launch_nt(const LinearStream& p, cudaStream_t st) {
    const int base = base_smem(NT);
    const int64_t with_x = base + x_smem(p.P, p.K);
    if (!p.offsets && with_x <= MAX_SMEM) return launch_one<CB, NT, true>(p, (int)with_x, st);
    return launch_one<CB, NT, false>(p, base, st);
}

template <int CB>
cudaError_t launch_cb(const LinearStream& p, cudaStream_t st) {
    // grouped rows are few per expert
    return p.P <= 8 || p.offsets ? launch_nt<CB, 1>(p, st) : launch_nt<CB, 2>(p, st);
}

}  // namespace

// Streamed / on the tensor-core tiles, us, in NF4 (MXFP4 for 2880) and in bf16:
//   dense, 8 rows, 4096 by 14336: 21 / 72, 24 / 71; 16 rows: 51 / 40, 31 / 39 (they do not fit);
//   16 rows that fit, 2048 by 2048: 8.5 / 14.1, 8.4 / 13.8; 2880 by 2880: 11.7 / 18.9, 13.5 / 19.7;
//   64 experts of 2048 by 1024, 256 rows: 51 / 76, 47 / 70; 384: 64 / 76, 50 / 71; 512: 80 / 76, 58 / 72;
//   128 experts of 2048 by 768, 512 rows: 79 / 109, 72 / 101; 768: 96 / 110, 75 / 103; 1024 (NF4): 119 / 110.
// So the limit of 4 rows per expert is on the safe side: at 6 the streamed form is still ahead.
bool linear_streams(bool grouped, int E, int64_t P, int K) {
    if (grouped) return P <= std::min<int64_t>(4LL * E, kStreamGroupedRows);
    return P <= 8 || (P <= 16 && base_smem(2) + x_smem(P, K) <= MAX_SMEM);
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
