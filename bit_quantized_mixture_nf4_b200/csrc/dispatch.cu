// Tokens to expert-sorted rows and back, as entry points of their own.
//
//   dispatch           rows[r] = x[perm[r] / k], pairs p = t*k + j stable by expert
//   dispatch backward  grad_x[t] = sum_j grad_rows[inv_perm[t,j]]
//   combine            y[t] = sum_j w[t,j] rows[inv_perm[t,j]]
//   combine backward   grad_rows[r] = w[t,j] grad_y[t],  grad_w[t,j] = <grad_y[t], rows[r]>
//
// All four are bound by HBM: per pair one row of H elements is written or read (both in
// the combine's backward) next to one row per token.  Sums run in fp32 in slot order and
// are rounded once, so results do not depend on the launch.  Tokens are the outer unit
// everywhere: a token's row is read once and written to its k places (or summed from
// them), which moves 1/k of the token bytes that a copy per pair would.  Measured (of the
// HBM rate of a copy): dispatch of 4096 tokens to 8 of 64 experts, rows of 2048 bf16, 33 us
// (70%; 8 us of it make the maps before the copies start); combine of 8192 x 8, 48 us (95%);
// its backward over 16384 x 2 rows of 4096, 109 us (94%).
#include <algorithm>
#include <initializer_list>

#include "../../include/e4b.h"
#include "rowops.cuh"

namespace e4b {

constexpr int kMaxE = 256, kMaxK = 8;
constexpr int kDispThreads = 256, kDispWarps = kDispThreads / 32;
// Up to this many pairs every block sorts all of them for itself, in one launch; above
// it two chained launches (histogram, place and copy) share the sorting, three (a scan
// between them) where a placing block would read more than kOwnCounts integers.
// Rows of 2048 bf16, 8 experts a token, us:
//   128 tokens, 64 experts: one launch 4.3, chained 9.5.  A limit of 2048 pairs costs the
//   small calls its larger tables (128 tokens: 5.2) and loses at 256 tokens (10.3 against 9.6).
//   own counts / with the scan: 1024 tokens, 256 experts (2560 integers) 14.8 / 17.1;
//   4096, 128 (1024 + 2048) 31.2 / 32.9; 8192, 128 (4096) 57.9 / 56.9; 16384, 256 (rows of 512)
//   56.5 / 38.9.
constexpr int kOneLaunchPairs = 1024;
constexpr int kOwnCounts = 3500;

// Tokens of one placing block: at most 64 pairs and 16 tokens (enough blocks to keep the
// copies' loads in flight).
static int disp_tokens(int k) { return std::min(16, 64 / k); }

// The histogram's chunks: `subs` placing blocks each, so that a placing block reads the
// fewest integers; a scan kernel adds the counts where those are too many all the same.
struct Chunks {
    int subs, n;
    bool scan;
    Chunks(int E, int k, int64_t P) {
        const int64_t block = (int64_t)disp_tokens(k) * k;
        auto chunks = [&](int s) { return (P + block * s - 1) / (block * s); };
        auto cost = [&](int s) { return chunks(s) * E + block * s / 2; };   // integers a placing block reads
        subs = 16;
        if (cost(64) < cost(subs)) subs = 64;
        scan = cost(subs) > kOwnCounts;
        if (scan) subs = 16;
        n = (int)chunks(subs);
    }
};

__device__ __forceinline__ int pair_expert(const int32_t* idx, int64_t p, int E) {
    const int e = __ldcg(idx + p);
    return e >= 0 && e < E ? e : -1;   // experts outside [0, E): the pair is dropped
}

// Exclusive sum over the block's kDispThreads values, in thread order; *total their sum.
__device__ __forceinline__ int block_exclusive(int v, int* s_warp, int* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int base = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kDispWarps; ++w) {
        const int t = s_warp[w];
        base += w < warp ? t : 0;
        sum += t;
    }
    *total = sum;
    return base + x - v;
}

// Copies `n_tok` tokens from t0 on to the rows in inv_s (their k rows each; -1: none).
// A unit is U x 32 vectors of one token: U loads and U k stores per lane.  The first loads
// are issued by start(), before the rows are known; every next ones before the stores.
template <typename R, int U>
struct RowCopy {
    const void* x;
    void* rows;
    int64_t t0;
    int n_tok, nvec, k;
    int segs, step, tl, sg;
    R val[U];
    __device__ __forceinline__ bool live() const { return tl < n_tok; }
    __device__ __forceinline__ int vec() const { return sg * (32 * U) + (threadIdx.x & 31); }
    __device__ __forceinline__ void fetch() {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (live() && vec() + 32 * u < nvec) val[u] = ld_once<R>(x, (t0 + tl) * nvec + vec() + 32 * u);
    }
    __device__ __forceinline__ void start(int first, int stride) {
        segs = max(1, (nvec + 32 * U - 1) / (32 * U));   // without rows: one, so that first / segs is defined
        step = stride;
        tl = first / segs;
        sg = first - tl * segs;
        fetch();
    }
    __device__ __forceinline__ void run(const int* inv_s) {
        while (live()) {
            R cur[U];
#pragma unroll
            for (int u = 0; u < U; ++u) cur[u] = val[u];
            const int t = tl, v = vec();
            sg += step;
            while (sg >= segs) {
                sg -= segs;
                ++tl;
            }
            fetch();
            for (int j = 0; j < k; ++j) {
                const int r = inv_s[t * k + j];
                if (r < 0) continue;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (v + 32 * u < nvec) st_once<R>(rows, (int64_t)r * nvec + v + 32 * u, cur[u]);
            }
        }
    }
};

// One launch: every block sorts the P <= kOneLaunchPairs pairs in shared memory (warp w
// counts and ranks its own contiguous part, so the order stays stable) and copies its
// share of the rows; block 0 writes the maps.  Latency-bound: one read of the indices and a
// few barriers (8 tokens to 8 of 128 experts: 3.0 us in a graph).
template <typename R>
__global__ void __launch_bounds__(kDispThreads) dispatch_one_kernel(const int32_t* __restrict__ idx, int P, int E, int k,
                                                                    const void* __restrict__ x, void* __restrict__ rows,
                                                                    int nvec, int32_t* __restrict__ offsets,
                                                                    int32_t* __restrict__ perm,
                                                                    int32_t* __restrict__ inv_perm) {
    constexpr int PER_LANE = kOneLaunchPairs / kDispThreads;
    __shared__ int wbase[kDispWarps][kMaxE];
    __shared__ int inv_s[kOneLaunchPairs];
    __shared__ int s_warp[kDispWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kDispWarps * kMaxE; i += kDispThreads) (&wbase[0][0])[i] = 0;
    pdl_release();
    pdl_wait();
    const int rounds = (P + kDispThreads - 1) / kDispThreads;
    const int p0 = warp * rounds * 32 + lane;   // this warp's pairs: p0, p0 + 32, ... (rounds of them)
    int e[PER_LANE];
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q) e[q] = q < rounds && p0 + 32 * q < P ? pair_expert(idx, p0 + 32 * q, E) : -1;
    RowCopy<R, 1> copy{x, rows, 0, rows ? P / k : 0, nvec, k};
    copy.start(blockIdx.x * kDispWarps + warp, gridDim.x * kDispWarps);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q)
        if (e[q] >= 0) atomicAdd(&wbase[warp][e[q]], 1);
    __syncthreads();
    int c[kDispWarps], tot = 0;
#pragma unroll
    for (int w = 0; w < kDispWarps; ++w) {
        c[w] = wbase[w][tid];
        tot += c[w];
    }
    int n;
    int run = block_exclusive(tot, s_warp, &n);
    if (blockIdx.x == 0) {
        if (tid < E) offsets[tid] = run;
        if (tid == 0) offsets[E] = n;
    }
#pragma unroll
    for (int w = 0; w < kDispWarps; ++w) {
        wbase[w][tid] = run;
        run += c[w];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q) {
        if (q >= rounds) break;
        const int p = p0 + 32 * q;
        const uint32_t peers = __match_any_sync(0xffffffffu, e[q]);
        const int rank = __popc(peers & ((1u << lane) - 1u));
        const int r = e[q] >= 0 ? wbase[warp][e[q]] + rank : -1;
        __syncwarp();
        if (e[q] >= 0 && rank == 0) wbase[warp][e[q]] += __popc(peers);
        __syncwarp();
        if (p < P) {
            inv_s[p] = r;
            if (blockIdx.x == 0) {
                inv_perm[p] = r;
                if (r >= 0) perm[r] = p;
            }
        }
    }
    __syncthreads();
    copy.run(inv_s);
}

// counts[c][e]: pairs of expert e in chunk c (integer sums: the order does not matter).
__global__ void __launch_bounds__(1024) dispatch_hist_kernel(const int32_t* __restrict__ idx, int64_t P, int E,
                                                             int chunk_pairs, int32_t* __restrict__ counts) {
    __shared__ int cnt[kMaxE];
    if (threadIdx.x < kMaxE) cnt[threadIdx.x] = 0;
    pdl_release();
    pdl_wait();
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * chunk_pairs, p1 = min(P, p0 + chunk_pairs);
#pragma unroll 4
    for (int64_t p = p0 + threadIdx.x; p < p1; p += blockDim.x) {
        const int e = pair_expert(idx, p, E);
        if (e >= 0) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    if (threadIdx.x < E) counts[(int64_t)blockIdx.x * E + threadIdx.x] = cnt[threadIdx.x];
}

// One block of 1024 threads: counts become each chunk's first row of each expert, and the
// experts' offsets.  The chunks are cut into `slices` runs, a thread per (slice, expert).
__global__ void __launch_bounds__(1024) dispatch_scan_kernel(int32_t* __restrict__ counts, int nchunks, int E,
                                                             int slices, int32_t* __restrict__ offsets) {
    __shared__ int part[1024];
    __shared__ int first[kMaxE];
    const int tid = threadIdx.x, sl = tid / E, e = tid - sl * E;
    const bool live = sl < slices;
    const int per = (nchunks + slices - 1) / slices;
    const int c0 = min(nchunks, sl * per), c1 = min(nchunks, c0 + per);
    pdl_release();
    pdl_wait();
    int sum = 0;
    if (live) {
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += __ldcg(counts + (int64_t)c * E + e);
        part[tid] = sum;
    }
    __syncthreads();
    if (tid < 32) {   // exclusive sums over the experts
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            int tot = 0;
            if (e0 + tid < E)
                for (int s = 0; s < slices; ++s) tot += part[s * E + e0 + tid];
            int x = tot;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, o);
                if (tid >= o) x += u;
            }
            if (e0 + tid < E) {
                first[e0 + tid] = run + x - tot;
                offsets[e0 + tid] = run + x - tot;
            }
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (tid == 0) offsets[E] = run;
    }
    __syncthreads();
    if (!live) return;
    int run = first[e];
    for (int s = 0; s < sl; ++s) run += part[s * E + e];
#pragma unroll 8
    for (int c = c0; c < c1; ++c) {
        int32_t* at = counts + (int64_t)c * E + e;
        const int n = __ldcg(at);
        *at = run;
        run += n;
    }
}

// Block b places the pairs of its tokens and copies their rows.  Where its expert starts:
// SCANNED, from the scan kernel; else the block adds the chunk counts itself (a few thousand
// integers from L2, cheaper than the scan's launch).  The pairs of its chunk before its own
// are counted again, which costs less than a histogram as fine as the blocks.
template <typename R, bool SCANNED>
__global__ void __launch_bounds__(kDispThreads) dispatch_place_kernel(const int32_t* __restrict__ idx, int64_t T, int E,
                                                                      int k, int tokens, int subs, int nchunks,
                                                                      const int32_t* __restrict__ counts,
                                                                      const void* __restrict__ x, void* __restrict__ rows,
                                                                      int nvec, int32_t* __restrict__ offsets,
                                                                      int32_t* __restrict__ perm,
                                                                      int32_t* __restrict__ inv_perm) {
    __shared__ int cnt[kMaxE];
    __shared__ int part[2][kDispThreads];
    __shared__ int s_warp[kDispWarps];
    __shared__ int inv_s[64];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int chunk = blockIdx.x / subs;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int n_tok = (int)min((int64_t)tokens, T - t0);
    pdl_release();
    pdl_wait();
    RowCopy<R, 4> copy{x, rows, t0, rows ? n_tok : 0, nvec, k};
    copy.start(warp, kDispWarps);
    const int n_pair = n_tok * k;
    int own[2];   // warp 0: the experts of this block's pairs
#pragma unroll
    for (int q = 0; q < 2; ++q) own[q] = warp == 0 && 32 * q + lane < n_pair ? pair_expert(idx, t0 * k + 32 * q + lane, E) : -1;
    if (SCANNED) {
        if (tid < E) cnt[tid] = __ldcg(counts + (int64_t)chunk * E + tid);
    } else {
        const int slices = kDispThreads / E, sl = tid / E, e = tid - sl * E;
        int tot = 0, pre = 0;   // of the slice: all chunks, and those before this block's
        if (sl < slices) {
#pragma unroll 8
            for (int c = sl; c < nchunks; c += slices) {
                const int n = __ldcg(counts + c * E + e);
                tot += n;
                pre += c < chunk ? n : 0;
            }
        }
        part[0][tid] = tot;
        part[1][tid] = pre;
        __syncthreads();
        tot = pre = 0;
        if (tid < E)
            for (int s = 0; s < slices; ++s) {
                tot += part[0][s * E + tid];
                pre += part[1][s * E + tid];
            }
        int n;
        const int first = block_exclusive(tot, s_warp, &n);
        if (tid < E) cnt[tid] = first + pre;
        if (blockIdx.x == 0) {
            if (tid < E) offsets[tid] = first;
            if (tid == 0) offsets[E] = n;
        }
    }
    __syncthreads();
#pragma unroll 4
    for (int64_t p = (int64_t)chunk * subs * tokens * k + tid; p < t0 * k; p += kDispThreads) {
        const int e = pair_expert(idx, p, E);
        if (e >= 0) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int i = 32 * q + lane, e = own[q];
            if (32 * q >= n_pair) break;
            const uint32_t peers = __match_any_sync(0xffffffffu, e);
            const int rank = __popc(peers & ((1u << lane) - 1u));
            const int r = e >= 0 ? cnt[e] + rank : -1;
            __syncwarp();
            if (e >= 0 && rank == 0) cnt[e] += __popc(peers);
            __syncwarp();
            if (i < n_pair) {
                inv_s[i] = r;
                inv_perm[t0 * k + i] = r;
                if (r >= 0) perm[r] = (int32_t)(t0 * k + i);
            }
        }
    }
    __syncthreads();
    copy.run(inv_s);
}

// y[t] = sum_j w[t,j] rows[inv_perm[t,j]] (w null: 1).  A warp takes U x 32 vectors of one
// token, at least 4 row loads in flight per lane; lane j < k holds the j-th row and weight (the
// next unit's are on their way while the loads arrive).  Entries outside [0, P) add nothing.
template <typename E, int V, int K, int U>
__global__ void __launch_bounds__(256) combine_rows_kernel(const E* __restrict__ rows, const int32_t* __restrict__ inv_perm,
                                                           const float* __restrict__ w, int64_t T, int k, int nvec,
                                                           E* __restrict__ y) {
    using R = raw_t<E, V>;
    const int lane = threadIdx.x & 31, segs = (nvec + 32 * U - 1) / (32 * U);
    const int64_t first = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> 5, P = T * k;
    const int64_t dt = step / segs;
    const int ds = (int)(step - dt * segs);
    int64_t t = first / segs;
    int sg = (int)(first - t * segs);
    pdl_release();
    pdl_wait();
    int64_t r = -1;
    float wt = 0.0f;
    auto fetch = [&](int64_t at) {
        r = -1;
        if (at < T && lane < k) {
            r = __ldcg(inv_perm + at * k + lane);
            wt = w ? __ldcg(w + at * k + lane) : 1.0f;
            if (r >= P) r = -1;
        }
    };
    fetch(t);
    while (t < T) {
        const int v = sg * 32 * U + lane;
        const int64_t out = t * nvec + v;
        R raw[U][K];
        bool in[K];
        float wj[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int64_t rj = __shfl_sync(0xffffffffu, r, j);
            wj[j] = __shfl_sync(0xffffffffu, wt, j);
            in[j] = rj >= 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (in[j] && v + 32 * u < nvec) raw[u][j] = ld_once<R>(rows, rj * nvec + v + 32 * u);
        }
        t += dt;
        sg += ds;
        if (sg >= segs) {
            sg -= segs;
            ++t;
        }
        fetch(t);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v + 32 * u >= nvec) break;
            float acc[V];
#pragma unroll
            for (int c = 0; c < V; ++c) acc[c] = 0.0f;
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (!in[j]) continue;
                float f[V];
                unpack<E, V>(raw[u][j], f);
#pragma unroll
                for (int c = 0; c < V; ++c) acc[c] = fmaf(wj[j], f[c], acc[c]);
            }
            st_once<R>(y, out + 32 * u, pack<E, V>(acc));
        }
    }
}

// One block per token: every vector of grad_y is read once, scaled into the token's k rows
// and multiplied with them; the k dot products are reduced in a fixed order.
template <typename E, int V, int K>
__global__ void __launch_bounds__(256) combine_backward_kernel(const E* __restrict__ rows,
                                                               const int32_t* __restrict__ inv_perm,
                                                               const float* __restrict__ w, const E* __restrict__ gy,
                                                               int64_t T, int k, int nvec, E* __restrict__ grad_rows,
                                                               float* __restrict__ grad_w) {
    using R = raw_t<E, V>;
    __shared__ float s_dot[8][K];
    pdl_release();
    pdl_wait();
    const int64_t P = T * k, t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    int64_t row[K];
    float wj[K], dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int64_t r = j < k ? __ldcg(inv_perm + t * k + j) : -1;
        row[j] = r >= 0 && r < P ? r * nvec : -1;
        wj[j] = j < k && w ? __ldcg(w + t * k + j) : 1.0f;
        dot[j] = 0.0f;
    }
    for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
        R raw[K];
        if (grad_w) {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (row[j] >= 0) raw[j] = ld_once<R>(rows, row[j] + v);
        }
        float g[V];
        unpack<E, V>(ld_once<R>(gy, t * nvec + v), g);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (row[j] < 0) continue;
            float f[V];
            if (grad_w) {
                unpack<E, V>(raw[j], f);
#pragma unroll
                for (int c = 0; c < V; ++c) dot[j] = fmaf(g[c], f[c], dot[j]);
            }
            if (grad_rows) {
#pragma unroll
                for (int c = 0; c < V; ++c) f[c] = wj[j] * g[c];
                st_once<R>(grad_rows, row[j] + v, pack<E, V>(f));
            }
        }
    }
    if (!grad_w) return;
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (lane == 0) s_dot[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < k) {
        float s = 0.0f;
        for (int i = 0; i < nw; ++i) s += s_dot[i][threadIdx.x];
        grad_w[t * k + threadIdx.x] = s;
    }
}

// ------------------------------------------------------------------ host side

// f(E{}, integral_constant V) for the element type and vector width.
template <typename F>
static cudaError_t with_row_vector(e4b_dtype dt, int bytes, F f) {
    if (dt == E4B_BF16) {
        if (bytes == 16) return f((__nv_bfloat16*)nullptr, std::integral_constant<int, 8>());
        if (bytes == 4) return f((__nv_bfloat16*)nullptr, std::integral_constant<int, 2>());
        return f((__nv_bfloat16*)nullptr, std::integral_constant<int, 1>());
    }
    if (bytes == 16) return f((float*)nullptr, std::integral_constant<int, 4>());
    return f((float*)nullptr, std::integral_constant<int, 1>());
}

template <typename F>
static cudaError_t with_slots(int k, F f) {
    if (k <= 1) return f(std::integral_constant<int, 1>());
    if (k <= 2) return f(std::integral_constant<int, 2>());
    if (k <= 4) return f(std::integral_constant<int, 4>());
    return f(std::integral_constant<int, 8>());
}

template <typename R>
static cudaError_t launch_dispatch(const int32_t* idx, int64_t T, int E, int k, const void* x, void* rows,
                                   int64_t row_bytes, int32_t* offsets, int32_t* perm, int32_t* inv_perm, int32_t* counts,
                                   cudaStream_t st) {
    const int64_t P = T * k;
    const int nvec = (int)(row_bytes / (int64_t)sizeof(R));
    if (P <= kOneLaunchPairs) {
        const int64_t units = rows ? T * ((nvec + 31) / 32) : 1;
        const int grid = (int)std::min<int64_t>((units + kDispWarps - 1) / kDispWarps, 4 * num_sms());
        return launch_pdl(dispatch_one_kernel<R>, dim3(grid), dim3(kDispThreads), 0, st, idx, (int)P, E, k, x, rows, nvec,
                          offsets, perm, inv_perm);
    }
    const int tokens = disp_tokens(k), blocks = (int)((T + tokens - 1) / tokens);
    const Chunks ch(E, k, P);
    const int64_t chunk_pairs = (int64_t)ch.subs * tokens * k;
    cudaError_t err = launch_pdl(dispatch_hist_kernel, dim3(ch.n), dim3(chunk_pairs > 2048 ? 1024 : 256), 0, st, idx, P, E,
                                 (int)chunk_pairs, counts);
    if (err != cudaSuccess) return err;
    if (ch.scan) {
        err = launch_pdl(dispatch_scan_kernel, dim3(1), dim3(1024), 0, st, counts, ch.n, E, std::min(1024 / E, ch.n),
                         offsets);
        if (err != cudaSuccess) return err;
    }
    return launch_pdl(ch.scan ? dispatch_place_kernel<R, true> : dispatch_place_kernel<R, false>, dim3(blocks),
                      dim3(kDispThreads), 0, st, idx, T, E, k, tokens, ch.subs, ch.n, (const int32_t*)counts, x, rows,
                      nvec, offsets, perm, inv_perm);
}

static bool bad_rows(e4b_dtype dt, int64_t T, int H, int k) {
    return (dt != E4B_F32 && dt != E4B_BF16) || T < 0 || H < 1 || k < 1 || k > kMaxK || too_many_pairs(T, k);
}
static int elem_bytes(e4b_dtype dt) { return dt == E4B_BF16 ? 2 : 4; }

static e4b_status combine_impl(const void* rows, const int32_t* inv_perm, const float* w, e4b_dtype dt, int64_t T, int H,
                               int k, void* y, void* stream) {
    if (bad_rows(dt, T, H, k)) return E4B_ERR_INVALID_ARG;
    if (T == 0) return E4B_OK;
    if (!rows || !inv_perm || !y || off_boundary(4, {inv_perm, w})) return E4B_ERR_INVALID_ARG;
    const int vb = row_vector_bytes((int64_t)H * elem_bytes(dt), elem_bytes(dt), {rows, y});
    if (!vb) return E4B_ERR_INVALID_ARG;
    const cudaError_t err = with_row_vector(dt, vb, [&](auto* e, auto v) {
        using E = std::remove_pointer_t<decltype(e)>;
        constexpr int V = decltype(v)::value;
        return with_slots(k, [&](auto kk) {
            const int nvec = H / V;
            constexpr int K = decltype(kk)::value, U = K < 4 ? 4 / K : 1;
            const int64_t units = T * ((nvec + 32 * U - 1) / (32 * U));
            const int64_t blocks = std::min<int64_t>((units + 7) / 8, 24 * num_sms());
            return launch_pdl(combine_rows_kernel<E, V, K, U>, dim3((unsigned)blocks), dim3(256), 0,
                              static_cast<cudaStream_t>(stream), static_cast<const E*>(rows), inv_perm, w, T, k, nvec,
                              static_cast<E*>(y));
        });
    });
    return err == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

}  // namespace e4b

using namespace e4b;

extern "C" {

size_t e4b_moe_dispatch_workspace_size(int E, int top_k, int64_t T) {
    if (E < 1 || E > kMaxE || top_k < 1 || top_k > kMaxK || T < 0 || too_many_pairs(T, top_k)) return 0;
    const int64_t P = T * top_k, block = (int64_t)disp_tokens(top_k) * top_k;
    // the finest chunks that this or any smaller number of tokens may take
    return P <= kOneLaunchPairs ? 0 : (size_t)((P + 16 * block - 1) / (16 * block)) * E * 4;
}

e4b_status e4b_moe_dispatch(int E, int top_k, const int32_t* topk_idx, const void* x, e4b_dtype dtype, int64_t T, int H,
                            void* rows, int32_t* offsets, int32_t* perm, int32_t* inv_perm, void* workspace,
                            size_t ws_bytes, void* stream) {
    NvtxScope nvtx_scope("e4b_moe_dispatch");
    if (E < 1 || E > kMaxE || bad_rows(dtype, T, H, top_k)) return E4B_ERR_INVALID_ARG;
    if (off_boundary(4, {topk_idx, offsets, perm, inv_perm})) return E4B_ERR_INVALID_ARG;
    if (!offsets || (x == nullptr) != (rows == nullptr)) return E4B_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return cudaMemsetAsync(offsets, 0, (size_t)(E + 1) * 4, st) == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
    if (!topk_idx || !perm || !inv_perm) return E4B_ERR_INVALID_ARG;
    const size_t need = T * top_k <= kOneLaunchPairs ? 0 : (size_t)Chunks(E, top_k, T * top_k).n * E * 4;
    if (need && (!workspace || ws_bytes < need)) return E4B_ERR_WORKSPACE;
    if (need && off_boundary(16, {workspace})) return E4B_ERR_INVALID_ARG;
    const int64_t row_bytes = (int64_t)H * elem_bytes(dtype);
    int32_t* counts = static_cast<int32_t*>(workspace);
    cudaError_t err;
    switch (x ? row_vector_bytes(row_bytes, elem_bytes(dtype), {x, rows}) : 16) {
        case 0: return E4B_ERR_INVALID_ARG;
        case 16: err = launch_dispatch<uint4>(topk_idx, T, E, top_k, x, rows, row_bytes, offsets, perm, inv_perm, counts, st); break;
        case 4: err = launch_dispatch<uint32_t>(topk_idx, T, E, top_k, x, rows, row_bytes, offsets, perm, inv_perm, counts, st); break;
        default: err = launch_dispatch<uint16_t>(topk_idx, T, E, top_k, x, rows, row_bytes, offsets, perm, inv_perm, counts, st);
    }
    return err == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

e4b_status e4b_moe_dispatch_backward(const void* grad_rows, const int32_t* inv_perm, e4b_dtype dtype, int64_t T, int H,
                                     int top_k, void* grad_x, void* stream) {
    NvtxScope nvtx_scope("e4b_moe_dispatch_backward");
    return combine_impl(grad_rows, inv_perm, nullptr, dtype, T, H, top_k, grad_x, stream);
}

e4b_status e4b_moe_combine(const void* rows, const int32_t* inv_perm, const float* topk_w, e4b_dtype dtype, int64_t T,
                           int H, int top_k, void* y, void* stream) {
    NvtxScope nvtx_scope("e4b_moe_combine");
    return combine_impl(rows, inv_perm, topk_w, dtype, T, H, top_k, y, stream);
}

e4b_status e4b_moe_combine_backward(const void* rows, const int32_t* inv_perm, const float* topk_w, const void* grad_y,
                                    e4b_dtype dtype, int64_t T, int H, int top_k, void* grad_rows, float* grad_topk_w,
                                    void* stream) {
    NvtxScope nvtx_scope("e4b_moe_combine_backward");
    if (bad_rows(dtype, T, H, top_k)) return E4B_ERR_INVALID_ARG;
    if (T == 0) return E4B_OK;
    if (!inv_perm || !grad_y || (!grad_rows && !grad_topk_w) || (grad_topk_w && !rows)) return E4B_ERR_INVALID_ARG;
    if (off_boundary(4, {inv_perm, topk_w, grad_topk_w})) return E4B_ERR_INVALID_ARG;
    // an absent operand does not narrow the vectors
    const int vb = row_vector_bytes((int64_t)H * elem_bytes(dtype), elem_bytes(dtype),
                                    {grad_topk_w ? rows : nullptr, grad_y, grad_rows});
    if (!vb) return E4B_ERR_INVALID_ARG;
    const cudaError_t err = with_row_vector(dtype, vb, [&](auto* e, auto v) {
        using E = std::remove_pointer_t<decltype(e)>;
        constexpr int V = decltype(v)::value;
        return with_slots(top_k, [&](auto kk) {
            const int nvec = H / V, threads = std::min(256, (nvec + 31) / 32 * 32);
            return launch_pdl(combine_backward_kernel<E, V, decltype(kk)::value>, dim3((unsigned)T), dim3(threads), 0,
                              static_cast<cudaStream_t>(stream), static_cast<const E*>(rows), inv_perm, topk_w,
                              static_cast<const E*>(grad_y), T, top_k, nvec, static_cast<E*>(grad_rows), grad_topk_w);
        });
    });
    return err == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

}  // extern "C"
