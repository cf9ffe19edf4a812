// Block norm forward over long runs of rows (the formulas are in block_norm.cu, the ring in
// block_ring.cuh).
#include "block_ring.cuh"

namespace e4b {
namespace {


// FULL: both norms (with a branch), known at compile time: the conditions on them cost as many
// instructions as the arithmetic (register moves where their sides meet).
template <typename E, int V, int NV, bool BR, int GK, bool FULL, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) block_forward_ring_kernel(const BlockArgs a, const RingPlan pl) {
    using R = raw_t<E, V>;
    constexpr bool ALIGNED = V * sizeof(E) == 16;
    constexpr bool chan = BR && GK == E4B_GATE_CHANNEL, elem = BR && GK == E4B_GATE_ELEMENT;
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ uint64_t s_full[kRingGroups][kRingStages];
    __shared__ int s_abort;
    __shared__ RowSums<1> s_red[2];
    RowRing ring;
    const int64_t first = ring_setup<E>(ring, a, pl, 1 + BR + elem, dsm, s_full, s_abort);
    ring_source(ring, 0, a.h);
    if (BR) ring_source(ring, 1, a.f);
    if (elem) ring_source(ring, 2, a.gate);
    const int tx = pl.tx, x = threadIdx.x % tx, row_bytes = a.H * (int)sizeof(E), sb = pl.slot_bytes;
    if (x == 0)
        for (int i = 0; i < pl.stages; ++i) ring.issue<E, ALIGNED>();
    const bool post = BR && (FULL || a.post_w), pre = FULL || a.pre_w;
    float pw[NV][V], nw[NV][V];   // the channel gate multiplies the post-norm's weight
    load_channels<V, NV>(post ? a.post_w : nullptr, a.offset, tx, x, a.nvec, pw);
    load_channels<V, NV>(a.pre_w, a.offset, tx, x, a.nvec, nw);
    if (chan) {
        float cg[NV][V];
        load_channels<V, NV>(static_cast<const float*>(a.gate), 0.0f, tx, x, a.nvec, cg);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) pw[i][j] *= a.gate_sigmoid ? sigmoid<false>(cg[i][j]) : cg[i][j];
    }
    const float inv_h = 1.0f / (float)a.H;
    const bool token = BR && !chan && !elem && a.gate_kind == E4B_GATE_TOKEN;
    const float* gates = static_cast<const float*>(a.gate);
    float gt_next = token && first * pl.rows < a.T ? __ldcg(gates + first * pl.rows) : 1.0f;   // one row ahead
    for (int64_t u = first; u < ring.units; u += ring.step) {
        const uint8_t* row = ring.wait<ALIGNED>(u);
        const int64_t t0 = u * pl.rows, t1 = min(a.T, t0 + pl.rows);
        for (int64_t t = t0; t < t1; ++t, row += row_bytes) {
            const float gt = gt_next;
            if (token) {
                const int64_t next = t + 1 < t1 ? t + 1 : (u + ring.step) * pl.rows;
                if (next < a.T) gt_next = __ldcg(gates + next);
            }
            const int64_t at = t * a.nvec;
            float o[NV][V], f[NV][V];
            float s[1] = {0.0f};
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int v = q * tx + x;
                read_row<E, V>(row, v, a.nvec, o[q]);
                if (!BR) continue;
                read_row<E, V>(row + sb, v, a.nvec, f[q]);
#pragma unroll
                for (int j = 0; j < V; ++j) s[0] = fmaf(f[q][j], f[q][j], s[0]);
                if (elem) {
                    float g[V];
                    read_row<E, V>(row + 2 * sb, v, a.nvec, g);
#pragma unroll
                    for (int j = 0; j < V; ++j) f[q][j] *= a.gate_sigmoid ? sigmoid<kFastGate<E>>(g[j]) : g[j];
                }
            }
            float s2 = 0.0f;
            if (BR) {
                float r = a.scale;
                if (token) r *= a.gate_sigmoid ? sigmoid<false>(gt) : gt;
                if (post) {
                    row_sum<1>(s, tx, s_red[0]);
                    r *= rsqrtf(s[0] * inv_h + a.eps);
                }
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    const int v = q * tx + x;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        o[q][j] = fmaf(f[q][j] * pw[q][j], r, o[q][j]);
                        s2 = fmaf(o[q][j], o[q][j], s2);
                    }
                    if (v < a.nvec) st_once<R>(a.o, at + v, pack<E, V>(o[q]));
                }
            } else {
#pragma unroll
                for (int q = 0; q < NV; ++q)
#pragma unroll
                    for (int j = 0; j < V; ++j) s2 = fmaf(o[q][j], o[q][j], s2);
            }
            if (pre) {
                s[0] = s2;
                row_sum<1>(s, tx, s_red[1]);
                const float ro = rsqrtf(s[0] * inv_h + a.eps);
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    const int v = q * tx + x;
#pragma unroll
                    for (int j = 0; j < V; ++j) o[q][j] *= ro * nw[q][j];
                    if (v < a.nvec) st_once<R>(a.n, at + v, pack<E, V>(o[q]));
                }
            }
        }
        // the slot's last reads lie before the last row's first reduction, if there is one
        if (tx == 32) __syncwarp();
        else if (!post && !pre) __syncthreads();
        if (x == 0) ring.issue<E, ALIGNED>();
        ring.advance();
    }
}

}  // namespace

bool block_ring_forward(e4b_dtype dt, bool dense, const BlockArgs& args, cudaStream_t st, cudaError_t* err) {
    BlockArgs a = args;
    const int es = dt == E4B_BF16 ? 2 : 4;
    const int arrays = 1 + dense + (a.gate_kind == E4B_GATE_ELEMENT);
    // 16 elements a thread for long rows (16384 x 4096 bf16: 96 us against 104; 8191 x 2880: 69
    // against 60), with 640 threads of them on an SM, and 1024 otherwise; fewer where a row takes
    // a warp (longer copies: 16384 x 256 in 22 us instead of 38) or is read narrowly (80 registers)
    const bool wide = (int64_t)a.H * es % 16 == 0;
    const int elems = (wide && a.H >= 4096) || a.H > 4096 ? 16 : 8;
    const int per_sm = elems == 16 ? 640 : !wide ? 768 : a.H <= 256 ? 512 : 1024;
    const RingShape sh(a.H, es, arrays, a.T, elems, per_sm);
    if (!sh.fits) return false;
    *err = with_ring_vector(dt, a.H, [&](auto* e, auto vv) {
        using E = std::remove_pointer_t<decltype(e)>;
        constexpr int V = decltype(vv)::value;
        a.nvec = a.H / V;
        return with_gate(a.gate_kind, [&](auto gk) {
            constexpr int G = decltype(gk)::value;
            auto pick = [&](auto elems, auto maxt, auto minb) {
                constexpr int NV = decltype(elems)::value / V, MT = decltype(maxt)::value, MB = decltype(minb)::value;
                constexpr bool WIDE = V * sizeof(E) == 16;   // narrow rows keep the general instances
                return !dense ? block_forward_ring_kernel<E, V, NV, false, E4B_GATE_NONE, true, MT, MB>
                       : WIDE && a.post_w && a.pre_w ? block_forward_ring_kernel<E, V, NV, true, G, WIDE, MT, MB>
                                                     : block_forward_ring_kernel<E, V, NV, true, G, false, MT, MB>;
            };
            using std::integral_constant;
            using i = std::integral_constant<int, 8>;
            using j = std::integral_constant<int, 16>;
            constexpr bool W = V * sizeof(E) == 16;
            auto kern = elems == 8 ? (sh.threads <= 256 ? pick(i(), integral_constant<int, 256>(), integral_constant<int, W ? 4 : 3>())
                                                        : pick(i(), integral_constant<int, 512>(), integral_constant<int, W ? 2 : 1>()))
                                   : (sh.threads <= 256 ? pick(j(), integral_constant<int, 256>(), integral_constant<int, 2>())
                                                        : pick(j(), integral_constant<int, 512>(), integral_constant<int, 1>()));
            const cudaError_t r = allow_ring(reinterpret_cast<const void*>(kern));
            return r != cudaSuccess ? r : launch_pdl(kern, dim3(sh.blocks), dim3(sh.threads), sh.smem, st, a, sh.plan);
        });
    });
    return true;
}

}  // namespace e4b
