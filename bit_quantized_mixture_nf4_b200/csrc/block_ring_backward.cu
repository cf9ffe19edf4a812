// Block norm backward over long runs of rows (the formulas are in block_norm.cu, the ring in
// block_ring.cuh).
#include "block_ring.cuh"

namespace e4b {
namespace {

constexpr int kThreads = 512;   // of rows at work per SM (128 registers each)

// FULL: every optional part is there (both norms, grad_o), known at compile time: the conditions
// on them cost as many instructions as the arithmetic (register moves where their sides meet).
template <typename E, int V, int NV, bool BR, int GK, bool FULL, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) block_backward_ring_kernel(const BlockArgs a, const RingPlan pl) {
    using R = raw_t<E, V>;
    constexpr bool ALIGNED = V * sizeof(E) == 16;
    constexpr bool chan = BR && GK == E4B_GATE_CHANNEL, elem = BR && GK == E4B_GATE_ELEMENT;
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ uint64_t s_full[kRingGroups][kRingStages];
    __shared__ int s_abort;
    __shared__ RowSums<3> s_red1;
    __shared__ RowSums<2> s_red2;
    const bool post = BR && (FULL || a.post_w), pre = FULL || a.pre_w, has_go = FULL || a.grad_o;
    const bool token = BR && !chan && !elem && a.gate_kind == E4B_GATE_TOKEN;
    RowRing ring;
    const int64_t first = ring_setup<E>(ring, a, pl, BR + elem + 2 * pre + has_go, dsm, s_full, s_abort);
    // the row's arrays: [o, grad_n], [f], [gate], [grad_o]
    const int sb = pl.slot_bytes, row_bytes = a.H * (int)sizeof(E);
    const int at_f = pre ? 2 * sb : 0, at_g = at_f + (BR ? sb : 0), at_go = at_g + (elem ? sb : 0);
    if (pre) {
        ring_source(ring, 0, a.o);
        ring_source(ring, 1, a.grad_n);
    }
    if (BR) ring_source(ring, 2 * pre, a.f);
    if (elem) ring_source(ring, 2 * pre + 1, a.gate);
    if (has_go) ring_source(ring, 2 * pre + BR + elem, a.grad_o);
    const int tx = pl.tx, x = threadIdx.x % tx, ry = threadIdx.x / tx, rpb = blockDim.x / tx;
    if (x == 0)
        for (int i = 0; i < pl.stages; ++i) ring.issue<E, ALIGNED>();
    float pw[NV][V], nw[NV][V], cg[NV][V];
    load_channels<V, NV>(post ? a.post_w : nullptr, a.offset, tx, x, a.nvec, pw);
    load_channels<V, NV>(a.pre_w, a.offset, tx, x, a.nvec, nw);
    if (chan) load_channels<V, NV>(static_cast<const float*>(a.gate), 0.0f, tx, x, a.nvec, cg);
    // with a channel gate acc_post holds sum db f rf, which both channel gradients are multiples of
    float acc_post[NV][V], acc_pre[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            acc_post[i][j] = acc_pre[i][j] = 0.0f;
            if (chan && a.gate_sigmoid) cg[i][j] = sigmoid<false>(cg[i][j]);
        }
    const float inv_h = 1.0f / (float)a.H;
    const float* gates = static_cast<const float*>(a.gate);
    float gt_next = token && first * pl.rows < a.T ? __ldcg(gates + first * pl.rows) : 1.0f;   // one row ahead
    for (int64_t u = first; u < ring.units; u += ring.step) {
        const uint8_t* row = ring.wait<ALIGNED>(u);
        const int64_t t0 = u * pl.rows, t1 = min(a.T, t0 + pl.rows);
        for (int64_t t = t0; t < t1; ++t, row += row_bytes) {
            float gt = gt_next, slope = 1.0f;
            if (token) {
                const int64_t next = t + 1 < t1 ? t + 1 : (u + ring.step) * pl.rows;
                if (next < a.T) gt_next = __ldcg(gates + next);
                if (a.gate_sigmoid) logistic<false>(gt, gt, slope);
            }
            const int64_t at = t * a.nvec;
            float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int v = q * tx + x;
                if (pre) {
                    float o[V], gn[V];
                    read_row<E, V>(row, v, a.nvec, o);
                    read_row<E, V>(row + sb, v, a.nvec, gn);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        s[0] = fmaf(o[j], o[j], s[0]);
                        s[1] = fmaf(gn[j] * nw[q][j], o[j], s[1]);
                    }
                }
                if (post) {
                    float f[V];
                    read_row<E, V>(row + at_f, v, a.nvec, f);
#pragma unroll
                    for (int j = 0; j < V; ++j) s[2] = fmaf(f[j], f[j], s[2]);
                }
            }
            row_sum<3>(s, tx, s_red1);
            const float ro = rsqrtf(s[0] * inv_h + a.eps), rf = post ? rsqrtf(s[2] * inv_h + a.eps) : 1.0f;
            const float co = ro * (ro * s[1] * inv_h * ro), srf = a.scale * rf;
            // rf v, v = db (post_w + off), is what stays of the row: grad_f = rf v - f rf^2 m(rf v f)
            float q2[2] = {0.0f, 0.0f};
            float d[NV][V];
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int v = q * tx + x;
                if (has_go) {
                    read_row<E, V>(row + at_go, v, a.nvec, d[q]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) d[q][j] = 0.0f;
                }
                if (pre) {
                    float o[V], gn[V];
                    read_row<E, V>(row, v, a.nvec, o);
                    read_row<E, V>(row + sb, v, a.nvec, gn);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float ur = gn[j] * ro;
                        acc_pre[q][j] = fmaf(ur, o[j], acc_pre[q][j]);
                        d[q][j] = fmaf(ur, nw[q][j], fmaf(-co, o[j], d[q][j]));
                    }
                }
                if (a.grad_h && v < a.nvec) st_once<R>(a.grad_h, at + v, pack<E, V>(d[q]));
                if constexpr (BR) {
                    float f[V], g[V];
                    read_row<E, V>(row + at_f, v, a.nvec, f);
                    if (elem) read_row<E, V>(row + at_g, v, a.nvec, g);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float db = d[q][j] * srf, dfr = db * f[j];
                        float gv = chan ? cg[q][j] : gt;
                        if (elem) {
                            float gd = 1.0f;
                            gv = g[j];
                            if (a.gate_sigmoid) logistic<kFastGate<E>>(gv, gv, gd);
                            g[j] = dfr * pw[q][j] * gd;
                        }
                        if (token) q2[1] = fmaf(dfr, pw[q][j], q2[1]);
                        acc_post[q][j] = chan ? acc_post[q][j] + dfr : fmaf(dfr, gv, acc_post[q][j]);
                        d[q][j] = db * gv * pw[q][j];
                        q2[0] = fmaf(d[q][j], f[j], q2[0]);
                    }
                    if (elem && a.grad_gate && v < a.nvec) st_once<R>(a.grad_gate, at + v, pack<E, V>(g));
                }
            }
            if constexpr (BR) {
                row_sum<2>(q2, tx, s_red2);
                const float cf = post ? rf * (q2[0] * inv_h) * rf : 0.0f;
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    const int v = q * tx + x;
                    if (post) {
                        float f[V];
                        read_row<E, V>(row + at_f, v, a.nvec, f);
#pragma unroll
                        for (int j = 0; j < V; ++j) d[q][j] = fmaf(-cf, f[j], d[q][j]);
                    }
                    if (a.grad_f && v < a.nvec) st_once<R>(a.grad_f, at + v, pack<E, V>(d[q]));
                }
                if (token && a.grad_gate && x == 0)
                    static_cast<float*>(a.grad_gate)[t] = q2[1] * slope;
            }
        }
        if (tx == 32) __syncwarp();   // behind the slot's last reads
        else __syncthreads();
        if (x == 0) ring.issue<E, ALIGNED>();
        ring.advance();
    }
    if (!a.partials) return;
    // one partial per block: its groups are added in order through shared memory (behind a barrier;
    // nothing that a group requested is in flight any more)
    float* part = a.partials + (int64_t)blockIdx.x * 3 * a.H;
    float* sums = reinterpret_cast<float*>(dsm);
    const bool want[3] = {a.want_post != 0, a.want_pre != 0, chan && a.want_cgate};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (!want[k]) continue;
        for (int g = 0; g < rpb; ++g) {
            if (rpb > 1) __syncthreads();
            if (ry != g) continue;
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int v = q * tx + x;
                if (v >= a.nvec) continue;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float s = k == 1 ? acc_pre[q][j] : acc_post[q][j];
                    if (chan && k == 0) s *= cg[q][j];
                    if (chan && k == 2) s *= pw[q][j];   // times g (1 - g) where the partials are added
                    if (g > 0) s += sums[v * V + j];
                    if (g + 1 < rpb) sums[v * V + j] = s;
                    else __stcg(part + k * a.H + v * V + j, s);
                }
            }
        }
    }
}

}  // namespace

int64_t block_ring_parts(int H, int64_t T) {
    (void)H;   // one per block
    return std::min<int64_t>(T, (int64_t)num_sms() * (kThreads / 32));
}

bool block_ring_backward(e4b_dtype dt, bool branch, const BlockArgs& args, int* parts, cudaStream_t st, cudaError_t* err) {
    BlockArgs a = args;
    const int es = dt == E4B_BF16 ? 2 : 4;
    const int arrays = branch + (branch && a.gate_kind == E4B_GATE_ELEMENT) + 2 * (a.pre_w != nullptr) + (a.grad_o != nullptr);
    // 16 elements a thread for long bf16 rows, and for all that would take over 512 threads
    // (16384 x 2048 bf16: 105 us against 134; 8192 x 2048 fp32: 116 against 71)
    const bool wide = (int64_t)a.H * es % 16 == 0;
    const int elems = (wide && es == 2 && a.H >= 1024) || a.H > 4096 ? 16 : 8;
    const RingShape sh(a.H, es, arrays, a.T, elems, kThreads);
    if (!sh.fits) return false;
    *parts = sh.blocks;
    *err = with_ring_vector(dt, a.H, [&](auto* e, auto vv) {
        using E = std::remove_pointer_t<decltype(e)>;
        constexpr int V = decltype(vv)::value;
        a.nvec = a.H / V;
        return with_gate(a.gate_kind, [&](auto gk) {
            constexpr int G = decltype(gk)::value;
            auto pick = [&](auto elems, auto maxt, auto minb) {
                constexpr int NV = decltype(elems)::value / V, MT = decltype(maxt)::value, MB = decltype(minb)::value;
                constexpr bool WIDE = V * sizeof(E) == 16;   // narrow rows keep the general instances
                const bool full = WIDE && a.pre_w && a.grad_o && (!branch || a.post_w);
                if (!branch)
                    return full ? block_backward_ring_kernel<E, V, NV, false, E4B_GATE_NONE, WIDE, MT, MB>
                                : block_backward_ring_kernel<E, V, NV, false, E4B_GATE_NONE, false, MT, MB>;
                return full ? block_backward_ring_kernel<E, V, NV, true, G, WIDE, MT, MB>
                            : block_backward_ring_kernel<E, V, NV, true, G, false, MT, MB>;
            };
            using std::integral_constant;
            using i = std::integral_constant<int, 8>;
            using j = std::integral_constant<int, 16>;
            auto kern = elems == 8 ? (sh.threads <= 256 ? pick(i(), integral_constant<int, 256>(), integral_constant<int, 2>())
                                                        : pick(i(), integral_constant<int, 512>(), integral_constant<int, 1>()))
                                   : (sh.threads <= 256 ? pick(j(), integral_constant<int, 256>(), integral_constant<int, 2>())
                                                        : pick(j(), integral_constant<int, 512>(), integral_constant<int, 1>()));
            const cudaError_t r = allow_ring(reinterpret_cast<const void*>(kern));
            return r != cudaSuccess ? r : launch_pdl(kern, dim3(sh.blocks), dim3(sh.threads), sh.smem, st, a, sh.plan);
        });
    });
    return true;
}

}  // namespace e4b
