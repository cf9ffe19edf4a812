// The stretch between two expert layers in one pass over the residual stream:
//
//   f = the branch: a dense row, or the combine sum_j w_j rows[inv_perm[t,j]]
//   b = f rf (post_w + off),  rf = 1 / sqrt(mean f^2 + eps)     (b = f without post_w)
//   o = h + s g b             g = gate or sigmoid(gate), per token, channel or element
//   n = o ro (pre_w + off),   ro = 1 / sqrt(mean o^2 + eps)
//
// and its backward (do: the gradient that reaches o; m(.) the mean over the row):
//
//   do = grad_o + ro (u - o ro^2 m(u o)),  u = grad_n (pre_w + off);   grad_h = do
//   db = s g do;  dg = s do b (times g (1 - g) behind the sigmoid)
//   grad_f = rf (v - f rf^2 m(v f)),  v = db (post_w + off)
//   grad_post_w = sum_t db f rf,  grad_pre_w = sum_t grad_n o ro
//
// Bound by HBM over many tokens, by latency over a few: every row is read once and nothing
// between the two norms is stored.  Statistics, sums and everything between load and store are
// fp32; each output is rounded once (n comes from the unrounded o).  The backward keeps the
// channel gradients of a block's rows in registers; blocks leave one partial each and a second
// kernel adds them in block order (no atomics: the same bits every time).
//
// Two forms.  Here: rows straight into registers (8 elements a thread, a row per block, or per
// warp up to 256 elements), the next row's loads issued before the current row's reductions.
// It serves few rows (1 x 2048 with a combine of 8 rows: 6.2 us in a graph), the combine as
// branch, and tensors that start off a 16-byte boundary.  Long runs of rows take the rings of
// block_ring.cuh: 16384 x 4096 bf16 forward, 125 us here, 96 there (HBM floor 82); 8191 x 2880
// backward with an element gate, 199 here, 112 there (floor 58; bound by instructions and
// barriers: 53 instructions an element at 8192 x 4096, 16 warps an SM at 128 registers).
#include <algorithm>
#include <cmath>

#include "block_norm.cuh"

namespace e4b {

constexpr int kRowElems = 8;             // elements of a row per thread
constexpr int kForwardThreads = 1024;    // threads of rows at work per SM (64 registers each)
constexpr int kBackwardThreads = 512;    // and in the backward (128)

// BR: 0 no branch (norm of h alone), 1 a dense branch, 2 the combine of k rows.
template <typename E, int V, int NV, int BR>
__global__ void __launch_bounds__(1024) block_forward_kernel(const BlockArgs a, int tx) {
    using R = raw_t<E, V>;
    __shared__ RowSums<1> s_red[2];
    const int x = threadIdx.x % tx, ry = threadIdx.x / tx, rpb = blockDim.x / tx;
    const int64_t step = (int64_t)gridDim.x * rpb;
    pdl_release();
    pdl_wait();
    float pw[NV][V], nw[NV][V], cg[NV][V];
    load_channels<V, NV>(BR ? a.post_w : nullptr, a.offset, tx, x, a.nvec, pw);
    load_channels<V, NV>(a.pre_w, a.offset, tx, x, a.nvec, nw);
    const bool chan = BR && a.gate_kind == E4B_GATE_CHANNEL, elem = BR && a.gate_kind == E4B_GATE_ELEMENT;
    load_channels<V, NV>(chan ? static_cast<const float*>(a.gate) : nullptr, 0.0f, tx, x, a.nvec, cg);
    if (chan && a.gate_sigmoid) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) cg[i][j] = sigmoid<false>(cg[i][j]);
    }
    R rf[NV], rh[NV], rg[NV];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * tx + x;
            if (v >= a.nvec) continue;
            rh[i] = ld_once<R>(a.h, t * a.nvec + v);
            if (BR == 1) rf[i] = ld_once<R>(a.f, t * a.nvec + v);
            if (elem) rg[i] = ld_once<R>(a.gate, t * a.nvec + v);
        }
    };
    int64_t t = (int64_t)blockIdx.x * rpb + ry;
    if (t < a.T) fetch(t);
    for (; t < a.T; t += step) {
        float o[NV][V], f[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i) unpack<E, V>(rh[i], o[i]);
        if (BR) {
            float g[NV][V];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (BR == 1) unpack<E, V>(rf[i], f[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (BR == 2) f[i][j] = 0.0f;
                    g[i][j] = cg[i][j];
                }
                if (elem) unpack<E, V>(rg[i], g[i]);
            }
            if (BR == 2) {   // as combine_rows_kernel: fp32 in slot order, entries outside [0, P) add nothing
                const int64_t P = a.T * a.k;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = i * tx + x;
#pragma unroll
                    for (int j0 = 0; j0 < 8; j0 += 4) {
                        R raw[4];
                        float w[4];
                        bool in[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int64_t r = j0 + j < a.k ? __ldcg(a.inv_perm + t * a.k + j0 + j) : -1;
                            in[j] = r >= 0 && r < P && v < a.nvec;
                            if (in[j]) {
                                raw[j] = ld_once<R>(a.rows, r * a.nvec + v);
                                w[j] = a.topk_w ? __ldcg(a.topk_w + t * a.k + j0 + j) : 1.0f;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (!in[j]) continue;
                            float q[V];
                            unpack<E, V>(raw[j], q);
#pragma unroll
                            for (int c = 0; c < V; ++c) f[i][c] = fmaf(w[j], q[c], f[i][c]);
                        }
                    }
                    if (a.f_out && v < a.nvec) st_once<R>(a.f_out, t * a.nvec + v, pack<E, V>(f[i]));
                }
            }
            const int64_t next = t + step;
            if (next < a.T) fetch(next);
            float r = a.scale;
            if (a.gate_kind == E4B_GATE_TOKEN) {
                const float gt = __ldcg(static_cast<const float*>(a.gate) + t);
                r *= a.gate_sigmoid ? sigmoid<false>(gt) : gt;
            }
            if (a.post_w) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (i * tx + x < a.nvec) s[0] = fmaf(f[i][j], f[i][j], s[0]);
                row_sum<1>(s, tx, s_red[0]);
                r *= rsqrtf(s[0] / (float)a.H + a.eps);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * tx + x;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float gv = elem && a.gate_sigmoid ? sigmoid<kFastGate<E>>(g[i][j]) : g[i][j];
                    o[i][j] = fmaf(f[i][j] * pw[i][j] * gv, r, o[i][j]);
                }
                if (v < a.nvec) st_once<R>(a.o, t * a.nvec + v, pack<E, V>(o[i]));
            }
        } else {
            const int64_t next = t + step;
            if (next < a.T) fetch(next);
        }
        if (a.pre_w) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (i * tx + x < a.nvec) s[0] = fmaf(o[i][j], o[i][j], s[0]);
            // without a post-norm this is the row's only reduction: alternate over the rows
            row_sum<1>(s, tx, s_red[BR && a.post_w ? 1 : (int)((t / step) & 1)]);
            const float ro = rsqrtf(s[0] / (float)a.H + a.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * tx + x;
#pragma unroll
                for (int j = 0; j < V; ++j) o[i][j] *= ro * nw[i][j];
                if (v < a.nvec) st_once<R>(a.n, t * a.nvec + v, pack<E, V>(o[i]));
            }
        } else if (BR && a.post_w) {
            if (tx != 32) __syncthreads();   // s_red[0] is written again by the next row
        }
    }
}

template <typename E, int V, int NV, bool BR, int MAXT>
__global__ void __launch_bounds__(MAXT) block_backward_kernel(const BlockArgs a, int tx) {
    using R = raw_t<E, V>;
    __shared__ RowSums<3> s_red1;
    __shared__ RowSums<2> s_red2;
    const int x = threadIdx.x % tx, ry = threadIdx.x / tx, rpb = blockDim.x / tx;
    const int64_t step = (int64_t)gridDim.x * rpb;
    pdl_release();
    pdl_wait();
    const bool post = BR && a.post_w, pre = a.pre_w != nullptr;
    const bool chan = BR && a.gate_kind == E4B_GATE_CHANNEL, elem = BR && a.gate_kind == E4B_GATE_ELEMENT;
    const bool token = BR && a.gate_kind == E4B_GATE_TOKEN;
    float pw[NV][V], nw[NV][V], cg[NV][V];
    load_channels<V, NV>(post ? a.post_w : nullptr, a.offset, tx, x, a.nvec, pw);
    load_channels<V, NV>(a.pre_w, a.offset, tx, x, a.nvec, nw);
    load_channels<V, NV>(chan ? static_cast<const float*>(a.gate) : nullptr, 0.0f, tx, x, a.nvec, cg);
    float acc_post[NV][V], acc_pre[NV][V], acc_gate[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            acc_post[i][j] = acc_pre[i][j] = acc_gate[i][j] = 0.0f;
            if (chan && a.gate_sigmoid) cg[i][j] = sigmoid<false>(cg[i][j]);
        }
    const float inv_h = 1.0f / (float)a.H;
    R ro_[NV], rf_[NV], rgo[NV], rgn[NV], rg[NV];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * tx + x;
            if (v >= a.nvec) continue;
            const int64_t at = t * a.nvec + v;
            if (pre) {
                ro_[i] = ld_once<R>(a.o, at);
                rgn[i] = ld_once<R>(a.grad_n, at);
            }
            if (a.grad_o) rgo[i] = ld_once<R>(a.grad_o, at);
            if (BR) rf_[i] = ld_once<R>(a.f, at);
            if (elem) rg[i] = ld_once<R>(a.gate, at);
        }
    };
    int64_t t = (int64_t)blockIdx.x * rpb + ry;
    if (t < a.T) fetch(t);
    for (; t < a.T; t += step) {
        float o[NV][V], f[NV][V], d[NV][V], u[NV][V], g[NV][V];
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = i * tx + x < a.nvec;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[i][j] = f[i][j] = d[i][j] = u[i][j] = 0.0f;
                g[i][j] = cg[i][j];
            }
            if (in) {
                if (pre) {
                    unpack<E, V>(ro_[i], o[i]);
                    unpack<E, V>(rgn[i], u[i]);
                }
                if (a.grad_o) unpack<E, V>(rgo[i], d[i]);
                if (BR) unpack<E, V>(rf_[i], f[i]);
                if (elem) unpack<E, V>(rg[i], g[i]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[0] = fmaf(o[i][j], o[i][j], s[0]);
                s[1] = fmaf(u[i][j] * nw[i][j], o[i][j], s[1]);
                if (BR) s[2] = fmaf(f[i][j], f[i][j], s[2]);
            }
        }
        const int64_t next = t + step;
        if (next < a.T) fetch(next);
        float gt = 1.0f, slope = 1.0f;
        if (token) {
            gt = __ldcg(static_cast<const float*>(a.gate) + t);
            if (a.gate_sigmoid) logistic<false>(gt, gt, slope);
        }
        row_sum<3>(s, tx, s_red1);
        const float ro = rsqrtf(s[0] * inv_h + a.eps), rf = post ? rsqrtf(s[2] * inv_h + a.eps) : 1.0f;
        const float co = ro * ro * s[1] * inv_h;
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * tx + x;
            const bool in = v < a.nvec;
            if (pre) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    acc_pre[i][j] = fmaf(u[i][j] * o[i][j], ro, acc_pre[i][j]);
                    d[i][j] = fmaf(ro, u[i][j] * nw[i][j] - o[i][j] * co, d[i][j]);
                }
            }
            if (a.grad_h && in) st_once<R>(a.grad_h, t * a.nvec + v, pack<E, V>(d[i]));
            if constexpr (BR) {
                float ge[V];
    #pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float db = a.scale * d[i][j], b = f[i][j] * rf * pw[i][j];
                    float gv = g[i][j], gd = 1.0f;
                    if (elem && a.gate_sigmoid) logistic<kFastGate<E>>(gv, gv, gd);
                    ge[j] = db * b * gd;   // a channel's or token's g (1 - g) multiplies the sum
                    if (chan) acc_gate[i][j] += ge[j];
                    if (token) q[1] = fmaf(db, b, q[1]);
                    const float v1 = db * (token ? gt : gv);   // the gradient of b
                    acc_post[i][j] = fmaf(v1 * f[i][j], rf, acc_post[i][j]);
                    d[i][j] = v1 * pw[i][j];
                    q[0] = fmaf(d[i][j], f[i][j], q[0]);
                }
                if (elem && a.grad_gate && in) st_once<R>(a.grad_gate, t * a.nvec + v, pack<E, V>(ge));
            }
        }
        if (BR) {
            row_sum<2>(q, tx, s_red2);   // this barrier also frees s_red1 for the next row
            const float cf = post ? rf * rf * q[0] * inv_h : 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * tx + x;
#pragma unroll
                for (int j = 0; j < V; ++j) d[i][j] = rf * (d[i][j] - f[i][j] * cf);
                if (a.grad_f && v < a.nvec) st_once<R>(a.grad_f, t * a.nvec + v, pack<E, V>(d[i]));
            }
            if (token && a.grad_gate && x == 0)
                static_cast<float*>(a.grad_gate)[t] = q[1] * slope;
        } else if (tx != 32) {
            __syncthreads();
        }
    }
    if (!a.partials) return;
    float* part = a.partials + ((int64_t)blockIdx.x * rpb + ry) * 3 * a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * tx + x;
        if (v >= a.nvec) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (a.want_post) __stcg(part + v * V + j, acc_post[i][j]);
            if (a.want_pre) __stcg(part + a.H + v * V + j, acc_pre[i][j]);
            if (a.want_cgate) __stcg(part + 2 * a.H + v * V + j, acc_gate[i][j]);
        }
    }
}


// out[c] = sum over the parts, in part order within each of the block's 32 threads of a
// column and then in thread order.  blockIdx.y: post_w, pre_w or channel gate, whose sum is of
// db b: times g (1 - g) of `sigmoid_gate` (null: the gate is no logistic function).
__global__ void __launch_bounds__(1024) channel_sum_kernel(const float* __restrict__ partials, int parts, int H,
                                                           float* post, float* pre, float* gate,
                                                           const float* __restrict__ sigmoid_gate) {
    __shared__ float s[32][33];
    pdl_release();
    pdl_wait();
    float* out = blockIdx.y == 0 ? post : blockIdx.y == 1 ? pre : gate;
    if (!out) return;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float sum = 0.0f;
    if (c < H) {
#pragma unroll 4
        for (int p = y; p < parts; p += 32) sum += __ldcg(partials + ((int64_t)p * 3 + blockIdx.y) * H + c);
    }
    s[y][x] = sum;
    __syncthreads();
    if (y == 0 && c < H) {
        float r = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) r += s[i][x];
        if (blockIdx.y == 2 && sigmoid_gate) {
            float g, slope;
            logistic<false>(__ldcg(sigmoid_gate + c), g, slope);
            r *= slope;
        }
        out[c] = r;
    }
}

// ------------------------------------------------------------------ host side

struct BlockShape {
    int tx, threads, rpb;   // threads per row and block, rows per block
    explicit BlockShape(int H) {
        tx = ((H + kRowElems - 1) / kRowElems + 31) / 32 * 32;
        threads = tx == 32 ? 256 : tx;
        rpb = threads / tx;
    }
    // rows of `per_sm` threads in flight on every SM
    int blocks(int64_t T, int per_sm) const {
        return (int)std::min<int64_t>((T + rpb - 1) / rpb, (int64_t)num_sms() * std::max(1, per_sm / threads));
    }
};

template <typename F>
static cudaError_t with_row_shape(e4b_dtype dt, int bytes, F f) {
    if (dt == E4B_BF16) {
        if (bytes == 16) return f((__nv_bfloat16*)nullptr, std::integral_constant<int, 8>());
        if (bytes == 4) return f((__nv_bfloat16*)nullptr, std::integral_constant<int, 2>());
        return f((__nv_bfloat16*)nullptr, std::integral_constant<int, 1>());
    }
    if (bytes == 16) return f((float*)nullptr, std::integral_constant<int, 4>());
    return f((float*)nullptr, std::integral_constant<int, 1>());
}

static e4b_status check_block(const e4b_block_desc* d, int64_t T, const void* gate) {
    if (!d || T < 0 || d->H < 1) return E4B_ERR_INVALID_ARG;
    if (d->H > kMaxRow) return E4B_ERR_UNSUPPORTED;
    if (T > INT64_MAX / (8 * kMaxRow)) return E4B_ERR_INVALID_ARG;   // byte offsets of rows in 64 bits
    if (d->dtype != E4B_F32 && d->dtype != E4B_BF16) return E4B_ERR_INVALID_ARG;
    if (!(d->eps >= 0.0f) || !std::isfinite(d->eps) || !std::isfinite(d->weight_offset) ||
        !std::isfinite(d->residual_scale))
        return E4B_ERR_INVALID_ARG;
    if (d->gate < E4B_GATE_NONE || d->gate > E4B_GATE_ELEMENT) return E4B_ERR_INVALID_ARG;
    if (T > 0 && (d->gate != E4B_GATE_NONE) != (gate != nullptr)) return E4B_ERR_INVALID_ARG;
    return E4B_OK;
}

static BlockArgs base_args(const e4b_block_desc* d, int64_t T) {
    BlockArgs a{};
    a.T = T;
    a.H = d->H;
    a.gate_kind = d->gate;
    a.gate_sigmoid = d->gate_sigmoid != 0 && d->gate != E4B_GATE_NONE;
    a.eps = d->eps;
    a.offset = d->weight_offset;
    a.scale = d->residual_scale;
    a.status = device_status_ptr();
    return a;
}

// Partials that a backward of T tokens may leave: one per row in flight.
static int64_t backward_parts(const e4b_block_desc* d, int64_t T) {
    const BlockShape sh(d->H);
    return std::max<int64_t>((int64_t)sh.blocks(T, kBackwardThreads) * sh.rpb, block_ring_parts(d->H, T));
}

}  // namespace e4b

using namespace e4b;

extern "C" {

e4b_status e4b_block_norm_forward(const e4b_block_desc* d, const e4b_block_branch* br, const void* h, int64_t T,
                                  const float* post_w, const void* gate, const float* pre_w, void* f_out, void* o,
                                  void* n, void* stream) {
    NvtxScope nvtx_scope("e4b_block_norm_forward");
    e4b_status s = check_block(d, T, gate);
    if (s != E4B_OK) return s;
    const bool dense = br && br->f, gather = br && br->rows;
    if (dense && gather) return E4B_ERR_INVALID_ARG;
    if (T == 0) return E4B_OK;
    const bool branch = dense || gather;
    if (gather && (br->top_k < 1 || br->top_k > 8 || !br->inv_perm || too_many_pairs(T, br->top_k)))
        return E4B_ERR_INVALID_ARG;
    if (!h || (pre_w != nullptr) != (n != nullptr) || branch != (o != nullptr) || (!branch && !pre_w))
        return E4B_ERR_INVALID_ARG;
    if (!branch && (post_w || gate)) return E4B_ERR_INVALID_ARG;
    if (f_out && !gather) return E4B_ERR_INVALID_ARG;
    if (off_boundary(4, {post_w, pre_w, d->gate == E4B_GATE_ELEMENT ? nullptr : gate}) ||
        (gather && off_boundary(4, {br->inv_perm, br->topk_w})))
        return E4B_ERR_INVALID_ARG;
    BlockArgs a = base_args(d, T);
    a.h = h;
    a.gate = gate;
    a.post_w = post_w;
    a.pre_w = pre_w;
    a.f_out = f_out;
    a.o = o;
    a.n = n;
    if (dense) a.f = br->f;
    if (gather) {
        a.rows = br->rows;
        a.inv_perm = br->inv_perm;
        a.topk_w = br->topk_w;
        a.k = br->top_k;
    }
    const int es = d->dtype == E4B_BF16 ? 2 : 4;
    const int vb = row_vector_bytes((int64_t)d->H * es, es,
                                    {h, a.f, a.rows, f_out, o, n, d->gate == E4B_GATE_ELEMENT ? gate : nullptr});
    const bool vb16 = !off_boundary(16, {h, a.f, o, n, d->gate == E4B_GATE_ELEMENT ? gate : nullptr});
    if (!vb) return E4B_ERR_INVALID_ARG;
    const BlockShape sh(d->H);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (vb16 && !gather && block_ring_forward(d->dtype, dense, a, st, &err)) return err == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
    err = with_row_shape(d->dtype, vb, [&](auto* e, auto v) {
        using E = std::remove_pointer_t<decltype(e)>;
        constexpr int V = decltype(v)::value;
        a.nvec = d->H / V;
        auto kern = gather ? block_forward_kernel<E, V, kRowElems / V, 2>
                    : dense ? block_forward_kernel<E, V, kRowElems / V, 1> : block_forward_kernel<E, V, kRowElems / V, 0>;
        return launch_pdl(kern, dim3(sh.blocks(T, kForwardThreads)), dim3(sh.threads), 0, st, a, sh.tx);
    });
    return err == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

size_t e4b_block_norm_workspace_size(const e4b_block_desc* d, int64_t T) {
    if (!d || d->H < 1 || d->H > kMaxRow || T < 0) return 0;
    return (size_t)backward_parts(d, T) * 3 * d->H * 4;
}

e4b_status e4b_block_norm_backward(const e4b_block_desc* d, const void* o, const void* f, int64_t T, const float* post_w,
                                   const void* gate, const float* pre_w, const void* grad_o, const void* grad_n,
                                   void* grad_h, void* grad_f, float* grad_post_w, void* grad_gate, float* grad_pre_w,
                                   void* workspace, size_t ws_bytes, void* stream) {
    NvtxScope nvtx_scope("e4b_block_norm_backward");
    e4b_status s = check_block(d, T, gate);
    if (s != E4B_OK) return s;
    if ((pre_w == nullptr && (grad_n || grad_pre_w)) || (!post_w && grad_post_w) || (!gate && grad_gate && T > 0))
        return E4B_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // no tokens: the channel gradients are zero
        float* chan = d->gate == E4B_GATE_CHANNEL ? static_cast<float*>(grad_gate) : nullptr;
        for (float* p : {grad_post_w, grad_pre_w, chan})
            if (p && cudaMemsetAsync(p, 0, (size_t)d->H * 4, st) != cudaSuccess) return E4B_ERR_CUDA;
        return E4B_OK;
    }
    if (pre_w ? (!o || !grad_n) : !grad_o) return E4B_ERR_INVALID_ARG;
    if (!f && (post_w || gate || grad_f)) return E4B_ERR_INVALID_ARG;
    const bool chan = d->gate == E4B_GATE_CHANNEL && grad_gate;
    const bool sums = grad_post_w || grad_pre_w || chan;
    if (!grad_h && !grad_f && !grad_gate && !sums) return E4B_ERR_INVALID_ARG;
    if (sums && (!workspace || ws_bytes < e4b_block_norm_workspace_size(d, T))) return E4B_ERR_WORKSPACE;
    const bool elem = d->gate == E4B_GATE_ELEMENT;
    if ((sums && off_boundary(16, {workspace})) || off_boundary(4, {post_w, pre_w, grad_post_w, grad_pre_w}) ||
        (!elem && off_boundary(4, {gate, grad_gate})))
        return E4B_ERR_INVALID_ARG;
    BlockArgs a = base_args(d, T);
    a.o = const_cast<void*>(o);
    a.f = f;
    a.gate = gate;
    a.post_w = post_w;
    a.pre_w = pre_w;
    a.grad_o = grad_o;
    a.grad_n = grad_n;
    a.grad_h = grad_h;
    a.grad_f = grad_f;
    a.grad_gate = grad_gate;
    a.partials = sums ? static_cast<float*>(workspace) : nullptr;
    a.want_post = grad_post_w != nullptr;
    a.want_pre = grad_pre_w != nullptr;
    a.want_cgate = chan;
    const int es = d->dtype == E4B_BF16 ? 2 : 4;
    const int vb = row_vector_bytes((int64_t)d->H * es, es,
                                    {pre_w ? o : nullptr, f, grad_o, grad_n, grad_h, grad_f, elem ? gate : nullptr,
                                     elem ? grad_gate : nullptr});
    const bool vb16 = !off_boundary(16, {pre_w ? o : nullptr, f, grad_o, grad_n, grad_h, grad_f, elem ? gate : nullptr,
                                         elem ? grad_gate : nullptr});
    if (!vb) return E4B_ERR_INVALID_ARG;
    const BlockShape sh(d->H);
    int parts = sh.blocks(T, kBackwardThreads) * sh.rpb;
    cudaError_t err = cudaSuccess;
    const bool ring = vb16 && block_ring_backward(d->dtype, f != nullptr, a, &parts, st, &err);
    if (!ring) err = with_row_shape(d->dtype, vb, [&](auto* e, auto v) {
        using E = std::remove_pointer_t<decltype(e)>;
        constexpr int V = decltype(v)::value;
        a.nvec = d->H / V;
        auto kern = sh.threads <= 512
                        ? (f ? block_backward_kernel<E, V, kRowElems / V, true, 512>
                             : block_backward_kernel<E, V, kRowElems / V, false, 512>)
                        : (f ? block_backward_kernel<E, V, kRowElems / V, true, 1024>
                             : block_backward_kernel<E, V, kRowElems / V, false, 1024>);
        return launch_pdl(kern, dim3(sh.blocks(T, kBackwardThreads)), dim3(sh.threads), 0, st, a, sh.tx);
    });
    if (err == cudaSuccess && sums)
        err = launch_pdl(channel_sum_kernel, dim3((d->H + 31) / 32, 3), dim3(1024), 0, st, (const float*)a.partials,
                         parts, d->H, grad_post_w, grad_pre_w,
                         chan ? static_cast<float*>(grad_gate) : nullptr,
                         a.gate_sigmoid ? static_cast<const float*>(gate) : nullptr);
    return err == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

}  // extern "C"
