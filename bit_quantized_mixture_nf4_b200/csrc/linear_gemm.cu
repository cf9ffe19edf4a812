// The quantized linear on the 5th-generation tensor cores (tcgen05, TMEM accumulators).
//
//   forward   D = X_e W_e^T;  z = D + b_e;  y = residual + act(z), saved = act'(z)
//   backward  D = dZ_e W_e;   grad_x = D
// for the rows of expert e (one expert: a dense linear), W_e stored [out, in] in a 4-bit
// format or bf16.  The pipeline is the expert layer's (grouped_gemm.cu): 256-row tiles on
// CTA pairs, 256 columns, 64-deep k-stages; weights come in packed, are decoded to bf16 by
// six warps into the operand's swizzled shared-memory layout and meet the rows that TMA
// brings in.  Bound by the decoding chain and the issuing thread, not by HBM: 16384 x 14336
// by 4096 (backward, NF4) takes 1.50 ms alone, 1280 TFLOP/s, and 1.77 ms (1090) in a row of
// calls; 32768 rows over 64 experts of 2048 by 1024 take 167 us, 820 TFLOP/s, and 207 us with
// GELU and its derivative stored.  What is its own:
//   * the epilogue: bias, activation and its derivative on the accumulator in registers;
//     the residual's 32 x 32 chunk arrives by TMA while the previous chunk is finished,
//     is added in place in shared memory and leaves as y;
//   * K split over CTA pairs where a dense product has too few tiles to fill the GPU
//     (fp32 partial sums, added in a fixed order by a finishing kernel with the epilogue):
//     2880 by 2880, 96 rows, 31.2 us unsplit, 18.3 in 6 parts; 512 rows, 33.6 and 24.3;
//     1024 rows (one part by the rule), 34.
#include <mutex>

#include "linear.h"
#include "rowops.cuh"

namespace e4b {
namespace {

constexpr int BN = 256, BK = 64, CTAS = 2;
constexpr int THREADS = 512;
constexpr int A_WARP = 4, MMA_WARP = 5, RAW_WARP = 6, DEQ_WARP0 = 8;
constexpr int TMEM_COLS = 2 * BN;   // two accumulator buffers
constexpr int TILE_M = 128 * CTAS, N_CTA = BN / CTAS;
constexpr int A_BYTES = 128 * BK * 2, B_BYTES = N_CTA * BK * 2;
constexpr int RAW_BYTES = N_CTA * BK / 2, RAW_STAGE = RAW_BYTES + N_CTA * 4;
constexpr int ASTAGES = 6, STAGES = 4;
constexpr int RSTAGES = 6;   // the packed ring gives its last stages' room to the epilogue's buffers
constexpr int DEQ_GROUPS = 3, DEQ_GROUP_WARPS = 2, TPG = 32 * DEQ_GROUP_WARPS;
constexpr int BLOCKS_PER_THREAD = N_CTA / TPG;
static_assert(STAGES >= DEQ_GROUPS && RSTAGES >= DEQ_GROUPS, "a ring slot per decoding group");
constexpr int BUF = 2048, WARP_BUFS = 4;   // per epilogue warp: two (y, saved) pairs of 32 x 32 bf16
constexpr int RINGS = ASTAGES * A_BYTES + STAGES * B_BYTES + RSTAGES * RAW_STAGE;
constexpr int SMEM = RINGS + 1024 + 4 * WARP_BUFS * BUF + 1024;
static_assert(RINGS % 1024 == 0 && SMEM <= 232448, "shared memory per block");

struct Ctl {
    uint64_t a_full[ASTAGES], a_empty[ASTAGES];
    uint64_t b_full[STAGES], b_empty[STAGES];
    uint64_t raw_full[RSTAGES], raw_empty[RSTAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t res_full[4][2];   // residual chunk landed (per epilogue warp and buffer pair)
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Ctl) <= 1024, "control block");

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct Tile {
    int e, row0, rows, nt, k0, k1;   // k0, k1: the item's k-stages
};

constexpr int kTileGroup = 16;   // n-tiles that share their m-tiles' rows, as in the expert layer

// Work item -> tile and part of K.
__device__ __forceinline__ Tile decode_item(const LinearGemm& p, int item, int nk) {
    Tile t;
    const int tile = item / p.splits, part = item - tile * p.splits;
    t.k0 = (int)((int64_t)part * nk / p.splits);
    t.k1 = (int)((int64_t)(part + 1) * nk / p.splits);
    const int n = p.n_tiles;
    int m0 = 0, me;
    if (p.tile_prefix) {
        const int mt = tile / n;   // locates the expert: the last one whose first m-tile is at or before mt
        int lo = 0, hi = p.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.tile_prefix[mid] <= mt) lo = mid;
            else hi = mid;
        }
        m0 = p.tile_prefix[lo];
        me = p.tile_prefix[lo + 1] - m0;
    } else {
        me = (int)((p.P + TILE_M - 1) / TILE_M);
    }
    const int l = tile - m0 * n, g = min(kTileGroup, n), full = n / g;
    int m;
    if (l < full * g * me) {
        const int grp = l / (g * me), r = l - grp * g * me;
        m = r / g;
        t.nt = grp * g + (r - m * g);
    } else {
        const int gw = n - full * g, r = l - full * g * me;
        m = r / gw;
        t.nt = full * g + (r - m * gw);
    }
    if (p.tile_prefix) {
        const int4 v = p.sched[m0 + m];
        t.e = v.x;
        t.row0 = v.y;
        t.rows = v.z;
    } else {
        t.e = 0;
        t.row0 = m * TILE_M;
        t.rows = (int)min((int64_t)TILE_M, p.P - t.row0);
    }
    return t;
}

// Block b (0..N_CTA-1) of this CTA's B half at k-stage 0: its stored row (within the
// stack) and 64-column block, or row -1 outside the stored matrix.
//   forward (K-major): B column rank*N_CTA + b, k-block ks;  backward (MN-major): k-row
//   b & 63 of the stage, column block b >> 6 of the CTA's half
template <bool FWD>
__device__ __forceinline__ int64_t block_row(const LinearGemm& p, const Tile& t, int b, int rank, int& blk) {
    int64_t row;
    if (FWD) {
        row = (int64_t)t.e * p.b_rows_per_expert + t.nt * BN + rank * N_CTA + b;
        blk = 0;
    } else {
        row = (int64_t)t.e * p.b_rows_per_expert + (b & 63);
        blk = (t.nt * BN + rank * N_CTA) / 64 + (b >> 6);
        if (blk >= p.b_blocks_per_row) return -1;
    }
    return row < p.b_rows_total ? row : -1;
}

// FWD: the forward with its epilogue; else the input gradient.  CB: weight format.
// SPLIT: fp32 partial sums instead of the epilogue.
template <bool FWD, int CB, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
linear_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                   const __grid_constant__ CUtensorMap tmap_out, const __grid_constant__ CUtensorMap tmap_saved,
                   const __grid_constant__ CUtensorMap tmap_res, const LinearGemm p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + ASTAGES * A_BYTES;
    uint8_t* sRaw = sB + STAGES * B_BYTES;
    Ctl* ctl = reinterpret_cast<Ctl*>(sRaw + RSTAGES * RAW_STAGE);
    uint8_t* sBuf = reinterpret_cast<uint8_t*>(ctl) + 1024;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster_id = blockIdx.x / CTAS, nclusters = gridDim.x / CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ASTAGES; ++s) {
            mbar_init(smem_u32(&ctl->a_full[s]), 1);
            mbar_init(smem_u32(&ctl->a_empty[s]), 1);
        }
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&ctl->b_full[s]), DEQ_GROUP_WARPS * CTAS);
            mbar_init(smem_u32(&ctl->b_empty[s]), 1);
        }
        for (int s = 0; s < RSTAGES; ++s) {
            mbar_init(smem_u32(&ctl->raw_full[s]), 1 + 32);   // TMA + the warp's scale copies
            mbar_init(smem_u32(&ctl->raw_empty[s]), DEQ_GROUP_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctl->acc_full[b]), 1);
            mbar_init(smem_u32(&ctl->acc_empty[b]), 4 * CTAS);
            for (int w = 0; w < 4; ++w) mbar_init(smem_u32(&ctl->res_full[w][b]), 1);
        }
        ctl->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == MMA_WARP) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), TMEM_COLS);
        tmem_relinquish_pair();
    }
    if (warp == A_WARP && lane == 0) {
        tma_prefetch_desc(&tmap_a);
        tma_prefetch_desc(&tmap_w);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // the peer's barriers are initialised before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    volatile int* abort_flag = &ctl->abort_flag;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return mbar_wait(smem_u32(bar), parity, abort_flag, p.status);
    };
    auto arrive_leader = [&](uint64_t* bar) {
        if (!leader) mbar_arrive_cluster(mapa_shared(smem_u32(bar), 0));
        else mbar_arrive(smem_u32(bar));
    };
    pdl_wait();   // everything above touches this CTA's own memory only

    const int m_tiles = p.tile_prefix ? __ldcg(p.tile_prefix + p.E) : (int)((p.P + TILE_M - 1) / TILE_M);
    const int items = m_tiles * p.n_tiles * p.splits;
    const int nk = p.K / BK;

    if (warp == A_WARP) {
        // rows: TMA into a 6-stage ring, each box prefetched into L2 8 stages ahead
        if (lane == 0) {
            constexpr int APF = 8;
            const int a_off = 128 * rank;
            int pf_item = cluster_id, pf_ks = 0;
            Tile pf{};
            if (pf_item < items) {
                pf = decode_item(p, pf_item, nk);
                pf_ks = pf.k0;
            }
            auto prefetch_next = [&]() {
                if (pf_item >= items) return;
                tma_prefetch_l2_2d(&tmap_a, pf_ks * BK, pf.row0 + a_off);
                if (++pf_ks == pf.k1) {
                    pf_item += nclusters;
                    if (pf_item < items) {
                        pf = decode_item(p, pf_item, nk);
                        pf_ks = pf.k0;
                    }
                }
            };
            for (int i = 0; i < APF; ++i) prefetch_next();
            uint32_t it = 0;
            bool ok = true;
            for (int item = cluster_id; item < items && ok; item += nclusters) {
                const Tile t = decode_item(p, item, nk);
                for (int ks = t.k0; ks < t.k1; ++ks, ++it) {
                    prefetch_next();
                    const int s = it % ASTAGES;
                    if (!wait(&ctl->a_empty[s], ((it / ASTAGES) & 1) ^ 1)) { ok = false; break; }
                    if (leader) mbar_arrive_expect_tx(smem_u32(&ctl->a_full[s]), 2 * A_BYTES);
                    tma_load_2d_pair(smem_u32(sA + s * A_BYTES), &tmap_a, mapa_shared(smem_u32(&ctl->a_full[s]), 0),
                                     ks * BK, t.row0 + a_off);
                }
            }
        }
    } else if (warp == RAW_WARP) {
        // packed weights (TMA) and their block scales (cp.async by every lane)
        constexpr int PER_LANE = N_CTA / 32;
        uint32_t it = 0;
        for (int item = cluster_id; item < items; item += nclusters) {
            const Tile t = decode_item(p, item, nk);
            const int ebase = t.e * p.b_rows_per_expert;
            const uint8_t* src[PER_LANE];
            bool valid[PER_LANE];
#pragma unroll
            for (int i = 0; i < PER_LANE; ++i) {
                const int b = lane + 32 * i;
                int blk;
                const int64_t row = block_row<FWD>(p, t, b, rank, blk);
                valid[i] = row >= 0;
                if (CB == 2) {   // the 4 scale bytes that hold the block's two 32-element scales
                    const int64_t off = FWD ? row * p.mx_stride
                                            : row * p.mx_stride + (t.nt * BN + rank * N_CTA) / 32 + 4 * ((b >> 6) >> 1);
                    src[i] = p.mx_scales + (valid[i] ? off : 0);
                } else {
                    src[i] = reinterpret_cast<const uint8_t*>(p.absmax +
                                                              (valid[i] ? row * p.b_blocks_per_row + blk : 0));
                }
            }
            const int64_t step = CB == 2 ? (FWD ? 0 : (int64_t)BK * p.mx_stride)
                                         : 4 * (FWD ? 1 : (int64_t)BK * p.b_blocks_per_row);
            bool ok = true;
            for (int ks = t.k0; ks < t.k1; ++ks, ++it) {
                const int s = it % RSTAGES;
                if (lane == 0) ok = mbar_wait(smem_u32(&ctl->raw_empty[s]), ((it / RSTAGES) & 1) ^ 1, abort_flag, p.status);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const uint32_t rb = smem_u32(&ctl->raw_full[s]);
                if (CB == 3) {   // bf16 weights come straight into the operand ring
                    if (lane == 0) mbar_arrive(rb);
                    mbar_arrive(rb);
                    continue;
                }
                uint8_t* stage = sRaw + s * RAW_STAGE;
                if (lane == 0) {
                    mbar_arrive_expect_tx(rb, RAW_BYTES);
                    if (FWD)
                        tma_load_2d(smem_u32(stage), &tmap_w, rb, ks * (BK / 2), ebase + t.nt * BN + rank * N_CTA);
                    else
                        tma_load_2d(smem_u32(stage), &tmap_w, rb, (t.nt * BN + rank * N_CTA) / 2, ebase + ks * BK);
                }
                const uint32_t am = smem_u32(stage + RAW_BYTES) + 4u * lane;
#pragma unroll
                for (int i = 0; i < PER_LANE; ++i) {
                    const uint8_t* a = src[i] + ks * step + ((CB == 2 && FWD) ? 4 * (ks >> 1) : 0);
                    cp_async_4(am + 128u * i, valid[i] ? a : src[i], valid[i] ? 4u : 0u);
                }
                cp_async_mbar_arrive_noinc(rb);
            }
            if (!ok) break;
        }
    } else if (warp == MMA_WARP) {
        if (lane == 0 && leader) {
            constexpr uint32_t idesc = idesc_bf16(TILE_M, BN, FWD ? 0 : 1);
            uint32_t it = 0, lt = 0;
            bool ok = true;
            for (int item = cluster_id; item < items && ok; item += nclusters, ++lt) {
                const Tile t = decode_item(p, item, nk);
                const uint32_t ab = lt & 1;
                if (!wait(&ctl->acc_empty[ab], ((lt >> 1) & 1) ^ 1)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + ab * BN;
                for (int ks = t.k0; ks < t.k1; ++ks, ++it) {
                    const int s = it % STAGES, sa = it % ASTAGES;
                    if (!wait(&ctl->a_full[sa], (it / ASTAGES) & 1) || !wait(&ctl->b_full[s], (it / STAGES) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(sA + sa * A_BYTES), b_addr = smem_u32(sB + s * B_BYTES);
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        const uint64_t ad = smem_desc_sw128(a_addr + kk * 32, 16, 1024);
                        const uint64_t bd = FWD ? smem_desc_sw128(b_addr + kk * 32, 16, 1024)
                                                : smem_desc_sw128(b_addr + kk * 2048, 8192, 1024);
                        mma_bf16_ss_pair(d_tmem, ad, bd, idesc, ks != t.k0 || kk != 0);
                    }
                    mma_commit_pair(smem_u32(&ctl->b_empty[s]));
                    mma_commit_pair(smem_u32(&ctl->a_empty[sa]));
                }
                if (ok) mma_commit_pair(smem_u32(&ctl->acc_full[ab]));
            }
        }
    } else if (warp >= DEQ_WARP0 && (warp & 3) != (MMA_WARP & 3)) {
        // decoding: group g takes this CTA's k-stages g, g+3, ...; thread tg its blocks tg, tg + 64
        const int w8 = warp - DEQ_WARP0;
        const int dq = w8 - (w8 > (MMA_WARP & 3)) - (w8 > 4 + (MMA_WARP & 3));
        const int grp = dq / DEQ_GROUP_WARPS, tg = (dq % DEQ_GROUP_WARPS) * 32 + lane;
        uint32_t it = grp;
        int item = cluster_id, pos = grp;   // pos: stage within the item
        Tile t{};
        if (item < items) t = decode_item(p, item, nk);
        auto normalize = [&]() {   // carry pos past the end of an item into the next one(s)
            while (item < items && pos >= t.k1 - t.k0) {
                pos -= t.k1 - t.k0;
                item += nclusters;
                if (item < items) t = decode_item(p, item, nk);
            }
        };
        normalize();
        while (item < items) {
            const int s = it % STAGES, rs = it % RSTAGES;
            const uint32_t r = it / STAGES, rr = it / RSTAGES;
            const int cur_ks = t.k0 + pos;
            uint8_t* dst = sB + s * B_BYTES;
            if (!mbar_wait(smem_u32(&ctl->raw_full[rs]), rr & 1, abort_flag, p.status)) break;
            if (CB == 3) {
                // the group's first warp loads this CTA's part of the tile by TMA, completing on the
                // first CTA's barrier; the other warps only arrive
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->raw_empty[rs]));
                if (!wait(&ctl->b_empty[s], (r & 1) ^ 1)) break;
                if (lane == 0) {
                    const uint32_t bar = smem_u32(&ctl->b_full[s]);
                    if (tg == 0) {
                        if (leader) mbar_arrive_expect_tx(bar, CTAS * B_BYTES);
                        else mbar_arrive_cluster(mapa_shared(bar, 0));
                        const int ebase = t.e * p.b_rows_per_expert;
                        if (FWD) {
                            tma_load_2d_pair(smem_u32(dst), &tmap_w, mapa_shared(bar, 0), cur_ks * BK,
                                             ebase + t.nt * BN + rank * N_CTA);
                        } else {
#pragma unroll
                            for (int j = 0; j < N_CTA / 64; ++j)
                                tma_load_2d_pair(smem_u32(dst) + j * 8192, &tmap_w, mapa_shared(bar, 0),
                                                 t.nt * BN + rank * N_CTA + 64 * j, ebase + cur_ks * BK);
                        }
                    } else {
                        arrive_leader(&ctl->b_full[s]);
                    }
                }
            } else {
                const uint8_t* raw = sRaw + rs * RAW_STAGE;
                const float* am = reinterpret_cast<const float*>(raw + RAW_BYTES);
                uint4 pk[BLOCKS_PER_THREAD][2];
                float sc[BLOCKS_PER_THREAD];
#pragma unroll
                for (int i = 0; i < BLOCKS_PER_THREAD; ++i) {
                    const int b = tg + TPG * i;
                    sc[i] = am[b];
                    if (FWD) {   // raw [N_CTA rows][32 B]
                        pk[i][0] = *reinterpret_cast<const uint4*>(raw + b * 32);
                        pk[i][1] = *reinterpret_cast<const uint4*>(raw + b * 32 + 16);
                    } else {     // raw [64 k-rows][64 B], 64B-swizzled
                        const int k = b & 63, j = b >> 6, sw = (k >> 1) & 3;
                        pk[i][0] = *reinterpret_cast<const uint4*>(raw + k * (N_CTA / 2) + (((2 * j) ^ sw) << 4));
                        pk[i][1] = *reinterpret_cast<const uint4*>(raw + k * (N_CTA / 2) + (((2 * j + 1) ^ sw) << 4));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->raw_empty[rs]));
                if (!wait(&ctl->b_empty[s], (r & 1) ^ 1)) break;
#pragma unroll
                for (int i = 0; i < BLOCKS_PER_THREAD; ++i) {
                    const int b = tg + TPG * i;
                    BlockTable tb, tb1;
                    if (CB == 2) {   // two 32-element scales: bytes sel, sel + 1 of the four copied
                        const uint32_t q = __float_as_uint(sc[i]);
                        const int sel = FWD ? 2 * (cur_ks & 1) : 2 * ((b >> 6) & 1);
                        tb = make_table<2>(mx_scale((q >> (8 * sel)) & 0xFFu));
                        tb1 = make_table<2>(mx_scale((q >> (8 * sel + 8)) & 0xFFu));
                    } else {
                        tb = make_table<(CB < 3 ? CB : 0)>(sc[i]);
                    }
                    const uint32_t words[8] = {pk[i][0].x, pk[i][0].y, pk[i][0].z, pk[i][0].w,
                                               pk[i][1].x, pk[i][1].y, pk[i][1].z, pk[i][1].w};
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t o[4];
                        decode_word((CB == 2 && c >= 4) ? tb1 : tb, words[c], o);
                        const uint32_t off = FWD ? sw128_offset(b, c) : (b >> 6) * 8192 + sw128_offset(b & 63, c);
                        *reinterpret_cast<uint4*>(dst + off) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive_leader(&ctl->b_full[s]);
            }
            it += DEQ_GROUPS;
            pos += DEQ_GROUPS;
            normalize();
        }
    } else if (warp < 4) {
        // epilogue: lane l holds accumulator row 32*warp + l of this CTA's half
        const int wrow0 = 128 * rank + 32 * warp, rtile = wrow0 + lane;
        uint8_t* bufs = sBuf + warp * WARP_BUFS * BUF;   // pair b: y (and residual) at 2b, saved at 2b + 1
        uint32_t nload = 0, nuse = 0;                    // chunks whose residual was requested / used
        uint32_t nstore = 0;                             // chunks stored (no residual)
        const bool has_res = FWD && p.residual != nullptr;
        const int sw = (lane >> 1) & 3;                  // 64-byte swizzle of the lane's row
        // pair b's stores have been read out; request the residual chunk into it
        auto load_res = [&](int c0, int srow) {
            const uint32_t b = nload & 1;
            if (lane == 0) {
                bulk_wait_read<0>();
                const uint32_t bar = smem_u32(&ctl->res_full[warp][b]);
                mbar_arrive_expect_tx(bar, BUF);
                tma_load_2d(smem_u32(bufs + 2 * b * BUF), &tmap_res, bar, c0, srow);
            }
            __syncwarp();
            ++nload;
        };
        uint32_t lt = 0;
        bool aborted = false;
        for (int item = cluster_id; item < items && !aborted; item += nclusters, ++lt) {
            const Tile t = decode_item(p, item, nk);
            const uint32_t ab = lt & 1;
            const bool bulk = t.rows - wrow0 >= 32;   // all 32 rows inside the tile
            const bool any = t.rows > wrow0, valid = rtile < t.rows;
            const int64_t row = (int64_t)t.row0 + rtile;
            const int srow = t.row0 + wrow0;
            const int c_first = t.nt * BN;
            if (!SPLIT && has_res && bulk) load_res(c_first, srow);
            if (!wait(&ctl->acc_full[ab], (lt >> 1) & 1)) break;
            tc_fence_after();
            const uint32_t tbase = tmem_base + ((uint32_t)(warp * 32) << 16) + ab * BN;
#pragma unroll 1
            for (int q = 0; q < BN / 32; ++q) {
                const int c0 = c_first + 32 * q;
                if (c0 >= p.N) break;   // the same for the whole CTA
                float v[32];
                tmem_load32(tbase + 32 * q, v);
                if (!any) continue;
                if (SPLIT) {
                    const int part = item - (item / p.splits) * p.splits;
                    // few rows: straight from the registers.  2880 by 2880, us here / below: 32 rows 14.2 / 17.6,
                    // 64 rows 16.1 / 17.8, 80 rows 17.0 / 18.1, 96 rows 18.3 / 18.4, 128 rows 20.0 / 18.8
                    if (t.rows <= 64) {
                        float4* d = reinterpret_cast<float4*>(p.partial + ((int64_t)part * p.P + row) * p.N + c0);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (valid) d[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        continue;
                    }
                    // through shared memory (16-byte pieces rotated by the row), so that the warp's
                    // stores are whole 128-byte lines (200 rows: 19.5 us, 20.5 above)
                    uint8_t* chunk = bufs + (q & 1) * 4096;   // its last readers are behind the barrier in between
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(chunk + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + (lane >> 3), c = lane & 7;
                        if (wrow0 + r < t.rows)   // (warps past the tile's rows left above)
                            reinterpret_cast<float4*>(p.partial + ((int64_t)part * p.P + srow + r) * p.N + c0)[c] =
                                *reinterpret_cast<const float4*>(chunk + r * 128 + ((c ^ (r & 7)) << 4));
                    }
                    continue;
                }
                if (has_res && bulk && q + 1 < BN / 32 && c0 + 32 < p.N) load_res(c0 + 32, srow);
                uint32_t sv[16];   // act' packed
                if (FWD) {
                    if (p.bias) {
                        const float4* bs = reinterpret_cast<const float4*>(p.bias + (int64_t)t.e * p.N + c0);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 f = bs[i];
                            v[4 * i] += f.x; v[4 * i + 1] += f.y; v[4 * i + 2] += f.z; v[4 * i + 3] += f.w;
                        }
                    }
                    const bool save = p.saved != nullptr;
                    if (p.act != E4B_LINEAR_ACT_NONE || save)
                        with_act(p.act, [&](auto kind) {
                            constexpr int ACT = decltype(kind)::value;
                            float d0, d1;
                            if (save) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    linear_act<ACT>(v[2 * i], v[2 * i], d0);
                                    linear_act<ACT>(v[2 * i + 1], v[2 * i + 1], d1);
                                    sv[i] = pack_bf16x2(d0, d1);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i) linear_act<ACT>(v[i], v[i], d0);
                            }
                        });
                }
                if (bulk) {
                    const uint32_t b = has_res ? nuse & 1 : nstore & 1;
                    uint8_t* yb = bufs + 2 * b * BUF + lane * 64;
                    if (has_res) {
                        if (!wait(&ctl->res_full[warp][nuse & 1], (nuse >> 1) & 1)) {
                            aborted = true;
                            break;
                        }
                        ++nuse;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 rv = *reinterpret_cast<const uint4*>(yb + ((c ^ sw) << 4));
                            const uint32_t w[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                v[8 * c + 2 * j] += __uint_as_float(w[j] << 16);
                                v[8 * c + 2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
                            }
                        }
                    } else if (nstore++ >= 2) {   // the pair's last stores have been read out
                        if (lane == 0) bulk_wait_read<1>();
                        __syncwarp();
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (p.out)
                            *reinterpret_cast<uint4*>(yb + ((c ^ sw) << 4)) =
                                make_uint4(pack_bf16x2(v[8 * c], v[8 * c + 1]), pack_bf16x2(v[8 * c + 2], v[8 * c + 3]),
                                           pack_bf16x2(v[8 * c + 4], v[8 * c + 5]), pack_bf16x2(v[8 * c + 6], v[8 * c + 7]));
                        if (FWD && p.saved)
                            *reinterpret_cast<uint4*>(yb + BUF + ((c ^ sw) << 4)) =
                                make_uint4(sv[4 * c], sv[4 * c + 1], sv[4 * c + 2], sv[4 * c + 3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (p.out) tma_store_2d(&tmap_out, smem_u32(bufs + 2 * b * BUF), c0, srow);
                        if (FWD && p.saved) tma_store_2d(&tmap_saved, smem_u32(bufs + (2 * b + 1) * BUF), c0, srow);
                        bulk_commit();
                    }
                } else if (valid) {   // the partial slab at the end of an expert's rows
                    const int64_t at = row * p.N + c0;
                    if (has_res) {
                        const uint4* rp = reinterpret_cast<const uint4*>(p.residual + at);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 rv = rp[c];
                            const uint32_t w[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                v[8 * c + 2 * j] += __uint_as_float(w[j] << 16);
                                v[8 * c + 2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
                            }
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (p.out)
                            reinterpret_cast<uint4*>(p.out + at)[c] =
                                make_uint4(pack_bf16x2(v[8 * c], v[8 * c + 1]), pack_bf16x2(v[8 * c + 2], v[8 * c + 3]),
                                           pack_bf16x2(v[8 * c + 4], v[8 * c + 5]), pack_bf16x2(v[8 * c + 6], v[8 * c + 7]));
                        if (FWD && p.saved)
                            reinterpret_cast<uint4*>(p.saved + at)[c] =
                                make_uint4(sv[4 * c], sv[4 * c + 1], sv[4 * c + 2], sv[4 * c + 3]);
                    }
                }
            }
            if (aborted) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(&ctl->acc_empty[ab]);
        }
        if (lane == 0) {
            bulk_wait_all();
            for (; nuse < nload; ++nuse)   // residual loads still in flight (bounded)
                mbar_wait_drain(smem_u32(&ctl->res_full[warp][nuse & 1]), (nuse >> 1) & 1);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // the peer's shared memory and TMEM stay alive until the pair is done
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// y = residual + act(sum of the parts + bias), saved = act': the split product's epilogue.
// A thread takes 8 columns of a row; the parts are added in order.
__global__ void __launch_bounds__(256) linear_finish_kernel(const LinearGemm p) {
    pdl_release();
    pdl_wait();
    const int nv = p.N / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.P * nv) return;
    const int64_t row = i / nv, c = (i - row * nv) * 8, at = row * p.N + c;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p.bias ? p.bias[c + j] : 0.0f;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int q = 0; q < p.splits; ++q) {
        const float4* f = reinterpret_cast<const float4*>(p.partial + ((int64_t)q * p.P) * p.N + at);
        const float4 lo = __ldcg(f), hi = __ldcg(f + 1);
        s[0] += lo.x; s[1] += lo.y; s[2] += lo.z; s[3] += lo.w;
        s[4] += hi.x; s[5] += hi.y; s[6] += hi.z; s[7] += hi.w;
    }
    float d[8];
    with_act(p.act, [&](auto kind) {
#pragma unroll
        for (int j = 0; j < 8; ++j) linear_act<decltype(kind)::value>(s[j] + v[j], v[j], d[j]);
    });
    if (p.residual) {
        float r[8];
        unpack<__nv_bfloat16, 8>(__ldcg(reinterpret_cast<const uint4*>(p.residual + at)), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
    if (p.out) *reinterpret_cast<uint4*>(p.out + at) = pack<__nv_bfloat16, 8>(v);
    if (p.saved) *reinterpret_cast<uint4*>(p.saved + at) = pack<__nv_bfloat16, 8>(d);
}

// One block: the m-tiles of every expert's rows.  Offsets are taken as the running
// maximum of their values clamped to [0, P], so any input gives ranges inside the rows.
__global__ void __launch_bounds__(256) linear_schedule_kernel(const int32_t* __restrict__ offsets, int E, int64_t P,
                                                              int tile_rows, int* __restrict__ tile_prefix,
                                                              int4* __restrict__ sched) {
    __shared__ int s_off[257];
    __shared__ int s_first[257];
    pdl_release();
    pdl_wait();
    for (int e = threadIdx.x; e <= E; e += blockDim.x)
        s_off[e] = offsets ? (int)min(max((int64_t)__ldcg(offsets + e), (int64_t)0), P) : (e == 0 ? 0 : (int)P);
    __syncthreads();
    if (threadIdx.x < 32) {   // running maximum and m-tile prefix, 32 experts at a time
        const int lane = threadIdx.x;
        int top = s_off[0], run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            int end = e < E ? s_off[e + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end = max(end, u);
            }
            end = max(end, top);
            int begin = __shfl_up_sync(0xffffffffu, end, 1);
            if (lane == 0) begin = top;
            const int n = e < E ? (end - begin + tile_rows - 1) / tile_rows : 0;
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += u;
            }
            __syncwarp();
            if (e < E) {
                s_off[e + 1] = end;
                s_first[e] = run + x - n;
            }
            top = __shfl_sync(0xffffffffu, end, 31);
            run += __shfl_sync(0xffffffffu, x, 31);
            __syncwarp();
        }
        if (lane == 0) s_first[E] = run;
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += blockDim.x) tile_prefix[e] = s_first[e];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = warp; e < E; e += 8) {
        const int begin = s_off[e], n = s_off[e + 1] - begin, first = s_first[e];
        for (int m = lane; m * (int64_t)tile_rows < n; m += 32)
            sched[first + m] = make_int4(e, begin + m * tile_rows, min(tile_rows, n - m * tile_rows), 0);
    }
}

template <bool FWD, int CB, bool SPLIT>
cudaError_t launch_one(const CUtensorMap& ma, const CUtensorMap& mw, const CUtensorMap& mo, const CUtensorMap& ms,
                       const CUtensorMap& mr, const LinearGemm& p, int grid, cudaStream_t st) {
    auto kern = linear_gemm_kernel<FWD, CB, SPLIT>;
    {   // the shared-memory limit is an attribute per device and instance
        static std::mutex mu;
        static bool set[64] = {false};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        if (!set[dev]) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
            if (e != cudaSuccess) return e;
            set[dev] = true;
        }
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CTAS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kern, ma, mw, mo, ms, mr, p);
}

template <bool FWD, bool SPLIT>
cudaError_t launch_cb(int cb, const CUtensorMap& ma, const CUtensorMap& mw, const CUtensorMap& mo, const CUtensorMap& ms,
                      const CUtensorMap& mr, const LinearGemm& p, int grid, cudaStream_t st) {
    switch (cb) {
        case 0: return launch_one<FWD, 0, SPLIT>(ma, mw, mo, ms, mr, p, grid, st);
        case 1: return launch_one<FWD, 1, SPLIT>(ma, mw, mo, ms, mr, p, grid, st);
        case 2: return launch_one<FWD, 2, SPLIT>(ma, mw, mo, ms, mr, p, grid, st);
        default: return launch_one<FWD, 3, SPLIT>(ma, mw, mo, ms, mr, p, grid, st);
    }
}

bool map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer, uint64_t row_bytes,
            uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw) {
    const uint64_t dims[2] = {inner, outer}, strides[1] = {row_bytes};
    const uint32_t box[2] = {box_inner, box_outer};
    return make_tensor_map(m, dt, 2, base, dims, strides, box, sw);
}

}  // namespace

int linear_tile_rows() { return TILE_M; }

int linear_splits(int64_t P, int N, int K) {
    const int64_t tiles = (P + TILE_M - 1) / TILE_M * ((N + BN - 1) / BN);
    const int64_t pairs = num_sms() / CTAS, nk = K / BK;
    // at least 4 k-stages per part, as many parts as fill the pairs
    return (int)std::max<int64_t>(1, std::min<int64_t>(pairs / std::max<int64_t>(1, tiles), nk / 4));
}

cudaError_t launch_linear_schedule(const int32_t* offsets, int E, int64_t P, int tile_rows, int* tile_prefix, int4* sched,
                                   cudaStream_t st) {
    return launch_pdl(linear_schedule_kernel, dim3(1), dim3(256), 0, st, offsets, E, P, tile_rows, tile_prefix, sched);
}

cudaError_t launch_linear_gemm(bool forward, int codebook, const LinearGemm& p, int max_m_tiles, cudaStream_t st) {
    CUtensorMap ma, mw, mo, ms, mr;
    if (!map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.a, (uint64_t)p.K, (uint64_t)p.P, (uint64_t)p.K * 2, 64, 128,
                CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    const uint64_t cols = forward ? (uint64_t)p.K : (uint64_t)p.N;   // stored row length
    if (codebook == 3) {
        if (!map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.bf16_b, cols, (uint64_t)p.b_rows_total, cols * 2, 64,
                    forward ? N_CTA : BK, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    } else if (!map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.packed, cols / 2, (uint64_t)p.b_rows_total, cols / 2,
                       forward ? BK / 2 : N_CTA / 2, forward ? N_CTA : BK,
                       forward ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B)) {
        return cudaErrorInvalidValue;
    }
    auto rows32 = [&](CUtensorMap* m, const void* base) {
        return map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, (uint64_t)p.N, (uint64_t)p.P, (uint64_t)p.N * 2, 32, 32,
                      CU_TENSOR_MAP_SWIZZLE_64B);
    };
    // absent operands take another operand's map (never used)
    mo = ms = mr = ma;
    if (p.out && !rows32(&mo, p.out)) return cudaErrorInvalidValue;
    if (p.saved && !rows32(&ms, p.saved)) return cudaErrorInvalidValue;
    if (p.residual && !rows32(&mr, p.residual)) return cudaErrorInvalidValue;
    const int64_t items = (int64_t)max_m_tiles * p.n_tiles * p.splits;
    if (items > INT32_MAX / 2) return cudaErrorInvalidValue;
    const int grid = (int)std::min<int64_t>(items * CTAS, (num_sms() / CTAS) * CTAS);
    if (grid <= 0) return cudaSuccess;
    if (p.splits == 1)
        return forward ? launch_cb<true, false>(codebook, ma, mw, mo, ms, mr, p, grid, st)
                       : launch_cb<false, false>(codebook, ma, mw, mo, ms, mr, p, grid, st);
    cudaError_t err = forward ? launch_cb<true, true>(codebook, ma, mw, mo, ms, mr, p, grid, st)
                              : launch_cb<false, true>(codebook, ma, mw, mo, ms, mr, p, grid, st);
    if (err != cudaSuccess) return err;
    const int64_t blocks = (p.P * (p.N / 8) + 255) / 256;
    return launch_pdl(linear_finish_kernel, dim3((unsigned)blocks), dim3(256), 0, st, p);
}

}  // namespace e4b
