// Rows through shared memory: the long-run form of the block norm kernels.
//
// Each group of tx threads (a warp, or the whole block) keeps a ring of rows in shared
// memory, filled by bulk copies that one thread issues several rows ahead, so that enough
// bytes are in flight whatever the barriers of the row at hand cost.  A row's slot is
// refilled after the barrier behind its last read.  Rows whose length is no multiple of 16
// bytes are copied as the 16-byte units around them and read at their offset: 4 bytes or one
// element at a time from shared memory, without narrow loads from HBM.
#pragma once
#include <algorithm>
#include <mutex>
#include <set>
#include <utility>

#include "block_norm.cuh"

namespace e4b {

constexpr int kRingStages = 8, kRingGroups = 8;
constexpr int kRingSmem = 222 * 1024;   // dynamic shared memory of an SM that its blocks' rings share

constexpr int64_t kNoMore = 1LL << 62;   // RowRing::next after a wait that ran out

struct RowRing {
    uint32_t data, bars;               // shared addresses of the group's slots and barriers
    const uint8_t* slots;
    volatile int* abort_flag;
    uint32_t* status;
    int stages, arrays, unit_bytes, slot_bytes;   // slot: one array's part of a stage
    int64_t step, next, units, end;    // next: the unit to request; end: bytes of the tensor
    const uint8_t* src[5];
    uint32_t put_data = 0, put_bar = 0;   // offsets of the next request
    int get = 0;                       // stage of the unit at hand, and its parity
    uint32_t phase = 0;

    // Requests the next unit.  ALIGNED: rows are multiples of 16 bytes.  By the group's first thread,
    // which has waited for what the slot held.
    template <typename E, bool ALIGNED>
    __device__ __forceinline__ void issue() {
        if (next < units) {
            const uint32_t bar = bars + put_bar, dst = data + put_data;
            const int64_t begin = next * unit_bytes, stop_row = min(begin + unit_bytes, end);
            int64_t from = begin, stop = stop_row;
            if (!ALIGNED) {
                // the copy ends at the last 16-byte unit that lies inside the tensor; elements behind
                // it (of the last row) are stored by hand, before the arrival that announces the rows
                from = begin & ~(int64_t)15;
                stop = min((stop_row + 15) & ~(int64_t)15, end & ~(int64_t)15);
                if (stop < stop_row) {
                    uint8_t* at = const_cast<uint8_t*>(slots) + put_data;
                    for (int i = 0; i < arrays; ++i)
                        for (int64_t p = max(stop, begin); p < stop_row; p += (int)sizeof(E)) {
                            if constexpr (sizeof(E) == 2)
                                *reinterpret_cast<uint16_t*>(at + i * slot_bytes + (p - from)) =
                                    __ldcg(reinterpret_cast<const uint16_t*>(src[i] + p));
                            else
                                *reinterpret_cast<uint32_t*>(at + i * slot_bytes + (p - from)) =
                                    __ldcg(reinterpret_cast<const uint32_t*>(src[i] + p));
                        }
                }
            }
            const int bytes = (int)max(stop - from, (int64_t)0);
            mbar_arrive_expect_tx(bar, arrays * bytes);
            if (ALIGNED || bytes > 0) {
#pragma unroll
                for (int i = 0; i < 5; ++i)
                    if (i < arrays) bulk_g2s(dst + i * slot_bytes, src[i] + from, bytes, bar);
            }
        }
        next += step;
        put_bar += 8;
        put_data += arrays * slot_bytes;
        if (put_bar == 8u * stages) put_bar = put_data = 0;
    }
    // Waits for unit u, the unit at hand; its first element in the slot's first array.  A wait
    // that runs out is recorded in the status word; the kernel then runs on through its rows without
    // requesting any (its barriers stay whole, its outputs are void; its later waits give up at once).
    template <bool ALIGNED>
    __device__ __forceinline__ const uint8_t* wait(int64_t u) {
        if (!mbar_wait(bars + 8 * get, phase, abort_flag, status)) give_up(u);
        const uint8_t* slot = slots + get * arrays * slot_bytes;
        return ALIGNED ? slot : slot + ((uint32_t)(u * unit_bytes) & 15u);
    }
    __device__ __forceinline__ void advance() {
        if (++get == stages) {
            get = 0;
            phase ^= 1u;
        }
    }
    // The thread that requests stops doing so and lets what it has in flight land (with a limit): unit u
    // and those requested behind it.  So a slot whose copy has not landed is never requested again, and
    // none is in flight at the kernel's end.
    __device__ __forceinline__ void give_up(int64_t u) {
        if (next < step || next >= kNoMore) return;   // a thread that does not request, or has stopped
        next = kNoMore;
        const uint64_t t0 = globaltimer_ns();
        for (int i = 0, g = get; i < stages && u < units; ++i, u += step) {
            const uint32_t parity = g < get ? phase ^ 1u : phase;
            while (!mbar_try_wait(bars + 8 * g, parity) && globaltimer_ns() - t0 <= kWaitLimitNs) {}
            if (++g == stages) g = 0;
        }
    }
};

// Vector v of a row in shared memory; zeros behind the row's end (a predicated load: branches
// around the vectors' arithmetic cost more than it, they keep the vectors' chains apart).
template <typename E, int V>
__device__ __forceinline__ void read_row(const uint8_t* row, int v, int nvec, float (&out)[V]) {
    raw_t<E, V> r = {};
    if (v < nvec) r = reinterpret_cast<const raw_t<E, V>*>(row)[v];
    unpack<E, V>(r, out);
}

// How a block's groups share out the rows (set by the host).
struct RingPlan {
    int tx, stages, rows, slot_bytes;   // threads per group, ring depth, rows per unit, bytes per slot
};

// The block's barriers, its predecessor's end, and this group's ring; its first unit.
template <typename E>
__device__ __forceinline__ int64_t ring_setup(RowRing& r, const BlockArgs& a, const RingPlan& pl, int arrays, uint8_t* dsm,
                                              uint64_t (&s_full)[kRingGroups][kRingStages], int& s_abort) {
    const int ry = threadIdx.x / pl.tx, rpb = blockDim.x / pl.tx;
    if (threadIdx.x < rpb * kRingStages) mbar_init(smem_u32(&s_full[0][0] + threadIdx.x), 1);
    if (threadIdx.x == 0) s_abort = 0;
    fence_barrier_init();
    pdl_release();
    pdl_wait();
    __syncthreads();
    const int row_bytes = a.H * (int)sizeof(E);
    r.unit_bytes = pl.rows * row_bytes;
    r.slot_bytes = pl.slot_bytes;
    r.arrays = arrays;
    r.stages = pl.stages;
    r.slots = dsm + (int64_t)ry * pl.stages * arrays * pl.slot_bytes;
    r.data = smem_u32(r.slots);
    r.bars = smem_u32(s_full[ry]);
    r.abort_flag = &s_abort;
    r.status = a.status;
    r.next = (int64_t)blockIdx.x * rpb + ry;
    r.step = (int64_t)gridDim.x * rpb;
    r.units = (a.T + pl.rows - 1) / pl.rows;
    r.end = a.T * row_bytes;
    return r.next;
}
// Array i of the rows.
__device__ __forceinline__ void ring_source(RowRing& r, int i, const void* p) {
#pragma unroll
    for (int j = 0; j < 5; ++j)
        if (j == i) r.src[j] = static_cast<const uint8_t*>(p);
}

// ------------------------------------------------------------------ host side

// Threads per row and block, groups per block and blocks per SM for `elems` elements a thread
// and `per_sm` threads on an SM; rows per unit, ring depth and grid for T rows of `arrays` arrays.  A bulk copy has a fixed
// cost, so short rows are copied several at a time, up to 4 KB.
struct RingShape {
    int threads, rpb, per, blocks = 0;
    RingPlan plan{};
    RingShape(int H, int es, int arrays, int64_t T, int elems, int per_sm) {
        plan.tx = ((H + elems - 1) / elems + 31) / 32 * 32;
        threads = plan.tx == 32 ? 256 : plan.tx;
        rpb = threads / plan.tx;
        per = std::max(1, per_sm / threads);
        const int64_t rb = (int64_t)H * es, groups = (int64_t)num_sms() * per * rpb;
        plan.rows = (int)std::max<int64_t>(1, std::min<int64_t>(4096 / rb, T / (2 * groups)));
        const int64_t unit = plan.rows * rb;
        plan.slot_bytes = (int)(rb % 16 == 0 ? unit : ((unit + 15) & ~15LL) + 16);
        plan.stages = (int)std::min<int64_t>(kRingStages, kRingSmem / per / ((int64_t)rpb * arrays * plan.slot_bytes));
        const int64_t units = (T + plan.rows - 1) / plan.rows;
        blocks = (int)std::min<int64_t>((units + rpb - 1) / rpb, (int64_t)num_sms() * per);
        fits = plan.stages >= 1 && units >= 2LL * blocks * rpb;
        smem = (size_t)plan.stages * rpb * arrays * plan.slot_bytes;
    }
    bool fits = false;   // at least two units per group, and one of them in shared memory
    size_t smem = 0;
};

// Raises a kernel's dynamic shared memory limit, once per kernel and device.
inline cudaError_t allow_ring(const void* kern) {
    static std::mutex mu;
    static std::set<std::pair<const void*, int>> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    try {   // nothing may be thrown through the C entry points
        std::lock_guard<std::mutex> lock(mu);
        if (done.count({kern, dev})) return cudaSuccess;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
        if (e == cudaSuccess) done.insert({kern, dev});
    } catch (...) {
        return cudaErrorMemoryAllocation;
    }
    return e;
}

// f(integral_constant gate): the ring kernels' instances (a token gate takes the plain one).
template <typename F>
cudaError_t with_gate(int gate, F f) {
    if (gate == E4B_GATE_CHANNEL) return f(std::integral_constant<int, E4B_GATE_CHANNEL>());
    if (gate == E4B_GATE_ELEMENT) return f(std::integral_constant<int, E4B_GATE_ELEMENT>());
    return f(std::integral_constant<int, E4B_GATE_NONE>());
}

// f(E*, integral_constant V): the vectors that rows of H elements can be read and written in.
template <typename F>
cudaError_t with_ring_vector(e4b_dtype dt, int H, F f) {
    if (dt == E4B_BF16) {
        if (H % 8 == 0) return f((__nv_bfloat16*)nullptr, std::integral_constant<int, 8>());
        if (H % 2 == 0) return f((__nv_bfloat16*)nullptr, std::integral_constant<int, 2>());
        return f((__nv_bfloat16*)nullptr, std::integral_constant<int, 1>());
    }
    if (H % 4 == 0) return f((float*)nullptr, std::integral_constant<int, 4>());
    return f((float*)nullptr, std::integral_constant<int, 1>());
}

}  // namespace e4b
