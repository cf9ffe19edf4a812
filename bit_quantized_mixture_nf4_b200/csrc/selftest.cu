// Watchdog self-test: one thread waits on an mbarrier that nothing will ever
// arrive at, through the same bounded wait every pipelined kernel uses.  After
// the wait's time limit (2 s) it records the timeout in the device status word
// and returns; nothing faults, traps or hangs, and the context stays usable.
//
// Ring self-test: two groups of the block norm kernels' shared-memory ring read rows; one row
// of the first group never counts as landed (its barrier expects 16 bytes more than come).
// That group must stop requesting there, let its other copies land and return.
#include "../../include/e4b.h"
#include "block_ring.cuh"

namespace e4b {

__global__ void watchdog_selftest_kernel(uint32_t* status) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x != 0) return;
    const uint32_t b = smem_u32(&bar);
    abort_flag = 0;
    mbar_init(b, 1);   // one arrival expected, none will come
    fence_barrier_init();
    mbar_wait(b, 0, &abort_flag, status);
}

constexpr int kTestRow = 128, kTestStages = 4;   // floats of a row

// out[2 g]: rows that group g read, all as in src; out[2 g + 1]: rows that it still had in flight,
// all of them in their slots by the end.  -1 where one was not.
__global__ void __launch_bounds__(64) ring_selftest_kernel(const BlockArgs a, const RingPlan pl, int lost, int32_t* out) {
    __shared__ __align__(128) uint8_t dsm[2 * kTestStages * kTestRow * 4];
    __shared__ uint64_t s_full[kRingGroups][kRingStages];
    __shared__ int s_abort;
    RowRing ring;
    const int64_t first = ring_setup<float>(ring, a, pl, 1, dsm, s_full, s_abort);
    ring_source(ring, 0, a.h);
    const int x = threadIdx.x % pl.tx, g = threadIdx.x / pl.tx;
    const float4* src = static_cast<const float4*>(a.h);
    auto same = [&](const uint8_t* slot, int64_t row) {
        const float4 p = reinterpret_cast<const float4*>(slot)[x], q = src[row * (kTestRow / 4) + x];
        return __all_sync(0xffffffffu, p.x == q.x && p.y == q.y && p.z == q.z && p.w == q.w) != 0;
    };
    auto request = [&]() {
        if (ring.next == lost) mbar_expect_tx(ring.bars + ring.put_bar, 16);
        ring.issue<float, true>();
    };
    if (x == 0)
        for (int i = 0; i < pl.stages; ++i) request();
    int used = 0, landed = 0;
    bool live = true;   // until a wait of this group ran out
    for (int64_t u = first; u < ring.units; u += ring.step) {
        const uint8_t* row = ring.wait<true>(u);
        live = live && mbar_test_wait(ring.bars + 8 * ring.get, ring.phase);
        live = __all_sync(0xffffffffu, live) != 0;
        if (live && used >= 0) used = same(row, u) ? used + 1 : -1;
        __syncwarp();
        if (x == 0) request();
        ring.advance();
    }
    const int64_t asked = min(ring.units, first + (max(used, 0) + pl.stages) * ring.step);   // the end of it
    for (int64_t i = max(used, 0); !live && first + i * ring.step < asked; ++i)
        if (landed >= 0) landed = same(ring.slots + i % pl.stages * pl.slot_bytes, first + i * ring.step) ? landed + 1 : -1;
    if (x == 0) {
        out[2 * g] = used;
        out[2 * g + 1] = landed;
    }
}

}  // namespace e4b

extern "C" e4b_status e4b_ring_selftest(const float* src, int rows, int lost, int32_t* out, void* stream) {
    using namespace e4b;
    if (!src || !out || rows < 1 || off_boundary(16, {src}) || off_boundary(4, {out})) return E4B_ERR_INVALID_ARG;
    BlockArgs a{};
    a.h = src;
    a.T = rows;
    a.H = kTestRow;
    a.status = device_status_ptr();
    if (!a.status) return E4B_ERR_CUDA;
    const RingPlan pl{32, kTestStages, 1, kTestRow * 4};
    return launch_pdl(ring_selftest_kernel, dim3(1), dim3(64), 0, static_cast<cudaStream_t>(stream), a, pl, lost, out) ==
                   cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}

extern "C" e4b_status e4b_watchdog_selftest(void* stream) {
    uint32_t* status = e4b::device_status_ptr();
    if (!status) return E4B_ERR_CUDA;
    e4b::watchdog_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(status);
    e4b::count_launch();
    return cudaGetLastError() == cudaSuccess ? E4B_OK : E4B_ERR_CUDA;
}
