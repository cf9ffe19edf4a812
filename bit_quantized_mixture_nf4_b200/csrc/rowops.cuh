// Row kernels' shared pieces: rows of H elements (bf16 or fp32) read and written in
// vectors of V elements, arithmetic in fp32.
#pragma once
#include <initializer_list>
#include <type_traits>

#include "e4b_internal.h"

namespace e4b {

template <int BYTES> struct RawVec;
template <> struct RawVec<16> { using type = uint4; };
template <> struct RawVec<8> { using type = uint2; };
template <> struct RawVec<4> { using type = uint32_t; };
template <> struct RawVec<2> { using type = uint16_t; };
template <typename E, int V> using raw_t = typename RawVec<V * (int)sizeof(E)>::type;

// The V elements of a raw vector as fp32.
template <typename E, int V>
__device__ __forceinline__ void unpack(const raw_t<E, V>& r, float (&v)[V]) {
    if constexpr (std::is_same<E, float>::value) {
        static_assert(sizeof(r) == 4 * V, "fp32 vector");
        const float* f = reinterpret_cast<const float*>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = f[i];
    } else if constexpr (V == 1) {
        v[0] = __uint_as_float((uint32_t)r << 16);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// fp32 values rounded once to E (bf16: nearest-even).
template <typename E, int V>
__device__ __forceinline__ raw_t<E, V> pack(const float (&v)[V]) {
    raw_t<E, V> r;
    if constexpr (std::is_same<E, float>::value) {
        float* f = reinterpret_cast<float*>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = v[i];
    } else if constexpr (V == 1) {
        r = (uint16_t)(pack_bf16x2(v[0], 0.0f) & 0xFFFFu);
    } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    return r;
}

// Vectors that are read or written once (evict-first in L2).
template <typename R> __device__ __forceinline__ R ld_once(const void* p, int64_t i) {
    return __ldcs(static_cast<const R*>(p) + i);
}
template <typename R> __device__ __forceinline__ void st_once(void* p, int64_t i, R v) {
    __stcs(static_cast<R*>(p) + i, v);
}

// Programmatic dependent launch: a chained kernel starts while its predecessor drains
// and waits here, before it touches memory that an earlier kernel writes or still reads.
// What a predecessor may have written is read with coherent loads only (plain, .cg or .cs),
// never through the non-coherent path: it changes during this kernel's lifetime.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;"); }

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Bytes of the widest vector (16, 4 or one element) that every row of rows of row_bytes
// at these bases can be read in; 0 where a base is not aligned to its elements.
inline int row_vector_bytes(int64_t row_bytes, int elem, std::initializer_list<const void*> bases) {
    uintptr_t a = (uintptr_t)row_bytes;
    for (const void* b : bases) a |= (uintptr_t)b;
    if (a % 16 == 0) return 16;
    return a % elem ? 0 : a % 4 == 0 ? 4 : elem;
}

// Whether one of the given pointers is off a boundary of `bytes` (a power of two).
inline bool off_boundary(int bytes, std::initializer_list<const void*> ptrs) {
    uintptr_t a = 0;
    for (const void* p : ptrs) a |= (uintptr_t)p;
    return a % bytes != 0;
}

}  // namespace e4b
