// hc_ops.cuh -- device-side building blocks of the training operators
// (hc_embedding.cu, hc_block_norm.cu, hc_distill.cu, hc_clip.cu, hc_expert.cu,
// hc_expert_matmul.cu): element access in binary32, reductions over the threads
// of a row, programmatic launches.
// Internal; not installed.
#pragma once

#include <cuda_runtime.h>

#include "hc_device.cuh"
#include "hc_ops.h"

namespace hc {
namespace {

struct Bf16 {
    uint16_t u;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(Bf16 v) { return __uint_as_float((uint32_t)v.u << 16); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(Bf16* p, float v) { p->u = (uint16_t)pack_bf16x2(v, 0.0f); }

// A 16-byte vector of T and its elements in binary32.
template <class T>
constexpr int kVecOf = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = bf_lo(u[i]);
        v[2 * i + 1] = bf_hi(u[i]);
    }
}
__device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// N consecutive elements of a row, of which the first n (any value) are in
// range; the others read as 0 and are not written.  Accesses of 8 or 16 bytes
// when N > 1 elements make them (the caller then guarantees 16-byte aligned
// rows and N-element aligned places) and all N are in range.
template <class T, int N>
__device__ __forceinline__ void load_n(const T* p, int n, float (&v)[N]) {
    constexpr int E = kVecOf<T>;
    if constexpr (N % E == 0) {
        if (n >= N) {
#pragma unroll
            for (int i = 0; i < N / E; i++) {
                float e[E];
                unpack(((const uint4*)p)[i], e);
#pragma unroll
                for (int j = 0; j < E; j++) v[i * E + j] = e[j];
            }
            return;
        }
    } else if constexpr (2 * N == E && sizeof(T) == 2) {  // half a vector of bf16
        if (n >= N) {
            const uint2 u = *(const uint2*)p;
            v[0] = bf_lo(u.x);
            v[1] = bf_hi(u.x);
            v[2] = bf_lo(u.y);
            v[3] = bf_hi(u.y);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = i < n ? to_f32(p[i]) : 0.0f;
}
template <class T, int N>
__device__ __forceinline__ void store_n(T* p, int n, const float (&v)[N]) {
    constexpr int E = kVecOf<T>;
    if constexpr (N % E == 0) {
        if (n >= N) {
#pragma unroll
            for (int i = 0; i < N / E; i++) {
                float e[E];
#pragma unroll
                for (int j = 0; j < E; j++) e[j] = v[i * E + j];
                ((uint4*)p)[i] = pack(e);
            }
            return;
        }
    } else if constexpr (2 * N == E && sizeof(T) == 2) {
        if (n >= N) {
            *(uint2*)p = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; i++)
        if (i < n) put(p + i, v[i]);
}

// N consecutive elements that are in range as a whole or not at all.
template <class T, int N>
__device__ __forceinline__ void load_whole(const T* p, bool in, float (&v)[N]) {
    if (in) {
        load_n<T, N>(p, N, v);
    } else {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = 0.0f;
    }
}
template <class T, int N>
__device__ __forceinline__ void store_whole(T* p, bool in, const float (&v)[N]) {
    if (in) store_n<T, N>(p, N, v);
}

// Pairs of binary32 numbers, one instruction for both.
struct Pair {
    unsigned long long v;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
    __device__ __forceinline__ void get(float& lo, float& hi) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma_pair(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The id of a token, whatever its width.
__device__ __forceinline__ int64_t load_id(const void* ids, int64_t t, bool wide) {
    return wide ? ((const int64_t*)ids)[t] : (int64_t)((const int32_t*)ids)[t];
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// ---------------------------------------------------------------------------
// clusters
// ---------------------------------------------------------------------------
constexpr int kMaxCluster = 8;
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Write to the same shared-memory variable of another block of the cluster.
__device__ __forceinline__ void store_remote(float* local, unsigned rank, float v) {
    asm volatile(
        "{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %0, %1;\n st.shared::cluster.f32 [r], %2;\n}\n" ::"r"(
            smem_addr(local)),
        "r"(rank), "f"(v)
        : "memory");
}

// Makes freshly initialised barriers visible to the bulk copies.
__device__ __forceinline__ void mbar_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// mbar_wait_bounded without reading the clock when the phase is over.
__device__ __forceinline__ bool mbar_wait_quick(uint64_t* m, unsigned parity, unsigned long long limit_ns) {
    return mbar_try_wait(m, parity) || mbar_wait_bounded(m, parity, limit_ns);
}

// Programmatic dependent launch: the kernel may start while the one before it
// on the stream drains, waits for its results before it touches memory, and
// then lets its own dependent start.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace

inline cudaError_t launch_op(const void* fn, dim3 grid, dim3 block, void** args, size_t smem,
                             cudaStream_t stream, int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace hc
