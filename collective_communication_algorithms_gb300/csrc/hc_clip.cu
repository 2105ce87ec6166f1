// hc_clip.cu -- the norm over all gradients and the gradients scaled by it
// (hc_clip_grads, hc_grad_norm).
//
//   norm = |scale| sqrt(sum g^2),  out = scale min(1, max_norm / (norm + eps)) g
//
// Bound by bytes: every gradient is read for the norm, read again for the
// product, and written.  Two kernels: the first leaves one binary64 partial
// sum a block, the second adds those up in every block (in the same order, so
// all get the same factor) and scales.  The second goes through the tensors
// from the end, so that what the first read last still comes from L2.
//
// The tensors' table travels in the kernel's parameters (up to 32 KB), so a
// call needs no copy to the device and can be captured; longer lists take
// several launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "hc_ops.cuh"

namespace hc {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipBatch = 8;        // 16-byte loads of one thread under way
constexpr int kChunkBytes = kClipThreads * kClipBatch * 16;

struct ClipTensor {
    uintptr_t in, out;
    uint64_t count : 56;
    uint64_t peel : 3;      // elements before the first 8 that lie on whole 16 (bf16) or 32 bytes (fp32)
    uint64_t scalar : 1;    // in and out never do at the same place
    uint64_t in_bf : 1, out_bf : 1;
    uint64_t in_place : 1;
};
static_assert(sizeof(ClipTensor) == 24, "ClipTensor layout");

template <int MAXT>
struct ClipParams {
    double* part;          // partial sums of all launches
    float* norm;
    float* factor;
    int first_part;        // of this launch
    int parts;             // of all launches
    int num;
    int chunks;
    float scale, max_norm, eps;
    int write_norm;        // this launch writes norm and factor
    int chunk_end[MAXT];   // chunks up to and with this tensor
    ClipTensor t[MAXT];
};
// Kernel parameters end at 32764 bytes; small lists take a small table, which
// is copied faster at every launch.
constexpr int kFewTensors = 32, kMoreTensors = 256, kMostTensors = 1160;
static_assert(sizeof(ClipParams<kMostTensors>) <= 32764, "kernel parameters");

// Tensor of a chunk: the first whose last chunk lies behind it.
template <class P>
__device__ __forceinline__ int tensor_of(const P& p, int chunk) {
    int lo = 0, hi = p.num - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (chunk < p.chunk_end[mid]) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ float load_one(uintptr_t p, bool bf, uint64_t i) {
    return bf ? to_f32(((const Bf16*)p)[i]) : ((const float*)p)[i];
}
__device__ __forceinline__ void store_one(uintptr_t p, bool bf, uint64_t i, float v) {
    if (bf) put((Bf16*)p + i, v);
    else ((float*)p)[i] = v;
}

// A running sum of squares: binary32 with the error of every addition kept,
// and a binary64 side for what binary32 squares cannot hold.
struct SquareSum {
    float hi = 0.0f, lo = 0.0f;
    double wide = 0.0;
    // s: the sum of some squares.  Between 2^-90 and 2^100 no square of weight
    // underflowed (one below 2^-126 loses at most 2^-150, against 64 terms of
    // 2^-90) and no sum overflows; outside, the caller squares in binary64.
    static __device__ __forceinline__ bool fits(float s) { return s >= 8.0779357e-28f && s <= 1.2676506e30f; }
    __device__ __forceinline__ void add(float s) {  // two-sum
        const float t = __fadd_rn(hi, s);
        const float b = __fadd_rn(t, -hi);
        lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(hi, -__fadd_rn(t, -b)), __fadd_rn(s, -b)));
        hi = t;
    }
    __device__ __forceinline__ double total() const { return wide + (double)hi + (double)lo; }
};

template <bool BF>
__device__ __forceinline__ void words_of(const uint4& w, float (&v)[BF ? 8 : 4]) {
    unpack(w, v);
}

// The squares of up to kClipBatch vectors held in registers.
template <bool BF>
__device__ __forceinline__ void add_vectors(SquareSum& q, const uint4 (&w)[kClipBatch]) {
    float a = 0.0f, b = 0.0f, c = 0.0f, d = 0.0f;
#pragma unroll
    for (int i = 0; i < kClipBatch; i++) {
        float v[BF ? 8 : 4];
        words_of<BF>(w[i], v);
#pragma unroll
        for (int j = 0; j < (BF ? 8 : 4); j += 4) {
            a = fmaf(v[j], v[j], a);
            b = fmaf(v[j + 1], v[j + 1], b);
            c = fmaf(v[j + 2], v[j + 2], c);
            d = fmaf(v[j + 3], v[j + 3], d);
        }
    }
    const float s = (a + b) + (c + d);
    if (SquareSum::fits(s)) {
        q.add(s);
        return;
    }
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kClipBatch; i++) any |= w[i].x | w[i].y | w[i].z | w[i].w;
    if (!(any & (BF ? 0x7FFF7FFFu : 0x7FFFFFFFu))) return;  // zeros
#pragma unroll 1
    for (int i = 0; i < kClipBatch; i++) {
        uint4 x = w[0];
#pragma unroll
        for (int k = 1; k < kClipBatch; k++)
            if (k == i) x = w[k];
        float v[BF ? 8 : 4];
        words_of<BF>(x, v);
#pragma unroll
        for (int j = 0; j < (BF ? 8 : 4); j++) q.wide = fma((double)v[j], (double)v[j], q.wide);
    }
}

template <bool BF>
__device__ __forceinline__ void add_chunk(SquareSum& q, const ClipTensor& t, int chunk_in_tensor) {
    const uint64_t body = (t.count - (t.peel < t.count ? t.peel : t.count)) / (BF ? 8 : 4);  // whole vectors
    const uint4* base = (const uint4*)(t.in + t.peel * (BF ? 2 : 4));
    const uint64_t start = (uint64_t)chunk_in_tensor * (kClipThreads * kClipBatch);
    base += start;
    const int left = (int)min(body > start ? body - start : 0, (uint64_t)(kClipThreads * kClipBatch));
    uint4 w[kClipBatch];
#pragma unroll
    for (int i = 0; i < kClipBatch; i++) {
        const int k = (int)threadIdx.x + i * kClipThreads;
        w[i] = k < left ? base[k] : make_uint4(0, 0, 0, 0);
    }
    add_vectors<BF>(q, w);
    if (chunk_in_tensor == 0) {  // what lies before and behind the vectors: at most 7 elements each
        const int tid = threadIdx.x;
        const uint64_t tail = t.peel + body * (BF ? 8 : 4);
        uint64_t i = t.count;
        if (tid < 8) i = tid < (int)t.peel ? tid : t.count;
        else if (tid < 16) i = tail + tid - 8;
        if (i < t.count) {
            const double v = load_one(t.in, BF, i);
            q.wide = fma(v, v, q.wide);
        }
    }
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double sh[kClipThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kClipThreads / 32; i++) s += sh[i];
    return s;
}

// 64 registers: four blocks an SM.
template <int MAXT>
__global__ void __launch_bounds__(kClipThreads, 4) square_kernel(const __grid_constant__ ClipParams<MAXT> p) {
    grid_wait();
    grid_release();
    SquareSum q;
    for (int c = blockIdx.x; c < p.chunks; c += gridDim.x) {
        const int k = tensor_of(p, c);
        const ClipTensor t = p.t[k];
        const int first = k ? p.chunk_end[k - 1] : 0;
        if (t.in_bf) add_chunk<true>(q, t, c - first);
        else add_chunk<false>(q, t, c - first);
    }
    const double s = block_sum(q.total());
    if (threadIdx.x == 0) p.part[p.first_part + blockIdx.x] = s;
}

struct Factor {
    float norm, factor;
};
// Every block adds the partial sums up in the same order.
template <class P>
__device__ __forceinline__ Factor factor_of(const P& p) {
    double s = 0.0;
    for (int i = threadIdx.x; i < p.parts; i += kClipThreads) s += p.part[i];
    s = block_sum(s);
    const double norm = sqrt(s) * fabs((double)p.scale);
    double c = isinf(p.max_norm) ? 1.0 : (double)p.max_norm / (norm + (double)p.eps);
    if (c > 1.0) c = 1.0;  // a NaN stays
    return Factor{(float)norm, (float)(c * (double)p.scale)};
}

// Eight elements, which lie on whole 16 bytes (bf16) or 32 (fp32).
template <bool BF>
struct Eight {
    uint4 w;
    __device__ __forceinline__ void load(const uint4* p) { w = *p; }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack(w, v); }
};
template <>
struct Eight<false> {
    ulonglong4_32a w;  // one access of 32 bytes
    __device__ __forceinline__ void load(const uint4* p) { w = *(const ulonglong4_32a*)p; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const unsigned long long u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; j++) asm("mov.b64 {%0, %1}, %2;" : "=f"(v[2 * j]), "=f"(v[2 * j + 1]) : "l"(u[j]));
    }
};
template <bool IB, bool OB>
__device__ __forceinline__ void scale_eight(const Eight<IB>& x, uint4* out, float f) {
    float v[8];
    x.get(v);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] *= f;
    if constexpr (OB) {
        *out = pack(v);
    } else {
        unsigned long long u[4];
#pragma unroll
        for (int j = 0; j < 4; j++) asm("mov.b64 %0, {%1, %2};" : "=l"(u[j]) : "f"(v[2 * j]), "f"(v[2 * j + 1]));
        *(ulonglong4_32a*)out = ulonglong4_32a{u[0], u[1], u[2], u[3]};
    }
}

template <bool IB, bool OB>
__device__ __noinline__ void scale_chunk(uintptr_t tin, uintptr_t tout, uint64_t count, unsigned peel, int chunk, float f) {
    constexpr int VI = IB ? 1 : 2, VO = OB ? 1 : 2;      // 16-byte accesses of 8 elements
    constexpr int N = IB ? kClipBatch : kClipBatch / 2;  // places of a thread
    if (peel > count) peel = (unsigned)count;
    const uint64_t body = (count - peel) / 8;
    const uint64_t start = (uint64_t)chunk * (kClipThreads * N);
    const uint4* in = (const uint4*)(tin + peel * (IB ? 2 : 4)) + start * VI;
    uint4* out = (uint4*)(tout + peel * (OB ? 2 : 4)) + start * VO;
    const int left = (int)min(body > start ? body - start : 0, (uint64_t)(kClipThreads * N));
    const int tid = threadIdx.x;
    if (left == kClipThreads * N) {
        Eight<IB> x[N];
#pragma unroll
        for (int i = 0; i < N; i++) x[i].load(in + (tid + i * kClipThreads) * VI);
#pragma unroll
        for (int i = 0; i < N; i++) scale_eight<IB, OB>(x[i], out + (tid + i * kClipThreads) * VO, f);
    } else {
#pragma unroll 1
        for (int k = tid; k < left; k += kClipThreads) {
            Eight<IB> x;
            x.load(in + k * VI);
            scale_eight<IB, OB>(x, out + k * VO, f);
        }
    }
    if (chunk == 0) {
        uint64_t i = count;
        if (tid < 8) i = tid < (int)peel ? tid : count;
        else if (tid < 16) i = peel + body * 8 + tid - 8;
        if (i < count) store_one(tout, OB, i, load_one(tin, IB, i) * f);
    }
}

template <int MAXT>
__global__ void __launch_bounds__(kClipThreads, 4) scale_kernel(const __grid_constant__ ClipParams<MAXT> p) {
    grid_wait();
    grid_release();
    const Factor f = factor_of(p);
    if (p.write_norm && blockIdx.x == 0 && threadIdx.x == 0) {
        *p.norm = f.norm;
        if (p.factor) *p.factor = f.factor;
    }
    for (int c = p.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
        const int k = tensor_of(p, c);
        const ClipTensor t = p.t[k];
        if (t.in_place && f.factor == 1.0f) continue;
        const int n = c - (k ? p.chunk_end[k - 1] : 0);
        if (t.scalar) {
            const uint64_t per = kChunkBytes / (t.in_bf ? 2 : 4);
            const uint64_t end = min((uint64_t)t.count, (uint64_t)(n + 1) * per);
#pragma unroll 4
            for (uint64_t i = (uint64_t)n * per + threadIdx.x; i < end; i += kClipThreads)
                store_one(t.out, t.out_bf, i, load_one(t.in, t.in_bf, i) * f.factor);
        } else if (t.in_bf) {
            if (t.out_bf) scale_chunk<true, true>(t.in, t.out, t.count, t.peel, n, f.factor);
            else scale_chunk<true, false>(t.in, t.out, t.count, t.peel, n, f.factor);
        } else {
            if (t.out_bf) scale_chunk<false, true>(t.in, t.out, t.count, t.peel, n, f.factor);
            else scale_chunk<false, false>(t.in, t.out, t.count, t.peel, n, f.factor);
        }
    }
}

template <int MAXT>
__global__ void __launch_bounds__(kClipThreads) norm_only_kernel(const __grid_constant__ ClipParams<MAXT> p) {
    grid_wait();
    grid_release();
    const Factor f = factor_of(p);
    if (threadIdx.x == 0) *p.norm = f.norm;
}

int64_t chunks_of(const hc_grad_t& g) {
    const uint64_t per = kChunkBytes / elem_bytes(g.in_dtype);
    return (int64_t)((g.count + per - 1) / per);
}

// Launches of a list: runs of tensors that fit a table, and the partial sums
// of each.  A block has at least one chunk, and several once all SMs are full.
constexpr int kClipMaxBlocks = 152 * 4;
int clip_blocks(int64_t chunks) { return (int)std::min<int64_t>(chunks, kClipMaxBlocks); }

template <class F>
cudaError_t for_each_run(const hc_clip_grads_t& a, F f) {
    size_t at = 0;
    do {
        size_t n = 0;
        int64_t chunks = 0;
        while (at + n < a.num && n < (size_t)kMostTensors && chunks + chunks_of(a.tensors[at + n]) <= INT32_MAX / 2) {
            chunks += chunks_of(a.tensors[at + n]);
            n++;
        }
        if (!n && at < a.num) return cudaErrorInvalidValue;
        const cudaError_t e = f(at, n, chunks);
        if (e != cudaSuccess) return e;
        at += n;
    } while (at < a.num);
    return cudaSuccess;
}

ClipTensor describe(const hc_grad_t& g) {
    ClipTensor t;
    std::memset(&t, 0, sizeof t);
    const bool in_place = !g.out || g.out == g.in;
    t.in = (uintptr_t)g.in;
    t.out = (uintptr_t)(in_place ? g.in : g.out);
    t.count = g.count;
    t.in_bf = g.in_dtype == HC_BFLOAT16;
    t.out_bf = in_place ? t.in_bf : g.out_dtype == HC_BFLOAT16;
    t.in_place = in_place;
    const int is = t.in_bf ? 2 : 4, os = t.out_bf ? 2 : 4;
    int peel = -1, in_peel = -1;
    for (int k = 0; k < 8; k++) {
        // eight elements on whole 16 bytes (bf16) or 32 (fp32)
        const bool i = (t.in + (uintptr_t)(k * is)) % (8 * is) == 0, o = (t.out + (uintptr_t)(k * os)) % (8 * os) == 0;
        if (i && in_peel < 0) in_peel = k;
        if (i && o && peel < 0) peel = k;
    }
    t.scalar = peel < 0;
    t.peel = (uint64_t)(peel >= 0 ? peel : in_peel);
    return t;
}

template <int MAXT>
cudaError_t launch_run(const hc_clip_grads_t& a, size_t at, size_t n, int64_t chunks, int stage, int first_part,
                       int parts, bool last, cudaStream_t stream) {
    ClipParams<MAXT> p;
    p.part = (double*)a.scratch;
    p.norm = a.norm;
    p.factor = a.factor;
    p.first_part = first_part;
    p.parts = parts;
    p.num = (int)n;
    p.chunks = (int)chunks;
    p.scale = a.scale;
    p.max_norm = a.max_norm;
    p.eps = a.eps;
    p.write_norm = last;
    int end = 0;
    for (size_t i = 0; i < n; i++) {
        end += (int)chunks_of(a.tensors[at + i]);
        p.chunk_end[i] = end;
        p.t[i] = describe(a.tensors[at + i]);
    }
    void* args[] = {&p};
    const void* fn = stage == 0 ? (const void*)square_kernel<MAXT>
                                : stage == 1 ? (const void*)scale_kernel<MAXT> : (const void*)norm_only_kernel<MAXT>;
    const int blocks = stage == 2 ? 1 : std::max(1, clip_blocks(chunks));
    return launch_op(fn, dim3((unsigned)blocks), dim3(kClipThreads), args, 0, stream);
}

cudaError_t launch_any(const hc_clip_grads_t& a, size_t at, size_t n, int64_t chunks, int stage, int first_part,
                       int parts, bool last, cudaStream_t stream) {
    if (n <= (size_t)kFewTensors) return launch_run<kFewTensors>(a, at, n, chunks, stage, first_part, parts, last, stream);
    if (n <= (size_t)kMoreTensors) return launch_run<kMoreTensors>(a, at, n, chunks, stage, first_part, parts, last, stream);
    return launch_run<kMostTensors>(a, at, n, chunks, stage, first_part, parts, last, stream);
}

}  // namespace

size_t clip_scratch_bytes(const hc_clip_grads_t& a) {
    size_t parts = 0;
    if (for_each_run(a, [&](size_t, size_t, int64_t chunks) {
            parts += (size_t)clip_blocks(chunks);
            return cudaSuccess;
        }) != cudaSuccess)
        return 0;
    return parts * sizeof(double);
}

cudaError_t launch_clip(const hc_clip_grads_t& a, bool apply, cudaStream_t stream) {
    int parts = 0;
    cudaError_t e = for_each_run(a, [&](size_t at, size_t n, int64_t chunks) {
        if (!chunks) return cudaSuccess;
        const int first = parts;
        parts += clip_blocks(chunks);
        return launch_any(a, at, n, chunks, 0, first, 0, false, stream);
    });
    if (e != cudaSuccess) return e;
    if (!apply) return launch_any(a, 0, 0, 0, 2, 0, parts, true, stream);
    bool first_run = true;
    return for_each_run(a, [&](size_t at, size_t n, int64_t chunks) {
        const bool writes = first_run;
        if (!chunks && !writes) return cudaSuccess;
        first_run = false;
        return launch_any(a, at, n, chunks, 1, 0, parts, writes, stream);
    });
}

}  // namespace hc
