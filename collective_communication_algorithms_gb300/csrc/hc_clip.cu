// hc_clip.cu -- the norm over all gradients and the gradients scaled by it
// (hc_clip_grads, hc_grad_norm).
//
//   norm = |scale| sqrt(sum g^2),  out = scale min(1, max_norm / (norm + eps)) g
//
// Bound by bytes: every gradient is read for the norm, read again for the
// product, and written.  Two kernels: the first leaves one partial sum a block,
// the second adds those up in every block (in the same order, so all get the same
// factor) and scales.  A block has the same run of the tensors in both and goes
// through it forwards, then backwards, so that what it read last still comes from
// L2.
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
constexpr int kClipBatch = 8;     // 16-byte loads of one thread at a time
constexpr int kClipResident = 4;  // blocks of an SM, whose loads and stores overlap
constexpr int kChunkBytes = 16384;  // tensors are divided among blocks in pieces of this

// A sum of squares: binary32 with the error of every addition kept, and a
// binary64 side for what binary32 squares cannot hold.  Binary64 arithmetic is
// slow here (about two operations a cycle and SM), and is kept to that side.
struct SquareSum {
    float hi, lo;
    double wide;
    // s: the sum of some squares.  Between 2^-90 and 2^80 no square of weight
    // underflowed (one below 2^-126 loses at most 2^-150, against 64 terms that
    // make 2^-90) and no sum of these overflows; outside, the caller squares in
    // binary64.
    static __device__ __forceinline__ bool fits(float s) { return s >= 8.0779357e-28f && s <= 1.2089258e24f; }
    __device__ __forceinline__ void add(float s) {  // two-sum
        const float t = __fadd_rn(hi, s);
        const float b = __fadd_rn(t, -hi);
        lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(hi, -__fadd_rn(t, -b)), __fadd_rn(s, -b)));
        hi = t;
    }
    __device__ __forceinline__ void add(const SquareSum& o) {
        add(o.hi);
        lo = __fadd_rn(lo, o.lo);
        if (o.wide != 0.0) wide += o.wide;  // a NaN is not 0 either
    }
};
static_assert(sizeof(SquareSum) == 16, "a partial sum's place in scratch");

struct ClipTensor {
    uintptr_t in, out;
    uint64_t count : 56;
    uint64_t peel : 3;      // elements before the first 8 that lie on whole 16 bytes
    uint64_t scalar : 1;    // in and out never do at the same place
    uint64_t in_bf : 1, out_bf : 1;
    uint64_t in_place : 1;
};
static_assert(sizeof(ClipTensor) == 24, "ClipTensor layout");

template <int MAXT>
struct ClipParams {
    SquareSum* part;       // partial sums of all launches
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

// Tensor of a chunk: the first whose chunks end behind it.
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

// The squares of up to kClipBatch vectors held in registers.
template <bool BF>
__device__ __forceinline__ void add_vectors(SquareSum& q, const uint4 (&w)[kClipBatch]) {
    float a = 0.0f, b = 0.0f, c = 0.0f, d = 0.0f;
#pragma unroll
    for (int i = 0; i < kClipBatch; i++) {
        float v[BF ? 8 : 4];
        unpack(w[i], v);
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
        unpack(x, v);
#pragma unroll
        for (int j = 0; j < (BF ? 8 : 4); j++) q.wide = fma((double)v[j], (double)v[j], q.wide);
    }
}

// Elements before and behind a tensor's vectors of V, at most 7 each: f(index)
// on a thread of its own.
template <class F>
__device__ __forceinline__ void for_ends(const ClipTensor& t, int V, F f) {
    const uint64_t peel = min((uint64_t)t.peel, (uint64_t)t.count), body = (t.count - peel) / V * V;
    const unsigned tid = threadIdx.x;
    if (tid < peel) f((uint64_t)tid);
    else if (tid >= 8 && tid < 16 && peel + body + tid - 8 < t.count) f(peel + body + tid - 8);
}

// The squares of the chunks [c0, c1) of a tensor.
template <bool BF>
__device__ __forceinline__ void add_chunks(SquareSum& q, const ClipTensor& t, int c0, int c1) {
    constexpr int V = BF ? 8 : 4, CHUNK = kChunkBytes / 16, STEP = kClipThreads * kClipBatch;
    const uint64_t peel = min((uint64_t)t.peel, (uint64_t)t.count), body = (t.count - peel) / V;  // whole vectors
    const uint64_t begin = (uint64_t)c0 * CHUNK, end = min((uint64_t)c1 * CHUNK, body);
    const uint4* base = (const uint4*)(t.in + t.peel * (BF ? 2 : 4)) + begin;
    // vectors of this thread's column; a block's share of any list that fits
    // the memory ends well below 2^31
    const int n = end > begin ? (int)(end - begin) - (int)threadIdx.x : 0;
    base += threadIdx.x;
#pragma unroll 1
    for (int at = 0; at < n; at += STEP) {
        uint4 w[kClipBatch];
#pragma unroll
        for (int i = 0; i < kClipBatch; i++) {
            w[i] = make_uint4(0, 0, 0, 0);
            if (at + i * kClipThreads < n) w[i] = base[at + i * kClipThreads];
        }
        add_vectors<BF>(q, w);
    }
    if (c0 == 0)
        for_ends(t, V, [&](uint64_t i) {
            const double v = load_one(t.in, BF, i);
            q.wide = fma(v, v, q.wide);
        });
}

// The chunks of a block, tensor by tensor: f(tensor, its chunks c0, c1), from
// the first on or from the last.
template <bool FORWARDS, class P, class F>
__device__ __forceinline__ void for_block(const P& p, F f) {
    const int from = (int)((int64_t)p.chunks * blockIdx.x / gridDim.x), to = (int)((int64_t)p.chunks * (blockIdx.x + 1) / gridDim.x);
    if (from >= to) return;
    int k = tensor_of(p, FORWARDS ? from : to - 1);
    for (int c = FORWARDS ? from : to; FORWARDS ? c < to : c > from; k += FORWARDS ? 1 : -1) {
        const int first = k ? p.chunk_end[k - 1] : 0, last = p.chunk_end[k];
        const int lo = max(from, first), hi = min(to, last);
        if (lo < hi) f(p.t[k], lo - first, hi - first);
        c = FORWARDS ? hi : lo;
    }
}

// The sum over `lanes` lanes (a power of two), in the first of them.
__device__ __forceinline__ void lanes_sum(SquareSum& q, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) {
        SquareSum x;
        x.hi = __shfl_down_sync(0xFFFFFFFFu, q.hi, o);
        x.lo = __shfl_down_sync(0xFFFFFFFFu, q.lo, o);
        x.wide = __shfl_down_sync(0xFFFFFFFFu, q.wide, o);
        q.add(x);
    }
}
// The sum over the block's threads, in the first.
__device__ __forceinline__ void block_sum(SquareSum& q) {
    __shared__ SquareSum sh[kClipThreads / 32];
    lanes_sum(q, 32);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = q;
    __syncthreads();
    if (threadIdx.x < 32) {
        q = sh[threadIdx.x % (kClipThreads / 32)];
        lanes_sum(q, kClipThreads / 32);
    }
}

template <int MAXT>
__global__ void __launch_bounds__(kClipThreads, kClipResident) square_kernel(const __grid_constant__ ClipParams<MAXT> p) {
    grid_wait();
    grid_release();
    SquareSum q = {0.0f, 0.0f, 0.0};
    for_block<true>(p, [&](const ClipTensor& t, int c0, int c1) {
        if (t.in_bf) add_chunks<true>(q, t, c0, c1);
        else add_chunks<false>(q, t, c0, c1);
    });
    block_sum(q);
    if (threadIdx.x == 0) p.part[p.first_part + blockIdx.x] = q;
}

struct Factor {
    float norm, factor;
};
// Every block adds the partial sums up in the same order.
template <class P>
__device__ __forceinline__ Factor factor_of(const P& p) {
    __shared__ Factor f;
    SquareSum q = {0.0f, 0.0f, 0.0};
    for (int i = threadIdx.x; i < p.parts; i += kClipThreads) q.add(p.part[i]);
    block_sum(q);
    if (threadIdx.x == 0) {
        const float norm = __fsqrt_rn(__fadd_rn(q.hi, q.lo)), scaled = norm * fabsf(p.scale), limit = p.max_norm;
        // all that follows lies well inside binary32's range
        const auto middling = [](float v) { return v > 1e-18f && v < 1e18f; };
        if (q.wide == 0.0 && middling(scaled) && middling(scaled + p.eps) && middling(fabsf(p.scale)) &&
            (middling(limit) || isinf(limit))) {
            f.norm = scaled;
            f.factor = fminf(1.0f, __fdiv_rn(limit, scaled + p.eps)) * p.scale;
        } else {
            const double n = sqrt(q.wide + (double)q.hi + (double)q.lo) * fabs((double)p.scale);
            double c = isinf(limit) ? 1.0 : (double)limit / (n + (double)p.eps);
            if (c > 1.0) c = 1.0;  // a NaN stays
            f.norm = (float)n;
            f.factor = (float)(c * (double)p.scale);
        }
    }
    __syncthreads();
    return f;
}

// Eight elements, which lie on whole 16 bytes in both tensors.
template <bool BF>
struct Eight {
    uint4 w[BF ? 1 : 2];
    __device__ __forceinline__ void load(const uint4* p, uint64_t policy) {
#pragma unroll
        for (int j = 0; j < (BF ? 1 : 2); j++) w[j] = ld_vec_hint((uintptr_t)(p + j), policy);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (BF) {
            unpack(w[0], v);
        } else {
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = __uint_as_float(u[j]);
        }
    }
};
template <bool IB, bool OB>
__device__ __forceinline__ void scale_eight(const Eight<IB>& x, uint4* out, float f, uint64_t policy) {
    float v[8];
    x.get(v);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] *= f;
    if constexpr (OB) {
        st_vec_hint((uintptr_t)out, pack(v), policy);
    } else {
        const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
        st_vec_hint((uintptr_t)out, pack(lo), policy);
        st_vec_hint((uintptr_t)(out + 1), pack(hi), policy);
    }
}

// The chunks [c0, c1) of a tensor, from the last on.
template <bool IB, bool OB>
__device__ __forceinline__ void scale_chunks(const ClipTensor& t, int c0, int c1, float f, uint64_t policy) {
    constexpr int VI = IB ? 1 : 2, VO = OB ? 1 : 2;                // 16-byte vectors of 8 elements
    constexpr int N = IB ? kClipBatch : kClipBatch / 2, STEP = kClipThreads * N;  // places of a thread, of a step
    constexpr int CHUNK = kChunkBytes / 16 / VI;
    const uint64_t peel = min((uint64_t)t.peel, (uint64_t)t.count), body = (t.count - peel) / 8;
    const uint64_t begin = (uint64_t)c0 * CHUNK, end = min((uint64_t)c1 * CHUNK, body);
    const uint4* in = (const uint4*)(t.in + peel * (IB ? 2 : 4)) + (begin + threadIdx.x) * VI;
    uint4* out = (uint4*)(t.out + peel * (OB ? 2 : 4)) + (begin + threadIdx.x) * VO;
    const int all = end > begin ? (int)(end - begin) : 0;
    const int n = all - (int)threadIdx.x;
    if (n > 0) {
        int at = (all - 1) / STEP * STEP;
        const auto step = [&](bool whole) {
            Eight<IB> x[N];
#pragma unroll
            for (int i = 0; i < N; i++)  // beyond the end: the last place again
                x[i].load(in + (whole ? at + i * kClipThreads : min(at + i * kClipThreads, n - 1)) * VI, policy);
#pragma unroll
            for (int i = 0; i < N; i++)
                if (whole || at + i * kClipThreads < n) scale_eight<IB, OB>(x[i], out + (at + i * kClipThreads) * VO, f, policy);
        };
        step(false);
#pragma unroll 1
        for (at -= STEP; at >= 0; at -= STEP) step(true);
    }
    if (c0 == 0) for_ends(t, 8, [&](uint64_t i) { store_one(t.out, OB, i, load_one(t.in, IB, i) * f); });
}

template <int MAXT>
__global__ void __launch_bounds__(kClipThreads, kClipResident) scale_kernel(const __grid_constant__ ClipParams<MAXT> p) {
    grid_wait();
    grid_release();
    const Factor f = factor_of(p);
    if (p.write_norm && blockIdx.x == 0 && threadIdx.x == 0) {
        *p.norm = f.norm;
        if (p.factor) *p.factor = f.factor;
    }
    // neither what is read for the last time nor what is written stays in L2 in
    // the place of gradients that are still to be read
    const uint64_t policy = l2_evict_first_policy();
    for_block<false>(p, [&](const ClipTensor& t, int c0, int c1) {
        if (t.in_place && f.factor == 1.0f) return;
        if (t.scalar) {
            const uint64_t per = kChunkBytes / (t.in_bf ? 2 : 4), end = min((uint64_t)t.count, c1 * per);
#pragma unroll 4
            for (uint64_t i = c0 * per + threadIdx.x; i < end; i += kClipThreads)
                store_one(t.out, t.out_bf, i, load_one(t.in, t.in_bf, i) * f.factor);
        } else if (t.in_bf) {
            if (t.out_bf) scale_chunks<true, true>(t, c0, c1, f.factor, policy);
            else scale_chunks<true, false>(t, c0, c1, f.factor, policy);
        } else {
            if (t.out_bf) scale_chunks<false, true>(t, c0, c1, f.factor, policy);
            else scale_chunks<false, false>(t, c0, c1, f.factor, policy);
        }
    });
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
constexpr int kClipMaxBlocks = 152 * kClipResident;
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
        const bool i = (t.in + (uintptr_t)(k * is)) % 16 == 0, o = (t.out + (uintptr_t)(k * os)) % 16 == 0;
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
    p.part = (SquareSum*)a.scratch;
    p.norm = a.norm;
    p.factor = a.factor;
    p.first_part = first_part;
    p.parts = parts;
    p.num = (int)n;
    p.chunks = (int)chunks;
    p.scale = a.scale;
    p.max_norm = stage == 2 ? INFINITY : a.max_norm;  // the norm alone
    p.eps = stage == 2 ? 0.0f : a.eps;
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
    return parts * sizeof(SquareSum);
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
