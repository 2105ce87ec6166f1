// hc_distill.cu -- distillation from a teacher's top logits, with its
// gradient.
//
// Per row, with c = log2(e) / temperature: q_j = 2^((x_j - m) c) / l, m the
// row's largest logit and l the sum of the numerators.  The loss needs m and
// l and the few logits that the teacher names; the gradient needs every x_j
// again.  A row is therefore held in shared memory between the two, split
// over the blocks of a cluster (a row of 131072 bf16 logits is 256 KB), so
// that it is read once and its gradient written once.  Bulk copies bring a
// block's share in; the threads reduce each piece as it lands, rescaling
// their running sums when their maximum grows; the blocks exchange (m, l)
// through distributed shared memory and write the gradient.
//
// Rows need not start on 16-byte boundaries: a share is a run of aligned
// 16-byte vectors of memory, the vectors that also hold a neighbouring row's
// elements (or lie past the matrix) are fetched element by element, the
// foreign elements set to -inf.
#include "hc_ops.cuh"

namespace hc {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPieces = 16;  // bulk copies (and barriers) of a share at most

struct DistillParams {
    const void* logits;
    const void* teacher;
    const void* ids;
    const float* weight;
    float* loss;
    float* stats;
    void* grad;
    int64_t tokens, logits_stride, teacher_stride, grad_stride;
    int vocab, top, cs;
    int share;        // vectors of a block's share
    int piece;        // vectors of one bulk copy
    bool wide_ids, bf16_teacher;
    float temperature, scale;
    int* err;
    unsigned long long wait_ns;
    int hold;
};

struct Shared {
    uint64_t full[kPieces];
    float warp_m[kWarps], warp_l[kWarps];
    float rank_m[8], rank_l[8];
    int failed;
    int entries;     // of the row, valid ones
    float t_top, t_log;  // teacher: largest logit, log of its sum
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Joins the lanes' (maximum, sum of 2^((x - maximum) c)) of a warp.
__device__ __forceinline__ void warp_join(float& m, float& l, float c) {
    const float mx = warp_max(m);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    l = warp_sum(l * exp2_fast((m - ref) * c));
    m = mx;
}

__device__ __forceinline__ float teacher_logit(const DistillParams& p, int64_t at) {
    return p.bf16_teacher ? to_f32(((const Bf16*)p.teacher)[at]) : ((const float*)p.teacher)[at];
}

// One warp: the row's entries -> ids (-1: none) and probabilities in shared
// memory.  Returns the number of entries with a probability.
__device__ int teacher_softmax(const DistillParams& p, int64_t t, float c, int* ids, float* prob, Shared& sh) {
    const int lane = threadIdx.x & 31;
    float top = -INFINITY;
    int n = 0;
    for (int k = lane; k < p.top; k += 32) {
        const int64_t id = load_id(p.ids, t * p.teacher_stride + k, p.wide_ids);
        const float v = teacher_logit(p, t * p.teacher_stride + k);
        const bool has = id >= 0 && id < p.vocab && v != -INFINITY;
        ids[k] = has ? (int)id : -1;
        prob[k] = v;
        if (has) {
            top = v > top || v != v ? v : top;
            n++;
        }
    }
    top = warp_max(top);
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    float sum = 0.0f;
    for (int k = lane; k < p.top; k += 32) {
        const float v = ids[k] >= 0 ? exp2_fast((prob[k] - top) * c) : 0.0f;
        sum += v;
    }
    sum = warp_sum(sum);
    for (int k = lane; k < p.top; k += 32)
        prob[k] = ids[k] >= 0 ? exp2_fast((prob[k] - top) * c) / sum : 0.0f;
    if (lane == 0) {
        sh.t_top = top;
        sh.t_log = logf(sum);
        sh.entries = n;
    }
    return n;
}

// A row's 16-byte vectors: vector i holds elements [i E - shift, i E - shift + E).
template <class T>
struct Window {
    static constexpr int E = kVecOf<T>;
    uintptr_t base;  // of vector 0, 16-byte aligned
    int shift;       // elements of vector 0 that precede the row
    int count;       // vectors
    int len;         // elements of the row
    __device__ __forceinline__ Window(const void* row, int n) {
        base = (uintptr_t)row & ~(uintptr_t)15;
        shift = (int)(((uintptr_t)row & 15) / sizeof(T));
        count = (shift + n + E - 1) / E;
        len = n;
    }
    __device__ __forceinline__ bool whole(int i) const { return i * E >= shift && (i + 1) * E - shift <= len; }
    // first and one past the last whole vector
    __device__ __forceinline__ int whole_lo() const { return shift ? 1 : 0; }
    __device__ __forceinline__ int whole_hi() const { return (shift + len) / E; }
};

template <class T>
__device__ __forceinline__ void edge_vector(const Window<T>& w, int i, float (&v)[kVecOf<T>]) {
#pragma unroll
    for (int j = 0; j < kVecOf<T>; j++) {
        const int e = i * kVecOf<T> - w.shift + j;
        v[j] = e >= 0 && e < w.len ? to_f32(((const T*)w.base)[i * kVecOf<T> + j]) : -INFINITY;
    }
}

// Store the gradient of vector i: whole vectors where the gradient's row has
// the logits' alignment, elements otherwise.
template <class T>
__device__ __forceinline__ void store_grad(const Window<T>& w, T* row, bool same, int i, const float (&v)[kVecOf<T>]) {
    T* q = row + (i * kVecOf<T> - w.shift);
    if (same && w.whole(i)) {
        *(uint4*)q = pack(v);
        return;
    }
#pragma unroll
    for (int j = 0; j < kVecOf<T>; j++) {
        const int e = i * kVecOf<T> - w.shift + j;
        if (e >= 0 && e < w.len) put(q + j, v[j]);
    }
}

// Zero gradient of a row without loss: vectors [lo, hi).
template <class T>
__device__ __forceinline__ void zero_grad(const Window<T>& w, T* row, bool same, int lo, int hi) {
    const float z[kVecOf<T>] = {};
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) store_grad<T>(w, row, same, i, z);
}

// Gradient of the entries this block's vectors [lo, hi) hold, over what the
// block has stored: g * (q - sum of the p with the same id).  x_of(k): the
// logit of entry k.
template <class T, class X>
__device__ __forceinline__ void entry_grads(const DistillParams& p, const Window<T>& w, T* row, int lo, int hi,
                                            const int* ids, const float* prob, float m, float l_inv, float c, float g,
                                            X x_of) {
    for (int k = threadIdx.x; k < p.top; k += kThreads) {
        const int id = ids[k];
        if (id < 0) continue;
        const int i = (w.shift + id) / kVecOf<T>;
        if (i < lo || i >= hi) continue;
        float sum = 0.0f;
        for (int o = 0; o < p.top; o++) sum += ids[o] == id ? prob[o] : 0.0f;
        put(row + id, g * (exp2_fast((x_of(k) - m) * c) * l_inv - sum));
    }
}

// MODE 0: the loss, 1: the loss and the gradient (DISTILL_LOSS, DISTILL_BOTH).
template <class T, int MODE>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillParams p) {
    constexpr int E = kVecOf<T>;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ Shared sh;
    uint4* const buf = (uint4*)dyn;
    int* const ids = (int*)(buf + p.share);
    float* const prob = (float*)(ids + p.top);
    float* const named = prob + p.top;  // block 0: the logits the teacher names
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = blockIdx.x % p.cs;
    const int64_t t = blockIdx.x / p.cs;
    const float c = 1.4426950408889634f / p.temperature;
    if (p.cs > 1) cluster_arrive();
    if (tid == 0) {
        for (int i = 0; i < kPieces; i++) mbar_init(&sh.full[i], 1 + (i == 0 ? p.hold : 0));
        sh.failed = 0;
        mbar_init_fence();
    }
    __syncthreads();
    grid_wait();
    grid_release();
    const float wt = p.scale * (p.weight ? p.weight[t] : 1.0f);
    const Window<T> w((const T*)p.logits + t * p.logits_stride, p.vocab);
    T* const grow = (T*)p.grad + t * p.grad_stride;
    const bool same = (((uintptr_t)grow ^ (uintptr_t)((const T*)p.logits + t * p.logits_stride)) & 15) == 0;
    const int lo = min((int)rank * p.share, w.count), hi = min(lo + p.share, w.count);
    if (wt == 0.0f) {  // the same in every block of the cluster
        if (p.cs > 1) cluster_wait();
        if (MODE == DISTILL_BOTH) zero_grad<T>(w, grow, same, lo, hi);
        if (rank == 0 && tid == 0) {
            p.loss[t] = 0.0f;
            if (p.stats) p.stats[2 * t] = p.stats[2 * t + 1] = 0.0f;
        }
        return;
    }
    // whole vectors of the share by bulk copies, the edges by hand
    const int wlo = max(lo, w.whole_lo()), whi = max(wlo, min(hi, w.whole_hi()));
    const int pieces = (whi - wlo + p.piece - 1) / p.piece;
    if (tid == 0) {
        for (int i = 0; i < pieces; i++) {
            const int a = wlo + i * p.piece, n = min(p.piece, whi - a);
            mbar_arrive_expect_tx(&sh.full[i], (unsigned)n * 16);
            bulk_g2s(buf + (a - lo), w.base + (uintptr_t)a * 16, (unsigned)n * 16, &sh.full[i]);
        }
    }
    if (tid >= 32 && tid < 64) {
        const int i = tid == 32 ? lo : tid == 33 ? hi - 1 : -1;
        if (i >= lo && i < hi && (i < wlo || i >= whi)) {
            float v[E];
            edge_vector<T>(w, i, v);
            buf[i - lo] = pack(v);
        }
    }
    if (warp == 0) {
        teacher_softmax(p, t, c, ids, prob, sh);
        __syncwarp();
        if (rank == 0)
            for (int k = lane; k < p.top; k += 32)
                named[k] = ids[k] >= 0 ? to_f32(((const T*)p.logits + t * p.logits_stride)[ids[k]]) : 0.0f;
    }
    __syncthreads();
    // running maximum and sum of this thread's vectors
    float m = -INFINITY, l = 0.0f;
    auto take = [&](const uint4& u) {
        float v[E];
        unpack(u, v);
        float mx = v[0];
#pragma unroll
        for (int j = 1; j < E; j++) mx = fmaxf(mx, v[j]);
        if (mx > m) {
            l *= exp2_fast((m - mx) * c);  // 0 * 2^-inf at first
            m = mx;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int j = 0; j < E; j++) l += exp2_fast((v[j] - ref) * c);
    };
    if (tid == 0 && lo < wlo) take(buf[0]);
    if (tid == 32 && whi < hi && !(hi - 1 == lo && lo < wlo)) take(buf[hi - 1 - lo]);
    bool ok = true;
    for (int i = 0; i < pieces && ok; i++) {
        if (!mbar_wait_quick(&sh.full[i], 0, i == 0 ? p.wait_ns : kWaitLimitNs)) {
            mbar_expired(&sh.full[i], p.err, i == 0 ? p.hold : 0, tid == 0);
            ok = false;
            break;
        }
        const int a = wlo + i * p.piece - lo, b = min(a + p.piece, whi - lo);
        for (int j = a + tid; j < b; j += kThreads) take(buf[j]);
    }
    if (!ok) {
        for (int i = 0; i < pieces; i++) mbar_wait_bounded(&sh.full[i], 0, kWaitLimitNs);
        sh.failed = 1;
    }
    warp_join(m, l, c);
    if (lane == 0) {
        sh.warp_m[warp] = m;
        sh.warp_l[warp] = l;
    }
    __syncthreads();
    m = lane < kWarps ? sh.warp_m[lane] : -INFINITY;
    l = lane < kWarps ? sh.warp_l[lane] : 0.0f;
    warp_join(m, l, c);
    if (p.cs > 1) {
        cluster_wait();  // every block of the cluster has started
        if (tid < p.cs) {
            store_remote(&sh.rank_m[rank], tid, m);
            store_remote(&sh.rank_l[rank], tid, l);
        }
        cluster_arrive();
        cluster_wait();
        m = lane < p.cs ? sh.rank_m[lane] : -INFINITY;
        l = lane < p.cs ? sh.rank_l[lane] : 0.0f;
        warp_join(m, l, c);
    }
    if (sh.failed) return;
    const bool empty = sh.entries == 0;
    if (rank == 0 && warp == 0) {
        float sum = 0.0f;
        const float log_l = logf(l), inv_t = 1.0f / p.temperature;
        for (int k = lane; k < p.top; k += 32) {
            const float q = prob[k];
            if (ids[k] >= 0 && q != 0.0f) {
                const float tv = teacher_logit(p, t * p.teacher_stride + k);
                sum += q * (((tv - sh.t_top) * inv_t - sh.t_log) - ((named[k] - m) * inv_t - log_l));
            }
        }
        sum = warp_sum(sum);
        if (lane == 0) {
            p.loss[t] = empty ? 0.0f : wt * p.temperature * p.temperature * sum;
            if (p.stats) {
                p.stats[2 * t] = empty ? 0.0f : m;
                p.stats[2 * t + 1] = empty ? 0.0f : l;
            }
        }
    }
    if (MODE != DISTILL_BOTH) return;
    if (empty) {
        zero_grad<T>(w, grow, same, lo, hi);
        return;
    }
    const float g = wt * p.temperature, l_inv = 1.0f / l, gl = g * l_inv;
    for (int i = lo + tid; i < hi; i += kThreads) {
        float v[E];
        unpack(buf[i - lo], v);
#pragma unroll
        for (int j = 0; j < E; j++) v[j] = exp2_fast((v[j] - m) * c) * gl;
        store_grad<T>(w, grow, same, i, v);
    }
    __syncthreads();
    entry_grads<T>(p, w, grow, lo, hi, ids, prob, m, l_inv, c, g, [&](int k) {
        return to_f32(((const T*)(buf))[w.shift + ids[k] - lo * E]);
    });
}

// The gradient alone, from stats: blocks of `share` vectors, independent.
template <class T>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(const DistillParams p) {
    constexpr int E = kVecOf<T>;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ Shared sh;
    int* const ids = (int*)dyn;
    float* const prob = (float*)(ids + p.top);
    float* const named = prob + p.top;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x / p.cs;
    const float c = 1.4426950408889634f / p.temperature;
    grid_wait();
    grid_release();
    const float wt = p.scale * (p.weight ? p.weight[t] : 1.0f);
    const T* const row = (const T*)p.logits + t * p.logits_stride;
    const Window<T> w(row, p.vocab);
    T* const grow = (T*)p.grad + t * p.grad_stride;
    const bool same = (((uintptr_t)grow ^ (uintptr_t)row) & 15) == 0;
    const int lo = min((int)(blockIdx.x % p.cs) * p.share, w.count), hi = min(lo + p.share, w.count);
    if (wt == 0.0f) {
        zero_grad<T>(w, grow, same, lo, hi);
        return;
    }
    if (warp == 0) {
        teacher_softmax(p, t, c, ids, prob, sh);
        __syncwarp();
        // in place, only this block's own elements are still as they were
        for (int k = lane; k < p.top; k += 32) {
            const int i = ids[k] >= 0 ? (w.shift + ids[k]) / E : -1;
            named[k] = i >= lo && i < hi ? to_f32(row[ids[k]]) : 0.0f;
        }
    }
    __syncthreads();
    if (sh.entries == 0) {
        zero_grad<T>(w, grow, same, lo, hi);
        return;
    }
    const float m = p.stats[2 * t], l_inv = 1.0f / p.stats[2 * t + 1];
    const float g = wt * p.temperature, gl = g * l_inv;
    constexpr int B = 4;  // vectors in flight
    for (int i0 = lo + tid; i0 < hi; i0 += B * kThreads) {
        float v[B][E];
#pragma unroll
        for (int b = 0; b < B; b++) {
            const int i = i0 + b * kThreads;
            if (i >= hi) break;
            if (w.whole(i)) unpack(*(const uint4*)(w.base + (uintptr_t)i * 16), v[b]);
            else edge_vector<T>(w, i, v[b]);
        }
#pragma unroll
        for (int b = 0; b < B; b++) {
            const int i = i0 + b * kThreads;
            if (i >= hi) break;
#pragma unroll
            for (int j = 0; j < E; j++) v[b][j] = exp2_fast((v[b][j] - m) * c) * gl;
            store_grad<T>(w, grow, same, i, v[b]);
        }
    }
    __syncthreads();
    entry_grads<T>(p, w, grow, lo, hi, ids, prob, m, l_inv, c, g, [&](int k) { return named[k]; });
}

// Shared memory of a block's share: three blocks fit an SM.
constexpr int kShareBytes = 64 << 10;
constexpr int kMaxShareBytes = 200 << 10;

}  // namespace

cudaError_t launch_distill(const hc_distill_t& a, DistillMode mode, cudaStream_t stream, int sms) {
    DistillParams p = {};
    p.logits = a.logits;
    p.teacher = a.teacher_logits;
    p.ids = a.teacher_ids;
    p.weight = a.row_weight;
    p.loss = a.loss;
    p.stats = a.stats;
    p.grad = a.grad_logits;
    p.tokens = (int64_t)a.tokens;
    p.logits_stride = (int64_t)a.logits_stride;
    p.teacher_stride = (int64_t)a.teacher_stride;
    p.grad_stride = (int64_t)a.grad_stride;
    p.vocab = (int)a.vocab;
    p.top = (int)a.top;
    p.wide_ids = a.id_type == HC_ID64;
    p.bf16_teacher = a.teacher_dtype == HC_BFLOAT16;
    p.temperature = a.temperature;
    p.scale = a.scale;
    const bool bf = a.dtype == HC_BFLOAT16;
    const int E = bf ? 8 : 4;
    const int vecs = (p.vocab + 2 * E - 2) / E;  // of a row at any alignment
    void* args[] = {&p};
    const int entry_bytes = p.top * 12;
    if (mode == DISTILL_GRAD) {
        p.share = 4 * kThreads;
        p.cs = (vecs + p.share - 1) / p.share;
        const int64_t grid = p.tokens * p.cs;
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        const void* fn = bf ? (const void*)distill_grad_kernel<Bf16> : (const void*)distill_grad_kernel<float>;
        return launch_op(fn, dim3((unsigned)grid), dim3(kThreads), args, (size_t)entry_bytes, stream);
    }
    p.cs = 1;
    while (p.cs < 8 && ((int64_t)vecs * 16 > (int64_t)kShareBytes * p.cs ||
                        (p.tokens * p.cs < sms && vecs / p.cs > kThreads)))
        p.cs *= 2;
    p.share = (vecs + p.cs - 1) / p.cs;
    if (p.share * 16 > kMaxShareBytes) return cudaErrorInvalidValue;
    p.piece = (p.share + kPieces - 1) / kPieces;
    if (p.piece < kThreads) p.piece = kThreads;
    p.err = device_error_flag();
    if (!p.err) return cudaErrorInvalidValue;
    p.hold = expiring_waits() ? 1 : 0;
    p.wait_ns = p.hold ? kTestWaitLimitNs : kWaitLimitNs;
    const void* fn = mode == DISTILL_BOTH
                         ? (bf ? (const void*)distill_kernel<Bf16, DISTILL_BOTH> : (const void*)distill_kernel<float, DISTILL_BOTH>)
                         : (bf ? (const void*)distill_kernel<Bf16, DISTILL_LOSS> : (const void*)distill_kernel<float, DISTILL_LOSS>);
    const int smem = p.share * 16 + entry_bytes;
    if (!allow_smem((void*)fn, smem)) return cudaErrorInvalidValue;
    const int64_t grid = p.tokens * p.cs;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_op(fn, dim3((unsigned)grid), dim3(kThreads), args, (size_t)smem, stream, p.cs);
}

}  // namespace hc
