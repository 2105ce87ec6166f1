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
// through distributed shared memory and write the gradient.  A warp of its own
// starts the copies and works on the teacher's entries meanwhile: their
// probabilities, the loss, and the gradient where they point, which it stores
// over the others' when those are done.
//
// Rows need not start on 16-byte boundaries: a share is a run of aligned
// 16-byte vectors of memory, the vectors that also hold a neighbouring row's
// elements (or lie past the matrix) are fetched element by element, the
// foreign elements set to -inf.
//
// What bounds it: one pass over the logits and one over the gradient, 2.15 GB
// for 4096 x 131072 bf16, 317 us at the copy bandwidth.  Measured: 360 us
// (6.0 TB/s) with a tenth of the rows masked off, 384 us with none; the
// instructions (13 an element: unpack, maximum, two exponentials, three sums
// and products, pack) take half of the issue slots, and the chain of waits in
// a cluster (copies, block sum, (m, l) of the others, stores) is covered by
// the other five blocks of an SM.  That is why four vectors are taken at a
// time (one comparison with the running maximum; 409 us with single vectors),
// pairs of binary32 go through one instruction, and blocks are small.  With no
// row masked, where six blocks an SM take 384 us, five take 444, and six with
// prefetches of later rows into L2 take 414.  One row a cluster measured faster
// than clusters that keep rows in registers and work through many (570 us
// against 428 at the time: one row under way is too few).
#include "hc_ops.cuh"

namespace hc {
namespace {

constexpr int kThreads = 128;               // that go through the logits
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = kThreads + 32;       // and the teacher's warp
constexpr int kResident = 6;                // blocks of an SM
constexpr int kPieces = 16;  // bulk copies (and barriers) of a share at most
constexpr int kUnroll = 4;   // vectors that a thread takes at a time

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
    bool in_place;    // the gradient replaces the logits
};

struct Shared {
    uint64_t full[kPieces];
    float warp_m[kWarps], warp_l[kWarps];
    float rank_m[kMaxCluster], rank_l[kMaxCluster];
    int failed;
    int entries;     // of the row, valid ones
    float t_top, t_log;  // teacher: largest logit, log of its sum
};

// 2^x within 2^-22 of itself, and 0 where it is below 2^-126: one instruction,
// since two exponentials an element are what counts beside the memory.  The
// gradient's own error in binary32 is then about 1e-7 of a row's largest; next to
// a row's largest term of 1, what is taken as 0 changes no sum.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ Pair exp2_pair(Pair a) {
    float lo, hi;
    a.get(lo, hi);
    return Pair(exp2_fast(lo), exp2_fast(hi));
}
// A 16-byte vector as pairs, and its largest element (NaN left out).
__device__ __forceinline__ void pairs_of(const uint4& u, Pair (&v)[2]) {
    v[0] = Pair(__uint_as_float(u.x), __uint_as_float(u.y));
    v[1] = Pair(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ void pairs_of(const uint4& u, Pair (&v)[4]) {
    v[0] = Pair(bf_lo(u.x), bf_hi(u.x));
    v[1] = Pair(bf_lo(u.y), bf_hi(u.y));
    v[2] = Pair(bf_lo(u.z), bf_hi(u.z));
    v[3] = Pair(bf_lo(u.w), bf_hi(u.w));
}
__device__ __forceinline__ uint4 pack_pairs(const Pair (&v)[2]) {
    float a, b, c, d;
    v[0].get(a, b);
    v[1].get(c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}
__device__ __forceinline__ uint4 pack_pairs(const Pair (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float a, b;
        v[i].get(a, b);
        w[i] = pack_bf16x2(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <class T>
__device__ __forceinline__ float largest(const uint4& u) {
    if (sizeof(T) == 2) {
        const uint32_t m = max_bf16x2(max_bf16x2(u.x, u.y), max_bf16x2(u.z, u.w));
        return fmaxf(bf_lo(m), bf_hi(m));
    }
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}
// Waits of the threads that go through the logits, and of the teacher's warp
// for them.
__device__ __forceinline__ void logits_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void stored_arrive() { asm volatile("bar.arrive 2, %0;" ::"n"(kBlock) : "memory"); }
__device__ __forceinline__ void stored_wait() { asm volatile("bar.sync 2, %0;" ::"n"(kBlock) : "memory"); }

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
    for (int i = lo + threadIdx.x; i < hi; i += kBlock) store_grad<T>(w, row, same, i, z);
}

__host__ __device__ inline int bucket_count(int top) {
    int n = 64;
    while (n < 4 * top) n *= 2;
    return n;
}

// The teacher's warp: gradient of the entries that this block's vectors [lo,
// hi) hold, g * (q - sum of the p with the same id), kept in prob's place until
// the other threads have stored theirs.  x_of(k): the logit of entry k.
template <class T, class X>
__device__ __forceinline__ void entry_grads(const DistillParams& p, const Window<T>& w, T* row, int lo, int hi,
                                            const int* ids, const float* prob, float* value, int* buckets, float m,
                                            float l_inv, float c, float g, X x_of) {
    const int lane = threadIdx.x & 31, mask = bucket_count(p.top) - 1;
    // entries by a hash of their id: only one that shares its bucket can have
    // a twin, and looks for it among all
    auto bucket = [&](int id) { return (int)((unsigned)id * 2654435761u >> 16) & mask; };
    for (int i = lane; i <= mask; i += 32) buckets[i] = 0;
    __syncwarp();
    for (int k = lane; k < p.top; k += 32)
        if (ids[k] >= 0) atomicAdd(&buckets[bucket(ids[k])], 1);
    __syncwarp();
    for (int k = lane; k < p.top; k += 32) {
        const int id = ids[k], i = id < 0 ? -1 : (w.shift + id) / kVecOf<T>;
        if (i < lo || i >= hi) continue;
        float sum = prob[k];
        if (buckets[bucket(id)] > 1) {
            sum = 0.0f;
            for (int o = 0; o < p.top; o++) sum += ids[o] == id ? prob[o] : 0.0f;
        }
        value[k] = g * (exp2_fast((x_of(k) - m) * c) * l_inv - sum);
    }
    stored_wait();
    for (int k = lane; k < p.top; k += 32) {
        const int id = ids[k], i = id < 0 ? -1 : (w.shift + id) / kVecOf<T>;
        if (i >= lo && i < hi) put(row + id, value[k]);
    }
}

// Gradient of the other columns: 2^((x - m) c) * gl.  What is rounded to bf16
// takes the exponent as x c - m c (ROUGH) where m c is small: it is off by half
// a unit of binary32, at most 2^-17 there, the result by 5e-6 of itself, far
// below a bf16 rounding.  Larger ones (a row of the type's lowest value would
// overflow) and binary32 results take the difference first.
constexpr float kRoughLimit = 256.0f;
template <class T>
__device__ __forceinline__ bool rough_exponents(float m, float c) {
    return sizeof(T) == 2 && fabsf(m * c) < kRoughLimit;
}
template <class T, bool ROUGH>
__device__ __forceinline__ uint4 column_grads(const uint4& u, Pair minus_m, Pair minus_mc, Pair c, Pair gl) {
    Pair v[kVecOf<T> / 2];
    pairs_of(u, v);
#pragma unroll
    for (int j = 0; j < kVecOf<T> / 2; j++)
        v[j] = exp2_pair(ROUGH ? fma_pair(v[j], c, minus_mc) : (v[j] + minus_m) * c) * gl;
    return pack_pairs(v);
}
template <class T>
__device__ __forceinline__ void store_vector(const Window<T>& w, T* row, bool same, int i, const uint4& u) {
    if (same) {
        *(uint4*)(row + (i * kVecOf<T> - w.shift)) = u;
    } else {
        float v[kVecOf<T>];
        unpack(u, v);
#pragma unroll
        for (int j = 0; j < kVecOf<T>; j++) put(row + (i * kVecOf<T> - w.shift) + j, v[j]);
    }
}

// MODE 0: the loss, 1: the loss and the gradient (DISTILL_LOSS, DISTILL_BOTH).
template <class T, int MODE>
__global__ void __launch_bounds__(kBlock, kResident) distill_kernel(const DistillParams p) {
    constexpr int E = kVecOf<T>;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ Shared sh;
    uint4* const buf = (uint4*)dyn;
    int* const ids = (int*)(buf + p.share);
    float* const prob = (float*)(ids + p.top);
    float* const named = prob + p.top;  // block 0: the logits the teacher names; then entries' gradients
    int* const buckets = (int*)(named + p.top);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool teacher = warp == kWarps;
    const unsigned rank = blockIdx.x % p.cs;
    const int64_t t = blockIdx.x / p.cs;
    const float c = 1.4426950408889634f / p.temperature;
    if (p.cs > 1) cluster_arrive_relaxed();
    grid_wait();
    grid_release();
    const float wt = p.scale * (p.weight ? p.weight[t] : 1.0f);
    if (tid == 0) {
        for (int i = 0; i < kPieces; i++) mbar_init(&sh.full[i], 1 + (i == 0 ? p.hold : 0));
        sh.failed = 0;
        mbar_init_fence();
    }
    __syncthreads();
    const T* const row = (const T*)p.logits + t * p.logits_stride;
    const Window<T> w(row, p.vocab);
    T* const grow = (T*)p.grad + t * p.grad_stride;
    const bool same = (((uintptr_t)grow ^ (uintptr_t)row) & 15) == 0;
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
    float m = -INFINITY, l = 0.0f;
    if (teacher) {
        if (lane < pieces) {  // kPieces <= 32
            const int a = wlo + lane * p.piece, n = min(p.piece, whi - a);
            mbar_arrive_expect_tx(&sh.full[lane], (unsigned)n * 16);
            bulk_g2s(buf + (a - lo), w.base + (uintptr_t)a * 16, (unsigned)n * 16, &sh.full[lane]);
        }
        __syncwarp();
        teacher_softmax(p, t, c, ids, prob, sh);
        __syncwarp();
        if (rank == 0)
            for (int k = lane; k < p.top; k += 32) named[k] = ids[k] >= 0 ? to_f32(row[ids[k]]) : 0.0f;
    } else {
        // running maximum and sum of this thread's vectors
        Pair sum(0.0f, 0.0f);
        const Pair cc(c, c);
        auto take = [&](const uint4* u, int n, int step) {  // n vectors, `step` apart; kUnroll or fewer
            uint4 x[kUnroll];
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < kUnroll; k++)
                if (k < n) {
                    x[k] = u[k * step];
                    mx = fmaxf(mx, largest<T>(x[k]));
                }
            if (mx > m) {
                const float f = exp2_fast((m - mx) * c);  // 0 at first
                sum = sum * Pair(f, f);
                m = mx;
            }
            const float ref = m == -INFINITY ? 0.0f : -m;
            const Pair minus(ref, ref);
#pragma unroll
            for (int k = 0; k < kUnroll; k++)
                if (k < n) {
                    Pair v[E / 2];
                    pairs_of(x[k], v);
#pragma unroll
                    for (int j = 0; j < E / 2; j++) sum = sum + exp2_pair((v[j] + minus) * cc);
                }
        };
        const int edge = tid == 0 && lo < wlo ? lo : tid == 32 && whi < hi && !(hi - 1 == lo && lo < wlo) ? hi - 1 : -1;
        if (edge >= 0) {
            float v[E];
            edge_vector<T>(w, edge, v);
            buf[edge - lo] = pack(v);
            take(buf + (edge - lo), 1, 0);
        }
        bool ok = true;
        for (int i = 0; i < pieces; i++) {
            if (!mbar_wait_quick(&sh.full[i], 0, i == 0 ? p.wait_ns : kWaitLimitNs)) {
                mbar_expired(&sh.full[i], p.err, i == 0 ? p.hold : 0, tid == 0);
                ok = false;
                break;
            }
            const int a = wlo + i * p.piece - lo, b = min(a + p.piece, whi - lo);
            for (int j = a + tid; j < b; j += kUnroll * kThreads) {
                const int n = (b - j + kThreads - 1) / kThreads;
                if (n >= kUnroll) take(buf + j, kUnroll, kThreads);
                else take(buf + j, n, kThreads);
            }
        }
        if (!ok) {
            for (int i = 0; i < pieces; i++) mbar_wait_bounded(&sh.full[i], 0, kWaitLimitNs);
            sh.failed = 1;
            __threadfence_block();
        }
        float l2;
        sum.get(l, l2);
        l += l2;
        warp_join(m, l, c);
        if (lane == 0) {
            sh.warp_m[warp] = m;
            sh.warp_l[warp] = l;
        }
        logits_sync();
        m = lane < kWarps ? sh.warp_m[lane] : -INFINITY;
        l = lane < kWarps ? sh.warp_l[lane] : 0.0f;
        warp_join(m, l, c);
    }
    // the row's (m, l), and the teacher's entries, to every thread
    if (p.cs > 1) cluster_wait();  // every block of the cluster has started
    if (tid < p.cs) {
        if (p.cs > 1) {
            store_remote(&sh.rank_m[rank], tid, m);
            store_remote(&sh.rank_l[rank], tid, l);
        } else {
            sh.rank_m[0] = m;
            sh.rank_l[0] = l;
        }
    }
    __syncwarp();
    if (p.cs > 1) {
        // only these two warps have something for others (a releasing arrival
        // waits for what its warp has under way)
        if (warp == 0 || teacher) cluster_arrive();
        else cluster_arrive_relaxed();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (sh.failed) return;
    m = lane < p.cs ? sh.rank_m[lane] : -INFINITY;
    l = lane < p.cs ? sh.rank_l[lane] : 0.0f;
    warp_join(m, l, c);
    const bool empty = sh.entries == 0;
    if (rank == 0 && teacher) {
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
    if (teacher) {
        __syncwarp();
        entry_grads<T>(p, w, grow, lo, hi, ids, prob, named, buckets, m, l_inv, c, g, [&](int k) {
            return to_f32(((const T*)(buf))[w.shift + ids[k] - lo * E]);
        });
        return;
    }
    const Pair minus(-m, -m), minus_c(-m * c, -m * c), cc(c, c), gg(gl, gl);
    if (rough_exponents<T>(m, c)) {
#pragma unroll 4
        for (int i = wlo + tid; i < whi; i += kThreads)
            store_vector<T>(w, grow, same, i, column_grads<T, true>(buf[i - lo], minus, minus_c, cc, gg));
    } else {
#pragma unroll 4
        for (int i = wlo + tid; i < whi; i += kThreads)
            store_vector<T>(w, grow, same, i, column_grads<T, false>(buf[i - lo], minus, minus_c, cc, gg));
    }
    const int edge = tid == 0 && lo < wlo ? lo : tid == 32 && whi < hi && !(hi - 1 == lo && lo < wlo) ? hi - 1 : -1;
    if (edge >= 0) {
        float v[E];
        unpack(column_grads<T, false>(buf[edge - lo], minus, minus_c, cc, gg), v);
        store_grad<T>(w, grow, same, edge, v);
    }
    stored_arrive();
}

// The gradient alone, from stats: blocks of `share` vectors, independent of
// each other, four vectors a thread in flight; 4096 x 131072 bf16: 307 us, 7.0
// TB/s.
template <class T>
__global__ void __launch_bounds__(kBlock, 2) distill_grad_kernel(const DistillParams p) {
    constexpr int E = kVecOf<T>;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ Shared sh;
    int* const ids = (int*)dyn;
    float* const prob = (float*)(ids + p.top);
    float* const named = prob + p.top;
    int* const buckets = (int*)(named + p.top);
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
    // stats of 0 mark a row without weight or entries
    const float m = p.stats[2 * t], l = p.stats[2 * t + 1];
    if (wt == 0.0f || (m == 0.0f && l == 0.0f)) {
        zero_grad<T>(w, grow, same, lo, hi);
        return;
    }
    const float l_inv = 1.0f / l, g = wt * p.temperature, gl = g * l_inv;
    if (warp == kWarps) {
        teacher_softmax(p, t, c, ids, prob, sh);
        __syncwarp();
        for (int k = lane; k < p.top; k += 32) {
            const int i = ids[k] >= 0 ? (w.shift + ids[k]) / E : -1;
            named[k] = i >= lo && i < hi ? to_f32(row[ids[k]]) : 0.0f;
        }
        if (p.in_place) __syncthreads();
        else __syncwarp();
        entry_grads<T>(p, w, grow, lo, hi, ids, prob, named, buckets, m, l_inv, c, g, [&](int k) { return named[k]; });
        return;
    }
    const int wlo = max(lo, w.whole_lo()), whi = max(wlo, min(hi, w.whole_hi()));
    const int edge = tid == 0 && lo < wlo ? lo : tid == 32 && whi < hi && !(hi - 1 == lo && lo < wlo) ? hi - 1 : -1;
    float ev[E];
    if (edge >= 0) edge_vector<T>(w, edge, ev);
    const Pair minus(-m, -m), minus_c(-m * c, -m * c), cc(c, c), gg(gl, gl);
    const bool rough = rough_exponents<T>(m, c);
    constexpr int B = 4;  // vectors in flight
    for (int i0 = wlo; i0 < whi; i0 += B * kThreads) {
        uint4 v[B];
#pragma unroll
        for (int b = 0; b < B; b++) {
            const int i = i0 + tid + b * kThreads;
            if (i < whi) v[b] = *(const uint4*)(w.base + (uintptr_t)i * 16);
        }
        // in place, the teacher's warp reads its logits before they are replaced
        if (p.in_place && i0 == wlo) __syncthreads();
#pragma unroll
        for (int b = 0; b < B; b++) {
            const int i = i0 + tid + b * kThreads;
            if (i >= whi) continue;
            v[b] = rough ? column_grads<T, true>(v[b], minus, minus_c, cc, gg) : column_grads<T, false>(v[b], minus, minus_c, cc, gg);
            store_vector<T>(w, grow, same, i, v[b]);
        }
    }
    if (p.in_place && wlo >= whi) __syncthreads();
    if (edge >= 0) {
        float v[E];
        unpack(column_grads<T, false>(pack(ev), minus, minus_c, cc, gg), v);
        store_grad<T>(w, grow, same, edge, v);
    }
    stored_arrive();
}

// A block's share of a row: six blocks fit an SM (and 128 KB or 256 KB rows of
// any alignment are four or eight shares).
constexpr int kShareBytes = 33 << 10;
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
    p.in_place = a.grad_logits == a.logits;
    const bool bf = a.dtype == HC_BFLOAT16;
    const int E = bf ? 8 : 4;
    const int vecs = (p.vocab + 2 * E - 2) / E;  // of a row at any alignment
    void* args[] = {&p};
    const int entry_bytes = p.top * 12 + bucket_count(p.top) * 4;
    if (mode == DISTILL_GRAD) {
        // shares of 32 KB once they fill the SMs several times over (4096 x 131072
        // bf16: 307 us, 379 with 8 KB), of 8 KB for few rows (8 x 32768: 3.0 us, 3.4)
        p.share = 16 * kThreads;
        if (p.tokens * ((vecs + p.share - 1) / p.share) < 4 * sms) p.share = 4 * kThreads;
        p.cs = (vecs + p.share - 1) / p.share;
        const int64_t grid = p.tokens * p.cs;
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        const void* fn = bf ? (const void*)distill_grad_kernel<Bf16> : (const void*)distill_grad_kernel<float>;
        return launch_op(fn, dim3((unsigned)grid), dim3(kBlock), args, (size_t)entry_bytes, stream);
    }
    p.cs = 1;
    while (p.cs < kMaxCluster && ((int64_t)vecs * 16 > (int64_t)kShareBytes * p.cs ||
                        (p.tokens * p.cs < sms && vecs / p.cs > kThreads)))
        p.cs *= 2;
    p.share = (vecs + p.cs - 1) / p.cs;
    if (p.share * 16 > kMaxShareBytes) return cudaErrorInvalidValue;
    p.piece = (p.share + kPieces - 1) / kPieces;
    if (p.piece < kUnroll * kThreads) p.piece = kUnroll * kThreads;
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
    return launch_op(fn, dim3((unsigned)grid), dim3(kBlock), args, (size_t)smem, stream, p.cs);
}

}  // namespace hc
