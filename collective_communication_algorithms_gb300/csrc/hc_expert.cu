// hc_expert.cu -- around the products of an expert layer: the plan that sorts
// a batch's assignments by expert (hc_expert_plan), the weighted sum back to
// the tokens (hc_expert_combine) and its gradient.
#include <algorithm>

#include "hc_ops.cuh"

namespace hc {
namespace {

// ---------------------------------------------------------------------------
// plan: a stable counting sort of n = tokens * top assignments into E groups.
//
// Bound by latency: a few MB at most pass through, but a row's place depends
// on every assignment before it.  Few assignments: one block counts, scans
// and places them.  More: a first kernel counts each block's run, a second
// one adds up the counts before its own and places.  Within a block every
// warp owns a run too, so that places in a warp follow from which lanes hold
// the same expert (match) and nothing depends on the order of atomics: those
// only add to counters.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanBatch = 8;         // ids of a lane loaded together
constexpr int kPlanMaxBlocks = 128;   // also the pitch of an expert's counts

struct PlanParams {
    const void* ids;
    int32_t* offsets;
    int32_t* row_tokens;
    int32_t* slots;
    int32_t* counts;  // E x kPlanMaxBlocks
    int64_t first;
    int64_t n;
    int64_t run;      // assignments of a block, a multiple of kPlanThreads
    uint32_t top;
    int E, blocks, wide;
};

// Local expert of an assignment, E for none.
__device__ __forceinline__ int expert_at(const PlanParams& p, int64_t i) {
    const int64_t e = (p.wide ? ((const int64_t*)p.ids)[i] : (int64_t)((const int32_t*)p.ids)[i]);
    // the difference of ids that lie far apart wraps round, but only one below
    // E comes out as one
    const uint64_t d = (uint64_t)e - (uint64_t)p.first;
    return d < (uint64_t)p.E ? (int)d : p.E;
}

// f(assignment, its expert) for a warp's run, 32 neighbours at a time; E and an
// assignment behind the end for lanes without one.
template <class F>
__device__ __forceinline__ void for_run(const PlanParams& p, int64_t begin, int64_t end, F f) {
    const int lane = threadIdx.x & 31;
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kPlanBatch) {
        int e[kPlanBatch];
#pragma unroll
        for (int k = 0; k < kPlanBatch; k++) {
            const int64_t i = i0 + 32 * k + lane;
            e[k] = i < end ? expert_at(p, i) : p.E;
        }
#pragma unroll
        for (int k = 0; k < kPlanBatch; k++)
            if (i0 + 32 * k < end) f(i0 + 32 * k + lane, e[k]);
    }
}

__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(const PlanParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    int32_t* cnt = (int32_t*)smem;
    for (int e = threadIdx.x; e < p.E; e += kPlanThreads) cnt[e] = 0;
    __syncthreads();
    grid_wait();
    grid_release();
    const int64_t begin = (int64_t)blockIdx.x * p.run, end = min(p.n, begin + p.run);
    const int64_t per = p.run / kPlanWarps, wb = begin + (threadIdx.x >> 5) * per;
    for_run(p, wb, min(end, wb + per), [&](int64_t, int e) {
        if (e < p.E) atomicAdd(&cnt[e], 1);
    });
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kPlanThreads) p.counts[e * kPlanMaxBlocks + blockIdx.x] = cnt[e];
}

// Exclusive sums of v over the block's threads (every thread's v), and the total.
__device__ __forceinline__ int block_exclusive(int v, int* sh, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) sh[warp] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; w++) {
        const int x = sh[w];
        if (w < warp) before += x;
        all += x;
    }
    __syncthreads();
    *total = all;
    return before + s - v;
}

// Shared memory: the next place per warp and expert [kPlanWarps][E]; of several
// blocks also the experts' totals and what the blocks before hold [2][E].
template <bool SINGLE>
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int sh[kPlanWarps];
    const int E = p.E, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* places = (int32_t*)smem;
    int32_t* place = places + warp * E;
    int32_t *total = places + kPlanWarps * E, *before = total + E;
    for (int e = lane; e < E; e += 32) place[e] = 0;
    __syncwarp();
    grid_wait();
    grid_release();
    const int64_t begin = (int64_t)blockIdx.x * p.run, end = min(p.n, begin + p.run);
    const int64_t per = p.run / kPlanWarps;  // a multiple of 32
    const int64_t wb = begin + warp * per, we = min(end, wb + per);
    for_run(p, wb, we, [&](int64_t, int e) {
        if (e < E) atomicAdd(&place[e], 1);
    });
    if (!SINGLE) {  // a warp takes an expert's counts of all blocks, four a lane
        static_assert(kPlanMaxBlocks == 128, "four counts a lane");
        const int b = lane * 4, me = blockIdx.x;
        constexpr int AT_ONCE = 8;  // experts whose counts are under way together
        for (int e0 = warp; e0 < E; e0 += kPlanWarps * AT_ONCE) {
            int4 some[AT_ONCE];
#pragma unroll
            for (int k = 0; k < AT_ONCE; k++) {
                const int e = e0 + k * kPlanWarps;
                some[k] = make_int4(0, 0, 0, 0);
                if (e < E && b < p.blocks) some[k] = *(const int4*)&p.counts[e * kPlanMaxBlocks + b];
            }
#pragma unroll
            for (int k = 0; k < AT_ONCE; k++) {
                const int e = e0 + k * kPlanWarps;
                if (e >= E) break;
                int4 c = some[k];
                if (b + 1 >= p.blocks) c.y = 0;
                if (b + 2 >= p.blocks) c.z = 0;
                if (b + 3 >= p.blocks) c.w = 0;
                const int all = __reduce_add_sync(0xFFFFFFFFu, c.x + c.y + c.z + c.w);
                const int mine = __reduce_add_sync(
                    0xFFFFFFFFu, (b < me ? c.x : 0) + (b + 1 < me ? c.y : 0) + (b + 2 < me ? c.z : 0) + (b + 3 < me ? c.w : 0));
                if (lane == 0) {
                    total[e] = all;
                    before[e] = mine;
                }
            }
        }
    }
    __syncthreads();
    // experts in runs of kPlanThreads: where each begins, and this block's and its warps' places in it
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
        const int e = e0 + tid;
        int all = 0;
        if (e < E) {
            if (SINGLE)
                for (int w = 0; w < kPlanWarps; w++) all += places[w * E + e];
            else
                all = total[e];
        }
        int sum;
        const int start = carry + block_exclusive(all, sh, &sum);
        carry += sum;
        if (e < E) {
            int at = start + (SINGLE ? 0 : before[e]);
            for (int w = 0; w < kPlanWarps; w++) {
                const int c = places[w * E + e];
                places[w * E + e] = at;
                at += c;
            }
            if (blockIdx.x == 0) p.offsets[e] = start;
        }
    }
    if (blockIdx.x == 0 && tid == 0) p.offsets[E] = carry;
    __syncthreads();
    for_run(p, wb, we, [&](int64_t i, int e) {
        const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
        const int at = e < E ? place[e] + __popc(same & ((1u << lane) - 1)) : -1;
        __syncwarp();
        if (e < E) {
            if (p.row_tokens) p.row_tokens[at] = (int32_t)((uint32_t)i / p.top);
            if (lane == __ffs(same) - 1) place[e] += __popc(same);
        }
        if (p.slots && i < we) p.slots[i] = at;
        __syncwarp();
    });
    if (p.row_tokens)  // behind the last row
        for (int64_t i = carry + (int64_t)blockIdx.x * kPlanThreads + tid; i < p.n; i += (int64_t)p.blocks * kPlanThreads)
            p.row_tokens[i] = -1;
}

// ---------------------------------------------------------------------------
// combine and its gradient: a token's row belongs to W warps, which take 32 V
// elements a step; rows of the experts are read once each.
//
// Bound by bytes: a token reads `top` rows scattered over y.  All of a step's
// loads over up to kSlots choices are under way together; rows of whole 16
// bytes take them in pieces of 16, others element by element.
// ---------------------------------------------------------------------------
constexpr int kCombineWarps = 8, kSlots = 8;

struct CombineParams {
    const void* y;         // forward: rows; gradient: NULL if grad_weights is not wanted
    const void* grad_out;
    const int32_t* slots;
    const void* weights;
    void* out;             // forward: tokens x dim; gradient: grad_y or NULL
    void* grad_weights;
    int64_t tokens, rows, dim;
    int64_t y_stride, out_stride, grad_out_stride;
    int top, weight_bf, warps;  // warps of a token
};

__device__ __forceinline__ float weight_at(const CombineParams& p, int64_t i) {
    if (!p.weights) return 1.0f;
    return p.weight_bf ? to_f32(((const Bf16*)p.weights)[i]) : ((const float*)p.weights)[i];
}

// V elements as they lie in memory: 16 bytes, or one element.
template <class T, int V>
struct Piece {
    uint4 w;
    __device__ __forceinline__ void load(const T* p) { w = *(const uint4*)p; }
    __device__ __forceinline__ void get(float (&v)[V]) const { unpack(w, v); }
    static __device__ __forceinline__ void store(T* p, const float (&v)[V]) { *(uint4*)p = pack(v); }
};
template <class T>
struct Piece<T, 1> {
    T w;
    __device__ __forceinline__ void load(const T* p) { w = *p; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f32(w); }
    static __device__ __forceinline__ void store(T* p, const float (&v)[1]) { put(p, v[0]); }
};

// Rows of a token's choices j0 .. j0 + kSlots, -1 for none.
__device__ __forceinline__ void slots_at(const CombineParams& p, int64_t t, int j0, int (&s)[kSlots]) {
#pragma unroll
    for (int j = 0; j < kSlots; j++) {
        s[j] = j0 + j < p.top ? p.slots[t * p.top + j0 + j] : -1;
        if ((uint64_t)(uint32_t)s[j] >= (uint64_t)p.rows) s[j] = -1;
    }
}

template <class T, int V>
__global__ void __launch_bounds__(kCombineWarps * 32) combine_kernel(const CombineParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kCombineWarps / p.warps) + warp / p.warps;
    grid_wait();
    grid_release();
    if (t >= p.tokens) return;
    const T* y = (const T*)p.y;
    T* out = (T*)p.out + t * p.out_stride;
    const int64_t step = (int64_t)p.warps * 32 * V, c0 = ((int64_t)(warp % p.warps) * 32 + lane) * V;
    int s[kSlots];
    float w[kSlots];
    const auto choices = [&](int j0) {
        slots_at(p, t, j0, s);
#pragma unroll
        for (int j = 0; j < kSlots; j++) w[j] = s[j] >= 0 ? weight_at(p, t * p.top + j0 + j) : 0.0f;
    };
    choices(0);
    for (int64_t c = c0; c < p.dim; c += step) {
        float acc[V];
#pragma unroll
        for (int v = 0; v < V; v++) acc[v] = 0.0f;
        for (int j0 = 0; j0 < p.top; j0 += kSlots) {
            if (p.top > kSlots) choices(j0);
            Piece<T, V> x[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; j++)
                if (s[j] >= 0) x[j].load(y + s[j] * p.y_stride + c);
#pragma unroll
            for (int j = 0; j < kSlots; j++)
                if (s[j] >= 0) {
                    float v[V];
                    x[j].get(v);
#pragma unroll
                    for (int k = 0; k < V; k++) acc[k] = fmaf(w[j], v[k], acc[k]);
                }
        }
        Piece<T, V>::store(out + c, acc);
    }
}

template <class T, int V>
__global__ void __launch_bounds__(kCombineWarps * 32) combine_grad_kernel(const CombineParams p) {
    __shared__ float part[kCombineWarps][kSlots];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = warp % p.warps;
    const int64_t t = (int64_t)blockIdx.x * (kCombineWarps / p.warps) + warp / p.warps;
    grid_wait();
    grid_release();
    const T* y = (const T*)p.y;
    const T* g = (const T*)p.grad_out + t * p.grad_out_stride;
    T* gy = (T*)p.out;
    const int64_t step = (int64_t)p.warps * 32 * V, c0 = ((int64_t)mine * 32 + lane) * V;
    for (int j0 = 0; j0 < p.top; j0 += kSlots) {
        float dot[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; j++) dot[j] = 0.0f;
        if (t < p.tokens) {
            int s[kSlots];
            float w[kSlots];
            slots_at(p, t, j0, s);
#pragma unroll
            for (int j = 0; j < kSlots; j++) w[j] = s[j] >= 0 ? weight_at(p, t * p.top + j0 + j) : 0.0f;
            for (int64_t c = c0; c < p.dim; c += step) {
                Piece<T, V> go, x[kSlots];
                go.load(g + c);
                if (p.grad_weights)
#pragma unroll
                    for (int j = 0; j < kSlots; j++)
                        if (s[j] >= 0) x[j].load(y + s[j] * p.y_stride + c);
                float gv[V];
                go.get(gv);
                if (p.grad_weights)
#pragma unroll
                    for (int j = 0; j < kSlots; j++)
                        if (s[j] >= 0) {
                            float v[V];
                            x[j].get(v);
#pragma unroll
                            for (int k = 0; k < V; k++) dot[j] = fmaf(gv[k], v[k], dot[j]);
                        }
                if (gy)
#pragma unroll
                    for (int j = 0; j < kSlots; j++)
                        if (s[j] >= 0) {
                            float o[V];
#pragma unroll
                            for (int k = 0; k < V; k++) o[k] = w[j] * gv[k];
                            Piece<T, V>::store(gy + s[j] * p.out_stride + c, o);
                        }
            }
        }
        if (!p.grad_weights) continue;
#pragma unroll
        for (int j = 0; j < kSlots; j++) dot[j] = warp_sum(dot[j]);
        if (p.warps > 1) {  // the same for the whole block
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < kSlots; j++) part[warp][j] = dot[j];
            __syncthreads();
            if (mine == 0)
#pragma unroll
                for (int j = 0; j < kSlots; j++)
                    for (int k = 1; k < p.warps; k++) dot[j] += part[warp + k][j];
            __syncthreads();
        }
        if (t < p.tokens && mine == 0 && lane == 0)
#pragma unroll
            for (int j = 0; j < kSlots; j++)
                if (j0 + j < p.top) {
                    const int64_t at = t * p.top + j0 + j;
                    if (p.weight_bf) put((Bf16*)p.grad_weights + at, dot[j]);
                    else ((float*)p.grad_weights)[at] = dot[j];
                }
    }
}

// Warps of a token: one while tokens alone fill the SMs with a block of eight
// warps each twice over, more for fewer tokens as far as the row has steps.
int warps_of(int64_t tokens, int64_t dim, int per_lane, int sms) {
    int w = 1;
    while (w < kCombineWarps && tokens * w < (int64_t)sms * 2 * kCombineWarps && dim > (int64_t)w * 32 * per_lane) w *= 2;
    return w;
}

template <template <class, int> class Pick>
cudaError_t launch_rows(CombineParams p, hc_dtype_t dtype, bool vectors, int sms, cudaStream_t stream) {
    const int es = elem_bytes(dtype), V = vectors ? 16 / es : 1;
    p.warps = warps_of(p.tokens, p.dim, V, sms);
    const int per_block = kCombineWarps / p.warps;
    const int64_t blocks = (p.tokens + per_block - 1) / per_block;
    void* args[] = {&p};
    const void* fn = dtype == HC_BFLOAT16 ? (vectors ? Pick<Bf16, 8>::fn() : Pick<Bf16, 1>::fn())
                                          : (vectors ? Pick<float, 4>::fn() : Pick<float, 1>::fn());
    return launch_op(fn, dim3((unsigned)blocks), dim3(kCombineWarps * 32), args, 0, stream);
}
template <class T, int V>
struct PickCombine {
    static const void* fn() { return (const void*)combine_kernel<T, V>; }
};
template <class T, int V>
struct PickCombineGrad {
    static const void* fn() { return (const void*)combine_grad_kernel<T, V>; }
};

bool wide_rows(const void* p, size_t stride, size_t dim, int es) {
    return !p || ((uintptr_t)p % 16 == 0 && stride * es % 16 == 0 && dim * es % 16 == 0);
}

}  // namespace

// Runs of the counting kernels: none up to this many assignments.
constexpr int64_t kPlanSingle = 8192, kPlanMinRun = 4096;

ExpertPlanShape expert_plan_shape(int64_t n, int64_t experts) {
    ExpertPlanShape s;
    const int64_t unit = kPlanThreads;
    if (n <= kPlanSingle) {
        s.blocks = 1;
        s.run = std::max<int64_t>(1, (n + unit - 1) / unit) * unit;
        s.bytes = 0;
        return s;
    }
    s.run = std::max(kPlanMinRun, (n + kPlanMaxBlocks - 1) / kPlanMaxBlocks);
    s.run = (s.run + unit - 1) / unit * unit;
    s.blocks = (int)((n + s.run - 1) / s.run);
    s.bytes = (size_t)kPlanMaxBlocks * experts * sizeof(int32_t);
    return s;
}

cudaError_t launch_expert_plan(const hc_expert_plan_t& a, cudaStream_t stream) {
    PlanParams p;
    p.ids = a.expert_ids;
    p.offsets = a.offsets;
    p.row_tokens = a.row_tokens;
    p.slots = a.slots;
    p.counts = (int32_t*)a.scratch;
    p.first = a.first_expert;
    p.n = (int64_t)(a.tokens * a.top);
    p.top = (uint32_t)a.top;
    p.E = (int)a.experts;
    p.wide = a.id_type == HC_ID64;
    const ExpertPlanShape s = expert_plan_shape(p.n, p.E);
    p.run = s.run;
    p.blocks = s.blocks;
    void* args[] = {&p};
    const int smem = (kPlanWarps + (s.blocks > 1 ? 2 : 0)) * p.E * (int)sizeof(int32_t);
    const void* fn = s.blocks > 1 ? (const void*)plan_place_kernel<false> : (const void*)plan_place_kernel<true>;
    // asked for at any size: what a block has without asking, 48 KiB, counts
    // the kernel's own variables too
    if (!allow_smem((void*)fn, smem)) return cudaErrorInvalidValue;
    if (s.blocks > 1) {
        const cudaError_t e = launch_op((const void*)plan_count_kernel, dim3((unsigned)s.blocks), dim3(kPlanThreads), args,
                                        p.E * sizeof(int32_t), stream);
        if (e != cudaSuccess) return e;
    }
    return launch_op(fn, dim3((unsigned)s.blocks), dim3(kPlanThreads), args, smem, stream);
}

cudaError_t launch_expert_combine(const hc_expert_combine_t& a, cudaStream_t stream, int sms) {
    CombineParams p = {};
    p.y = a.y;
    p.slots = a.slots;
    p.weights = a.weights;
    p.out = a.out;
    p.tokens = (int64_t)a.tokens;
    p.rows = (int64_t)a.rows;
    p.dim = (int64_t)a.dim;
    p.y_stride = (int64_t)a.y_stride;
    p.out_stride = (int64_t)a.out_stride;
    p.top = (int)a.top;
    p.weight_bf = a.weight_dtype == HC_BFLOAT16;
    const int es = elem_bytes(a.dtype);
    const bool vectors = wide_rows(a.y, a.y_stride, a.dim, es) && wide_rows(a.out, a.out_stride, a.dim, es);
    return launch_rows<PickCombine>(p, a.dtype, vectors, sms, stream);
}

cudaError_t launch_expert_combine_grad(const hc_expert_combine_grad_t& a, cudaStream_t stream, int sms) {
    CombineParams p = {};
    p.y = a.y;
    p.grad_out = a.grad_out;
    p.slots = a.slots;
    p.weights = a.weights;
    p.out = a.grad_y;
    p.grad_weights = a.grad_weights;
    p.tokens = (int64_t)a.tokens;
    p.rows = (int64_t)a.rows;
    p.dim = (int64_t)a.dim;
    p.y_stride = (int64_t)a.y_stride;
    p.out_stride = (int64_t)a.grad_y_stride;
    p.grad_out_stride = (int64_t)a.grad_out_stride;
    p.top = (int)a.top;
    p.weight_bf = a.weight_dtype == HC_BFLOAT16;
    const int es = elem_bytes(a.dtype);
    const bool vectors = wide_rows(a.grad_weights ? a.y : nullptr, a.y_stride, a.dim, es) &&
                         wide_rows(a.grad_y, a.grad_y_stride, a.dim, es) &&
                         wide_rows(a.grad_out, a.grad_out_stride, a.dim, es);
    return launch_rows<PickCombineGrad>(p, a.dtype, vectors, sms, stream);
}

}  // namespace hc
