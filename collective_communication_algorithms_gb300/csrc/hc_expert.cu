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

struct PlanParams {
    const void* ids;
    int32_t* offsets;
    int32_t* row_tokens;
    int32_t* slots;
    int32_t* counts;  // blocks x E
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

__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(const PlanParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    int32_t* cnt = (int32_t*)smem;
    for (int e = threadIdx.x; e < p.E; e += kPlanThreads) cnt[e] = 0;
    __syncthreads();
    grid_wait();
    grid_release();
    const int64_t begin = (int64_t)blockIdx.x * p.run, end = min(p.n, begin + p.run);
    for (int64_t i = begin + threadIdx.x; i < end; i += kPlanThreads) {
        const int e = expert_at(p, i);
        if (e < p.E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kPlanThreads) p.counts[(int64_t)blockIdx.x * p.E + e] = cnt[e];
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

// Shared memory: the next place per warp and expert [kPlanWarps][E].
template <bool SINGLE>
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    int32_t* places = (int32_t*)smem;
    __shared__ int sh[kPlanWarps];
    const int E = p.E, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* place = places + warp * E;
    for (int e = lane; e < E; e += 32) place[e] = 0;
    __syncwarp();
    grid_wait();
    grid_release();
    const int64_t begin = (int64_t)blockIdx.x * p.run, end = min(p.n, begin + p.run);
    const int64_t per = p.run / kPlanWarps;  // a multiple of 32
    const int64_t wb = begin + warp * per, we = min(end, wb + per);
    for (int64_t i = wb + lane; i < we; i += 32) {
        const int e = expert_at(p, i);
        if (e < E) atomicAdd(&place[e], 1);
    }
    __syncthreads();
    // experts in runs of kPlanThreads: totals, their sums, and this block's start
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
        const int e = e0 + tid;
        int all = 0, before = 0;
        if (e < E) {
            if (SINGLE) {
                for (int w = 0; w < kPlanWarps; w++) all += places[w * E + e];
            } else {
#pragma unroll 8
                for (int b = 0; b < p.blocks; b++) {
                    const int c = p.counts[(int64_t)b * E + e];
                    all += c;
                    if (b < (int)blockIdx.x) before += c;
                }
            }
        }
        int total;
        const int start = carry + block_exclusive(all, sh, &total);
        carry += total;
        if (e < E) {
            int at = start + before;
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
    for (int64_t i0 = wb; i0 < we; i0 += 32) {
        const int64_t i = i0 + lane;
        const int e = i < we ? expert_at(p, i) : E;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
        int at = -1;
        if (e < E) at = place[e] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (e < E) {
            if (p.row_tokens) p.row_tokens[at] = (int32_t)((uint32_t)i / p.top);
            if (lane == __ffs(same) - 1) place[e] += __popc(same);
        }
        if (p.slots && i < we) p.slots[i] = at;
        __syncwarp();
    }
    if (p.row_tokens)  // behind the last row
        for (int64_t i = carry + (int64_t)blockIdx.x * kPlanThreads + tid; i < p.n; i += (int64_t)p.blocks * kPlanThreads)
            p.row_tokens[i] = -1;
}

// ---------------------------------------------------------------------------
// combine and its gradient: a token's row belongs to W warps, which take 32 V
// elements a step; rows of the experts are read once each.
//
// Bound by bytes: a token reads `top` rows scattered over y.  All of a step's
// loads over up to kSlots choices are under way together.
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

template <class T, int V>
__global__ void __launch_bounds__(kCombineWarps * 32) combine_kernel(const CombineParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kCombineWarps / p.warps) + warp / p.warps;
    grid_wait();
    grid_release();
    if (t >= p.tokens) return;
    const T* y = (const T*)p.y;
    T* out = (T*)p.out + t * p.out_stride;
    const int64_t step = (int64_t)p.warps * 32 * V;
    for (int64_t c = ((int64_t)(warp % p.warps) * 32 + lane) * V; c < p.dim; c += step) {
        const int64_t left = p.dim - c;
        const int n = left < V ? (int)left : V;
        float acc[V];
#pragma unroll
        for (int v = 0; v < V; v++) acc[v] = 0.0f;
        for (int j0 = 0; j0 < p.top; j0 += kSlots) {
            float x[kSlots][V], w[kSlots];
            bool in[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; j++) {
                const int64_t at = t * p.top + j0 + j;
                const int s = j0 + j < p.top ? p.slots[at] : -1;
                in[j] = (uint32_t)s < (uint64_t)p.rows && s >= 0;
                if (in[j]) {
                    w[j] = weight_at(p, at);
                    load_n<T, V>(y + s * p.y_stride + c, n, x[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < kSlots; j++)
                if (in[j])
#pragma unroll
                    for (int v = 0; v < V; v++) acc[v] = fmaf(w[j], x[j][v], acc[v]);
        }
        store_n<T, V>(out + c, n, acc);
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
    const int64_t step = (int64_t)p.warps * 32 * V;
    for (int j0 = 0; j0 < p.top; j0 += kSlots) {
        float dot[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; j++) dot[j] = 0.0f;
        if (t < p.tokens) {
            int s[kSlots];
            float w[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; j++) {
                const int64_t at = t * p.top + j0 + j;
                s[j] = j0 + j < p.top ? p.slots[at] : -1;
                if ((uint64_t)(uint32_t)s[j] >= (uint64_t)p.rows) s[j] = -1;
                w[j] = s[j] >= 0 ? weight_at(p, at) : 0.0f;
            }
            for (int64_t c = ((int64_t)mine * 32 + lane) * V; c < p.dim; c += step) {
                const int64_t left = p.dim - c;
                const int n = left < V ? (int)left : V;
                float gv[V], x[kSlots][V];
                load_n<T, V>(g + c, n, gv);
                if (p.grad_weights) {
#pragma unroll
                    for (int j = 0; j < kSlots; j++)
                        if (s[j] >= 0) load_n<T, V>(y + s[j] * p.y_stride + c, n, x[j]);
#pragma unroll
                    for (int j = 0; j < kSlots; j++)
                        if (s[j] >= 0)
#pragma unroll
                            for (int v = 0; v < V; v++) dot[j] = fmaf(gv[v], x[j][v], dot[j]);
                }
                if (gy) {
#pragma unroll
                    for (int j = 0; j < kSlots; j++)
                        if (s[j] >= 0) {
                            float o[V];
#pragma unroll
                            for (int v = 0; v < V; v++) o[v] = w[j] * gv[v];
                            store_n<T, V>(gy + s[j] * p.out_stride + c, n, o);
                        }
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
constexpr int64_t kPlanSingle = 8192;
constexpr int64_t kPlanMaxBlocks = 128, kPlanMinRun = 4096;

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
    s.bytes = (size_t)s.blocks * experts * sizeof(int32_t);
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
    const int smem = kPlanWarps * p.E * (int)sizeof(int32_t);
    if (s.blocks > 1) {
        const cudaError_t e = launch_op((const void*)plan_count_kernel, dim3((unsigned)s.blocks), dim3(kPlanThreads), args,
                                        p.E * sizeof(int32_t), stream);
        if (e != cudaSuccess) return e;
    }
    const void* fn = s.blocks > 1 ? (const void*)plan_place_kernel<false> : (const void*)plan_place_kernel<true>;
    if (smem > 48 * 1024 && !allow_smem((void*)fn, smem)) return cudaErrorInvalidValue;
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
