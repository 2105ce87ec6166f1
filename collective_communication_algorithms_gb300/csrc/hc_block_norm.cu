// hc_block_norm.cu -- the norm after a block, its gate, the scaled residual
// and the norm before the next block, and their gradient.
//
// A row stays in the registers of its threads from its loads to its stores:
// forward, y and x are read once and r and z written once, with two row sums
// between (y^2, then r^2, which needs the first); backward, grad_r, grad_z, y
// and x are read once and grad_x and grad_y written once, again with two row
// sums.  Rows longer than one block holds are split over a cluster, whose
// blocks exchange their sums through distributed shared memory.
//
// Weight gradients: sums over tokens of dz * rhat (pre) and A = D * yhat,
// from which the others follow: d gate = post_weight * sum A over the gate's
// tokens, d post_weight = sum gate * A.  A block sums its own run of tokens in
// registers and leaves partial sums in scratch; a second kernel adds them in
// a fixed order.
#include "hc_ops.cuh"

namespace hc {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kNormThreads = 1024;
constexpr int kNormGradThreads = 512;  // up to 128 registers a thread

// Cluster-wide barrier (every thread of every block of the cluster).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void store_remote(float* local, unsigned rank, float v) {
    const unsigned a = (unsigned)__cvta_generic_to_shared(local);
    asm volatile(
        "{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %0, %1;\n st.shared::cluster.f32 [r], %2;\n}\n" ::"r"(a),
        "r"(rank), "f"(v)
        : "memory");
}

// Sum of v over the blockDim.x threads of a row (and the blocks of the
// cluster), in a fixed order.  Calls alternate between two slots of shared
// memory: a call's slot is written again only after the barrier of the call
// between, which every thread reaches after its reads.
struct RowSum {
    float (*warp)[32];         // [2][row * warps + warp]
    float (*rank)[kMaxCluster];  // [2][rank], clusters have one row a block
    int cs;
    int slot;
    __device__ __forceinline__ float operator()(float v) {
        slot ^= 1;
        v = warp_sum(v);
        const int warps = blockDim.x >> 5;
        if (warps > 1) {
            const int w = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0) warp[slot][threadIdx.y * warps + w] = v;
            __syncthreads();
            v = 0.0f;
            for (int i = 0; i < warps; i++) v += warp[slot][threadIdx.y * warps + i];
        }
        if (cs > 1) {
            if (threadIdx.x < (unsigned)cs) store_remote(&rank[slot][cluster_rank()], threadIdx.x, v);
            cluster_sync();
            v = 0.0f;
            for (int i = 0; i < cs; i++) v += rank[slot][i];
        }
        return v;
    }
};

struct NormParams {
    const void *y, *x, *post_weight, *gate, *pre_weight;
    void *r, *z;
    float *post_rstd, *pre_rstd;
    int64_t tokens, per_gate, y_stride, x_stride, r_stride, z_stride;
    int dim, cs;
    bool bf16_weights;
    float residual_scale, eps;
};

// N elements of a weight vector (ones where there is none).
template <int N>
__device__ __forceinline__ void load_weight(const void* w, bool bf16, int64_t at, int n, float (&v)[N]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = 1.0f;
    } else if (bf16) {
        load_n<Bf16, N>((const Bf16*)w + at, n, v);
    } else {
        load_n<float, N>((const float*)w + at, n, v);
    }
}

// blockDim = (threads of a row, rows of a block); a thread holds V vectors of
// N columns, blockDim.x * N columns apart.
template <class T, int N, int V>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormParams p) {
    __shared__ float warp_sums[2][32];
    __shared__ float rank_sums[2][kMaxCluster];
    RowSum row_sum{warp_sums, rank_sums, p.cs, 0};
    const int64_t t = (int64_t)(blockIdx.x / p.cs) * blockDim.y + threadIdx.y;
    const int c0 = ((int)(blockIdx.x % p.cs) * blockDim.x * V + threadIdx.x) * N;
    const int step = blockDim.x * N;
    const bool live = t < p.tokens;
    if (p.cs > 1) cluster_sync();  // every block of the cluster runs
    grid_wait();
    grid_release();
    float y[V][N], x[V][N];
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int c = c0 + v * step, n = live ? p.dim - c : 0;
        load_n<T, N>((const T*)p.y + t * p.y_stride + c, n, y[v]);
        load_n<T, N>((const T*)p.x + t * p.x_stride + c, n, x[v]);
    }
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
        for (int i = 0; i < N; i++) s = fmaf(y[v][i], y[v][i], s);
    const float post = rsqrtf(row_sum(s) / (float)p.dim + p.eps);
    const int64_t g = live ? t / p.per_gate : 0;
    s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int c = c0 + v * step, n = live ? p.dim - c : 0;
        float w[N], gt[N];
        load_weight<N>(p.post_weight, p.bf16_weights, c, n, w);
        load_weight<N>(p.gate, p.bf16_weights, g * p.dim + c, n, gt);
#pragma unroll
        for (int i = 0; i < N; i++) {
            x[v][i] = fmaf(p.residual_scale, x[v][i], gt[i] * (y[v][i] * post * w[i]));
            s = fmaf(x[v][i], x[v][i], s);
        }
        store_n<T, N>((T*)p.r + t * p.r_stride + c, n, x[v]);
    }
    const bool first = threadIdx.x == 0 && blockIdx.x % p.cs == 0 && live;
    if (first && p.post_rstd) p.post_rstd[t] = post;
    if (!p.z) return;
    const float pre = rsqrtf(row_sum(s) / (float)p.dim + p.eps);
    if (first && p.pre_rstd) p.pre_rstd[t] = pre;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int c = c0 + v * step, n = live ? p.dim - c : 0;
        float w[N];
        load_weight<N>(p.pre_weight, p.bf16_weights, c, n, w);
#pragma unroll
        for (int i = 0; i < N; i++) x[v][i] *= pre * w[i];
        store_n<T, N>((T*)p.z + t * p.z_stride + c, n, x[v]);
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
struct NormGradParams {
    const void *grad_r, *grad_z, *y, *x, *post_weight, *gate, *pre_weight;
    const float *post_rstd, *pre_rstd;
    void *grad_y, *grad_x, *grad_post_weight, *grad_gate, *grad_pre_weight;
    float* part;         // [block][slot][pitch]: gate * A, dz * rhat, A
    int64_t tokens, gates, per_gate;
    int64_t grad_r_stride, grad_z_stride, y_stride, x_stride, grad_y_stride, grad_x_stride;
    int64_t blocks, unit, per_group, pitch, jobs;
    int dim, cs, slots;
    bool bf16_weights;
    float residual_scale;
};

// Add the rows' sums of a block into row 0's, in row order, and store them.
template <int N>
__device__ __forceinline__ void store_part(float* joined, float* part, int c, int n, float (&acc)[N]) {
    if (blockDim.y > 1) {
        float* mine = joined + (threadIdx.y * blockDim.x + threadIdx.x) * N;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; i++) mine[i] = acc[i];
        __syncthreads();
        if (threadIdx.y) return;
        for (unsigned r = 1; r < blockDim.y; r++)
#pragma unroll
            for (int i = 0; i < N; i++) acc[i] += joined[(r * blockDim.x + threadIdx.x) * N + i];
    }
    store_n<float, N>(part + c, n, acc);
}

// GROUPS false: the block's run of `unit` tokens lies in one gate row, its
// rows are dealt to the blockDim.y rows of threads.  true: the block has
// `unit` whole gate rows, dealt to the rows of threads.
template <class T, int N, int V, bool GROUPS>
__global__ void __launch_bounds__(kNormGradThreads) norm_grad_kernel(const NormGradParams p) {
    extern __shared__ float joined[];
    __shared__ float warp_sums[2][32];
    __shared__ float rank_sums[2][kMaxCluster];
    RowSum row_sum{warp_sums, rank_sums, p.cs, 0};
    const int64_t block = blockIdx.x / p.cs;
    const int c0 = ((int)(blockIdx.x % p.cs) * blockDim.x * V + threadIdx.x) * N;
    const int step = blockDim.x * N;
    if (p.cs > 1) cluster_sync();
    grid_wait();
    grid_release();
    float a[V][N] = {}, ga[V][N] = {}, pre_acc[V][N] = {};
    // tokens [begin + k * stride, k < count) of this row of threads; a barrier
    // in every step, so the count is the block's
    int64_t gate_row, begin, end, count, stride, groups = 1;
    if (GROUPS) {
        gate_row = block * p.unit + threadIdx.y;
        groups = (p.unit + blockDim.y - 1) / blockDim.y;
    } else {
        gate_row = block / p.per_group;
    }
    for (int64_t k = 0; k < groups; k++) {
        if (GROUPS) {
            const bool has = k * blockDim.y + threadIdx.y < p.unit && gate_row < p.gates;
            begin = gate_row * p.per_gate;
            end = has ? begin + p.per_gate : begin;
            stride = 1;
            count = p.per_gate;
        } else {
            const int64_t lo = gate_row * p.per_gate + block % p.per_group * p.unit;
            const int64_t hi = (gate_row + 1) * p.per_gate;
            end = lo + p.unit < hi ? lo + p.unit : hi;
            begin = lo + threadIdx.y;
            stride = blockDim.y;
            count = (end - lo + stride - 1) / stride;
        }
        for (int64_t step_k = 0; step_k < count; step_k++) {
            const int64_t t = begin + step_k * stride;
            const bool live = t < end;
            float gr[V][N], gz[V][N], y[V][N], x[V][N];
#pragma unroll
            for (int v = 0; v < V; v++) {
                const int c = c0 + v * step, n = live ? p.dim - c : 0;
                load_n<T, N>((const T*)p.grad_r + t * p.grad_r_stride + c, p.grad_r ? n : 0, gr[v]);
                load_n<T, N>((const T*)p.grad_z + t * p.grad_z_stride + c, p.grad_z ? n : 0, gz[v]);
                load_n<T, N>((const T*)p.y + t * p.y_stride + c, n, y[v]);
                load_n<T, N>((const T*)p.x + t * p.x_stride + c, n, x[v]);
            }
            const float post = live ? p.post_rstd[t] : 0.0f;
            const float pre = live && p.grad_z ? p.pre_rstd[t] : 0.0f;
            // y -> yhat; x -> rhat; gz -> h = gz * pre_weight after its use
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) {
                const int c = c0 + v * step, n = live ? p.dim - c : 0;
                float w[N], gt[N], pw[N];
                load_weight<N>(p.post_weight, p.bf16_weights, c, n, w);
                load_weight<N>(p.gate, p.bf16_weights, gate_row * p.dim + c, n, gt);
                load_weight<N>(p.pre_weight, p.bf16_weights, c, n, pw);
#pragma unroll
                for (int i = 0; i < N; i++) {
                    y[v][i] *= post;
                    x[v][i] = fmaf(p.residual_scale, x[v][i], gt[i] * (y[v][i] * w[i])) * pre;
                    pre_acc[v][i] = fmaf(gz[v][i], x[v][i], pre_acc[v][i]);
                    gz[v][i] *= pw[i];
                    s = fmaf(gz[v][i], x[v][i], s);
                }
            }
            const float m1 = p.grad_z ? row_sum(s) / (float)p.dim : 0.0f;
            s = 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) {
                const int c = c0 + v * step, n = live ? p.dim - c : 0;
                float w[N], gt[N], out[N];
                load_weight<N>(p.post_weight, p.bf16_weights, c, n, w);
                load_weight<N>(p.gate, p.bf16_weights, gate_row * p.dim + c, n, gt);
#pragma unroll
                for (int i = 0; i < N; i++) {
                    const float d = fmaf(pre, fmaf(-x[v][i], m1, gz[v][i]), gr[v][i]);
                    a[v][i] = fmaf(d, y[v][i], a[v][i]);
                    out[i] = p.residual_scale * d;
                    gr[v][i] = d * gt[i] * w[i];
                    s = fmaf(gr[v][i], y[v][i], s);
                }
                store_n<T, N>((T*)p.grad_x + t * p.grad_x_stride + c, n, out);
            }
            const float m2 = row_sum(s) / (float)p.dim;
#pragma unroll
            for (int v = 0; v < V; v++) {
                const int c = c0 + v * step, n = live ? p.dim - c : 0;
#pragma unroll
                for (int i = 0; i < N; i++) gr[v][i] = post * fmaf(-y[v][i], m2, gr[v][i]);
                store_n<T, N>((T*)p.grad_y + t * p.grad_y_stride + c, n, gr[v]);
            }
        }
        // A of this gate row is complete (GROUPS), or of the block's run
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int c = c0 + v * step, n = p.dim - c;
            const bool has = !GROUPS || end > begin;
            float gt[N];
            load_weight<N>(p.gate, p.bf16_weights, gate_row * p.dim + c, has ? n : 0, gt);
#pragma unroll
            for (int i = 0; i < N; i++) ga[v][i] = has ? fmaf(gt[i], a[v][i], ga[v][i]) : ga[v][i];
            if (GROUPS) {
                if (p.grad_gate && has) {
                    float w[N];
                    load_weight<N>(p.post_weight, p.bf16_weights, c, n, w);
#pragma unroll
                    for (int i = 0; i < N; i++) w[i] *= a[v][i];
                    if (p.bf16_weights) store_n<Bf16, N>((Bf16*)p.grad_gate + gate_row * p.dim + c, n, w);
                    else store_n<float, N>((float*)p.grad_gate + gate_row * p.dim + c, n, w);
                }
#pragma unroll
                for (int i = 0; i < N; i++) a[v][i] = 0.0f;
            }
        }
        if (GROUPS) gate_row += blockDim.y;
    }
    float* part = p.part + block * p.slots * p.pitch;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int c = c0 + v * step, n = p.dim - c;
        store_part<N>(joined, part, c, n, ga[v]);
        store_part<N>(joined, part + p.pitch, c, n, pre_acc[v]);
        if (!GROUPS) store_part<N>(joined, part + 2 * p.pitch, c, n, a[v]);
    }
}

// Sums of the partial rows: blockIdx.y 0: post weight, 1: pre weight, 2 + g:
// gate row g.  The warps add equal parts of the list, joined in order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) norm_sum_kernel(const NormGradParams p) {
    __shared__ float4 sums[kSumWarps][32];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t job = blockIdx.y; job < p.jobs; job += gridDim.y) {
        void* out = job == 0 ? p.grad_post_weight : job == 1 ? p.grad_pre_weight : p.grad_gate;
        if (!out) continue;
        const int64_t g = job - 2;
        const int64_t first = job < 2 ? 0 : g * p.per_group, count = job < 2 ? p.blocks : p.per_group;
        const int c = (blockIdx.x * 32 + lane) * 4;  // the pitch is a multiple of 4 columns
        const float* src = p.part + (first * p.slots + (job < 2 ? job : 2)) * p.pitch + c;
        const int64_t per = (count + kSumWarps - 1) / kSumWarps;
        const int64_t a = warp * per, b = a + per < count ? a + per : count;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < p.dim) {
#pragma unroll 4
            for (int64_t k = a; k < b; k++) {
                const float4 v = *(const float4*)(src + k * p.slots * p.pitch);
                acc.x += v.x;
                acc.y += v.y;
                acc.z += v.z;
                acc.w += v.w;
            }
        }
        __syncthreads();  // the last job's sums have been read
        sums[warp][lane] = acc;
        __syncthreads();
        if (warp || c >= p.dim) continue;
        for (int w = 1; w < kSumWarps && w * per < count; w++) {
            const float4 v = sums[w][lane];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        float v[4] = {acc.x, acc.y, acc.z, acc.w};
        const int n = p.dim - c < 4 ? p.dim - c : 4;
        const int64_t at = (job < 2 ? 0 : g * p.dim) + c;
        for (int i = 0; i < n; i++) {
            if (job >= 2 && p.post_weight)
                v[i] *= p.bf16_weights ? to_f32(((const Bf16*)p.post_weight)[c + i]) : ((const float*)p.post_weight)[c + i];
            if (p.bf16_weights) put((Bf16*)out + at + i, v[i]);
            else put((float*)out + at + i, v[i]);
        }
    }
}

// Threads of a row, rows of a block and blocks of a cluster for `dim` columns
// held C to a thread.
struct Shape {
    int tx, ty, cs;
};
Shape row_shape(int64_t dim, int C, int most_threads, int64_t rows) {
    Shape s;
    const int64_t threads = (dim + C - 1) / C;
    s.cs = 1;
    while (threads > (int64_t)most_threads * s.cs) s.cs *= 2;
    const int64_t per = (threads + s.cs - 1) / s.cs;
    s.tx = (int)((per + 31) / 32 * 32);
    s.ty = 1;
    while (s.cs == 1 && s.tx * s.ty < 128 && s.ty < rows) s.ty *= 2;
    return s;
}

template <class T>
bool wide(const void* p, int64_t stride) {
    return ((uintptr_t)p & 15) == 0 && (stride * (int64_t)sizeof(T) & 15) == 0;
}
bool wide_weight(const void* w, bool bf16, int64_t stride) {
    return bf16 ? wide<Bf16>(w, stride) : wide<float>(w, stride);
}

template <class T>
cudaError_t run_norm(NormParams& p, cudaStream_t stream) {
    constexpr int E = kVecOf<T>;
    const bool vec = wide<T>(p.y, p.y_stride) && wide<T>(p.x, p.x_stride) && wide<T>(p.r, p.r_stride) &&
                     (!p.z || wide<T>(p.z, p.z_stride)) && wide_weight(p.post_weight, p.bf16_weights, 0) &&
                     wide_weight(p.gate, p.bf16_weights, p.dim) && wide_weight(p.pre_weight, p.bf16_weights, 0);
    const Shape s = row_shape(p.dim, 8, kNormThreads, p.tokens);
    p.cs = s.cs;
    const int64_t grid = (p.tokens + s.ty - 1) / s.ty * s.cs;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const void* fn = vec ? (const void*)norm_kernel<T, E, 8 / E> : (const void*)norm_kernel<T, 1, 8>;
    void* args[] = {&p};
    return launch_op(fn, dim3((unsigned)grid), dim3(s.tx, s.ty), args, 0, stream, s.cs);
}

template <class T>
cudaError_t run_norm_grad(NormGradParams& p, bool by_group, cudaStream_t stream) {
    constexpr int E = kVecOf<T>;
    const bool vec = (!p.grad_r || wide<T>(p.grad_r, p.grad_r_stride)) &&
                     (!p.grad_z || wide<T>(p.grad_z, p.grad_z_stride)) && wide<T>(p.y, p.y_stride) &&
                     wide<T>(p.x, p.x_stride) && wide<T>(p.grad_y, p.grad_y_stride) &&
                     wide<T>(p.grad_x, p.grad_x_stride) && wide_weight(p.post_weight, p.bf16_weights, 0) &&
                     wide_weight(p.gate, p.bf16_weights, p.dim) && wide_weight(p.pre_weight, p.bf16_weights, 0) &&
                     wide_weight(p.grad_gate, p.bf16_weights, p.dim);
    const Shape s = row_shape(p.dim, 8, kNormGradThreads, p.unit);
    p.cs = s.cs;
    const void* fn = vec ? (by_group ? (const void*)norm_grad_kernel<T, E, 8 / E, true>
                                     : (const void*)norm_grad_kernel<T, E, 8 / E, false>)
                         : (by_group ? (const void*)norm_grad_kernel<T, 1, 8, true>
                                     : (const void*)norm_grad_kernel<T, 1, 8, false>);
    void* args[] = {&p};
    if (p.blocks > 0) {
        if (p.blocks * s.cs > INT32_MAX) return cudaErrorInvalidValue;
        const size_t smem = s.ty > 1 ? (size_t)s.tx * s.ty * E * sizeof(float) : 0;
        const cudaError_t e = launch_op(fn, dim3((unsigned)(p.blocks * s.cs)), dim3(s.tx, s.ty), args, smem, stream, s.cs);
        if (e != cudaSuccess) return e;
    }
    // gate rows by_group blocks have not written; without tokens all are zeros
    p.jobs = 2 + (p.grad_gate && (!by_group || p.blocks == 0) ? p.gates : 0);
    if (!p.grad_post_weight && !p.grad_pre_weight && p.jobs == 2) return cudaSuccess;
    return launch_op((const void*)norm_sum_kernel,
                     dim3((unsigned)((p.dim + 127) / 128), (unsigned)(p.jobs < 65535 ? p.jobs : 65535)),
                     dim3(kSumWarps * 32), args, 0, stream);
}

constexpr int64_t kGradBlocks = 304;  // partial sums aimed at

}  // namespace

cudaError_t launch_block_norm(const hc_block_norm_t& a, cudaStream_t stream, int sms) {
    (void)sms;
    NormParams p = {};
    p.y = a.y;
    p.x = a.x;
    p.post_weight = a.post_weight;
    p.gate = a.gate;
    p.pre_weight = a.pre_weight;
    p.r = a.r;
    p.z = a.z;
    p.post_rstd = a.post_rstd;
    p.pre_rstd = a.pre_rstd;
    p.tokens = (int64_t)a.tokens;
    p.per_gate = a.gate ? p.tokens / (int64_t)a.gate_rows : p.tokens;
    p.y_stride = (int64_t)a.y_stride;
    p.x_stride = (int64_t)a.x_stride;
    p.r_stride = (int64_t)a.r_stride;
    p.z_stride = (int64_t)a.z_stride;
    p.dim = (int)a.dim;
    p.bf16_weights = a.weight_dtype == HC_BFLOAT16;
    p.residual_scale = a.residual_scale;
    p.eps = a.eps;
    return a.dtype == HC_BFLOAT16 ? run_norm<Bf16>(p, stream) : run_norm<float>(p, stream);
}

BlockNormPlan block_norm_plan(int64_t tokens, int64_t dim, int64_t gate_rows, bool gate) {
    BlockNormPlan q = {};
    const int64_t gates = gate ? gate_rows : 1;
    const int64_t per_gate = tokens / gates;
    q.pitch = (dim + 7) / 8 * 8;
    q.slots = 2;
    if (!tokens) {
        q.by_group = gates >= kGradBlocks;  // nothing to divide: unit, per_group and blocks are 0
    } else if (gates < kGradBlocks) {
        const int64_t want = (kGradBlocks + gates - 1) / gates;
        q.unit = (per_gate + want - 1) / want;
        if (q.unit < 1) q.unit = 1;
        q.per_group = (per_gate + q.unit - 1) / q.unit;
        q.blocks = gates * q.per_group;
        q.slots = 3;
    } else {
        q.by_group = 1;
        q.unit = (gates + kGradBlocks - 1) / kGradBlocks;
        q.blocks = (gates + q.unit - 1) / q.unit;
    }
    q.bytes = (size_t)q.blocks * q.slots * q.pitch * sizeof(float);
    return q;
}

cudaError_t launch_block_norm_grad(const hc_block_norm_grad_t& a, cudaStream_t stream, int sms) {
    (void)sms;
    const BlockNormPlan q = block_norm_plan((int64_t)a.tokens, (int64_t)a.dim, (int64_t)a.gate_rows, a.gate != nullptr);
    NormGradParams p = {};
    p.grad_r = a.grad_r;
    p.grad_z = a.grad_z;
    p.y = a.y;
    p.x = a.x;
    p.post_weight = a.post_weight;
    p.gate = a.gate;
    p.pre_weight = a.pre_weight;
    p.post_rstd = a.post_rstd;
    p.pre_rstd = a.pre_rstd;
    p.grad_y = a.grad_y;
    p.grad_x = a.grad_x;
    p.grad_post_weight = a.grad_post_weight;
    p.grad_gate = a.grad_gate;
    p.grad_pre_weight = a.grad_pre_weight;
    p.part = (float*)a.scratch;
    p.tokens = (int64_t)a.tokens;
    p.gates = a.gate ? (int64_t)a.gate_rows : 1;
    p.per_gate = p.tokens / p.gates;
    p.grad_r_stride = (int64_t)a.grad_r_stride;
    p.grad_z_stride = (int64_t)a.grad_z_stride;
    p.y_stride = (int64_t)a.y_stride;
    p.x_stride = (int64_t)a.x_stride;
    p.grad_y_stride = (int64_t)a.grad_y_stride;
    p.grad_x_stride = (int64_t)a.grad_x_stride;
    p.blocks = q.blocks;
    p.unit = q.unit;
    p.per_group = q.per_group;
    p.pitch = q.pitch;
    p.slots = q.slots;
    p.dim = (int)a.dim;
    p.bf16_weights = a.weight_dtype == HC_BFLOAT16;
    p.residual_scale = a.residual_scale;
    return a.dtype == HC_BFLOAT16 ? run_norm_grad<Bf16>(p, q.by_group, stream) : run_norm_grad<float>(p, q.by_group, stream);
}

}  // namespace hc
