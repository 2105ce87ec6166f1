// hc_block_norm.cu -- the norm after a block, its gate, the scaled residual
// and the norm before the next block, and their gradient.
//
// A row stays on chip from its loads to its stores: forward, y and x are read
// once and r and z written once, with two row sums between (y^2, then r^2,
// which needs the first); backward, grad_r, grad_z, y and x are read once and
// grad_x and grad_y written once, again with two row sums.  What bounds both
// is the memory, so the kernels are built to keep loads in flight while rows
// wait for their sums:
//  - rows of up to 256 columns: a power of two of lanes of one warp has a row
//    (8 or 16 columns a lane); the sums are shuffles and many warps hide the loads;
//  - longer rows: a group of threads (as many columns each) works through its rows
//    while bulk copies bring the next ones into a ring of shared-memory
//    stages; a stage is free again after the row's first sum, when every
//    thread holds its columns in registers;
//  - rows longer than a block's threads hold are split over a cluster, whose
//    blocks exchange their sums through distributed shared memory.
//
// Rows that do not start on 16-byte boundaries: where all inputs' rows lie
// alike (contiguous ones of an odd dim), every vectors-of-an-alignment-period-th
// row starts at the same place in its first vector (the row's shift), so a
// group of threads keeps to rows of one shift and its threads to the aligned
// vectors of memory ("window"), the first and last of which hold only a part
// of the row.  Otherwise (gradients of gate rows of a few tokens, or of another
// type than the values, among them) the same kernels take one element per
// access, neighbouring threads on neighbouring columns.
//
// Measured, 16384 x 4096 bf16: forward 84 us (6.4 TB/s, 94 % of the copy
// bandwidth), gradient 144 us (5.6 TB/s, 82 %, with the sums of the weight
// gradients); one token 3.0 us.  Once loads are always on their way, what
// counts is instructions and the two barriers a row, hence pairs of binary32
// (forward 104 -> 84 us), weights kept across rows (165 -> 104) and 16 columns
// a thread.
//
// Weight gradients: sums over tokens of dz * rhat (pre) and A = D * yhat,
// from which the others follow: d gate = post_weight * sum A over the gate's
// tokens, d post_weight = sum gate * A.  A block sums its own run of tokens in
// registers and leaves partial sums in scratch; a second kernel adds them in
// a fixed order.
#include <algorithm>

#include "hc_ops.cuh"

namespace hc {
namespace {

// Columns of a thread.  More of them share the row sums' shuffles and barriers
// (16384 x 4096 bf16, gradient: 176 us with 8, 145 with 16), as far as the
// registers go: the gradient holds three rows' values and two sums, with 16
// columns the weights stay in shared memory, and with a sum more, for gate rows
// that end within a block, 8 columns are what fits.
constexpr int kCols = 16, kGradCols = 16, kGradFewCols = 8;
constexpr int kNormThreads = 512;  // of a block at most: up to 128 registers a thread
constexpr int kStages = 4;         // rows in flight of a group of threads at most
constexpr int kMaxGroups = 8;      // groups of threads (rows) of a block at most

// What the bulk copies of a row need of a matrix.
struct Operand {
    const void* base;
    int64_t stride;
};

// The ring of one group of threads: OPS operands a stage, operand o brought by
// lane o of the group's first warp (so that a row's copies are set up side by
// side).  ALIGNED: every row and slice starts and ends on 16 bytes.
template <class T, int OPS, bool ALIGNED>
struct Ring {
    unsigned char* data;
    uint64_t* full;
    const RowLayout& lay;
    int64_t tokens;
    int first, cols;  // this block's slice of the columns
    bool ok = true;
    int failed_at = 0;  // row whose wait gave up

    __device__ __forceinline__ static int shift_of(const T* p) {
        return ALIGNED ? 0 : (int)(((uintptr_t)p & 15) / sizeof(T));
    }
    __device__ __forceinline__ unsigned char* slot(int stage, int op) const {
        return data + (stage * OPS + op) * lay.slot;
    }
    // One thread of the group, before the block's first barrier.
    __device__ void init() const {
        for (int i = 0; i < lay.stages; i++) mbar_init(&full[i], OPS + (i == 0 ? lay.hold : 0));
        mbar_init_fence();
    }
    // Lane o: bring token t's row of its operand into a stage.  The copy takes
    // the whole 16-byte vectors that hold the slice, with neighbouring elements
    // of the matrix; only before its first and after its last element there
    // may be nothing, so those two vectors are filled element by element.
    __device__ __forceinline__ void load(int stage, int64_t t, int o, const Operand& op) const {
        if (!op.base || (ALIGNED && cols <= 0)) {  // the last block of a cluster may have no columns
            mbar_arrive(&full[stage]);
            return;
        }
        const T* p = (const T*)op.base + t * op.stride + first;
        unsigned char* to = slot(stage, o);
        if (ALIGNED) {
            mbar_arrive_expect_tx(&full[stage], (unsigned)cols * (unsigned)sizeof(T));
            bulk_g2s(to, (uintptr_t)p, (unsigned)cols * (unsigned)sizeof(T), &full[stage]);
            return;
        }
        const int shift = shift_of(p), end = shift + cols;
        if (end <= 0) {
            mbar_arrive(&full[stage]);
            return;
        }
        int lo = 0, hi = (end * (int)sizeof(T) + 15) / 16;
        T* q = (T*)to;
        if (shift && t == 0 && first == 0) {
            lo = 1;
            for (int i = shift; i < kVecOf<T> && i < end; i++) q[i] = p[i - shift];
        }
        if (end % kVecOf<T> && t == tokens - 1) {
            hi--;
            for (int i = max(hi * kVecOf<T>, first ? 0 : shift); i < end; i++) q[i] = p[i - shift];
        }
        const unsigned bytes = hi > lo ? (unsigned)(hi - lo) * 16 : 0u;
        mbar_arrive_expect_tx(&full[stage], bytes);
        if (bytes) bulk_g2s(to + lo * 16, ((uintptr_t)p & ~(uintptr_t)15) + (uintptr_t)lo * 16, bytes, &full[stage]);
    }
    // Wait for the k-th row (a whole warp).  After a wait that gave up the warp
    // goes on without waiting (its outputs are undefined) to the end of its
    // rows, and brings no more.
    __device__ __forceinline__ void wait(int stage, unsigned phase, bool first_row, bool leader) {
        if (!ok) return;
        const bool came = mbar_wait_quick(&full[stage], phase & 1, first_row ? lay.wait_ns : kWaitLimitNs);
        if (__all_sync(0xFFFFFFFFu, came)) return;
        ok = false;
        failed_at = (int)phase * lay.stages + stage;
        mbar_expired(&full[stage], lay.err, first_row ? lay.hold : 0, leader);
    }
    // After a wait gave up: let the copies of the first `issued` rows land
    // before the block leaves.
    __device__ void drain(int issued) const {
        for (int k = max(0, issued - lay.stages); k < issued; k++)
            mbar_wait_bounded(&full[k % lay.stages], (unsigned)(k / lay.stages) & 1, kWaitLimitNs);
    }
};

// Sum of v over the threads of a row (and the blocks of the cluster), in a
// fixed order.  Calls alternate between two slots of shared memory: a call's
// slot is written again only after the barrier of the call between, which
// every thread reaches after its reads.
constexpr int kRowWarps = kNormThreads / 32;
template <bool RING>
struct RowSum {
    float (*warp)[kMaxGroups * 4 + kRowWarps];  // [2][group * padded warps + warp], unused ones 0
    float (*rank)[kMaxCluster];                 // [2][rank], clusters have one group a block
    int tx, ty, cs;                             // threads of a row, this row's number
    int slot = 0;
    __device__ __forceinline__ int padded() const { return ((tx >> 5) + 3) & ~3; }
    // All threads of the block, before its first barrier.
    __device__ __forceinline__ void init(int thread, int threads) const {
        for (int i = thread; i < kMaxGroups * 4 + kRowWarps; i += threads) warp[0][i] = warp[1][i] = 0.0f;
    }
    __device__ __forceinline__ float operator()(float v) {
        if (!RING) {
            for (int o = tx >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            return v;
        }
        slot ^= 1;
        v = warp_sum(v);
        const int n = padded();
        float* const mine = &warp[slot][ty * n];
        if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(ty + 1), "r"(tx) : "memory");
        v = 0.0f;
        for (int i = 0; i < n; i += 4) {
            const float4 f = *(const float4*)(mine + i);
            v += (f.x + f.y) + (f.z + f.w);
        }
        if (cs > 1) {
            unsigned me;
            asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(me));
            if (threadIdx.x < (unsigned)cs) store_remote(&rank[slot][me], threadIdx.x, v);
            cluster_arrive();
            cluster_wait();
            v = 0.0f;
            for (int i = 0; i < cs; i++) v += rank[slot][i];
        }
        return v;
    }
};

// A thread's columns, in pairs: vectors v of N neighbouring ones, tx * N apart.
// N is 1, or dim is a multiple of N and every row aligned, so that a vector
// lies in the row as a whole or not at all; FULL: every vector lies in it.
// WIN: N elements are 16 aligned bytes of every row of this shift.
template <class T, int N, int C, bool FULL, bool WIN>
struct Columns {
    static constexpr int V = C / N;
    int begin, step, first, dim;  // vector 0's column, columns between vectors, the block's slice
    __device__ __forceinline__ Columns(int tid, int tx, int first_, int dim_, int shift)
        : begin(first_ + tid * N - (WIN ? shift : 0)), step(tx * N), first(first_), dim(dim_) {}
    __device__ __forceinline__ int at(int v) const { return begin + v * step; }
    // the whole vector lies in the row
    __device__ __forceinline__ bool in(int v) const {
        return FULL || (WIN ? at(v) >= 0 && at(v) + N <= dim : at(v) < dim);
    }

    // ALIGNED: of a row with the shift (weights have none); SLOT: in shared
    // memory, where a vector that only partly lies in the row may be read
    template <class S, bool ALIGNED = true, bool SLOT = false>
    __device__ __forceinline__ void get(const S* row, bool live, Pair (&x)[C / 2]) const {
        float f[C];
#pragma unroll
        for (int v = 0; v < V; v++) {
            float e[N];
            if (!WIN) {
                load_whole<S, N>(row + at(v), live && in(v), e);
            } else if (SLOT) {
                load_whole<S, N>(row + at(v), at(v) < dim, e);
                if (!in(v)) {
#pragma unroll
                    for (int i = 0; i < N; i++) e[i] = (unsigned)(at(v) + i) < (unsigned)dim ? e[i] : 0.0f;
                }
            } else if (ALIGNED && in(v)) {
                load_whole<S, N>(row + at(v), live, e);
            } else {
#pragma unroll
                for (int i = 0; i < N; i++)
                    e[i] = live && (unsigned)(at(v) + i) < (unsigned)dim ? to_f32(row[at(v) + i]) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < N; i++) f[v * N + i] = e[i];
        }
#pragma unroll
        for (int i = 0; i < C / 2; i++) x[i] = Pair(f[2 * i], f[2 * i + 1]);
    }
    __device__ __forceinline__ void load(const T* row, bool live, Pair (&x)[C / 2]) const { get<T>(row, live, x); }
    // from a ring's slot, whose element `place` is column `first`
    __device__ __forceinline__ void load(const unsigned char* slot, int place, Pair (&x)[C / 2]) const {
        get<T, true, true>((const T*)slot + place - first, true, x);
    }
    // aligned: the row has the shift
    template <class S>
    __device__ __forceinline__ void put_all(S* row, bool live, const Pair (&x)[C / 2], bool aligned) const {
        float f[C];
#pragma unroll
        for (int i = 0; i < C / 2; i++) x[i].get(f[2 * i], f[2 * i + 1]);
#pragma unroll
        for (int v = 0; v < V; v++) {
            float e[N];
#pragma unroll
            for (int i = 0; i < N; i++) e[i] = f[v * N + i];
            if (!WIN || (aligned && in(v))) {
                store_whole<S, N>(row + at(v), live && in(v), e);
            } else {
#pragma unroll
                for (int i = 0; i < N; i++)
                    if (live && (unsigned)(at(v) + i) < (unsigned)dim) put(row + at(v) + i, e[i]);
            }
        }
    }
    // a weight vector (ones where there is none)
    __device__ __forceinline__ void weight(const void* w, bool bf16, int64_t row, Pair (&x)[C / 2]) const {
        if (!w) {
#pragma unroll
            for (int i = 0; i < C / 2; i++) x[i] = Pair(1.0f, 1.0f);
        } else if (bf16) {
            get<Bf16, false>((const Bf16*)w + row * dim, true, x);
        } else {
            get<float, false>((const float*)w + row * dim, true, x);
        }
    }
};
__device__ __forceinline__ float both(Pair a) {
    float lo, hi;
    a.get(lo, hi);
    return lo + hi;
}

struct NormParams {
    Operand in[2];  // y, x
    const void *post_weight, *gate, *pre_weight;
    void *r, *z;
    float *post_rstd, *pre_rstd;
    int64_t tokens, r_stride, z_stride;
    unsigned per_gate;
    int dim;
    bool bf16_weights, alike[2];  // r and z lie in their vectors as y and x do
    float residual_scale, eps;
    RowLayout lay;
};

// blockDim = (tx, ty) for a ring, (tx * ty) for rows in warps.
template <class T, int N, bool RING, bool FULL, bool WIN>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormParams p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ uint64_t full[kMaxGroups][kStages];
    __shared__ __align__(16) float warp_sums[2][kMaxGroups * 4 + kRowWarps];
    __shared__ float rank_sums[2][kMaxCluster];
    const RowLayout& L = p.lay;
    const int tid = RING ? threadIdx.x : threadIdx.x % L.tx;
    const int ty = RING ? threadIdx.y : threadIdx.x / L.tx;
    const int rank = RING ? blockIdx.x % L.cs : 0;
    constexpr int H = kCols / 2;
    RowSum<RING> row_sum{warp_sums, rank_sums, L.tx, ty, L.cs};
    const int64_t start = (int64_t)(blockIdx.x / L.cs) * L.ty + ty;
    const int64_t step = (int64_t)(gridDim.x / L.cs) * L.ty;
    // with a window, the rows of this group of threads all have this shift
    const int shift = WIN ? (int)((uintptr_t)((const T*)p.in[0].base + start * p.in[0].stride) & 15) / (int)sizeof(T) : 0;
    const Columns<T, N, kCols, FULL, WIN> col(tid, L.tx, rank * L.tx * kCols, p.dim, shift);
    Ring<T, 2, (N > 1 && !WIN)> ring{dyn + (size_t)ty * L.stages * 2 * L.slot, full[ty], L, p.tokens, col.first,
                             min(L.tx * kCols, p.dim - col.first)};
    if (RING) {
        if (tid == 0) ring.init();
        row_sum.init(threadIdx.y * L.tx + tid, L.tx * L.ty);
        if (L.cs > 1) cluster_arrive();
        __syncthreads();
        if (L.cs > 1) cluster_wait();  // every block of the cluster runs
    }
    grid_wait();
    grid_release();
    int64_t next = start;  // token of the next row to bring
    int issued = 0;
    if (RING && tid < 2)
        for (; issued < L.stages && next < p.tokens; issued++, next += step) ring.load(issued, next, tid, p.in[tid]);
    const float inv_dim = 1.0f / (float)p.dim;
    const Pair scale(p.residual_scale, p.residual_scale);
    Pair wg[H], pw[H];  // post_weight * gate, pre_weight
    int64_t gate_end = -1;       // of the tokens that wg is for
    col.weight(p.pre_weight, p.bf16_weights, 0, pw);
    int stage = 0;
    unsigned phase = 0;
    for (int64_t t = start;; t += step) {
        // rows in warps: every lane takes part in the shuffles of its one row
        const bool live = t < p.tokens;
        if (RING && !live) break;
        Pair y[H], x[H];
        const T* yrow = (const T*)p.in[0].base + t * p.in[0].stride;
        const T* xrow = (const T*)p.in[1].base + t * p.in[1].stride;
        if (!RING) {
            col.load(yrow, live, y);
            col.load(xrow, live, x);
        }
        if (t >= gate_end) {
            const int64_t g = live ? (unsigned)t / p.per_gate : 0;
            gate_end = (g + 1) * p.per_gate;
            Pair gt[H];
            col.weight(p.post_weight, p.bf16_weights, 0, wg);
            col.weight(p.gate, p.bf16_weights, g, gt);
#pragma unroll
            for (int i = 0; i < H; i++) wg[i] = wg[i] * gt[i];
        }
        if (RING) {
            ring.wait(stage, phase, t == start, tid == 0);
            col.load(ring.slot(stage, 0), ring.shift_of(yrow + col.first), y);
            col.load(ring.slot(stage, 1), ring.shift_of(xrow + col.first), x);
        }
        Pair s(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < H; i++) s = fma_pair(y[i], y[i], s);
        const float post = rsqrtf(fmaf(row_sum(both(s)), inv_dim, p.eps));
        const Pair post2(post, post);
        if (RING) {
            if (tid < 2 && ring.ok && next < p.tokens) {
                ring.load(stage, next, tid, p.in[tid]);
                issued++;
                next += step;
            }
            if (++stage == L.stages) {
                stage = 0;
                phase++;
            }
        }
        s = Pair(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < H; i++) {
            x[i] = fma_pair(wg[i], y[i] * post2, scale * x[i]);
            s = fma_pair(x[i], x[i], s);
        }
        col.put_all((T*)p.r + t * p.r_stride, live, x, p.alike[0]);
        const bool first = tid == 0 && rank == 0 && live;
        if (first && p.post_rstd) p.post_rstd[t] = post;
        if (p.z) {
            const float pre = rsqrtf(fmaf(row_sum(both(s)), inv_dim, p.eps));
            if (first && p.pre_rstd) p.pre_rstd[t] = pre;
            const Pair pre2(pre, pre);
#pragma unroll
            for (int i = 0; i < H; i++) x[i] = x[i] * (pre2 * pw[i]);
            col.put_all((T*)p.z + t * p.z_stride, live, x, p.alike[1]);
        }
        if (!RING) break;
    }
    if (RING && tid == 0 && !ring.ok) ring.drain(issued);
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
struct NormGradParams {
    Operand in[5];  // grad_r, grad_z, y, x, and the gate where every token has its own
    const void *post_weight, *gate, *pre_weight;
    const float *post_rstd, *pre_rstd;
    void *grad_y, *grad_x, *grad_post_weight, *grad_gate, *grad_pre_weight;
    float* part;         // [block][slot][pitch]: gate * A, dz * rhat, A
    int64_t tokens, gates;
    int64_t grad_y_stride, grad_x_stride;
    int64_t blocks, per_group, pitch, jobs;
    unsigned per_gate, unit;
    int dim, slots;
    bool bf16_weights, alike[3];  // grad_x, grad_y (grad_gate, if each token's) lie in their vectors as the inputs do
    bool direct;  // one block: no partial sums
    float residual_scale;
    RowLayout lay;
};

// Add the rows' sums of a block into row 0's, in row order.
template <int C>
__device__ __forceinline__ void join_rows(int tid, int tx, int ty, int rows, float* joined, Pair (&sums)[C / 2]) {
    if (rows == 1) return;
    float acc[C];
#pragma unroll
    for (int i = 0; i < C / 2; i++) sums[i].get(acc[2 * i], acc[2 * i + 1]);
    float* mine = joined + ty * tx + tid;
    const int pitch = rows * tx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C; i++) mine[i * pitch] = acc[i];
    __syncthreads();
    if (ty) return;
    for (int r = 1; r < rows; r++)
#pragma unroll
        for (int i = 0; i < C; i++) acc[i] += mine[i * pitch + r * tx];
#pragma unroll
    for (int i = 0; i < C / 2; i++) sums[i] = Pair(acc[2 * i], acc[2 * i + 1]);
}
// The joined sums as a row of partial sums.
template <class T, int N, int C, bool FULL, bool WIN>
__device__ __forceinline__ void store_part(const Columns<T, N, C, FULL, WIN>& col, int tid, int tx, int ty, int rows,
                                           float* joined, float* part, Pair (&sums)[C / 2]) {
    join_rows<C>(tid, tx, ty, rows, joined, sums);
    if (ty == 0) col.put_all(part, true, sums, false);
}
// The joined sums as a weight's gradient (which may not be wanted).
template <class T, int N, int C, bool FULL, bool WIN>
__device__ __forceinline__ void store_direct(const Columns<T, N, C, FULL, WIN>& col, int tid, int tx, int ty, int rows,
                                             float* joined, void* out, bool bf16, Pair (&sums)[C / 2]) {
    join_rows<C>(tid, tx, ty, rows, joined, sums);
    if (ty || !out) return;
    if (bf16) col.put_all((Bf16*)out, true, sums, false);
    else col.put_all((float*)out, true, sums, false);
}

// GROUPS false: the block's run of `unit` tokens lies in one gate row, its
// tokens are dealt to the block's rows of threads; with a window, the run is
// of every kClasses-th token, which all have the same shift.  true: the block
// has `unit` whole gate rows, dealt to the rows of threads.
// EACH: every token has a gate row, of the values' type: one more operand of
// its row, brought ahead with the others, and grad_gate one more output; else
// as without gates.
constexpr int kClasses = 8;
template <class T, int N, bool RING, bool GROUPS, bool FULL, bool WIN, int C, bool EACH = false>
__global__ void __launch_bounds__(kNormThreads) norm_grad_kernel(const NormGradParams p) {
    constexpr int H = C / 2;
    constexpr bool SHARED_WEIGHTS = C == kGradCols;
    constexpr int OPS = EACH ? 5 : 4;
    // yhat between the sums: out of the stage again instead of 16 registers
    // that spill (144 us instead of 158 for 16384 x 4096 bf16; in a window, whose
    // reads take more, 240 us instead of 213 for 16384 x 3001)
    constexpr bool REREAD = RING && C == kGradCols && !WIN;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ uint64_t full[kMaxGroups][kStages];
    __shared__ __align__(16) float warp_sums[2][kMaxGroups * 4 + kRowWarps];
    __shared__ float rank_sums[2][kMaxCluster];
    const RowLayout& L = p.lay;
    const int tid = RING ? threadIdx.x : threadIdx.x % L.tx;
    const int ty = RING ? threadIdx.y : threadIdx.x / L.tx;
    const int rank = RING ? blockIdx.x % L.cs : 0;
    const int64_t block = blockIdx.x / L.cs;
    RowSum<RING> row_sum{warp_sums, rank_sums, L.tx, ty, L.cs};
    // this row of threads has `count` tokens; steps: what the warp goes
    // through together (rows in warps)
    unsigned count, steps;
    int64_t gate_row, base;
    if (GROUPS) {
        const int64_t first = block * p.unit;
        const unsigned have = (unsigned)min((int64_t)p.unit, p.gates - first);
        count = ((unsigned)ty < have ? (have - ty - 1) / L.ty + 1 : 0u) * p.per_gate;
        steps = (p.unit + L.ty - 1) / L.ty * p.per_gate;
        gate_row = first + ty;
        base = 0;
    } else {
        gate_row = block / p.per_group;
        const unsigned b = (unsigned)(block % p.per_group), klass = WIN ? b % kClasses : 0, apart = WIN ? kClasses : 1;
        const unsigned lo = b / apart * p.unit, all = (p.per_gate - klass + apart - 1) / apart;  // tokens of the class
        const unsigned have = lo < all ? min(p.unit, all - lo) : 0u;
        count = (unsigned)ty < have ? (have - ty - 1) / L.ty + 1 : 0u;
        steps = (p.unit + L.ty - 1) / L.ty;
        base = gate_row * p.per_gate + klass + (int64_t)apart * (lo + ty);
    }
    const int shift = WIN ? (int)((uintptr_t)((const T*)p.in[2].base + base * p.in[2].stride) & 15) / (int)sizeof(T) : 0;
    const Columns<T, N, C, FULL, WIN> col(tid, L.tx, rank * L.tx * C, p.dim, shift);
    Ring<T, OPS, (N > 1 && !WIN)> ring{dyn + (size_t)ty * L.stages * OPS * L.slot, full[ty], L, p.tokens, col.first,
                             min(L.tx * C, p.dim - col.first)};
    // the tokens in order: the one to do, and (lanes that bring rows) the next
    // one to bring
    struct Walk {
        int64_t t, gate;
        unsigned in_gate;
    };
    auto advance = [&](Walk& w) {
        if (!GROUPS) {
            w.t += WIN ? kClasses * L.ty : L.ty;
        } else if (++w.in_gate == p.per_gate) {
            w.in_gate = 0;
            w.gate += L.ty;
            w.t = w.gate * p.per_gate;
        } else {
            w.t++;
        }
    };
    Walk now{GROUPS ? gate_row * p.per_gate : base, gate_row, 0};
    if (RING) {
        if (tid == 0) ring.init();
        row_sum.init(threadIdx.y * L.tx + tid, L.tx * L.ty);
        if (L.cs > 1) cluster_arrive();
        __syncthreads();
        if (L.cs > 1) cluster_wait();
        steps = count;
    }
    grid_wait();
    grid_release();
    Walk next = now;
    if (RING && tid < OPS)
        for (unsigned i = 0; i < (unsigned)L.stages && i < count; i++) {
            ring.load((int)i, next.t, tid, p.in[tid]);
            advance(next);
        }
    const float inv_dim = 1.0f / (float)p.dim;
    const Pair zero(0.0f, 0.0f), scale(p.residual_scale, p.residual_scale);
    Pair a[H], ga[H], pre_acc[H];
#pragma unroll
    for (int i = 0; i < H; i++) a[i] = ga[i] = pre_acc[i] = zero;
    // post_weight * gate (EACH: post_weight) and pre_weight: in registers, or a pair of columns
    // each in shared memory (one copy a block: its tokens share the gate)
    Pair wg_[SHARED_WEIGHTS ? 1 : H], pw_[SHARED_WEIGHTS ? 1 : H];
    float4* const shared_weights = (float4*)(dyn + (size_t)L.ty * L.stages * OPS * L.slot) + tid;
    auto load_gate = [&](int64_t g) {
        Pair wg[H], gt[H];
        col.weight(p.post_weight, p.bf16_weights, 0, wg);
        if (!EACH) col.weight(p.gate, p.bf16_weights, g, gt);
#pragma unroll
        for (int i = 0; i < H; i++) {
            if (!EACH) wg[i] = wg[i] * gt[i];
            if constexpr (!SHARED_WEIGHTS) wg_[i] = wg[i];
        }
        if constexpr (SHARED_WEIGHTS) {
            Pair pw[H];
            col.weight(p.pre_weight, p.bf16_weights, 0, pw);
#pragma unroll
            for (int i = 0; i < H; i++) {
                float4 f;
                wg[i].get(f.x, f.y);
                pw[i].get(f.z, f.w);
                if (ty == 0) shared_weights[i * L.tx] = f;
            }
        }
    };
    auto weights = [&](int i, Pair& wg, Pair& pw) {
        if constexpr (SHARED_WEIGHTS) {
            const float4 f = shared_weights[i * L.tx];
            wg = Pair(f.x, f.y);
            pw = Pair(f.z, f.w);
        } else {
            wg = wg_[i];
            pw = pw_[i];
        }
    };
    if constexpr (SHARED_WEIGHTS) {
        load_gate(now.gate);
        __syncthreads();
    } else {
        col.weight(p.pre_weight, p.bf16_weights, 0, pw_);
        if (count) load_gate(now.gate);
    }
    int stage = 0;
    unsigned phase = 0;
    for (unsigned k = 0; k < steps; k++) {
        const bool live = k < count;
        const int64_t t = now.t;
        // every thread has taken its columns: bring the next row in their place
        auto bring = [&]() {
            if (tid < OPS && ring.ok && k + L.stages < count) {
                ring.load(stage, GROUPS ? next.t : t + (WIN ? kClasses : 1) * L.ty * L.stages, tid, p.in[tid]);
                if (GROUPS) advance(next);
            }
            if (++stage == L.stages) {
                stage = 0;
                phase++;
            }
        };
        Pair d0[H], y[H], rh[H], gt[H];  // gt: EACH, the gate, then its gradient
#pragma unroll
        for (int i = 0; i < H; i++) d0[i] = y[i] = rh[i] = zero;
        const float post = live ? p.post_rstd[t] : 0.0f;
        const float pre = live && p.in[1].base ? p.pre_rstd[t] : 0.0f;
        // y -> yhat; x -> rhat; h = gz * pre_weight; d0 = gr + pre * h
        const Pair post2(post, post), pre2(pre, pre);
        auto load = [&](int o, Pair (&v)[H]) {
            const T* row = (const T*)p.in[o].base + t * p.in[o].stride;
            if (!p.in[o].base) {
#pragma unroll
                for (int i = 0; i < H; i++) v[i] = zero;
            } else if (RING) {
                col.load(ring.slot(stage, o), ring.shift_of(row + col.first), v);
            } else {
                col.load(row, true, v);
            }
        };
        Pair s = zero;
        if (RING || live) {
            Pair gz[H];
            if (RING) ring.wait(stage, phase, k == 0, tid == 0);
            load(0, d0);
            load(1, gz);
            load(2, y);
            load(3, rh);
            if constexpr (EACH) load(4, gt);
#pragma unroll
            for (int i = 0; i < H; i++) {
                Pair wg, pw;
                weights(i, wg, pw);
                if (EACH) wg = wg * gt[i];
                y[i] = y[i] * post2;
                rh[i] = fma_pair(wg, y[i], scale * rh[i]) * pre2;
                pre_acc[i] = fma_pair(gz[i], rh[i], pre_acc[i]);
                const Pair h = gz[i] * pw;
                s = fma_pair(h, rh[i], s);
                d0[i] = fma_pair(pre2, h, d0[i]);
            }
        }
        const float m1 = -pre * (row_sum(both(s)) * inv_dim);
        if (RING && !REREAD) bring();
        // d = gr + pre (h - rhat mean(h rhat)), k = d * gate * post_weight
        s = zero;
        const Pair m12(m1, m1);
        if (RING || live) {
            if (REREAD) load(2, y);
            if constexpr (EACH && REREAD) load(4, gt);
#pragma unroll
            for (int i = 0; i < H; i++) {
                Pair wg, pw;
                weights(i, wg, pw);
                if (REREAD) y[i] = y[i] * post2;
                const Pair d = fma_pair(m12, rh[i], d0[i]);
                if (EACH) {
                    const Pair dy = d * y[i], g = gt[i];
                    ga[i] = fma_pair(g, dy, ga[i]);
                    gt[i] = wg * dy;
                    wg = wg * g;
                } else {
                    a[i] = fma_pair(d, y[i], a[i]);
                }
                rh[i] = scale * d;
                d0[i] = d * wg;
                s = fma_pair(d0[i], y[i], s);
            }
        }
        col.put_all((T*)p.grad_x + t * p.grad_x_stride, live, rh, p.alike[0]);
        if (EACH && p.grad_gate) col.put_all((T*)p.grad_gate + t * p.dim, live, gt, p.alike[2]);
        const float m2 = -row_sum(both(s)) * inv_dim;
        if (REREAD) bring();
        const Pair m22(m2, m2);
#pragma unroll
        for (int i = 0; i < H; i++) d0[i] = post2 * fma_pair(m22, y[i], d0[i]);
        col.put_all((T*)p.grad_y + t * p.grad_y_stride, live, d0, p.alike[1]);
        if (GROUPS && now.in_gate + 1 == p.per_gate) {  // A of this gate row is complete
            Pair w[H];
            col.weight(p.gate, p.bf16_weights, live ? now.gate : 0, w);
            if (RING || live) {
#pragma unroll
                for (int i = 0; i < H; i++) ga[i] = fma_pair(w[i], a[i], ga[i]);
            }
            if (p.grad_gate && live) {
                col.weight(p.post_weight, p.bf16_weights, 0, w);
#pragma unroll
                for (int i = 0; i < H; i++) w[i] = w[i] * a[i];
                if (p.bf16_weights) col.put_all((Bf16*)p.grad_gate + now.gate * p.dim, true, w, false);
                else col.put_all((float*)p.grad_gate + now.gate * p.dim, true, w, false);
            }
#pragma unroll
            for (int i = 0; i < H; i++) a[i] = zero;
            if (k + 1 < count) load_gate(now.gate + L.ty);
        }
        advance(now);
    }
    if (RING && tid == 0 && !ring.ok) ring.drain((int)min(count, (unsigned)(ring.failed_at + L.stages)));
    __syncthreads();  // every row has left the ring, whose memory the sums reuse
    if (!GROUPS && !EACH) {
        Pair gt[H];
        col.weight(p.gate, p.bf16_weights, gate_row, gt);
#pragma unroll
        for (int i = 0; i < H; i++) ga[i] = gt[i] * a[i];
    }
    float* joined = (float*)dyn;
    if (!WIN && !EACH && p.direct) {  // the only block: these are the sums
        store_direct(col, tid, L.tx, ty, L.ty, joined, p.grad_post_weight, p.bf16_weights, ga);
        store_direct(col, tid, L.tx, ty, L.ty, joined, p.grad_pre_weight, p.bf16_weights, pre_acc);
        if (!GROUPS) {
            join_rows<C>(tid, L.tx, ty, L.ty, joined, a);
            Pair w[H];
            col.weight(p.post_weight, p.bf16_weights, 0, w);
#pragma unroll
            for (int i = 0; i < H; i++) a[i] = a[i] * w[i];
            store_direct(col, tid, L.tx, ty, 1, joined, p.grad_gate, p.bf16_weights, a);
        }
        return;
    }
    float* part = p.part + block * p.slots * p.pitch;
    store_part(col, tid, L.tx, ty, L.ty, joined, part, ga);
    store_part(col, tid, L.tx, ty, L.ty, joined, part + p.pitch, pre_acc);
    if (!GROUPS && !EACH) store_part(col, tid, L.tx, ty, L.ty, joined, part + 2 * p.pitch, a);
}

// Sums of the partial rows: job 0: post weight, 1: pre weight, 2 + g: gate
// row g.  The warps add equal parts of the list, joined in order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) norm_sum_kernel(const NormGradParams p) {
    __shared__ float sums[kSumWarps][32];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t job = blockIdx.y; job < p.jobs; job += gridDim.y) {
        void* out = job == 0 ? p.grad_post_weight : job == 1 ? p.grad_pre_weight : p.grad_gate;
        if (!out) continue;
        const int64_t g = job - 2;
        const int64_t first = job < 2 ? 0 : g * p.per_group, count = job < 2 ? p.blocks : p.per_group;
        const int c = blockIdx.x * 32 + lane;
        const float* src = p.part + (first * p.slots + (job < 2 ? job : 2)) * p.pitch + c;
        const int64_t per = (count + kSumWarps - 1) / kSumWarps;
        const int64_t a = warp * per, b = a + per < count ? a + per : count;
        float acc = 0.0f;
        if (c < p.dim) {
#pragma unroll 8
            for (int64_t k = a; k < b; k++) acc += src[k * p.slots * p.pitch];
        }
        __syncthreads();  // the last job's sums have been read
        sums[warp][lane] = acc;
        __syncthreads();
        if (warp || c >= p.dim) continue;
        for (int w = 1; w < kSumWarps && w * per < count; w++) acc += sums[w][lane];
        if (job >= 2 && p.post_weight && count)  // no tokens: zeros (0 * inf)
            acc *= p.bf16_weights ? to_f32(((const Bf16*)p.post_weight)[c]) : ((const float*)p.post_weight)[c];
        const int64_t at = (job < 2 ? 0 : g * p.dim) + c;
        if (p.bf16_weights) put((Bf16*)out + at, acc);
        else put((float*)out + at, acc);
    }
}

// Launch shape for rows of `dim` columns of es bytes, `ops` operands loaded.
// Rows in one warp up to here: 32768 x 256 bf16 takes 14.3 us forward, 20.7 in a
// ring; 16384 x 512 takes 14.7 in a warp (16 columns a lane), 11.8 in a ring.
constexpr int64_t kWarpDim = 256;
constexpr int kStageBytes = 192 << 10;  // of an SM's blocks together
// Rows of up to 256 columns are one warp's, in_warp columns a lane.
RowLayout row_layout(int64_t dim, int es, int ops, RowAccess access, int in_warp, int per_thread, int block_threads) {
    RowLayout L = {};
    // a window begins up to a vector less one element before the row
    const int64_t wide = dim + (access == ROWS_WINDOW ? 16 / es - 1 : 0), threads = (wide + per_thread - 1) / per_thread;
    L.cs = 1;
    if (wide <= kWarpDim) {
        L.tx = 1;
        while (L.tx * in_warp < wide) L.tx *= 2;
        L.ty = 256 / L.tx;
        return L;
    }
    // four fp32 rows of 8192 columns leave no room for a second stage
    const bool weights = per_thread == kGradCols && ops >= 4;
    while (threads > (int64_t)(weights && es == 4 ? kNormThreads / 2 : kNormThreads) * L.cs) L.cs *= 2;
    L.tx = (int)(((threads + L.cs - 1) / L.cs + 31) / 32 * 32);
    L.ty = L.cs > 1 ? 1 : std::max(1, std::min(kMaxGroups, block_threads / L.tx));
    const int64_t cols = std::min<int64_t>(dim, (int64_t)L.tx * per_thread);
    L.slot = (int)((cols * es + (access == ROWS_VECTORS ? 0 : 16) + 15) / 16 * 16);
    if (weights) L.weights = L.tx * kGradCols * 2 * (int)sizeof(float);
    const int64_t stage = (int64_t)L.slot * ops * L.ty;
    L.stages = (int)std::min<int64_t>(kStages, (kStageBytes / (kNormThreads / (L.tx * L.ty)) - L.weights) / stage);
    // one block an SM, and on top of its bytes what two stages of unaligned slots
    // have more (bf16, gradient of 4096 x 8185: 127 us, 141 with the one stage that
    // fits otherwise; 2048 x 15355, in clusters: 205 and 205)
    const int more = access == ROWS_VECTORS ? 0 : 2 * 16 * ops * L.ty;
    if (L.stages < 2) L.stages = (int)((kStageBytes + more - L.weights) / stage);
    return L;
}

template <class T>
bool wide(const void* p, int64_t stride, int64_t dim) {
    return ((uintptr_t)p & 15) == 0 && (stride * (int64_t)sizeof(T) & 15) == 0 && (dim * (int64_t)sizeof(T) & 15) == 0;
}
// Places matrices' rows in 16-byte vectors: whether all lie alike.
struct Alike {
    bool any = false, alike = true;
    uintptr_t phase = 0, pitch = 0;
    template <class T>
    void add(const T*, const void* p, int64_t stride) {
        if (!p) return;
        const uintptr_t a = (uintptr_t)p & 15, b = (uintptr_t)(stride * (int64_t)sizeof(T)) & 15;
        if (any && (a != phase || b != pitch)) alike = false;
        any = true;
        phase = a;
        pitch = b;
    }
    template <class T>
    bool with(const T* t, const void* p, int64_t stride) const {
        Alike both = *this;
        both.add(t, p, stride);
        return both.alike;
    }
};
bool wide_weight(const void* w, bool bf16, int64_t dim) {
    return !w || (bf16 ? wide<Bf16>(w, dim, dim) : wide<float>(w, dim, dim));
}

// Fills the parts of the layout that depend on the device, and launches.
cudaError_t launch_rows(const void* fn, RowLayout* L, int ops, int64_t grid, void** args, size_t least_smem, cudaStream_t stream) {
    L->err = device_error_flag();
    if (!L->err || L->cs > kMaxCluster) return cudaErrorInvalidValue;
    L->hold = expiring_waits() ? 1 : 0;
    L->wait_ns = L->hold ? kTestWaitLimitNs : kWaitLimitNs;
    if (grid * L->cs > INT32_MAX) return cudaErrorInvalidValue;
    const size_t smem = std::max(least_smem, (size_t)L->slot * ops * L->stages * L->ty + L->weights);
    if (!allow_smem((void*)fn, (int)smem)) return cudaErrorInvalidValue;
    const dim3 block = L->stages ? dim3(L->tx, L->ty) : dim3(L->tx * L->ty);
    return launch_op(fn, dim3((unsigned)(grid * L->cs)), block, args, smem, stream, L->cs);
}

template <class T>
cudaError_t run_norm(NormParams& p, cudaStream_t stream, int sms) {
    constexpr int E = kVecOf<T>;
    const bool vec = wide<T>(p.in[0].base, p.in[0].stride, p.dim) && wide<T>(p.in[1].base, p.in[1].stride, p.dim) &&
                     wide<T>(p.r, p.r_stride, p.dim) && (!p.z || wide<T>(p.z, p.z_stride, p.dim)) &&
                     wide_weight(p.post_weight, p.bf16_weights, p.dim) && wide_weight(p.gate, p.bf16_weights, p.dim) &&
                     wide_weight(p.pre_weight, p.bf16_weights, p.dim);
    Alike rows;
    rows.add((const T*)nullptr, p.in[0].base, p.in[0].stride);
    rows.add((const T*)nullptr, p.in[1].base, p.in[1].stride);
    p.alike[0] = rows.with((const T*)nullptr, p.r, p.r_stride);
    p.alike[1] = rows.with((const T*)nullptr, p.z, p.z_stride);
    const BlockNormRows shape = block_norm_rows(p.dim, sizeof(T), vec, rows.alike);
    const RowAccess access = shape.access;
    p.lay = shape.lay;
    const bool ring = p.lay.stages > 0;
    int64_t grid = (p.tokens + p.lay.ty - 1) / p.lay.ty;
    if (ring) {
        const int64_t resident = std::max(1, sms * (kNormThreads / (p.lay.tx * p.lay.ty)) / p.lay.cs);
        // in a window, rows of a group are a multiple of 8 apart (or it has one):
        // they have the same shift
        if (grid > resident) grid = access != ROWS_WINDOW ? resident : resident >= 8 ? resident / 8 * 8 : grid;
    }
    const bool full = (int64_t)p.lay.tx * p.lay.cs * kCols == p.dim;
    const void* fn;
    if (access == ROWS_VECTORS)
        fn = ring ? (full ? (const void*)norm_kernel<T, E, true, true, false> : (const void*)norm_kernel<T, E, true, false, false>)
                  : (const void*)norm_kernel<T, E, false, false, false>;
    else if (access == ROWS_WINDOW)
        fn = ring ? (const void*)norm_kernel<T, E, true, false, true> : (const void*)norm_kernel<T, E, false, false, true>;
    else
        fn = ring ? (const void*)norm_kernel<T, 1, true, false, false> : (const void*)norm_kernel<T, 1, false, false, false>;
    void* args[] = {&p};
    return launch_rows(fn, &p.lay, 2, grid, args, 0, stream);
}

template <class T, int N, bool RING, bool FULL>
const void* pick_grad(bool by_group) {
    return by_group ? (const void*)norm_grad_kernel<T, N, RING, true, FULL, false, kGradFewCols>
                    : (const void*)norm_grad_kernel<T, N, RING, false, FULL, false, (RING && N > 1 ? kGradCols : kGradFewCols)>;
}

// Blocks (and partial sums) aimed at: two of 256 threads an SM, or one of 512.
constexpr int64_t kGradBlocks = 152;

// Threads of 16 bf16 columns whose stages of five operands fit twice beside
// their weights: 2 * 5 * 32 + 128 bytes a thread.
constexpr int kEachThreads = 416;
static_assert(kEachThreads * (2 * 5 * kGradCols * 2 + kGradCols * 2 * 4) <= kStageBytes, "two stages");

template <class T>
cudaError_t run_norm_grad(NormGradParams& p, const BlockNormPlan& q, cudaStream_t stream) {
    constexpr int E = kVecOf<T>;
    bool vec = wide<T>(p.grad_y, p.grad_y_stride, p.dim) && wide<T>(p.grad_x, p.grad_x_stride, p.dim) &&
               wide_weight(p.post_weight, p.bf16_weights, p.dim) && wide_weight(p.gate, p.bf16_weights, p.dim) &&
               wide_weight(p.pre_weight, p.bf16_weights, p.dim) && wide_weight(p.grad_gate, p.bf16_weights, p.dim) &&
               (!p.direct || (wide_weight(p.grad_post_weight, p.bf16_weights, p.dim) &&
                              wide_weight(p.grad_pre_weight, p.bf16_weights, p.dim)));
    for (const Operand& o : p.in) vec = vec && (!o.base || wide<T>(o.base, o.stride, p.dim));
    Alike rows;
    for (const Operand& o : p.in) rows.add((const T*)nullptr, o.base, o.stride);
    p.alike[0] = rows.with((const T*)nullptr, p.grad_x, p.grad_x_stride);
    p.alike[1] = rows.with((const T*)nullptr, p.grad_y, p.grad_y_stride);
    p.alike[2] = rows.with((const T*)nullptr, p.grad_gate, p.dim);
    BlockNormPlan plan = q;
    const BlockNormRows shape = block_norm_grad_rows(&plan, p.tokens, p.dim, sizeof(T), vec, rows.alike);
    p.unit = (unsigned)plan.unit;
    p.per_group = plan.per_group;
    p.blocks = plan.blocks;
    p.lay = shape.lay;
    const RowAccess access = shape.access;
    const int cols = shape.cols, ops = shape.ops;
    const bool by_group = plan.by_group, each = plan.each, one_block = each && cols == kGradCols;
    const bool ring = p.lay.stages > 0;
    const bool full = (int64_t)p.lay.tx * p.lay.cs * cols == p.dim;
    const void* fn;
    if (each)  // rows of more than kWarpDim columns: always a ring
        fn = one_block ? (const void*)norm_grad_kernel<Bf16, kVecOf<Bf16>, true, false, false, false, kGradCols, true>
             : access == ROWS_VECTORS ? (const void*)norm_grad_kernel<T, E, true, false, false, false, kGradFewCols, true>
             : access == ROWS_WINDOW ? (const void*)norm_grad_kernel<T, E, true, false, false, true, kGradFewCols, true>
                                : (const void*)norm_grad_kernel<T, 1, true, false, false, false, kGradFewCols, true>;
    else if (access == ROWS_VECTORS)
        fn = ring ? (full ? pick_grad<T, E, true, true>(by_group) : pick_grad<T, E, true, false>(by_group))
                  : pick_grad<T, E, false, false>(by_group);
    else if (access == ROWS_WINDOW)
        fn = ring ? (const void*)norm_grad_kernel<T, E, true, false, false, true, (sizeof(T) == 2 ? kGradCols : kGradFewCols)>
                  : (const void*)norm_grad_kernel<T, E, false, false, false, true, kGradFewCols>;
    else
        fn = ring ? pick_grad<T, 1, true, false>(by_group) : pick_grad<T, 1, false, false>(by_group);
    void* args[] = {&p};
    if (p.blocks > 0) {
        const size_t joined = p.lay.ty > 1 ? (size_t)p.lay.tx * p.lay.ty * cols * sizeof(float) : 0;
        const cudaError_t e = launch_rows(fn, &p.lay, ops, p.blocks, args, joined, stream);
        if (e != cudaSuccess) return e;
    }
    // gate rows by_group blocks have not written; without tokens all are zeros
    p.jobs = 2 + (p.grad_gate && !each && (!by_group || p.blocks == 0) ? p.gates : 0);
    if (p.direct || (!p.grad_post_weight && !p.grad_pre_weight && p.jobs == 2)) return cudaSuccess;
    return launch_op((const void*)norm_sum_kernel,
                     dim3((unsigned)((p.dim + 31) / 32), (unsigned)(p.jobs < 65535 ? p.jobs : 65535)),
                     dim3(kSumWarps * 32), args, 0, stream);
}

}  // namespace

cudaError_t launch_block_norm(const hc_block_norm_t& a, cudaStream_t stream, int sms) {
    NormParams p = {};
    p.in[0] = {a.y, (int64_t)a.y_stride};
    p.in[1] = {a.x, (int64_t)a.x_stride};
    p.post_weight = a.post_weight;
    p.gate = a.gate;
    p.pre_weight = a.pre_weight;
    p.r = a.r;
    p.z = a.z;
    p.post_rstd = a.post_rstd;
    p.pre_rstd = a.pre_rstd;
    p.tokens = (int64_t)a.tokens;
    p.per_gate = (unsigned)(a.gate ? a.tokens / a.gate_rows : a.tokens);
    p.r_stride = (int64_t)a.r_stride;
    p.z_stride = (int64_t)a.z_stride;
    p.dim = (int)a.dim;
    p.bf16_weights = a.weight_dtype == HC_BFLOAT16;
    p.residual_scale = a.residual_scale;
    p.eps = a.eps;
    return a.dtype == HC_BFLOAT16 ? run_norm<Bf16>(p, stream, sms) : run_norm<float>(p, stream, sms);
}

namespace {
// Rows of threads of a block with kGradFewCols columns a thread.
int64_t few_rows(int64_t dim) {
    const int64_t threads = (dim + kGradFewCols - 1) / kGradFewCols;
    if (dim <= kWarpDim) {
        int64_t lanes = 1;
        while (lanes < threads) lanes *= 2;
        return 256 / lanes;
    }
    return std::max<int64_t>(1, std::min<int64_t>(kMaxGroups, kNormThreads / ((threads + 31) / 32 * 32)));
}
}  // namespace

BlockNormPlan block_norm_plan(int64_t tokens, int64_t dim, int64_t gate_rows, bool gate, bool same_types) {
    BlockNormPlan q = {};
    int64_t gates = gate ? gate_rows : 1, per_gate = tokens / gates;
    q.pitch = (dim + 7) / 8 * 8;
    q.slots = 2;
    if (!tokens) {
        q.by_group = gates >= kGradBlocks;  // nothing to divide: unit, per_group and blocks are 0
    } else if (dim <= kGradFewCols * kNormThreads &&
               (gates == 1 ? (tokens + few_rows(dim) - 1) / few_rows(dim)
                           : (gates + few_rows(dim) - 1) / few_rows(dim) * per_gate) <= 3) {
        // up to three tokens a group of threads: one block, whose sums are final
        // (4 tokens of 1832 columns: 7.9 us instead of 8.4 with a second kernel)
        q.direct = q.blocks = 1;
        q.by_group = gates > 1;
        q.unit = gates > 1 ? gates : tokens;
        q.per_group = gates > 1 ? 0 : 1;
    } else if (gates < kGradBlocks || (per_gate == 1 && same_types && dim > kWarpDim)) {
        // gate rows of every token's own and of the values' type: as one more
        // operand (16384 x 1024 bf16: 59 us, 82 by gate rows; 4096 x 3001: 88,
        // 143; 509 x 1001 fp32: 10.2, 12.5; 509 x 4096 bf16: 17, 20)
        q.each = gates >= kGradBlocks;
        if (q.each) gates = 1, per_gate = tokens;
        const int64_t want = ((dim <= kGradCols * kNormThreads / 2 ? 2 : 1) * kGradBlocks + gates - 1) / gates;
        q.unit = std::max<int64_t>((per_gate + want - 1) / want, std::min<int64_t>(per_gate, 4));
        q.per_group = (per_gate + q.unit - 1) / q.unit;
        q.blocks = gates * q.per_group;
        q.slots = q.each ? 2 : 3;
    } else {
        q.by_group = 1;
        q.unit = (gates + kGradBlocks - 1) / kGradBlocks;
        q.blocks = (gates + q.unit - 1) / q.unit;
    }
    q.bytes = q.direct ? 0 : (size_t)q.blocks * q.slots * q.pitch * sizeof(float);
    return q;
}

BlockNormRows block_norm_rows(int64_t dim, int es, bool vectors, bool alike) {
    BlockNormRows r = {};
    r.access = vectors ? ROWS_VECTORS : alike ? ROWS_WINDOW : ROWS_ONE_BY_ONE;
    r.cols = kCols;
    r.ops = 2;
    r.lay = row_layout(dim, es, r.ops, r.access, kCols, kCols, kNormThreads / 2);
    return r;
}

BlockNormRows block_norm_grad_rows(BlockNormPlan* q, int64_t tokens, int64_t dim, int es, bool vectors, bool alike) {
    BlockNormRows r = {};
    // with 8 columns a thread a cluster has just enough for the longest rows, and
    // none for what a window begins before them (fp32 rows of 32766 columns):
    // those are taken element by element
    const int window_cols = !q->each && es == 2 ? kGradCols : kGradFewCols;
    const bool window = !vectors && alike && !q->by_group && q->per_group >= kClasses &&
                        dim + 16 / es - 1 <= (int64_t)kMaxCluster * kNormThreads * window_cols;
    if (window) {  // as many blocks for each class of tokens
        const int64_t gates = q->blocks / q->per_group, parts = q->per_group / kClasses, per_gate = tokens / gates;
        q->unit = ((per_gate + kClasses - 1) / kClasses + parts - 1) / parts;
        q->per_group = parts * kClasses;
        q->blocks = gates * q->per_group;
    }
    r.access = vectors ? ROWS_VECTORS : window ? ROWS_WINDOW : ROWS_ONE_BY_ONE;
    // fp32 windows are faster with 8 (8192 x 3001: 125 us against 182), bf16 ones
    // with 16 (16384 x 3001: 235 us against 281)
    // with each token's gate 8, which leave no spills (8192 x 4096 bf16: 117 us
    // against 222; 4096 x 3001: 88 against 93), but for bf16 rows that 8 would
    // split over a cluster of half-filled blocks and 16 leave room for two stages
    // (3600 x 4512: 113 us against 160)
    const bool one_block = q->each && r.access == ROWS_VECTORS && es == 2 && dim > kNormThreads * kGradFewCols &&
                           dim <= kEachThreads * kGradCols;
    r.cols = one_block || (!q->by_group && !q->each && (r.access == ROWS_VECTORS || (r.access == ROWS_WINDOW && es == 2)))
                 ? kGradCols : kGradFewCols;
    // more blocks than SMs are halved (16384 x 1024 bf16, each token's gate: 59 us
    // with 256 threads, 66 with 512; fewer keep a row a group: 509 x 1001 fp32)
    r.ops = q->each ? 5 : 4;
    r.lay = row_layout(dim, es, r.ops, r.access, kGradFewCols, r.cols,
                       r.cols == kGradCols || (q->each && q->blocks > kGradBlocks) ? kNormThreads / 2 : kNormThreads);
    if (!r.lay.stages) r.cols = kGradFewCols;
    return r;
}

cudaError_t launch_block_norm_grad(const hc_block_norm_grad_t& a, cudaStream_t stream) {
    const BlockNormPlan q = block_norm_plan((int64_t)a.tokens, (int64_t)a.dim, (int64_t)a.gate_rows, a.gate != nullptr,
                                            a.dtype == a.weight_dtype);
    NormGradParams p = {};
    p.in[0] = {a.grad_r, (int64_t)a.grad_r_stride};
    p.in[1] = {a.grad_z, (int64_t)a.grad_z_stride};
    p.in[2] = {a.y, (int64_t)a.y_stride};
    // without a next norm, x and its weight are no operands: what they hold (0 *
    // inf) is kept out of the gradients, and x is not read
    p.in[3] = {a.grad_z ? a.x : nullptr, (int64_t)a.x_stride};
    p.post_weight = a.post_weight;
    p.gate = a.gate;
    p.pre_weight = a.grad_z ? a.pre_weight : nullptr;
    p.post_rstd = a.post_rstd;
    p.pre_rstd = a.pre_rstd;
    p.grad_y = a.grad_y;
    p.grad_x = a.grad_x;
    p.grad_post_weight = a.grad_post_weight;
    p.grad_gate = a.grad_gate;
    p.grad_pre_weight = a.grad_pre_weight;
    p.part = (float*)a.scratch;
    p.tokens = (int64_t)a.tokens;
    if (q.each) p.in[4] = {a.gate, (int64_t)a.dim};
    p.gates = a.gate && !q.each ? (int64_t)a.gate_rows : 1;
    p.per_gate = (unsigned)(p.tokens / p.gates);
    p.grad_y_stride = (int64_t)a.grad_y_stride;
    p.grad_x_stride = (int64_t)a.grad_x_stride;
    p.pitch = q.pitch;
    p.slots = q.slots;
    p.direct = q.direct;
    p.dim = (int)a.dim;
    p.bf16_weights = a.weight_dtype == HC_BFLOAT16;
    p.residual_scale = a.residual_scale;
    return a.dtype == HC_BFLOAT16 ? run_norm_grad<Bf16>(p, q, stream) : run_norm_grad<float>(p, q, stream);
}

}  // namespace hc
