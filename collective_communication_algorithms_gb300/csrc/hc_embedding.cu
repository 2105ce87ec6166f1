// hc_embedding.cu -- the embedding lookup and its gradient.
//
// Lookup: out[t] = scale * table[ids[t] - first], a gather of rows; every
// byte of a token's row is read and written once, so the memory bounds it:
// 16384 tokens of 4096 fp32 columns to bf16 take 40 us, 6.2 TB/s (91 % of the
// copy bandwidth) of the distinct rows and the output; one token 2.1 us, the
// time of a launch.
//
// Gradient: grad_table[v] = scale * sum of grad_out[t] over the tokens of row
// v.  Adding rows with atomics would make the sums depend on the order in
// which blocks run, so the tokens are grouped by row first:
//  - up to kEmbeddingFewTokens tokens, every block finds the tokens of its
//    own row by comparing all ids (one launch, no scratch);
//  - above, a stable radix sort of (row, token), in the shared memory of one
//    cluster while it holds the tokens, else in passes over global memory;
//    then sums over groups of sorted tokens.  A row whose tokens all lie in
//    one group is written by it; a row cut by a group's end leaves partial
//    sums in scratch and its place on a list, and a last kernel adds up the
//    listed rows' partial sums in group order.
#include <algorithm>

#include "hc_ops.cuh"

namespace hc {
namespace {

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
struct LookupParams {
    const void* table;
    const void* ids;
    void* out;
    int64_t tokens, rows, first, table_stride, out_stride;
    int dim, col_blocks, tx_log2;
    bool wide_ids;
    float scale;
};

constexpr int kLookupThreads = 256;
// Tokens of a thread, whose rows are on their way together (65536 x 256 bf16:
// 8.5 us, 9.9 with one; no slower for a single token).
constexpr int kLookupTokens = 4;

// Columns of a thread: one vector of 8 (or of the wider type's 4), or 8 single
// ones, so that rows that are not aligned have as much on its way (19384 x 1694
// fp32 to bf16: 28 us, 51 with one column a thread).
constexpr int kLookupCols = 8;

// A block takes (2^tx_log2 x kLookupCols) columns, in vectors of N a thread, 2^tx_log2
// N apart, of (256 >> tx_log2) * kLookupTokens tokens.
template <class TI, class TO, int N>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(const LookupParams p) {
    constexpr int U = kLookupTokens, V = N == 1 ? kLookupCols : 1;
    const int tx = threadIdx.x & ((1 << p.tx_log2) - 1), ty = threadIdx.x >> p.tx_log2;
    const int ny = kLookupThreads >> p.tx_log2;
    const int64_t t0 = (int64_t)(blockIdx.x / p.col_blocks) * (ny * U) + ty;
    const int c = (((int)(blockIdx.x % p.col_blocks) * V << p.tx_log2) + tx) * N, step = N << p.tx_log2;
    grid_wait();
    grid_release();
    if (c >= p.dim) return;
    uint64_t row[U];
    float v[U][V][N];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int64_t t = t0 + u * ny;
        // rows of other tables wrap to large values
        row[u] = t < p.tokens ? (uint64_t)load_id(p.ids, t, p.wide_ids) - (uint64_t)p.first : ~0ull;
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        const TI* from = (const TI*)p.table + (int64_t)row[u] * p.table_stride + c;
#pragma unroll
        for (int k = 0; k < V; k++)
            load_whole<TI, N>(from + k * step, row[u] < (uint64_t)p.rows && c + k * step < p.dim, v[u][k]);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int64_t t = t0 + u * ny;
        if (t >= p.tokens) break;
        TO* to = (TO*)p.out + t * p.out_stride + c;
#pragma unroll
        for (int k = 0; k < V; k++) {
#pragma unroll
            for (int i = 0; i < N; i++) v[u][k][i] *= p.scale;
            store_whole<TO, N>(to + k * step, c + k * step < p.dim, v[u][k]);
        }
    }
}

template <class TI, class TO>
cudaError_t launch_lookup(LookupParams& p, bool vec, cudaStream_t stream) {
    constexpr int W = std::max(kVecOf<TI>, kVecOf<TO>);
    const int per_thread = vec ? W : kLookupCols;
    const int nv = (p.dim + per_thread - 1) / per_thread;
    p.tx_log2 = 5;
    while (p.tx_log2 < 8 && (1 << p.tx_log2) < nv) p.tx_log2++;
    p.col_blocks = (nv + (1 << p.tx_log2) - 1) >> p.tx_log2;
    const int64_t per = (int64_t)(kLookupThreads >> p.tx_log2) * kLookupTokens;
    const int64_t grid = (p.tokens + per - 1) / per * p.col_blocks;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const void* fn = vec ? (const void*)lookup_kernel<TI, TO, W> : (const void*)lookup_kernel<TI, TO, 1>;
    void* args[] = {&p};
    return launch_op(fn, dim3((unsigned)grid), dim3(kLookupThreads), args, 0, stream);
}

// ---------------------------------------------------------------------------
// gradient: shared pieces
// ---------------------------------------------------------------------------
struct GradParams {
    const void* grad;   // grad_out
    const void* ids;
    void* table;        // grad_table
    int64_t tokens, rows, first, padding, grad_stride, table_stride;
    int dim;
    bool wide_ids, accumulate, has_padding;
    float scale;
    // sorted path
    uint32_t *keys_in, *pos_in, *keys_out, *pos_out;
    uint32_t *hist, *hist_next, *hist_after;  // this pass's digit counts, the next's, the one after's
    float* part;
    unsigned char* touched;  // rows with tokens (NULL when adding to the table)
    uint32_t* cut;      // [0]: rows cut by a group's end, then the groups they begin in
    int64_t pitch, chunks, sum_chunks;
    int chunk, shift, bits, next_shift, passes, sum_chunk;
    int tiles;          // column tiles of a row
    int64_t sum_blocks;  // few tokens: the blocks after them write the rows without tokens
};

// Row of token t in this table, or rows when it has none (padding, another
// rank's id).
__device__ __forceinline__ uint32_t row_of(const GradParams& p, int64_t t) {
    const int64_t id = load_id(p.ids, t, p.wide_ids);
    const uint64_t r = (uint64_t)id - (uint64_t)p.first;  // ids below first wrap to large values
    return r < (uint64_t)p.rows && !(p.has_padding && id == p.padding) ? (uint32_t)r : (uint32_t)p.rows;
}

template <class TT, int N>
__device__ __forceinline__ void write_row(const GradParams& p, uint32_t row, int c, const float (&acc)[N]) {
    TT* q = (TT*)p.table + (int64_t)row * p.table_stride + c;
    const int n = p.dim - c;
    float v[N];
    if (p.accumulate) {
        load_n<TT, N>(q, n, v);
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = fmaf(acc[i], p.scale, v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = acc[i] * p.scale;
    }
    store_n<TT, N>(q, n, v);
}

template <class TT, int N>
__device__ __forceinline__ void zero_row(const GradParams& p, int64_t row, int tid, int threads) {
    const float z[N] = {};
    TT* q = (TT*)p.table + row * p.table_stride;
    for (int c = tid * N; c < p.dim; c += threads * N) store_n<TT, N>(q + c, p.dim - c, z);
}

constexpr int kFewThreads = 128;
constexpr int kFewWords = (int)kEmbeddingFewTokens / 32;
constexpr int kFillRows = 32;

// ---------------------------------------------------------------------------
// gradient of a few tokens: block (token, column tile); the block of a row's
// first token sums the row's tokens in token order, the others leave.  One
// launch and two waits for memory: 33 tokens of 1024 columns take 2.6 us.  A
// block compares all ids, and a row of many tokens is one block's chain, which
// is what ends it: 500 tokens of 1024 columns take 9.2 us here and 12.7 sorted
// (500 of one row: 32 and 15), 100 tokens 3.5 and 11.7.
// ---------------------------------------------------------------------------
template <class TO, class TT, int N>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const GradParams p) {
    __shared__ uint32_t same[kFewWords];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int T = (int)p.tokens;
    if ((int64_t)blockIdx.x >= p.sum_blocks) {  // rows without tokens
        const int64_t v0 = ((int64_t)blockIdx.x - p.sum_blocks) * kFillRows;
        __shared__ uint32_t touched;
        if (threadIdx.x == 0) touched = 0;
        __syncthreads();
        for (int s = threadIdx.x; s < T; s += kFewThreads) {
            const int64_t r = (int64_t)row_of(p, s) - v0;
            if (r >= 0 && r < kFillRows) atomicOr(&touched, 1u << r);
        }
        __syncthreads();
        for (int r = warp; r < kFillRows; r += kFewThreads / 32)
            if (v0 + r < p.rows && !(touched >> r & 1)) zero_row<TT, N>(p, v0 + r, lane, 32);
        return;
    }
    const int t = (int)(blockIdx.x / p.tiles);
    const int c = ((int)(blockIdx.x % p.tiles) * kFewThreads + threadIdx.x) * N;
    const uint32_t row = row_of(p, t);
    if (row == (uint32_t)p.rows) return;
    const int words = (T + 31) / 32;
    for (int w = warp; w < words; w += kFewThreads / 32) {
        const int s = w * 32 + lane;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, s < T && row_of(p, s) == row);
        if (lane == 0) same[w] = m;
    }
    __syncthreads();
    for (int w = 0; w < t / 32; w++)
        if (same[w]) return;  // an earlier token's block has the row
    if (same[t / 32] & ((1u << (t & 31)) - 1)) return;
    if (c >= p.dim) return;
    float acc[N] = {};
    for (int w = t / 32; w < words; w++) {
        uint32_t m = same[w];
        while (m) {
            constexpr int B = 8;  // rows in flight
            float v[B][N];
#pragma unroll
            for (int b = 0; b < B; b++) {
                const int s = m ? w * 32 + __ffs(m) - 1 : -1;
                m &= m - 1;  // 0 stays 0
                load_whole<TO, N>((const TO*)p.grad + (int64_t)s * p.grad_stride + c, s >= 0, v[b]);
            }
#pragma unroll
            for (int b = 0; b < B; b++)
#pragma unroll
                for (int i = 0; i < N; i++) acc[i] += v[b][i];
        }
    }
    write_row<TT, N>(p, row, c, acc);
}

// ---------------------------------------------------------------------------
// stable radix sort of (row, token) in the shared memory of one cluster: block
// r holds places [r * chunk, (r + 1) * chunk).  In every pass a warp takes a
// run of its block's tokens; a token's new place is (tokens of smaller
// digits) + (tokens of its digit in earlier blocks, in earlier warps, earlier
// in its warp).  The last pass writes to global memory.  Bound by the chain of
// steps (two passes of 9-bit digits, four cluster barriers): 16411 tokens take
// about 11 us; 30000 tokens of 1024 columns 48 us in all, 54 with the passes
// over global memory below, which from 32768 tokens use more SMs (60000: 84 us,
// 87 with one cluster).
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 512;  // digits of at most 9 bits
constexpr int64_t kClusterSortTokens = kMaxCluster * 4096;

struct ClusterSort {
    uint32_t warp_at[kSortWarps][kMaxBins];     // tokens of a warp, then the place of its next one
    uint32_t counts[kMaxCluster][kMaxBins];     // tokens of every block of the cluster
    uint32_t scan[kSortWarps];
};

__device__ __forceinline__ unsigned remote_addr(const void* local, unsigned rank) {
    unsigned a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    return a;
}

__global__ void __launch_bounds__(kSortThreads) cluster_sort_kernel(const GradParams p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    ClusterSort& sh = *(ClusterSort*)dyn;
    uint2* const buf = (uint2*)(dyn + sizeof(ClusterSort));  // two of chunk places
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = blockIdx.x, blocks = gridDim.x;
    const int bins = 1 << p.bits;
    const int64_t place0 = (int64_t)rank * p.chunk;
    const int have = (int)max((int64_t)0, min((int64_t)p.chunk, p.tokens - place0));
    const int per_warp = p.chunk / kSortWarps;  // a multiple of 32
    const int begin = warp * per_warp, end = min(begin + per_warp, have);
    grid_wait();
    grid_release();
    if (rank == 0 && tid == 0) p.cut[0] = 0;
    if (p.touched)
        for (int64_t v = rank * kSortThreads + tid; v < (p.rows + 15) / 16; v += (int64_t)blocks * kSortThreads)
            ((uint4*)p.touched)[v] = make_uint4(0, 0, 0, 0);
    if (blocks > 1) cluster_arrive();
    // the first pass reads the second buffer
#pragma unroll 8
    for (int i = tid; i < have; i += kSortThreads)
        buf[p.chunk + i] = make_uint2(row_of(p, place0 + i), (uint32_t)(place0 + i));
    if (blocks > 1) cluster_wait();  // every block runs, every flag is clear
    else __syncthreads();
    if (p.touched)
        for (int i = tid; i < have; i += kSortThreads) {
            const uint32_t row = buf[p.chunk + i].x;
            if (row < (uint32_t)p.rows) p.touched[row] = 1;
        }
    for (int pass = 0; pass < p.passes; pass++) {
        const int shift = pass * p.bits;
        const bool last = pass + 1 == p.passes;
        const uint2* from = buf + (size_t)((pass + 1) & 1) * p.chunk;
        const unsigned to = smem_addr(buf + (size_t)(pass & 1) * p.chunk);
        for (int w = 0; w < kSortWarps; w++)
            if (tid < bins) sh.warp_at[w][tid] = 0;
        __syncthreads();
        for (int i = begin + lane; i < end; i += 32) atomicAdd(&sh.warp_at[warp][(from[i].x >> shift) & (bins - 1)], 1u);
        __syncthreads();
        if (tid < bins) {
            uint32_t n = 0;
            for (int w = 0; w < kSortWarps; w++) n += sh.warp_at[w][tid];
            for (unsigned r = 0; r < blocks; r++)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote_addr(&sh.counts[rank][tid], r)), "r"(n) : "memory");
        }
        if (blocks > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        uint32_t before = 0, total = 0;
        if (tid < bins)
            for (unsigned r = 0; r < blocks; r++) {
                const uint32_t n = sh.counts[r][tid];
                if (r < rank) before += n;
                total += n;
            }
        uint32_t inc = total;  // inclusive sum over the digits
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) sh.scan[warp] = inc;
        __syncthreads();
        if (tid < bins) {
            uint32_t at = inc - total + before;
            for (int w = 0; w < warp; w++) at += sh.scan[w];
            for (int w = 0; w < kSortWarps; w++) {
                const uint32_t n = sh.warp_at[w][tid];
                sh.warp_at[w][tid] = at;
                at += n;
            }
        }
        __syncthreads();
        for (int b = begin; b < end; b += 32) {
            const bool in = b + lane < end;
            const uint2 e = in ? from[b + lane] : make_uint2(0u, 0u);
            const uint32_t d = in ? (e.x >> shift) & (bins - 1) : (uint32_t)bins;
            const uint32_t peers = __match_any_sync(0xFFFFFFFFu, d);
            const uint32_t lower = __popc(peers & ((1u << lane) - 1));
            const uint32_t at = in ? sh.warp_at[warp][d] : 0u;
            __syncwarp();
            if (in && lower == 0) sh.warp_at[warp][d] = at + __popc(peers);
            __syncwarp();
            if (!in) continue;
            const uint32_t place = at + lower;
            if (last) {
                p.keys_out[place] = e.x;
                p.pos_out[place] = e.y;
            } else {
                const unsigned r = place / (unsigned)p.chunk, o = place - r * (unsigned)p.chunk;
                unsigned a;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(to + o * 8), "r"(r));
                asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(e.x), "r"(e.y) : "memory");
            }
        }
        if (!last) {
            if (blocks > 1) {
                cluster_arrive();
                cluster_wait();
            } else {
                __syncthreads();
            }
        }
    }
}

// ---------------------------------------------------------------------------
// the same sort in passes over global memory: a block orders `chunk` tokens.
// Every block reads the digit counts of all chunks, which is quadratic in them:
// nothing up to a million tokens (128 chunks; 191 us of 8 columns), about a
// third of the time of 2^24 (2048 chunks; 4.8 ms).
// ---------------------------------------------------------------------------
// Digit counts of every chunk for the first pass; zeroes the next pass's.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const GradParams p) {
    __shared__ uint32_t count[kMaxBins];
    grid_wait();
    grid_release();
    const int bins = 1 << p.bits;
    if (blockIdx.x == 0 && threadIdx.x == 0) p.cut[0] = 0;
    if (p.touched)
        for (int64_t v = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; v < (p.rows + 15) / 16; v += (int64_t)gridDim.x * kSortThreads)
            ((uint4*)p.touched)[v] = make_uint4(0, 0, 0, 0);
    for (int b = threadIdx.x; b < bins; b += kSortThreads) count[b] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
    for (int i = threadIdx.x; i < p.chunk; i += kSortThreads)
        if (t0 + i < p.tokens) atomicAdd(&count[row_of(p, t0 + i) & (bins - 1)], 1u);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
        p.hist[(int64_t)blockIdx.x * bins + b] = count[b];
        p.hist_next[(int64_t)blockIdx.x * bins + b] = 0;
    }
}

// One pass: every token's place is (tokens of smaller digits) + (tokens of
// its digit in earlier chunks, in earlier warps, earlier in its warp).  Also
// counts the next pass's digits at their new places (integer adds, so their
// order does not matter), and zeroes the counts of the pass after that.
template <int ITEMS, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_pass_kernel(const GradParams p) {
    __shared__ uint32_t warp_count[kSortWarps][kMaxBins];
    __shared__ uint32_t base[kMaxBins];
    __shared__ uint32_t scan[kSortWarps];
    grid_wait();
    grid_release();
    const int bins = 1 << p.bits;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int w = 0; w < kSortWarps; w++)
        if (tid < bins) warp_count[w][tid] = 0;
    // digit tid: its tokens in earlier chunks, and in all
    uint32_t before = 0, total = 0;
    if (tid < bins) {
#pragma unroll 8
        for (int64_t c = 0; c < p.chunks; c++) {
            const uint32_t h = p.hist[c * bins + tid];
            if (c < (int64_t)blockIdx.x) before += h;
            total += h;
        }
        if (p.hist_after) p.hist_after[(int64_t)blockIdx.x * bins + tid] = 0;
    }
    // exclusive sum of the totals over the digits
    uint32_t inc = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    uint32_t off = 0;
    for (int w = 0; w < warp; w++) off += scan[w];
    if (tid < bins) base[tid] = off + inc - total + before;
    // rank of every token in its warp
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk + (int64_t)warp * 32 * ITEMS + lane;
    uint32_t key[ITEMS], pos[ITEMS], rank[ITEMS];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        const int64_t t = t0 + i * 32;
        const bool in = t < p.tokens;
        key[i] = in ? (FIRST ? row_of(p, t) : p.keys_in[t]) : 0u;
        pos[i] = in ? (FIRST ? (uint32_t)t : p.pos_in[t]) : 0u;
    }
    if (FIRST && p.touched)
#pragma unroll
        for (int i = 0; i < ITEMS; i++)
            if (t0 + i * 32 < p.tokens && key[i] < (uint32_t)p.rows) p.touched[key[i]] = 1;
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        const bool in = t0 + i * 32 < p.tokens;
        const uint32_t d = in ? (key[i] >> p.shift) & (bins - 1) : (uint32_t)bins;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, d);
        const uint32_t lower = __popc(peers & ((1u << lane) - 1));
        uint32_t seen = 0;
        if (in) seen = warp_count[warp][d];
        __syncwarp();
        if (in && lower == 0) warp_count[warp][d] = seen + __popc(peers);
        __syncwarp();
        rank[i] = seen + lower;
    }
    __syncthreads();
    if (tid < bins) {  // counts of the warps -> places of their first tokens
        uint32_t at = base[tid];
        for (int w = 0; w < kSortWarps; w++) {
            const uint32_t n = warp_count[w][tid];
            warp_count[w][tid] = at;
            at += n;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        if (t0 + i * 32 >= p.tokens) break;
        const uint32_t to = warp_count[warp][(key[i] >> p.shift) & (bins - 1)] + rank[i];
        p.keys_out[to] = key[i];
        p.pos_out[to] = pos[i];
        if (p.hist_next)
            atomicAdd(&p.hist_next[(int64_t)(to / (uint32_t)p.chunk) * bins + ((key[i] >> p.next_shift) & (bins - 1))], 1u);
    }
}

// ---------------------------------------------------------------------------
// sums over sorted tokens: a warp takes 256 columns of sum_chunk tokens, of
// which eight (or four, and the table's rows that they end, when adding to
// them) are on their way at a time, as they lie in memory.  Bound by the
// memory, with few tokens by the waits: 65536 tokens of 2048 bf16 columns to a
// dense fp32 table of 131072 rows take 253 us with the sort, 5.3 TB/s; adding
// to the 19845 rows with tokens 143 us.
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kLaneCols = 8;       // columns of a lane

// A lane's columns of a row of T: vectors of W neighbouring ones, 32 W apart
// (so that a warp's accesses are contiguous).
template <class T, int W>
struct Lane {
    static constexpr int kVecs = kLaneCols / W, kBytes = W * (int)sizeof(T);
    union {
        uint4 v16[kLaneCols * sizeof(T) / 16];
        uint2 v8[kLaneCols * sizeof(T) / 8];
        T e[kLaneCols];
    };
    // n: columns of the row from the lane's first, whole vectors of them (a
    // branch for parts of vectors kept the rows' loads from overlapping: 250 us
    // instead of 150 for 65536 tokens of 2048 columns)
    __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
        for (int v = 0; v < kVecs; v++) {
            const int o = v * 32 * W;
            if (o >= n) continue;
            if constexpr (kBytes == 16) v16[v] = *(const uint4*)(p + o);
            else if constexpr (kBytes == 8) v8[v] = *(const uint2*)(p + o);
            else e[v] = p[o];
        }
    }
    __device__ __forceinline__ float get(int i) const { return to_f32(e[i]); }
};
template <class T, int W>
__device__ __forceinline__ void store_lane(T* p, int n, const float (&x)[kLaneCols]) {
#pragma unroll
    for (int v = 0; v < kLaneCols / W; v++) {
        float e[W];
#pragma unroll
        for (int i = 0; i < W; i++) e[i] = x[v * W + i];
        store_whole<T, W>(p + v * 32 * W, v * 32 * W < n, e);
    }
}

template <class TO, class TT, int W, bool ACC>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const GradParams p) {
    constexpr int kRowsInFlight = ACC ? 4 : 8;
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t none = (uint32_t)p.rows;
    const int64_t item = (int64_t)blockIdx.x * kSumWarps + warp;
    constexpr int kZeroBytes = 4096;
    __shared__ __align__(16) unsigned char zeros[ACC || W == 1 ? 16 : kZeroBytes];
    struct Leave {  // the copies out of `zeros` read it before the block leaves
        __device__ __forceinline__ ~Leave() {
            if (!ACC && W > 1) bulk_wait_read_all();
        }
    } leave;
    if (!ACC && W > 1) {
        for (int i = threadIdx.x; i < kZeroBytes / 16; i += kSumThreads) ((uint4*)zeros)[i] = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
    }
    if (!ACC) {
        // every warp zeroes an equal share of the rows without tokens, by bulk
        // copies where rows are aligned, which queue apart from the loads
        // below
        const int64_t warps = (int64_t)gridDim.x * kSumWarps, share = (p.rows + warps - 1) / warps;
        const int64_t v1 = min((item + 1) * share, p.rows);
        for (int64_t v0 = item * share; v0 < v1; v0 += 32) {
            const int64_t v = v0 + lane;
            const bool empty = v < v1 && !p.touched[v];
            if (W > 1) {
                if (empty) {
                    const uintptr_t q = (uintptr_t)((TT*)p.table + v * p.table_stride);
                    const int bytes = p.dim * (int)sizeof(TT);
                    for (int o = 0; o < bytes; o += kZeroBytes) bulk_s2g(q + o, zeros, (unsigned)min(kZeroBytes, bytes - o));
                }
            } else {
                uint32_t todo = __ballot_sync(0xFFFFFFFFu, empty);
                while (todo) {
                    zero_row<TT, 1>(p, v0 + __ffs(todo) - 1, lane, 32);
                    todo &= todo - 1;
                }
            }
        }
        bulk_commit();
    }
    const int64_t chunk = item / p.tiles;
    if (chunk >= p.sum_chunks) return;
    const int tile = (int)(item % p.tiles);
    const int c = tile * 32 * kLaneCols + lane * W;
    const int n = p.dim - c;
    const int64_t s0 = chunk * p.sum_chunk, s1 = min(s0 + p.sum_chunk, p.tokens);
    // whether the row under way began before s0
    bool head = s0 > 0 && p.keys_in[s0 - 1] == p.keys_in[s0];
    float acc[kLaneCols] = {};
    for (int64_t b = s0; b < s1; b += 32) {
        const int64_t s = b + lane;
        const uint32_t key = s < s1 ? p.keys_in[s] : none;
        const uint32_t pos = s < s1 ? p.pos_in[s] : 0u;
        const uint32_t next = s + 1 < p.tokens ? p.keys_in[s + 1] : none;
        const int m = __popc(__ballot_sync(0xFFFFFFFFu, key != none));  // a prefix: tokens without a row come last
        // a row's last token, or the group's; of a row that goes on after it
        const uint32_t end_mask = __ballot_sync(0xFFFFFFFFu, lane < m && (next != key || s + 1 == s1));
        const uint32_t on_mask = __ballot_sync(0xFFFFFFFFu, lane < m && next == key && s + 1 == s1);
        // written to the table, not to a partial sum
        const uint32_t whole_mask = end_mask & ~on_mask & ~(head ? end_mask & (0u - end_mask) : 0u);
        for (int j = 0; j < m; j += kRowsInFlight) {
            Lane<TO, W> v[kRowsInFlight];
            Lane<TT, W> old[kRowsInFlight];
#pragma unroll
            for (int k = 0; k < kRowsInFlight; k++) {
                const uint32_t t = __shfl_sync(0xFFFFFFFFu, pos, j + k), r = __shfl_sync(0xFFFFFFFFu, key, j + k);
                if (j + k < m) v[k].load((const TO*)p.grad + (int64_t)t * p.grad_stride + c, n);
                if (ACC && (whole_mask >> (j + k) & 1)) old[k].load((const TT*)p.table + (int64_t)r * p.table_stride + c, n);
            }
#pragma unroll
            for (int k = 0; k < kRowsInFlight; k++) {
                const uint32_t bit = 1u << (j + k);
                const uint32_t r = __shfl_sync(0xFFFFFFFFu, key, j + k);
                if (j + k < m)
#pragma unroll
                    for (int i = 0; i < kLaneCols; i++) acc[i] += v[k].get(i);
                if (!(end_mask & bit)) continue;
                if (whole_mask & bit) {
                    if (ACC) {
#pragma unroll
                        for (int i = 0; i < kLaneCols; i++) acc[i] = fmaf(acc[i], p.scale, old[k].get(i));
                    } else {
#pragma unroll
                        for (int i = 0; i < kLaneCols; i++) acc[i] *= p.scale;
                    }
                    store_lane<TT, W>((TT*)p.table + (int64_t)r * p.table_stride + c, n, acc);
                } else {
                    const bool tail = (on_mask & bit) && !head;
                    store_lane<float, W>(p.part + (chunk * 2 + (tail ? 1 : 0)) * p.pitch + c, n, acc);
                    if (tail && tile == 0 && lane == 0) p.cut[1 + atomicAdd(p.cut, 1u)] = (uint32_t)chunk;
                }
                head = false;
#pragma unroll
                for (int i = 0; i < kLaneCols; i++) acc[i] = 0.0f;
            }
        }
        if (m < 32) break;
    }
}

// The rows on the list: slot 1 of the group where a row begins and slot 0 of
// the groups after it.  An item is a tile of 32 N columns of a row; eight
// items of the same tile and different rows are a block's at a time.  A warp
// adds up its item's short list by itself; long lists are taken in turn by all
// warps, which add equal parts of it, joined in order.
constexpr int kJoinWarps = 8;
constexpr int kShortList = 8;  // 16000 x 1024: 31 us, 37 with all lists taken by all warps
template <class TT, int N>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const GradParams p) {
    __shared__ float sums[kJoinWarps][32 * N];
    __shared__ int64_t chunks[kJoinWarps], counts[kJoinWarps];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t rows = p.cut[0], per_tile = (rows + kJoinWarps - 1) / kJoinWarps, items = per_tile * p.tiles;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int c = ((int)(item / per_tile) * 32 + lane) * N;
        // neighbours on the list, which tend to be alike, go to different blocks
        const int64_t at = item % per_tile + warp * per_tile;
        auto add = [&](int64_t chunk, int64_t a, int64_t b, float (&acc)[N]) {
#pragma unroll 4
            for (int64_t k = a; k < b; k++) {
                float v[N];
                load_n<float, N>(p.part + ((chunk + k) * 2 + (k == 0 ? 1 : 0)) * p.pitch + c, p.dim - c, v);
#pragma unroll
                for (int i = 0; i < N; i++) acc[i] += v[i];
            }
        };
        int64_t count = 0;
        if (at < rows) {
            const int64_t chunk = p.cut[1 + at];
            const uint32_t key = p.keys_in[(chunk + 1) * p.sum_chunk];
            // the last group whose first token is of this row: doubling, then halving
            int64_t lo = chunk + 1, hi = chunk + 2, step = 1;
            while (hi < p.sum_chunks && p.keys_in[hi * p.sum_chunk] == key) {
                lo = hi;
                step *= 2;
                hi += step;
            }
            hi = min(hi, p.sum_chunks);
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (p.keys_in[mid * p.sum_chunk] == key) lo = mid;
                else hi = mid;
            }
            count = lo - chunk + 1;
            if (count <= kShortList) {
                float acc[N] = {};
                add(chunk, 0, count, acc);
                write_row<TT, N>(p, key, c, acc);
                count = 0;
            }
            if (lane == 0) chunks[warp] = chunk;
        }
        if (lane == 0) counts[warp] = count;
        __syncthreads();
        for (int i = 0; i < kJoinWarps; i++) {
            if (!counts[i]) continue;  // the same for every thread
            const int64_t per = (counts[i] + kJoinWarps - 1) / kJoinWarps;
            float acc[N] = {};
            add(chunks[i], warp * per, min((warp + 1) * per, counts[i]), acc);
#pragma unroll
            for (int j = 0; j < N; j++) sums[warp][j * 32 + lane] = acc[j];
            __syncthreads();
            if (warp == i) {
                // this warp's item: its own part again, in the list's order
#pragma unroll
                for (int j = 0; j < N; j++) acc[j] = sums[0][j * 32 + lane];
                for (int w = 1; w < kJoinWarps && w * per < counts[i]; w++)
#pragma unroll
                    for (int j = 0; j < N; j++) acc[j] += sums[w][j * 32 + lane];
                write_row<TT, N>(p, p.keys_in[(chunks[i] + 1) * p.sum_chunk], c, acc);
            }
            __syncthreads();
        }
        __syncthreads();  // counts and chunks have been read
    }
}

template <class TO, class TT>
cudaError_t launch_grad(GradParams& p, const EmbeddingScratch& sc, unsigned char* scratch, bool vec,
                        cudaStream_t stream, int sms) {
    constexpr int W = std::min(kVecOf<TO>, kVecOf<TT>);
    const int64_t nv = (p.dim + (vec ? W : 1) - 1) / (vec ? W : 1);
    void* args[] = {&p};
    auto grid_ok = [](int64_t g) { return g <= INT32_MAX; };
    if (p.tokens <= (int64_t)kEmbeddingFewTokens) {
        p.tiles = (int)((nv + kFewThreads - 1) / kFewThreads);
        p.sum_blocks = p.tokens * p.tiles;
        const int64_t grid = p.sum_blocks + (p.accumulate ? 0 : (p.rows + kFillRows - 1) / kFillRows);
        if (grid == 0) return cudaSuccess;
        if (!grid_ok(grid)) return cudaErrorInvalidValue;
        const void* fn = vec ? (const void*)few_kernel<TO, TT, W> : (const void*)few_kernel<TO, TT, 1>;
        return launch_op(fn, dim3((unsigned)grid), dim3(kFewThreads), args, 0, stream);
    }
    uint32_t *keys[2], *pos[2];
    for (int i = 0; i < 2; i++) {
        keys[i] = (uint32_t*)(scratch + sc.keys[i]);
        pos[i] = (uint32_t*)(scratch + sc.pos[i]);
    }
    p.part = (float*)(scratch + sc.part);
    p.cut = (uint32_t*)(scratch + sc.cut);
    p.touched = p.accumulate ? nullptr : scratch + sc.touched;
    p.pitch = sc.pitch;
    p.chunk = sc.chunk;
    p.chunks = sc.chunks;
    p.bits = sc.bits;
    p.passes = sc.passes;
    p.sum_chunk = sc.sum_chunk;
    p.sum_chunks = sc.sum_chunks;
    cudaError_t e;
    if (sc.cluster) {
        p.keys_out = keys[0];
        p.pos_out = pos[0];
        const int smem = (int)sizeof(ClusterSort) + sc.chunk * 16;
        if (!allow_smem((void*)cluster_sort_kernel, smem)) return cudaErrorInvalidValue;
        e = launch_op((const void*)cluster_sort_kernel, dim3((unsigned)sc.cluster), dim3(kSortThreads), args, (size_t)smem, stream, sc.cluster);
        if (e != cudaSuccess) return e;
        p.keys_in = keys[0];
        p.pos_in = pos[0];
    } else {
        uint32_t* const hist = (uint32_t*)(scratch + sc.hist);
        const size_t hist_len = (size_t)sc.chunks << sc.bits;
        p.hist = hist;
        p.hist_next = hist + hist_len;
        e = launch_op((const void*)sort_count_kernel, dim3((unsigned)p.chunks), dim3(kSortThreads), args, 0, stream);
        if (e != cudaSuccess) return e;
        for (int i = 0; i < sc.passes; i++) {
            p.shift = i * sc.bits;
            p.next_shift = p.shift + sc.bits;
            p.keys_in = keys[(i + 1) & 1];
            p.pos_in = pos[(i + 1) & 1];
            p.keys_out = keys[i & 1];
            p.pos_out = pos[i & 1];
            p.hist = hist + (size_t)(i % 3) * hist_len;
            p.hist_next = i + 1 < sc.passes ? hist + (size_t)((i + 1) % 3) * hist_len : nullptr;
            p.hist_after = i + 2 < sc.passes ? hist + (size_t)((i + 2) % 3) * hist_len : nullptr;
            const bool small = sc.chunk <= kSortThreads * 4;
            const void* fn = i == 0 ? (small ? (const void*)sort_pass_kernel<4, true> : (const void*)sort_pass_kernel<16, true>)
                                    : (small ? (const void*)sort_pass_kernel<4, false> : (const void*)sort_pass_kernel<16, false>);
            e = launch_op(fn, dim3((unsigned)p.chunks), dim3(kSortThreads), args, 0, stream);
            if (e != cudaSuccess) return e;
        }
        p.keys_in = keys[(sc.passes - 1) & 1];
        p.pos_in = pos[(sc.passes - 1) & 1];
    }
    p.tiles = (p.dim + 32 * kLaneCols - 1) / (32 * kLaneCols);
    p.sum_blocks = (p.sum_chunks * p.tiles + kSumWarps - 1) / kSumWarps;
    // enough warps for the rows without tokens, too
    const int64_t sum_grid = std::max<int64_t>(p.sum_blocks, p.accumulate ? 1 : std::min<int64_t>((p.rows + kSumWarps - 1) / kSumWarps, 4 * sms));
    if (!grid_ok(sum_grid)) return cudaErrorInvalidValue;
    const void* fn = p.accumulate ? (vec ? (const void*)sum_kernel<TO, TT, W, true> : (const void*)sum_kernel<TO, TT, 1, true>)
                                  : (vec ? (const void*)sum_kernel<TO, TT, W, false> : (const void*)sum_kernel<TO, TT, 1, false>);
    e = launch_op(fn, dim3((unsigned)sum_grid), dim3(kSumThreads), args, 0, stream);
    if (e != cudaSuccess || p.sum_chunks < 2) return e;
    // partial rows are 16-byte aligned, the table's may not be
    constexpr int J = 4;
    const int64_t jv = (p.dim + (vec ? J : 1) - 1) / (vec ? J : 1);
    p.tiles = (int)((jv + 31) / 32);
    const int64_t grid = std::min<int64_t>((p.sum_chunks + kJoinWarps - 2) / kJoinWarps * p.tiles, (int64_t)sms * 8);
    return launch_op(vec ? (const void*)join_kernel<TT, J> : (const void*)join_kernel<TT, 1>, dim3((unsigned)grid),
                     dim3(kJoinWarps * 32), args, 0, stream);
}

// Rows that take accesses of W elements: on 16-byte boundaries, whole vectors.
bool aligned16(const void* p, int64_t stride, int dim, int es) {
    return ((uintptr_t)p & 15) == 0 && (stride * es & 15) == 0 && dim % 8 == 0;
}

}  // namespace

cudaError_t launch_embedding(const hc_embedding_t& a, cudaStream_t stream) {
    LookupParams p = {};
    p.table = a.table;
    p.ids = a.ids;
    p.out = a.out;
    p.tokens = (int64_t)a.tokens;
    p.rows = (int64_t)a.rows;
    p.first = a.first_id;
    p.table_stride = (int64_t)a.table_stride;
    p.out_stride = (int64_t)a.out_stride;
    p.dim = (int)a.dim;
    p.wide_ids = a.id_type == HC_ID64;
    p.scale = a.scale;
    const bool vec = aligned16(a.table, p.table_stride, p.dim, elem_bytes(a.table_dtype)) &&
                     aligned16(a.out, p.out_stride, p.dim, elem_bytes(a.out_dtype));
    const bool bi = a.table_dtype == HC_BFLOAT16, bo = a.out_dtype == HC_BFLOAT16;
    if (bi) return bo ? launch_lookup<Bf16, Bf16>(p, vec, stream) : launch_lookup<Bf16, float>(p, vec, stream);
    return bo ? launch_lookup<float, Bf16>(p, vec, stream) : launch_lookup<float, float>(p, vec, stream);
}

EmbeddingScratch embedding_scratch(int64_t tokens, int64_t rows, int64_t dim) {
    EmbeddingScratch s = {};
    if (tokens <= (int64_t)kEmbeddingFewTokens) return s;
    // tokens without a row sort as `rows`, so the largest key is rows
    int bits = 1;
    while (bits < 32 && (rows >> bits)) bits++;
    s.passes = (bits + 8) / 9;
    s.bits = (bits + s.passes - 1) / s.passes;
    if (tokens <= kClusterSortTokens) {
        // at least 2048 tokens a block
        s.cluster = 1;
        while (s.cluster < kMaxCluster && tokens > 2048 * s.cluster) s.cluster *= 2;
        const int64_t per = (tokens + s.cluster - 1) / s.cluster;
        s.chunk = (int)((per + kSortThreads - 1) / kSortThreads * kSortThreads);
    } else {
        s.chunk = kSortThreads * (tokens <= (1 << 18) ? 4 : 16);
    }
    s.chunks = (tokens + s.chunk - 1) / s.chunk;
    // groups of 8 to 128 tokens, at least a round of the warps that the SMs hold (24 each)
    s.sum_chunk = 128;
    const int64_t tiles = (dim + 32 * kLaneCols - 1) / (32 * kLaneCols);
    while (s.sum_chunk > 8 && tokens * tiles < 24 * 152 * s.sum_chunk) s.sum_chunk /= 2;
    s.sum_chunks = (tokens + s.sum_chunk - 1) / s.sum_chunk;
    s.pitch = (dim + 7) / 8 * 8;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    for (int i = 0; i < (s.cluster ? 1 : 2); i++) {
        s.keys[i] = take((size_t)tokens * 4);
        s.pos[i] = take((size_t)tokens * 4);
    }
    if (!s.cluster) s.hist = take((size_t)3 * s.chunks << (s.bits + 2));
    s.cut = take(((size_t)s.sum_chunks + 1) * 4);
    s.touched = take((size_t)rows);
    s.part = take((size_t)s.sum_chunks * 2 * (size_t)s.pitch * 4);
    s.bytes = at;
    return s;
}

cudaError_t launch_embedding_grad(const hc_embedding_grad_t& a, cudaStream_t stream, int sms) {
    GradParams p = {};
    p.grad = a.grad_out;
    p.ids = a.ids;
    p.table = a.grad_table;
    p.tokens = (int64_t)a.tokens;
    p.rows = (int64_t)a.rows;
    p.first = a.first_id;
    p.padding = a.padding_id;
    p.has_padding = a.padding_id >= 0;
    p.grad_stride = (int64_t)a.grad_out_stride;
    p.table_stride = (int64_t)a.grad_table_stride;
    p.dim = (int)a.dim;
    p.wide_ids = a.id_type == HC_ID64;
    p.accumulate = a.accumulate != 0;
    p.scale = a.scale;
    const EmbeddingScratch sc = embedding_scratch(p.tokens, p.rows, p.dim);
    const bool vec = aligned16(a.grad_out, p.grad_stride, p.dim, elem_bytes(a.grad_out_dtype)) &&
                     aligned16(a.grad_table, p.table_stride, p.dim, elem_bytes(a.grad_table_dtype));
    unsigned char* s = (unsigned char*)a.scratch;
    const bool bo = a.grad_out_dtype == HC_BFLOAT16, bt = a.grad_table_dtype == HC_BFLOAT16;
    if (bo) return bt ? launch_grad<Bf16, Bf16>(p, sc, s, vec, stream, sms) : launch_grad<Bf16, float>(p, sc, s, vec, stream, sms);
    return bt ? launch_grad<float, Bf16>(p, sc, s, vec, stream, sms) : launch_grad<float, float>(p, sc, s, vec, stream, sms);
}

}  // namespace hc
