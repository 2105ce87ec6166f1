// hc_expert_matmul.cu -- the products of an expert layer: each expert's rows
// with its weight (hc_expert_matmul), and their gradients.
//
// Three products over the groups of rows that `offsets` (on the device) names:
//   forward      out[r]     = sum_i W[e][o][i] x[r][i]
//   rows'        grad_x[r]  = sum_o W[e][o][i] grad_out[r][o]
//   weights'     grad_W[e]  = sum over e's rows of grad_out[r][o] x[r][i]
// The first two are one kernel: a tile of one group's rows times a tile of
// the weight's columns, summed along the rows' own direction.  In the third
// the rows are what is summed along, and every expert has all of its tiles.
#include <algorithm>

#include "hc_tensor.cuh"

namespace hc {
namespace {

// ---------------------------------------------------------------------------
// groups: bound[e] .. bound[e + 1] are the rows of expert e, tile[e] the tiles
// of rows before it
// ---------------------------------------------------------------------------
// By one warp: offsets clamped to [0, rows] and made non-decreasing, and the
// sums of ceil(rows of a group / tile_rows).
__device__ __forceinline__ void read_groups(const int32_t* offsets, int E, int64_t rows, int tile_rows, int* bound,
                                            int* tile) {
    const int lane = threadIdx.x & 31;
    const int most = (int)rows;
    int carry = 0, tiles = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int lo = e <= E ? min(max(offsets[e], 0), most) : 0;
        int hi = e < E ? min(max(offsets[e + 1], 0), most) : 0;
        hi = max(hi, lo);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, hi, o);
            if (lane >= o) hi = max(hi, u);
        }
        hi = max(hi, carry);
        int before = __shfl_up_sync(0xFFFFFFFFu, hi, 1);
        if (lane == 0) before = e0 ? carry : lo;
        lo = max(lo, before);
        if (lane > 0) lo = before;
        const int n = e < E ? (int)(((int64_t)hi - lo + tile_rows - 1) / tile_rows) : 0;
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += u;
        }
        if (e < E) {
            if (e == 0) {
                bound[0] = lo;
                tile[0] = 0;
            }
            bound[e + 1] = hi;
            tile[e + 1] = tiles + s;
        }
        carry = __shfl_sync(0xFFFFFFFFu, hi, 31);
        tiles += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
}

// The group that a tile of rows belongs to.
__device__ __forceinline__ int group_of(const int* tile, int E, int m) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (m < tile[mid + 1]) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// ---------------------------------------------------------------------------
// binary32 multiplications on the ordinary cores
// ---------------------------------------------------------------------------
struct PlainParams {
    const void* a;  // forward: x; rows': grad_out; weights': the operand along the gradient's rows
    const void* b;  // the weight; weights': the operand along the gradient's columns
    void* out;
    const int32_t* offsets;
    int64_t rows, a_stride, b_stride, b_expert, out_stride, out_expert;
    int E, M, N, K;           // M: weights' gradient's rows; K: of the first two products
    int a_vec, b_vec;         // whole 16 bytes
    int accumulate;
    int splits;               // blocks of a tile
};

constexpr int kPThreads = 256, kPEach = 8, kPPad = 4;

// One operand's T x PK elements of a step, kPEach of them a thread's: in pieces
// of four where rows lie on whole 16 bytes, else one by one, neighbours in a
// row going to neighbouring threads.  ALONG: k runs along the operand's rows.
template <bool ALONG, int T, int PK>
__device__ __forceinline__ void load_step(const float* p, int64_t stride, int k0, int K, int len, bool vec, float (&v)[kPEach]) {
    const int tid = threadIdx.x;
    if (vec) {
        constexpr int PER = (ALONG ? PK : T) / kPEach;  // threads of a row
        const int row = tid / PER + (ALONG ? 0 : k0), col = tid % PER * kPEach + (ALONG ? k0 : 0);
        const int n = row < (ALONG ? len : K) ? (ALONG ? K : len) - col : 0;
        const float* at = p + row * stride + col;
        if (n >= kPEach) {
#pragma unroll
            for (int i = 0; i < kPEach; i += 4) {
                const float4 w = *(const float4*)(at + i);
                v[i] = w.x; v[i + 1] = w.y; v[i + 2] = w.z; v[i + 3] = w.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPEach; i++) v[i] = i < n ? at[i] : 0.0f;
        }
    } else {
        constexpr int PER = ALONG ? PK : T / kPEach;
#pragma unroll
        for (int i = 0; i < kPEach; i++) {
            const int row = ALONG ? tid / PER + kPThreads / PER * i : k0 + tid / PER;
            const int col = ALONG ? k0 + tid % PER : tid % PER + PER * i;
            v[i] = row < (ALONG ? len : K) && col < (ALONG ? K : len) ? p[row * stride + col] : 0.0f;
        }
    }
}
// Keeps them as [k][row or column of the sums].
template <bool ALONG, int T, int PK>
__device__ __forceinline__ void keep_step(float (&to)[PK][T + kPPad], bool vec, const float (&v)[kPEach]) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int i = 0; i < kPEach; i++) {
        if (vec) {
            constexpr int PER = (ALONG ? PK : T) / kPEach;
            to[ALONG ? tid % PER * kPEach + i : tid / PER][ALONG ? tid / PER : tid % PER * kPEach + i] = v[i];
        } else {
            constexpr int PER = ALONG ? PK : T / kPEach;
            to[ALONG ? tid % PER : tid / PER][ALONG ? tid / PER + kPThreads / PER * i : tid % PER + PER * i] = v[i];
        }
    }
}

__device__ __forceinline__ float load_remote(const float* local, unsigned rank) {
    float v;
    asm volatile("{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %1, %2;\n ld.shared::cluster.f32 %0, [r];\n}\n"
                 : "=f"(v)
                 : "r"(smem_addr(local)), "r"(rank)
                 : "memory");
    return v;
}

// ROWS: the first two products, whose sums run along a's rows; b is summed
// along its rows (BK) or across them.
// T x T sums a block, L x L a thread, in pieces of four.  SPLIT: the blocks of a
// cluster share a tile, each with a run of the sum's steps; every block then
// adds up its part of the tile's rows over the blocks, in their order.
template <class TO, bool ROWS, bool BK, int T, bool SPLIT>
__global__ void __launch_bounds__(kPThreads) plain_product_kernel(const PlainParams p) {
    constexpr int L = T / 16, PK = kPThreads * kPEach / T;  // steps of 16 or 32 of the sum
    __shared__ __align__(16) float as[2][PK][T + kPPad], bs[2][PK][T + kPPad];
    __shared__ int bound[kMaxExperts + 1], tile[kMaxExperts + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    grid_wait();
    // no early release: the next kernel's blocks would pile up on the SMs with
    // room, and stay there (two products in turn: 108 us, against 57 apart)
    if (tid < 32) read_groups(p.offsets, p.E, p.rows, T, bound, tile);
    __syncthreads();
    const int nt = (p.N + T - 1) / T;
    const int64_t mt = ROWS ? tile[p.E] : (int64_t)((p.M + T - 1) / T) * p.E;
    const int splits = SPLIT ? p.splits : 1, rank = SPLIT ? (int)blockIdx.x % splits : 0;
    for (int64_t i = blockIdx.x / splits; i < mt * nt; i += gridDim.x / splits) {
        const int m = (int)(i / nt), n0 = (int)(i % nt) * T;
        int e, m0, mlen, K;
        int64_t first;  // ROWS: the tile's first row; else the group's
        if (ROWS) {
            e = group_of(tile, p.E, m);
            first = bound[e] + (int64_t)(m - tile[e]) * T;
            m0 = 0;
            mlen = (int)min((int64_t)T, bound[e + 1] - first);
            K = p.K;
        } else {
            const int per = (p.M + T - 1) / T;
            e = m / per;
            m0 = (m % per) * T;
            mlen = min(T, p.M - m0);
            first = bound[e];
            K = bound[e + 1] - bound[e];
            if (!K && p.accumulate) continue;
        }
        const int nlen = min(T, p.N - n0);
        const float* a = (const float*)p.a + first * p.a_stride + m0;
        const float* b = (const float*)p.b + (ROWS ? e * p.b_expert + (BK ? (int64_t)n0 * p.b_stride : n0)
                                                   : first * p.b_stride + n0);
        const int run = ((K + PK - 1) / PK + splits - 1) / splits * PK, begin = rank * run;
        K = min(K, begin + run);  // this block's steps end there
        float av[kPEach], bv[kPEach];
        Pair acc[L][L / 2];  // two columns each
#pragma unroll
        for (int x = 0; x < L; x++)
#pragma unroll
            for (int y = 0; y < L / 2; y++) acc[x][y] = Pair(0.0f, 0.0f);
        auto fetch = [&](int k0) {
            load_step<ROWS, T, PK>(a, p.a_stride, k0, K, mlen, p.a_vec, av);
            load_step<BK, T, PK>(b, p.b_stride, k0, K, nlen, p.b_vec, bv);
        };
        auto keep = [&](int h) {
            keep_step<ROWS, T, PK>(as[h], p.a_vec, av);
            keep_step<BK, T, PK>(bs[h], p.b_vec, bv);
        };
        __syncthreads();  // the tile before has been read
        if (begin < K) {
            fetch(begin);
            keep(0);
        }
        __syncthreads();
        int h = 0;
        for (int k0 = begin; k0 < K; k0 += PK, h ^= 1) {
            if (k0 + PK < K) fetch(k0 + PK);
#pragma unroll
            for (int k = 0; k < PK; k++) {
                float x[L];
                Pair y[L / 2];
#pragma unroll
                for (int g = 0; g < L / 4; g++) {
                    const float4 u = *(const float4*)&as[h][k][g * 64 + ty * 4];
                    const ulonglong2 w = *(const ulonglong2*)&bs[h][k][g * 64 + tx * 4];
                    x[4 * g] = u.x; x[4 * g + 1] = u.y; x[4 * g + 2] = u.z; x[4 * g + 3] = u.w;
                    y[2 * g].v = w.x; y[2 * g + 1].v = w.y;
                }
#pragma unroll
                for (int q = 0; q < L; q++) {
                    const Pair xx(x[q], x[q]);
#pragma unroll
                    for (int r = 0; r < L / 2; r++) acc[q][r] = fma_pair(xx, y[r], acc[q][r]);
                }
            }
            if (k0 + PK < K) keep(h ^ 1);
            __syncthreads();
        }
        TO* out = (TO*)p.out + (ROWS ? first * p.out_stride : e * p.out_expert + (int64_t)m0 * p.out_stride) + n0;
        if constexpr (SPLIT) {
            static_assert(T * (T + kPPad) <= 2 * PK * (T + kPPad), "the sums take the place of one operand");
            float(*part)[T + kPPad] = (float(*)[T + kPPad]) & as[0][0][0];
#pragma unroll
            for (int q = 0; q < L; q++)
#pragma unroll
                for (int r = 0; r < L / 2; r++) {
                    float2 v;
                    acc[q][r].get(v.x, v.y);
                    *(float2*)&part[(q / 4) * 64 + ty * 4 + q % 4][(r / 2) * 64 + tx * 4 + r % 2 * 2] = v;
                }
            cluster_arrive();
            cluster_wait();
            for (int j = tid; j < T / splits * T; j += kPThreads) {
                const int row = j / T * splits + rank, col = j % T;
                if (row >= mlen || col >= nlen) continue;
                float sum = 0.0f;
                for (int q = 0; q < splits; q++) sum += load_remote(&part[row][col], q);
                TO* at = out + row * p.out_stride + col;
                put(at, (!ROWS && p.accumulate ? to_f32(*at) : 0.0f) + sum);
            }
            cluster_arrive();  // all have read before the next tile, or the end
            cluster_wait();
        } else {
#pragma unroll
            for (int q = 0; q < L; q++) {
                const int row = (q / 4) * 64 + ty * 4 + q % 4;
                if (row >= mlen) continue;
                float sums[L];
#pragma unroll
                for (int r = 0; r < L / 2; r++) acc[q][r].get(sums[2 * r], sums[2 * r + 1]);
#pragma unroll
                for (int r = 0; r < L; r++) {
                    const int col = (r / 4) * 64 + tx * 4 + r % 4;
                    if (col >= nlen) continue;
                    TO* at = out + row * p.out_stride + col;
                    put(at, (!ROWS && p.accumulate ? to_f32(*at) : 0.0f) + sums[r]);
                }
            }
        }
    }
}

// The 16 bytes that begin s (even) bytes behind the first of two vectors.
__device__ __forceinline__ uint4 bytes_from(const uint4& u, const uint4& v, int s) {
    uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    if (s & 8)
#pragma unroll
        for (int i = 0; i < 6; i++) w[i] = w[i + 2];
    if (s & 4)
#pragma unroll
        for (int i = 0; i < 5; i++) w[i] = w[i + 1];
    const int bits = (s & 2) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}

// Elements 8 c .. 8 c + 7 of a row of `cols` that begins anywhere, from the
// aligned vectors that hold them (none without a byte of the row); zeros behind
// the row's end.
__device__ __forceinline__ uint4 row_vector(const Bf16* row, int c, int cols) {
    const uintptr_t from = (uintptr_t)row, end = from + 2 * (uintptr_t)cols, at = (from & ~(uintptr_t)15) + 16 * (uintptr_t)c;
    const int s = (int)(from & 15);
    uint4 u = make_uint4(0, 0, 0, 0), v = u;
    if (at < end) u = *(const uint4*)at;
    if (s && at + 16 < end) v = *(const uint4*)(at + 16);
    uint4 w = bytes_from(u, v, s);
    const int left = cols - 8 * c;
    if (left < 8) {
        uint32_t* x = &w.x;
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (2 * i + 2 > left) x[i] = 2 * i + 1 > left ? 0u : x[i] & 0xFFFFu;
    }
    return w;
}
// ---------------------------------------------------------------------------
// bf16 products of few rows (of all groups together), the weight summed along
// its rows
//
// Bound by the bytes of the weights that have rows: a warp takes a row of the
// weight, in aligned vectors of 16 bytes wherever it begins, and multiplies it
// by up to four of the group's rows, which lie in shared memory.  One token
// through two experts of 4096 x 1024: 16.8 MB.
// ---------------------------------------------------------------------------
constexpr int64_t kFewRows = 16, kFewDim = 8192;
constexpr int kFewThreads = 256, kFewAtOnce = 4, kFewBatch = 4;
constexpr int kFewEach = 4, kFewBlock = kFewThreads / 32 * kFewEach;  // weight rows of a warp, of a block

struct FewParams {
    const Bf16* x;
    const Bf16* w;
    void* out;
    const int32_t* offsets;
    int64_t rows, x_stride, w_stride, w_expert, out_stride;
    int E, N, K;
};

template <class TO>
__global__ void __launch_bounds__(kFewThreads) few_rows_kernel(const FewParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int bound[kMaxExperts + 1], before[kMaxExperts + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_wait();
    grid_release();
    if (warp == 0) read_groups(p.offsets, p.E, p.rows, 1 << 30, bound, before);  // before: groups with rows
    __syncthreads();
    if ((int)blockIdx.y >= before[p.E]) return;
    const int e = group_of(before, p.E, blockIdx.y), o0 = blockIdx.x * kFewBlock + warp * kFewEach;
    const int each = max(0, min(kFewEach, p.N - o0));  // weight rows of this warp
    const int vectors = (p.K + 7) / 8, batches = (vectors + 32 * kFewBatch - 1) / (32 * kFewBatch);
    const Bf16* w0 = p.w + e * p.w_expert + o0 * p.w_stride;
    Bf16* xs = (Bf16*)smem;  // kFewAtOnce rows of whole vectors
    for (int r0 = bound[e]; r0 < bound[e + 1]; r0 += kFewAtOnce) {
        const int n = min(kFewAtOnce, bound[e + 1] - r0);
        // batch i of the warp's rows: the vectors that hold it, one batch ahead
        uint4 u[2][kFewBatch], v[2][kFewBatch];
        const auto load = [&](int i, uint4 (&a)[kFewBatch], uint4 (&b)[kFewBatch]) {
            const uintptr_t from = (uintptr_t)(w0 + (i / batches) * p.w_stride), end = from + 2 * (uintptr_t)p.K;
            const uintptr_t at = (from & ~(uintptr_t)15) + 16 * (uintptr_t)(i % batches * 32 * kFewBatch + lane);
#pragma unroll
            for (int k = 0; k < kFewBatch; k++) {
                a[k] = b[k] = make_uint4(0, 0, 0, 0);
                if (i < each * batches && at + 512 * k < end) a[k] = *(const uint4*)(at + 512 * k);
                if ((from & 15) && i < each * batches && at + 512 * k + 16 < end) b[k] = *(const uint4*)(at + 512 * k + 16);
            }
        };
        load(0, u[0], v[0]);
        __syncthreads();  // the rows before have been read
        for (int j = threadIdx.x; j < n * vectors; j += kFewThreads) {
            const int r = j / vectors, c = j - r * vectors;
            ((uint4*)xs)[j] = row_vector(p.x + (int64_t)(r0 + r) * p.x_stride, c, p.K);
        }
        __syncthreads();
        float acc[kFewAtOnce] = {};
        for (int i0 = 0; i0 < each * batches; i0 += 2)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int i = i0 + h;
                if (i >= each * batches) break;
                load(i + 1, u[h ^ 1], v[h ^ 1]);
                const int f = i / batches, c0 = (i - f * batches) * 32 * kFewBatch + lane;
                const int shift = (int)((uintptr_t)(w0 + f * p.w_stride) & 15);
#pragma unroll
                for (int k = 0; k < kFewBatch; k++) {
                    const int c = c0 + 32 * k;
                    if (c >= vectors) continue;
                    float w[8];
                    unpack(bytes_from(u[h][k], v[h][k], shift), w);
                    if (c * 8 + 8 > p.K)  // behind the row lies another's, of any value
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            if (c * 8 + j >= p.K) w[j] = 0.0f;
#pragma unroll
                    for (int r = 0; r < kFewAtOnce; r++) {
                        if (r >= n) break;
                        float y[8];
                        unpack(((const uint4*)xs)[r * vectors + c], y);
#pragma unroll
                        for (int j = 0; j < 8; j++) acc[r] = fmaf(w[j], y[j], acc[r]);
                    }
                }
                if (i + 1 == (f + 1) * batches) {  // the row's last
#pragma unroll
                    for (int r = 0; r < kFewAtOnce; r++) {
                        const float sum = warp_sum(acc[r]);
                        if (lane == 0 && r < n) put((TO*)p.out + (int64_t)(r0 + r) * p.out_stride + o0 + f, sum);
                        acc[r] = 0.0f;
                    }
                }
            }
    }
}

// ---------------------------------------------------------------------------
// bf16 products on the tensor cores
//
// G = 2: the two blocks of a cluster, on two neighbouring SMs, take tiles of
// 256 x 256 sums in turn; each brings in half of both operands, so that a byte
// of shared memory serves twice the products.  G = 1: single blocks and tiles
// of 128 x 128, for products with few tiles or few rows a group.
//
// In a block one thread starts tiled copies of 64 steps of the sum into a ring
// of stages, one (of the first block) issues the products of each stage, and
// four warps bring finished sums from tensor memory through shared memory to
// the output while the next tile's products run (two sets of sums).
//
// The first two products have the weight's columns as m and a group's rows as
// n, whose number in an instruction is any multiple of 32: the last tile of a
// group multiplies at most 31 rows of the next one, which it does not store
// (sums of different rows have nothing to do with each other).  In the
// weights' gradient the rows are what is summed along, so those behind the
// group's last are overwritten with zeros in shared memory, by a warp of their
// own, before the products may start.
// ---------------------------------------------------------------------------
constexpr int kTM = 128, kTK = 64, kTStages = 6;  // kTM: of one block, of both operands
constexpr int kTOperandBytes = kTM * kTK * 2, kTStageBytes = 2 * kTOperandBytes;
constexpr int kTStagingBytes = 4 * 32 * 128;
// The tensor cores bring the 16 products of a step and the sum so far to the
// largest one's exponent and cut off what lies two bits or more below binary32's
// last place, so that a sum of n terms of one sign ends short by at most n
// 1.25 2^-26 of itself (n 2^-26 for the terms, each cut off below 2^-25 of a sum
// that is half of its end on average, n / 16 2^-24 for the sums).  Measured, bf16
// values of [0.5, 1): 3.2e-5 after 8192, 3.8e-4 after 65536 terms.
// LONG: sums are taken out every kTSegment steps and added up, rounded, in
// registers, so that no length costs more than a segment does: 9.5e-6 of it for
// binary32 results, 1.5e-4 for bf16 ones, whose own rounding is up to 2e-3.
// binary32 results are always made so (476 us instead of 412 for weight gradients
// of 32768 rows of 16, 2048 x 4096; 369 to 408 instead of 348 for the forward
// product of as many, 4096 -> 2048), bf16 ones from sums of more than kTPlain terms (353 us
// either way for those weight gradients, but with plain sums four warps are
// enough).
template <class TO>
constexpr int kTSegment = sizeof(TO) == 4 ? 512 : 8192;
constexpr int64_t kTPlain = 16384;
template <bool LONG>
constexpr int kTThreadsOf = LONG ? 384 : 256;

struct TensorParams {
    CUtensorMap a, b;
    void* out;
    const int32_t* offsets;
    int64_t rows, out_stride, out_expert;
    int E, M, N, K;           // M: weights' gradient's rows; K: of the first two products
    int accumulate, out_vec;  // out: whole 16 bytes
    int* err;
    unsigned long long wait_ns;
    int hold;                 // wait-expiry test mode
};

struct TensorBarriers {
    uint64_t full[kTStages], empty[kTStages], raw[kTStages];  // raw: landed, to be overwritten in part
    uint64_t zeroed[kTStages];  // by the other block, which may be stages ahead
    uint64_t sums_full[2], sums_empty[2], drain;
    uint32_t tmem;
    volatile uint32_t copied;  // stages whose copies this block has begun
};
constexpr int kTSmem = 1024 + kTStages * kTStageBytes + kTStagingBytes + (int)sizeof(TensorBarriers) + 8;

// A place in the ring of stages: the stage, and the parity of its turn.
struct Ring {
    int s = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next() {
        if (++s == kTStages) {
            s = 0;
            turn ^= 1;
        }
    }
    __device__ __forceinline__ void skip(int n) {  // n stages on
        s += n % kTStages;
        turn ^= n / kTStages & 1;
        if (s >= kTStages) {
            s -= kTStages;
            turn ^= 1;
        }
    }
};

// One tile: sums m0 .. m0 + mlen, n0 .. n0 + nlen of expert e, over K steps.
// The first two products: m counts the weight's columns, n rows from `first`
// on; the weights' gradient: m and n count its rows and columns, the steps are
// the rows from `first` on.
struct TensorTile {
    int e, m0, mlen, n0, nlen, K;
    int64_t first;
    __device__ __forceinline__ int n() const { return (nlen + 31) / 32 * 32; }  // of an instruction
};
// Tile i of T x T sums, of `across` in a row.
template <bool ROWS, int T>
__device__ __forceinline__ TensorTile tensor_tile(const TensorParams& p, const int* bound, const int* tile, int64_t i, int across) {
    TensorTile t;
    const int down = (int)(i / across), at = (int)(i - (int64_t)down * across) * T;
    if (ROWS) {
        t.m0 = at;
        t.mlen = min(T, p.N - at);
        t.e = group_of(tile, p.E, down);
        t.first = bound[t.e] + (int64_t)(down - tile[t.e]) * T;
        t.n0 = 0;
        t.nlen = (int)min((int64_t)T, bound[t.e + 1] - t.first);
        t.K = p.K;
    } else {
        t.n0 = at;
        t.nlen = min(T, p.N - at);
        const int per = (p.M + T - 1) / T;
        t.e = down / per;
        t.m0 = (down - t.e * per) * T;
        t.mlen = min(T, p.M - t.m0);
        t.first = bound[t.e];
        t.K = bound[t.e + 1] - bound[t.e];
    }
    return t;
}

// The way out of long sums, by eight warps: each has a half of the columns of 32
// rows of sums in registers and adds the segments up as they come.  In the
// forward product a column of sums is a row of the output, which the 32 lanes
// store as it is; the weights' gradient goes through shared memory, 16 columns at
// a time.
// What a binary32 output holds is added by L2 (a rounded addition to each
// element, one in a call, so the order is fixed all the same): 478 us where waiting for old
// values took 675, and bringing them into L2 beforehand 590 (32768 rows of 16,
// 2048 x 4096; 462 without adding).
template <bool ROWS, int G, int T, class TO, class Wait>
__device__ __forceinline__ void long_sums_to_output(const TensorParams& p, const int* bound, const int* tile, unsigned char* staging,
                                                    uint64_t* sums_full, uint64_t* sums_empty, uint32_t tmem, int64_t tiles, int across,
                                                    int rank, Wait warp_wait) {
    constexpr int W = T / 2;  // columns of a warp
    const int warp = (threadIdx.x >> 5) - 4, lane = threadIdx.x & 31, q = warp & 3, c0 = (warp >> 2) * W;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + c0;
    unsigned char* mine = staging + warp * 2048;
    const int r0 = lane / 4, at = lane % 4 * 4, m = rank * kTM + q * 32;
    uint32_t n = 0;
    for (int64_t i = blockIdx.x / G; i < tiles; i += gridDim.x / G) {
        const TensorTile t = tensor_tile<ROWS, T>(p, bound, tile, i, across);
        if (!t.K && p.accumulate) continue;
        const int cols = t.nlen - c0, rows = t.mlen - m;  // of this warp
        float sum[W];
#pragma unroll
        for (int j = 0; j < W; j++) sum[j] = 0.0f;
        bool ok = true;
        for (int k = 0; k < t.K; k += kTSegment<TO>, n++) {
            const uint32_t set = n & 1;
            if (!(ok = warp_wait([&] { return mbar_wait_quick(&sums_full[set], (n >> 1) & 1, p.wait_ns); }))) break;
            tensor_fence_after();
#pragma unroll
            for (int c = 0; c < W; c += 16)
                if (c < cols) {
                    uint32_t v[16];
                    tmem_load16(lanes + set * T + c, v);
#pragma unroll
                    for (int j = 0; j < 16; j++) sum[c + j] += __uint_as_float(v[j]);
                }
            tensor_fence_before();
            __syncwarp();
            if (lane == 0) first_arrive<G>(&sums_empty[set]);
        }
        if (!ok) break;
        if constexpr (ROWS) {
            TO* to = (TO*)p.out + (t.first + c0) * p.out_stride + t.m0 + m + lane;
#pragma unroll
            for (int c = 0; c < W; c += 16) {
                if (c >= cols) break;
#pragma unroll
                for (int j = 0; j < 16; j++)
                    if (c + j < cols && lane < rows) put(to + (c + j) * p.out_stride, sum[c + j]);
            }
            continue;
        }
        TO* out = (TO*)p.out + t.e * p.out_expert + (int64_t)(t.m0 + m + r0) * p.out_stride + t.n0 + c0 + at;
        const bool fast = p.out_vec && t.nlen % 4 == 0, add = p.accumulate;
#pragma unroll
        for (int c = 0; c < W; c += 16) {
            if (c >= cols) break;
            __syncwarp();  // the step before has been read
#pragma unroll
            for (int j = 0; j < 4; j++)
                *(float4*)(mine + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                    make_float4(sum[c + 4 * j], sum[c + 4 * j + 1], sum[c + 4 * j + 2], sum[c + 4 * j + 3]);
            __syncwarp();
            if (fast) {
                uint2 old[4];  // bf16: what is added to
                if constexpr (sizeof(TO) == 2)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (add && j * 8 + r0 < rows && c + at < cols) old[j] = *(const uint2*)(out + (int64_t)(j * 8) * p.out_stride + c);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int r = j * 8 + r0;
                    float4 x = *(const float4*)(mine + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
                    TO* to = out + (int64_t)(j * 8) * p.out_stride + c;
                    if (r >= rows || c + at >= cols) continue;
                    if constexpr (sizeof(TO) == 2) {
                        if (add) {
                            x.x += bf_lo(old[j].x);
                            x.y += bf_hi(old[j].x);
                            x.z += bf_lo(old[j].y);
                            x.w += bf_hi(old[j].y);
                        }
                        *(uint2*)to = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
                    } else if (add)
                        asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
                                     : "memory");
                    else
                        *(float4*)to = x;
                }
            } else {  // element by element: a lane has a column of every other row
                TO* to = out - (int64_t)r0 * p.out_stride - at + (lane >> 4) * p.out_stride + (lane & 15) + c;
                if (c + (lane & 15) < cols)
#pragma unroll
                    for (int r = 0; r < 16; r++) {
                        const int row = 2 * r + (lane >> 4);
                        const float x = *(const float*)(mine + row * 64 + ((((lane >> 2) & 3) ^ ((row >> 1) & 3)) << 4) + (lane & 3) * 4);
                        if (row >= rows) continue;
                        TO* one = to + 2 * r * p.out_stride;
                        if constexpr (sizeof(TO) == 2) put(one, add ? to_f32(*one) + x : x);
                        else if (add) asm volatile("red.global.add.f32 [%0], %1;" ::"l"(one), "f"(x) : "memory");
                        else *one = x;
                    }
                __syncwarp();
            }
        }
    }
}

// ROWS: the first two products; WK: their weight is summed along its rows.
template <bool ROWS, bool WK, int G, class TO, bool LONG>
__global__ void __launch_bounds__(kTThreadsOf<LONG>, 1) tensor_product_kernel(const __grid_constant__ TensorParams p) {
    constexpr int T = kTM * G;
    constexpr int SEGMENT = LONG ? kTSegment<TO> : 1 << 30;  // steps of a sum taken out at once
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int bound[kMaxExperts + 1], tile[kMaxExperts + 1];
    unsigned char* stages = smem + (1024 - (smem_addr(smem) & 1023)) % 1024;
    unsigned char* staging = stages + kTStages * kTStageBytes;
    TensorBarriers& bar = *(TensorBarriers*)(staging + kTStagingBytes);
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int rank = G == 1 ? 0 : (int)(blockIdx.x % G);  // in the cluster
    if (tid == 0) {
        for (int s = 0; s < kTStages; s++) {
            mbar_init(&bar.full[s], 1 + p.hold);
            mbar_init(&bar.empty[s], 1);
            mbar_init(&bar.raw[s], 1);
            mbar_init(&bar.zeroed[s], 1);
        }
        for (int s = 0; s < 2; s++) {
            mbar_init(&bar.sums_full[s], 1);
            mbar_init(&bar.sums_empty[s], (LONG ? 8 : 4) * G);
        }
        mbar_init(&bar.drain, 1);
        bar.copied = 0;
        mbar_init_fence();
        prefetch_map(&p.a);
        prefetch_map(&p.b);
    }
    if (warp == 2) tmem_alloc<G>(&bar.tmem, 2 * T);
    grid_wait();
    // no early release: the next kernel's blocks would take up registers beside
    // this one's and wait there
    if (warp == 3) read_groups(p.offsets, p.E, p.rows, T, bound, tile);
    tensor_fence_before();
    __syncthreads();
    if constexpr (G > 1) {  // the other block's barriers are set up
        cluster_arrive();
        cluster_wait();
    }
    tensor_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar.tmem, 0);
    const int across = (p.N + T - 1) / T;
    const int64_t tiles = (ROWS ? (int64_t)tile[p.E] : (int64_t)((p.M + T - 1) / T) * p.E) * across;
    const int64_t step = gridDim.x / G;
    const auto expired = [&] { atomicExch(p.err, (int)HC_ERR_TIMEOUT); };
    // A whole warp's wait: one lane polls, and the warp is together again
    // afterwards, as elections and loads from tensor memory need it, with one
    // answer for all.  What is waited for may lie any number of stages ahead (a
    // tile's sums, the next group with a remainder), so the wait only gives up
    // when the block's copies have stood still for as long; they stop by
    // themselves once the ring is full.
    const auto warp_wait = [&](auto wait) {
        bool ok = true;
        if (lane == 0) {
            ok = wait();
            for (bool on = true; !ok && on;) {
                const uint32_t before = bar.copied;
                ok = wait();
                on = bar.copied != before;
            }
            if (!ok) expired();
        }
        ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
        __syncwarp();  // what the lane has seen, all have
        return ok;
    };

    if (warp == 0 && lane == 0) {  // copies
        Ring at;
        int issued = 0;           // stages that hold copies, at most all
        uint32_t copied = 0;
        uint32_t turns = 0;       // the parity of each stage's last turn
        uint32_t raw_used = 0;    // stages whose last copies went to raw
        uint32_t raw_phase = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x / G; ok && i < tiles; i += step) {
            const TensorTile t = tensor_tile<ROWS, T>(p, bound, tile, i, across);
            const int am = t.m0 + rank * kTM, half = t.n() / G, bn = (ROWS ? (int)t.first : t.n0) + rank * half;
            const int boxes = (half + 63) / 64;  // of 64 n
            const unsigned bytes = kTOperandBytes + boxes * 8192;
            for (int k0 = 0; k0 < t.K; k0 += kTK, at.next()) {
                const int s = at.s;
                if (!mbar_wait_quick(&bar.empty[s], at.turn ^ 1, p.wait_ns)) {
                    expired();
                    ok = false;
                    break;
                }
                issued = max(issued, s + 1);
                turns = (turns & ~(1u << s)) | at.turn << s;
                unsigned char* a = stages + s * kTStageBytes;
                unsigned char* b = a + kTOperandBytes;
                const bool part = !ROWS && t.K - k0 < kTK;
                uint32_t to;
                if (part) {
                    raw_used |= 1u << s;
                    raw_phase ^= 1u << s;
                    to = smem_addr(&bar.raw[s]);
                    mbar_arrive_expect_tx(&bar.raw[s], bytes);
                } else {
                    raw_used &= ~(1u << s);
                    // both blocks' copies land on the first one's barrier (the
                    // other's may do so before the bytes are announced)
                    to = first_blocks<G>(&bar.full[s]);
                    if (rank == 0) mbar_arrive_expect_tx(&bar.full[s], G * bytes);
                }
                if (ROWS && WK) {
                    tile_g2s<G>(a, &p.a, k0, am, t.e, to);
                } else {
#pragma unroll
                    for (int j = 0; j < kTM / 64; j++) {
                        if (ROWS) tile_g2s<G>(a + j * 8192, &p.a, am + 64 * j, k0, t.e, to);
                        else tile_g2s<G>(a + j * 8192, &p.a, am + 64 * j, (int)t.first + k0, to);
                    }
                }
                for (int j = 0; j < boxes; j++) {
                    if (ROWS) tile_g2s<G>(b + j * 8192, &p.b, k0, bn + 64 * j, to);
                    else tile_g2s<G>(b + j * 8192, &p.b, bn + 64 * j, (int)t.first + k0, to);
                }
                bar.copied = ++copied;
            }
        }
        // A block does not leave while copies into its shared memory are under
        // way, nor before the last arrivals on its barriers: those of finished
        // products come by themselves, from the first block to both, and one that
        // came late would find the next block's barriers in this one's place.
        for (int s = 0; ok && s < issued; s++)
            if (!(ok = mbar_wait_quick(&bar.empty[s], turns >> s & 1, p.wait_ns))) expired();
        if (!ok) {  // the first block waits for the copies of both
            for (int s = 0; s < issued; s++) {
                if (raw_used >> s & 1) {
                    mbar_wait_quick(&bar.raw[s], (raw_phase >> s & 1) ^ 1, kWaitLimitNs);
                } else if (rank == 0) {
                    if (p.hold) mbar_arrive(&bar.full[s]);
                    mbar_wait_quick(&bar.full[s], turns >> s & 1, kWaitLimitNs);
                }
            }
            if (G > 1)  // and either for some time beyond any copy's or arrival's
                for (const unsigned long long t0 = global_ns(); global_ns() - t0 < kTestWaitLimitNs;) {}
        }
    } else if (warp == 1 && rank == 0) {  // products
        // 16 steps of the sum further on, in units of a descriptor's address
        constexpr bool AK = ROWS && WK, BK = ROWS;  // summed along rows in shared memory
        constexpr uint32_t a_on = (AK ? 32 : 2048) >> 4, b_on = (BK ? 32 : 2048) >> 4;
        const uint32_t base = smem_addr(stages);
        const uint64_t a0 = AK ? operand_along(base) : operand_across(base, 8192);
        const uint64_t b0 = BK ? operand_along(base + kTOperandBytes) : operand_across(base + kTOperandBytes, 8192);
        Ring at;
        uint32_t n = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x / G; ok && i < tiles; i += step) {
            const TensorTile t = tensor_tile<ROWS, T>(p, bound, tile, i, across);
            if (!t.K) continue;
            const uint32_t shape = product_shape(!AK, !BK, T, t.n());
            for (int k0 = 0; k0 < t.K; k0 += kTK, at.next()) {
                const uint32_t set = n & 1, sums = tmem + set * T;
                const int k = k0 % SEGMENT;
                if (!k) {
                    if (!(ok = warp_wait([&] { return first_wait<G>(&bar.sums_empty[set], ((n >> 1) & 1) ^ 1, p.wait_ns); }))) break;
                    tensor_fence_after();
                }
                const int s = at.s;
                if (!(ok = warp_wait([&] { return mbar_wait_quick(&bar.full[s], at.turn, p.wait_ns); }))) break;
                tensor_fence_after();
                const uint64_t a = a0 + (uint32_t)(s * (kTStageBytes >> 4)), b = b0 + (uint32_t)(s * (kTStageBytes >> 4));
                const bool last = k + kTK == SEGMENT || k0 + kTK >= t.K;
                if (elected()) {
                    if (t.K - k0 >= kTK) {
#pragma unroll
                        for (int j = 0; j < kTK / 16; j++) product16<G>(sums, a + j * a_on, b + j * b_on, shape, k > 0 || j > 0);
                    } else {
                        for (int j = 0; j < (t.K - k0 + 15) / 16; j++)
                            product16<G>(sums, a + j * a_on, b + j * b_on, shape, k > 0 || j > 0);
                    }
                    products_arrive<G>(&bar.empty[s]);
                    if (last) products_arrive<G>(&bar.sums_full[set]);
                }
                __syncwarp();
                n += last;
            }
        }
        if (elected()) products_arrive<G>(&bar.drain, false);  // tensor memory is freed after the last products
        __syncwarp();
        if (lane == 0) mbar_wait_quick(&bar.drain, 0, kWaitLimitNs);
    } else if (!ROWS && warp == 3) {  // zeros behind the last row of a group
        Ring at;
        uint32_t phase = 0;  // of each stage's turns with such rows
        for (int64_t i = blockIdx.x / G; i < tiles; i += step) {
            const TensorTile t = tensor_tile<ROWS, T>(p, bound, tile, i, across);
            const int rest = t.K % kTK;
            at.skip(t.K / kTK);
            if (!rest) continue;
            const int s = at.s;
            at.next();
            const uint32_t turn = phase >> s & 1;
            phase ^= 1u << s;
            if (!warp_wait([&] { return mbar_wait_quick(&bar.raw[s], turn, p.wait_ns); })) break;
            const int zeros = (16 - rest % 16) % 16 * 8;  // rows that a product reads, 16 bytes each
            for (int j = lane; j < zeros * (kTStageBytes / 8192); j += 32)  // in all boxes
                *(uint4*)(stages + s * kTStageBytes + j / zeros * 8192 + rest * 128 + j % zeros * 16) = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (rank > 0) {
                if (lane == 0) first_arrive<G>(&bar.zeroed[s]);
            } else {
                if (G > 1 && !warp_wait([&] { return first_wait<G>(&bar.zeroed[s], turn, p.wait_ns); })) break;
                if (lane == 0) mbar_arrive(&bar.full[s]);
            }
        }
    } else if constexpr (LONG) {
        if (warp >= 4)
            long_sums_to_output<ROWS, G, T, TO>(p, bound, tile, staging, bar.sums_full, bar.sums_empty, tmem, tiles, across, rank, warp_wait);
    } else if (warp >= 4) {  // sums to the output
        constexpr int V = 16 / (int)sizeof(TO), PER = 32 / V, N = 32 / V;  // elements of a lane, lanes and steps of 32 columns
        const int q = warp - 4;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        unsigned char* mine = staging + q * 32 * 128;  // 32 rows of 32 sums, whose 16-byte pieces are swapped about
        const int r0 = lane / PER, at = lane % PER * V;  // of the lane, when it stores
        uint32_t n = 0;
        for (int64_t i = blockIdx.x / G; i < tiles; i += step) {
            const TensorTile t = tensor_tile<ROWS, T>(p, bound, tile, i, across);
            if (!t.K && p.accumulate) continue;
            const uint32_t set = n & 1;
            const int m = rank * kTM + q * 32;  // of this warp's 32 lanes of sums
            // the tile's place in the output, and the lane's in the warp's part
            TO* out = ROWS ? (TO*)p.out + (t.first + r0) * p.out_stride + t.m0 + m + at
                           : (TO*)p.out + t.e * p.out_expert + (int64_t)(t.m0 + m + r0) * p.out_stride + t.n0 + at;
            // c: columns of sums; the step's rows of output left for the lane
            const auto rows_left = [&](int c, int j) { return (ROWS ? t.nlen - c : t.mlen - m) - j * V - r0; };
            const auto place = [&](int c, int j) { return out + (ROWS ? (int64_t)(c + j * V) * p.out_stride : (int64_t)(j * V) * p.out_stride + c); };
            const bool add = !ROWS && p.accumulate;
            const auto cols_left = [&](int c) { return ROWS ? t.mlen - m : t.nlen - c; };
            // 16-byte accesses, of which a lane makes all or none at its columns:
            // branches about parts of them would keep loads from overlapping
            const bool fast = p.out_vec && (ROWS ? t.mlen : t.nlen) % V == 0;
            constexpr int AHEAD = ROWS ? 1 : 4;  // steps of 32 columns that what is added to is loaded ahead
            uint4 old[AHEAD][N];
            const auto fetch = [&](int c, uint4 (&v)[N]) {
#pragma unroll
                for (int j = 0; j < N; j++)
                    if (rows_left(c, j) > 0 && at < cols_left(c)) v[j] = *(const uint4*)place(c, j);
            };
            if (add && fast)
#pragma unroll
                for (int h = 0; h < AHEAD; h++)
                    if (h * 32 < t.nlen) fetch(h * 32, old[h]);
            if (t.K) {
                if (!warp_wait([&] { return mbar_wait_quick(&bar.sums_full[set], (n >> 1) & 1, p.wait_ns); })) break;
                tensor_fence_after();
                n++;
            }
            for (int c0 = 0; c0 < t.nlen; c0 += 32 * AHEAD)
#pragma unroll
                for (int h = 0; h < AHEAD; h++) {
                    const int c = c0 + 32 * h;
                    if (c >= t.nlen) break;
                    uint32_t v[32];
                    if (t.K) {
                        __syncwarp();
                        tmem_load32(lanes + set * T + c, v);
                        if (c + 32 >= t.nlen) {
                            tensor_fence_before();
                            __syncwarp();
                            if (lane == 0) first_arrive<G>(&bar.sums_empty[set]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j++) v[j] = 0;
                    }
                    __syncwarp();  // the sums of the step before have been read
                    if constexpr (ROWS) {  // a column of sums is a row of the output
#pragma unroll
                        for (int j = 0; j < 32; j++)
                            *(uint32_t*)(mine + j * 128 + (((lane >> 2) ^ (j & 7)) << 4) + (lane & 3) * 4) = v[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            *(uint4*)(mine + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                    __syncwarp();
                    if (!fast) {  // element by element: a lane has a column
                        const int rows = min(32, ROWS ? t.nlen - c : t.mlen - m);
                        TO* to = place(c, 0) - r0 * p.out_stride - at + lane;
                        if (lane < cols_left(c))
#pragma unroll
                            for (int r0 = 0; r0 < 32; r0 += 16) {
                                float y[16];
#pragma unroll
                                for (int r = 0; r < 16; r++) y[r] = add && r0 + r < rows ? to_f32(to[(r0 + r) * p.out_stride]) : 0.0f;
#pragma unroll
                                for (int r = 0; r < 16; r++) {
                                    const float x = *(const float*)(mine + (r0 + r) * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                                    if (r0 + r < rows) put(to + (r0 + r) * p.out_stride, x + y[r]);
                                }
                            }
                        __syncwarp();
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < N; j++) {
                        const int r = j * V + r0;
                        float x[V];
#pragma unroll
                        for (int g = 0; g < V / 4; g++) {
                            const uint4 w = *(const uint4*)(mine + r * 128 + (((at / 4 + g) ^ (r & 7)) << 4));
                            x[4 * g] = __uint_as_float(w.x);
                            x[4 * g + 1] = __uint_as_float(w.y);
                            x[4 * g + 2] = __uint_as_float(w.z);
                            x[4 * g + 3] = __uint_as_float(w.w);
                        }
                        if (add) {
                            float y[V];
                            unpack(old[h][j], y);
#pragma unroll
                            for (int g = 0; g < V; g++) x[g] += y[g];
                        }
                        if (rows_left(c, j) > 0 && at < cols_left(c)) *(uint4*)place(c, j) = pack(x);
                    }
                    if (add && fast && c + 32 * AHEAD < t.nlen) fetch(c + 32 * AHEAD, old[h]);
                }
        }
    }
    __syncwarp();
    tensor_fence_before();
    __syncthreads();
    if constexpr (G > 1) {  // neither block's shared or tensor memory goes while the other uses it
        cluster_arrive();
        cluster_wait();
    }
    tensor_fence_after();
    if (warp == 2) tmem_free<G>(tmem, 2 * T);
}

bool whole(const void* p, size_t stride, size_t expert, int es) {
    return (uintptr_t)p % 16 == 0 && stride * es % 16 == 0 && expert * es % 16 == 0;
}

template <class TO, bool ROWS, bool BK>
cudaError_t launch_plain(PlainParams p, cudaStream_t stream, int sms) {
    const auto tiles = [&](int64_t T) {
        return (ROWS ? p.rows / T + std::min<int64_t>(p.E, p.rows) + 1 : (p.M + T - 1) / T * p.E) * ((p.N + T - 1) / T);
    };
    // tiles of 128 (half the loads a product) while there are two for every SM, of 64 for fewer
    const bool large = tiles(128) >= 2 * (int64_t)sms;
    // less than one for every SM: their sums are split among blocks, each of
    // which keeps eight steps or more (26 rows an expert, 96 x 3843: 51 us, by
    // single blocks 173)
    const int64_t steps = (ROWS ? p.K : p.rows / p.E) / 32;
    p.splits = 1;
    while (!large && p.splits < kMaxCluster && tiles(64) * p.splits <= sms && steps >= p.splits * 16) p.splits *= 2;
    const int64_t grid = std::min<int64_t>(tiles(large ? 128 : 64) * p.splits, (int64_t)sms * (large || p.splits > 1 ? 2 : 3) / p.splits * p.splits);
    void* args[] = {&p};
    const void* fn = large          ? (const void*)plain_product_kernel<TO, ROWS, BK, 128, false>
                     : p.splits > 1 ? (const void*)plain_product_kernel<TO, ROWS, BK, 64, true>
                                    : (const void*)plain_product_kernel<TO, ROWS, BK, 64, false>;
    return launch_op(fn, dim3((unsigned)grid), dim3(kPThreads), args, 0, stream, p.splits);
}
template <bool ROWS, bool BK>
cudaError_t launch_plain(const PlainParams& p, hc_dtype_t out, cudaStream_t stream, int sms) {
    return out == HC_BFLOAT16 ? launch_plain<Bf16, ROWS, BK>(p, stream, sms) : launch_plain<float, ROWS, BK>(p, stream, sms);
}

// ---------------------------------------------------------------------------
// operands that tiled copies cannot take (pointers or strides that are not
// whole 16 bytes) are copied row by row into scratch first
// ---------------------------------------------------------------------------
struct PackJob {
    const Bf16* from;
    Bf16* to;
    int64_t rows, per;          // rows in all, rows of one expert
    int64_t stride, expert;     // of `from`
    int cols, pitch;            // pitch: of `to`
    int weights;                // experts without rows are left out
};
constexpr int kPackJobs = 3;
struct PackParams {
    PackJob job[kPackJobs];
    const int32_t* offsets;
    int jobs, experts;
};
constexpr int kPackThreads = 256;

// A warp takes a row, a lane eight elements.
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackParams p) {
    __shared__ bool used[kMaxExperts];
    grid_wait();
    grid_release();
    // offsets that do not rise give no rows, whatever is before them
    for (int e = threadIdx.x; e < p.experts; e += kPackThreads) used[e] = p.offsets[e + 1] > p.offsets[e];
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int first = blockIdx.x * (kPackThreads / 32) + threadIdx.x / 32, step = gridDim.x * (kPackThreads / 32);
    for (int j = 0; j < p.jobs; j++) {
        const PackJob& q = p.job[j];
        const int vectors = q.pitch / 8;
        for (int64_t r = first; r < q.rows; r += step) {
            const int64_t e = r / q.per;
            if (q.weights && !used[e]) continue;
            const uintptr_t from = (uintptr_t)(q.from + e * q.expert + (r - e * q.per) * q.stride);
            const uintptr_t end = from + 2 * (uintptr_t)q.cols, base = from & ~(uintptr_t)15;
            const int s = (int)(from & 15);
            uint4* to = (uint4*)(q.to + r * q.pitch);
            for (int c0 = lane; c0 < vectors; c0 += 128) {
                uint4 u[4], v[4];  // as in row_vector, but nobody reads what lies behind a row
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uintptr_t a = base + 16 * (uintptr_t)(c0 + 32 * k);
                    u[k] = v[k] = make_uint4(0, 0, 0, 0);
                    if (a < end) u[k] = *(const uint4*)a;
                    if (s && a + 16 < end) v[k] = *(const uint4*)(a + 16);
                }
#pragma unroll
                for (int k = 0; k < 4; k++)
                    if (c0 + 32 * k < vectors) to[c0 + 32 * k] = bytes_from(u[k], v[k], s);
            }
        }
    }
}

// A bf16 operand of the tensor cores: `experts` times `rows` rows of `cols`.
struct Operand {
    const void* p;
    int64_t experts, rows, cols, stride, expert;
    bool weights;
    bool aligned() const { return (uintptr_t)p % 16 == 0 && stride % 8 == 0 && expert % 8 == 0; }
    int64_t pitch() const { return (cols + 7) / 8 * 8; }
    size_t packed_bytes() const { return (size_t)(experts * rows * pitch() * 2 + 255) / 256 * 256; }
};

// Whether the first two products take the kernel for few rows: where tiles
// would first need a copy of the weights (1 token through 2 of 8 experts of
// 4096 x 1024, aligned: 8.1 us against 7.2 in tiles; of 4095 x 1023: 8 against 12).
bool few_rows(const Operand& a, const Operand& w, bool along) {
    return along && !(a.aligned() && w.aligned()) && a.rows <= kFewRows && a.cols <= kFewDim;
}

// Copies those of the operands that need it into scratch, and points them there.
cudaError_t pack(Operand* const* list, int n, const int32_t* offsets, size_t experts, void* scratch, cudaStream_t stream, int sms) {
    PackParams p = {};
    p.offsets = offsets;
    p.experts = (int)experts;
    unsigned char* at = (unsigned char*)scratch;
    int64_t most = 0;
    for (int i = 0; i < n; i++) {
        Operand& x = *list[i];
        if (x.aligned()) continue;
        PackJob& q = p.job[p.jobs++];
        q.from = (const Bf16*)x.p;
        q.to = (Bf16*)at;
        q.rows = x.experts * x.rows;
        q.per = x.rows;
        q.stride = x.stride;
        q.expert = x.expert;
        q.cols = (int)x.cols;
        q.pitch = (int)x.pitch();
        q.weights = x.weights;
        at += x.packed_bytes();
        most = std::max(most, q.rows);
        x.p = q.to;
        x.stride = q.pitch;
        x.expert = x.rows * q.pitch;
    }
    if (!most) return cudaSuccess;
    const int64_t blocks = std::min<int64_t>((most + kPackThreads / 32 - 1) / (kPackThreads / 32), (int64_t)sms * 8);
    void* args[] = {&p};
    return launch_op((const void*)pack_kernel, dim3((unsigned)blocks), dim3(kPackThreads), args, 0, stream);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (EncodeTiled)f;
    }();
    return fn;
}
// Boxes of box_rows rows of 64 columns; what lies outside reads as zeros.
cudaError_t describe(CUtensorMap* map, const Operand& x, int box_rows, bool experts) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)x.cols, (cuuint64_t)std::max<int64_t>(1, x.rows), (cuuint64_t)x.experts};
    const cuuint64_t strides[2] = {(cuuint64_t)x.stride * 2, (cuuint64_t)x.expert * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, experts ? 3 : 2, const_cast<void*>(x.p), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <bool ROWS, bool WK, int G, class TO, bool LONG>
cudaError_t launch_tensor(TensorParams& p, const Operand& a, const Operand& b, cudaStream_t stream, int sms) {
    constexpr int T = kTM * G;
    cudaError_t e = describe(&p.a, a, ROWS && WK ? kTM : 64, ROWS);
    if (e == cudaSuccess) e = describe(&p.b, b, 64, false);
    if (e != cudaSuccess) return e;
    p.err = device_error_flag();
    if (!p.err) return cudaErrorInvalidValue;
    p.hold = expiring_waits() ? 1 : 0;
    p.wait_ns = p.hold ? kTestWaitLimitNs : kWaitLimitNs;
    const void* fn = (const void*)tensor_product_kernel<ROWS, WK, G, TO, LONG>;
    if (!allow_smem((void*)fn, kTSmem)) return cudaErrorInvalidValue;
    const int64_t nt = (p.N + T - 1) / T;
    const int64_t mt = ROWS ? p.rows / T + std::min<int64_t>(p.E, p.rows) + 1 : (int64_t)((p.M + T - 1) / T) * p.E;
    void* args[] = {&p};
    const int64_t grid = std::min<int64_t>(mt * nt, sms / G) * G;
    return launch_op(fn, dim3((unsigned)grid), dim3(kTThreadsOf<LONG>), args, kTSmem, stream, G);
}
template <bool ROWS, bool WK>
cudaError_t launch_tensor(TensorParams& p, const Operand& a, const Operand& b, hc_dtype_t out, cudaStream_t stream, int sms) {
    // Two blocks a tile, unless that leaves pairs of SMs without one.
    const int64_t mt = ROWS ? (p.rows + 255) / 256 : (int64_t)((p.M + 255) / 256) * p.E;
    const bool two = mt * ((p.N + 255) / 256) >= sms / 2;
    if (out == HC_FLOAT32)
        return two ? launch_tensor<ROWS, WK, 2, float, true>(p, a, b, stream, sms)
                   : launch_tensor<ROWS, WK, 1, float, true>(p, a, b, stream, sms);
    if ((ROWS ? p.K : p.rows) > kTPlain)  // a group's rows are the device's to know: all of them at most
        return two ? launch_tensor<ROWS, WK, 2, Bf16, true>(p, a, b, stream, sms)
                   : launch_tensor<ROWS, WK, 1, Bf16, true>(p, a, b, stream, sms);
    return two ? launch_tensor<ROWS, WK, 2, Bf16, false>(p, a, b, stream, sms)
               : launch_tensor<ROWS, WK, 1, Bf16, false>(p, a, b, stream, sms);
}

Operand rows_operand(const void* p, size_t rows, size_t cols, size_t stride) {
    // a single row has no next one: any stride will do
    return Operand{p, 1, (int64_t)rows, (int64_t)cols, rows > 1 ? (int64_t)stride : ((int64_t)cols + 7) / 8 * 8, 0, false};
}
Operand weight_operand(const void* p, size_t experts, size_t in, size_t out, hc_weight_layout_t layout, size_t stride, size_t expert) {
    const bool out_in = layout == HC_WEIGHT_OUT_IN;
    return Operand{p, (int64_t)experts, (int64_t)(out_in ? out : in), (int64_t)(out_in ? in : out), (int64_t)stride, (int64_t)expert, true};
}
size_t packed(const Operand& x) { return x.aligned() ? 0 : x.packed_bytes(); }

// The first two products: rows of `a` times the weight, which is summed along
// its own rows (along) or across them.
cudaError_t rows_product(const Operand& a, const Operand& w, bool along, void* out, size_t out_stride, size_t N, hc_dtype_t in,
                         hc_dtype_t to, const int32_t* offsets, cudaStream_t stream, int sms) {
    if (in == HC_FLOAT32) {
        PlainParams p = {};
        p.a = a.p;
        p.b = w.p;
        p.out = out;
        p.offsets = offsets;
        p.rows = a.rows;
        p.a_stride = a.stride;
        p.b_stride = w.stride;
        p.b_expert = w.expert;
        p.out_stride = (int64_t)out_stride;
        p.E = (int)w.experts;
        p.N = (int)N;
        p.K = (int)a.cols;
        p.a_vec = whole(a.p, (size_t)a.stride, 0, 4);
        p.b_vec = whole(w.p, (size_t)w.stride, (size_t)w.expert, 4);
        return along ? launch_plain<true, true>(p, to, stream, sms) : launch_plain<true, false>(p, to, stream, sms);
    }
    if (few_rows(a, w, along)) {
        FewParams p;
        p.x = (const Bf16*)a.p;
        p.w = (const Bf16*)w.p;
        p.out = out;
        p.offsets = offsets;
        p.rows = a.rows;
        p.x_stride = a.stride;
        p.w_stride = w.stride;
        p.w_expert = w.expert;
        p.out_stride = (int64_t)out_stride;
        p.E = (int)w.experts;
        p.N = (int)N;
        p.K = (int)a.cols;
        void* args[] = {&p};
        const dim3 grid((unsigned)((N + kFewBlock - 1) / kFewBlock), (unsigned)std::min<int64_t>(w.experts, a.rows));
        const void* fn = to == HC_BFLOAT16 ? (const void*)few_rows_kernel<Bf16> : (const void*)few_rows_kernel<float>;
        const int smem = kFewAtOnce * (int)a.pitch() * 2;
        if (!allow_smem((void*)fn, smem)) return cudaErrorInvalidValue;
        return launch_op(fn, grid, dim3(kFewThreads), args, smem, stream);
    }
    TensorParams p;
    p.out = out;
    p.offsets = offsets;
    p.rows = a.rows;
    p.out_stride = (int64_t)out_stride;
    p.out_expert = 0;
    p.E = (int)w.experts;
    p.M = 0;
    p.N = (int)N;
    p.K = (int)a.cols;
    p.accumulate = 0;
    p.out_vec = whole(out, out_stride, 0, elem_bytes(to));
    return along ? launch_tensor<true, true>(p, w, a, to, stream, sms) : launch_tensor<true, false>(p, w, a, to, stream, sms);
}

}  // namespace

size_t expert_matmul_scratch(const hc_expert_matmul_t& a) {
    if (a.dtype != HC_BFLOAT16 || !a.rows) return 0;
    const Operand x = rows_operand(a.x, a.rows, a.in_dim, a.x_stride);
    const Operand w = weight_operand(a.weight, a.experts, a.in_dim, a.out_dim, a.weight_layout, a.weight_stride, a.expert_stride);
    return few_rows(x, w, a.weight_layout == HC_WEIGHT_OUT_IN) ? 0 : packed(x) + packed(w);
}

size_t expert_matmul_grad_scratch(const hc_expert_matmul_grad_t& a) {
    if (a.dtype != HC_BFLOAT16 || !a.rows) return 0;
    const Operand go = rows_operand(a.grad_out, a.rows, a.out_dim, a.grad_out_stride);
    const Operand w = weight_operand(a.weight, a.experts, a.in_dim, a.out_dim, a.weight_layout, a.weight_stride, a.expert_stride);
    const bool few = a.grad_x && few_rows(go, w, a.weight_layout == HC_WEIGHT_IN_OUT);
    size_t n = few && !a.grad_weight ? 0 : packed(go);
    if (a.grad_x && !few) n += packed(w);
    if (a.grad_weight) n += packed(rows_operand(a.x, a.rows, a.in_dim, a.x_stride));
    return n;
}

cudaError_t launch_expert_matmul(const hc_expert_matmul_t& a, cudaStream_t stream, int sms) {
    Operand x = rows_operand(a.x, a.rows, a.in_dim, a.x_stride);
    Operand w = weight_operand(a.weight, a.experts, a.in_dim, a.out_dim, a.weight_layout, a.weight_stride, a.expert_stride);
    if (a.dtype == HC_BFLOAT16 && !few_rows(x, w, a.weight_layout == HC_WEIGHT_OUT_IN)) {
        Operand* const list[] = {&x, &w};
        const cudaError_t e = pack(list, 2, a.offsets, a.experts, a.scratch, stream, sms);
        if (e != cudaSuccess) return e;
    }
    return rows_product(x, w, a.weight_layout == HC_WEIGHT_OUT_IN, a.out, a.out_stride, a.out_dim, a.dtype, a.out_dtype, a.offsets,
                        stream, sms);
}

cudaError_t launch_expert_matmul_grad(const hc_expert_matmul_grad_t& a, cudaStream_t stream, int sms) {
    const bool out_in = a.weight_layout == HC_WEIGHT_OUT_IN;
    Operand go = rows_operand(a.grad_out, a.rows, a.out_dim, a.grad_out_stride);
    Operand x = rows_operand(a.x, a.rows, a.in_dim, a.x_stride);
    Operand w = weight_operand(a.weight, a.experts, a.in_dim, a.out_dim, a.weight_layout, a.weight_stride, a.expert_stride);
    const Operand given = go;
    const bool few = a.dtype == HC_BFLOAT16 && a.grad_x && few_rows(go, w, !out_in);
    if (a.dtype == HC_BFLOAT16 && a.rows) {
        Operand* list[kPackJobs];
        int n = 0;
        if (!few || a.grad_weight) list[n++] = &go;
        if (a.grad_x && !few) list[n++] = &w;
        if (a.grad_weight) list[n++] = &x;
        const cudaError_t e = pack(list, n, a.offsets, a.experts, a.scratch, stream, sms);
        if (e != cudaSuccess) return e;
    }
    if (a.grad_x && a.rows) {
        const cudaError_t e =
            rows_product(few ? given : go, w, !out_in, a.grad_x, a.grad_x_stride, a.in_dim, a.dtype, a.dtype, a.offsets, stream, sms);
        if (e != cudaSuccess) return e;
    }
    if (!a.grad_weight) return cudaSuccess;
    const size_t M = out_in ? a.out_dim : a.in_dim, N = out_in ? a.in_dim : a.out_dim;
    if (a.dtype == HC_FLOAT32) {
        const Operand &m = out_in ? go : x, &n = out_in ? x : go;
        PlainParams p = {};
        p.a = m.p;
        p.b = n.p;
        p.out = a.grad_weight;
        p.offsets = a.offsets;
        p.rows = (int64_t)a.rows;
        p.a_stride = m.stride;
        p.b_stride = n.stride;
        p.out_stride = (int64_t)a.grad_weight_stride;
        p.out_expert = (int64_t)a.grad_expert_stride;
        p.E = (int)a.experts;
        p.M = (int)M;
        p.N = (int)N;
        p.a_vec = whole(m.p, (size_t)m.stride, 0, 4);
        p.b_vec = whole(n.p, (size_t)n.stride, 0, 4);
        p.accumulate = a.accumulate;
        return launch_plain<false, false>(p, a.grad_weight_dtype, stream, sms);
    }
    if (!a.rows) {  // no row is read, but a copy's description wants an address and a stride
        go.p = x.p = (const void*)((uintptr_t)a.grad_weight / 16 * 16);
        go.stride = go.pitch();
        x.stride = x.pitch();
    }
    TensorParams p;
    p.out = a.grad_weight;
    p.offsets = a.offsets;
    p.rows = (int64_t)a.rows;
    p.out_stride = (int64_t)a.grad_weight_stride;
    p.out_expert = (int64_t)a.grad_expert_stride;
    p.E = (int)a.experts;
    p.M = (int)M;
    p.N = (int)N;
    p.K = 0;
    p.accumulate = a.accumulate;
    p.out_vec = whole(a.grad_weight, a.grad_weight_stride, a.grad_expert_stride, elem_bytes(a.grad_weight_dtype));
    return launch_tensor<false, false>(p, out_in ? go : x, out_in ? x : go, a.grad_weight_dtype, stream, sms);
}

}  // namespace hc
