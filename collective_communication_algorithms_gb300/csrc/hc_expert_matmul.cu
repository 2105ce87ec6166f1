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

#include "hc_ops.cuh"

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
};

constexpr int kPT = 128, kPK = 16, kPThreads = 256, kPPad = 4;

template <class T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&v)[8]) {
    if (vec && n >= 8) {
        load_n<T, 8>(p, 8, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = i < n ? to_f32(p[i]) : 0.0f;
    }
}

// ROWS: the first two products, whose sums run along a's rows; b is summed
// along its rows (BK) or across them.
template <class T, class TO, bool ROWS, bool BK>
__global__ void __launch_bounds__(kPThreads) plain_product_kernel(const PlainParams p) {
    __shared__ __align__(16) float as[kPK][kPT + kPPad], bs[kPK][kPT + kPPad];
    __shared__ int bound[kMaxExperts + 1], tile[kMaxExperts + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    grid_wait();
    grid_release();
    if (tid < 32) read_groups(p.offsets, p.E, p.rows, kPT, bound, tile);
    __syncthreads();
    const int nt = (p.N + kPT - 1) / kPT;
    const int64_t mt = ROWS ? tile[p.E] : (int64_t)((p.M + kPT - 1) / kPT) * p.E;
    for (int64_t i = blockIdx.x; i < mt * nt; i += gridDim.x) {
        const int m = (int)(i / nt), n0 = (int)(i % nt) * kPT;
        int e, m0, mlen, K;
        int64_t first;  // ROWS: the tile's first row; else the group's
        if (ROWS) {
            e = group_of(tile, p.E, m);
            first = bound[e] + (int64_t)(m - tile[e]) * kPT;
            m0 = 0;
            mlen = (int)min((int64_t)kPT, bound[e + 1] - first);
            K = p.K;
        } else {
            const int per = (p.M + kPT - 1) / kPT;
            e = m / per;
            m0 = (m % per) * kPT;
            mlen = min(kPT, p.M - m0);
            first = bound[e];
            K = bound[e + 1] - bound[e];
            if (!K && p.accumulate) continue;
        }
        const int nlen = min(kPT, p.N - n0);
        const T* a = (const T*)p.a + first * p.a_stride + m0;
        const T* b = (const T*)p.b + (ROWS ? e * p.b_expert + (BK ? (int64_t)n0 * p.b_stride : n0)
                                           : first * p.b_stride + n0);
        // places of this thread's 8 elements: along k (row, k) or along m (k, column)
        const int kr = tid / 2, kc = (tid % 2) * 8, mr = tid / 16, mc = (tid % 16) * 8;
        float av[8], bv[8], acc[8][8];
#pragma unroll
        for (int x = 0; x < 8; x++)
#pragma unroll
            for (int y = 0; y < 8; y++) acc[x][y] = 0.0f;
        auto fetch = [&](int k0) {
            if (ROWS) load8(a + kr * p.a_stride + k0 + kc, kr < mlen ? K - k0 - kc : 0, p.a_vec, av);
            else load8(a + (int64_t)(k0 + mr) * p.a_stride + mc, k0 + mr < K ? mlen - mc : 0, p.a_vec, av);
            if (BK) load8(b + kr * p.b_stride + k0 + kc, kr < nlen ? K - k0 - kc : 0, p.b_vec, bv);
            else load8(b + (int64_t)(k0 + mr) * p.b_stride + mc, k0 + mr < K ? nlen - mc : 0, p.b_vec, bv);
        };
        if (K) fetch(0);
        for (int k0 = 0; k0 < K; k0 += kPK) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (ROWS) as[kc + j][kr] = av[j];
                else as[mr][mc + j] = av[j];
                if (BK) bs[kc + j][kr] = bv[j];
                else bs[mr][mc + j] = bv[j];
            }
            __syncthreads();
            if (k0 + kPK < K) fetch(k0 + kPK);
#pragma unroll
            for (int k = 0; k < kPK; k++) {
                float x[8], y[8];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float4 u = *(const float4*)&as[k][h * 64 + ty * 4], w = *(const float4*)&bs[k][h * 64 + tx * 4];
                    x[4 * h] = u.x; x[4 * h + 1] = u.y; x[4 * h + 2] = u.z; x[4 * h + 3] = u.w;
                    y[4 * h] = w.x; y[4 * h + 1] = w.y; y[4 * h + 2] = w.z; y[4 * h + 3] = w.w;
                }
#pragma unroll
                for (int q = 0; q < 8; q++)
#pragma unroll
                    for (int r = 0; r < 8; r++) acc[q][r] = fmaf(x[q], y[r], acc[q][r]);
            }
        }
        TO* out = (TO*)p.out + (ROWS ? first * p.out_stride : e * p.out_expert + (int64_t)m0 * p.out_stride) + n0;
#pragma unroll
        for (int q = 0; q < 8; q++) {
            const int row = (q / 4) * 64 + ty * 4 + q % 4;
            if (row >= mlen) continue;
#pragma unroll
            for (int r = 0; r < 8; r++) {
                const int col = (r / 4) * 64 + tx * 4 + r % 4;
                if (col >= nlen) continue;
                TO* at = out + row * p.out_stride + col;
                put(at, (!ROWS && p.accumulate ? to_f32(*at) : 0.0f) + acc[q][r]);
            }
        }
    }
}

bool whole(const void* p, size_t stride, size_t expert, int es) {
    return (uintptr_t)p % 16 == 0 && stride * es % 16 == 0 && expert * es % 16 == 0;
}

template <class T, class TO, bool ROWS, bool BK>
cudaError_t launch_plain(PlainParams p, cudaStream_t stream, int sms) {
    const int64_t nt = (p.N + kPT - 1) / kPT;
    const int64_t mt = ROWS ? p.rows / kPT + std::min<int64_t>(p.E, p.rows) + 1 : (int64_t)((p.M + kPT - 1) / kPT) * p.E;
    const int64_t grid = std::min<int64_t>(mt * nt, (int64_t)sms * 2);
    void* args[] = {&p};
    return launch_op((const void*)plain_product_kernel<T, TO, ROWS, BK>, dim3((unsigned)grid), dim3(kPThreads), args, 0, stream);
}
template <bool ROWS, bool BK>
cudaError_t launch_plain(const PlainParams& p, hc_dtype_t in, hc_dtype_t out, cudaStream_t stream, int sms) {
    if (in == HC_BFLOAT16)
        return out == HC_BFLOAT16 ? launch_plain<Bf16, Bf16, ROWS, BK>(p, stream, sms)
                                  : launch_plain<Bf16, float, ROWS, BK>(p, stream, sms);
    return out == HC_BFLOAT16 ? launch_plain<float, Bf16, ROWS, BK>(p, stream, sms)
                              : launch_plain<float, float, ROWS, BK>(p, stream, sms);
}

}  // namespace

size_t expert_matmul_scratch(const hc_expert_matmul_t&) { return 0; }
size_t expert_matmul_grad_scratch(const hc_expert_matmul_grad_t&) { return 0; }

cudaError_t launch_expert_matmul(const hc_expert_matmul_t& a, cudaStream_t stream, int sms) {
    PlainParams p = {};
    const int es = elem_bytes(a.dtype);
    p.a = a.x;
    p.b = a.weight;
    p.out = a.out;
    p.offsets = a.offsets;
    p.rows = (int64_t)a.rows;
    p.a_stride = (int64_t)a.x_stride;
    p.b_stride = (int64_t)a.weight_stride;
    p.b_expert = (int64_t)a.expert_stride;
    p.out_stride = (int64_t)a.out_stride;
    p.E = (int)a.experts;
    p.N = (int)a.out_dim;
    p.K = (int)a.in_dim;
    p.a_vec = whole(a.x, a.x_stride, 0, es);
    p.b_vec = whole(a.weight, a.weight_stride, a.expert_stride, es);
    return a.weight_layout == HC_WEIGHT_OUT_IN ? launch_plain<true, true>(p, a.dtype, a.out_dtype, stream, sms)
                                               : launch_plain<true, false>(p, a.dtype, a.out_dtype, stream, sms);
}

cudaError_t launch_expert_matmul_grad(const hc_expert_matmul_grad_t& a, cudaStream_t stream, int sms) {
    const int es = elem_bytes(a.dtype);
    PlainParams p = {};
    p.offsets = a.offsets;
    p.rows = (int64_t)a.rows;
    p.E = (int)a.experts;
    if (a.grad_x && a.rows) {
        p.a = a.grad_out;
        p.b = a.weight;
        p.out = a.grad_x;
        p.a_stride = (int64_t)a.grad_out_stride;
        p.b_stride = (int64_t)a.weight_stride;
        p.b_expert = (int64_t)a.expert_stride;
        p.out_stride = (int64_t)a.grad_x_stride;
        p.N = (int)a.in_dim;
        p.K = (int)a.out_dim;
        p.a_vec = whole(a.grad_out, a.grad_out_stride, 0, es);
        p.b_vec = whole(a.weight, a.weight_stride, a.expert_stride, es);
        const cudaError_t e = a.weight_layout == HC_WEIGHT_OUT_IN
                                  ? launch_plain<true, false>(p, a.dtype, a.dtype, stream, sms)
                                  : launch_plain<true, true>(p, a.dtype, a.dtype, stream, sms);
        if (e != cudaSuccess) return e;
    }
    if (!a.grad_weight) return cudaSuccess;
    const bool out_in = a.weight_layout == HC_WEIGHT_OUT_IN;
    p.a = out_in ? a.grad_out : a.x;
    p.b = out_in ? a.x : a.grad_out;
    p.a_stride = (int64_t)(out_in ? a.grad_out_stride : a.x_stride);
    p.b_stride = (int64_t)(out_in ? a.x_stride : a.grad_out_stride);
    p.M = (int)(out_in ? a.out_dim : a.in_dim);
    p.N = (int)(out_in ? a.in_dim : a.out_dim);
    p.out = a.grad_weight;
    p.out_stride = (int64_t)a.grad_weight_stride;
    p.out_expert = (int64_t)a.grad_expert_stride;
    p.a_vec = whole(p.a, (size_t)p.a_stride, 0, es);
    p.b_vec = whole(p.b, (size_t)p.b_stride, 0, es);
    p.accumulate = a.accumulate;
    return launch_plain<false, false>(p, a.dtype, a.grad_weight_dtype, stream, sms);
}

}  // namespace hc
