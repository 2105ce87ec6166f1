// hc_ops.cpp -- the C ABI of the training operators (see include/hc.h):
// argument validation, strides, overlap checks and dispatch to the kernels.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "hc_ops.h"

using namespace hc;

namespace {

bool float_dtype(hc_dtype_t d) { return d == HC_FLOAT32 || d == HC_BFLOAT16; }
bool known_dtype(hc_dtype_t d) { return float_dtype(d) || d == HC_INT32; }
bool known_id(hc_id_t i) { return i == HC_ID32 || i == HC_ID64; }
size_t id_bytes(hc_id_t i) { return i == HC_ID64 ? 8 : 4; }

// INVALID_ARG for values that are no dtype, UNSUPPORTED for int32
hc_status_t check_float(hc_dtype_t d) {
    if (!known_dtype(d)) return HC_ERR_INVALID_ARG;
    return float_dtype(d) ? HC_OK : HC_ERR_UNSUPPORTED;
}

constexpr size_t kMaxTokens = 0x7FFFFFFFu;
constexpr size_t kMaxEmbeddingDim = 1u << 24;

// A matrix operand: rows x cols elements of es bytes, `stride` elements apart.
struct Matrix {
    uintptr_t base = 0;
    size_t rows = 0, row_bytes = 0, pitch = 0;
    bool empty() const { return !base || !rows || !row_bytes; }
    uintptr_t end() const { return base + (rows - 1) * pitch + row_bytes; }
};

// Resolves a stride (0: the row length) and describes the operand.
hc_status_t matrix(const void* p, size_t rows, size_t cols, size_t* stride, size_t es, Matrix* out) {
    if (*stride == 0) *stride = cols;
    if (*stride < cols) return HC_ERR_INVALID_ARG;
    if (cols > (size_t)INT64_MAX / 16 || *stride > (size_t)INT64_MAX / 16 / (rows ? rows : 1)) return HC_ERR_INVALID_ARG;
    *out = Matrix();
    out->base = (uintptr_t)p;
    out->rows = rows;
    out->row_bytes = cols * es;
    out->pitch = *stride * es;
    if (!p) return HC_OK;
    return (uintptr_t)p % es ? HC_ERR_ALIGN : HC_OK;
}
hc_status_t vector(const void* p, size_t n, size_t es, Matrix* out) {
    size_t stride = 0;
    return matrix(p, 1, n, &stride, es, out);
}

// Whether two operands share a byte.  Exact for equal pitches (rows may
// interleave), conservative (address ranges) otherwise.
bool overlap(const Matrix& a, const Matrix& b) {
    if (a.empty() || b.empty()) return false;
    if (a.end() <= b.base || b.end() <= a.base) return false;
    if (a.pitch != b.pitch || a.rows == 1 || b.rows == 1) return true;
    const Matrix& lo = a.base <= b.base ? a : b;
    const Matrix& hi = a.base <= b.base ? b : a;
    const size_t d = (hi.base - lo.base) % lo.pitch;
    return !(d >= lo.row_bytes && d + hi.row_bytes <= lo.pitch);
}
bool same_place(const Matrix& a, const Matrix& b) {
    return a.base == b.base && (a.pitch == b.pitch || a.rows == 1) && a.row_bytes == b.row_bytes;
}

struct Use {
    Matrix m;
    bool write;
    bool in_place;  // an input that an output may replace, or an output that may do so
};
hc_status_t check_overlaps(const Use* u, int n) {
    for (int i = 0; i < n; i++)
        for (int j = 0; j < n; j++) {
            if (i == j || !u[i].write || (u[j].write && j < i) || !overlap(u[i].m, u[j].m)) continue;
            if (!u[j].write && u[i].in_place && u[j].in_place && same_place(u[i].m, u[j].m)) continue;
            return HC_ERR_INVALID_ARG;
        }
    return HC_OK;
}

#define HC_TRY(expr)                          \
    do {                                      \
        const hc_status_t st_ = (expr);       \
        if (st_ != HC_OK) return st_;         \
    } while (0)

hc_status_t check_scratch(const void* p, size_t have, size_t need) {
    if (!need) return HC_OK;
    if (!p || have < need) return HC_ERR_SCRATCH;
    return (uintptr_t)p & 15 ? HC_ERR_ALIGN : HC_OK;
}

// Runs a launcher on the current device.
template <class F>
hc_status_t launch(F f) {
    const int sms = sm_count_of_current_device();
    if (sms <= 0) return cuda_status(cudaErrorNoDevice);
    return cuda_status(f(sms));
}

hc_status_t embedding_sizes(size_t tokens, size_t rows, size_t dim) {
    if (!dim || !rows) return HC_ERR_INVALID_ARG;
    if (tokens > kMaxTokens || rows > kMaxTokens || dim > kMaxEmbeddingDim) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}

hc_status_t norm_sizes(size_t tokens, size_t dim, bool gate, size_t gate_rows) {
    if (!dim) return HC_ERR_INVALID_ARG;
    if (gate && (!gate_rows || tokens % gate_rows)) return HC_ERR_INVALID_ARG;
    if (dim > kBlockNormMaxDim || tokens > kMaxTokens || (gate && gate_rows > kMaxTokens)) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}

// ---------------------------------------------------------------- clipping
struct Span {
    uintptr_t lo, hi;
    bool write;
};

hc_status_t clip_tensors(const hc_clip_grads_t& a, bool apply) {
    if (a.num && !a.tensors) return HC_ERR_INVALID_ARG;
    if (a.num > kMaxTokens) return HC_ERR_UNSUPPORTED;
    for (size_t i = 0; i < a.num; i++) {
        const hc_grad_t& g = a.tensors[i];
        HC_TRY(check_float(g.in_dtype));
        if (g.count >> 56) return HC_ERR_UNSUPPORTED;
        if (g.count && !g.in) return HC_ERR_INVALID_ARG;
        if ((uintptr_t)g.in % elem_bytes(g.in_dtype)) return HC_ERR_ALIGN;
        if (!apply || !g.out) continue;
        HC_TRY(check_float(g.out_dtype));
        if ((uintptr_t)g.out % elem_bytes(g.out_dtype)) return HC_ERR_ALIGN;
        if (g.out == g.in && g.out_dtype != g.in_dtype) return HC_ERR_INVALID_ARG;
    }
    return HC_OK;
}

// Whether an output shares a byte with another operand.
hc_status_t clip_overlaps(const hc_clip_grads_t& a, bool apply, size_t scratch) {
    std::unique_ptr<Span[]> s(new (std::nothrow) Span[2 * a.num + 3]);
    if (!s) return cuda_status(cudaErrorMemoryAllocation);
    size_t n = 0;
    for (size_t i = 0; i < a.num; i++) {
        const hc_grad_t& g = a.tensors[i];
        if (!g.count) continue;
        const bool in_place = !g.out || g.out == g.in;
        s[n++] = Span{(uintptr_t)g.in, (uintptr_t)g.in + g.count * elem_bytes(g.in_dtype), apply && in_place};
        if (apply && !in_place) s[n++] = Span{(uintptr_t)g.out, (uintptr_t)g.out + g.count * elem_bytes(g.out_dtype), true};
    }
    s[n++] = Span{(uintptr_t)a.norm, (uintptr_t)a.norm + sizeof(float), true};
    if (apply && a.factor) s[n++] = Span{(uintptr_t)a.factor, (uintptr_t)a.factor + sizeof(float), true};
    if (scratch) s[n++] = Span{(uintptr_t)a.scratch, (uintptr_t)a.scratch + scratch, true};
    const auto before = [](const Span& x, const Span& y) { return x.lo < y.lo; };
    if (!std::is_sorted(s.get(), s.get() + n, before)) std::sort(s.get(), s.get() + n, before);
    uintptr_t any = 0, written = 0;  // where the spans so far end
    for (size_t i = 0; i < n; i++) {
        if (s[i].lo < (s[i].write ? any : written)) return HC_ERR_INVALID_ARG;
        any = std::max(any, s[i].hi);
        if (s[i].write) written = std::max(written, s[i].hi);
    }
    return HC_OK;
}

hc_status_t clip(const hc_clip_grads_t* args, bool apply, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_clip_grads_t)) return HC_ERR_INVALID_ARG;
    const hc_clip_grads_t a = *args;
    if (!std::isfinite(a.scale) || !a.norm) return HC_ERR_INVALID_ARG;
    if (apply && (!(a.max_norm > 0.0f) || !(a.eps >= 0.0f) || !std::isfinite(a.eps))) return HC_ERR_INVALID_ARG;
    HC_TRY(clip_tensors(a, apply));
    if ((uintptr_t)a.norm % sizeof(float) || (apply && (uintptr_t)a.factor % sizeof(float))) return HC_ERR_ALIGN;
    const size_t need = clip_scratch_bytes(a);
    HC_TRY(check_scratch(a.scratch, a.scratch_bytes, need));
    HC_TRY(clip_overlaps(a, apply, need));
    const TraceRange range(apply ? "hc_clip_grads" : "hc_grad_norm", 0, (uint64_t)a.num);
    return launch([&](int) { return launch_clip(a, apply, (cudaStream_t)stream); });
}

// ---------------------------------------------------------------- expert layer
// The weights of all experts: `rows` rows of `cols` elements each, experts
// `expert` elements apart.
hc_status_t weights(const void* p, size_t experts, size_t rows, size_t cols, size_t* stride, size_t* expert, size_t es,
                    Matrix* out) {
    Matrix one;
    HC_TRY(matrix(p, rows, cols, stride, es, &one));
    const size_t extent = (rows - 1) * *stride + cols;
    if (*expert == 0 || experts == 1) *expert = rows * *stride;
    if (experts > 1 && *expert < extent) return HC_ERR_INVALID_ARG;
    if (*expert > (size_t)INT64_MAX / 16 / experts) return HC_ERR_INVALID_ARG;
    *out = one;
    if (*expert == rows * *stride) {
        out->rows = rows * experts;
    } else {  // taken as one piece
        out->rows = 1;
        out->row_bytes = ((experts - 1) * *expert + extent) * es;
        out->pitch = out->row_bytes;
    }
    return HC_OK;
}

hc_status_t matmul_sizes(size_t rows, size_t experts, size_t in_dim, size_t out_dim) {
    if (!experts || !in_dim || !out_dim) return HC_ERR_INVALID_ARG;
    if (experts > kMaxExperts || rows > kMaxExpertRows || in_dim > kMaxExpertDim || out_dim > kMaxExpertDim)
        return HC_ERR_UNSUPPORTED;
    return HC_OK;
}
bool known_layout(hc_weight_layout_t l) { return l == HC_WEIGHT_OUT_IN || l == HC_WEIGHT_IN_OUT; }

// Strides and operands of the products, without the scratch.
hc_status_t matmul_operands(hc_expert_matmul_t& a, Use* u) {
    HC_TRY(check_float(a.dtype));
    HC_TRY(check_float(a.out_dtype));
    if (!known_layout(a.weight_layout)) return HC_ERR_INVALID_ARG;
    HC_TRY(matmul_sizes(a.rows, a.experts, a.in_dim, a.out_dim));
    const size_t es = elem_bytes(a.dtype);
    const bool out_in = a.weight_layout == HC_WEIGHT_OUT_IN;
    HC_TRY(matrix(a.x, a.rows, a.in_dim, &a.x_stride, es, &u[0].m));
    HC_TRY(weights(a.weight, a.experts, out_in ? a.out_dim : a.in_dim, out_in ? a.in_dim : a.out_dim, &a.weight_stride,
                   &a.expert_stride, es, &u[1].m));
    HC_TRY(vector(a.offsets, a.experts + 1, sizeof(int32_t), &u[2].m));
    HC_TRY(matrix(a.out, a.rows, a.out_dim, &a.out_stride, elem_bytes(a.out_dtype), &u[3].m));
    u[3].write = true;
    return HC_OK;
}
hc_status_t matmul_grad_operands(hc_expert_matmul_grad_t& a, Use* u) {
    HC_TRY(check_float(a.dtype));
    HC_TRY(check_float(a.grad_weight_dtype));
    if (!known_layout(a.weight_layout) || (a.accumulate != 0 && a.accumulate != 1)) return HC_ERR_INVALID_ARG;
    HC_TRY(matmul_sizes(a.rows, a.experts, a.in_dim, a.out_dim));
    const size_t es = elem_bytes(a.dtype);
    const bool out_in = a.weight_layout == HC_WEIGHT_OUT_IN;
    const size_t wr = out_in ? a.out_dim : a.in_dim, wc = out_in ? a.in_dim : a.out_dim;
    HC_TRY(matrix(a.grad_out, a.rows, a.out_dim, &a.grad_out_stride, es, &u[0].m));
    HC_TRY(matrix(a.grad_weight ? a.x : nullptr, a.rows, a.in_dim, &a.x_stride, es, &u[1].m));
    HC_TRY(weights(a.grad_x ? a.weight : nullptr, a.experts, wr, wc, &a.weight_stride, &a.expert_stride, es, &u[2].m));
    HC_TRY(vector(a.offsets, a.experts + 1, sizeof(int32_t), &u[3].m));
    HC_TRY(matrix(a.grad_x, a.rows, a.in_dim, &a.grad_x_stride, es, &u[4].m));
    HC_TRY(weights(a.grad_weight, a.experts, wr, wc, &a.grad_weight_stride, &a.grad_expert_stride,
                   elem_bytes(a.grad_weight_dtype), &u[5].m));
    u[4].write = u[5].write = true;
    return HC_OK;
}

hc_status_t combine_sizes(size_t tokens, size_t top, size_t rows, size_t dim) {
    if (!top || !dim) return HC_ERR_INVALID_ARG;
    if (tokens > kMaxTokens / top || rows > kMaxTokens || dim > kMaxEmbeddingDim) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}

}  // namespace

extern "C" {

hc_status_t hc_embedding(const hc_embedding_t* args, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_embedding_t)) return HC_ERR_INVALID_ARG;
    hc_embedding_t a = *args;
    HC_TRY(check_float(a.table_dtype));
    HC_TRY(check_float(a.out_dtype));
    if (!known_id(a.id_type)) return HC_ERR_INVALID_ARG;
    HC_TRY(embedding_sizes(a.tokens, a.rows, a.dim));
    if (!std::isfinite(a.scale)) return HC_ERR_INVALID_ARG;  // would make NaN of the zero rows
    Use u[3] = {};
    u[2].write = true;
    if (a.tokens && (!a.table || !a.ids || !a.out)) return HC_ERR_INVALID_ARG;
    HC_TRY(matrix(a.table, a.rows, a.dim, &a.table_stride, elem_bytes(a.table_dtype), &u[0].m));
    HC_TRY(vector(a.ids, a.tokens, id_bytes(a.id_type), &u[1].m));
    HC_TRY(matrix(a.out, a.tokens, a.dim, &a.out_stride, elem_bytes(a.out_dtype), &u[2].m));
    HC_TRY(check_overlaps(u, 3));
    if (!a.tokens) return HC_OK;
    const TraceRange range("hc_embedding", 0, (uint64_t)a.tokens);
    return launch([&](int) { return launch_embedding(a, (cudaStream_t)stream); });
}

size_t hc_embedding_grad_scratch_bytes(const hc_embedding_grad_t* a) {
    if (!a || a->struct_size < sizeof(hc_embedding_grad_t)) return 0;
    if (embedding_sizes(a->tokens, a->rows, a->dim) != HC_OK) return 0;
    return embedding_scratch((int64_t)a->tokens, (int64_t)a->rows, (int64_t)a->dim).bytes;
}

hc_status_t hc_embedding_grad(const hc_embedding_grad_t* args, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_embedding_grad_t)) return HC_ERR_INVALID_ARG;
    hc_embedding_grad_t a = *args;
    HC_TRY(check_float(a.grad_out_dtype));
    HC_TRY(check_float(a.grad_table_dtype));
    if (!known_id(a.id_type) || (a.accumulate != 0 && a.accumulate != 1)) return HC_ERR_INVALID_ARG;
    HC_TRY(embedding_sizes(a.tokens, a.rows, a.dim));
    Use u[4] = {};
    u[2].write = u[3].write = true;
    if ((a.tokens && (!a.grad_out || !a.ids)) || !a.grad_table) return HC_ERR_INVALID_ARG;
    HC_TRY(matrix(a.grad_out, a.tokens, a.dim, &a.grad_out_stride, elem_bytes(a.grad_out_dtype), &u[0].m));
    HC_TRY(vector(a.ids, a.tokens, id_bytes(a.id_type), &u[1].m));
    HC_TRY(matrix(a.grad_table, a.rows, a.dim, &a.grad_table_stride, elem_bytes(a.grad_table_dtype), &u[2].m));
    const size_t need = hc_embedding_grad_scratch_bytes(&a);
    HC_TRY(check_scratch(a.scratch, a.scratch_bytes, need));
    if (need) HC_TRY(vector(a.scratch, need, 1, &u[3].m));
    HC_TRY(check_overlaps(u, 4));
    if (!a.tokens && a.accumulate) return HC_OK;
    const TraceRange range("hc_embedding_grad", 0, (uint64_t)a.tokens);
    return launch([&](int sms) { return launch_embedding_grad(a, (cudaStream_t)stream, sms); });
}

hc_status_t hc_block_norm(const hc_block_norm_t* args, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_block_norm_t)) return HC_ERR_INVALID_ARG;
    hc_block_norm_t a = *args;
    HC_TRY(check_float(a.dtype));
    HC_TRY(check_float(a.weight_dtype));
    HC_TRY(norm_sizes(a.tokens, a.dim, a.gate != nullptr, a.gate_rows));
    if (!(a.eps >= 0.0f) || !std::isfinite(a.eps)) return HC_ERR_INVALID_ARG;
    if (a.tokens && (!a.y || !a.x || !a.r)) return HC_ERR_INVALID_ARG;
    if (a.pre_rstd && !a.z) return HC_ERR_INVALID_ARG;
    const size_t es = elem_bytes(a.dtype), ws = elem_bytes(a.weight_dtype);
    Use u[9] = {};
    HC_TRY(matrix(a.y, a.tokens, a.dim, &a.y_stride, es, &u[0].m));
    HC_TRY(matrix(a.x, a.tokens, a.dim, &a.x_stride, es, &u[1].m));
    HC_TRY(vector(a.post_weight, a.dim, ws, &u[2].m));
    HC_TRY(vector(a.gate, a.gate ? a.dim * a.gate_rows : 0, ws, &u[3].m));
    HC_TRY(vector(a.pre_weight, a.dim, ws, &u[4].m));
    HC_TRY(matrix(a.r, a.tokens, a.dim, &a.r_stride, es, &u[5].m));
    HC_TRY(matrix(a.z, a.tokens, a.dim, &a.z_stride, es, &u[6].m));
    HC_TRY(vector(a.post_rstd, a.tokens, sizeof(float), &u[7].m));
    HC_TRY(vector(a.pre_rstd, a.tokens, sizeof(float), &u[8].m));
    for (int i = 5; i < 9; i++) u[i].write = true;
    u[0].in_place = u[1].in_place = u[5].in_place = u[6].in_place = true;
    HC_TRY(check_overlaps(u, 9));
    if (!a.tokens) return HC_OK;
    const TraceRange range("hc_block_norm", 0, (uint64_t)a.tokens);
    return launch([&](int sms) { return launch_block_norm(a, (cudaStream_t)stream, sms); });
}

size_t hc_block_norm_grad_scratch_bytes(const hc_block_norm_grad_t* a) {
    if (!a || a->struct_size < sizeof(hc_block_norm_grad_t)) return 0;
    // a gate that is NULL only because no pointer is known yet counts by its
    // rows, so one size serves calls with and without it; a call without a gate
    // does not look at them
    if (norm_sizes(a->tokens, a->dim, false, 0) != HC_OK) return 0;
    const size_t without = block_norm_plan((int64_t)a->tokens, (int64_t)a->dim, 1, false, false).bytes;
    const size_t rows = a->gate_rows ? a->gate_rows : 1;
    if (norm_sizes(a->tokens, a->dim, true, rows) != HC_OK) return without;
    const size_t with = block_norm_plan((int64_t)a->tokens, (int64_t)a->dim, (int64_t)rows, true, a->dtype == a->weight_dtype).bytes;
    return with > without ? with : without;
}

hc_status_t hc_block_norm_grad(const hc_block_norm_grad_t* args, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_block_norm_grad_t)) return HC_ERR_INVALID_ARG;
    hc_block_norm_grad_t a = *args;
    HC_TRY(check_float(a.dtype));
    HC_TRY(check_float(a.weight_dtype));
    HC_TRY(norm_sizes(a.tokens, a.dim, a.gate != nullptr, a.gate_rows));
    if (a.tokens && ((!a.grad_r && !a.grad_z) || !a.y || !a.x || !a.post_rstd || (a.grad_z && !a.pre_rstd) ||
                     !a.grad_y || !a.grad_x))
        return HC_ERR_INVALID_ARG;
    if (a.grad_gate && !a.gate) return HC_ERR_INVALID_ARG;
    const size_t es = elem_bytes(a.dtype), ws = elem_bytes(a.weight_dtype);
    Use u[15] = {};
    HC_TRY(matrix(a.grad_r, a.tokens, a.dim, &a.grad_r_stride, es, &u[0].m));
    HC_TRY(matrix(a.grad_z, a.tokens, a.dim, &a.grad_z_stride, es, &u[1].m));
    HC_TRY(matrix(a.y, a.tokens, a.dim, &a.y_stride, es, &u[2].m));
    HC_TRY(matrix(a.x, a.tokens, a.dim, &a.x_stride, es, &u[3].m));
    HC_TRY(vector(a.post_weight, a.dim, ws, &u[4].m));
    HC_TRY(vector(a.gate, a.gate ? a.dim * a.gate_rows : 0, ws, &u[5].m));
    HC_TRY(vector(a.pre_weight, a.dim, ws, &u[6].m));
    HC_TRY(vector(a.post_rstd, a.tokens, sizeof(float), &u[7].m));
    HC_TRY(vector(a.pre_rstd, a.tokens, sizeof(float), &u[8].m));
    HC_TRY(matrix(a.grad_y, a.tokens, a.dim, &a.grad_y_stride, es, &u[9].m));
    HC_TRY(matrix(a.grad_x, a.tokens, a.dim, &a.grad_x_stride, es, &u[10].m));
    HC_TRY(vector(a.grad_post_weight, a.dim, ws, &u[11].m));
    HC_TRY(vector(a.grad_gate, a.gate ? a.dim * a.gate_rows : 0, ws, &u[12].m));
    HC_TRY(vector(a.grad_pre_weight, a.dim, ws, &u[13].m));
    const size_t need =
        block_norm_plan((int64_t)a.tokens, (int64_t)a.dim, (int64_t)a.gate_rows, a.gate != nullptr,
                        a.dtype == a.weight_dtype).bytes;
    HC_TRY(check_scratch(a.scratch, a.scratch_bytes, need));
    if (need) HC_TRY(vector(a.scratch, need, 1, &u[14].m));
    for (int i = 9; i < 15; i++) u[i].write = true;
    for (int i = 0; i < 4; i++) u[i].in_place = true;
    u[9].in_place = u[10].in_place = true;
    HC_TRY(check_overlaps(u, 15));
    const TraceRange range("hc_block_norm_grad", 0, (uint64_t)a.tokens);
    return launch([&](int) { return launch_block_norm_grad(a, (cudaStream_t)stream); });
}

static hc_status_t distill(const hc_distill_t* args, bool grad_only, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_distill_t)) return HC_ERR_INVALID_ARG;
    hc_distill_t a = *args;
    HC_TRY(check_float(a.dtype));
    HC_TRY(check_float(a.teacher_dtype));
    if (!known_id(a.id_type) || !a.vocab || !a.top) return HC_ERR_INVALID_ARG;
    if (!(a.temperature > 0.0f) || !std::isfinite(a.temperature) || !std::isfinite(1.4426950408889634f / a.temperature) ||
        !std::isfinite(a.scale))
        return HC_ERR_INVALID_ARG;
    const size_t es = elem_bytes(a.dtype);
    if (a.top > kDistillMaxTop || a.vocab > kDistillMaxVocab || a.vocab * es > kDistillMaxRowBytes ||
        a.tokens > kMaxTokens)
        return HC_ERR_UNSUPPORTED;
    if (a.tokens && (!a.logits || !a.teacher_logits || !a.teacher_ids)) return HC_ERR_INVALID_ARG;
    if (a.tokens && (grad_only ? !a.stats || !a.grad_logits : !a.loss)) return HC_ERR_INVALID_ARG;
    Use u[7] = {};
    size_t ids_stride = a.teacher_stride;
    HC_TRY(matrix(a.logits, a.tokens, a.vocab, &a.logits_stride, es, &u[0].m));
    HC_TRY(matrix(a.teacher_logits, a.tokens, a.top, &a.teacher_stride, elem_bytes(a.teacher_dtype), &u[1].m));
    HC_TRY(matrix(a.teacher_ids, a.tokens, a.top, &ids_stride, id_bytes(a.id_type), &u[2].m));
    HC_TRY(vector(a.row_weight, a.tokens, sizeof(float), &u[3].m));
    HC_TRY(vector(a.stats, 2 * a.tokens, sizeof(float), &u[4].m));
    HC_TRY(vector(grad_only ? nullptr : a.loss, a.tokens, sizeof(float), &u[5].m));
    HC_TRY(matrix(a.grad_logits, a.tokens, a.vocab, &a.grad_stride, es, &u[6].m));
    u[4].write = !grad_only;
    u[5].write = u[6].write = true;
    u[0].in_place = u[6].in_place = true;
    HC_TRY(check_overlaps(u, 7));
    if (!a.tokens) return HC_OK;
    const TraceRange range(grad_only ? "hc_distill_grad" : "hc_distill", 0, (uint64_t)a.tokens);
    const DistillMode mode = grad_only ? DISTILL_GRAD : a.grad_logits ? DISTILL_BOTH : DISTILL_LOSS;
    return launch([&](int sms) { return launch_distill(a, mode, (cudaStream_t)stream, sms); });
}

hc_status_t hc_distill(const hc_distill_t* args, hc_stream_t stream) { return distill(args, false, stream); }
hc_status_t hc_distill_grad(const hc_distill_t* args, hc_stream_t stream) { return distill(args, true, stream); }

hc_status_t hc_clip_grads(const hc_clip_grads_t* args, hc_stream_t stream) { return clip(args, true, stream); }
hc_status_t hc_grad_norm(const hc_clip_grads_t* args, hc_stream_t stream) { return clip(args, false, stream); }
size_t hc_clip_grads_scratch_bytes(const hc_clip_grads_t* a) {
    if (!a || a->struct_size < sizeof(hc_clip_grads_t) || clip_tensors(*a, false) != HC_OK) return 0;
    return clip_scratch_bytes(*a);
}

static hc_status_t plan_sizes(const hc_expert_plan_t& a) {
    if (!a.top || !a.experts) return HC_ERR_INVALID_ARG;
    if (a.experts > kMaxExperts || a.top > kMaxTokens || a.tokens > kMaxTokens / a.top) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}
size_t hc_expert_plan_scratch_bytes(const hc_expert_plan_t* a) {
    if (!a || a->struct_size < sizeof(hc_expert_plan_t) || plan_sizes(*a) != HC_OK) return 0;
    return expert_plan_shape((int64_t)(a->tokens * a->top), (int64_t)a->experts).bytes;
}
hc_status_t hc_expert_plan(const hc_expert_plan_t* args, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_expert_plan_t)) return HC_ERR_INVALID_ARG;
    const hc_expert_plan_t a = *args;
    if (!known_id(a.id_type)) return HC_ERR_INVALID_ARG;
    HC_TRY(plan_sizes(a));
    const size_t n = a.tokens * a.top;
    if ((n && !a.expert_ids) || !a.offsets) return HC_ERR_INVALID_ARG;
    Use u[5] = {};
    HC_TRY(vector(a.expert_ids, n, id_bytes(a.id_type), &u[0].m));
    HC_TRY(vector(a.offsets, a.experts + 1, sizeof(int32_t), &u[1].m));
    HC_TRY(vector(a.row_tokens, n, sizeof(int32_t), &u[2].m));
    HC_TRY(vector(a.slots, n, sizeof(int32_t), &u[3].m));
    const size_t need = hc_expert_plan_scratch_bytes(&a);
    HC_TRY(check_scratch(a.scratch, a.scratch_bytes, need));
    if (need) HC_TRY(vector(a.scratch, need, 1, &u[4].m));
    for (int i = 1; i < 5; i++) u[i].write = true;
    HC_TRY(check_overlaps(u, 5));
    const TraceRange range("hc_expert_plan", 0, (uint64_t)a.tokens);
    return launch([&](int) { return launch_expert_plan(a, (cudaStream_t)stream); });
}

size_t hc_expert_matmul_scratch_bytes(const hc_expert_matmul_t* args) {
    if (!args || args->struct_size < sizeof(hc_expert_matmul_t)) return 0;
    hc_expert_matmul_t a = *args;
    Use u[4] = {};
    return matmul_operands(a, u) == HC_OK ? expert_matmul_scratch(a) : 0;
}
hc_status_t hc_expert_matmul(const hc_expert_matmul_t* args, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_expert_matmul_t)) return HC_ERR_INVALID_ARG;
    hc_expert_matmul_t a = *args;
    Use u[5] = {};
    HC_TRY(matmul_operands(a, u));
    if (a.rows && (!a.x || !a.weight || !a.offsets || !a.out)) return HC_ERR_INVALID_ARG;
    const size_t need = expert_matmul_scratch(a);
    HC_TRY(check_scratch(a.scratch, a.scratch_bytes, need));
    if (need) HC_TRY(vector(a.scratch, need, 1, &u[4].m));
    u[4].write = true;
    HC_TRY(check_overlaps(u, 5));
    if (!a.rows) return HC_OK;
    const TraceRange range("hc_expert_matmul", 0, (uint64_t)a.rows);
    return launch([&](int sms) { return launch_expert_matmul(a, (cudaStream_t)stream, sms); });
}

size_t hc_expert_matmul_grad_scratch_bytes(const hc_expert_matmul_grad_t* args) {
    if (!args || args->struct_size < sizeof(hc_expert_matmul_grad_t)) return 0;
    hc_expert_matmul_grad_t a = *args;
    Use u[6] = {};
    return matmul_grad_operands(a, u) == HC_OK ? expert_matmul_grad_scratch(a) : 0;
}
hc_status_t hc_expert_matmul_grad(const hc_expert_matmul_grad_t* args, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_expert_matmul_grad_t)) return HC_ERR_INVALID_ARG;
    hc_expert_matmul_grad_t a = *args;
    Use u[7] = {};
    HC_TRY(matmul_grad_operands(a, u));
    if ((!a.grad_x && !a.grad_weight && a.rows) || !a.offsets) return HC_ERR_INVALID_ARG;
    if (a.rows && (!a.grad_out || (a.grad_x && !a.weight) || (a.grad_weight && !a.x))) return HC_ERR_INVALID_ARG;
    const size_t need = expert_matmul_grad_scratch(a);
    HC_TRY(check_scratch(a.scratch, a.scratch_bytes, need));
    if (need) HC_TRY(vector(a.scratch, need, 1, &u[6].m));
    u[6].write = true;
    HC_TRY(check_overlaps(u, 7));
    if (!a.rows && (a.accumulate || !a.grad_weight)) return HC_OK;
    const TraceRange range("hc_expert_matmul_grad", 0, (uint64_t)a.rows);
    return launch([&](int sms) { return launch_expert_matmul_grad(a, (cudaStream_t)stream, sms); });
}

hc_status_t hc_expert_combine(const hc_expert_combine_t* args, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_expert_combine_t)) return HC_ERR_INVALID_ARG;
    hc_expert_combine_t a = *args;
    HC_TRY(check_float(a.dtype));
    if (a.weights) HC_TRY(check_float(a.weight_dtype));
    HC_TRY(combine_sizes(a.tokens, a.top, a.rows, a.dim));
    if (a.tokens && ((a.rows && !a.y) || !a.slots || !a.out)) return HC_ERR_INVALID_ARG;
    const size_t es = elem_bytes(a.dtype), n = a.tokens * a.top;
    Use u[4] = {};
    HC_TRY(matrix(a.y, a.rows, a.dim, &a.y_stride, es, &u[0].m));
    HC_TRY(vector(a.slots, n, sizeof(int32_t), &u[1].m));
    if (a.weights) HC_TRY(vector(a.weights, n, elem_bytes(a.weight_dtype), &u[2].m));
    HC_TRY(matrix(a.out, a.tokens, a.dim, &a.out_stride, es, &u[3].m));
    u[3].write = true;
    HC_TRY(check_overlaps(u, 4));
    if (!a.tokens) return HC_OK;
    const TraceRange range("hc_expert_combine", 0, (uint64_t)a.tokens);
    return launch([&](int sms) { return launch_expert_combine(a, (cudaStream_t)stream, sms); });
}

hc_status_t hc_expert_combine_grad(const hc_expert_combine_grad_t* args, hc_stream_t stream) {
    if (!args || args->struct_size < sizeof(hc_expert_combine_grad_t)) return HC_ERR_INVALID_ARG;
    hc_expert_combine_grad_t a = *args;
    HC_TRY(check_float(a.dtype));
    if (a.weights || a.grad_weights) HC_TRY(check_float(a.weight_dtype));
    HC_TRY(combine_sizes(a.tokens, a.top, a.rows, a.dim));
    if (a.tokens && (!a.grad_out || !a.slots || (!a.grad_y && !a.grad_weights) || (a.rows && a.grad_weights && !a.y)))
        return HC_ERR_INVALID_ARG;
    const size_t es = elem_bytes(a.dtype), n = a.tokens * a.top;
    Use u[6] = {};
    HC_TRY(matrix(a.grad_out, a.tokens, a.dim, &a.grad_out_stride, es, &u[0].m));
    HC_TRY(matrix(a.grad_weights ? a.y : nullptr, a.rows, a.dim, &a.y_stride, es, &u[1].m));
    HC_TRY(vector(a.slots, n, sizeof(int32_t), &u[2].m));
    if (a.weights) HC_TRY(vector(a.weights, n, elem_bytes(a.weight_dtype), &u[3].m));
    HC_TRY(matrix(a.grad_y, a.rows, a.dim, &a.grad_y_stride, es, &u[4].m));
    if (a.grad_weights) HC_TRY(vector(a.grad_weights, n, elem_bytes(a.weight_dtype), &u[5].m));
    u[4].write = u[5].write = true;
    u[1].in_place = u[4].in_place = true;
    HC_TRY(check_overlaps(u, 6));
    if (!a.tokens) return HC_OK;
    const TraceRange range("hc_expert_combine_grad", 0, (uint64_t)a.tokens);
    return launch([&](int sms) { return launch_expert_combine_grad(a, (cudaStream_t)stream, sms); });
}

}  // extern "C"
