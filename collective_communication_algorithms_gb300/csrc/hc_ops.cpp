// hc_ops.cpp -- the C ABI of the training operators (see include/hc.h):
// argument validation, strides, overlap checks and dispatch to the kernels.
#include <cmath>

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

}  // extern "C"
