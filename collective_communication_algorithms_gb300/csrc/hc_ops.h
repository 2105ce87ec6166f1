// hc_ops.h -- launchers of the training operators, called by hc_ops.cpp on
// validated arguments (strides resolved, sizes in range).  Internal.
#pragma once

#include "hc_internal.h"

namespace hc {

cudaError_t launch_embedding(const hc_embedding_t& a, cudaStream_t stream);

// Tokens up to which the gradient of the lookup needs no sort (and no
// scratch), and the layout of its scratch above that.
constexpr size_t kEmbeddingFewTokens = 512;
struct EmbeddingScratch {
    size_t keys[2], pos[2], hist, cut, touched, part;  // byte offsets
    size_t bytes;
    int cluster;          // blocks of the one-cluster sort; 0: passes over global memory
    int chunk;            // tokens per sorting block
    int64_t chunks;
    int passes, bits;     // radix passes, bits of one pass's digit
    int sum_chunk;        // sorted tokens summed by one warp
    int64_t sum_chunks;   // groups of them
    int64_t pitch;        // floats in one row of partial sums
};
EmbeddingScratch embedding_scratch(int64_t tokens, int64_t rows, int64_t dim);
cudaError_t launch_embedding_grad(const hc_embedding_grad_t& a, cudaStream_t stream, int sms);

constexpr size_t kBlockNormMaxDim = 32768;
// How the threads of a block norm's kernels take their rows: one element an
// access, 16-byte vectors of 16-byte aligned rows, or the aligned vectors of
// memory that hold rows which all lie alike.
enum RowAccess { ROWS_ONE_BY_ONE, ROWS_VECTORS, ROWS_WINDOW };
// Shape of a launch: tx threads (or lanes) have a row, ty rows a block.
struct RowLayout {
    int tx, ty, cs;     // cs: blocks of a cluster
    int stages;         // 0: rows in a warp, loaded directly
    int slot;           // bytes of one row (slice) of one operand in a stage
    int weights;        // bytes of weights kept after the stages
    int* err;
    unsigned long long wait_ns;
    int hold;           // wait-expiry test mode
};
struct BlockNormRows {
    RowAccess access;
    int cols, ops;      // columns of a thread, operands of a stage
    RowLayout lay;      // without the fields that depend on the device
};
// vectors: every operand takes 16-byte accesses; alike: the inputs' rows lie
// alike in their 16-byte vectors; es: bytes of an element.
BlockNormRows block_norm_rows(int64_t dim, int es, bool vectors, bool alike);
cudaError_t launch_block_norm(const hc_block_norm_t& a, cudaStream_t stream, int sms);
// How the rows are divided among the blocks that sum weight gradients.
struct BlockNormPlan {
    int64_t blocks;      // blocks (clusters) = rows of partial sums
    int64_t unit;        // tokens (by_group 0) or groups (1) of one block
    int64_t per_group;   // by_group 0: blocks of one group
    int by_group;
    int each;            // 1: every token has a gate row, taken along with its other rows
    int direct;          // 1: one block, no partial sums
    int slots;           // partial sums kept by a block
    int64_t pitch;       // floats in one row of partial sums
    size_t bytes;
};
BlockNormPlan block_norm_plan(int64_t tokens, int64_t dim, int64_t gate_rows, bool gate, bool same_types);
// Windows divide the tokens by their rows' shift: they change unit, per_group and blocks.
BlockNormRows block_norm_grad_rows(BlockNormPlan* q, int64_t tokens, int64_t dim, int es, bool vectors, bool alike);
cudaError_t launch_block_norm_grad(const hc_block_norm_grad_t& a, cudaStream_t stream);

constexpr size_t kDistillMaxTop = 1024;
constexpr size_t kDistillMaxVocab = 1u << 20;
constexpr size_t kDistillMaxRowBytes = 3u << 19;
enum DistillMode { DISTILL_LOSS = 0, DISTILL_BOTH = 1, DISTILL_GRAD = 2 };
cudaError_t launch_distill(const hc_distill_t& a, DistillMode mode, cudaStream_t stream, int sms);

size_t clip_scratch_bytes(const hc_clip_grads_t& a);  // 0 also for lists that no launch takes
cudaError_t launch_clip(const hc_clip_grads_t& a, bool apply, cudaStream_t stream);

constexpr size_t kMaxExperts = 1024;
// How the plan's assignments are divided among blocks.
struct ExpertPlanShape {
    int64_t run;   // assignments of a block
    int blocks;    // 1: no scratch, no counting kernel
    size_t bytes;  // scratch
};
ExpertPlanShape expert_plan_shape(int64_t assignments, int64_t experts);
cudaError_t launch_expert_plan(const hc_expert_plan_t& a, cudaStream_t stream);
cudaError_t launch_expert_combine(const hc_expert_combine_t& a, cudaStream_t stream, int sms);
cudaError_t launch_expert_combine_grad(const hc_expert_combine_grad_t& a, cudaStream_t stream, int sms);

constexpr size_t kMaxExpertDim = 65536;
constexpr size_t kMaxExpertRows = 1u << 30;
size_t expert_matmul_scratch(const hc_expert_matmul_t& a);
size_t expert_matmul_grad_scratch(const hc_expert_matmul_grad_t& a);
cudaError_t launch_expert_matmul(const hc_expert_matmul_t& a, cudaStream_t stream, int sms);
cudaError_t launch_expert_matmul_grad(const hc_expert_matmul_grad_t& a, cudaStream_t stream, int sms);

// hc_api.cpp / hc_kernels.cu
hc_status_t cuda_status(cudaError_t e);
int sm_count_of_current_device();
int* device_error_flag();
bool allow_smem(void* fn, int bytes);
bool expiring_waits();  // hc_test_expire_waits is on

}  // namespace hc
