// Internal interface of the paged key/value cache: the host side (tb_kv.cpp),
// the page kernels (tb_pages.cu) and the tree attention (tb_tree.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tb.h"
#include "tb_internal.h"

namespace tb {

// The cache as the kernels see it: tb_kv_cache after the host's checks, with
// the bytes of one (token, head) row and how the rows of a page join up.
struct KvView {
    char *pool[2];  // keys, values
    int32_t *table, *held, *lens, *refs;
    int32_t layers, pages, page_tokens, heads, row_bytes, slots, width;
    int64_t layer_stride, page_stride, token_stride, head_stride;
};

// Launchers of tb_pages.cu.  pdl: programmatic dependent launch.
cudaError_t launch_copy_pages(const KvView &c, const int32_t *src, const int32_t *dst,
                              const int32_t *tokens, int32_t n, bool pdl,
                              cudaStream_t stream);
cudaError_t launch_kv_resize(const KvView &c, const int32_t *capacity, int32_t *status, bool pdl,
                             cudaStream_t stream);
cudaError_t launch_kv_fork(const KvView &c, const int32_t *parents, int32_t *table_out,
                           int32_t *held_out, int32_t *lens_out, int32_t *status, bool pdl,
                           cudaStream_t stream);
cudaError_t launch_kv_compact(const KvView &c, const int32_t *start, const int32_t *keep,
                              int32_t keep_stride, const int32_t *count, int32_t *status,
                              bool pdl, cudaStream_t stream);

// One tree-attention launch, after the host's checks.
struct TreePlan {
    KvView c;  // pools moved to the layer
    bool bf16;
    int32_t head_dim, seqs, rows, q_heads, group, mask_words;
    const int32_t *seq_slots, *q_start;
    const char *q;
    char *out;
    int64_t q_row, q_head, o_row, o_head;  // strides in bytes
    float *lse;
    const uint32_t *mask;
    void *workspace;
    float scale;
    uint32_t *status;  // device-visible: 1 if a bounded wait expired
    uint64_t wait_ns;  // limit of each wait inside the kernel
};

uint64_t tree_workspace_bytes(int num_sms, int head_dim);
cudaError_t launch_tree(const TreePlan &p, int num_sms, bool pdl, cudaStream_t stream);

}  // namespace tb
