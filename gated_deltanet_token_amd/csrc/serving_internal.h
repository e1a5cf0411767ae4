// Internal launch interface between serving_api.hip and the kernel files of
// the attention layers' operators and the block norms.  Arguments arrive here
// already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

struct StepTablesArgs {
    const int32_t *context_lens;
    const int32_t *query_lens;
    const int32_t *free_pages;
    const int32_t *num_free;
    int32_t *block_table;
    int64_t block_table_stride;
    int32_t *query_start_loc;
    int32_t *seq_lens;
    int32_t *positions;
    int64_t *slot_mapping;
    gdn_conv_chunk *chunks;      // nullptr with n_chunks == 0
    int32_t *counts;
    int num_seqs;
    int free_capacity;
    int max_pages;
    int page_shift;              // log2 of page_size
    int num_tokens;
    int n_chunks;
};

struct RopeAppendArgs {
    const uint16_t *q;           // nullptr: no q
    const uint16_t *k;
    const uint16_t *v;
    uint16_t *q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const int32_t *positions;
    const int64_t *slots;
    const double *freq;
    uint8_t *k_cache;
    uint8_t *v_cache;
    float *k_scale;
    float *v_scale;
    double rope_scale;
    int rot;
    int interleaved;
    int num_pages;
    int page;
    int num_tokens;
    int num_q_heads;
    int num_kv_heads;
    int d;
};

struct AttentionArgs {
    const uint16_t *q;
    int64_t q_stride;
    const uint8_t *k_cache;
    const uint8_t *v_cache;
    const float *k_scale;
    const float *v_scale;
    const int32_t *block_table;
    int64_t block_table_stride;
    const int32_t *seq_lens;
    const int32_t *qsl;
    uint16_t *o;
    int64_t o_stride;
    float *workspace;
    int num_pages;
    int page;
    int max_pages;
    int max_seq_len;
    int num_seqs;
    int num_tokens;
    int num_q_heads;
    int num_kv_heads;
    int d;
    float scale;
    int causal;
    int window;
};

struct HeadNormArgs {
    const uint16_t *x;
    const uint16_t *gate;        // nullptr: none
    const uint16_t *weight;
    uint16_t *y;
    int64_t x_stride, gate_stride, y_stride;
    int num_tokens;
    int num_heads;
    int d;
    float eps;
    float offset;
};

struct ResidualNormArgs {
    const uint16_t *x;
    const uint16_t *residual;
    const uint16_t *post_weight; // nullptr: no norm after the block
    const uint16_t *gate;        // nullptr: none
    const uint16_t *weight;
    uint16_t *new_residual;
    uint16_t *y;
    int64_t x_stride, residual_stride, gate_stride, new_residual_stride, y_stride;
    int rows;
    int hidden;
    float residual_scale;
    float eps;
    float offset;
};

hipError_t launch_step_tables(const StepTablesArgs &a, hipStream_t stream);
hipError_t launch_rope_append(const RopeAppendArgs &a, hipStream_t stream);
int64_t attention_workspace_bytes(int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int d,
                                  int max_seq_len);
hipError_t launch_attention(const AttentionArgs &a, hipStream_t stream);
hipError_t launch_head_norm(const HeadNormArgs &a, hipStream_t stream);
hipError_t launch_residual_norm(const ResidualNormArgs &a, hipStream_t stream);

}  // namespace gdn
