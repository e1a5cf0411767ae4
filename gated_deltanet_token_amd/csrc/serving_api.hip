// C-ABI entry points of the attention layers' operators and the block norms:
// host-side argument validation and kernel launches on the caller's stream.
// Every check runs before anything is enqueued; a failing call enqueues
// nothing.
#include <math.h>

#include "api_check.h"
#include "gdn.h"
#include "serving_internal.h"

using namespace gdn;

namespace {

Span array_span(const void *p, int64_t n, int64_t elem) { return row_span(p, 1, 0, n, elem); }

bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// Whether two strided row buffers of `rows` rows share an element.  Rows of
// one wider activation (equal strides) share none when their columns are
// disjoint, although their byte ranges interleave.
bool rows_overlap(const void *a, int64_t a_stride, int64_t a_cols, const void *b, int64_t b_stride, int64_t b_cols,
                  int64_t rows, int64_t elem) {
    if (!overlap(row_span(a, rows, a_stride, a_cols, elem), row_span(b, rows, b_stride, b_cols, elem))) return false;
    if (a_stride != b_stride || rows <= 1) return true;
    const int64_t pitch = a_stride * elem;
    int64_t d = ((int64_t)((uintptr_t)b - (uintptr_t)a)) % pitch;   // b's first column, seen from a's
    if (d < 0) d += pitch;
    return d < a_cols * elem || d + b_cols * elem > pitch;
}

bool same_rows(const void *a, int64_t a_stride, const void *b, int64_t b_stride) { return a == b && a_stride == b_stride; }

int check_cache(const uint8_t *k_cache, const uint8_t *v_cache, const float *k_scale, const float *v_scale,
                int32_t num_pages, int32_t page_size, int32_t num_kv_heads, int32_t head_dim) {
    if (!k_cache || !v_cache || !k_scale || !v_scale)
        return fail(GDN_ERR_INVALID, "k_cache, v_cache, k_scale and v_scale are required");
    if (num_pages < 1) return fail(GDN_ERR_INVALID, "num_pages must be >= 1");
    if (num_kv_heads < 1) return fail(GDN_ERR_INVALID, "num_kv_heads must be >= 1");
    if (page_size != 16 && page_size != 32 && page_size != 64)
        return fail(GDN_ERR_UNSUPPORTED, "page_size %d: supported 16, 32, 64", page_size);
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(GDN_ERR_UNSUPPORTED, "head_dim %d: supported 64, 128, 256", head_dim);
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return fail(GDN_ERR_UNSUPPORTED, "the caches must be 16-byte aligned, the scales 4-byte");
    return ok();
}

}  // namespace

GDN_EXPORT int gdn_build_step_tables(const int32_t *context_lens, const int32_t *query_lens, int32_t num_seqs,
                                     const int32_t *free_pages, const int32_t *num_free, int32_t free_capacity,
                                     int32_t *block_table, int64_t block_table_stride, int32_t max_pages,
                                     int32_t page_size, int32_t *query_start_loc, int32_t *seq_lens,
                                     int32_t *positions, int64_t *slot_mapping, int32_t num_tokens,
                                     gdn_conv_chunk *chunks, int32_t n_chunks, int32_t *counts, void *stream) {
    if (num_seqs < 0 || num_tokens < 0 || free_capacity < 0 || n_chunks < 0)
        return fail(GDN_ERR_INVALID, "negative num_seqs, num_tokens, free_capacity or n_chunks");
    if (!query_start_loc || !counts || !num_free)
        return fail(GDN_ERR_INVALID, "query_start_loc, counts and num_free are required");
    if (num_seqs > 0 && (!context_lens || !query_lens || !block_table || !seq_lens))
        return fail(GDN_ERR_INVALID, "context_lens, query_lens, block_table and seq_lens are required");
    if (num_tokens > 0 && (!positions || !slot_mapping))
        return fail(GDN_ERR_INVALID, "positions and slot_mapping are required");
    if (free_capacity > 0 && !free_pages) return fail(GDN_ERR_INVALID, "free_pages is required");
    if ((chunks == nullptr) != (n_chunks == 0))
        return fail(GDN_ERR_INVALID, "chunks and n_chunks must be given together");
    if (page_size < 1 || page_size > 1024 || (page_size & (page_size - 1)))
        return fail(GDN_ERR_INVALID, "page_size %d: must be a power of two from 1 to 1024", page_size);
    if (max_pages < 1 || block_table_stride < max_pages)
        return fail(GDN_ERR_INVALID, "max_pages must be >= 1 and at most block_table_stride");
    if (num_seqs > GDN_STEP_MAX_SEQS)
        return fail(GDN_ERR_UNSUPPORTED, "%d requests: at most %d in one call", num_seqs, GDN_STEP_MAX_SEQS);
    if (!aligned(context_lens, 4) || !aligned(query_lens, 4) || !aligned(free_pages, 4) || !aligned(num_free, 4) ||
        !aligned(block_table, 4) || !aligned(query_start_loc, 4) || !aligned(seq_lens, 4) || !aligned(positions, 4) ||
        !aligned(slot_mapping, 8) || !aligned(chunks, 8) || !aligned(counts, 4))
        return fail(GDN_ERR_UNSUPPORTED, "slot_mapping and chunks must be 8-byte aligned, the other arrays 4-byte");
    const Span in[] = {array_span(context_lens, num_seqs, 4), array_span(query_lens, num_seqs, 4),
                       array_span(free_pages, free_capacity, 4), array_span(num_free, 1, 4)};
    const Span out[] = {row_span(block_table, num_seqs, block_table_stride, max_pages, 4),
                        array_span(query_start_loc, (int64_t)num_seqs + 1, 4), array_span(seq_lens, num_seqs, 4),
                        array_span(positions, num_tokens, 4), array_span(slot_mapping, num_tokens, 8),
                        array_span(chunks, n_chunks, 8), array_span(counts, 4, 4)};
    const int n_out = (int)(sizeof out / sizeof out[0]);
    for (int i = 0; i < n_out; ++i) {
        for (const Span &r : in)
            if (overlap(out[i], r)) return fail(GDN_ERR_INVALID, "an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return fail(GDN_ERR_INVALID, "two outputs overlap");
    }
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    const StepTablesArgs a{context_lens, query_lens, free_pages, num_free, block_table, block_table_stride,
                           query_start_loc, seq_lens, positions, slot_mapping, chunks, counts, num_seqs,
                           free_capacity, max_pages, shift, num_tokens, n_chunks};
    return hip_status(launch_step_tables(a, (hipStream_t)stream), "step tables launch");
}

GDN_EXPORT int gdn_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor,
                                    double original_context, double beta_fast, double beta_slow, double *out,
                                    double *rope_scale) {
    if (!out || !rope_scale) return fail(GDN_ERR_INVALID, "out and rope_scale are required");
    if (rotary_dim < 2 || rotary_dim % 2) return fail(GDN_ERR_INVALID, "rotary_dim %d: must be even and >= 2", rotary_dim);
    if (!(base > 1.0) || !isfinite(base)) return fail(GDN_ERR_INVALID, "base must be above 1");
    if (scaling < GDN_ROPE_PLAIN || scaling > GDN_ROPE_YARN) return fail(GDN_ERR_INVALID, "scaling %d is none", scaling);
    if (scaling != GDN_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor)))
        return fail(GDN_ERR_INVALID, "factor must be at least 1");
    if (scaling == GDN_ROPE_NTK && rotary_dim == 2) return fail(GDN_ERR_INVALID, "the raised base needs rotary_dim > 2");
    if (scaling == GDN_ROPE_YARN && (!(original_context >= 1.0) || !isfinite(original_context) || !isfinite(beta_fast) ||
                                     !isfinite(beta_slow) || !(beta_fast > beta_slow)))
        return fail(GDN_ERR_INVALID, "original_context must be at least 1 and beta_fast above beta_slow");
    const double r = rotary_dim, two_pi = 6.283185307179586476925286766559;
    const double b = scaling == GDN_ROPE_NTK ? base * pow(factor, r / (r - 2.0)) : base;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(b, -2.0 * i / r);
        if (scaling == GDN_ROPE_LINEAR) f /= factor;
        if (scaling == GDN_ROPE_YARN) {
            const double turns = original_context * f / two_pi;
            const double keep = fmin(fmax((turns - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0);
            f = f * keep + f / factor * (1.0 - keep);
        }
        out[i] = f;
    }
    *rope_scale = scaling == GDN_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
    return ok();
}

GDN_EXPORT int gdn_rope_append_kv8(const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k, int64_t k_stride,
                                   const gdn_bf16 *v, int64_t v_stride, const int32_t *positions,
                                   const int64_t *slot_mapping, const double *frequencies, int32_t rotary_dim,
                                   int32_t interleaved, double rope_scale, gdn_bf16 *q_out, int64_t q_out_stride,
                                   uint8_t *k_cache, uint8_t *v_cache, float *k_scale, float *v_scale,
                                   int32_t num_pages, int32_t page_size, int32_t num_tokens, int32_t num_q_heads,
                                   int32_t num_kv_heads, int32_t head_dim, void *stream) {
    if (num_tokens < 0) return fail(GDN_ERR_INVALID, "negative num_tokens");
    if (num_tokens == 0) return ok();
    if (!k || !v || !positions || !slot_mapping)
        return fail(GDN_ERR_INVALID, "k, v, positions and slot_mapping are required");
    if ((q == nullptr) != (q_out == nullptr)) return fail(GDN_ERR_INVALID, "q and q_out must be given together");
    if (q && num_q_heads < 1) return fail(GDN_ERR_INVALID, "num_q_heads must be >= 1");
    int rc = check_cache(k_cache, v_cache, k_scale, v_scale, num_pages, page_size, num_kv_heads, head_dim);
    if (rc) return rc;
    if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16)
        return fail(GDN_ERR_UNSUPPORTED, "rotary_dim %d: must be a multiple of 16 from 0 to head_dim", rotary_dim);
    if (rotary_dim > 0 && !frequencies) return fail(GDN_ERR_INVALID, "frequencies is required");
    const int64_t qw = q ? (int64_t)num_q_heads * head_dim : 0, kw = (int64_t)num_kv_heads * head_dim;
    if (k_stride < kw || v_stride < kw || (q && (q_stride < qw || q_out_stride < qw)))
        return fail(GDN_ERR_INVALID, "a token stride is smaller than its row of heads");
    if (k_stride % 8 || v_stride % 8 || (q && (q_stride % 8 || q_out_stride % 8)))
        return fail(GDN_ERR_UNSUPPORTED, "token strides must be multiples of 8 elements");
    // the kernel addresses a page's rows with 32-bit byte offsets
    if (k_stride >= (1 << 24) || v_stride >= (1 << 24))
        return fail(GDN_ERR_UNSUPPORTED, "k's and v's token strides must be below 2^24 elements");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out))
        return fail(GDN_ERR_UNSUPPORTED, "q, k, v and q_out must be 16-byte aligned");
    if (!aligned(positions, 4) || !aligned(slot_mapping, 8) || !aligned(frequencies, 8))
        return fail(GDN_ERR_UNSUPPORTED, "positions must be 4-byte aligned, slot_mapping and frequencies 8-byte");
    if (q && ((rows_overlap(q_out, q_out_stride, qw, q, q_stride, qw, num_tokens, 2) &&
               !same_rows(q_out, q_out_stride, q, q_stride)) ||
              rows_overlap(q_out, q_out_stride, qw, k, k_stride, kw, num_tokens, 2) ||
              rows_overlap(q_out, q_out_stride, qw, v, v_stride, kw, num_tokens, 2)))
        return fail(GDN_ERR_INVALID, "q_out overlaps q, k or v");
    const int64_t heads = (int64_t)num_pages * num_kv_heads, codes = heads * page_size * head_dim;
    const Span out[] = {array_span(k_cache, codes, 1), array_span(v_cache, codes, 1), array_span(k_scale, heads, 4),
                        array_span(v_scale, heads, 4), row_span(q_out, q ? num_tokens : 0, q_out_stride, qw, 2)};
    const Span in[] = {row_span(k, num_tokens, k_stride, kw, 2), row_span(v, num_tokens, v_stride, kw, 2),
                       row_span(q, q ? num_tokens : 0, q_stride, qw, 2), array_span(positions, num_tokens, 4),
                       array_span(slot_mapping, num_tokens, 8), array_span(frequencies, rotary_dim / 2, 8)};
    for (int i = 0; i < 5; ++i) {
        for (int j = i == 4 ? 3 : 0; j < 6; ++j)      // q_out against q, k and v: above
            if (overlap(out[i], in[j])) return fail(GDN_ERR_INVALID, "an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return fail(GDN_ERR_INVALID, "two outputs overlap");
    }
    const RopeAppendArgs a{q, k, v, q_out, q_stride, k_stride, v_stride, q_out_stride, positions, slot_mapping,
                           frequencies, k_cache, v_cache, k_scale, v_scale, rope_scale, rotary_dim, interleaved != 0,
                           num_pages, page_size, num_tokens, q ? num_q_heads : 0, num_kv_heads, head_dim};
    return hip_status(launch_rope_append(a, (hipStream_t)stream), "rope append launch");
}

GDN_EXPORT size_t gdn_paged_attention_kv8_workspace_size(int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                                                         int32_t num_kv_heads, int32_t head_dim, int32_t max_seq_len) {
    if (num_tokens <= 0 || num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        head_dim <= 0 || max_seq_len <= 0)
        return 0;
    return (size_t)attention_workspace_bytes(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, max_seq_len);
}

GDN_EXPORT int gdn_paged_attention_kv8(const gdn_bf16 *q, int64_t q_stride, const uint8_t *k_cache,
                                       const uint8_t *v_cache, const float *k_scale, const float *v_scale,
                                       int32_t num_pages, int32_t page_size, const int32_t *block_table,
                                       int64_t block_table_stride, int32_t max_pages, const int32_t *seq_lens,
                                       const int32_t *query_start_loc, int32_t max_seq_len, gdn_bf16 *o,
                                       int64_t o_stride, int32_t num_seqs, int32_t num_tokens, int32_t num_q_heads,
                                       int32_t num_kv_heads, int32_t head_dim, float scale, int32_t causal,
                                       int32_t window, void *workspace, size_t workspace_bytes, void *stream) {
    if (num_seqs < 0 || num_tokens < 0) return fail(GDN_ERR_INVALID, "negative num_seqs or num_tokens");
    if (num_seqs == 0 || num_tokens == 0) return ok();
    if (!q || !o || !block_table || !seq_lens || !query_start_loc)
        return fail(GDN_ERR_INVALID, "q, o, block_table, seq_lens and query_start_loc are required");
    int rc = check_cache(k_cache, v_cache, k_scale, v_scale, num_pages, page_size, num_kv_heads, head_dim);
    if (rc) return rc;
    if (num_q_heads < 1 || num_q_heads % num_kv_heads)
        return fail(GDN_ERR_INVALID, "num_q_heads must be a positive multiple of num_kv_heads");
    // offsets within a page are 32-bit where prompts are read
    if ((int64_t)num_kv_heads * page_size * head_dim > 0x7fffffff)
        return fail(GDN_ERR_UNSUPPORTED, "a page of %d heads x %d tokens x %d elements passes 2^31 - 1 bytes", num_kv_heads, page_size,
                    head_dim);
    if (max_pages < 1 || block_table_stride < max_pages)
        return fail(GDN_ERR_INVALID, "max_pages must be >= 1 and at most block_table_stride");
    if (max_pages > (0x7fffffff - 1024) / page_size)     // key numbers, a few tiles past the end too, are 32-bit
        return fail(GDN_ERR_UNSUPPORTED, "a row of %d pages of %d tokens passes 2^31 - 1024 tokens", max_pages, page_size);
    if (max_seq_len < 1) return fail(GDN_ERR_INVALID, "max_seq_len must be >= 1");
    if (window < 0) return fail(GDN_ERR_INVALID, "negative window");
    const int64_t w = (int64_t)num_q_heads * head_dim;
    if (q_stride < w || o_stride < w) return fail(GDN_ERR_INVALID, "a token stride is smaller than its row of heads");
    if (q_stride % 8 || o_stride % 8) return fail(GDN_ERR_UNSUPPORTED, "token strides must be multiples of 8 elements");
    if (!aligned16(q) || !aligned16(o)) return fail(GDN_ERR_UNSUPPORTED, "q and o must be 16-byte aligned");
    if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4))
        return fail(GDN_ERR_UNSUPPORTED, "block_table, seq_lens and query_start_loc must be 4-byte aligned");
    const size_t need = gdn_paged_attention_kv8_workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads,
                                                               head_dim, max_seq_len);
    if (need > 0) {
        if (!workspace) return fail(GDN_ERR_INVALID, "workspace is required (%zu bytes)", need);
        if (!aligned(workspace, 256)) return fail(GDN_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
        if (workspace_bytes < need)
            return fail(GDN_ERR_CAPACITY, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    }
    const int64_t heads = (int64_t)num_pages * num_kv_heads, codes = heads * page_size * head_dim;
    const Span os = row_span(o, num_tokens, o_stride, w, 2), ws = array_span(workspace, (int64_t)need, 1);
    const Span in[] = {array_span(k_cache, codes, 1), array_span(v_cache, codes, 1), array_span(k_scale, heads, 4),
                       array_span(v_scale, heads, 4), row_span(block_table, num_seqs, block_table_stride, max_pages, 4),
                       array_span(seq_lens, num_seqs, 4), array_span(query_start_loc, (int64_t)num_seqs + 1, 4),
                       row_span(q, num_tokens, q_stride, w, 2)};
    for (const Span &r : in)
        if (overlap(ws, r)) return fail(GDN_ERR_INVALID, "the workspace overlaps an operand");
    for (int i = 0; i < 7; ++i)
        if (overlap(os, in[i])) return fail(GDN_ERR_INVALID, "o overlaps an operand");
    if (rows_overlap(o, o_stride, w, q, q_stride, w, num_tokens, 2)) return fail(GDN_ERR_INVALID, "o overlaps q");
    if (overlap(ws, os)) return fail(GDN_ERR_INVALID, "the workspace overlaps o");
    const AttentionArgs a{q, q_stride, k_cache, v_cache, k_scale, v_scale, block_table, block_table_stride, seq_lens,
                          query_start_loc, o, o_stride, (float *)workspace, num_pages, page_size, max_pages,
                          max_seq_len, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, scale, causal != 0,
                          window};
    return hip_status(launch_attention(a, (hipStream_t)stream), "paged attention launch");
}

GDN_EXPORT int gdn_gated_rms_norm(const gdn_bf16 *x, int64_t x_stride, const gdn_bf16 *gate, int64_t gate_stride,
                                  const gdn_bf16 *weight, gdn_bf16 *y, int64_t y_stride, int32_t num_tokens,
                                  int32_t num_heads, int32_t head_dim, float eps, float weight_offset, void *stream) {
    if (num_tokens < 0 || num_heads < 1) return fail(GDN_ERR_INVALID, "negative num_tokens or num_heads < 1");
    if (num_tokens == 0) return ok();
    if (!x || !weight || !y) return fail(GDN_ERR_INVALID, "x, weight and y are required");
    if (head_dim < 8 || head_dim % 8 || head_dim > 512)
        return fail(GDN_ERR_UNSUPPORTED, "head_dim %d: must be a multiple of 8 up to 512", head_dim);
    const int64_t w = (int64_t)num_heads * head_dim;
    if (x_stride < w || y_stride < w || (gate && gate_stride < w))
        return fail(GDN_ERR_INVALID, "a token stride is smaller than its row of heads");
    if (x_stride % 8 || y_stride % 8 || (gate && gate_stride % 8))
        return fail(GDN_ERR_UNSUPPORTED, "token strides must be multiples of 8 elements");
    if (!aligned16(x) || !aligned16(gate) || !aligned16(weight) || !aligned16(y))
        return fail(GDN_ERR_UNSUPPORTED, "x, gate, weight and y must be 16-byte aligned");
    if ((rows_overlap(y, y_stride, w, x, x_stride, w, num_tokens, 2) && !same_rows(y, y_stride, x, x_stride)) ||
        (gate && rows_overlap(y, y_stride, w, gate, gate_stride, w, num_tokens, 2)) ||
        overlap(row_span(y, num_tokens, y_stride, w, 2), array_span(weight, head_dim, 2)))
        return fail(GDN_ERR_INVALID, "y overlaps x (other than in place), gate or weight");
    const HeadNormArgs a{x, gate, weight, y, x_stride, gate_stride, y_stride, num_tokens, num_heads, head_dim, eps,
                         weight_offset};
    return hip_status(launch_head_norm(a, (hipStream_t)stream), "gated norm launch");
}

GDN_EXPORT int gdn_residual_rms_norm(const gdn_bf16 *x, int64_t x_stride, const gdn_bf16 *residual,
                                     int64_t residual_stride, const gdn_bf16 *post_weight, const gdn_bf16 *gate,
                                     int64_t gate_stride, const gdn_bf16 *weight, gdn_bf16 *new_residual,
                                     int64_t new_residual_stride, gdn_bf16 *y, int64_t y_stride, int32_t rows,
                                     int32_t hidden, float residual_scale, float eps, float weight_offset,
                                     void *stream) {
    if (rows < 0) return fail(GDN_ERR_INVALID, "negative rows");
    if (rows == 0) return ok();
    if (!x || !residual || !weight || !new_residual || !y)
        return fail(GDN_ERR_INVALID, "x, residual, weight, new_residual and y are required");
    if (hidden < 8 || hidden % 8 || hidden > 16384)
        return fail(GDN_ERR_UNSUPPORTED, "hidden %d: must be a multiple of 8 up to 16384", hidden);
    if (x_stride < hidden || residual_stride < hidden || new_residual_stride < hidden || y_stride < hidden ||
        (gate && gate_stride < hidden))
        return fail(GDN_ERR_INVALID, "a row stride is smaller than hidden");
    if (x_stride % 8 || residual_stride % 8 || new_residual_stride % 8 || y_stride % 8 || (gate && gate_stride % 8))
        return fail(GDN_ERR_UNSUPPORTED, "row strides must be multiples of 8 elements");
    if (!aligned16(x) || !aligned16(residual) || !aligned16(post_weight) || !aligned16(gate) || !aligned16(weight) ||
        !aligned16(new_residual) || !aligned16(y))
        return fail(GDN_ERR_UNSUPPORTED, "every operand must be 16-byte aligned");
    struct Rows {
        const void *p;
        int64_t stride;
    };
    const Rows xr{x, x_stride}, rr{residual, residual_stride}, gr{gate, gate_stride};
    const Rows nr{new_residual, new_residual_stride}, yr{y, y_stride};
    auto clash = [&](const Rows &o, const Rows &i, bool in_place) {
        return i.p && rows_overlap(o.p, o.stride, hidden, i.p, i.stride, hidden, rows, 2) &&
               !(in_place && same_rows(o.p, o.stride, i.p, i.stride));
    };
    const Span ns = row_span(new_residual, rows, new_residual_stride, hidden, 2);
    const Span ys = row_span(y, rows, y_stride, hidden, 2);
    const Span ws = array_span(weight, hidden, 2), ps = array_span(post_weight, post_weight ? hidden : 0, 2);
    if (clash(nr, xr, true) || clash(nr, rr, true) || clash(nr, gr, false) || clash(yr, xr, true) ||
        clash(yr, rr, false) || clash(yr, gr, false) || clash(yr, nr, false) || overlap(ns, ws) || overlap(ns, ps) ||
        overlap(ys, ws) || overlap(ys, ps))
        return fail(GDN_ERR_INVALID, "an output overlaps an operand (other than in place) or the other output");
    const ResidualNormArgs a{x, residual, post_weight, gate, weight, new_residual, y, x_stride, residual_stride,
                             gate_stride, new_residual_stride, y_stride, rows, hidden, residual_scale, eps,
                             weight_offset};
    return hip_status(launch_residual_norm(a, (hipStream_t)stream), "residual norm launch");
}
