// latent.h -- host-side launcher interfaces of the latent cache and of the
// step's page tables, between latent_api.cpp and the kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"

namespace pkv {

constexpr int kLatentDim = 512;                     // values, and keys but for the rotary part
constexpr int kLatentRope = 64;                     // rotary part of a key
constexpr int kLatentRow = kLatentDim + kLatentRope;
constexpr int kNopeDim = 128;                       // expanded form: per-head key part ...
constexpr int kExpandedQ = kNopeDim + kLatentRope;  // ... and the whole query or key
constexpr int kExpandedV = 128;

struct StepPagesArgs {
    const int32_t* new_lens;
    const int32_t* kv_lens;
    const int32_t* num_free;
    int32_t* free_pages;
    int64_t free_capacity;
    int32_t* block_table;
    int64_t block_table_stride;
    int batch, max_tokens;
    int32_t* kv_lens_out;
    int32_t* num_free_out;
    int32_t* q_indptr;
    int64_t* slots;
    int64_t* positions;
    int32_t* err;
};
cudaError_t launch_step_pages(const StepPagesArgs& a, cudaStream_t s);

struct LatentAppendArgs {
    const void* src;
    int64_t src_stride, num_tokens;
    const void* norm_weight;
    float eps;
    const int64_t* positions;
    const float* cos_sin;
    int64_t max_position;
    bool interleaved;
    const int64_t* slots;
    void* pool;
    int64_t num_pages, page_stride;
    const void* q_pe;
    int64_t q_pe_token_stride, q_pe_head_stride;
    void* q_out;
    int64_t q_out_token_stride, q_out_head_stride;
    int num_heads;
    bool checked;
    int32_t* err;
};
cudaError_t launch_append_latent(const LatentAppendArgs& a, cudaStream_t s);

// Absorbed attention.  A column is one (query row, head) pair of a sequence,
// row-major: column c is row c / heads, head c % heads.
struct LatentParams {
    const void* q;
    int64_t q_token_stride, q_head_stride;
    const void* pool;
    int64_t num_pages, page_stride;
    const int32_t* block_table;
    int64_t block_table_stride;
    const int32_t* kv_lens;
    const int32_t* q_indptr;
    const int32_t* q_real;
    int batch, max_q_rows, max_kv_len, heads;
    bool causal;
    float scale_log2;
    void* out;
    bool out_f32;
    float* lse;
    bool checked;
    int32_t* err;
};
struct LatentPlan {
    int cols, ctas;  // columns a CTA holds, CTAs of a worker (all on the same key tiles)
    int workers;     // one or a pair of CTAs each
    int groups;      // column groups (cols * ctas) of a sequence, at the host bounds
    bool whole;      // a worker for every group, which then has no states to join
    size_t ws_bytes;
};
LatentPlan plan_latent(int batch, int max_q_rows, int heads, int max_kv_len, int sms);
// What any call whose bounds are none above these needs at most: a smaller batch may take
// shares where this one's units all run at once, fewer columns may have more workers.
size_t latent_workspace_bytes(int batch, int max_q_rows, int heads, int max_kv_len, int sms);
// tmap: the pool as {576, 32, pages}, boxes of a page's 64 columns.  q_boxes: tmap_q holds
// the queries as {576, heads, rows} in boxes of 64 columns x pl.cols (row, head) pairs,
// which takes heads that divide pl.cols or are a multiple of it.
cudaError_t launch_latent_attn(const LatentParams& p, const LatentPlan& pl, void* workspace, const void* tmap,
                               const void* tmap_q, bool q_boxes, cudaStream_t s);

// Expanded attention over ragged K and V.
struct RaggedParams {
    const void* q;
    int64_t q_token_stride, q_head_stride;
    const void* k;
    int64_t k_token_stride, k_head_stride;
    const void* k_pe;
    int64_t k_pe_stride;
    const void* v;
    int64_t v_token_stride, v_head_stride;
    int64_t num_keys;
    const int32_t* q_indptr;
    const int32_t* kv_indptr;
    int batch, max_q_rows, max_kv_len, heads;
    bool causal;
    float scale_log2;
    void* out;
    bool out_f32;
    float* lse;
    bool checked;
    int32_t* err;
};
// Tensor maps: k and v as {128, heads, keys}, k_pe as {64, keys}; with q_boxes q as {192, heads, rows}.
cudaError_t launch_ragged_attn(const RaggedParams& p, const void* tmap_k, const void* tmap_pe, const void* tmap_v,
                               const void* tmap_q, bool q_boxes, cudaStream_t s);

// Generic kernels (one warp a query row and head): a slow cross-check.
cudaError_t launch_latent_simt(const LatentParams& p, cudaStream_t s);
cudaError_t launch_ragged_simt(const RaggedParams& p, cudaStream_t s);

}  // namespace pkv
