// latent_api.cpp -- C entry points of the latent cache and of the step's page
// tables: argument checks, kernel choice, TMA tensor maps.  Nothing here
// touches device memory; every check runs before anything is enqueued.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "latent.h"
#include "pkv.h"
#include "pkv_internal.h"

namespace {

pkv_status fail(pkv_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
pkv_status fail(pkv_status st, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return pkv::report(st, buf);
}
pkv_status ok() { return pkv::report(PKV_OK, ""); }
pkv_status from_cuda(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return ok();
    return fail(PKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
// a stride of whole 16 bytes of bf16
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

constexpr int64_t kMaxCount = (int64_t(1) << 31) - 256;
constexpr int64_t kMaxStride = (int64_t(1) << 39) / 2 - 8;  // elements: tensor maps hold strides below 2^40 bytes

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A bf16 tensor, 128-byte swizzled boxes of 64 columns; strides in elements, outermost last.
pkv_status make_map(CUtensorMap* m, const void* base, int rank, const int64_t* dims, const int64_t* strides,
                    const int* box) {
    auto fn = encode_fn();
    if (!fn) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    cuuint64_t d[4], st[3];
    cuuint32_t bx[4], es[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = static_cast<cuuint64_t>(dims[i]);
        bx[i] = static_cast<cuuint32_t>(box[i]);
        if (i > 0) st[i - 1] = static_cast<cuuint64_t>(strides[i - 1]) * 2;
    }
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, st, bx, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed: %d", static_cast<int>(r));
    return PKV_OK;
}

// Whether rows of `width` elements at i * a_stride + j * b_stride (i < na, j < nb) are
// apart: one axis' rows lie within a step of the other's, as slices of a tensor and
// transposed ones do.
bool rows_apart(int64_t na, int64_t a_stride, int64_t nb, int64_t b_stride, int64_t width) {
    if (na > 1 && nb > 1 && a_stride < b_stride) return rows_apart(nb, b_stride, na, a_stride, width);
    const __int128 inner = nb > 1 ? static_cast<__int128>(nb - 1) * b_stride + width : width;
    return (nb <= 1 || b_stride >= width) && (na <= 1 || a_stride >= inner);
}

// SM count of the current device (152 where none can be queried), as the workspace sizes of paged_attention
int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
        cudaGetLastError();
        return 152;
    }
    return sms;
}

// What paged_attention_latent counts in 32 bits: columns of a sequence, column
// groups of the call, and a worker's share of the key tiles.
bool counts_ok(int batch, int max_q_rows, int num_heads, int max_kv_len) {
    if (max_kv_len > kMaxCount || max_q_rows > kMaxCount / num_heads || batch > 65535) return false;
    const int64_t groups = static_cast<int64_t>(batch) * ((static_cast<int64_t>(max_q_rows) * num_heads + 15) / 16);
    return groups <= kMaxCount && groups * (max_kv_len / 64 + 8) <= (int64_t(1) << 36);
}

bool dims_ok(int latent_dim, int rope_dim) {
    return latent_dim == pkv::kLatentDim && rope_dim == pkv::kLatentRope;
}

}  // namespace

extern "C" {

pkv_status assign_step_pages(const int32_t* new_lens, const int32_t* kv_lens, const int32_t* num_free,
                             int32_t* free_pages, int64_t free_capacity, int32_t* block_table,
                             int64_t block_table_stride, int batch, int max_tokens, int page_size,
                             int32_t* kv_lens_out, int32_t* num_free_out, int32_t* q_indptr, int64_t* slots,
                             int64_t* positions, int32_t* err, void* stream) {
    if (batch < 0 || max_tokens < 0 || free_capacity < 0 || block_table_stride < 0)
        return fail(PKV_ERR_INVALID_ARG, "step pages: negative size");
    if (batch == 0) return ok();
    if (!new_lens || !kv_lens || !num_free || !kv_lens_out || !num_free_out || !q_indptr)
        return fail(PKV_ERR_INVALID_ARG, "step pages: null pointer");
    if ((max_tokens > 0 && (!slots || !positions)) || (free_capacity > 0 && !free_pages) ||
        (block_table_stride > 0 && !block_table))
        return fail(PKV_ERR_INVALID_ARG, "step pages: null pointer");
    if (page_size != 32) return fail(PKV_ERR_UNSUPPORTED, "step pages: page_size %d (only 32-token pages)", page_size);
    if (batch > 4096) return fail(PKV_ERR_UNSUPPORTED, "step pages: batch %d (at most 4096)", batch);
    if (max_tokens > (1 << 30)) return fail(PKV_ERR_UNSUPPORTED, "step pages: max_tokens above 2^30");
    if (free_capacity > kMaxCount || block_table_stride > kMaxCount / 32)
        return fail(PKV_ERR_UNSUPPORTED, "step pages: more pages than 32 bits of slots count");
    if (!aligned(new_lens, 4) || !aligned(kv_lens, 4) || !aligned(num_free, 4) || !aligned(free_pages, 4) ||
        !aligned(block_table, 4) || !aligned(kv_lens_out, 4) || !aligned(num_free_out, 4) || !aligned(q_indptr, 4) ||
        !aligned(slots, 8) || !aligned(positions, 8))
        return fail(PKV_ERR_INVALID_ARG, "step pages: misaligned pointer");
    const pkv::StepPagesArgs a{new_lens,    kv_lens,      num_free, free_pages, free_capacity, block_table, block_table_stride,
                               batch,       max_tokens,   kv_lens_out, num_free_out, q_indptr, slots,       positions,
                               err};
    return from_cuda(pkv::launch_step_pages(a, static_cast<cudaStream_t>(stream)), "step pages");
}

pkv_status kv_append_latent(const void* src, int64_t src_stride, int64_t num_tokens, const void* norm_weight, float eps,
                            const int64_t* positions, const float* cos_sin, int64_t max_position, int interleaved,
                            const int64_t* slots, void* pool, int64_t num_pages, int page_size, int64_t page_stride,
                            int latent_dim, int rope_dim, const void* q_pe, int64_t q_pe_token_stride,
                            int64_t q_pe_head_stride, void* q_out, int64_t q_out_token_stride,
                            int64_t q_out_head_stride, int num_heads, unsigned flags, int32_t* err, void* stream) {
    if (num_tokens < 0 || max_position < 0 || num_pages < 0 || num_heads < 0)
        return fail(PKV_ERR_INVALID_ARG, "latent append: negative size");
    if (num_tokens == 0) return ok();
    if (!dims_ok(latent_dim, rope_dim))
        return fail(PKV_ERR_UNSUPPORTED, "latent append: rows of %d + %d (only 512 + 64)", latent_dim, rope_dim);
    if (page_size != 32)
        return fail(PKV_ERR_UNSUPPORTED, "latent append: page_size %d (only 32-token pages)", page_size);
    if (!src || !positions || !cos_sin || !slots || !pool || (num_heads > 0 && (!q_pe || !q_out)))
        return fail(PKV_ERR_INVALID_ARG, "latent append: null pointer");
    if (max_position == 0) return fail(PKV_ERR_INVALID_ARG, "latent append: empty cos/sin table");
    if (!(eps >= 0.f) || std::isinf(eps)) return fail(PKV_ERR_INVALID_ARG, "latent append: eps must be finite and >= 0");
    if (page_stride < 32 * pkv::kLatentRow || page_stride % 8)
        return fail(PKV_ERR_INVALID_ARG, "latent append: page_stride must cover a page, a multiple of 8");
    if (num_heads > 65535 || num_tokens > kMaxCount || (num_heads > 0 && num_tokens > kMaxCount / num_heads))
        return fail(PKV_ERR_UNSUPPORTED, "latent append: more than 65535 heads or 2^31 rows");
    if (!aligned(src, 16) || !aligned(pool, 16) || !aligned(cos_sin, 16) || !aligned(norm_weight, 16) ||
        !aligned(positions, 8) || !aligned(slots, 8) || !stride_ok(src_stride))
        return fail(PKV_ERR_INVALID_ARG, "latent append: 16-byte aligned pointers and strides multiple of 8");
    if (num_heads > 0 && (!aligned(q_pe, 16) || !aligned(q_out, 16) || !stride_ok(q_pe_token_stride) ||
                          !stride_ok(q_pe_head_stride) || !stride_ok(q_out_token_stride) || !stride_ok(q_out_head_stride)))
        return fail(PKV_ERR_INVALID_ARG, "latent append: 16-byte aligned queries and strides multiple of 8");
    if (num_heads > 0 && !rows_apart(num_tokens, q_out_token_stride, num_heads, q_out_head_stride, rope_dim))
        return fail(PKV_ERR_INVALID_ARG, "latent append: rows of q_out overlap");
    if (num_heads > 0 && q_pe == q_out &&
        ((num_tokens > 1 && q_pe_token_stride != q_out_token_stride) || (num_heads > 1 && q_pe_head_stride != q_out_head_stride)))
        return fail(PKV_ERR_INVALID_ARG, "latent append: queries rotated in place need equal strides");
    if ((flags & PKV_FLAG_CHECKED) && !err)
        return fail(PKV_ERR_INVALID_ARG, "latent append: checked mode needs an error flag");
    const pkv::LatentAppendArgs a{src, src_stride, num_tokens, norm_weight, eps, positions, cos_sin, max_position,
                                  interleaved != 0, slots, pool, num_pages, page_stride, q_pe, q_pe_token_stride,
                                  q_pe_head_stride, q_out, q_out_token_stride, q_out_head_stride, num_heads,
                                  (flags & PKV_FLAG_CHECKED) != 0, err};
    return from_cuda(pkv::launch_append_latent(a, static_cast<cudaStream_t>(stream)), "latent append");
}

size_t paged_attention_latent_workspace_size(int batch, int max_q_rows, int num_heads, int max_kv_len, int latent_dim,
                                             int rope_dim, unsigned flags) {
    if (batch <= 0 || max_q_rows <= 0 || num_heads <= 0 || max_kv_len < 0 || !dims_ok(latent_dim, rope_dim) ||
        (flags & PKV_FLAG_SIMT_ONLY) || !counts_ok(batch, max_q_rows, num_heads, max_kv_len))
        return 0;
    return pkv::latent_workspace_bytes(batch, max_q_rows, num_heads, max_kv_len, device_sms());
}

pkv_status paged_attention_latent(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* pool,
                                  int64_t num_pages, int page_size, int64_t page_stride, const int32_t* block_table,
                                  int64_t block_table_stride, const int32_t* kv_lens, const int32_t* q_indptr,
                                  const int32_t* q_real, int batch, int max_q_rows, int max_kv_len, int num_heads,
                                  int latent_dim, int rope_dim, pkv_mask mask, float scale, void* out,
                                  pkv_dtype out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                                  unsigned flags, int32_t* err, void* stream) {
    if (batch < 0 || max_q_rows < 0 || max_kv_len < 0 || num_heads < 0 || num_pages < 0)
        return fail(PKV_ERR_INVALID_ARG, "latent attention: negative size");
    if (batch == 0 || max_q_rows == 0 || num_heads == 0) return ok();
    if (!dims_ok(latent_dim, rope_dim))
        return fail(PKV_ERR_UNSUPPORTED, "latent attention: rows of %d + %d (only 512 + 64)", latent_dim, rope_dim);
    if (page_size != 32)
        return fail(PKV_ERR_UNSUPPORTED, "latent attention: page_size %d (only 32-token pages)", page_size);
    if (!q || (max_kv_len > 0 && (!pool || !block_table)) || !kv_lens || !q_indptr || !out)
        return fail(PKV_ERR_INVALID_ARG, "latent attention: null pointer");
    if (mask == PKV_MASK_BLOCK_CAUSAL) return fail(PKV_ERR_UNSUPPORTED, "latent attention: no block-causal mask");
    if (mask != PKV_MASK_NONE && mask != PKV_MASK_CAUSAL)
        return fail(PKV_ERR_INVALID_ARG, "latent attention: unknown mask %d", static_cast<int>(mask));
    if (out_dtype != PKV_BF16 && out_dtype != PKV_F32)
        return fail(PKV_ERR_UNSUPPORTED, "latent attention: output dtype must be bf16 or f32");
    if (!(scale > 0.f) || std::isinf(scale))
        return fail(PKV_ERR_INVALID_ARG, "latent attention: scale must be finite and > 0");
    if (num_pages > kMaxCount || !counts_ok(batch, max_q_rows, num_heads, max_kv_len))
        return fail(PKV_ERR_UNSUPPORTED, "latent attention: sizes above 2^31 - 256, or 2^36 tiles of 16 columns and 64 keys");
    if (max_kv_len > 0 && num_pages == 0) return fail(PKV_ERR_INVALID_ARG, "latent attention: a pool without pages");
    if (page_stride < 32 * pkv::kLatentRow || page_stride % 8)
        return fail(PKV_ERR_INVALID_ARG, "latent attention: page_stride must cover a page, a multiple of 8");
    if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4)) ||
        !stride_ok(q_token_stride) || !stride_ok(q_head_stride))
        return fail(PKV_ERR_INVALID_ARG, "latent attention: 16-byte aligned pointers and strides multiple of 8");
    if (!aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(q_indptr, 4) || !aligned(q_real, 4))
        return fail(PKV_ERR_INVALID_ARG, "latent attention: misaligned index pointer");
    if (block_table_stride < (static_cast<int64_t>(max_kv_len) + 31) / 32)
        return fail(PKV_ERR_INVALID_ARG, "latent attention: block_table_stride %lld is too short for max_kv_len",
                    static_cast<long long>(block_table_stride));
    if (flags & ~(PKV_FLAG_CHECKED | PKV_FLAG_SIMT_ONLY))
        return fail(PKV_ERR_UNSUPPORTED, "latent attention: flags %#x", flags);
    if ((flags & PKV_FLAG_CHECKED) && !err)
        return fail(PKV_ERR_INVALID_ARG, "latent attention: checked mode needs an error flag");
    const pkv::LatentParams p{q, q_token_stride, q_head_stride, pool, num_pages, page_stride, block_table,
                              block_table_stride, kv_lens, q_indptr, q_real, batch, max_q_rows, max_kv_len, num_heads,
                              mask == PKV_MASK_CAUSAL, scale * 1.4426950408889634f, out, out_dtype == PKV_F32, lse,
                              (flags & PKV_FLAG_CHECKED) != 0, err};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // (without keys every row is empty: the generic kernel writes them)
    if ((flags & PKV_FLAG_SIMT_ONLY) || max_kv_len == 0)
        return from_cuda(pkv::launch_latent_simt(p, s), "latent attention (simt)");
    const pkv::LatentPlan pl = pkv::plan_latent(batch, max_q_rows, num_heads, max_kv_len, device_sms());
    if (!workspace || workspace_bytes < pl.ws_bytes || !aligned(workspace, 256))
        return fail(PKV_ERR_WORKSPACE, "latent attention: workspace needs %zu bytes, 256-byte aligned", pl.ws_bytes);
    CUtensorMap tm;
    const int64_t dims[3] = {pkv::kLatentRow, 32, num_pages}, st[2] = {pkv::kLatentRow, page_stride};
    const int box[3] = {64, 32, 1};
    const pkv_status m = make_map(&tm, pool, 3, dims, st, box);
    if (m != PKV_OK) return m;
    // queries as boxes of a CTA's columns, where its (row, head) pairs are whole rows of
    // heads or a part of one, and the strides can stand in a tensor map
    CUtensorMap tq = tm;
    const int hbox = num_heads < pl.cols ? num_heads : pl.cols;
    bool boxes = (pl.cols % num_heads == 0 || num_heads % pl.cols == 0) && (num_heads == 1 || q_head_stride >= pkv::kLatentRow) &&
                 q_token_stride >= pkv::kLatentRow && q_token_stride < kMaxStride && q_head_stride < kMaxStride;
    if (boxes) {
        const int64_t qd[3] = {pkv::kLatentRow, num_heads, kMaxCount};
        const int64_t qs[2] = {num_heads == 1 ? int64_t(pkv::kLatentRow) : q_head_stride, q_token_stride};
        const int qbox[3] = {64, hbox, pl.cols / hbox};
        boxes = make_map(&tq, q, 3, qd, qs, qbox) == PKV_OK;
    }
    return from_cuda(pkv::launch_latent_attn(p, pl, workspace, &tm, &tq, boxes, s), "latent attention");
}

pkv_status ragged_attention_latent(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                                   int64_t k_token_stride, int64_t k_head_stride, const void* k_pe, int64_t k_pe_stride,
                                   const void* v, int64_t v_token_stride, int64_t v_head_stride, int64_t num_keys,
                                   const int32_t* q_indptr, const int32_t* kv_indptr, int batch, int max_q_rows,
                                   int max_kv_len, int num_heads, int nope_dim, int rope_dim, int v_dim, pkv_mask mask,
                                   float scale, void* out, pkv_dtype out_dtype, float* lse, unsigned flags, int32_t* err,
                                   void* stream) {
    if (batch < 0 || max_q_rows < 0 || max_kv_len < 0 || num_heads < 0 || num_keys < 0)
        return fail(PKV_ERR_INVALID_ARG, "ragged attention: negative size");
    if (batch == 0 || max_q_rows == 0 || num_heads == 0) return ok();
    if (nope_dim != pkv::kNopeDim || rope_dim != pkv::kLatentRope || v_dim != pkv::kExpandedV)
        return fail(PKV_ERR_UNSUPPORTED, "ragged attention: keys of %d + %d, values of %d (only 128 + 64, 128)", nope_dim,
                    rope_dim, v_dim);
    if (!q || !q_indptr || !kv_indptr || !out || (num_keys > 0 && (!k || !k_pe || !v)))
        return fail(PKV_ERR_INVALID_ARG, "ragged attention: null pointer");
    if (mask == PKV_MASK_BLOCK_CAUSAL) return fail(PKV_ERR_UNSUPPORTED, "ragged attention: no block-causal mask");
    if (mask != PKV_MASK_NONE && mask != PKV_MASK_CAUSAL)
        return fail(PKV_ERR_INVALID_ARG, "ragged attention: unknown mask %d", static_cast<int>(mask));
    if (out_dtype != PKV_BF16 && out_dtype != PKV_F32)
        return fail(PKV_ERR_UNSUPPORTED, "ragged attention: output dtype must be bf16 or f32");
    if (!(scale > 0.f) || std::isinf(scale))
        return fail(PKV_ERR_INVALID_ARG, "ragged attention: scale must be finite and > 0");
    if (batch > 65535 || num_heads > 65535) return fail(PKV_ERR_UNSUPPORTED, "ragged attention: batch or heads above 65535");
    if (max_kv_len > kMaxCount || max_q_rows > kMaxCount / num_heads || num_keys > kMaxCount)
        return fail(PKV_ERR_UNSUPPORTED, "ragged attention: sizes above 2^31 - 256");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(k_pe, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        (lse && !aligned(lse, 4)) || !stride_ok(q_token_stride) || !stride_ok(q_head_stride) ||
        !stride_ok(k_token_stride) || !stride_ok(k_head_stride) || !stride_ok(k_pe_stride) ||
        !stride_ok(v_token_stride) || !stride_ok(v_head_stride))
        return fail(PKV_ERR_INVALID_ARG, "ragged attention: 16-byte aligned pointers and strides multiple of 8");
    if (!aligned(q_indptr, 4) || !aligned(kv_indptr, 4))
        return fail(PKV_ERR_INVALID_ARG, "ragged attention: misaligned index pointer");
    if (k_token_stride > kMaxStride || k_head_stride > kMaxStride || k_pe_stride > kMaxStride ||
        v_token_stride > kMaxStride || v_head_stride > kMaxStride)
        return fail(PKV_ERR_UNSUPPORTED, "ragged attention: strides above 2^39 bytes");
    if (flags & ~(PKV_FLAG_CHECKED | PKV_FLAG_SIMT_ONLY))
        return fail(PKV_ERR_UNSUPPORTED, "ragged attention: flags %#x", flags);
    if ((flags & PKV_FLAG_CHECKED) && !err)
        return fail(PKV_ERR_INVALID_ARG, "ragged attention: checked mode needs an error flag");
    const pkv::RaggedParams p{q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, k_pe, k_pe_stride, v,
                              v_token_stride, v_head_stride, num_keys, q_indptr, kv_indptr, batch, max_q_rows, max_kv_len,
                              num_heads, mask == PKV_MASK_CAUSAL, scale * 1.4426950408889634f, out, out_dtype == PKV_F32,
                              lse, (flags & PKV_FLAG_CHECKED) != 0, err};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // (without keys every row is empty: the generic kernel writes them)
    if ((flags & PKV_FLAG_SIMT_ONLY) || num_keys == 0 || max_kv_len == 0)
        return from_cuda(pkv::launch_ragged_simt(p, s), "ragged attention (simt)");
    CUtensorMap tk, tp, tv;
    // a tensor of one head or one key may come with any stride there: its own width then
    auto st1 = [](int64_t s, int64_t n, int64_t w) { return n > 1 || s >= w ? s : w; };
    const int64_t kd[3] = {pkv::kNopeDim, num_heads, num_keys}, pd[2] = {pkv::kLatentRope, num_keys};
    const int64_t ks[2] = {st1(k_head_stride, num_heads, pkv::kNopeDim), st1(k_token_stride, num_keys, pkv::kNopeDim)};
    const int64_t vs[2] = {st1(v_head_stride, num_heads, pkv::kExpandedV), st1(v_token_stride, num_keys, pkv::kExpandedV)};
    const int64_t ps[1] = {st1(k_pe_stride, num_keys, pkv::kLatentRope)};
    const int box3[3] = {64, 1, 128}, box2[2] = {64, 128};
    pkv_status m = make_map(&tk, k, 3, kd, ks, box3);
    if (m == PKV_OK) m = make_map(&tv, v, 3, kd, vs, box3);
    if (m == PKV_OK) m = make_map(&tp, k_pe, 2, pd, ps, box2);
    if (m != PKV_OK) return m;
    // queries as boxes of 128 rows, where their strides can stand in a tensor map
    CUtensorMap tq = tk;
    const int64_t qd[3] = {pkv::kExpandedQ, num_heads, kMaxCount};
    const int64_t qs[2] = {num_heads == 1 ? int64_t(pkv::kExpandedQ) : q_head_stride, q_token_stride};
    const bool boxes = qs[0] >= pkv::kExpandedQ && qs[1] >= pkv::kExpandedQ && qs[0] < kMaxStride && qs[1] < kMaxStride &&
                       make_map(&tq, q, 3, qd, qs, box3) == PKV_OK;
    return from_cuda(pkv::launch_ragged_attn(p, &tk, &tp, &tv, &tq, boxes, s), "ragged attention");
}

}  // extern "C"
