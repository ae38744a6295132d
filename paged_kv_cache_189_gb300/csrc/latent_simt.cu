// latent_simt.cu -- generic attention over latent rows and over expanded keys
// and values: one warp a (query row, head), f32 throughout, any number of rows.
// A slow cross-check of the tensor-core kernels (PKV_FLAG_SIMT_ONLY).
//
//   s_j = scale q . k_j;  m = max s_j;  out = sum 2^(s_j - m) v_j / sum 2^(s_j - m)
// in one pass over the keys with a running maximum (scores in base 2).
#include "latent.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

// Running softmax state of a warp; each lane holds V of the output's elements.
template <int V>
struct Running {
    float m = -INFINITY, l = 0.f, o[V];
    __device__ Running() {
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = 0.f;
    }
    __device__ __forceinline__ void add(float s, const float (&v)[V]) {
        const float m_new = fmaxf(m, s);
        if (s == -INFINITY && m_new == -INFINITY) return;  // -inf before any other score: weight 0
        const float alpha = fast_exp2(m - m_new), w = fast_exp2(s - m_new);
        l = l * alpha + w;
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = fmaf(w, v[j], o[j] * alpha);
        m = m_new;
    }
    // element j of the lane is element lane * V + j of the row
    __device__ __forceinline__ void store(void* out, bool f32, float* lse, int64_t st, int lane) const {
        const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t at = st * (32 * V) + lane * V + j;
            if (f32) static_cast<float*>(out)[at] = o[j] * inv;
            else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(o[j] * inv);
        }
        if (lse && lane == 0) lse[st] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
    }
};

__device__ __forceinline__ float to_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__global__ void __launch_bounds__(128) latent_simt_kernel(LatentParams p) {
    constexpr int V = kLatentDim / 32, R = kLatentRope / 32;
    const int lane = threadIdx.x & 31;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int b = blockIdx.y;
    const int i = static_cast<int>(col / p.heads), h = static_cast<int>(col - static_cast<int64_t>(i) * p.heads);
    const int r0 = p.q_indptr[b], rows = p.q_indptr[b + 1] - r0, nrows = min(rows, p.max_q_rows);
    const int kv_all = p.kv_lens[b];
    if (p.checked && lane == 0 && col == 0 &&
        (kv_all > p.max_kv_len || kv_all < 0 || rows > p.max_q_rows || (p.q_real && p.q_real[b] > rows)))
        set_err(p.err, PKV_ERRBIT_LEN);
    if (i >= nrows) return;
    const int qreal = max(min(p.q_real ? p.q_real[b] : nrows, nrows), 0);
    const int kv = min(max(kv_all, 0), p.max_kv_len);
    const int nvis = i >= qreal ? 0 : p.causal ? max(0, kv - qreal + i + 1) : kv;

    float q[V + R];
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(r0 + i) * p.q_token_stride +
                              static_cast<int64_t>(h) * p.q_head_stride;
#pragma unroll
    for (int j = 0; j < V; ++j) q[j] = to_f(qp + lane * V + j) * p.scale_log2;
#pragma unroll
    for (int j = 0; j < R; ++j) q[V + j] = to_f(qp + kLatentDim + lane * R + j) * p.scale_log2;

    const int32_t* bt = p.block_table + static_cast<int64_t>(b) * p.block_table_stride;
    Running<V> st;
    for (int key = 0; key < nvis; ++key) {
        const int page = bt[key >> 5];
        const bool held = page >= 0 && page < p.num_pages;  // else a page of zeros
        if (!held && p.checked && lane == 0) set_err(p.err, PKV_ERRBIT_PAGE);
        float x[V], dot = 0.f;
        const __nv_bfloat16* c = static_cast<const __nv_bfloat16*>(p.pool) +
                                 (held ? static_cast<int64_t>(page) * p.page_stride + (key & 31) * kLatentRow : 0);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            x[j] = held ? to_f(c + lane * V + j) : 0.f;
            dot = fmaf(q[j], x[j], dot);
        }
#pragma unroll
        for (int j = 0; j < R; ++j) dot = fmaf(q[V + j], held ? to_f(c + kLatentDim + lane * R + j) : 0.f, dot);
        st.add(warp_sum(dot), x);
    }
    st.store(p.out, p.out_f32, p.lse, static_cast<int64_t>(r0 + i) * p.heads + h, lane);
}

__global__ void __launch_bounds__(128) ragged_simt_kernel(RaggedParams p) {
    constexpr int V = kExpandedV / 32, N = kNopeDim / 32, R = kLatentRope / 32;
    const int lane = threadIdx.x & 31;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int b = blockIdx.y;
    const int i = static_cast<int>(col / p.heads), h = static_cast<int>(col - static_cast<int64_t>(i) * p.heads);
    const int r0 = p.q_indptr[b], rows = p.q_indptr[b + 1] - r0, nrows = min(rows, p.max_q_rows);
    const int k0 = p.kv_indptr[b], kv_all = p.kv_indptr[b + 1] - k0;
    if (p.checked && lane == 0 && col == 0 &&
        (kv_all > p.max_kv_len || kv_all < 0 || rows > p.max_q_rows || k0 < 0 || k0 + int64_t(kv_all) > p.num_keys))
        set_err(p.err, PKV_ERRBIT_LEN);
    if (i >= nrows) return;
    const int kv = min(max(kv_all, 0), p.max_kv_len);
    const int nvis = p.causal ? max(0, kv - nrows + i + 1) : kv;

    float q[N + R];
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(r0 + i) * p.q_token_stride +
                              static_cast<int64_t>(h) * p.q_head_stride;
#pragma unroll
    for (int j = 0; j < N; ++j) q[j] = to_f(qp + lane * N + j) * p.scale_log2;
#pragma unroll
    for (int j = 0; j < R; ++j) q[N + j] = to_f(qp + kNopeDim + lane * R + j) * p.scale_log2;

    Running<V> st;
    for (int j0 = 0; j0 < nvis; ++j0) {
        const int64_t key = static_cast<int64_t>(k0) + j0;
        const bool held = key >= 0 && key < p.num_keys;  // rows past num_keys count as zeros
        const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + key * p.k_token_stride + h * p.k_head_stride;
        const __nv_bfloat16* pe = static_cast<const __nv_bfloat16*>(p.k_pe) + key * p.k_pe_stride;
        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + key * p.v_token_stride + h * p.v_head_stride;
        float x[V], dot = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) dot = fmaf(q[j], held ? to_f(k + lane * N + j) : 0.f, dot);
#pragma unroll
        for (int j = 0; j < R; ++j) dot = fmaf(q[N + j], held ? to_f(pe + lane * R + j) : 0.f, dot);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = held ? to_f(v + lane * V + j) : 0.f;
        st.add(warp_sum(dot), x);
    }
    st.store(p.out, p.out_f32, p.lse, static_cast<int64_t>(r0 + i) * p.heads + h, lane);
}

unsigned column_blocks(int rows, int heads) {
    return static_cast<unsigned>((static_cast<int64_t>(rows) * heads + 3) / 4);
}

}  // namespace

cudaError_t launch_latent_simt(const LatentParams& p, cudaStream_t s) {
    latent_simt_kernel<<<dim3(column_blocks(p.max_q_rows, p.heads), p.batch), 128, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_ragged_simt(const RaggedParams& p, cudaStream_t s) {
    ragged_simt_kernel<<<dim3(column_blocks(p.max_q_rows, p.heads), p.batch), 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
