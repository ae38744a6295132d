// expand.cu -- pages of an 8-bit cache as bf16, for the tile kernel.
//
// element = bf16(code * scale): exact while the scale is a power of two (an
// e4m3 code has 4 significant bits, bf16 holds 8), one rounding otherwise.
// The tile kernel's products want 16-bit operands in shared memory, each K/V
// tile is read by every pair of row tiles of its sequence and head, and the
// softmax warps are what that kernel waits for; widening inside it would repeat
// the conversion per pair on busy issue slots, this pass makes it once per
// call.  It costs 1 byte read and 2 written per element, which the tiles read
// back: 30 us of the 475 of four prompt chunks of 1024-2048 tokens, 56 of 270 at
// 256 tokens in each of 16 sequences, but 195 of 380 at 24 tokens (of 4 grouped
// heads) in each of 64, where one pair of tiles covers a sequence.
// Bound: HBM; a block takes one page of one sequence, 16 codes a thread and step.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

__device__ __forceinline__ void widen(const uint4& v, float scale, uint4 (&out)[2]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] & 0xffffu), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> 16), __NV_E4M3);
        const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
        o[2 * i] = pack_bf16x2(a.x * scale, a.y * scale);
        o[2 * i + 1] = pack_bf16x2(b.x * scale, b.y * scale);
    }
    out[0] = make_uint4(o[0], o[1], o[2], o[3]);
    out[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

__global__ void __launch_bounds__(256) expand_fp8_kernel(const AttnParams p, __nv_bfloat16* k_out,
                                                          __nv_bfloat16* v_out, int pages) {
    const int b = blockIdx.y, c = blockIdx.x;
    const int nrows = min(p.q_indptr[b + 1] - p.q_indptr[b], p.max_q_rows);
    const int qreal = max(min(p.q_real ? p.q_real[b] : nrows, nrows), 0);
    const int kv_len = min(max(p.kv_lens[b], 0), p.max_kv_len);
    if (qreal == 0) return;
    // the keys of the sequence's first row on, and the sinks before them
    const int near = (p.window > 0 ? max(0, kv_len - qreal - p.window + 1) : 0) / 32;
    const int sinks = min((min(p.num_sinks, kv_len) + 31) / 32, near);
    const int lp = c < sinks ? c : near + c - sinks;
    if (lp * 32 >= kv_len) return;
    const int page = p.block_table[b * p.block_table_stride + lp];
    const bool valid = page >= 0 && page < p.num_pages;
    if (!valid && p.checked && threadIdx.x == 0) set_err(p.err, PKV_ERRBIT_PAGE);
    const int D = p.head_dim;
    const int per_slot = p.num_kv_heads * D / 16;  // 16-code vectors of a slot
    const int64_t dst = (static_cast<int64_t>(b) * pages + c) * 32 * per_slot;
    const uint4* src[2] = {
        reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_pool) + (valid ? page * p.page_stride : 0)),
        reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.v_pool) + (valid ? page * p.page_stride : 0))};
    const float* scale[2] = {p.k_scale + (valid ? page * p.scale_stride : 0),
                             p.v_scale + (valid ? page * p.scale_stride : 0)};
    uint4* out[2] = {reinterpret_cast<uint4*>(k_out) + 2 * dst, reinterpret_cast<uint4*>(v_out) + 2 * dst};
    const int live = min(32, kv_len - lp * 32) * per_slot;  // slots past the last key stay as they are
#pragma unroll
    for (int w = 0; w < 2; ++w)
        for (int i = threadIdx.x; i < live; i += 256) {
            const float s = valid ? __ldg(scale[w] + (i % per_slot) * 16 / D) : 0.f;
            const uint4 v = valid ? __ldg(src[w] + i) : make_uint4(0u, 0u, 0u, 0u);
            uint4 o[2];
            widen(v, s, o);
            out[w][2 * i] = o[0];
            out[w][2 * i + 1] = o[1];
        }
}

}  // namespace

cudaError_t launch_expand_fp8(const AttnParams& p, void* k_out, void* v_out, int pages, cudaStream_t s) {
    const dim3 grid(pages, p.batch);
    expand_fp8_kernel<<<grid, 256, 0, s>>>(p, static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out),
                                           pages);
    return cudaGetLastError();
}

}  // namespace pkv
