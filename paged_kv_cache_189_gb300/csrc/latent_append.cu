// latent_append.cu -- kv_append_latent: RMS norm, rotation and paged write of
// the step's latent rows, and the rotation of their query heads, in one launch.
//
//   row = [x / sqrt(mean x^2 + eps) * w | R(position) x_pe],  q_out = R(position) q_pe
// A call is bound by its loads' latency, one chain position -> angles -> store a token;
// prompts by how many of them are under way: one CTA a token, its first warp
// the latent row (two 16-byte chunks a lane, the sum of squares over the warp),
// the others eight query heads each at a time, four lanes a head with two
// 16-byte chunks each, so both elements of every pair, in either order of
// pairs, are in one lane.  Measured, replayed as a graph: 2.2 us for 64 tokens of
// 16 heads; 19.9 us for 7.7 k tokens of 32 heads (82.6 MB, 0.61 of the copy rate).  There
// counters show the algorithmic bytes (41.6 MB read, the writes still in L2), DRAM at
// 29 %, 45 % of the warps and 15 cycles of waiting for loads an instruction.  1216 to
// 3648 CTAs that walk the tokens took 19.6 to 24.7 us.
#include "latent.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kHeadWarps = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16lo(w[i]);
        f[2 * i + 1] = bf16hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Chunks c and c + 4 (of eight) of a rotary part: pairs (a[j], b[j]), or the
// neighbours inside each chunk.  cs: the position's cosines, then its sines.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate_chunks(const float* cs, int c, uint4& av, uint4& bv) {
    float a[8], b[8], x[8], y[8], cc[8], ss[8];
    unpack8(av, a);
    unpack8(bv, b);
    // angles of the eight pairs: 8 c .. 8 c + 7, or 4 c .. and 16 + 4 c ..
    const int i0 = INTERLEAVED ? 4 * c : 8 * c, i1 = INTERLEAVED ? 16 + 4 * c : 8 * c + 4;
    *reinterpret_cast<float4*>(cc) = *reinterpret_cast<const float4*>(cs + i0);
    *reinterpret_cast<float4*>(cc + 4) = *reinterpret_cast<const float4*>(cs + i1);
    *reinterpret_cast<float4*>(ss) = *reinterpret_cast<const float4*>(cs + kLatentRope / 2 + i0);
    *reinterpret_cast<float4*>(ss + 4) = *reinterpret_cast<const float4*>(cs + kLatentRope / 2 + i1);
    if constexpr (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = a[2 * j] * cc[j] - a[2 * j + 1] * ss[j];
            x[2 * j + 1] = a[2 * j + 1] * cc[j] + a[2 * j] * ss[j];
            y[2 * j] = b[2 * j] * cc[4 + j] - b[2 * j + 1] * ss[4 + j];
            y[2 * j + 1] = b[2 * j + 1] * cc[4 + j] + b[2 * j] * ss[4 + j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = a[j] * cc[j] - b[j] * ss[j];
            y[j] = b[j] * cc[j] + a[j] * ss[j];
        }
    }
    av = pack8(x);
    bv = pack8(y);
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(32 * (1 + kHeadWarps)) append_latent_kernel(const LatentAppendArgs a) {
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t pos = a.positions[t];
    const bool in_table = pos >= 0 && pos < a.max_position;
    pos = min(max(pos, int64_t(0)), a.max_position - 1);
    const float* cs = a.cos_sin + pos * kLatentRope;
    if (warp > 0) {
        const int c = lane & 3;
        for (int h = (warp - 1) * 8 + (lane >> 2); h < a.num_heads; h += kHeadWarps * 8) {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q_pe) +
                                                              t * a.q_pe_token_stride + h * a.q_pe_head_stride);
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.q_out) + t * a.q_out_token_stride +
                                                  h * a.q_out_head_stride);
            uint4 x = src[c], y = src[c + 4];
            rotate_chunks<INTERLEAVED>(cs, c, x, y);
            dst[c] = x;
            dst[c + 4] = y;
        }
        return;
    }
    if (a.checked && !in_table && lane == 0) set_err(a.err, PKV_ERRBIT_LEN);
    const int64_t slot = a.slots[t];
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.src) + t * a.src_stride);
    if (slot < 0) return;
    if (slot >= a.num_pages * 32) {
        if (a.checked && lane == 0) set_err(a.err, PKV_ERRBIT_SLOT);
        return;
    }
    uint4 v[2] = {src[lane], src[lane + 32]}, x, y;
    if (lane < 4) {
        x = src[64 + lane];
        y = src[68 + lane];
    }
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.pool) + (slot >> 5) * a.page_stride +
                                          (slot & 31) * kLatentRow);
    if (a.norm_weight) {
        const uint4* wp = static_cast<const uint4*>(a.norm_weight);
        const uint4 wv[2] = {wp[lane], wp[lane + 32]};
        float f[2][8], w[8], sum = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            unpack8(v[k], f[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(f[k][j], f[k][j], sum);
        }
        const float r = 1.0f / sqrtf(warp_sum(sum) * (1.0f / kLatentDim) + a.eps);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            unpack8(wv[k], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[k][j] = f[k][j] * r * w[j];
            v[k] = pack8(f[k]);
        }
    }
    dst[lane] = v[0];
    dst[lane + 32] = v[1];
    if (lane < 4) {
        rotate_chunks<INTERLEAVED>(cs, lane, x, y);
        dst[64 + lane] = x;
        dst[68 + lane] = y;
    }
}

}  // namespace

cudaError_t launch_append_latent(const LatentAppendArgs& a, cudaStream_t s) {
    const int head_warps = min(kHeadWarps, (a.num_heads + 7) / 8);
    const unsigned tokens = static_cast<unsigned>(a.num_tokens);
    if (a.interleaved) append_latent_kernel<true><<<tokens, 32 * (1 + head_warps), 0, s>>>(a);
    else append_latent_kernel<false><<<tokens, 32 * (1 + head_warps), 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
