// kv_append.cu -- kv_append_fp8: quantise new K/V rows into an 8-bit paged cache.
//
// An element is code * scale with an e4m3 code and one f32 scale per (32-token
// page, K/V head), K and V apart.  The scale is a power of two, 2^e with the
// smallest e for which the largest magnitude fits 448 * 2^e: dividing by it
// changes no bit, so an element carries exactly one rounding, and when a later
// token raises the scale of a page that already holds tokens, moving the old
// codes to it only lowers their exponents -- no second rounding until a code
// becomes subnormal.  e4m3 keeps 4 significant bits over 2^-6 .. 448 whatever
// the scale, so the up-to-one bit of range a power of two gives away costs
// nothing; an amax / 448 scale would round every old code again at each growth.
//
// One warp per (sequence, touched page, K/V head, K or V): it owns the page's
// 32 slots of that head, so nothing is shared between warps and the result does
// not depend on their order.  Rows of 2-byte elements (16-byte vectors, D / 8
// lanes a row) are all loaded at once, before the page is looked up, and stay
// in registers between the maximum (packed, two elements an instruction) and
// the conversion: every source byte is read once.  4-byte rows would take 128
// registers; they are loaded twice, both times marked for early eviction as the
// others are.
// Bound: HBM for chunks (2 bytes read and 1 written per bf16 element), launch
// and one chain of dependent loads (lengths, page id, old scale) for one token
// per sequence.  Measured: 48.3 MB of four ragged prompt chunks (eight heads of
// 128) 13 us, 0.56 of the copy peak, from bf16 or f16 rows (1040 blocks on the 608
// places there are, two waves, each with the chain of loads: about 4 us with the
// launch); 80.6 MB from f32 rows 32 us, 0.38 of it; one token into each of 64
// sequences 6 us.  Streaming loads took the 2-byte chunks from 14.6 to 13 us (the
// rows are read once); 4 blocks of 4 warps an SM beat 5 to 8 with spills (16.4) and
// a second read instead of registers (16.9).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <algorithm>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kPage = 32;
constexpr int kWarps = 4;

// two f32 -> two e4m3 codes (round to nearest even, saturating; NaN stays NaN)
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t pair) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3);
    return __half22float2(__half2(h));
}

// One 16-byte vector of the source type: its values as f32, the largest
// magnitude so far (NaN passed over), the type's largest finite value.
template <typename T>
struct Src;
template <>
struct Src<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static constexpr float kTop = 3.3895313892515355e38f;
    __nv_bfloat162 peak = __floats2bfloat162_rn(0.f, 0.f);
    __device__ void see(const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) peak = __hmax2(peak, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
    }
    __device__ float top() const { return fmaxf(__low2float(peak), __high2float(peak)); }
    __device__ static void widen(const uint4& v, float (&x)[kVec]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16lo(w[i]);
            x[2 * i + 1] = bf16hi(w[i]);
        }
    }
};
template <>
struct Src<__half> {
    static constexpr int kVec = 8;
    static constexpr float kTop = 65504.f;
    __half2 peak = __floats2half2_rn(0.f, 0.f);
    __device__ void see(const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) peak = __hmax2(peak, __habs2(*reinterpret_cast<const __half2*>(&w[i])));
    }
    __device__ float top() const { return fmaxf(__low2float(peak), __high2float(peak)); }
    __device__ static void widen(const uint4& v, float (&x)[kVec]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Src<float> {
    static constexpr int kVec = 4;
    static constexpr float kTop = 3.4028234663852886e38f;
    float peak = 0.f;
    __device__ void see(const uint4& v) {
        float x[kVec];
        widen(v, x);
#pragma unroll
        for (int i = 0; i < kVec; ++i) peak = fmaxf(peak, fabsf(x[i]));
    }
    __device__ float top() const { return peak; }
    __device__ static void widen(const uint4& v, float (&x)[kVec]) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
};

// 2^e, the smallest e >= -126 with amax <= 448 * 2^e = 1.75 * 2^(e + 8); 0 for 0
__device__ __forceinline__ float scale_for(float amax) {
    if (!(amax > 0.f)) return 0.f;
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7);
    return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}

template <int N>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&y)[N]) {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        w[i] = to_e4m3x2(y[4 * i], y[4 * i + 1]) | (to_e4m3x2(y[4 * i + 2], y[4 * i + 3]) << 16);
    if constexpr (N == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 4 : 8)
    append_fp8_kernel(const __grid_constant__ AppendArgs a, int pages_bound) {
    constexpr int kVec = Src<T>::kVec;          // elements of a lane's vector
    constexpr int kLanes = D / kVec;            // lanes a row takes
    constexpr int kRows = 32 / kLanes;          // rows of one warp-wide load
    constexpr int kSteps = kPage / kRows;
    constexpr bool kKeep = sizeof(T) == 2;
    const int lane = threadIdx.x & 31;
    const int Hkv = a.num_kv_heads;
    const int b = blockIdx.y;
    const int item = blockIdx.x * kWarps + (threadIdx.x >> 5);  // (page, K or V, head), heads fastest
    const int t = item / (2 * Hkv);
    if (t >= pages_bound) return;
    const int rest = item - t * 2 * Hkv;
    const int which = rest >= Hkv ? 1 : 0, h = rest - which * Hkv;

    const int r0 = a.q_indptr[b];
    const int rows = a.q_indptr[b + 1] - r0;
    const int real = a.q_real ? a.q_real[b] : rows, kv_len = a.kv_lens[b];
    if (a.checked && item == 0 && lane == 0 &&
        (kv_len > a.max_kv_len || kv_len < 0 || rows > a.max_q_rows || real > rows))
        set_err(a.err, PKV_ERRBIT_LEN);
    const int first = max(kv_len, 0) - max(real, 0);  // position of the first new row (may be below 0)
    // new rows end here: as many as there are, below the host bounds
    const int last = min(first + min(min(real, rows), a.max_q_rows), a.max_kv_len);
    if (real <= 0 || first >= last || last <= 0) return;
    const int logical = max(first, 0) / kPage + t;
    if (logical > (last - 1) / kPage) return;  // in pages: at the widest bounds the position would pass 2^31
    const int pos0 = logical * kPage;          // this page's first position
    const int begin = max(first - pos0, 0), end = min(last - pos0, kPage);  // slots that receive rows

    const int sub = lane / kLanes, col = (lane % kLanes) * kVec;
    const T* src = static_cast<const T*>(a.src[which]) +
                   (static_cast<int64_t>(r0) - first + pos0 + sub) * a.src_token_stride +
                   static_cast<int64_t>(h) * a.src_head_stride + col;
    const int64_t step = a.src_token_stride * kRows;
    auto row = [&](int s) {
        return s * kRows + sub >= begin && s * kRows + sub < end
                   ? __ldcs(reinterpret_cast<const uint4*>(src + s * step)) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 v[kKeep ? kSteps : 1];
    if constexpr (kKeep) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) v[s] = row(s);
    }
    const int page = a.block_table[b * a.block_table_stride + logical];
    if (page < 0 || page >= a.num_pages) {
        if (a.checked && lane == 0) set_err(a.err, PKV_ERRBIT_PAGE);
        return;
    }
    float* sp = a.scale[which] + page * a.scale_stride + h;
    const float had = begin > 0 ? *sp : 0.f;

    Src<T> peak;
    if constexpr (kKeep) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) peak.see(v[s]);
    } else {
#pragma unroll 8
        for (int s = 0; s < kSteps; ++s) peak.see(row(s));
    }
    const float amax = warp_max(peak.top());
    const float scale = fmaxf(had, scale_for(fminf(amax, Src<T>::kTop)));
    const float inv = scale > 0.f ? 1.0f / scale : 0.f;
    const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0;  // a power of two: its reciprocal is exact
    const int64_t slot_stride = static_cast<int64_t>(Hkv) * D;
    uint8_t* dst = a.pool[which] + page * a.page_stride + sub * slot_stride + static_cast<int64_t>(h) * D + col;
    // the scale grew: the page's earlier codes, to the new one
    if (begin > 0 && scale != had) {
#pragma unroll 1
        for (int s = 0; s * kRows + sub < begin; ++s) {
            uint8_t* at = dst + s * kRows * slot_stride;
            uint32_t w[kVec / 4];
            if constexpr (kVec == 8) {
                const uint2 c = *reinterpret_cast<const uint2*>(at);
                w[0] = c.x;
                w[1] = c.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t*>(at);
            }
            float y[kVec];
#pragma unroll
            for (int i = 0; i < kVec / 4; ++i) {
                const float2 lo = from_e4m3x2(w[i] & 0xffffu), hi = from_e4m3x2(w[i] >> 16);
                const float o[4] = {lo.x * had, lo.y * had, hi.x * had, hi.y * had};
#pragma unroll
                for (int e = 0; e < 4; ++e) y[4 * i + e] = exact ? o[e] * inv : o[e] / scale;
            }
            store_codes<kVec>(at, y);
        }
    }
    if (exact && amax != INFINITY) {
#pragma unroll(kKeep ? kSteps : 4)
        for (int s = 0; s < kSteps; ++s) {
            if (s * kRows + sub >= begin && s * kRows + sub < end) {
                float x[kVec];
                if constexpr (kKeep) Src<T>::widen(v[s], x);
                else Src<T>::widen(row(s), x);
#pragma unroll
                for (int i = 0; i < kVec; ++i) x[i] *= inv;
                store_codes<kVec>(dst + s * kRows * slot_stride, x);
            }
        }
    } else {
        // infinities among the rows, or an old scale that is no power of two
#pragma unroll 1
        for (int s = 0; s < kSteps; ++s) {
            if (s * kRows + sub >= begin && s * kRows + sub < end) {
                float x[kVec];
                Src<T>::widen(row(s), x);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    if (fabsf(x[i]) == INFINITY) x[i] = copysignf(Src<T>::kTop, x[i]);
                    x[i] = exact ? x[i] * inv : x[i] / scale;
                }
                store_codes<kVec>(dst + s * kRows * slot_stride, x);
            }
        }
    }
    if (lane == 0) *sp = scale;
}

template <typename T>
cudaError_t launch_t(const AppendArgs& a, cudaStream_t s) {
    // n rows touch at most (n + 30) / 32 + 1 pages, whatever slot they start at,
    // and none past the cache's bound (either limit may be close to 2^31)
    const int64_t touched = (static_cast<int64_t>(a.max_q_rows) + kPage - 2) / kPage + 1;
    const int pages = static_cast<int>(std::min<int64_t>(touched, (static_cast<int64_t>(a.max_kv_len) + kPage - 1) / kPage));
    const int64_t items = static_cast<int64_t>(pages) * 2 * a.num_kv_heads;
    const dim3 grid(static_cast<unsigned>((items + kWarps - 1) / kWarps), a.batch);
    if (a.head_dim == 128) append_fp8_kernel<T, 128><<<grid, kWarps * 32, 0, s>>>(a, pages);
    else append_fp8_kernel<T, 64><<<grid, kWarps * 32, 0, s>>>(a, pages);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_fp8(const AppendArgs& a, cudaStream_t s) {
    switch (a.src_dtype) {
        case PKV_BF16: return launch_t<__nv_bfloat16>(a, s);
        case PKV_F16: return launch_t<__half>(a, s);
        default: return launch_t<float>(a, s);
    }
}

}  // namespace pkv
