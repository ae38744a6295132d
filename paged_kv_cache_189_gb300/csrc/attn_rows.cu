// attn_rows.cu -- attention of few query rows per sequence over a paged cache
// held in 8 bits or in bf16, with a sliding window and sinks: the decode and
// small multi-token form of paged_attention_fp8 and paged_attention_window.
//
// Mathematics, per (query row, head) over its visible keys j, in base 2:
//   a_j = s log2(e) q.k_j,   out = sum_j 2^(a_j - M) v_j / sum_j 2^(a_j - M)
// with a running reference M; states (M, l, O) over disjoint keys join exactly.
// For 8-bit pools k_j = ks c_j and v_j = vs d_j with one ks and vs a page, so
// the kernel contracts the codes and applies the scales to scores and weights.
//
// Bound: HBM.  Every K/V byte is read once for the query heads that share it;
// at 8 bits the multiply-adds per byte are twice bf16's, more than the FP32
// pipes take at full bandwidth for 4 heads, so both products run on mma.sync.
// (tcgen05 wants 128 rows; 4 to 16 leave it idle, and its operands would have
// to be widened through shared memory first.)
//  * Keys take the M side of both products, query rows the N side: S^T = K Q^T
//    and O^T = V^T P^T in m16n8k16 steps, so 8 rows (2 tokens of 4 grouped
//    heads, say) fill a tile that a row-major form would half waste.
//  * e4m3 codes widen to f16 exactly in registers.  The contraction may take
//    its dimensions in any order that K and Q share: a lane loads 16-byte runs
//    of a key and feeds them to consecutive steps.  V comes through transposing
//    16-bit ldmatrix; a byte permute separates the two dimensions it pairs.
//  * q is bf16; for 8-bit pools each row is brought to 2^8 by a power of two
//    (undone in the score's factor) and held in f16: exact but for elements
//    2^-22 below the row's largest.
//  * Weights are rounded once: to bf16 for bf16 pools, and w = 2^(a - M) vs to
//    f16 for 8-bit ones, M following a + log2(vs), so w stays at or below 2^9
//    whatever the scales.  Sums, maxima and outputs are f32.
//  * A warp owns whole chunks of keys (32 in 8 bits, 16 in bf16) with its own
//    ring of TMA copies and its own softmax state: no barrier between warps
//    until a unit's end.  8 warps an SM keep 192 KB in flight.
//  * Work: a unit is (sequence, K/V head, tile of 8 or 16 rows); its chunks are
//    the pages its rows see.  All units' chunks form one line that is cut into
//    equal shares, one per resident CTA; a unit cut between CTAs leaves partial
//    states that a second launch joins in a fixed order.  The cut follows the
//    lengths on the device (each CTA sums them itself), so a captured call
//    replays with other lengths.  Small calls skip the cut: one CTA a unit.
#include <cuda.h>
#include <cuda_fp16.h>
#include <algorithm>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kPage = 32;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kRingBytes = 24 * 1024;  // per warp
constexpr int kMinShare = 2 * kWarps;  // chunks a CTA takes at least
constexpr float kLazy = 8.0f;          // move the reference only past 2^8 growth
constexpr float kLowScale = -90.0f;    // log2 of the smallest V scale M follows

template <int D, bool FP8, int NT>
struct Cfg {
    static constexpr int kKeys = FP8 ? 32 : 16;          // keys of a chunk
    static constexpr int kTile = kKeys * D * (FP8 ? 1 : 2);
    static constexpr int kStage = 2 * kTile;             // K, V
    static constexpr int kStages = kRingBytes / kStage;  // 3 (head dim 128), 6 (64)
    static constexpr int kRows = 8 * NT;
    static constexpr int kRedStride = D + 4;
    static constexpr int kRedOff = kWarps * kStages * kStage;          // [warps][4][kRedStride] f32
    static constexpr int kStatOff = kRedOff + kWarps * 4 * kRedStride * 4;  // m, l, l_b: [warps][kRows]
    static constexpr int kMetaOff = kStatOff + 3 * kWarps * kRows * 4;  // [warps][stages] (ks, vs, key0)
    static constexpr int kBarOff = kMetaOff + kWarps * kStages * 16;
    static constexpr int kBytes = kBarOff + kWarps * kStages * 8;
    static_assert((kBytes + 2048) * kCtasPerSm <= 228 * 1024, "CTAs per SM must fit in shared memory");
    static_assert(kMetaOff % 16 == 0 && kBarOff % 8 == 0, "alignment");
};

struct RowsArgs {
    AttnParams p;
    int ctas;       // shares of the line (0: one CTA a unit)
    int tiles_max;  // row tiles of a sequence at the host bound
    float* frag_o;    // [ctas][2][rows][D] normalised partial outputs
    float* frag_lse;  // [ctas][2][rows] (natural log)
    int4* frag_dir;   // [ctas][2] (sequence, K/V head, row tile, flags)
};
constexpr int kFragValid = 1, kFragStarts = 2, kFragEnds = 4;

// ---------------------------------------------------------------------------
// Geometry
// ---------------------------------------------------------------------------
__device__ __forceinline__ int row_limit(const AttnParams& p, int t, int qreal, int kv_len) {
    const int first = kv_len - qreal;
    int end = kv_len;
    if (p.mask == PKV_MASK_CAUSAL) end = first + t + 1;
    else if (p.mask == PKV_MASK_BLOCK_CAUSAL) end = first + min(qreal, (t / p.causal_block + 1) * p.causal_block);
    return min(max(end, 0), kv_len);
}

struct Seq {
    int r0, nrows, qreal, kv_len, tiles;
};
template <int ROWS>
__device__ __forceinline__ Seq sequence(const AttnParams& p, int b, int G) {
    Seq s;
    s.r0 = p.q_indptr[b];
    s.nrows = max(min(p.q_indptr[b + 1] - s.r0, p.max_q_rows), 0);
    s.qreal = max(min(p.q_real ? p.q_real[b] : s.nrows, s.nrows), 0);
    s.kv_len = min(max(p.kv_lens[b], 0), p.max_kv_len);
    s.tiles = static_cast<int>((static_cast<int64_t>(s.nrows) * G + ROWS - 1) / ROWS);
    return s;
}

// The keys some row of tile mt sees are inside [0, sinks) and [lo, hi); its
// chunks are the first nsc of the cache and those from loc on, n in all.
struct Span {
    int lo, hi, nsc, loc, n;
};
template <int ROWS, int KEYS>
__device__ __forceinline__ Span span_of(const AttnParams& p, const Seq& s, int mt, int G) {
    Span u{0, 0, 0, 0, 0};
    const int tf = mt * ROWS / G, tl = min((mt * ROWS + ROWS - 1) / G, s.qreal - 1);
    if (tf >= s.qreal) return u;
    u.hi = row_limit(p, tl, s.qreal, s.kv_len);
    if (u.hi <= 0) return u;
    u.lo = p.window > 0 ? max(0, s.kv_len - s.qreal + tf - p.window + 1) : 0;
    u.loc = u.lo / KEYS;
    u.nsc = min((min(p.num_sinks, u.hi) + KEYS - 1) / KEYS, u.loc);
    u.n = u.nsc + (u.hi + KEYS - 1) / KEYS - u.loc;
    return u;
}

// A CTA's share of the line of units, as segments: chunks [ps, pe) of a unit
// (n = 0: a unit of rows that see nothing takes one place, with no chunk).
template <int ROWS, int KEYS>
struct Walk {
    int b, kvh, mt, at;  // next unit, and the place in it
    int64_t left;        // places of the share still to come
    // the current segment
    Seq s;
    Span u;
    int sb, skvh, smt, ps, pe;
    bool starts, ends;

    __device__ __forceinline__ bool next(const AttnParams& p, int G) {
        while (left > 0 && b < p.batch) {
            s = sequence<ROWS>(p, b, G);
            if (mt >= s.tiles) {
                at = 0;
                mt = 0;
                if (s.tiles == 0 || ++kvh == p.num_kv_heads) {
                    kvh = 0;
                    ++b;
                }
                continue;
            }
            u = span_of<ROWS, KEYS>(p, s, mt, G);
            const int places = max(u.n, 1);
            sb = b;
            skvh = kvh;
            smt = mt;
            ps = at;
            pe = static_cast<int>(min(static_cast<int64_t>(places), at + left));
            starts = ps == 0;
            ends = pe == places;
            left -= pe - ps;
            if (ends) {
                at = 0;
                ++mt;
            } else {
                at = pe;
            }
            pe = min(pe, u.n);
            return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------------------
// Matrix instructions and conversions
// ---------------------------------------------------------------------------
template <bool FP8>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FP8)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// four e4m3 codes -> two f16 pairs (exact)
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A warp's softmax state and output tile; rows 8j + 2t + e of lane 4g + t.
template <int D, int NT>
struct State {
    float m[NT][2], l[NT][2], lb[NT][2];
    float o[NT][D / 16][4];
};

// What a chunk needs of its segment.
template <int NT>
struct RowInfo {
    int lim[NT][2], lo[NT][2];  // of this lane's rows
    int all_end, all_lo;        // keys [all_lo, all_end) are visible to every real row
    int any_lo, any_end, sinks; // keys outside [any_lo, any_end) and [0, sinks) to none
    float fq[NT][2];            // score factor of this lane's rows
};

// One chunk: scores, weights and the output update.  MASKED: some key of it is
// hidden from some row.
template <int D, bool FP8, int NT, bool MASKED>
__device__ __forceinline__ void chunk_step(State<D, NT>& st, const uint32_t (&qf)[NT][D / 16][2],
                                           const RowInfo<NT>& ri, uint32_t kb, uint32_t vb, float ks, float vs,
                                           int key0, int lane) {
    using C = Cfg<D, FP8, NT>;
    constexpr int MI = C::kKeys / 16;
    const int g = lane >> 2, t = lane & 3;
    // ---- S^T = K Q^T
    float s[MI][NT][4];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mi][j][e] = 0.f;
        const int r0 = 16 * mi + g;  // this lane's keys r0 and r0 + 8
        if constexpr (FP8) {
            constexpr int kLoads = D / 64;
            constexpr int kRowB = D;
            const uint32_t x = D == 128 ? ((2 * t) ^ g) << 4 : (t ^ ((r0 >> 1) & 3)) << 4;
            const uint32_t a0 = kb + r0 * kRowB + x;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint4 u = lds128(a0 ^ (i << 4)), v = lds128((a0 ^ (i << 4)) + 8 * kRowB);
                const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t a[4];
                    widen4(uw[k], a[0], a[2]);
                    widen4(vw[k], a[1], a[3]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma<FP8>(s[mi][j], a, qf[j][4 * i + k][0], qf[j][4 * i + k][1]);
                }
            }
        } else {
            const uint32_t a0 = kb + r0 * 128 + (((2 * t) ^ g) << 4);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t ad = (a0 ^ ((i & 1) << 4)) + (i >> 1) * (C::kKeys * 128);
                const uint4 u = lds128(ad), v = lds128(ad + 8 * 128);
                const uint32_t x0[4] = {u.x, v.x, u.y, v.y}, x1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma<FP8>(s[mi][j], x0, qf[j][2 * i][0], qf[j][2 * i][1]);
                    mma<FP8>(s[mi][j], x1, qf[j][2 * i + 1][0], qf[j][2 * i + 1][1]);
                }
            }
        }
    }
    // ---- weights
    float lv = 0.f;  // log2 of the V scale, rounded down
    if constexpr (FP8)
        lv = fmaxf(static_cast<float>(static_cast<int>((__float_as_uint(vs) >> 23) & 255u) - 127), kLowScale);
    uint32_t pb[NT][MI][2];
    bool moved = false;
    float alpha[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float ref[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float f = FP8 ? ri.fq[j][e] * ks : ri.fq[j][e];
            float mx = -INFINITY;
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float x = s[mi][j][2 * hh + e] * f;
                    if constexpr (MASKED) {
                        const int key = key0 + 16 * mi + 8 * hh + g;
                        if (!(key < ri.lim[j][e] && (key >= ri.lo[j][e] || key < ri.sinks))) x = -INFINITY;
                    }
                    s[mi][j][2 * hh + e] = x;
                    mx = fmaxf(mx, x);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if constexpr (FP8) mx += lv;
            alpha[j][e] = 1.f;
            if (mx > st.m[j][e] + kLazy) {  // also the first visible key
                alpha[j][e] = fast_exp2(st.m[j][e] - mx);
                st.m[j][e] = mx;
                moved = true;
            }
            ref[e] = st.m[j][e] == -INFINITY ? 0.f : st.m[j][e];
        }
        float sum[2] = {0.f, 0.f}, sumb[2] = {0.f, 0.f};
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const float p0 = fast_exp2(s[mi][j][2 * hh] - ref[0]), p1 = fast_exp2(s[mi][j][2 * hh + 1] - ref[1]);
                sum[0] += p0;
                sum[1] += p1;
                uint32_t w;
                if constexpr (FP8) {
                    w = pack_f16x2(p0 * vs, p1 * vs);
                } else {
                    w = pack_bf16x2(p0, p1);
                    sumb[0] += bf16lo(w);
                    sumb[1] += bf16hi(w);
                }
                pb[j][mi][hh] = movmatrix(w);  // (key g; rows 2t, 2t + 1) -> (row g; keys 2t, 2t + 1)
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            st.l[j][e] = st.l[j][e] * alpha[j][e] + sum[e];
            if constexpr (!FP8) st.lb[j][e] = st.lb[j][e] * alpha[j][e] + sumb[e];
        }
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.o[j][c][e] *= alpha[j][e & 1];
    }
    // ---- O^T += V^T P^T; the V of keys that no row sees may hold anything
    uint32_t vm[2 * MI];
    if constexpr (MASKED) {
#pragma unroll
        for (int k = 0; k < 2 * MI; ++k) {
            uint32_t keep = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int key = key0 + 8 * k + 2 * t + e;
                if (key < ri.any_end && (key >= ri.any_lo || key < ri.sinks)) keep |= 0xffffu << (16 * e);
            }
            vm[k] = keep;
        }
    }
    if constexpr (FP8) {
        constexpr int kRowB = D;
        const uint32_t x = D == 128 ? (lane & 7) << 4 : ((lane >> 1) & 3) << 4;
        const uint32_t a0 = vb + lane * kRowB + x;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            uint32_t r[4];
            ldmatrix_x4_trans(r, a0 ^ (c << 4));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t a[4];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t w = r[2 * k + q];
                    if constexpr (MASKED) w &= vm[2 * k + q];
                    // (key 2t: dims d, d + 1; key 2t + 1: dims d, d + 1) -> d of both keys, d + 1 of both
                    widen4(__byte_perm(w, w, 0x3120), a[2 * q], a[2 * q + 1]);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) mma<FP8>(st.o[j][c], a, pb[j][k][0], pb[j][k][1]);
            }
        }
    } else {
        const int row = (lane & 7) + ((lane >> 4) << 3);
        const uint32_t a0 = vb + row * 128 + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            uint32_t r[4];
            ldmatrix_x4_trans(r, (a0 ^ ((2 * c & 7) << 4)) + (c >> 2) * (C::kKeys * 128));
            if constexpr (MASKED) {
                r[0] &= vm[0];
                r[1] &= vm[0];
                r[2] &= vm[1];
                r[3] &= vm[1];
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) mma<FP8>(st.o[j][c], r, pb[j][0][0], pb[j][0][1]);
        }
    }
}

// Query rows 8j + g of a tile into the score product's B operand, in the order
// the K loads give the dimensions; returns the factor that undoes the row's
// scaling (1 for bf16 pools).
template <int D, bool FP8>
__device__ __forceinline__ float load_q(const AttnParams& p, const __nv_bfloat16* q, bool exists, int t,
                                        uint32_t (&f)[D / 16][2]) {
    uint4 v[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        // 8-bit: D / 4 elements from t D / 4 on; bf16: 16 of each 64 from 16 t on
        const int at = FP8 ? t * (D / 4) + 8 * i : (i >> 1) * 64 + t * 16 + (i & 1) * 8;
        v[i] = exists ? __ldg(reinterpret_cast<const uint4*>(q + at)) : make_uint4(0u, 0u, 0u, 0u);
    }
    float undo = 1.f;
    if constexpr (FP8) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max((w[k] >> 7) & 255u, (w[k] >> 23) & 255u));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = max(top, 9u);
        const float up = __uint_as_float((262u - top) << 23);  // the largest exponent to 2^8
        undo = __uint_as_float((top - 8u) << 23);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                f[2 * i + (k >> 1)][k & 1] = pack_f16x2(bf16lo(w[k]) * up, bf16hi(w[k]) * up);
        }
    } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            f[2 * i][0] = v[i].x;
            f[2 * i][1] = v[i].y;
            f[2 * i + 1][0] = v[i].z;
            f[2 * i + 1][1] = v[i].w;
        }
    }
    return undo;
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    attn_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ RowsArgs a) {
    using C = Cfg<D, FP8, NT>;
    using W = Walk<C::kRows, C::kKeys>;
    constexpr int S = C::kStages;
    const AttnParams& p = a.p;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long scan[kWarps];
    __shared__ int begin[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.num_q_heads / p.num_kv_heads, Hkv = p.num_kv_heads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid's end

    if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle needs 1024-byte aligned tiles
        if (threadIdx.x == 0) set_err(p.err, PKV_ERRBIT_TIMEOUT);
        return;
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff) + warp * S;
    float4* meta = reinterpret_cast<float4*>(smem + C::kMetaOff) + warp * S;
    uint8_t* ring = smem + warp * S * C::kStage;
    if (lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
    }

    // ---- this CTA's share
    W cw;
    if (a.ctas == 0) {
        const int x = blockIdx.x;
        cw.mt = x % a.tiles_max;
        cw.kvh = (x / a.tiles_max) % Hkv;
        cw.b = x / a.tiles_max / Hkv;
        cw.at = 0;
        const Seq s = sequence<C::kRows>(p, cw.b, G);
        if (cw.mt >= s.tiles) return;
        cw.left = max(span_of<C::kRows, C::kKeys>(p, s, cw.mt, G).n, 1);
    } else {
        auto weight = [&](int b) {  // places of one K/V head
            const Seq s = sequence<C::kRows>(p, b, G);
            long long w = 0;
            for (int mt = 0; mt < s.tiles; ++mt) w += max(span_of<C::kRows, C::kKeys>(p, s, mt, G).n, 1);
            return w;
        };
        const int per = (p.batch + kThreads - 1) / kThreads;
        const int b0 = min(static_cast<int>(threadIdx.x) * per, p.batch), b1 = min(b0 + per, p.batch);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += weight(b) * Hkv;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        long long before = incl - mine, total = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += scan[w];
            total += scan[w];
        }
        const long long shares = min(static_cast<long long>(a.ctas), max(total / kMinShare, 1ll));
        const long long c = blockIdx.x;
        const long long from = c < shares ? total * c / shares : total;
        const long long to = c < shares ? total * (c + 1) / shares : total;
        if (from >= to) {
            if (threadIdx.x < 2) a.frag_dir[c * 2 + threadIdx.x] = make_int4(0, 0, 0, 0);
            return;
        }
        if (from >= before && from < before + mine) {
            long long rem = from - before;
            int b = b0;
            for (; b < b1; ++b) {
                const long long w = weight(b) * Hkv;
                if (rem < w) break;
                rem -= w;
            }
            const long long w = weight(b);
            begin[0] = b;
            begin[1] = static_cast<int>(rem / w);
            rem %= w;
            const Seq s = sequence<C::kRows>(p, b, G);
            int mt = 0;
            for (;; ++mt) {
                const int n = max(span_of<C::kRows, C::kKeys>(p, s, mt, G).n, 1);
                if (rem < n) break;
                rem -= n;
            }
            begin[2] = mt;
            begin[3] = static_cast<int>(rem);
        }
        __syncthreads();
        cw.b = begin[0];
        cw.kvh = begin[1];
        cw.mt = begin[2];
        cw.at = begin[3];
        cw.left = to - from;
    }

    // ---- the warp's copies: every kWarps-th chunk of every segment, in order,
    // S ahead of what it consumes
    W iw = cw;
    iw.ps = iw.pe = 0;
    int ipos = 0, ibase = 0;  // next chunk to copy; chunk of lane 0's cached page
    int my_page = 0;
    float my_ks = 1.f, my_vs = 1.f;
    int issued = 0;
    bool more = true;
    auto key_of = [](const W& w, int i) { return (i < w.u.nsc ? i : w.u.loc + i - w.u.nsc) * C::kKeys; };
    auto look_up = [&] {  // pages and scales of this warp's next 32 chunks, one a lane
        ibase = ipos;
        const int i = ipos + kWarps * lane;
        my_page = static_cast<int>(p.num_pages);  // outside the tensor: the copy fills zeros
        my_ks = my_vs = 0.f;
        if (i < iw.pe) {
            const int page = p.block_table[iw.sb * p.block_table_stride + key_of(iw, i) / kPage];
            if (page >= 0 && page < p.num_pages) {
                my_page = page;
                if constexpr (FP8) {
                    my_ks = __ldg(p.k_scale + page * p.scale_stride + iw.skvh);
                    my_vs = __ldg(p.v_scale + page * p.scale_stride + iw.skvh);
                }
            } else if (p.checked) {
                set_err(p.err, PKV_ERRBIT_PAGE);
            }
        }
    };
    auto issue = [&] {
        while (more && ipos >= iw.pe) {
            more = iw.next(p, G);
            if (more) {
                ipos = iw.ps + warp;
                if (ipos < iw.pe) look_up();
            }
        }
        if (!more) return;
        if (ipos - ibase >= 32 * kWarps) look_up();
        const int l = (ipos - ibase) / kWarps;
        const int page = __shfl_sync(0xffffffffu, my_page, l);
        const float ks = __shfl_sync(0xffffffffu, my_ks, l), vs = __shfl_sync(0xffffffffu, my_vs, l);
        if (lane == 0) {
            const int st = issued % S, key0 = key_of(iw, ipos);
            uint8_t* kd = ring + st * C::kStage;
            uint8_t* vd = kd + C::kTile;
            meta[st] = make_float4(ks, vs, __int_as_float(key0), 0.f);
            mbar_arrive_expect_tx(&bars[st], C::kStage);
            if constexpr (FP8) {
                tma_load_4d(kd, &tm_k, &bars[st], 0, iw.skvh, 0, page);
                tma_load_4d(vd, &tm_v, &bars[st], 0, iw.skvh, 0, page);
            } else {
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    tma_load_4d(kd + h * (C::kKeys * 128), &tm_k, &bars[st], h * 64, iw.skvh, key0 % kPage, page);
                    tma_load_4d(vd + h * (C::kKeys * 128), &tm_v, &bars[st], h * 64, iw.skvh, key0 % kPage, page);
                }
            }
        }
        ipos += kWarps;
        ++issued;
    };
    __syncwarp();
    for (int s = 0; s < S; ++s) issue();

    // ---- segments
    const int g = lane >> 2, t = lane & 3;
    float* red = reinterpret_cast<float*>(smem + C::kRedOff);
    float* red_m = reinterpret_cast<float*>(smem + C::kStatOff);
    float* red_l = red_m + kWarps * C::kRows;
    float* red_lb = red_l + kWarps * C::kRows;
    const uint32_t ring_u = smem_u32(ring);
    int consumed = 0;
    bool dead = false;
    int4 dir0 = make_int4(0, 0, 0, 0), dir1 = dir0;
    int nseg = 0;
    for (; cw.next(p, G); ++nseg) {
        const int R0 = cw.smt * C::kRows;
        const Seq& s = cw.s;
        if (p.checked && threadIdx.x == 0 && cw.starts && cw.skvh == 0 && cw.smt == 0) {
            const int rows = p.q_indptr[cw.sb + 1] - s.r0, kv = p.kv_lens[cw.sb];
            if (kv > p.max_kv_len || kv < 0 || rows > p.max_q_rows || (p.q_real && p.q_real[cw.sb] > rows))
                set_err(p.err, PKV_ERRBIT_LEN);
        }
        RowInfo<NT> ri;
        uint32_t qf[NT][D / 16][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int R = R0 + 8 * j + g;
            const int tok = R / G, h = cw.skvh * G + R % G;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                                     static_cast<int64_t>(s.r0 + tok) * p.q_token_stride +
                                     static_cast<int64_t>(h) * p.q_head_stride;
            const float undo = load_q<D, FP8>(p, q, tok < s.nrows, t, qf[j]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ri.fq[j][e] = p.scale_log2;
                if constexpr (FP8) ri.fq[j][e] *= __shfl_sync(0xffffffffu, undo, (2 * t + e) * 4);
                const int tk = (R0 + 8 * j + 2 * t + e) / G;
                ri.lim[j][e] = tk < s.qreal ? row_limit(p, tk, s.qreal, s.kv_len) : 0;
                ri.lo[j][e] = p.window > 0 ? s.kv_len - s.qreal + tk - p.window + 1 : 0;
            }
        }
        {
            const int tf = R0 / G, tl = min((R0 + C::kRows - 1) / G, s.qreal - 1);
            ri.all_end = tf < s.qreal ? row_limit(p, tf, s.qreal, s.kv_len) : 0;
            ri.all_lo = p.window > 0 ? max(0, s.kv_len - s.qreal + tl - p.window + 1) : 0;
            ri.any_lo = cw.u.lo;
            ri.any_end = cw.u.hi;
            ri.sinks = p.num_sinks;
        }
        State<D, NT> st;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                st.m[j][e] = -INFINITY;
                st.l[j][e] = st.lb[j][e] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.o[j][c][e] = 0.f;
        }
        for (int pos = cw.ps + warp; pos < cw.pe && !dead; pos += kWarps) {
            const int sg = consumed % S;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars[sg], (consumed / S) & 1))) {
                if (lane == 0) set_err(p.err, PKV_ERRBIT_TIMEOUT);
                dead = true;
                break;
            }
            const float4 me = meta[sg];
            const int key0 = __float_as_int(me.z);
            const uint32_t kb = ring_u + sg * C::kStage;
            const bool whole = key0 + C::kKeys <= ri.all_end &&
                               (key0 >= ri.all_lo || key0 + C::kKeys <= ri.sinks);
            if (whole) chunk_step<D, FP8, NT, false>(st, qf, ri, kb, kb + C::kTile, me.x, me.y, key0, lane);
            else chunk_step<D, FP8, NT, true>(st, qf, ri, kb, kb + C::kTile, me.x, me.y, key0, lane);
            __syncwarp();
            ++consumed;
            issue();
        }
        // ---- join the warps' states, four rows at a time
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    st.l[j][e] += __shfl_xor_sync(0xffffffffu, st.l[j][e], o);
                    if constexpr (!FP8) st.lb[j][e] += __shfl_xor_sync(0xffffffffu, st.lb[j][e], o);
                }
                if (g == 0) {
                    const int r = warp * C::kRows + 8 * j + 2 * t + e;
                    red_m[r] = st.m[j][e];
                    red_l[r] = st.l[j][e];
                    if constexpr (!FP8) red_lb[r] = st.lb[j][e];
                }
            }
        const bool whole_unit = cw.starts && cw.ends;
        const int slot = nseg == 0 ? 0 : 1;
        if (!whole_unit) {
            const int4 x = make_int4(cw.sb, cw.skvh, cw.smt,
                                     kFragValid | (cw.starts ? kFragStarts : 0) | (cw.ends ? kFragEnds : 0));
            if (slot == 0) dir0 = x;
            else dir1 = x;
        }
        const int rows_here = min(C::kRows, s.nrows * G - R0);
#pragma unroll
        for (int rg = 0; rg < C::kRows / 4; ++rg) {
            if (4 * rg < rows_here) {
                if ((t >> 1) == (rg & 1)) {
                    constexpr int RS = C::kRedStride;
                    float* r0 = red + (warp * 4 + 2 * (t & 1)) * RS;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const float(&o)[4] = st.o[rg >> 1][c];
                        if constexpr (FP8) {
                            *reinterpret_cast<float2*>(r0 + 16 * c + 2 * g) = make_float2(o[0], o[2]);
                            *reinterpret_cast<float2*>(r0 + RS + 16 * c + 2 * g) = make_float2(o[1], o[3]);
                        } else {
                            r0[16 * c + g] = o[0];
                            r0[16 * c + 8 + g] = o[2];
                            r0[RS + 16 * c + g] = o[1];
                            r0[RS + 16 * c + 8 + g] = o[3];
                        }
                    }
                }
                __syncthreads();
                for (int e = threadIdx.x; e < 4 * D / 2; e += kThreads) {
                    const int rr = e / (D / 2), d = (e - rr * (D / 2)) * 2;
                    const int r = 4 * rg + rr;
                    if (r >= rows_here) continue;
                    const int tok = (R0 + r) / G, h = cw.skvh * G + (R0 + r) % G;
                    float M = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_m[w * C::kRows + r]);
                    float L = 0.f, Lb = 0.f;
                    float2 O = make_float2(0.f, 0.f);
                    if (M != -INFINITY && tok < s.qreal) {
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) {
                            const float f = fast_exp2(red_m[w * C::kRows + r] - M);
                            const float2 o = *reinterpret_cast<const float2*>(red + (w * 4 + rr) * C::kRedStride + d);
                            L = fmaf(f, red_l[w * C::kRows + r], L);
                            if constexpr (!FP8) Lb = fmaf(f, red_lb[w * C::kRows + r], Lb);
                            O.x = fmaf(f, o.x, O.x);
                            O.y = fmaf(f, o.y, O.y);
                        }
                    }
                    // bf16 weights: normalised by the sum of the rounded ones
                    const float div = FP8 ? L : Lb;
                    const float inv = div > 0.f ? 1.0f / div : (div == div ? 0.f : div);
                    O.x *= inv;
                    O.y *= inv;
                    const float lse = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
                    if (whole_unit) {
                        const int64_t ot = static_cast<int64_t>(s.r0 + tok) * p.num_q_heads + h;
                        if (p.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + ot * D + d) = O;
                        else
                            *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + ot * D + d) =
                                pack_bf16x2(O.x, O.y);
                        if (p.lse && d == 0) p.lse[ot] = lse;
                    } else {
                        const int64_t fr = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * C::kRows + r;
                        *reinterpret_cast<float2*>(a.frag_o + fr * D + d) = O;
                        if (d == 0) a.frag_lse[fr] = lse;
                    }
                }
                __syncthreads();
            }
        }
    }
    if (a.ctas > 0 && threadIdx.x < 2)
        a.frag_dir[static_cast<int64_t>(blockIdx.x) * 2 + threadIdx.x] = threadIdx.x == 0 ? dir0 : dir1;
    // after a wait that gave up: leave with no copy in flight
    for (int j = consumed; j < issued; ++j) mbar_wait(&bars[j % S], (j / S) & 1);
}

// Joins the partial states of the units cut between CTAs.  Block (c, r): the
// unit that starts in CTA c and goes on behind it, row r; its pieces are CTA
// c's last and the first of c + 1, c + 2, ... up to the one that ends it.
template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads) attn_rows_join_kernel(const __grid_constant__ RowsArgs a) {
    constexpr int DPL = D / 32;
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    const AttnParams& p = a.p;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x, r = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int slot = -1;
    int4 u = make_int4(0, 0, 0, 0);
    for (int s = 0; s < 2; ++s) {
        const int4 x = a.frag_dir[c * 2 + s];
        if ((x.w & kFragValid) && (x.w & kFragStarts) && !(x.w & kFragEnds)) {
            slot = s;
            u = x;
        }
    }
    if (slot < 0) return;
    const int G = p.num_q_heads / p.num_kv_heads;
    const int R = u.z * ROWS + r;
    const int r0 = p.q_indptr[u.x];
    const int nrows = min(p.q_indptr[u.x + 1] - r0, p.max_q_rows);
    const int tok = R / G, h = u.y * G + R % G;
    if (tok >= nrows) return;
    int n = 1;  // pieces: c's, then the first ones of the CTAs behind it
    while (c + n < a.ctas) {
        const int4 x = a.frag_dir[(c + n) * 2];
        ++n;
        if (!(x.w & kFragValid) || (x.w & kFragEnds)) break;
    }
    float M = -INFINITY, L = 0.f, O[DPL];
#pragma unroll
    for (int i = 0; i < DPL; ++i) O[i] = 0.f;
    constexpr int kAhead = 4;
    for (int k0 = warp; k0 < n; k0 += kWarps * kAhead) {
        float lv[kAhead], ov[kAhead][DPL];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int k = k0 + x * kWarps;
            lv[x] = -INFINITY;
            if (k < n) {
                const int64_t fr = (static_cast<int64_t>(c + k) * 2 + (k == 0 ? slot : 0)) * ROWS + r;
                lv[x] = __ldcg(a.frag_lse + fr);
#pragma unroll
                for (int i = 0; i < DPL; ++i) ov[x][i] = __ldcg(a.frag_o + fr * D + lane * DPL + i);
            }
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            if (lv[x] == -INFINITY) continue;
            const float Mn = fmaxf(M, lv[x]);
            const float f = __expf(M - Mn), w = __expf(lv[x] - Mn);
            L = fmaf(L, f, w);
#pragma unroll
            for (int i = 0; i < DPL; ++i) O[i] = fmaf(w, ov[x][i], O[i] * f);
            M = Mn;
        }
    }
    if (lane == 0) {
        sm[warp] = M;
        sl[warp] = L;
    }
#pragma unroll
    for (int i = 0; i < DPL; ++i) so[warp][lane * DPL + i] = O[i];
    __syncthreads();
    if (threadIdx.x >= D) return;
    const int d = threadIdx.x;
    M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float l = 0.f, o = 0.f;
    if (M != -INFINITY) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = __expf(sm[w] - M);
            l = fmaf(f, sl[w], l);
            o = fmaf(f, so[w][d], o);
        }
    }
    o *= l == 0.f ? 0.f : 1.0f / l;
    const int64_t ot = static_cast<int64_t>(r0 + tok) * p.num_q_heads + h;
    if (p.out_f32) static_cast<float*>(p.out)[ot * D + d] = o;
    else static_cast<__nv_bfloat16*>(p.out)[ot * D + d] = __float2bfloat16_rn(o);
    if (p.lse && d == 0) p.lse[ot] = l == 0.f ? -INFINITY : M + __logf(l);
}

template <int D, bool FP8, int NT>
cudaError_t launch_rows(RowsArgs a, const RowsPlan& pl, const void* tk, const void* tv, cudaStream_t s) {
    using C = Cfg<D, FP8, NT>;
    auto kern = attn_rows_kernel<D, FP8, NT>;
    static DeviceOnce opted;
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = opted.get(dev, &done, [&](int, int* v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
    });
    if (e != cudaSuccess) return e;
    const CUtensorMap &mk = *static_cast<const CUtensorMap*>(tk), &mv = *static_cast<const CUtensorMap*>(tv);
    const unsigned grid = static_cast<unsigned>(a.ctas > 0 ? a.ctas : a.tiles_max * a.p.num_kv_heads * a.p.batch);
    kern<<<grid, kThreads, C::kBytes, s>>>(mk, mv, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.ctas == 0) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.ctas), C::kRows);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_rows_join_kernel<D, C::kRows>, a);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// One CTA a unit while a unit is short (kDirectKeys keys at the host bound, a
// few chunks a warp); beyond that the cut line.
RowsPlan plan_attn_rows(int batch, int max_q_rows, int Hq, int Hkv, int D, int max_kv_len, int window,
                        int num_sinks, bool fp8, int sms) {
    constexpr int kDirectKeys = 512;
    RowsPlan pl{};
    const int64_t rows = static_cast<int64_t>(max_q_rows) * (Hq / Hkv);
    pl.row_tiles = rows <= 8 ? 1 : 2;
    const int R = 8 * pl.row_tiles;
    pl.tiles = (rows + R - 1) / R;
    int64_t keys = max_kv_len;
    if (window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(window) + R + std::min(num_sinks, max_kv_len) + 62);
    const int64_t units = pl.tiles * Hkv * batch;
    (void)fp8;
    if (keys <= kDirectKeys && units < (1ll << 31)) return pl;
    pl.ctas = kCtasPerSm * sms;
    pl.ws_bytes = align256(static_cast<size_t>(pl.ctas) * 2 * sizeof(int4)) +
                  align256(static_cast<size_t>(pl.ctas) * 2 * R * sizeof(float)) +
                  align256(static_cast<size_t>(pl.ctas) * 2 * R * D * sizeof(float));
    return pl;
}

cudaError_t launch_attn_rows(const AttnParams& p, const RowsPlan& pl, void* workspace, const void* tk,
                             const void* tv, cudaStream_t s) {
    RowsArgs a{};
    a.p = p;
    a.ctas = pl.ctas;
    a.tiles_max = static_cast<int>(std::min<int64_t>(pl.tiles, 0x7fffffff));
    if (pl.ctas > 0) {
        char* w = static_cast<char*>(workspace);
        const size_t R = 8 * pl.row_tiles;
        a.frag_dir = reinterpret_cast<int4*>(w);
        w += align256(static_cast<size_t>(pl.ctas) * 2 * sizeof(int4));
        a.frag_lse = reinterpret_cast<float*>(w);
        w += align256(static_cast<size_t>(pl.ctas) * 2 * R * sizeof(float));
        a.frag_o = reinterpret_cast<float*>(w);
    }
#define PKV_ROWS(D_, F_, N_) \
    if (p.head_dim == D_ && p.kv_fp8 == F_ && pl.row_tiles == N_) return launch_rows<D_, F_, N_>(a, pl, tk, tv, s);
    PKV_ROWS(128, true, 1) PKV_ROWS(128, true, 2) PKV_ROWS(128, false, 1) PKV_ROWS(128, false, 2)
    PKV_ROWS(64, true, 1) PKV_ROWS(64, true, 2) PKV_ROWS(64, false, 1) PKV_ROWS(64, false, 2)
#undef PKV_ROWS
    return cudaErrorInvalidValue;
}

}  // namespace pkv
