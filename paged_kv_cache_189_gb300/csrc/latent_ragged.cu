// latent_ragged.cu -- ragged_attention_latent on the tensor cores (tcgen05 /
// TMEM, TMA-fed): prompts over keys of 128 + 64 elements and values of 128.
//
//   S = Q K^T over 192 elements, P = 2^(S scale - m), O += P V, out = O / sum P
// A call is bound by the matrix rate: 640 flops a (row, key, head) against 640
// bytes a (key, head), shared by all rows of a sequence.
//
// One CTA takes two tiles of 128 query rows (A, B) of one head, so that one
// tile's softmax runs beside the other's products; both use every key tile (128
// keys).  P overlays S in TMEM and is the A operand of P V from there, which
// leaves shared memory to the two Q tiles (96 KB) and a ring of eight 16 KB blocks
// of 64 columns: a key tile is five of them (two of K's own part, the rotary
// one, two of V), which the ring takes in the order of use, K_0 V_0 K_1 V_1 ....
// TMEM columns: S_A 0, O_A 128, S_B 256, O_B 384.
//
// Measured (four prompts of 1500-2048 tokens over 2048-4096 keys, 32 heads, 303
// GFLOP visible): 257 us, 1.18 PFLOP/s, 0.62 of the bf16 rate.  A key tile takes
// ~3700 cycles for 2560 of products: the chain scores, softmax (~1550 cycles for a
// row's 128 keys in one thread), P V of one tile is longer than the other tile's
// products, and S reads both operands from shared memory at all of its bandwidth.
// Not kept: two threads a row (294 us), no running maximum but a check of the
// weights' sum (282), CTAs that take over waiting ones by cluster launch control (+2 %).
//
// Roles (320 threads): warps 0-3 softmax of tile A, 4-7 of tile B, one thread a
// row; warp 8 the TMA producer, warp 9 the MMA issuer.  Waits give up after ~2 s.
#include <cuda.h>

#include "latent.h"
#include "tc.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 320;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kRows = 128;             // query rows of a tile
constexpr int kKeys = 128;             // keys of a tile
constexpr int kBlock = 128 * 128;      // 128 rows x 64 columns
constexpr int kQTile = 3 * kBlock;
constexpr int kRing = 8;
constexpr int kRingOff = 2 * kQTile;
constexpr int kBarOff = kRingOff + kRing * kBlock;
constexpr int kNumBars = 1 + 4 * 2 + 3 * 2 + 1;
constexpr int kSlotOff = kBarOff + kNumBars * 8;
constexpr int kSmemBytes = kSlotOff + 16;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
constexpr float kLazyRescale = 8.0f;   // move a row's reference only past 2^8 growth

struct Geom {
    int r0, k0, nrows, kv, t0;
    int nt[2];   // key tiles of tile A and tile B (0: no rows, or none sees a key)
    int key_hi;  // keys that the pair's last row sees
};

__device__ __forceinline__ int row_limit(const RaggedParams& p, const Geom& g, int i) {
    if (i >= g.nrows) return 0;
    return p.causal ? max(0, g.kv - g.nrows + i + 1) : g.kv;
}

// Block q of the ring's sequence sits in slot q mod 8; tile j's are 5 j ... 5 j + 4.
// V's two blocks in ascending slots, so that the second lies a positive distance on.
struct ValueSlots {
    int lo, hi;
};
__device__ __forceinline__ ValueSlots value_slots(int j) {
    const int a = (5 * j + 3) & 7, b = (5 * j + 4) & 7;
    return {min(a, b), max(a, b)};
}

__global__ void __launch_bounds__(kThreads, 1)
    ragged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_pe,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
                       const RaggedParams p, const bool q_boxes) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    const int h = blockIdx.y, b = blockIdx.z;

    Geom g;
    g.r0 = p.q_indptr[b];
    const int rows = p.q_indptr[b + 1] - g.r0;
    g.nrows = min(rows, p.max_q_rows);
    g.k0 = p.kv_indptr[b];
    const int kv_all = p.kv_indptr[b + 1] - g.k0;
    g.kv = min(max(kv_all, 0), p.max_kv_len);
    // the last rows see most keys: their pairs go first
    g.t0 = static_cast<int>(gridDim.x - 1 - blockIdx.x) * 2 * kRows;
    if (p.checked && threadIdx.x == 0 && blockIdx.x == 0 && h == 0 &&
        (kv_all > p.max_kv_len || kv_all < 0 || rows > p.max_q_rows || g.k0 < 0 || g.k0 + int64_t(kv_all) > p.num_keys))
        set_err(p.err, PKV_ERRBIT_LEN);
    if (g.t0 >= g.nrows) return;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int first = g.t0 + x * kRows, last = min(first + kRows, g.nrows) - 1;
        g.nt[x] = first < g.nrows ? (row_limit(p, g, last) + kKeys - 1) / kKeys : 0;
    }
    g.key_hi = row_limit(p, g, min(g.t0 + 2 * kRows, g.nrows) - 1);
    const int nt = max(g.nt[0], g.nt[1]);

    auto whole_tile = [&](int x) { return q_boxes && g.t0 + (x + 1) * kRows <= g.nrows; };

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
    uint64_t* q_ready = bars;
    uint64_t* k_full = bars + 1;      // [2], by tile parity
    uint64_t* k_empty = k_full + 2;
    uint64_t* v_full = k_empty + 2;
    uint64_t* v_empty = v_full + 2;
    uint64_t* s_full = v_empty + 2;   // [2], by row tile
    uint64_t* p_full = s_full + 2;
    uint64_t* o_full = p_full + 2;
    uint64_t* mma_done = o_full + 2;
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kSlotOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSlotOff + 4);
    if (threadIdx.x == 0) {
        mbar_init(q_ready, (whole_tile(0) ? 1 : kRows) + (whole_tile(1) ? 1 : kRows));
        for (int x = 0; x < 2; ++x) {
            mbar_init(&k_full[x], 1);
            mbar_init(&k_empty[x], 1);
            mbar_init(&v_full[x], 1);
            mbar_init(&v_empty[x], 1);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], kRows);
            mbar_init(&o_full[x], 1);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tc_alloc(slot, 512);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *slot, sbase = smem_u32(smem);
    const bool aligned = (sbase & 1023u) == 0;  // the swizzles need it
    if (!aligned && threadIdx.x == 0) set_err(p.err, PKV_ERRBIT_TIMEOUT);

    // a completed phase passes at once; after one wait gave up, the others do not wait
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity)) return true;
        *abort_flag = 1;
        set_err(p.err, PKV_ERRBIT_TIMEOUT);
        return false;
    };

    if (warp == kProducerWarp) {
        // ============================ producer ==============================
        // K_j lies where V_{j-2} (and the end of K_{j-2}) was, V_j where K_{j-1} began
        if (aligned && elect_one()) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_pe);
            prefetch_tmap(&tm_v);
            auto at = [&](int s) { return smem + kRingOff + s * kBlock; };
            int nk = 0, nv = 0;
            // a row tile that lies whole inside the sequence: three boxes
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (nt == 0 || !whole_tile(x)) continue;
                mbar_arrive_expect_tx(q_ready, kQTile);
                for (int c = 0; c < 3; ++c)
                    tma_load_3d(smem + x * kQTile + c * kBlock, &tm_q, q_ready, c * 64, h, g.r0 + g.t0 + x * kRows);
            }
            for (int j = 0; j < nt; ++j) {
                const int key = g.k0 + j * kKeys, x = j & 1;
                const uint32_t again = ((j >> 1) & 1) ^ 1;  // the phase that tile j - 2 completed
                if (j >= 2 && !(wait(&v_empty[x], again) && wait(&k_empty[x], again))) break;
                mbar_arrive_expect_tx(&k_full[x], 3 * kBlock);
                tma_load_3d(at((5 * j) & 7), &tm_k, &k_full[x], 0, h, key);
                tma_load_3d(at((5 * j + 1) & 7), &tm_k, &k_full[x], 64, h, key);
                tma_load_2d(at((5 * j + 2) & 7), &tm_pe, &k_full[x], 0, key);
                ++nk;
                if (j >= 1 && !wait(&k_empty[x ^ 1], ((j - 1) >> 1) & 1)) break;
                const ValueSlots vs = value_slots(j);
                mbar_arrive_expect_tx(&v_full[x], 2 * kBlock);
                tma_load_3d(at(vs.lo), &tm_v, &v_full[x], 0, h, key);
                tma_load_3d(at(vs.hi), &tm_v, &v_full[x], 64, h, key);
                ++nv;
            }
            // do not leave with copies into this CTA's shared memory in flight
            for (int j = max(0, nk - 2); j < nk; ++j) mbar_wait(&k_full[j & 1], (j >> 1) & 1);
            for (int j = max(0, nv - 2); j < nv; ++j) mbar_wait(&v_full[j & 1], (j >> 1) & 1);
            if (nt > 0) mbar_wait(q_ready, 0);
        }
    } else if (warp == kMmaWarp) {
        // =============================== MMA ================================
        if (aligned && elect_one()) {
            constexpr uint32_t kIdescS = tc_idesc(kRows, kKeys, false, false);
            constexpr uint32_t kIdescO = tc_idesc(kRows, kExpandedV, false, true);
            const uint64_t dq = tc_desc(sbase, 16, 1024, 128), dk = tc_desc(sbase + kRingOff, 16, 1024, 128);
            bool ok = nt == 0 || wait(q_ready, 0);
            auto scores = [&](int x, int j, auto&& mid) {
                tc_after_sync();
                const uint64_t da = dq + x * (kQTile >> 4);
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    const uint64_t db = dk + ((5 * j + c) & 7) * (kBlock >> 4);
                    if (c == 2) mid();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma(tmem + x * 256, da + ((c * kBlock + kk * 32) >> 4), db + 2 * kk, kIdescS, c + kk > 0);
                }
                tc_commit(&s_full[x]);
            };
            auto values = [&](int x, int j, auto&& mid) {
                tc_after_sync();
                const ValueSlots vs = value_slots(j);
                const uint64_t db = tc_desc(sbase + kRingOff + vs.lo * kBlock, (vs.hi - vs.lo) * kBlock, 1024, 128);
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk) {  // 16 keys: 8 columns of packed P, 16 rows of V
                    if (kk == 4) mid();
                    tc_mma_ts(tmem + x * 256 + 128, tmem + x * 256 + kk * 8, db + kk * (2048 >> 4), kIdescO, j + kk > 0);
                }
            };
            // a copy's barrier is probed among the products before its use: a wait
            // between two batches would leave the pipe idle
            bool landed = false;
            auto probe = [&](uint64_t* bar, uint32_t parity) { landed = mbar_test(bar, parity); };
            auto settle = [&](uint64_t* bar, uint32_t parity) { return landed || wait(bar, parity); };
            if (ok && nt > 0) {
                ok = wait(&k_full[0], 0);
                if (g.nt[0] > 0) scores(0, 0, [] {});
                if (g.nt[1] > 0) scores(1, 0, [] {});
                tc_commit(&k_empty[0]);
                probe(&v_full[0], 0);
            }
            for (int j = 0; ok && j < nt; ++j) {
                const uint32_t ph = (j >> 1) & 1, ph1 = ((j + 1) >> 1) & 1;
                const int x1 = (j + 1) & 1;
                bool fresh = true;  // the step's first tile: its V_j, then its K_{j+1} may not have landed
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!ok || j >= g.nt[x]) continue;
                    ok = (!fresh || settle(&v_full[j & 1], ph)) && wait(&p_full[x], j & 1);
                    if (!ok) break;
                    values(x, j, [&] {
                        if (fresh && j + 1 < nt) probe(&k_full[x1], ph1);
                    });
                    if (x == 1 || j >= g.nt[1]) tc_commit(&v_empty[j & 1]);
                    if (j + 1 < g.nt[x]) {
                        ok = !fresh || settle(&k_full[x1], ph1);
                        fresh = false;
                        if (ok) scores(x, j + 1, [&] {
                            if (x == 1 || j + 1 >= g.nt[1]) probe(&v_full[x1], ph1);
                        });
                    } else {
                        tc_commit(&o_full[x]);
                    }
                }
                if (j + 1 < nt) tc_commit(&k_empty[x1]);
            }
            // nothing of this thread's still runs in the tensor pipe when the CTA
            // winds down (after a failed wait the last products may)
            tc_commit(mma_done);
            if (!mbar_wait(mma_done, 0)) set_err(p.err, PKV_ERRBIT_TIMEOUT);
        }
    } else {
        // ============================= softmax ==============================
        const int x = warp >> 2, r = threadIdx.x & (kRows - 1);
        const int i = g.t0 + x * kRows + r;
        const bool exists = i < g.nrows;
        const int limit = row_limit(p, g, i);
        const uint32_t s_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + x * 256, o_addr = s_addr + 128;
        if (nt > 0 && !whole_tile(x)) {
            // 24 chunks a row; eight lanes take one row's neighbouring chunks together
            const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(g.r0) * p.q_token_stride +
                                        static_cast<int64_t>(h) * p.q_head_stride;
#pragma unroll 4
            for (int k = 0; k < 24; ++k) {
                const int idx = k * kRows + r, row = idx / 24, ch = idx - row * 24, ri = g.t0 + x * kRows + row;
                copy16_async(sbase + x * kQTile + (ch >> 3) * kBlock + sw128_offset(row, ch & 7),
                             base + (ri < g.nrows ? ri * p.q_token_stride + ch * 8 : 0), ri < g.nrows);
            }
            copy_async_wait();
            fence_proxy_async_smem();
            mbar_arrive(q_ready);
        }
        float m = -INFINITY, l = 0.f;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        for (int j = 0; aligned && j < g.nt[x]; ++j) {
            wait(&s_full[x], j & 1);
            __syncwarp();
            tc_after_sync();
            uint32_t sv[kKeys];  // the row's scores, then its packed weights
            tc_load128(s_addr, sv);
            const int nvis = limit - j * kKeys;
            if (__any_sync(0xffffffffu, nvis < kKeys)) {
#pragma unroll
                for (int e = 0; e < kKeys; ++e) sv[e] = e < nvis ? sv[e] : __float_as_uint(-INFINITY);
            }
            float a[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) a[q] = __uint_as_float(sv[q]);
#pragma unroll
            for (int e = 8; e < kKeys - 8; e += 16) {
#pragma unroll
                for (int q = 0; q < 8; ++q) a[q] = max3(a[q], __uint_as_float(sv[e + q]), __uint_as_float(sv[e + 8 + q]));
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) a[q] = fmaxf(a[q], __uint_as_float(sv[kKeys - 8 + q]));
            const float mx = max3(max3(a[0], a[1], a[2]), max3(a[3], a[4], a[5]), fmaxf(a[6], a[7])) * p.scale_log2;
            float alpha = 1.f;
            if (mx > m + kLazyRescale) {   // also the first time a key is visible
                alpha = fast_exp2(m - mx);  // 0 when m was -inf
                m = mx;
            }
            const float nm = m == -INFINITY ? 0.f : -m;
            const float2 nm2 = make_float2(nm, nm);
            // weights, rounded to bf16 for the product; the sum takes them unrounded, for
            // the output's divisor too: roundings to nearest are off to either side, and a
            // second sum of the rounded ones cost 5 % of the kernel (277 against 264 us for
            // four prompts).  Keys 2 k, 2 k + 1 land in sv[k].
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kKeys / 2; ++k) {
                const float2 y = __ffma2_rn(make_float2(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1])), sc2, nm2);
                const float2 w = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                sv[k] = pack_bf16x2(w.x, w.y);
                sum = __fadd2_rn(sum, w);
            }
            tc_store32(s_addr, sv);
            tc_store32(s_addr + 32, sv + 32);
            if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                // (the previous tile's products were done before these scores)
#pragma unroll
                for (int c = 0; c < kExpandedV / 32; ++c) {
                    uint32_t o[32];
                    tc_load32(o_addr + c * 32, o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tc_store32(o_addr + c * 32, o);
                }
            }
            tc_wait_store();
            l = l * alpha + (sum.x + sum.y);
            // V rows of keys that no row of the pair sees may hold anything: zeros,
            // before the tile's first product (tile A's where it has this key tile)
            if ((j + 1) * kKeys > g.key_hi && (x == 0 || j >= g.nt[0])) {
                wait(&v_full[j & 1], (j >> 1) & 1);
                const ValueSlots vs = value_slots(j);
                if (j * kKeys + r >= g.key_hi) {
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        *reinterpret_cast<uint4*>(smem + kRingOff + (c < 8 ? vs.lo : vs.hi) * kBlock + sw128_offset(r, c & 7)) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tc_before_sync();
            mbar_arrive(&p_full[x]);
        }
        // ---- the row's output
        const bool any = l != 0.f;  // (NaN stays)
        const float inv = any ? 1.0f / l : 0.f;
        const int64_t st = static_cast<int64_t>(g.r0 + i) * p.heads + h;
        if (g.nt[x] > 0 && aligned) wait(&o_full[x], 0);
        __syncwarp();
        tc_after_sync();
        if (p.lse && exists) p.lse[st] = any ? (m + __log2f(l)) * kLn2 : -INFINITY;
#pragma unroll
        for (int c = 0; c < kExpandedV / 32; ++c) {
            uint32_t o[32];
            tc_load32(o_addr + c * 32, o);
            float f[32];
            // (without a key tile the accumulators hold nothing of this call)
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = g.nt[x] > 0 ? __uint_as_float(o[e]) * inv : 0.f;
            if (exists && p.out_f32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + st * kExpandedV + c * 32);
#pragma unroll
                for (int q = 0; q < 8; ++q) dst[q] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
            } else if (exists) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + st * kExpandedV + c * 32);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    dst[q] = make_uint4(pack_bf16x2(f[8 * q], f[8 * q + 1]), pack_bf16x2(f[8 * q + 2], f[8 * q + 3]),
                                        pack_bf16x2(f[8 * q + 4], f[8 * q + 5]), pack_bf16x2(f[8 * q + 6], f[8 * q + 7]));
            }
        }
    }

    __syncwarp();
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == kMmaWarp) tc_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_ragged_attn(const RaggedParams& p, const void* tmap_k, const void* tmap_pe, const void* tmap_v,
                               const void* tmap_q, bool q_boxes, cudaStream_t s) {
    static DeviceOnce opted;
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = opted.get(dev, &done, [&](int, int* v) {
        *v = 1;
        return cudaFuncSetAttribute(ragged_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    // a sequence's pairs run together and share its K and V in L2
    const dim3 grid(static_cast<unsigned>((p.max_q_rows + int64_t(2 * kRows) - 1) / (2 * kRows)), p.heads, p.batch);
    ragged_attn_kernel<<<grid, kThreads, kSmemBytes, s>>>(*static_cast<const CUtensorMap*>(tmap_k),
                                                          *static_cast<const CUtensorMap*>(tmap_pe),
                                                          *static_cast<const CUtensorMap*>(tmap_v),
                                                          *static_cast<const CUtensorMap*>(tmap_q), p, q_boxes);
    return cudaGetLastError();
}

}  // namespace pkv
