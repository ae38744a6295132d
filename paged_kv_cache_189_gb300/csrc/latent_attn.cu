// latent_attn.cu -- paged_attention_latent on the tensor cores (tcgen05 / TMEM,
// TMA-fed): every head reads the same latent rows, so a sequence's (query row,
// head) pairs are the columns of two matrix products with the keys as rows:
//   S^T [64 keys x N] = C [64 x 576] Q^T,   O^T [512 x N] += C[:, :512]^T P^T
// over 64-key tiles (two pages) with a running maximum and sum per column.
//
// Keys stand in the M dimension because a decode step has few columns (16 heads
// shared out over GPUs, 128 on one) and TMEM has no room for 128 rows of O beside
// S (128 x 512 f32 is all of it), while O^T takes 4 N columns.  A latent tile is
// read from DRAM once and used twice from shared memory: K-major for S^T, and as
// the same bytes MN-major for O^T.
//
// A CTA holds N = 16, 32 or 64 columns; more are held by a pair of neighbouring CTAs,
// which walk the same tiles side by side, each with copies of its own: a tile comes
// from DRAM for the first and from L2 for the second.  (One page a CTA, copied into
// both: 100.8 us against 99.8 for 128 columns, 195 against 191 for a prompt chunk.  The
// pair as a cluster without that: 99.5 and 192.5.)  The tiles of all units (a unit is a
// column group of a sequence) are one line that the workers (CTAs, or pairs of them)
// share out evenly, each unit's tiles behind a few more places that stand for what
// beginning it costs.  A worker goes through its share segment by segment (a
// segment is a range of one unit's tiles) and leaves a partial state where a unit
// was cut; a second launch joins those.
//
// What bounds it (64 sequences of 513-8193 keys, among others, us; floor = bytes at
// the copy rate): 16 columns 66 (50): DRAM for ~55 of them, then 2.5 us before the
// first copy, shares that end up to 4 us apart, 5 us launch and join; 64 columns 81
// (53) and 128 on pairs 100 (49): a tile's buffers are held through S^T, softmax
// and O^T (~4000 cycles) and shared memory holds two tiles beside 64 columns of Q,
// and each tile takes 36 x 32 + 16 x 48 = 1920 cycles of products (measured:
// 64 x 64 x 16 products issue every 32 cycles, 128 x 64 x 16 every 48).
//
// Roles (one CTA an SM): four softmax and output warps (eight for 64 columns: the
// softmax of a tile is part of the time its buffers are held), then the TMA
// producer, the issuers of S^T and of O^T (a wait costs an issuing thread the time
// of four small products, so each hides the other's) and the loader of the next
// segment's queries, which runs beside the last one's softmax and outputs.  Every
// wait gives up after ~2 s.
#include <cuda.h>

#include "latent.h"
#include "tc.cuh"

namespace pkv {
namespace {

constexpr int kKeys = 64;                  // keys of a tile
constexpr int kHalf = kKeys * 128;         // 64 keys x 64 dims
constexpr int kBlock = 2 * kHalf;          // 64 keys x 128 dims
constexpr int kBlocks = kLatentDim / 128;  // value blocks of a tile (the rotary half block is apart)
constexpr int kRopeBlock = kLatentDim / 64;
constexpr float kLazyRescale = 8.0f;       // move a column's reference only past 2^8 growth
constexpr int kNoPage = -2;                // look-up past the last page: zeros, and no error
// Tiles a worker takes at least: one sequence of 8192 keys takes 15.8 / 14.0 / 14.4 / 16.9
// us with 1 / 2 / 4 / 8, four of 500-1500 keys 12.3 / 13.6 / 14.7 / 18.1, two short ones (shared
// out) 10.3 / 8.7 / 11.4 / 11.6
constexpr int kMinShare = 2;
// What a segment costs beside its tiles (queries, first copies, outputs), in tiles.  With
// 0 / 1 / 3 and 0 / 2 / 5: 66.6 / 65.9 / 66.3 us (16 columns), 85.4 / 81.3 / 81.0 (64), 103.2 / 100.1 / 100.4 (128)
constexpr int kToll = 1, kTollWide = 2;
// Units of at most kWholeTiles tiles (at the host's bound) that all run at once go one
// to a worker, without shares and join, where that leaves no more than kIdleTiles of a
// unit's time idle over all workers.  Shares and join / one to a worker, us: two
// sequences of 128 / 256 / 512 / 1024 keys, 16 heads 8.5 / 7.3, 10.8 / 9.0, 11.5 / 12.3, 11.7 / 19.2,
// 128 heads 11.0 / 9.7, 15.7 / 12.2, 17.0 / 16.8, 17.6 / 26.0; 64 sequences of half to all of
// 512 / 1024 keys, 16 heads 19.4 / 14.7, 24.1 / 23.8, 128 heads 34.4 / 21.6, 41.7 / 31.5.  The bound is
// the host's: a captured step that passes the cache's cap takes shares at every length
constexpr int kWholeTiles = 16, kIdleTiles = 8;

// Shared memory: the queries, rings of value blocks and of rotary blocks, the
// weights of two tiles.  N = 64 leaves room for two tiles exactly.
template <int N>
struct Dim {
    static constexpr int kSoftmaxWarps = N == 64 ? 8 : 4;
    static constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
    static constexpr int kProducerWarp = kSoftmaxWarps;
    static constexpr int kScoreWarp = kSoftmaxWarps + 1;
    static constexpr int kValueWarp = kSoftmaxWarps + 2;
    static constexpr int kQueryWarp = kSoftmaxWarps + 3;
    static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
    static constexpr int kWarpCols = N / (kSoftmaxWarps / 4);   // columns a softmax warp works on
    static constexpr int kV = N == 64 ? 8 : N == 32 ? 10 : 11;  // ring of value blocks
    static constexpr int kR = N == 64 ? 1 : N == 32 ? 2 : 3;    // ring of rotary blocks
    static constexpr int kAhead = N == 64 ? 1 : 0;              // tiles asked for in L2 ahead of their copies
    static constexpr int kQBlock = N * 128;                     // N columns x 64 dims
    static constexpr int kPBytes = kKeys * N * 2;
    static constexpr int kVOff = 0;
    static constexpr int kROff = kVOff + kV * kBlock;
    static constexpr int kQOff = kROff + kR * kHalf;
    static constexpr int kPOff = kQOff + 9 * kQBlock;
    static constexpr int kBarOff = kPOff + 2 * kPBytes;
    static constexpr int kNumBars = 2 * kV + 2 * kR + 10;
    static constexpr int kRedOff = kBarOff + ((kNumBars * 8 + 127) / 128) * 128;  // [4][N] per-warp maxima or sums
    static constexpr int kColOff = kRedOff + 4 * N * 4;   // [N] factors (rescale, then 1 / sum)
    static constexpr int kLimOff = kColOff + N * 4;       // [N] keys each column sees
    static constexpr int kPlanOff = kLimOff + N * 4;      // plan: warp totals, the worker's first unit
    static constexpr int kBytes = kPlanOff + 16 + 8 * (kSoftmaxWarps + 4);
    static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
    static constexpr uint32_t kSCol = 4 * N;              // S^T behind O^T's four blocks
    static constexpr uint32_t kTmem = N == 64 ? 512 : N == 32 ? 256 : 128;
};

// A unit: column group `g` of sequence `b`.
struct Unit {
    int b, r0, kv, qreal, cols, c0;  // cols: the sequence's columns; c0: the group's first
    int vis, tiles;                  // keys its last real row sees
};

struct Sched {
    int workers, groups, cols;  // workers, column groups a sequence may have, columns of a group
    int toll;                   // places of the line ahead of each unit's tiles
    int4* dir;                  // [workers][2] where each worker starts: place in its unit (-1: no
                                // work), the unit's tiles, share; the unit's row, columns, first column
    float* lse;                 // [workers][2][cols] partial states: a first and a last segment
    float* o;                   // [workers][2][cols][512]
    bool q_boxes;               // a CTA's columns are a box of the queries' tensor map
    bool whole;                 // worker w takes unit w: nothing is cut, nothing joined
};

__device__ __forceinline__ Unit unit_of(const LatentParams& p, const Sched& sc, int u) {
    Unit w;
    w.b = u / sc.groups;
    w.r0 = p.q_indptr[w.b];
    const int nrows = max(0, min(p.q_indptr[w.b + 1] - w.r0, p.max_q_rows));
    w.qreal = max(0, min(p.q_real ? p.q_real[w.b] : nrows, nrows));
    w.kv = min(max(p.kv_lens[w.b], 0), p.max_kv_len);
    w.cols = nrows * p.heads;
    w.c0 = (u - w.b * sc.groups) * sc.cols;
    w.vis = 0;
    if (w.c0 < w.cols && w.c0 / p.heads < w.qreal) {
        const int last = min((min(w.c0 + sc.cols, w.cols) - 1) / p.heads, w.qreal - 1);
        w.vis = p.causal ? max(0, w.kv - w.qreal + last + 1) : w.kv;
    }
    w.tiles = (w.vis + kKeys - 1) / kKeys;
    return w;
}

// The places of the line that a unit takes.
__device__ __forceinline__ int unit_places(const Sched& sc, const Unit& w) { return w.tiles > 0 ? w.tiles + sc.toll : 0; }

// The segments of one worker's share, in order; every role walks them alike.
struct Segments {
    int u, o;      // unit and place in it that come next
    int64_t left;  // places of the share
    Unit w;
    int j0, j1;    // the segment: tiles [j0, j1) of w
    __device__ __forceinline__ bool next(const LatentParams& p, const Sched& sc) {
        while (left > 0) {
            w = unit_of(p, sc, u);
            const int places = unit_places(sc, w);
            const int to = static_cast<int>(min(static_cast<int64_t>(places), o + left));
            j0 = max(0, o - sc.toll);
            j1 = to - sc.toll;
            left -= max(0, to - o);
            o = to;
            if (o >= places) {
                o = 0;
                ++u;
            }
            if (j1 > j0) return true;
        }
        return false;
    }
};

// A place in a ring of R buffers and the parity of the phase it is in.
template <int R>
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == R) {
            s = 0;
            ph ^= 1;
        }
    }
};

template <int N, int CTAS>
__global__ void __launch_bounds__(Dim<N>::kThreads, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_q,
                       const LatentParams p, const Sched sc) {
    using D = Dim<N>;
    constexpr int kThreads = D::kThreads, kSoftmaxThreads = D::kSoftmaxThreads;
    constexpr int kProducerWarp = D::kProducerWarp, kScoreWarp = D::kScoreWarp, kValueWarp = D::kValueWarp;
    constexpr int kQueryWarp = D::kQueryWarp;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % CTAS;
    const int worker = blockIdx.x / CTAS;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid's end

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + D::kBarOff);
    uint64_t* v_full = bars;
    uint64_t* v_empty = v_full + D::kV;
    uint64_t* r_full = v_empty + D::kV;
    uint64_t* r_empty = r_full + D::kR;
    uint64_t* q_ready = r_empty + D::kR;
    uint64_t* q_free = q_ready + 1;
    uint64_t* s_full = q_free + 1;    // [2]
    uint64_t* p_full = s_full + 2;    // [2]
    uint64_t* pv_done = p_full + 2;   // [2]
    uint64_t* o_full = pv_done + 2;
    uint64_t* mma_done = o_full + 1;
    float* red = reinterpret_cast<float*>(smem + D::kRedOff);
    float* colf = reinterpret_cast<float*>(smem + D::kColOff);
    int* lim = reinterpret_cast<int*>(smem + D::kLimOff);
    int64_t* plan_tot = reinterpret_cast<int64_t*>(smem + D::kPlanOff);  // [warps]
    int* plan = reinterpret_cast<int*>(smem + D::kPlanOff + kThreads / 4);  // unit, tile, tmem, abort
    volatile int* abort_flag = plan + 3;

    // ---- the plan: the line of all units' tiles, and this worker's share of it
    const int units = p.batch * sc.groups;
    const int per = (units + kThreads - 1) / kThreads;
    const int u0 = sc.whole ? worker : min(units, static_cast<int>(threadIdx.x) * per);
    const int u1 = sc.whole ? worker + 1 : min(units, u0 + per);
    int64_t mine = 0;
    for (int u = u0; u < u1; ++u) mine += unit_places(sc, unit_of(p, sc, u));
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) plan_tot[warp] = x;
    if (warp == kQueryWarp && lane == 0) {
        for (int s = 0; s < D::kV; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int s = 0; s < D::kR; ++s) {
            mbar_init(&r_full[s], 1);
            mbar_init(&r_empty[s], 1);
        }
        mbar_init(q_ready, 32);
        mbar_init(q_free, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], D::kSoftmaxWarps);
            mbar_init(&pv_done[t], 1);
        }
        mbar_init(o_full, 1);
        mbar_init(mma_done, 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kValueWarp) tc_alloc(reinterpret_cast<uint32_t*>(plan + 2), D::kTmem);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    Segments seg0;
    if (sc.whole) {
        seg0.left = mine;
    } else {
        int64_t before = x - mine, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            before += w < warp ? plan_tot[w] : 0;
            total += plan_tot[w];
        }
        int64_t share = total + sc.workers - 1;
        share = share >> 32 ? share / sc.workers : static_cast<uint32_t>(share) / static_cast<uint32_t>(sc.workers);
        share = max(share, static_cast<int64_t>(kMinShare + sc.toll));
        const int64_t start = worker * share;
        seg0.left = max(min(share, total - start), static_cast<int64_t>(0));
        if (start >= before && start < before + mine) {  // one thread at most
            int64_t at = before;
            for (int u = u0; u < u1; ++u) {
                const Unit w = unit_of(p, sc, u);
                const int t = unit_places(sc, w);
                if (start < at + t) {
                    plan[0] = u;
                    plan[1] = static_cast<int>(start - at);
                    if (rank == 0) {
                        sc.dir[2 * worker] = make_int4(plan[1], w.tiles, static_cast<int>(share), 0);
                        sc.dir[2 * worker + 1] = make_int4(w.r0, w.cols, w.c0, 0);
                    }
                    break;
                }
                at += t;
            }
        }
        if (seg0.left == 0 && threadIdx.x == 0 && rank == 0) sc.dir[2 * worker] = make_int4(-1, 0, 0, 0);
    }
    __syncthreads();
    seg0.u = sc.whole ? worker : plan[0];
    seg0.o = sc.whole ? 0 : plan[1];
    const uint32_t tmem = static_cast<uint32_t>(plan[2]);
    const uint32_t sbase = smem_u32(smem);
    // the swizzles need 1024-byte aligned tiles
    if ((sbase & 1023u) != 0) {
        if (threadIdx.x == 0) set_err(p.err, PKV_ERRBIT_TIMEOUT);
        seg0.left = 0;
    }

    // a completed phase passes at once; after one wait gave up, the others do not wait
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity)) return true;
        *abort_flag = 1;
        set_err(p.err, PKV_ERRBIT_TIMEOUT);
        return false;
    };
    Segments it = seg0;

    if (warp == kProducerWarp) {
        // ============================ producer ==============================
        if (elect_one()) {
            prefetch_tmap(&tm);
            constexpr int kPages = kKeys / 32;  // of a tile
            Ring<D::kV> v;
            Ring<D::kR> r;
            // The pages are looked up a tile ahead of their use, on across segments.
            // Where two tiles are all that shared memory holds, pages are asked for in
            // L2 kAhead tiles before their copies: 64 columns take 83.5 / 81.1 / 88.4 / 98.9 us
            // with 0 / 1 / 2 / 4, 128 columns 109.3 / 99.4 / 102.0 / 104.7.  (Beside a deeper ring it
            // changes nothing: 65.9 / 65.6 us with 0 / 1 for 16 columns.)
            constexpr int kAhead = D::kAhead;
            int j = 0, last_page = 0;
            const int32_t* bt = nullptr;
            int queued = 0;  // tiles looked up and not yet copied
            it.j1 = 0;
            auto look_up = [&](int (&ph)[kPages]) {
                if (j >= it.j1) {
                    if (!it.next(p, sc)) return;  // (and again: nothing is left)
                    j = it.j0;
                    bt = p.block_table + static_cast<int64_t>(it.w.b) * p.block_table_stride;
                    last_page = (it.w.vis + 31) / 32;
                }
#pragma unroll
                for (int k = 0; k < kPages; ++k) {
                    const int lp = kPages * j + k;
                    ph[k] = lp < last_page ? max(bt[lp], -1) : kNoPage;
                }
                ++j;
                ++queued;
            };
            // checked pages; the sentinel reads as zeros
            auto ask = [&](int (&ph)[kPages]) {
#pragma unroll
                for (int k = 0; k < kPages; ++k) {
                    if (ph[k] < 0 || ph[k] >= p.num_pages) {
                        if (ph[k] != kNoPage && p.checked) set_err(p.err, PKV_ERRBIT_PAGE);
                        ph[k] = static_cast<int>(p.num_pages);
                    } else if (kAhead > 0) {
                        const char* page = static_cast<const char*>(p.pool) + static_cast<int64_t>(ph[k]) * p.page_stride * 2;
                        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(page), "r"(32 * kLatentRow * 2) : "memory");
                    }
                }
            };
            int next[kAhead + 1][kPages];
#pragma unroll
            for (int k = 0; k <= kAhead; ++k) {
#pragma unroll
                for (int q = 0; q < kPages; ++q) next[k][q] = kNoPage;
                look_up(next[k]);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) ask(next[k]);
            bool alive = true;
            for (int n = 0; alive && queued > 0; ++n, --queued) {
                ask(next[kAhead]);
                int ph[kPages];
#pragma unroll
                for (int q = 0; q < kPages; ++q) {
                    ph[q] = next[0][q];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) next[k][q] = next[k + 1][q];
                    next[kAhead][q] = kNoPage;
                }
                look_up(next[kAhead]);
                // 64 dims from d0 of the tile's pages to dst
                auto copy = [&](uint8_t* dst, uint64_t* bar, int d0) {
#pragma unroll
                    for (int k = 0; k < kPages; ++k) tma_load_3d(dst + k * 4096, &tm, bar, d0, 0, ph[k]);
                };
                // (a fresh barrier's previous phase counts as complete: the first round passes)
                for (int b = 0; alive && b < kBlocks; ++b) {
                    alive = wait(&v_empty[v.s], v.ph ^ 1);
                    if (!alive) break;
                    mbar_arrive_expect_tx(&v_full[v.s], kBlock);
                    uint8_t* dst = smem + D::kVOff + v.s * kBlock;
                    copy(dst, &v_full[v.s], b * 128);
                    copy(dst + kHalf, &v_full[v.s], b * 128 + 64);
                    v.next();
                }
                // the rotary block comes last in every tile: with one buffer its next copy has a
                // tile's time to land
                alive = alive && wait(&r_empty[r.s], r.ph ^ 1);
                if (!alive) break;
                mbar_arrive_expect_tx(&r_full[r.s], kHalf);
                copy(smem + D::kROff + r.s * kHalf, &r_full[r.s], kLatentDim);
                r.next();
            }
            // do not leave with copies into this CTA's shared memory in flight
            // (buffers behind `s` were last filled in this round, the others in the one before)
            for (int k = 0; k < D::kV; ++k) mbar_wait(&v_full[k], k < v.s ? v.ph : v.ph ^ 1);
            for (int k = 0; k < D::kR; ++k) mbar_wait(&r_full[k], k < r.s ? r.ph : r.ph ^ 1);
        }
    } else if (warp == kScoreWarp) {
        // =============================== S^T ================================
        if (elect_one()) {
            constexpr uint32_t kIdesc = tc_idesc(kKeys, N, false, false);
            const uint64_t dq = tc_desc(sbase + D::kQOff, 16, 1024, 128);
            const uint64_t dv = tc_desc(sbase + D::kVOff, 16, 1024, 128), dr = tc_desc(sbase + D::kROff, 16, 1024, 128);
            Ring<D::kV> v;
            Ring<D::kR> r;
            int n = 0, nseg = 0;
            bool ok = true, landed = false;
            // a block's barrier is probed among the products of the one before it: a
            // wait between two batches would leave the pipe idle for ~150 cycles
            auto probe = [&](uint64_t* bar, uint32_t parity) {
                landed = mbar_test(bar, parity);
                if (landed) tc_after_sync();
            };
            auto settle = [&](uint64_t* bar, uint32_t parity) {
                if (landed) return;
                ok = ok && wait(bar, parity);
                tc_after_sync();
            };
            while (ok && it.next(p, sc)) {
                ok = wait(q_ready, nseg++ & 1);
                for (int j = it.j0; ok && j < it.j1; ++j, ++n) {
                    const int t = n & 1;
                    const uint32_t d = tmem + D::kSCol + t * N;
                    // S^T (+)= 64 dims of the tile times block qb of the queries
                    auto half = [&](uint64_t da, int qb, bool acc) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma(d, da + 2 * kk, dq + ((qb * D::kQBlock + kk * 32) >> 4), kIdesc, acc || kk > 0);
                    };
                    ok = wait(&p_full[t], ((n >> 1) & 1) ^ 1);  // the softmax has read tile n - 2's scores
                    tc_after_sync();
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        settle(&v_full[v.s], v.ph);
                        const uint64_t da = dv + v.s * (kBlock >> 4);
                        half(da, 2 * b, b > 0);
                        v.next();
                        if (b + 1 < kBlocks) probe(&v_full[v.s], v.ph);
                        else probe(&r_full[r.s], r.ph);
                        half(da + (kHalf >> 4), 2 * b + 1, true);
                    }
                    settle(&r_full[r.s], r.ph);
                    half(dr + r.s * (kHalf >> 4), kRopeBlock, true);
                    tc_commit(&r_empty[r.s]);
                    r.next();
                    tc_commit(&s_full[t]);
                    probe(&v_full[v.s], v.ph);
                }
                tc_commit(q_free);
            }
            // nothing of this thread's still runs in the tensor pipe when the CTA
            // winds down (after a failed wait the last products may)
            tc_commit(mma_done);
            if (!mbar_wait(mma_done, 0)) set_err(p.err, PKV_ERRBIT_TIMEOUT);
        }
    } else if (warp == kValueWarp) {
        // =============================== O^T ================================
        if (elect_one()) {
            constexpr uint32_t kIdesc = tc_idesc(128, N, true, true);
            // the tiles once more, as dims x keys; P^T: rows of keys, N columns wide, one swizzle row each
            const uint64_t dv = tc_desc(sbase + D::kVOff, kHalf, 1024, 128);
            const uint64_t dp = tc_desc(sbase + D::kPOff, 16, 16 * N, 2 * N);
            int n = 0, s = 0;
            bool ok = true;
            while (ok && it.next(p, sc)) {
                for (int j = it.j0; ok && j < it.j1; ++j, ++n) {
                    const int t = n & 1;
                    ok = wait(&p_full[t], (n >> 1) & 1);
                    tc_after_sync();
                    const uint64_t db = dp + t * (D::kPBytes >> 4);
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        const uint64_t da = dv + s * (kBlock >> 4);
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            tc_mma(tmem + b * N, da + kk * (2048 >> 4), db + kk * (32 * N >> 4), kIdesc, j > it.j0 || kk > 0);
                        tc_commit(&v_empty[s]);
                        if (++s == D::kV) s = 0;
                    }
                    tc_commit(&pv_done[t]);
                }
                if (ok) tc_commit(o_full);
            }
            tc_commit(mma_done);
            if (!mbar_wait(mma_done, 0)) set_err(p.err, PKV_ERRBIT_TIMEOUT);
        }
    } else if (warp == kQueryWarp) {
        // ============================= queries ==============================
        int nseg = 0;
        while (it.next(p, sc)) {
            const int col0 = it.w.c0 + rank * N;
            wait(q_free, (nseg++ & 1) ^ 1);
            __syncwarp();
            int i = col0 / p.heads, h = col0 - i * p.heads;
            if (sc.q_boxes && col0 + N <= it.w.cols) {
                // whole rows of heads, or a part of one: nine boxes (all of them existing rows)
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_ready, 9 * D::kQBlock);
                    for (int k = 0; k < 9; ++k)
                        tma_load_3d(smem + D::kQOff + k * D::kQBlock, &tm_q, q_ready, k * 64, h, it.w.r0 + i);
                } else {
                    mbar_arrive(q_ready);
                }
                continue;
            }
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(it.w.r0) * p.q_token_stride;
#pragma unroll 2
            for (int c = 0; c < N; ++c) {  // columns past the last: zeros
                const bool held = col0 + c < it.w.cols;
                const __nv_bfloat16* row = held ? q + i * p.q_token_stride + h * p.q_head_stride : q;
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const int ch = lane + 32 * k;
                    if (ch < kLatentRow / 8)
                        copy16_async(sbase + D::kQOff + (ch >> 3) * D::kQBlock + sw128_offset(c, ch & 7),
                                     row + (held ? ch * 8 : 0), held);
                }
                if (++h == p.heads) {
                    h = 0;
                    ++i;
                }
            }
            copy_async_wait();
            fence_proxy_async_smem();
            mbar_arrive(q_ready);
        }
        // this worker's part of the units that see no key: zeros
        for (int u = worker; u < units; u += sc.workers) {
            const Unit w = unit_of(p, sc, u);
            if (p.checked && rank == 0 && lane == 0 && w.c0 == 0) {
                const int rows = p.q_indptr[w.b + 1] - w.r0, kv = p.kv_lens[w.b];
                if (kv > p.max_kv_len || kv < 0 || rows > p.max_q_rows || (p.q_real && p.q_real[w.b] > rows))
                    set_err(p.err, PKV_ERRBIT_LEN);
            }
            if (w.tiles > 0) continue;
            for (int c = w.c0 + rank * N; c < min(w.c0 + rank * N + N, w.cols); ++c) {
                const int64_t at = static_cast<int64_t>(w.r0) * p.heads + c;
                for (int d = lane * 4; d < kLatentDim; d += 128) {
                    if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at * kLatentDim + d) = make_float4(0, 0, 0, 0);
                    else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at * kLatentDim + d) = make_uint2(0, 0);
                }
                if (p.lse && lane == 0) p.lse[at] = -INFINITY;
            }
        }
        // do not leave with copies into this CTA's shared memory in flight
        if (nseg > 0) mbar_wait(q_ready, (nseg - 1) & 1);
    } else {
        // ===================== softmax and outputs ==========================
        // A warp holds 16 keys of the tile (its quadrant's first 16 lanes) and W
        // columns, a thread 2 keys and W / 4 columns: maxima and sums stay per thread,
        // and a column's reference moves (by all threads together) only when a score
        // passes it by 2^8, so most tiles exchange nothing but that one vote.
        constexpr int W = D::kWarpCols, NC = W / 4;
        const int wq = warp & 3, wc = (warp >> 2) * W;  // quadrant, first column
        const uint32_t quad = static_cast<uint32_t>(wq * 32) << 16;
        const int key_of = 16 * wq + (lane >> 2);       // and 8 further
        const int col_of = wc + 2 * (lane & 3);         // [2 f + e] is column col_of + 8 f + e
        int nseg = 0;
        int vfirst = 0;  // the tile's first value block in the ring
        int n = 0;
        int slot = 0;  // of a partial state: 0 for the share's first segment

        while (it.next(p, sc)) {
            const Unit& w = it.w;
            const int col0 = w.c0 + rank * N;  // this CTA's first column
            // ---- limits of the columns.  Those past the last (their
            // results go nowhere) see what the unit sees, so they mask nothing.
            if (threadIdx.x < N) {
                const int i = (col0 + threadIdx.x) / p.heads;
                int l = w.vis;
                if (col0 + threadIdx.x < w.cols)
                    l = i >= w.qreal ? 0 : p.causal ? max(0, w.kv - w.qreal + i + 1) : w.kv;
                lim[threadIdx.x] = l;
            }
            bar_sync(1, kSoftmaxThreads);
            int lim_min = lim[lane % N];
            if (N > 32) lim_min = min(lim_min, lim[(lane + 32) % N]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));

            float m[NC], l[NC], lb[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                m[c] = -INFINITY;
                l[c] = lb[c] = 0.f;
            }
            for (int j = it.j0; j < it.j1; ++j, ++n) {
                const int t = n & 1;
                const int key0 = j * kKeys;
                wait(&s_full[t], (n >> 1) & 1);
                __syncwarp();
                tc_after_sync();
                uint32_t v[W / 2];
                tc_load_frag<W>(tmem + quad + D::kSCol + t * N + wc, v);
                float s[W / 2];
#pragma unroll
                for (int e = 0; e < W / 2; ++e) s[e] = __uint_as_float(v[e]) * p.scale_log2;
                if (key0 + kKeys > lim_min) {
#pragma unroll
                    for (int f = 0; f < W / 8; ++f) {
                        const int2 lm = *reinterpret_cast<const int2*>(lim + col_of + 8 * f);
                        const int k = key0 + key_of;
                        s[4 * f] = k < lm.x ? s[4 * f] : -INFINITY;
                        s[4 * f + 1] = k < lm.y ? s[4 * f + 1] : -INFINITY;
                        s[4 * f + 2] = k + 8 < lm.x ? s[4 * f + 2] : -INFINITY;
                        s[4 * f + 3] = k + 8 < lm.y ? s[4 * f + 3] : -INFINITY;
                    }
                }
                bool past = false;
#pragma unroll
                for (int f = 0; f < W / 8; ++f)
#pragma unroll
                    for (int e = 0; e < 2; ++e) past |= fmaxf(s[4 * f + e], s[4 * f + 2 + e]) > m[2 * f + e] + kLazyRescale;
                if (bar_any(1, kSoftmaxThreads, past)) {
                    // new references: the tile's maxima where they pass the old ones by 2^8
                    float mx[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        mx[c] = fmaxf(s[4 * (c >> 1) + (c & 1)], s[4 * (c >> 1) + 2 + (c & 1)]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], o));
                    }
                    if (lane < 4) {
#pragma unroll
                        for (int c = 0; c < NC; ++c) red[wq * N + col_of + 8 * (c >> 1) + (c & 1)] = mx[c];
                    }
                    bar_sync(1, kSoftmaxThreads);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int at = col_of + 8 * (c >> 1) + (c & 1);
                        const float tm4 = fmaxf(fmaxf(red[at], red[N + at]), fmaxf(red[2 * N + at], red[3 * N + at]));
                        float alpha = 1.f;
                        if (tm4 > m[c] + kLazyRescale) {
                            alpha = fast_exp2(m[c] - tm4);  // 0 when no key was visible before
                            m[c] = tm4;
                        }
                        l[c] *= alpha;
                        lb[c] *= alpha;
                        if (wq == 0 && lane < 4) colf[at] = alpha;
                    }
                    // O^T's columns follow once the previous tile's products are done
                    if (j > it.j0) wait(&pv_done[t ^ 1], ((n - 1) >> 1) & 1);
                    __syncwarp();
                    bar_sync(1, kSoftmaxThreads);
                    if (j > it.j0) {
                        tc_after_sync();
                        for (int c16 = 0; c16 < kBlocks * W / 16; ++c16) {
                            const int c = wc + c16 % (W / 16) * 16;
                            const uint32_t at = tmem + quad + c16 / (W / 16) * N + c;
                            uint32_t o[16];
                            tc_load16(at, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * colf[c + e]);
                            tc_store16(at, o);
                        }
                        tc_wait_store();
                    }
                }
                // weights, rounded to bf16 for the product; their sums rounded (the
                // output's divisor) and not (the LSE)
                // tile n - 2's products are done with this buffer of weights (where the ring
                // holds two tiles, tile n has taken the blocks that they released last)
                if (D::kV > 2 * kBlocks) wait(&pv_done[t], ((n >> 1) & 1) ^ 1);
                uint8_t* pt = smem + D::kPOff + t * D::kPBytes;
#pragma unroll
                for (int f = 0; f < W / 8; ++f) {
                    const float m0 = m[2 * f] == -INFINITY ? 0.f : m[2 * f], m1 = m[2 * f + 1] == -INFINITY ? 0.f : m[2 * f + 1];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float w0 = fast_exp2(s[4 * f + 2 * r] - m0), w1 = fast_exp2(s[4 * f + 2 * r + 1] - m1);
                        const uint32_t pk = pack_bf16x2(w0, w1);
                        l[2 * f] += w0;
                        l[2 * f + 1] += w1;
                        lb[2 * f] += bf16lo(pk);
                        lb[2 * f + 1] += bf16hi(pk);
                        const int k = key_of + 8 * r;
                        uint32_t at = k * 2 * N + wc * 2 + f * 16;
                        at ^= ((at >> 7) & (N / 8 - 1)) << 4;
                        *reinterpret_cast<uint32_t*>(pt + at + (lane & 3) * 4) = pk;
                    }
                }
                // rows of keys that no column sees hold whatever the pool holds: zero
                // them (S^T has been computed), so that 0 * NaN does not reach O^T
                if (key0 + kKeys > w.vis) {
                    const int first = w.vis - key0;
                    for (int idx = threadIdx.x; idx < (kKeys - first) * 64; idx += kSoftmaxThreads) {
                        const int row = first + (idx >> 6), ch = idx & 63;
                        const int sl = (vfirst + (ch >> 4)) % D::kV;
                        *reinterpret_cast<uint4*>(smem + D::kVOff + sl * kBlock + ((ch >> 3) & 1) * kHalf +
                                                  sw128_offset(row, ch & 7)) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t]);
                vfirst = (vfirst + kBlocks) % D::kV;
            }
            // ---- the segment's columns: sums over the tile's rows, then O^T / sum
            const bool whole = it.j0 == 0 && it.j1 == w.tiles;
            float lsum = 0.f, lbsum = 0.f;  // of column threadIdx.x
#pragma unroll
            for (int pass = 0; pass < 2; ++pass) {
                bar_sync(1, kSoftmaxThreads);  // red has been read
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float sum = pass == 0 ? l[c] : lb[c];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane < 4) red[wq * N + col_of + 8 * (c >> 1) + (c & 1)] = sum;
                }
                bar_sync(1, kSoftmaxThreads);
                if (threadIdx.x < N) {
                    const float sum = (red[threadIdx.x] + red[N + threadIdx.x]) + (red[2 * N + threadIdx.x] + red[3 * N + threadIdx.x]);
                    if (pass == 0) lsum = sum;
                    else lbsum = sum;
                }
            }
            if (wq == 0 && lane < 4) {
#pragma unroll
                for (int c = 0; c < NC; ++c) colf[col_of + 8 * (c >> 1) + (c & 1)] = m[c];
            }
            bar_sync(1, kSoftmaxThreads);
            if (threadIdx.x < N) {
                const bool any = lsum != 0.f;  // (NaN stays)
                const float lse = any ? (colf[threadIdx.x] + __log2f(lsum)) * kLn2 : -INFINITY;
                const int col = col0 + threadIdx.x;
                if (whole) {
                    if (p.lse && col < w.cols) p.lse[static_cast<int64_t>(w.r0) * p.heads + col] = lse;
                } else {
                    sc.lse[(static_cast<int64_t>(worker) * 2 + slot) * sc.cols + rank * N + threadIdx.x] = lse;
                }
                colf[threadIdx.x] = any ? 1.0f / lbsum : 0.f;
            }
            wait(o_full, nseg++ & 1);
            __syncwarp();
            bar_sync(1, kSoftmaxThreads);
            tc_after_sync();
            const int64_t out_row = static_cast<int64_t>(w.r0) * p.heads + col0;
            float* part = sc.o + ((static_cast<int64_t>(worker) * 2 + slot) * sc.cols + rank * N) * kLatentDim;
            const int valid = min(N, w.cols - col0);  // columns that exist (uniform)
            for (int b = 0; b < kBlocks; ++b) {
                const int dim = b * 128 + wq * 32 + lane;
                uint32_t o[W];
                if constexpr (W == 16) tc_load16(tmem + quad + b * N + wc, o);
                else tc_load32(tmem + quad + b * N + wc, o);
                float f[W];
#pragma unroll
                for (int e = 0; e < W; ++e) f[e] = __uint_as_float(o[e]) * colf[wc + e];
                if (!whole || p.out_f32) {
                    float* dst = (whole ? static_cast<float*>(p.out) + out_row * kLatentDim : part) +
                                 static_cast<int64_t>(wc) * kLatentDim + dim;
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (wc + e < valid) dst[e * kLatentDim] = f[e];
                } else {
                    // lanes exchange one of two columns, so that each stores a pair of dims
                    const bool odd = lane & 1;
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                                         (out_row + wc + (odd ? 1 : 0)) * kLatentDim + (dim & ~1);
#pragma unroll
                    for (int e = 0; e < W; e += 2) {
                        const float got = __shfl_xor_sync(0xffffffffu, odd ? f[e] : f[e + 1], 1);
                        const uint32_t pk = odd ? pack_bf16x2(got, f[e + 1]) : pack_bf16x2(f[e], got);
                        if (wc + e + (odd ? 1 : 0) < valid) *reinterpret_cast<uint32_t*>(dst + e * kLatentDim) = pk;
                    }
                }
            }
            slot = 1;  // a later partial segment of this share is its last
            tc_before_sync();
        }
    }

    __syncwarp();
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == kValueWarp) tc_dealloc(tmem, D::kTmem);
}

// 4 E columns a CTA and cut: where worker c starts inside a unit, the unit's states,
// one a worker in line, are joined: out = sum w_i O_i / sum w_i with w_i = e^(lse_i -
// max).  Few states: the unit's first cut joins all the columns, E to each group of
// 128 threads, whose loads are under way together.  Many: its first cuts share the
// columns out, every group takes a quarter of the states.  E = 4 keeps units of 64
// and 128 columns to one wave of CTAs (with 1 the calls take 0.4 and 1 us longer), E = 1
// spreads those of 16 over the SMs (with 4: 0.7 us longer).
constexpr int kJoinGroups = 4;
constexpr int kJoinFew = 8;
template <int E>
__global__ void __launch_bounds__(128 * kJoinGroups, E == 1 ? 3 : 1) latent_join_kernel(const LatentParams p, const Sched sc) {
    const int c = blockIdx.x + 1, g = threadIdx.x >> 7, t = threadIdx.x & 127, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 d = sc.dir[2 * c], w = sc.dir[2 * c + 1];
    if (d.x <= sc.toll) return;
    const int64_t share = d.z, off = c * share - d.x, tile0 = off + sc.toll;  // the unit's places, its first tile's
    const int first = static_cast<int>(tile0 / share);                        // the worker that it begins in
    const int n = static_cast<int>((tile0 + d.y - 1) / share) - first + 1;
    const int first_slot = first * share < off ? 1 : 0;
    const int cut = c - first - 1;                                            // cuts of the unit before this one
    constexpr int kJoinCols = kJoinGroups * E;
    const int col0 = blockIdx.y * kJoinCols;
    const int valid = min(kJoinCols, w.y - w.z - col0);                       // columns that exist
    if (valid <= 0) return;
    auto piece = [&](int k, int col) {
        return (static_cast<int64_t>(first + k) * 2 + (k == 0 ? first_slot : 0)) * sc.cols + col0 + col;
    };
    auto add = [](float4& acc, float wk, const float4& o) {
        acc.x = fmaf(wk, o.x, acc.x);
        acc.y = fmaf(wk, o.y, acc.y);
        acc.z = fmaf(wk, o.z, acc.z);
        acc.w = fmaf(wk, o.w, acc.w);
    };
    auto state = [&](int64_t at) { return *reinterpret_cast<const float4*>(sc.o + at * kLatentDim + t * 4); };
    auto store = [&](int col, float m, float sum, const float4& acc) {
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
        const int64_t row = static_cast<int64_t>(w.x) * p.heads + w.z + col0 + col;
        if (p.out_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * kLatentDim + t * 4) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        } else {
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * kLatentDim + t * 4) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        }
        if (p.lse && t == 0) p.lse[row] = sum == 0.f ? -INFINITY : m + __log2f(sum) * kLn2;
    };
    if (n <= kJoinFew) {
        if (cut > 0) return;
        float lse[E], m[E], wk[E], sum[E];
        float4 acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {  // lane k: the k-th state's LSE, then its weight
            const int col = g * E + e;
            lse[e] = lane < n && col < valid ? sc.lse[piece(lane, col)] : -INFINITY;
            acc[e] = make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            m[e] = warp_max(lse[e]);
            if (m[e] == -INFINITY) m[e] = 0.f;
            wk[e] = fast_exp2((lse[e] - m[e]) * kLog2e);
            sum[e] = warp_sum(wk[e]);
        }
#pragma unroll 2
        for (int k = 0; k < n; ++k) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int col = g * E + e;
                const float x = __shfl_sync(0xffffffffu, wk[e], k);
                if (col < valid) add(acc[e], x, state(piece(k, col)));
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (g * E + e < valid) store(g * E + e, m[e], sum[e], acc[e]);
        return;
    }
    constexpr int kShare = E > 1 ? 2 : 1;  // columns a cut takes: a unit of many states has eight cuts
    if (cut >= kJoinCols / kShare) return;
    __shared__ float4 sh_o[kJoinGroups][128];
    __shared__ float sh_s[kJoinGroups];
    for (int col = kShare * cut; col < min(kShare * (cut + 1), valid); ++col) {
        float m = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0, 0, 0, 0);
        for (int k = lane; k < n; k += 32) m = fmaxf(m, sc.lse[piece(k, col)]);
        m = warp_max(m);
        if (m == -INFINITY) m = 0.f;
#pragma unroll 4
        for (int k = g; k < n; k += kJoinGroups) {
            const int64_t at = piece(k, col);
            const float x = fast_exp2((sc.lse[at] - m) * kLog2e);
            sum += x;
            add(acc, x, state(at));
        }
        sh_o[g][t] = acc;
        if (t == 0) sh_s[g] = sum;
        __syncthreads();
        if (g == 0) {
#pragma unroll
            for (int k = 1; k < kJoinGroups; ++k) {
                sum += sh_s[k];
                add(acc, 1.f, sh_o[k][t]);
            }
            store(col, m, sum, acc);
        }
        __syncthreads();
    }
}

template <int N, int CTAS>
cudaError_t launch(const LatentParams& p, const Sched& sc, const void* tmap, const void* tmap_q, cudaStream_t s) {
    static DeviceOnce opted;
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = opted.get(dev, &done, [&](int, int* v) {
        *v = 1;
        return cudaFuncSetAttribute(latent_attn_kernel<N, CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Dim<N>::kBytes);
    });
    if (e != cudaSuccess) return e;
    latent_attn_kernel<N, CTAS><<<static_cast<unsigned>(sc.workers * CTAS), Dim<N>::kThreads, Dim<N>::kBytes, s>>>(
        *static_cast<const CUtensorMap*>(tmap), *static_cast<const CUtensorMap*>(tmap_q), p, sc);
    e = cudaGetLastError();
    if (e != cudaSuccess || sc.workers == 1 || sc.whole) return e;
    constexpr int E = N == 16 ? 1 : 4;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t jc = {};
    jc.gridDim = dim3(static_cast<unsigned>(sc.workers - 1), static_cast<unsigned>(sc.cols / (kJoinGroups * E)));
    jc.blockDim = dim3(128 * kJoinGroups);
    jc.stream = s;
    jc.attrs = pdl;
    jc.numAttrs = 1;
    return cudaLaunchKernelEx(&jc, latent_join_kernel<E>, p, sc);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int64_t tiles_of(int max_kv_len) { return (static_cast<int64_t>(max_kv_len) + kKeys - 1) / kKeys; }
int columns_of(int64_t cols) { return cols <= 16 ? 16 : cols <= 32 ? 32 : cols <= 64 ? 64 : 128; }  // a worker holds
int64_t groups_of(int64_t cols) { return (cols + columns_of(cols) - 1) / columns_of(cols); }
int workers_at_once(int cols, int sms) { return cols <= 64 ? sms : max(sms / 2, 1); }
// no more workers than shares of the smallest size
int share_workers(int cols, int64_t units, int64_t unit_tiles, int sms) {
    return static_cast<int>(
        max(int64_t(1), min(int64_t(workers_at_once(cols, sms)), (units * unit_tiles + kMinShare - 1) / kMinShare)));
}
size_t share_bytes(int cols, int workers) {
    const size_t states = static_cast<size_t>(workers) * 2 * cols;
    return round256(workers * 2 * sizeof(int4)) + round256(states * 4) + states * kLatentDim * 4;
}

}  // namespace

LatentPlan plan_latent(int batch, int max_q_rows, int heads, int max_kv_len, int sms) {
    LatentPlan pl{};
    // The narrowest CTA that holds a sequence's columns, pairs of the widest beyond.  64
    // sequences of 513-8193 keys, us: 16 columns in CTAs of 16 / 32 / 64: 65.9 / 70.0 / 71.3;
    // 32 columns: 103.6 / 74.5 / 76.0; 64 columns: 183 / 112 / 82.3; 128 columns in CTAs of 64
    // one by one / in pairs: 124 / 100.  One width serves the whole call, from the bound of
    // rows: a prompt chunk beside decoding rows puts these in wide CTAs, mostly of zeros.
    const int64_t cols = static_cast<int64_t>(max_q_rows) * heads;
    const int held = columns_of(cols);
    pl.cols = min(held, 64);
    pl.ctas = held / pl.cols;
    pl.groups = static_cast<int>(groups_of(cols));
    const int64_t unit_tiles = tiles_of(max_kv_len);
    const int64_t units = static_cast<int64_t>(batch) * pl.groups, most = workers_at_once(held, sms);
    if (unit_tiles <= kWholeTiles && units <= most && unit_tiles * (most - units) <= kIdleTiles * most) {
        pl.whole = true;
        pl.workers = static_cast<int>(units);
        pl.ws_bytes = 256;
        return pl;
    }
    pl.workers = share_workers(held, units, unit_tiles, sms);
    pl.ws_bytes = share_bytes(held, pl.workers);
    return pl;
}

size_t latent_workspace_bytes(int batch, int max_q_rows, int heads, int max_kv_len, int sms) {
    const int64_t cols = static_cast<int64_t>(max_q_rows) * heads;
    size_t bytes = 256;
    for (int held = 16; held <= columns_of(cols); held *= 2)
        bytes = max(bytes, share_bytes(held, share_workers(held, batch * (held == 128 ? groups_of(cols) : 1),
                                                           tiles_of(max_kv_len), sms)));
    return bytes;
}

cudaError_t launch_latent_attn(const LatentParams& p, const LatentPlan& pl, void* workspace, const void* tmap,
                               const void* tmap_q, bool q_boxes, cudaStream_t s) {
    Sched sc;
    sc.workers = pl.workers;
    sc.groups = pl.groups;
    sc.toll = pl.cols == 64 ? kTollWide : kToll;
    sc.cols = pl.cols * pl.ctas;
    sc.q_boxes = q_boxes;
    sc.whole = pl.whole;
    char* w = static_cast<char*>(workspace);
    sc.dir = reinterpret_cast<int4*>(w);
    w += round256(pl.workers * 2 * sizeof(int4));
    sc.lse = reinterpret_cast<float*>(w);
    w += round256(static_cast<size_t>(pl.workers) * 2 * sc.cols * 4);
    sc.o = reinterpret_cast<float*>(w);
    if (pl.ctas == 2) return launch<64, 2>(p, sc, tmap, tmap_q, s);
    if (pl.cols == 64) return launch<64, 1>(p, sc, tmap, tmap_q, s);
    if (pl.cols == 32) return launch<32, 1>(p, sc, tmap, tmap_q, s);
    return launch<16, 1>(p, sc, tmap, tmap_q, s);
}

}  // namespace pkv
