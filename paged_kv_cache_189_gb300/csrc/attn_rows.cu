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
//    2^-22 below the row's largest.  A segment's rows sit in shared memory in
//    fragment order, staged once for all consumers.
//  * Weights are rounded once: to bf16 for bf16 pools, and w = 2^(a - M) vs to
//    f16 for 8-bit ones, M following a + log2(vs) - 6, so the largest w lies
//    between 2^6 and 2^15 for V scales of 2^-80 to 2^90.  Sums, maxima and outputs
//    are f32.
//  * Per CTA one warp looks up pages and scales ahead, 32 chunks at a time, and
//    one fills a ring of chunks (32 keys in 8 bits, 16 in bf16) by TMA, so the
//    chain length -> table -> scale stays off the copies' path; each of four
//    consumer warps owns every fourth stage and keeps its own softmax state: no
//    barrier joins the consumers until a unit's end.  2 CTAs an SM keep 128 KB in
//    flight (3 at 64-wide heads and 8 rows: 144 KB); 192 KB, six consumers at 128
//    registers, or two chunks a step were no faster (107, 114 and 121 us, of an
//    earlier build that took 107 for the first case below).
//  * Work: a unit is (sequence, K/V head, tile of 8 or 16 rows); its chunks are
//    the pages its rows see.  All units' chunks form one line, laid out on the
//    device (a captured call replays with other lengths), and the line is cut
//    into pieces: a first, fixed one per CTA, then smaller ones taken by
//    ticket.  SMs differ in the bandwidth they get (equal shares ended between
//    84 and 120 us), which the tickets absorb.  A planner clears the ticket and
//    writes where the pieces start while the CTAs, launched behind it with
//    programmatic serialisation, find their first piece themselves.
//  * A unit cut between pieces leaves one partial state per piece; a last launch
//    joins them in the line's order, so results do not depend on who took which
//    ticket.  (Joined by the CTA that completes a unit instead, the last CTAs
//    ended up to 75 us after the others on three sequences of 10^5 keys.)
//    Small calls skip all this: the resident CTAs take whole units in turn, the
//    next one's chunks on their way while one is joined.
// Measured (copy peak 6694 GB/s): 64 sequences of 513-8193 keys, 32 / 8 heads of
// 128, 8 bits, 524 MB: 105 us, 0.75 of the peak (the first chunk arrives after
// 6 us, the CTAs stream at 0.93 of it and end within 13 us of each other, the
// join takes 6); the same with 4 tokens a sequence 120 us, bound by the chunk's
// chain of dependent steps at 8 consumer warps an SM (the four that look up and
// copy hold 168 registers a thread too; one CTA of ten consumers an SM: 154, nothing
// streams while it joins a unit); 3 sequences of 60000-131072 keys 86 us (0.75);
// bf16 through a 4096-key window, 1020 MB: 167 us (0.91).  Rows beyond 16 walk and
// widen the keys again: 93, 161, 212, 283 and 321 us at 16, 32, 48, 64 and 80 rows
// of 64 sequences of 2000-4000 keys (400 MB).
#include <cuda.h>
#include <cuda_fp16.h>
#include <algorithm>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kPage = 32;
constexpr float kLazy = 8.0f;         // move the reference only past 2^8 growth
// 8-bit pools: M follows a + log2(vs) - kWeightUp for V scales of 2^kLowScale to
// 2^kHighScale.  A state's largest weight w is then 2^6 at least and below 2^15,
// whatever vs in that range: f16 keeps 11 bits of weights down to 2^-20 of it (from
// 2^-14 on without kWeightUp).  The sums of 2^(a - M), whose largest summand is
// 2^-84 to 2^94, neither vanish nor overflow for as many keys as there can be.
// Smaller scales (0 too) round the weights to within 2^-102 of an output a key;
// larger ones overflow f16 to infinity, where without kHighScale the sums would
// underflow and a row come out as zero.
constexpr float kWeightUp = 6.0f, kLowScale = -80.0f, kHighScale = 90.0f;
// PKV_FLAG_TEST_WAIT_TIMEOUT: the limit of the waits that are meant to run out
// (consumers on a barrier nothing completes, the other warps' as they follow)
constexpr uint64_t kTestWaitNs = 20000, kWaitNs = 2000000000ull;
constexpr int kDescs = 8;             // segments the look-up may be ahead
constexpr int kSelfBatch = 256;       // sequences up to which a CTA finds its first piece itself
constexpr int kBatches = 1;           // batches of 32 chunks it may be ahead

template <int D, bool FP8, int NT>
struct Cfg {
    static constexpr int kWarps = 4;                     // consumers
    // 64-wide heads leave ring space for a third CTA, at 96 registers a thread
    // (8-bit pools spill 36 bytes at that)
    static constexpr int kCtasPerSm = D == 64 && NT == 1 ? 3 : 2;
    static constexpr int kRingBytes = (kCtasPerSm == 3 ? 48 : 64) * 1024;
    static constexpr int kRedRows = 8;                   // rows joined at a time: a tile
    static constexpr int kThreads = (kWarps + 2) * 32;
    static constexpr int kKeys = FP8 ? 32 : 16;          // keys of a chunk
    static constexpr int kTile = kKeys * D * (FP8 ? 1 : 2);
    static constexpr int kStage = 2 * kTile;             // K, V
    static constexpr int kStages = kRingBytes / kStage;  // 8 (head dim 128), 16 (64; 12 with three CTAs)
    static constexpr int kOwn = kStages / kWarps;        // stages of one consumer
    static constexpr int kRows = 8 * NT;
    static constexpr int kRedStride = D + 4;
    static constexpr int kRedOff = kRingBytes;                              // [warps][kRedRows][kRedStride] f32
    static constexpr int kStatOff = kRedOff + kWarps * kRedRows * kRedStride * 4;  // m, l, l_b: [warps][kRows]
    static constexpr int kQOff = (kStatOff + 3 * kWarps * kRows * 4 + 15) & ~15;   // [NT][D / 32][lanes] 16 bytes
    static constexpr int kFacOff = kQOff + NT * (D / 32) * 512;                    // [kRows] score factors
    static constexpr int kMetaOff = kFacOff + kRows * 4;                    // [stages] (ks, vs, key0)
    static constexpr int kDescOff = kMetaOff + kStages * 16;
    static constexpr int kQueueOff = kDescOff + kDescs * 64;          // [batches][32] look-ups
    static constexpr int kHeadOff = kQueueOff + kBatches * 32 * 16;   // [batches] (chunks, K/V head)
    static constexpr int kFlagOff = kHeadOff + kBatches * 8;  // a consumer's wait gave up; segments staged
    // full, empty [stages], dfull, dempty [descs], bfull, bempty [batches], never
    static constexpr int kBarOff = kFlagOff + 8;
    static constexpr int kBytes = kBarOff + (2 * kStages + 2 * kDescs + 2 * kBatches + 1) * 8;
    static_assert(kStages % kWarps == 0, "each consumer owns whole stages");
    static_assert((kBytes + 1024) * kCtasPerSm <= 228 * 1024, "CTAs per SM must fit in shared memory");
    static_assert(kMetaOff % 16 == 0 && kDescOff % 16 == 0 && kBarOff % 8 == 0, "alignment");
};

struct RowsArgs {
    AttnParams p;
    int ctas;       // CTAs that share the line (0: whole units)
    int tiles_max;  // row tiles of a sequence at the host bound
    bool even;      // all pieces fixed
    // written by the planner
    int* ticket;
    int2* cuts;         // [units] first slot and number of its partial states; 0: none
    int* seq_at;        // [batch + 1] the line's place of each sequence's first unit, and its length
    int4* starts;       // [pieces] (sequence, K/V head, place in the head's units) each starts with
    // partial states: piece i of unit u in slot i + u (both grow along the line)
    float* frag_o;      // [pieces + units][rows][D] normalised outputs
    float* frag_lse;    // [pieces + units][rows] log2 of the sums
};

// The cut of a line of T places: `first` pieces of together A1, then pieces of
// q1 up to A2 and of q2 up to T.
struct Line {
    int T, A1, A2, first, size, longer, n1, n2, q1, q2;
    __device__ __forceinline__ Line(int total, int ctas, bool even) {
        // 85 % fixed, 10 % in tenths and 5 % in twentieths of a CTA's average
        // share; pieces of at least 12 and 6 chunks, fixed ones of at least 8.
        // Few long units: all fixed, else the last ones fall into a hundred
        // states each (three sequences of 10^5 keys: 88 us against 94; 64
        // ragged sequences: 114 against 108 the other way round).
        T = total;
        A1 = even ? T : T / 20 * 17;
        A2 = even ? T : T / 20 * 19;
        first = min(max(A1 / 8, 1), ctas);
        size = A1 / first;
        longer = A1 - size * first;  // the first so many pieces have one more
        q1 = max((T / 10 + ctas - 1) / ctas, 12);
        q2 = max((T / 20 + ctas - 1) / ctas, 6);
        n1 = (A2 - A1 + q1 - 1) / q1;
        n2 = (T - A2 + q2 - 1) / q2;
    }
    __device__ __forceinline__ int pieces() const { return first + n1 + n2; }
    // places [from, to) of piece i
    __device__ __forceinline__ void piece(int i, int& from, int& to) const {
        if (i < first) {
            from = i * size + min(i, longer);
            to = from + size + (i < longer ? 1 : 0);
        } else if (i < first + n1) {
            from = A1 + (i - first) * q1;
            to = min(from + q1, A2);
        } else {
            from = min(A2 + (i - first - n1) * q2, T);
            to = min(from + q2, T);
        }
    }
    __device__ __forceinline__ int piece_of(int at) const {
        if (at < A1) {
            const int x = longer * (size + 1);
            return at < x ? at / (size + 1) : longer + (at - x) / size;
        }
        if (at < A2) return first + (at - A1) / q1;
        return first + n1 + (at - A2) / q2;
    }
    static int most(int ctas) { return 6 * ctas + 8; }  // pieces, whatever T
};

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
    int left;            // places of the piece still to come
    // the current segment
    Seq s;
    Span u;
    int sb, skvh, smt, ps, pe;
    bool starts, ends;

    __device__ __forceinline__ bool next(const AttnParams& p, int G) {
        while (left > 0 && b < p.batch) {
            s = sequence<ROWS>(p, b, G);
            if (mt >= s.tiles) {
                mt = 0;
                if (s.tiles == 0 || ++kvh == p.num_kv_heads) {
                    kvh = 0;
                    ++b;
                }
                continue;
            }
            u = span_of<ROWS, KEYS>(p, s, mt, G);
            const int places = max(u.n, 1);
            if (at >= places) {  // a start counted from the head's first tile
                at -= places;
                ++mt;
                continue;
            }
            sb = b;
            skvh = kvh;
            smt = mt;
            ps = at;
            pe = min(places, at + left);
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
__device__ __forceinline__ uint32_t word(const uint4& v, int k) { return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w; }
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

// A segment as the look-up hands it to the consumers.
struct __align__(16) Desc {
    int r0, nrows, qreal, kv_len, lo, hi;  // hi, lo: of the unit's rows together
    int kvh, row0;                         // K/V head, first (row, head) of the tile
    int n;                                 // chunks; -1: no more segments
    int frag;                              // slot of the partial state; -1: the whole unit is here
    int all_lo, all_end;                   // keys [all_lo, all_end) are visible to every real row
    int pad[4];
};
static_assert(sizeof(Desc) == 64, "descriptor size");
// The keys [lo, lim) that token tok of the segment's sequence sees (and the sinks below lo).
__device__ __forceinline__ void row_range(const AttnParams& p, const Desc& s, int tok, int& lo, int& lim) {
    lim = tok < s.qreal ? row_limit(p, tok, s.qreal, s.kv_len) : 0;
    lo = p.window > 0 ? s.kv_len - s.qreal + tok - p.window + 1 : 0;
}

// A chunk: shared-memory address of its K (V follows), scales, first key.
struct Chunk {
    uint32_t kb;
    float ks, vs;
    int key0;
};

// One chunk: scores, weights and the output update.  MASKED: some key of it is
// hidden from some row.
template <int D, bool FP8, int NT, bool MASKED>
__device__ __forceinline__ void chunk_step(State<D, NT>& st, uint32_t qb, const float (&fq)[NT][2],
                                           const AttnParams& p, const Desc& ds, int G, const Chunk& ch, int lane) {
    using C = Cfg<D, FP8, NT>;
    constexpr int MI = C::kKeys / 16;  // 16-key tiles of a chunk
    const int g = lane >> 2, t = lane & 3;
    // ---- S^T = K Q^T, the steps of independent accumulators in turn
    constexpr int SA = 2;  // the two tiles of 32 keys; one tile: every other step to the second
    float s[SA][NT][4];
#pragma unroll
    for (int x = 0; x < SA; ++x)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[x][j][e] = 0.f;
    if constexpr (FP8) {
        // this lane's keys of a chunk: g, g + 8, g + 16, g + 24
        const uint32_t a0 = g * D + (D == 128 ? ((2 * t) ^ g) << 4 : (t ^ ((g >> 1) & 3)) << 4);
        constexpr int MG = NT == 1 ? 2 : 1;  // tiles in turn (two row tiles make two chains already)
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
            for (int m0 = 0; m0 < MI; m0 += MG) {
                uint4 w[2 * MG];
#pragma unroll
                for (int r = 0; r < 2 * MG; ++r)
                    w[r] = lds128(ch.kb + (a0 ^ (i << 4)) + (2 * m0 + r) * 8 * D);
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) {
                    uint4 q[NT];  // steps 2 k2 and 2 k2 + 1
#pragma unroll
                    for (int j = 0; j < NT; ++j) q[j] = lds128(qb + (j * (D / 32) + 2 * i + k2) * 512);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int mi = 0; mi < MG; ++mi) {
                            uint32_t a[4];
                            widen4(word(w[2 * mi], 2 * k2 + k), a[0], a[2]);
                            widen4(word(w[2 * mi + 1], 2 * k2 + k), a[1], a[3]);
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                mma<FP8>(s[m0 + mi][j], a, word(q[j], 2 * k), word(q[j], 2 * k + 1));
                        }
                }
            }
    } else {
        const uint32_t a0 = g * 128 + (((2 * t) ^ g) << 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            uint4 q[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) q[j] = lds128(qb + (j * (D / 32) + i) * 512);
            const uint32_t ad = ch.kb + (a0 ^ ((i & 1) << 4)) + (i >> 1) * (C::kKeys * 128);
            const uint4 u = lds128(ad), v = lds128(ad + 8 * 128);
            const uint32_t x0[4] = {u.x, v.x, u.y, v.y}, x1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
            for (int j = 0; j < NT; ++j) mma<FP8>(s[0][j], x0, q[j].x, q[j].y);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma<FP8>(s[1][j], x1, q[j].z, q[j].w);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[0][j][e] += s[1][j][e];
    }
    // ---- weights
    float lv = 0.f;  // what M adds to a: log2 of the V scale, rounded down, less kWeightUp
    if constexpr (FP8) {
        const float e = static_cast<float>(static_cast<int>((__float_as_uint(ch.vs) >> 23) & 255u) - 127);
        lv = fminf(fmaxf(e, kLowScale), kHighScale) - kWeightUp;
    }
    uint32_t pb[NT][MI][2];
    bool moved = false;
    float alpha[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float ref[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            int lim = 0, lo = 0;
            if constexpr (MASKED) row_range(p, ds, (ds.row0 + 8 * j + 2 * t + e) / G, lo, lim);
            const float f = FP8 ? fq[j][e] * ch.ks : fq[j][e];
            float mx = -INFINITY;
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float x = s[mi][j][2 * hh + e] * f;
                    if constexpr (MASKED) {
                        const int key = ch.key0 + 16 * mi + 8 * hh + g;
                        if (!(key < lim && (key >= lo || key < p.num_sinks))) x = -INFINITY;
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
        for (int m = 0; m < MI; ++m)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const float p0 = fast_exp2(s[m][j][2 * hh] - ref[0]), p1 = fast_exp2(s[m][j][2 * hh + 1] - ref[1]);
                sum[0] += p0;
                sum[1] += p1;
                uint32_t w;
                if constexpr (FP8) {
                    w = pack_f16x2(p0 * ch.vs, p1 * ch.vs);
                } else {
                    w = pack_bf16x2(p0, p1);
                    sumb[0] += bf16lo(w);
                    sumb[1] += bf16hi(w);
                }
                pb[j][m][hh] = movmatrix(w);  // (key g; rows 2t, 2t + 1) -> (row g; keys 2t, 2t + 1)
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
    const uint32_t vb = ch.kb + C::kTile;
    uint32_t vm[2 * MI];
    if constexpr (MASKED) {
#pragma unroll
        for (int k = 0; k < 2 * MI; ++k) {
            uint32_t keep = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int key = ch.key0 + 8 * k + 2 * t + e;
                if (key < ds.hi && (key >= ds.lo || key < p.num_sinks)) keep |= 0xffffu << (16 * e);
            }
            vm[k] = keep;
        }
    }
    if constexpr (FP8) {
        const uint32_t a0 = vb + lane * D + (D == 128 ? (lane & 7) << 4 : ((lane >> 1) & 3) << 4);
#pragma unroll
        for (int c0 = 0; c0 < D / 16; c0 += 2) {
            uint32_t r[2][4];
#pragma unroll
            for (int c = 0; c < 2; ++c) ldmatrix_x4_trans(r[c], a0 ^ ((c0 + c) << 4));
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t a[4];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t w = r[c][2 * k + q];
                        if constexpr (MASKED) w &= vm[2 * k + q];
                        // (key 2t: dims d, d + 1; key 2t + 1: dims d, d + 1) -> d of both keys, d + 1 of both
                        widen4(__byte_perm(w, w, 0x3120), a[2 * q], a[2 * q + 1]);
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        mma<FP8>(st.o[j][c0 + c], a, pb[j][k][0], pb[j][k][1]);
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

// A lane's part of a query row, in the order the K loads give the dimensions.
template <int D, bool FP8>
__device__ __forceinline__ void fetch_q_row(const __nv_bfloat16* q, bool exists, int t, uint4 (&v)[D / 32]) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        // 8-bit: D / 4 elements from t D / 4 on; bf16: 16 of each 64 from 16 t on
        const int at = FP8 ? t * (D / 4) + 8 * i : (i >> 1) * 64 + t * 16 + (i & 1) * 8;
        v[i] = exists ? __ldg(reinterpret_cast<const uint4*>(q + at)) : make_uint4(0u, 0u, 0u, 0u);
    }
}
// The same as the score product's B operand, two steps a vector; returns the
// factor that undoes the row's scaling (1 for bf16 pools).
template <int D, bool FP8>
__device__ __forceinline__ float pack_q(uint4 (&v)[D / 32]) {
    if constexpr (!FP8) return 1.f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t w = word(v[i], k);
            top = max(top, max((w >> 7) & 255u, (w >> 23) & 255u));
        }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = max(top, 9u);
    const float up = __uint_as_float((262u - top) << 23);  // the largest exponent to 2^8
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        v[i] = make_uint4(pack_f16x2(bf16lo(v[i].x) * up, bf16hi(v[i].x) * up),
                          pack_f16x2(bf16lo(v[i].y) * up, bf16hi(v[i].y) * up),
                          pack_f16x2(bf16lo(v[i].z) * up, bf16hi(v[i].z) * up),
                          pack_f16x2(bf16lo(v[i].w) * up, bf16hi(v[i].w) * up));
    return __uint_as_float((top - 8u) << 23);
}

struct Look {
    int page, key0;
    float ks, vs;
};

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__((Cfg<D, FP8, NT>::kThreads), (Cfg<D, FP8, NT>::kCtasPerSm))
    attn_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ RowsArgs a) {
    using C = Cfg<D, FP8, NT>;
    using W = Walk<C::kRows, C::kKeys>;
    constexpr int S = C::kStages, NW = C::kWarps;
    const AttnParams& p = a.p;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.num_q_heads / p.num_kv_heads, Hkv = p.num_kv_heads;

    if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle needs 1024-byte aligned tiles
        if (threadIdx.x == 0) set_err(p.err, PKV_ERRBIT_TIMEOUT);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint64_t* empty = full + S;
    uint64_t* dfull = empty + S;
    uint64_t* dempty = dfull + kDescs;
    uint64_t* bfull = dempty + kDescs;
    uint64_t* bempty = bfull + kBatches;
    uint64_t* never = bempty + kBatches;  // nothing completes it
    const uint64_t limit = p.test_wait_timeout ? kTestWaitNs : kWaitNs;
    float4* meta = reinterpret_cast<float4*>(smem + C::kMetaOff);
    Desc* desc = reinterpret_cast<Desc*>(smem + C::kDescOff);
    Look* queue = reinterpret_cast<Look*>(smem + C::kQueueOff);
    int2* head = reinterpret_cast<int2*>(smem + C::kHeadOff);
    if (threadIdx.x == 0) {
        *reinterpret_cast<int2*>(smem + C::kFlagOff) = make_int2(0, 0);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kDescs; ++s) {
            mbar_init(&dfull[s], 1);
            mbar_init(&dempty[s], NW);
        }
        for (int s = 0; s < kBatches; ++s) {
            mbar_init(&bfull[s], 32);
            mbar_init(&bempty[s], 32);
        }
        mbar_init(never, 1);
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == NW) {
        // ============================ look-up ===============================
        // The first piece of a small batch is found here, from the lengths, while
        // the planner (launched before this grid, with programmatic
        // serialisation) still runs; what it wrote is read behind await_planner.
        // (One small loop for both passes: at a launch's start, straight-line
        // code costs its instruction fetches.)
        if (a.ctas > 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join, behind this grid
        bool planned = false;
        auto await_planner = [&] {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            planned = true;
        };
        W w;
        w.b = w.kvh = w.mt = w.at = w.left = 0;
        int T = 0, piece = blockIdx.x;
        const bool self = p.batch <= kSelfBatch;
        if (a.ctas > 0 && !self) {
            await_planner();
            T = __ldcg(a.seq_at + p.batch);
        } else if (a.ctas > 0) {
            int at = -1;  // pass 0: the line's length; pass 1: the sequence that holds its place `at`
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                int base = 0;
#pragma unroll 1
                for (int b0 = 0; b0 < p.batch; b0 += 32) {
                    int per_head = 0;
                    if (b0 + lane < p.batch) {
                        const Seq s = sequence<C::kRows>(p, b0 + lane, G);
#pragma unroll 1
                        for (int mt = 0; mt < s.tiles; ++mt)
                            per_head += max(span_of<C::kRows, C::kKeys>(p, s, mt, G).n, 1);
                    }
                    int incl = per_head * Hkv;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += y;
                    }
                    const uint32_t ends = __ballot_sync(0xffffffffu, pass == 1 && base + incl > at);
                    if (ends) {  // the first sequence to end behind it
                        const int l = __ffs(ends) - 1;
                        per_head = __shfl_sync(0xffffffffu, per_head, l);
                        at -= base + __shfl_sync(0xffffffffu, incl, l) - per_head * Hkv;
                        w.b = b0 + l;
                        w.kvh = at / per_head;
                        w.at = at - w.kvh * per_head;
                        break;
                    }
                    base += __shfl_sync(0xffffffffu, incl, 31);
                }
                if (pass == 0) {
                    T = base;
                    const Line line(T, a.ctas, a.even);
                    if (piece >= line.first) break;
                    int to;
                    line.piece(piece, at, to);
                    w.left = to - at;
                    if (w.left == 0) break;
                }
            }
        }
        const Line line(T, max(a.ctas, 1), a.even);
        const int pieces = line.pieces();
        int nseg = 0, nbatch = 0;
        bool alive = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit)); };
        for (bool fixed = true; alive; fixed = false) {
            // ---- the next piece, by ticket; in a small call every gridDim-th unit, whole
            if (a.ctas == 0) {
                if (!fixed) piece += gridDim.x;
                if (piece >= a.tiles_max * Hkv * p.batch) break;
                w.mt = piece % a.tiles_max;
                w.kvh = (piece / a.tiles_max) % Hkv;
                w.b = piece / a.tiles_max / Hkv;
                w.at = 0;
                w.left = w.mt < sequence<C::kRows>(p, w.b, G).tiles ? 0x7fffffff : 0;
            } else if (!(fixed && self && piece < line.first)) {
                if (!planned) await_planner();
                if (!fixed || piece >= line.first) {
                    int tk = 0;
                    if (lane == 0) tk = atomicAdd(a.ticket, 1);
                    piece = line.first + __shfl_sync(0xffffffffu, tk, 0);
                }
                if (piece >= pieces) break;
                int from, to;
                line.piece(piece, from, to);
                const int4 at = __ldcg(a.starts + piece);
                w.b = at.x;
                w.kvh = at.y;
                w.mt = 0;
                w.at = at.z;
                w.left = to - from;
            }
            // ---- its segments
            while (alive && w.next(p, G)) {
                const int ds = nseg % kDescs;
                if (nseg >= kDescs && !wait(&dempty[ds], (nseg / kDescs - 1) & 1)) {
                    alive = false;
                    break;
                }
                if (lane == 0) {
                    Desc d;
                    d.r0 = w.s.r0;
                    d.nrows = w.s.nrows;
                    d.qreal = w.s.qreal;
                    d.kv_len = w.s.kv_len;
                    d.lo = w.u.lo;
                    d.hi = w.u.hi;
                    d.kvh = w.skvh;
                    d.row0 = w.smt * C::kRows;
                    d.n = max(w.pe - w.ps, 0);
                    {
                        const int tf = d.row0 / G, tl = min((d.row0 + C::kRows - 1) / G, d.qreal - 1);
                        d.all_end = tf < d.qreal ? row_limit(p, tf, d.qreal, d.kv_len) : 0;
                        d.all_lo = p.window > 0 ? max(0, d.kv_len - d.qreal + tl - p.window + 1) : 0;
                    }
                    d.frag = w.starts && w.ends ? -1 : piece + (w.sb * Hkv + w.skvh) * a.tiles_max + w.smt;
                    desc[ds] = d;
                    mbar_arrive(&dfull[ds]);
                    if (p.checked && w.starts && w.skvh == 0 && w.smt == 0) {
                        const int rows = p.q_indptr[w.sb + 1] - w.s.r0, kv = p.kv_lens[w.sb];
                        if (kv > p.max_kv_len || kv < 0 || rows > p.max_q_rows || (p.q_real && p.q_real[w.sb] > rows))
                            set_err(p.err, PKV_ERRBIT_LEN);
                    }
                }
                __syncwarp();
                ++nseg;
                if (a.ctas == 0) w.left = 0;  // its one unit
                for (int c0 = w.ps; c0 < w.pe; c0 += 32) {
                    // pages and scales of the next 32 chunks, one a lane
                    const int bs = nbatch % kBatches;
                    if (nbatch >= kBatches && !wait(&bempty[bs], (nbatch / kBatches - 1) & 1)) {
                        alive = false;
                        break;
                    }
                    const int i = c0 + lane;
                    Look k;
                    k.key0 = (i < w.u.nsc ? i : w.u.loc + i - w.u.nsc) * C::kKeys;
                    k.page = static_cast<int>(p.num_pages);  // outside the tensor: the copy fills zeros
                    k.ks = k.vs = 0.f;
                    if (i < w.pe) {
                        const int x = p.block_table[w.sb * p.block_table_stride + k.key0 / kPage];
                        if (x >= 0 && x < p.num_pages) {
                            k.page = x;
                            if constexpr (FP8) {
                                k.ks = __ldg(p.k_scale + x * p.scale_stride + w.skvh);
                                k.vs = __ldg(p.v_scale + x * p.scale_stride + w.skvh);
                            }
                        } else if (p.checked) {
                            set_err(p.err, PKV_ERRBIT_PAGE);
                        }
                    }
                    queue[bs * 32 + lane] = k;
                    if (lane == 0) head[bs] = make_int2(min(32, w.pe - c0), w.skvh);
                    mbar_arrive(&bfull[bs]);
                    ++nbatch;
                }
            }
        }
        if (!alive && lane == 0) set_err(p.err, PKV_ERRBIT_TIMEOUT);
        // the join waits for this grid alone and reads what the planner wrote, so
        // a look-up that gave up before it needed the planner waits for it here
        if (a.ctas > 0 && !planned) await_planner();
        // the end marks (where a wait gave up, the readers' own waits run out too)
        const int bs = nbatch % kBatches, ds = nseg % kDescs;
        if (nbatch < kBatches || wait(&bempty[bs], (nbatch / kBatches - 1) & 1)) {
            if (lane == 0) head[bs] = make_int2(-1, 0);
            mbar_arrive(&bfull[bs]);
        }
        if (nseg < kDescs || wait(&dempty[ds], (nseg / kDescs - 1) & 1)) {
            if (lane == 0) {
                desc[ds].n = -1;
                mbar_arrive(&dfull[ds]);
            }
        }
        return;
    }
    if (warp == NW + 1) {
        // ============================= copies ===============================
        if (lane == 0) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
        }
        int issued = 0, gave_up = -1;
        bool alive = true;
        for (int nb = 0; alive; ++nb) {
            const int bs = nb % kBatches;
            if (!__all_sync(0xffffffffu, mbar_wait(&bfull[bs], (nb / kBatches) & 1))) {
                alive = false;
                break;
            }
            const int2 h = head[bs];
            if (h.x < 0) break;
            const Look k = queue[bs * 32 + lane];
            mbar_arrive(&bempty[bs]);
            // as many chunks at once as there are stages: each lane copies one, as
            // soon as its stage is free (one after the other, a chunk took ~500
            // cycles of this warp, the limit at head dim 64)
            constexpr int kAtOnce = S < 32 ? S : 32;
            for (int l0 = 0; alive && l0 < h.x; l0 += kAtOnce) {
                const int n = min(kAtOnce, h.x - l0);
                const int src = l0 + lane;
                Look c;
                c.page = __shfl_sync(0xffffffffu, k.page, src & 31);
                c.key0 = __shfl_sync(0xffffffffu, k.key0, src & 31);
                c.ks = __shfl_sync(0xffffffffu, k.ks, src & 31);
                c.vs = __shfl_sync(0xffffffffu, k.vs, src & 31);
                const int at = issued + lane, st = at % S;
                bool todo = lane < n;
                uint64_t t0 = 0;
                for (uint32_t it = 0; __any_sync(0xffffffffu, todo); ++it) {
                    if (todo && (at < S || mbar_try_wait(&empty[st], (at / S - 1) & 1))) {
                        uint8_t* kd = smem + st * C::kStage;
                        uint8_t* vd = kd + C::kTile;
                        meta[st] = make_float4(c.ks, c.vs, __int_as_float(c.key0), 0.f);
                        mbar_arrive_expect_tx(&full[st], C::kStage);
                        if constexpr (FP8) {
                            tma_load_4d(kd, &tm_k, &full[st], 0, h.y, 0, c.page);
                            tma_load_4d(vd, &tm_v, &full[st], 0, h.y, 0, c.page);
                        } else {
#pragma unroll
                            for (int x = 0; x < D / 64; ++x) {
                                tma_load_4d(kd + x * (C::kKeys * 128), &tm_k, &full[st], x * 64, h.y, c.key0 % kPage, c.page);
                                tma_load_4d(vd + x * (C::kKeys * 128), &tm_v, &full[st], x * 64, h.y, c.key0 % kPage, c.page);
                            }
                        }
                        todo = false;
                    }
                    if ((it & 63u) == 63u) {
                        const uint64_t now = global_timer_ns();
                        if (t0 == 0) t0 = now;
                        if (__any_sync(0xffffffffu, now - t0 > limit)) {
                            alive = false;
                            break;
                        }
                    }
                }
                // (after a wait that gave up: the lanes that did issue are not one
                // run of stages; every one is waited for below)
                if (!alive) {
                    gave_up = todo || lane >= n ? -1 : at;
                    break;
                }
                issued += n;
            }
        }
        if (!alive && lane == 0) set_err(p.err, PKV_ERRBIT_TIMEOUT);
        // do not leave with copies into this CTA's shared memory in flight
        for (int j = max(0, issued - S); j < issued; ++j) mbar_wait(&full[j % S], (j / S) & 1);
        if (gave_up >= 0) mbar_wait(&full[gave_up % S], (gave_up / S) & 1);
        return;
    }

    // ============================== consumers ===============================
    const int g = lane >> 2, t = lane & 3;
    float* red = reinterpret_cast<float*>(smem + C::kRedOff);
    float* red_m = reinterpret_cast<float*>(smem + C::kStatOff);
    float* red_l = red_m + NW * C::kRows;
    float* red_lb = red_l + NW * C::kRows;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kFlagOff);
    const uint32_t ring_u = smem_u32(smem);
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"r"(NW * 32) : "memory"); };
    int own = 0;      // stage of the warp's next chunk among its own, and its phase
    uint32_t phase = 0;
    int turn = 0;     // consumer whose turn the segment's first chunk is
    // A segment's query rows, in fragment order in shared memory: tile j is
    // brought in by warp j, while the segment before it is joined if its
    // descriptor is there by then.
    uint4* qs = reinterpret_cast<uint4*>(smem + C::kQOff);
    float* facs = reinterpret_cast<float*>(smem + C::kFacOff);
    const uint32_t qb = smem_u32(qs + lane);
    volatile int* staged = reinterpret_cast<volatile int*>(smem + C::kFlagOff) + 1;  // segments staged
    uint4 raw[D / 32];
    auto fetch_q = [&](const Desc& s) {
        const int R = s.row0 + 8 * warp + g;
        const int tok = R / G, h = s.kvh * G + R % G;
        fetch_q_row<D, FP8>(static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(s.r0 + tok) * p.q_token_stride +
                                static_cast<int64_t>(h) * p.q_head_stride,
                            tok < s.nrows, t, raw);
    };
    auto stage_q = [&] {
        const float undo = pack_q<D, FP8>(raw);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) qs[(warp * (D / 32) + i) * 32 + lane] = raw[i];
        if (t == 0) facs[8 * warp + g] = p.scale_log2 * undo;
    };
    for (int nseg = 0;; ++nseg) {
        const int ds = nseg % kDescs;
        bool dead = !__all_sync(0xffffffffu, mbar_wait(&dfull[ds], (nseg / kDescs) & 1));
        const Desc& s = desc[ds];
        const bool run = !dead && s.n >= 0;
        const int R0 = s.row0;
        State<D, NT> st;
        if (*staged <= nseg) {  // the same for all: written before the last barrier
            if (run && warp < NT) {
                fetch_q(s);
                stage_q();
            }
            sync();
        }
        if (run) {
            float fq[NT][2];  // score factors of this lane's rows
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) fq[j][e] = facs[8 * j + 2 * t + e];
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
            // the test hook: a wait that runs out before the first chunk
            if (p.test_wait_timeout && !__all_sync(0xffffffffu, mbar_wait(never, 0, kTestWaitNs))) dead = true;
            for (int i = warp >= turn ? warp - turn : warp - turn + NW; i < s.n && !dead; i += NW) {
                const int sg = own * NW + warp;
                if (!__all_sync(0xffffffffu, mbar_wait(&full[sg], phase))) {
                    dead = true;
                    break;
                }
                const float4 me = meta[sg];
                const Chunk ch{ring_u + sg * C::kStage, me.x, me.y, __float_as_int(me.z)};
                const bool whole = ch.key0 + C::kKeys <= s.all_end &&
                                   (ch.key0 >= s.all_lo || ch.key0 + C::kKeys <= p.num_sinks);
                if (whole) chunk_step<D, FP8, NT, false>(st, qb, fq, p, s, G, ch, lane);
                else chunk_step<D, FP8, NT, true>(st, qb, fq, p, s, G, ch, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[sg]);
                if (++own == C::kOwn) {
                    own = 0;
                    phase ^= 1;
                }
            }
            // ---- join the warps' states, kRedRows rows at a time
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
        }
        if (dead && lane == 0) {
            set_err(p.err, PKV_ERRBIT_TIMEOUT);
            *abort_flag = 1;
        }
        constexpr int RR = C::kRedRows, RS = C::kRedStride;
        auto put_rows = [&](int rg) {  // rows RR rg .. RR rg + RR - 1: tile rg
            float* r0 = red + (warp * RR + 2 * t) * RS;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const float(&o)[4] = st.o[rg][c];
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
        };
        if (run) put_rows(0);
        // the next segment's query rows, on their way while this one is joined
        bool ahead = false;
        if (NT == 1 && run && warp == 0) {
            const int dn = (nseg + 1) % kDescs;
            ahead = __all_sync(0xffffffffu, mbar_test(&dfull[dn], ((nseg + 1) / kDescs) & 1)) && desc[dn].n >= 0;
            if (ahead) fetch_q(desc[dn]);
        }
        // every consumer passes here once a segment, whether its waits held or not
        sync();
        if (*abort_flag || !run) break;
        if (NT == 1 && ahead) {  // nobody reads this segment's rows any more
            stage_q();
            if (lane == 0) *staged = nseg + 2;
        }
        const int rows_here = min(C::kRows, s.nrows * G - R0);
        // rows RR rg .. RR rg + RR - 1 of the warps' states in red / red_m / red_l: joined and written,
        // as the result or as a partial state; four dimensions a thread (a row's
        // factors are computed by each of its threads: with two dimensions each
        // and four rows at a time, 16-row calls took 131 us instead of 120, with
        // eight dimensions 120 too)
        auto join_rows = [&](int rg) {
            for (int e = threadIdx.x; e < RR * D / 4; e += NW * 32) {
                const int rr = e / (D / 4), d = (e - rr * (D / 4)) * 4;
                const int r = RR * rg + rr;
                if (r >= rows_here) continue;
                const int tok = (R0 + r) / G, h = s.kvh * G + (R0 + r) % G;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < NW; ++w) M = fmaxf(M, red_m[w * C::kRows + r]);
                float L = 0.f, Lb = 0.f;
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                if (tok < s.qreal) {
                    // (no visible key: every l and o is 0, or NaN where a score was)
                    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
                    for (int k = 0; k < NW; ++k) {
                        // by the place of the warps' chunks in the segment, not by the warp's
                        // number: which warp had the first depends on what came before
                        const int w = (turn + k) % NW;
                        const float f = fast_exp2(red_m[w * C::kRows + r] - ref);
                        const float4 o = *reinterpret_cast<const float4*>(red + (w * RR + rr) * RS + d);
                        L = fmaf(f, red_l[w * C::kRows + r], L);
                        if constexpr (!FP8) Lb = fmaf(f, red_lb[w * C::kRows + r], Lb);
                        O.x = fmaf(f, o.x, O.x);
                        O.y = fmaf(f, o.y, O.y);
                        O.z = fmaf(f, o.z, O.z);
                        O.w = fmaf(f, o.w, O.w);
                    }
                }
                // bf16 weights: normalised by the sum of the rounded ones
                const float div = FP8 ? L : Lb;
                const float inv = div > 0.f ? 1.0f / div : (div == div ? 0.f : div);
                O.x *= inv;
                O.y *= inv;
                O.z *= inv;
                O.w *= inv;
                const float lse2 = L == 0.f ? -INFINITY : M + __log2f(L);
                if (s.frag < 0) {
                    const int64_t ot = static_cast<int64_t>(s.r0 + tok) * p.num_q_heads + h;
                    if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + ot * D + d) = O;
                    else
                        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + ot * D + d) =
                            make_uint2(pack_bf16x2(O.x, O.y), pack_bf16x2(O.z, O.w));
                    if (p.lse && d == 0) p.lse[ot] = lse2 * kLn2;
                } else {
                    const int64_t fr = static_cast<int64_t>(s.frag) * C::kRows + r;
                    __stcg(reinterpret_cast<float4*>(a.frag_o + fr * D + d), O);
                    if (d == 0) __stcg(a.frag_lse + fr, lse2);
                }
            }
        };
#pragma unroll
        for (int rg = 0; rg < C::kRows / RR; ++rg) {
            if (RR * rg < rows_here) {
                if (rg > 0) {
                    put_rows(rg);
                    sync();
                }
                join_rows(rg);
                sync();
            }
        }
        turn = (turn + s.n) % NW;
        __syncwarp();
        if (lane == 0) mbar_arrive(&dempty[ds]);
    }
}

// The line: where each sequence's units start, one place per chunk (and one for
// a unit without any), and what each piece starts with.  One CTA; also clears
// the ticket and the counts.
constexpr int kPlanThreads = 1024;
constexpr int kPlanSeqs = 2048;  // sequences whose places stay in shared memory
template <int ROWS, int KEYS>
__global__ void __launch_bounds__(kPlanThreads) attn_rows_plan_kernel(const __grid_constant__ RowsArgs a) {
    __shared__ int warp_sum[32];
    __shared__ int places[kPlanSeqs + 1];
    const AttnParams& p = a.p;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int G = p.num_q_heads / p.num_kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) *a.ticket = 0;
    int* seq_at = p.batch <= kPlanSeqs ? places : a.seq_at;
    int base = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int mine = 0;
        if (b < p.batch) {
            const Seq s = sequence<ROWS>(p, b, G);
            for (int mt = 0; mt < s.tiles; ++mt) mine += max(span_of<ROWS, KEYS>(p, s, mt, G).n, 1);
            mine *= p.num_kv_heads;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int v = warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        const int upto = __shfl_sync(0xffffffffu, v, max(warp - 1, 0));
        const int before = base + (warp > 0 ? upto : 0) + incl - mine;
        if (b < p.batch) {
            seq_at[b] = before;
            a.seq_at[b] = before;
        }
        base += __shfl_sync(0xffffffffu, v, 31);
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        seq_at[p.batch] = base;
        a.seq_at[p.batch] = base;
    }
    __syncthreads();
    const Line line(base, a.ctas, a.even);
    for (int i = threadIdx.x; i < line.pieces(); i += kPlanThreads) {
        int from, to;
        line.piece(i, from, to);
        if (from >= to) continue;
        int lo = 0, hi = p.batch - 1;  // the last sequence that starts at or before it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_at[mid] <= from) lo = mid;
            else hi = mid - 1;
        }
        const int per_head = (seq_at[lo + 1] - seq_at[lo]) / p.num_kv_heads;
        const int kvh = (from - seq_at[lo]) / per_head;
        a.starts[i] = make_int4(lo, kvh, from - seq_at[lo] - kvh * per_head, 0);
    }
    // the units that pieces cut
    const int units = a.tiles_max * p.num_kv_heads * p.batch;
    for (int u = threadIdx.x; u < units; u += kPlanThreads) {
        const int mt = u % a.tiles_max, kvh = u / a.tiles_max % p.num_kv_heads, b = u / a.tiles_max / p.num_kv_heads;
        const int per_head = (seq_at[b + 1] - seq_at[b]) / p.num_kv_heads;
        int at = seq_at[b] + kvh * per_head, n = per_head;
        bool exists = n > 0;
        if (a.tiles_max > 1) {
            const Seq s = sequence<ROWS>(p, b, G);
            exists = mt < s.tiles;
            for (int m = 0; m < mt && exists; ++m) at += max(span_of<ROWS, KEYS>(p, s, m, G).n, 1);
            if (exists) n = max(span_of<ROWS, KEYS>(p, s, mt, G).n, 1);
        }
        int2 cut = make_int2(0, 0);
        if (exists) {
            const int i0 = line.piece_of(at), i1 = line.piece_of(at + n - 1);
            if (i1 > i0) cut = make_int2(i0 + u, i1 - i0 + 1);
        }
        a.cuts[u] = cut;
    }
}

// Joins the partial states of the units that pieces cut: block (unit, four of
// its rows), PARTS warps a row that take every PARTS-th state, a lane D / 32
// dimensions.  One part where the units are many (a handful of states each,
// and a wave of blocks), four for few long units (up to a hundred each).
template <int D, int ROWS, int PARTS>
__global__ void __launch_bounds__(PARTS * 128) attn_rows_join_kernel(const __grid_constant__ RowsArgs a) {
    constexpr int DPL = D / 32, kAhead = 8;
    __shared__ float part_o[PARTS > 1 ? PARTS - 1 : 1][4][D];
    const AttnParams& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x;
    const int mt = unit % a.tiles_max, kvh = unit / a.tiles_max % p.num_kv_heads;
    const int b = unit / a.tiles_max / p.num_kv_heads;
    const int G = p.num_q_heads / p.num_kv_heads;
    const int q0 = p.q_indptr[b];
    const int nrows = min(p.q_indptr[b + 1] - q0, p.max_q_rows);
    const int row = warp & 3, part = warp >> 2;
    const int r = blockIdx.y * 4 + row, R = mt * ROWS + r;
    const bool exists = R / G < nrows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int2 cut = __ldcg(a.cuts + unit);
    if (cut.y == 0 || mt * ROWS + static_cast<int>(blockIdx.y) * 4 >= nrows * G) return;  // uniform
    float M = -INFINITY, L = 0.f, O[DPL];
#pragma unroll
    for (int i = 0; i < DPL; ++i) O[i] = 0.f;
    if (exists) {
        const float* lse = a.frag_lse + static_cast<int64_t>(cut.x) * ROWS + r;
        const float* o = a.frag_o + (static_cast<int64_t>(cut.x) * ROWS + r) * D + lane * DPL;
        // 32 states at a time: their sums in the lanes, this warp's outputs in flight with them
#pragma unroll 1
        for (int k0 = 0; k0 < cut.y; k0 += 32) {
            const int n = min(32, cut.y - k0);
            const float e = lane < n ? __ldcg(lse + static_cast<int64_t>(k0 + lane) * ROWS) : -INFINITY;
            float w = 0.f;
#pragma unroll 1
            for (int x0 = 0; x0 < n; x0 += PARTS * kAhead) {
                float v[kAhead][DPL];
#pragma unroll
                for (int x = 0; x < kAhead; ++x) {
                    const int k = x0 + PARTS * x + part;
                    const float* src = o + static_cast<int64_t>(k0 + k) * (ROWS * D);
                    if constexpr (DPL == 4) {
                        const float4 u = k < n ? __ldcg(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
                        v[x][0] = u.x;
                        v[x][1] = u.y;
                        v[x][2] = u.z;
                        v[x][3] = u.w;
                    } else {
                        const float2 u = k < n ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
                        v[x][0] = u.x;
                        v[x][1] = u.y;
                    }
                }
                if (x0 == 0) {
                    const float Mn = fmaxf(M, warp_max(e));
                    const float ref = Mn == -INFINITY ? 0.f : Mn;
                    const float f = fast_exp2(M - ref);
                    w = fast_exp2(e - ref);
                    M = Mn;
                    L = fmaf(L, f, warp_sum(w));
#pragma unroll
                    for (int i = 0; i < DPL; ++i) O[i] *= f;
                }
#pragma unroll
                for (int x = 0; x < kAhead; ++x) {
                    const float wx = __shfl_sync(0xffffffffu, w, (x0 + PARTS * x + part) & 31);
                    if (x0 + PARTS * x + part < n)
#pragma unroll
                        for (int i = 0; i < DPL; ++i) O[i] = fmaf(wx, v[x][i], O[i]);
                }
            }
        }
        if (part > 0)
#pragma unroll
            for (int i = 0; i < DPL; ++i) part_o[part - 1][row][lane * DPL + i] = O[i];
    }
    __syncthreads();
    if (!exists || part > 0) return;
    const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
    for (int i = 0; i < DPL; ++i) {
#pragma unroll
        for (int x = 0; x < PARTS - 1; ++x) O[i] += part_o[x][row][lane * DPL + i];
        O[i] *= inv;
    }
    const int64_t ot = static_cast<int64_t>(q0 + R / G) * p.num_q_heads + kvh * G + R % G;
#pragma unroll
    for (int i = 0; i < DPL; i += 2) {
        const int64_t at = ot * D + lane * DPL + i;
        if (p.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at) = make_float2(O[i], O[i + 1]);
        else *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at) = pack_bf16x2(O[i], O[i + 1]);
    }
    if (p.lse && lane == 0) p.lse[ot] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
}

template <int D, bool FP8, int NT>
cudaError_t launch_rows(const RowsArgs& a, int resident, const void* tk, const void* tv, cudaStream_t s) {
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
    const unsigned units = static_cast<unsigned>(a.tiles_max * a.p.num_kv_heads * a.p.batch);
    if (a.ctas == 0) {
        kern<<<std::min(units, static_cast<unsigned>(resident)), C::kThreads, C::kBytes, s>>>(mk, mv, a);
        return cudaGetLastError();
    }
    attn_rows_plan_kernel<C::kRows, C::kKeys><<<1, kPlanThreads, 0, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // each behind the one before with programmatic serialisation: it starts beside it
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, mk, mv, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(units, C::kRows / 4);
    cfg.blockDim = dim3(a.even ? 512 : 128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, a.even ? attn_rows_join_kernel<D, C::kRows, 4> : attn_rows_join_kernel<D, C::kRows, 1>,
                              a);
}

// The workspace of the cut line.
struct RowsSpace {
    size_t ticket, cuts, seq_at, starts, frag_lse, frag_o, bytes;
    RowsSpace(int batch, int64_t units, int ctas, int rows, int D) {
        auto take = [this](size_t n) {
            const size_t at = bytes;
            bytes += (n + 255) / 256 * 256;
            return at;
        };
        const size_t pieces = Line::most(ctas), frags = pieces + static_cast<size_t>(units);
        bytes = 0;
        ticket = take(sizeof(int));
        cuts = take(units * sizeof(int2));
        seq_at = take((static_cast<size_t>(batch) + 1) * sizeof(int));
        starts = take(pieces * sizeof(int4));
        frag_lse = take(frags * rows * sizeof(float));
        frag_o = take(frags * rows * D * sizeof(float));
    }
};

}  // namespace

// Whole units while a unit is short (kDirectBytes of K and V at the host
// bound, what a CTA streams in about 6 us) or the rows alone make units enough (more than kCutTiles
// tiles a sequence, whose places the planner would add up one by one); else
// the cut line.
RowsPlan plan_attn_rows(int batch, int max_q_rows, int Hq, int Hkv, int D, int max_kv_len, int window,
                        int num_sinks, bool fp8, int sms) {
    constexpr int64_t kDirectBytes = 384 * 1024;
    constexpr int kCutTiles = 16;
    RowsPlan pl{};
    const int64_t rows = static_cast<int64_t>(max_q_rows) * (Hq / Hkv);
    pl.row_tiles = rows <= 8 ? 1 : 2;
    const int R = 8 * pl.row_tiles;
    pl.tiles = (rows + R - 1) / R;
    pl.units = pl.tiles * Hkv * batch;
    int64_t keys = max_kv_len;
    if (window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(window) + R + std::min(num_sinks, max_kv_len) + 62);
    const double places = static_cast<double>(pl.units) * (std::min<double>(keys, max_kv_len) / 16 + 3);
    pl.resident = (D == 64 && pl.row_tiles == 1 ? Cfg<64, true, 1>::kCtasPerSm : Cfg<128, true, 1>::kCtasPerSm) * sms;
    if (keys * 2 * D * (fp8 ? 1 : 2) <= kDirectBytes || pl.tiles > kCutTiles || places > 2e9) return pl;  // the line is counted in 32 bits
    pl.ctas = pl.resident;
    pl.ws_bytes = RowsSpace(batch, pl.units, pl.ctas, R, D).bytes;
    return pl;
}

cudaError_t launch_attn_rows(const AttnParams& p, const RowsPlan& pl, void* workspace, const void* tk,
                             const void* tv, cudaStream_t s) {
    if (pl.units > 0x7fffffff - Line::most(pl.ctas)) return cudaErrorInvalidConfiguration;
    RowsArgs a{};
    a.p = p;
    a.ctas = pl.ctas;
    a.tiles_max = static_cast<int>(pl.tiles);
    a.even = pl.units < pl.ctas;
    if (pl.ctas > 0) {
        const RowsSpace x(p.batch, pl.units, pl.ctas, 8 * pl.row_tiles, p.head_dim);
        char* w = static_cast<char*>(workspace);
        a.ticket = reinterpret_cast<int*>(w + x.ticket);
        a.cuts = reinterpret_cast<int2*>(w + x.cuts);
        a.seq_at = reinterpret_cast<int*>(w + x.seq_at);
        a.starts = reinterpret_cast<int4*>(w + x.starts);
        a.frag_lse = reinterpret_cast<float*>(w + x.frag_lse);
        a.frag_o = reinterpret_cast<float*>(w + x.frag_o);
    }
#define PKV_ROWS(D_, F_, N_) \
    if (p.head_dim == D_ && p.kv_fp8 == F_ && pl.row_tiles == N_) return launch_rows<D_, F_, N_>(a, pl.resident, tk, tv, s);
    PKV_ROWS(128, true, 1) PKV_ROWS(128, true, 2) PKV_ROWS(128, false, 1) PKV_ROWS(128, false, 2)
    PKV_ROWS(64, true, 1) PKV_ROWS(64, true, 2) PKV_ROWS(64, false, 1) PKV_ROWS(64, false, 2)
#undef PKV_ROWS
    return cudaErrorInvalidValue;
}

}  // namespace pkv
