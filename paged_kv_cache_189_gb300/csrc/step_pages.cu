// step_pages.cu -- assign_step_pages: a step's block tables, query ranges and
// slot map from the requests' lengths, in one launch.
//
// The rules are running sums over the batch (tokens asked for, pages needed,
// pages given back), so every CTA of one cluster reads all lengths and computes
// them for itself; only the writes are shared out.  One cluster barrier
// separates reading the inputs and pushing the finished sequences' pages from
// everything that is written over them or read from the stack.  A call is
// latency: launch, lengths, five block scans, search, stack or table look-up,
// store.  Measured, replayed as a graph: 6.0 us for 64 decoding sequences (one CTA
// instead of the cluster: the same), 6.6 for 256 (7.7), 11.6 for 768 with 25 k
// tokens (41.6).
#include <cooperative_groups.h>

#include "latent.h"
#include "pkv_common.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxPer = 8;  // sequences a thread holds: 4096 / 512
constexpr int kCluster = 8;

// Exclusive running sum over the block of one 64-bit value a thread; the total in *total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* total) {
    __shared__ int64_t part[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous scan's parts have been read
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? part[w] : 0;
        all += part[w];
    }
    *total = all;
    return before + x - v;
}

__device__ __forceinline__ int64_t pages_of(int64_t keys) { return (keys + 31) >> 5; }

// The first index whose running sum lies past v (the last one has one that does).
__device__ __forceinline__ int upper(const int32_t* ends, int count, int v) {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > v) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) step_pages_kernel(const StepPagesArgs a) {
    // per sequence, running sums up to and with it: granted tokens, pages taken, pages
    // given back; and its keys before the step
    extern __shared__ int32_t state[];
    int32_t* tok_end = state;
    int32_t* take_end = state + a.batch;
    int32_t* back_end = state + 2 * a.batch;
    int32_t* kv_of = state + 3 * a.batch;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
    const int tid = threadIdx.x;
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int64_t stride = a.block_table_stride;

    int kv[kMaxPer], ask[kMaxPer];  // ask < 0: finished
    int64_t tokens = 0, need = 0, back = 0;
    int bad = 0;
#pragma unroll
    for (int k = 0; k < kMaxPer; ++k) {
        const int b = tid * per + k;
        kv[k] = ask[k] = 0;
        if (k >= per || b >= a.batch) continue;
        kv[k] = a.kv_lens[b];
        ask[k] = a.new_lens[b];
        if (kv[k] < 0) {
            kv[k] = 0;
            bad |= PKV_ERRBIT_PAGE;
        }
        tokens += max(ask[k], 0);
        if (ask[k] > 0) need += pages_of(int64_t(kv[k]) + ask[k]) - pages_of(kv[k]);
        if (ask[k] < 0) back += min(pages_of(kv[k]), stride);
    }
    const int free_in = *a.num_free;
    const int64_t height = min(max(int64_t(free_in), int64_t(0)), a.free_capacity);
    if (height != free_in) bad |= PKV_ERRBIT_PAGE;
    int64_t total, back_total;
    int64_t token_sum = block_scan(tokens, &total);
    int64_t need_sum = block_scan(need, &total);
    int64_t back_sum = block_scan(back, &back_total);
    const int64_t top = min(height + back_total, a.free_capacity);
    if (height + back_total > a.free_capacity) bad |= PKV_ERRBIT_PAGE;

    int take[kMaxPer];
    int64_t took = 0, granted = 0;
#pragma unroll
    for (int k = 0; k < kMaxPer; ++k) {
        take[k] = 0;
        const int b = tid * per + k;
        if (k >= per || b >= a.batch) continue;
        if (ask[k] < 0) back_sum += min(pages_of(kv[k]), stride);
        back_end[b] = static_cast<int32_t>(min(back_sum, a.free_capacity));  // (what lies past it is dropped)
        kv_of[b] = kv[k];
        if (ask[k] <= 0) continue;
        const int64_t n = pages_of(int64_t(kv[k]) + ask[k]) - pages_of(kv[k]);
        token_sum += ask[k];
        need_sum += n;
        const bool room = token_sum <= a.max_tokens && pages_of(int64_t(kv[k]) + ask[k]) <= stride;
        if (!room) bad |= PKV_ERRBIT_LEN;
        if (room && (n == 0 || need_sum <= top)) take[k] = static_cast<int>(n);
        else ask[k] = 0;
        took += take[k];
        granted += ask[k];
    }
    int64_t took_total, granted_total;
    int64_t took_sum = block_scan(took, &took_total);
    int64_t token_end = block_scan(granted, &granted_total);
#pragma unroll
    for (int k = 0; k < kMaxPer; ++k) {
        const int b = tid * per + k;
        if (k >= per || b >= a.batch) continue;
        took_sum += take[k];
        token_end += max(ask[k], 0);
        take_end[b] = static_cast<int32_t>(took_sum);
        tok_end[b] = static_cast<int32_t>(token_end);
        if (rank == 0) {
            // (the inputs, which these may be, are read by every CTA before the barrier below)
            kv[k] = ask[k] < 0 ? 0 : kv[k] + ask[k];
        }
    }
    if (bad && rank == 0) set_err(a.err, bad);
    __syncthreads();

    // what is done page by page or token by token is shared out over the cluster's
    // threads, each finding its sequence in the running sums
    const int first = rank * kThreads + tid, step = ranks * kThreads;
    // (counts are below 2^31, but not by as much as a step of the loops: 64 bits)
    const int64_t pushed = top - height;
    if (pushed > 0) {
        for (int64_t n = first; n < pushed; n += step) {
            const int b = upper(back_end, a.batch, static_cast<int>(n));
            a.free_pages[height + n] = a.block_table[b * stride + n - (b > 0 ? back_end[b - 1] : 0)];
        }
        __threadfence();
    }
    cluster.sync();

    // page number n of those taken lies n below the top
    auto stack_page = [&](int64_t n) { return a.free_pages[top - 1 - n]; };
    for (int64_t n = first; n < took_total; n += step) {
        const int b = upper(take_end, a.batch, static_cast<int>(n));
        a.block_table[b * stride + pages_of(kv_of[b]) + n - (b > 0 ? take_end[b - 1] : 0)] = stack_page(n);
    }
    constexpr int kAtOnce = 4;  // tokens whose look-ups are under way together
    for (int64_t t0 = first; t0 < a.max_tokens; t0 += static_cast<int64_t>(kAtOnce) * step) {
        int page[kAtOnce], pos[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int64_t t = t0 + static_cast<int64_t>(k) * step;
            page[k] = -1;
            pos[k] = 0;
            if (t >= granted_total) continue;
            const int b = upper(tok_end, a.batch, static_cast<int>(t));
            pos[k] = kv_of[b] + static_cast<int>(t) - (b > 0 ? tok_end[b - 1] : 0);
            const int lp = pos[k] >> 5, held = static_cast<int>(pages_of(kv_of[b]));
            page[k] = lp < held ? a.block_table[b * stride + lp] : stack_page((b > 0 ? take_end[b - 1] : 0) + lp - held);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int64_t t = t0 + static_cast<int64_t>(k) * step;
            if (t >= a.max_tokens) break;
            a.slots[t] = t < granted_total ? static_cast<int64_t>(page[k]) * 32 + (pos[k] & 31) : -1;
            a.positions[t] = pos[k];
        }
    }
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < kMaxPer; ++k) {
            const int b = tid * per + k;
            if (k >= per || b >= a.batch) continue;
            a.q_indptr[b + 1] = tok_end[b];
            a.kv_lens_out[b] = kv[k];
        }
        if (tid == 0) {
            a.q_indptr[0] = 0;
            *a.num_free_out = static_cast<int32_t>(top - took_total);
        }
    }
}

}  // namespace

cudaError_t launch_step_pages(const StepPagesArgs& a, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.batch) * 16;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static DeviceOnce opted;  // 4096 sequences take 64 KB
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = opted.get(dev, &done, [&](int, int* v) {
        *v = 1;
        return cudaFuncSetAttribute(step_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4096 * 16);
    });
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, step_pages_kernel, a);
}

}  // namespace pkv
