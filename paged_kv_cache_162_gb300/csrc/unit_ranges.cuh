// What the decode attention kernels that take a sequence's tokens head by head
// share (bounded.cu: 16-bit caches, q4_decode.cu: 4-bit caches): how the tiles
// of all units are cut into ranges and handed out, and how a row is gathered
// from the pieces that several ranges have of it.  The comment at the top of
// bounded.cu has the whole picture.
#pragma once

#include <climits>
#include <cmath>
#include <cstdio>
#include <mutex>

#include "bounded_place.h"
#include "pagedkv.h"
#include "pkv_device.cuh"
#include "tc_wait.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Tiles of a large range at least: a range of 8 is a chain of unit ends (100
// requests of 1..64 tokens: 19.9 us with 8, 10.9 with 2; one head of a
// 30000-token window: 16.5 and 14.0).
constexpr int kMinRange = 2;
constexpr int kMinSmall = 4;       // and of a small one: a ring is at most two ranges ahead
constexpr int kMaxGroup = 16;      // query heads per KV head
constexpr int kMaxCluster = 16;    // CTAs that share a unit in a direct call
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    void* out;
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int S, H, Hkv, G, NB, MB, bs_log2, max_ctx;
    int tile_log2;       // of a tile's tokens
    int window, sinks;   // accumulate: window = max_ctx
    int hw, nsplit, HB;  // KV heads per CTA, warps per KV head, units per sequence
    int cs;              // direct: CTAs per cluster
    int ranges0, ranges; // split: large ranges, and all of them
    float qscale;        // scale * log2(e)
    int2* place;         // [S * HB]: first and last range of each unit
    float* part_m;       // [2 * ranges][hw * G]
    float* part_l;
    float* part_acc;     // [2 * ranges][hw * G][D]
    float* row_m;        // [S][H]: M and L of units finished in one range
    float* row_l;
    float* z;            // [S][H][z_stride], accumulate only
    int64_t z_stride;
    float* scores;       // [S][Hkv][score_stride], accumulate only
    int64_t score_stride;
    int* err;
};

__device__ __forceinline__ int context_of(const Params& p, int s) {
    const int n = __ldg(p.context_lens + s);
    return n < 0 ? 0 : (n > p.max_ctx ? p.max_ctx : n);
}

__device__ __forceinline__ int visible_of(const Params& p, int n) {
    const long long most = (long long)p.window + p.sinks;
    return most < n ? (int)most : n;
}

// 1 / L, 0 for a row that sees nothing.
__device__ __forceinline__ float inverse_of(float L) { return L > 0.f || L != L ? 1.f / L : 0.f; }

// Tiles of a unit; an empty context has one, which writes zeros.
__device__ __forceinline__ int tiles_of(const Params& p, int n) {
    const int t = (visible_of(p, n) + (1 << p.tile_log2) - 1) >> p.tile_log2;
    return t < 1 ? 1 : t;
}

// How the tiles of a split call are cut (equal ranges alone: the SMs' rates differ
// and the slowest ended 10 % after the median): slots of one large range and `n_small`
// small ones after it, so that a unit has about as many pieces wherever it
// lies; kLargeShare / 16 of the tiles are in large ranges (all, where the small
// ones would be shorter than kMinSmall).  Ranges are numbered by place; CTAs are
// launched for the large ones first.
constexpr int kLargeShare = 14;
constexpr int kSmallRanges = 2;    // per large one

struct RangeMap {
    long long total, large, small, slot;
    int n_large, n_small;
    __device__ __forceinline__ void set(const Params& p, long long total_) {
        total = total_;
        n_large = p.ranges0;
        n_small = p.ranges / p.ranges0 - 1;
        const long long per = max((long long)kMinRange, (total + n_large - 1) / n_large);
        large = per;
        small = 0;
        if (n_small > 0) {
            small = per * (16 - kLargeShare) / 16 / n_small;
            // too little to share out: one range each, and numbers without gaps (a
            // unit's pieces are those of all ranges from its first to its last)
            if (small < kMinSmall) small = n_small = 0;
            large = per - n_small * small;
        }
        slot = per;
    }
    // the range of the id-th CTA launched
    __device__ __forceinline__ int of_cta(int id) const {
        if (id < n_large || n_small == 0) return id * (1 + n_small);  // n_large and up, no small ones: empty
        return (id - n_large) / n_small * (1 + n_small) + 1 + (id - n_large) % n_small;
    }
    __device__ __forceinline__ long long begin(int c) const {
        const int k = c % (1 + n_small);
        const long long x = c / (1 + n_small) * slot + (k ? large + (k - 1) * small : 0);
        return min(x, total);
    }
    __device__ __forceinline__ int of(long long tile) const {
        const int s = (int)(tile / slot);
        const long long in = tile % slot;
        return s * (1 + n_small) + (in < large ? 0 : 1 + (int)((in - large) / small));
    }
};

// A range's first unit and first tile of it.
struct Range {
    long long unit0;     // the unit's first tile, of all
    int c, s, hb, tb, n; // range, unit (s, hb), its tile, context of s
    int left;            // tiles in the range, 0: none
};

// The sequence whose units hold tile `want` * HB, by a whole warp.  before[i]:
// tiles of the sequences below run i of `per` sequences.
__device__ __forceinline__ int sequence_of(const Params& p, const long long* before, int per,
                                           long long want, int lane, long long& first) {
    int run = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k)
        run += __popc(__ballot_sync(kFull, before[32 * k + lane] <= want));
    run -= 1;  // before[0] = 0 <= want; equal entries are empty runs, the last one wins
    first = before[run];
    for (int s = run * per;; s += 32) {
        const int q = s + lane;
        const int tl = q < p.S && q < (run + 1) * per ? tiles_of(p, context_of(p, q)) : 0;
        long long in = tl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(kFull, in, o);
            if (lane >= o) in += x;
        }
        const unsigned past = __ballot_sync(kFull, first + in > want);
        if (past) {
            const int at = __ffs(past) - 1;
            first += __shfl_sync(kFull, in - tl, at);
            return s + at;
        }
        first += __shfl_sync(kFull, in, 31);
    }
}

// Shared by the CTAs' warps in a split call.
struct Plan {
    long long before[kThreads + 1];   // tiles of the sequences before each thread's run
    long long warp_sum[kWarps];
    RangeMap map;
    Range queue[kWarps][4];           // ranges a warp has begun to copy, not yet to use
    __align__(16) uint4 taken[2];     // answers of the launch control, in turn
    __align__(8) unsigned long long full[2], used[2];
    int abort;
};

// Range c as a warp finds it (whole warp; every lane returns it).
__device__ __forceinline__ Range range_at(const Params& p, const long long* before, const RangeMap& map,
                                          int c, int lane) {
    Range r;
    const long long at = map.begin(c);
    r.c = c;
    r.left = (int)(map.begin(c + 1) - at);
    if (r.left == 0) return r;
    long long first;
    const int per = (p.S + kThreads - 1) / kThreads;
    r.s = sequence_of(p, before, per, at / p.HB, lane, first);
    r.n = context_of(p, r.s);
    const long long inside = at - first * p.HB;
    const int T = tiles_of(p, r.n);
    r.hb = (int)(inside / T);
    r.tb = (int)(inside % T);
    r.unit0 = at - r.tb;
    return r;
}

__device__ __forceinline__ uint32_t smem_of(const void* x) {
    return (uint32_t)__cvta_generic_to_shared(x);
}

// Fills a CTA's plan: the tiles before each thread's run of sequences, the cuts,
// the barriers of the launch control.  By all threads; they meet at its end.
__device__ __forceinline__ void make_plan(const Params& p, Plan& plan, int tid) {
    const int warp = tid >> 5, lane = tid & 31;
    const int per = (p.S + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int i = 0; i < per; ++i) {
        const int q = tid * per + i;
        if (q < p.S) {
            const int raw = __ldg(p.context_lens + q);
            if ((raw < 0 || raw > p.max_ctx) && blockIdx.x == 0) pkv::report(p.err, PKV_DEVERR_CONTEXT);
            mine += tiles_of(p, context_of(p, q));
        }
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) plan.warp_sum[warp] = incl;
    if (tid == 0) {
        plan.abort = 0;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            tc_mbar_init(smem_of(&plan.full[b]), 1);
            tc_mbar_init(smem_of(&plan.used[b]), kWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    long long base = 0;
    for (int w = 0; w < warp; ++w) base += plan.warp_sum[w];
    plan.before[tid] = base + incl - mine;
    if (tid == kThreads - 1) {
        plan.before[kThreads] = base + incl;
        plan.map.set(p, (base + incl) * p.HB);
    }
    __syncthreads();
}

// Asks for the range of a CTA that has not been launched: request k of this
// CTA, by one thread.
__device__ __noinline__ void ask_range(Plan* plan, int k) {
    const int b = k & 1;
    // every warp has read the answer that was here
    if (k >= 2 && !tc_mbar_wait(smem_of(&plan->used[b]), ((k - 2) >> 1) & 1, &plan->abort)) return;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], 16;" ::"r"(smem_of(&plan->full[b])) : "memory");
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_of(&plan->taken[b])),
        "r"(smem_of(&plan->full[b]))
        : "memory");
}

// The next range for a warp, into its queue's entry at; false when there is
// none.  k: answers read so far.
__device__ __noinline__ bool next_range(const Params& p, Plan* plan, int warp, int lane, int& k, int at) {
    for (;;) {
        const int b = k & 1;
        const bool answered = tc_mbar_wait(smem_of(&plan->full[b]), (k >> 1) & 1, &plan->abort);
        if (!__all_sync(kFull, answered)) {
            pkv::report(p.err, PKV_DEVERR_TIMEOUT);
            *(volatile int*)&plan->abort = 1;
            return false;
        }
        uint32_t got, c;
        asm volatile(
            "{.reg .b128 h; .reg .pred ok;\n\t"
            "ld.shared.b128 h, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 ok, h;\n\t"
            "selp.u32 %0, 1, 0, ok;\n\t"
            "mov.u32 %1, 0;\n\t"
            "@ok clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;}"
            : "=r"(got), "=r"(c)
            : "r"(smem_of(&plan->taken[b]))
            : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_of(&plan->used[b])) : "memory");
        ++k;
        if (!got) return false;
        const Range r = range_at(p, plan->before, plan->map, plan->map.of_cta((int)c), lane);
        if (r.left > 0) {
            if (lane == 0) plan->queue[warp][at & 3] = r;
            __syncwarp();
            return true;
        }
        if (warp == 0 && lane == 0) ask_range(plan, k);
        __syncwarp();
    }
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Row i of a unit's hw * G over the pieces c, c + step, ... <= c1 (c0: the range
// where the unit begins), U pieces' loads in flight: (M, L) and the unnormalised
// output, D / 32 dims per lane.
template <int D, int U>
__device__ __forceinline__ void gather_row(const Params& p, int c0, int c, int c1, int step, int i, int lane,
                                           float& M, float& L, float (&o)[D / 32]) {
    constexpr int DPL = D / 32;
    const int rows = p.hw * p.G;
    M = -INFINITY;
    L = 0.f;
#pragma unroll
    for (int j = 0; j < DPL; ++j) o[j] = 0.f;
    for (; c <= c1; c += U * step) {
        float m[U], l[U], x[U][DPL];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cc = c + u * step;
            const int64_t at = (2 * (int64_t)cc + (cc == c0 ? 1 : 0)) * rows + i;
            const bool in = cc <= c1;
            m[u] = in ? p.part_m[at] : -INFINITY;
            l[u] = in ? p.part_l[at] : 0.f;
            const float* src = p.part_acc + at * D + lane * DPL;
            if constexpr (DPL == 4) {
                const float4 v = in ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
                x[u][0] = v.x; x[u][1] = v.y; x[u][2] = v.z; x[u][3] = v.w;
            } else {
                const float2 v = in ? *reinterpret_cast<const float2*>(src) : make_float2(0.f, 0.f);
                x[u][0] = v.x; x[u][1] = v.y;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float m_new = fmaxf(M, m[u]);
            const float use = m_new == -INFINITY ? 0.f : m_new;
            const float wo = exp2f(M - use), wn = exp2f(m[u] - use);
            L = L * wo + l[u] * wn;
            M = m_new;
#pragma unroll
            for (int j = 0; j < DPL; ++j) o[j] = fmaf(wn, x[u][j], o[j] * wo);
        }
    }
}

constexpr int kMinUnits = 16;       // of a split call, else fewer KV heads per unit
// Longest context: token numbers go up to the end of a fold's 512 past it.
constexpr int kMaxContext = INT32_MAX - 1024;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int heads_per_cta(int Hkv) { return Hkv % 4 == 0 ? 4 : (Hkv % 2 == 0 ? 2 : 1); }

using KernelFn = void (*)(Params);

// Resident CTAs per SM of an attention kernel with smem bytes of shared memory,
// after allowing it `most` (0: as many), once per kernel, size and device; 0 if it
// cannot run.
int resident_of(KernelFn fn, int smem, int threads = kThreads, int most = 0) {
    static std::mutex mu;
    static struct { KernelFn fn; int dev, smem, n; } cache[256];
    static int used = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < used; ++i)
        if (cache[i].fn == fn && cache[i].dev == dev && cache[i].smem == smem) return cache[i].n;
    int n = 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most > smem ? most : smem) != cudaSuccess ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (used < 256) cache[used++] = {fn, dev, smem, n};
    return n;
}

}  // namespace
