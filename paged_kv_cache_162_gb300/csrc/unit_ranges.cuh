// What the decode attention kernels that take a sequence's tokens head by head
// share (bounded.cu: 16-bit caches, q4_decode.cu: 4-bit caches): how the tiles
// of all units are cut into ranges and handed out, and the kernel that joins
// the pieces of units that several ranges have.  The comment at the top of
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

// What a weight of 1 is in P.V.  In fp16 a weight below 2^-25 would be nothing and
// one below 2^-14 lose digits, and a long context's can all be: one token of
// logit 0 among 2^20 of -18 has 1.6 % of the weight lost.  In units of 2^-15 (the
// largest weight is 1: 32768 of 65504) the same happens below 2^-40.  bf16 has the
// range of fp32.
template <class E>
constexpr float kWeightUnits = 1.f;
template <>
constexpr float kWeightUnits<pkv::F16> = 32768.f;

// What makes a row of P.V the output: 1 / L, and the units of the weights.
template <class E>
__device__ __forceinline__ float output_scale(float L) { return inverse_of(L) * (1.f / kWeightUnits<E>); }

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

// Row `row` of head hl in the piece that range c has of a unit beginning in c0.
__device__ __forceinline__ int64_t piece_row(const Params& p, int c, int c0, int hl, int row) {
    return ((2 * (int64_t)c + (c == c0 ? 1 : 0)) * p.hw + hl) * p.G + row;
}

// (M, L) of two parts of a row as one.
__device__ __forceinline__ void merge_ml(float& M, float& L, float m, float l) {
    const float m_new = fmaxf(M, m);
    const float use = m_new == -INFINITY ? 0.f : m_new;
    L = L * exp2f(M - use) + l * exp2f(m - use);
    M = m_new;
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

// Writes row i of unit `unit`.
template <class E, int D>
__device__ __forceinline__ void write_row(const Params& p, int unit, int i, int lane, float L,
                                          const float (&o)[D / 32]) {
    const float inv = output_scale<E>(L);
    const int64_t oh = (int64_t)(unit / p.HB) * p.H + (int64_t)(unit % p.HB) * p.hw * p.G + i;
    uint16_t* dst = static_cast<uint16_t*>(p.out) + oh * D + lane * (D / 32);
#pragma unroll
    for (int j = 0; j < D / 32; j += 2)
        *reinterpret_cast<uint32_t*>(dst + j) = E::from_float2(o[j] * inv, o[j + 1] * inv);
}

// M and 1 / L of query head `lane` (< G) of a KV head, by one warp: h0 its first
// query head in row_m and row_l, `place` the ranges of its unit, hl the head in
// it.  All loads of a round go out together.
__device__ __forceinline__ void group_ml(const Params& p, int64_t h0, int2 place, int hl, int lane,
                                         float& M, float& inv) {
    const int pieces = place.y - place.x + 1;
    float L = 0.f;
    M = -INFINITY;
    if (pieces == 1) {
        if (lane < p.G) {
            M = p.row_m[h0 + lane];
            L = p.row_l[h0 + lane];
        }
    } else if (pieces <= 4) {  // four lanes per head, eight heads per round
        for (int r0 = 0; r0 < p.G; r0 += 8) {
            const int row = r0 + lane / 4, c = place.x + lane % 4;
            float m = -INFINITY, l = 0.f;
            if (row < p.G && c <= place.y) {
                const int64_t at = piece_row(p, c, place.x, hl, row);
                m = p.part_m[at];
                l = p.part_l[at];
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1)
                merge_ml(m, l, __shfl_xor_sync(kFull, m, o), __shfl_xor_sync(kFull, l, o));
            const float mr = __shfl_sync(kFull, m, 4 * (lane & 7)), lr = __shfl_sync(kFull, l, 4 * (lane & 7));
            if (lane / 8 == r0 / 8) {
                M = mr;
                L = lr;
            }
        }
    } else {  // the warp on four heads per round
        for (int r0 = 0; r0 < p.G; r0 += 4) {
            float m[4], l[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                m[r] = -INFINITY;
                l[r] = 0.f;
            }
            for (int c = place.x + lane; c <= place.y; c += 32) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r0 + r < p.G) {
                        const int64_t at = piece_row(p, c, place.x, hl, r0 + r);
                        merge_ml(m[r], l[r], p.part_m[at], p.part_l[at]);
                    }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    merge_ml(m[r], l[r], __shfl_xor_sync(kFull, m[r], o), __shfl_xor_sync(kFull, l[r], o));
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (lane == r0 + r) {
                    M = m[r];
                    L = l[r];
                }
        }
    }
    inv = inverse_of(L);
}

// Adds the weights of tokens j0 + 4 (32 u + lane) .. + 3, u < RUNS, of KV head
// kvh of sequence s to their scores, by one warp; `place`: the ranges its unit
// begins and ends in, hl: the head in it.  z of the first HEADS query heads and
// the old scores are on their way while M and L are found.
template <int RUNS, int HEADS>
__device__ __forceinline__ void fold_stretch(const Params& p, int s, int kvh, int hl, int n, int2 place,
                                             int j0, int lane) {
    const int64_t h0 = (int64_t)s * p.H + (int64_t)kvh * p.G;
    const float* z = p.z + h0 * p.z_stride;
    float* sc = p.scores + ((int64_t)s * p.Hkv + kvh) * p.score_stride;
    const bool vec = (reinterpret_cast<uintptr_t>(sc) & 15u) == 0;
    float4 zz[RUNS][HEADS];
    float old[RUNS][4];
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
        const int j = j0 + 4 * (32 * u + lane);
#pragma unroll
        for (int r = 0; r < HEADS; ++r)
            zz[u][r] = j < n && r < p.G ? *reinterpret_cast<const float4*>(z + r * p.z_stride + j)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
        if (vec && j + 4 <= n) {
            const float4 v = *reinterpret_cast<const float4*>(sc + j);
            old[u][0] = v.x; old[u][1] = v.y; old[u][2] = v.z; old[u][3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) old[u][e] = j + e < n ? sc[j + e] : 0.f;
        }
    }
    float M, inv;
    group_ml(p, h0, place, hl, lane, M, inv);
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
        const int j = j0 + 4 * (32 * u + lane);
        float w[4] = {0.f, 0.f, 0.f, 0.f};
        auto add = [&](const float4& v, int r) {
            const float m = __shfl_sync(kFull, M, r), i = __shfl_sync(kFull, inv, r);
            if (i != 0.f) {
                w[0] = fmaf(exp2f(v.x - m), i, w[0]);
                w[1] = fmaf(exp2f(v.y - m), i, w[1]);
                w[2] = fmaf(exp2f(v.z - m), i, w[2]);
                w[3] = fmaf(exp2f(v.w - m), i, w[3]);
            }
        };
#pragma unroll
        for (int r = 0; r < HEADS; ++r)
            if (r < p.G) add(zz[u][r], r);
        if constexpr (HEADS > 1) {
#pragma unroll 4
            for (int r = HEADS; r < p.G; ++r)
                add(j < n ? *reinterpret_cast<const float4*>(z + r * p.z_stride + j) : make_float4(0.f, 0.f, 0.f, 0.f), r);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) old[u][e] += w[e];
        if (vec && j + 4 <= n) {
            *reinterpret_cast<float4*>(sc + j) = make_float4(old[u][0], old[u][1], old[u][2], old[u][3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < n) sc[j + e] = old[u][e];
        }
    }
}

// After split_kernel, one wave of CTAs that take items: first the joins, then,
// with scores, the fold.  Either is a short chain of loads (is there anything ->
// where -> the data), and most possible items do not exist: so the threads of a
// CTA look at 256 of its share at once, list those that do, and its warps do
// the listed ones in turn: 155 us for the 256 requests of 16..4096, where warps
// with items of their own took 160.  Fewer tokens per fold, two or four CTAs per
// SM: no faster (at three the score forms spill 4 to 28 bytes, at two nothing).
//  join: a row of a unit that lies in several ranges, by a warp, or by the
//        CTA's warps together (`wide`) where units have many pieces.
//  fold: 256 tokens (512 with one query head) of a KV head, by a warp.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
struct Item {
    int2 place;  // the ranges its unit begins and ends in
    int at;      // join: output row; fold: sequence * Hkv + KV head
    int n, j0;   // fold: context (join: 0), first token
};

template <class E, int D, bool kScores, bool kOne>
__global__ void __launch_bounds__(kJoinThreads, 3) join_kernel(const __grid_constant__ Params p, int wide) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int DPL = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.hw * p.G;
    const int joins = p.S * p.HB * rows;  // = S * H
    if (wide) {
        __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
        __shared__ __align__(16) float s_o[kJoinWarps][D];
        for (int i = blockIdx.x; i < joins; i += gridDim.x) {
            const int2 at = p.place[i / rows];
            if (pkv::pieces_of(at.x, at.y, p.ranges) < 2) continue;  // the same for the whole CTA
            float M, L, o[DPL];
            gather_row<D, 6>(p, at.x, at.x + warp, at.y, kJoinWarps, i % rows, lane, M, L, o);
            if (lane == 0) {
                s_m[warp] = M;
                s_l[warp] = L;
            }
#pragma unroll
            for (int j = 0; j < DPL; ++j) s_o[warp][lane * DPL + j] = o[j];
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int w = 1; w < kJoinWarps; ++w) {
                    const float m_new = fmaxf(M, s_m[w]);
                    const float use = m_new == -INFINITY ? 0.f : m_new;
                    const float wo = exp2f(M - use), wn = exp2f(s_m[w] - use);
                    L = L * wo + s_l[w] * wn;
                    M = m_new;
#pragma unroll
                    for (int j = 0; j < DPL; ++j) o[j] = fmaf(wn, s_o[w][lane * DPL + j], o[j] * wo);
                }
                write_row<E, D>(p, i / rows, i % rows, lane, L, o);
            }
            __syncthreads();  // the parts have been read
        }
    }
    constexpr int RUNS = kOne ? 4 : 2, HEADS = kOne ? 1 : 4, TOKENS = RUNS * 128;
    __shared__ int s_count[kJoinWarps];
    __shared__ Item s_item[kJoinThreads];
    const int heads = p.S * p.Hkv;
    const long long listed = wide ? 0 : joins;
    const long long items = listed + (kScores ? (long long)heads * ((p.max_ctx + TOKENS - 1) / TOKENS) : 0);
    // neighbouring items go to different SMs
    for (long long base = blockIdx.x; base < items; base += (long long)kJoinThreads * gridDim.x) {
        const long long mine = base + (long long)threadIdx.x * gridDim.x;
        Item it;
        it.n = 0;  // of a join
        bool live = false;
        if (mine < listed) {
            it.at = (int)mine;
            it.place = p.place[it.at / rows];
            live = pkv::pieces_of(it.place.x, it.place.y, p.ranges) > 1;
        } else if (kScores && mine < items) {
            // (stretch, sequence, KV head): the first stretches of all first
            const long long f = mine - listed;
            it.at = (int)(f % heads);
            it.j0 = (int)(f / heads) * TOKENS;
            it.n = context_of(p, it.at / p.Hkv);
            it.place = p.place[it.at / p.hw];
            live = it.j0 < it.n && pkv::pieces_of(it.place.x, it.place.y, p.ranges) > 0;
        }
        const unsigned alive = __ballot_sync(kFull, live);
        if (lane == 0) s_count[warp] = __popc(alive);
        __syncthreads();
        int before = 0, count = 0;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            if (w == warp) before = count;
            count += s_count[w];
        }
        if (live) s_item[before + __popc(alive & ((1u << lane) - 1u))] = it;
        __syncthreads();
        for (int k = warp; k < count; k += kJoinWarps) {
            const Item x = s_item[k];
            if (x.n == 0) {
                float M, L, o[DPL];
                gather_row<D, 2>(p, x.place.x, x.place.x, x.place.y, 1, x.at % rows, lane, M, L, o);
                write_row<E, D>(p, x.at / rows, x.at % rows, lane, L, o);
            } else if constexpr (kScores) {
                const int kvh = x.at % p.Hkv;
                fold_stretch<RUNS, HEADS>(p, x.at / p.Hkv, kvh, kvh % p.hw, x.n, x.place, x.j0, lane);
            }
        }
        __syncthreads();  // the list has been read
    }
}

constexpr int kJoinCtasPerSm = 3;   // of the join kernel
constexpr int kMinUnits = 16;       // of a split call, else fewer KV heads per unit
// Longest context: token numbers go up to the end of a fold's 512 past it.
constexpr int kMaxContext = INT32_MAX - 1024;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int heads_per_cta(int Hkv) { return Hkv % 4 == 0 ? 4 : (Hkv % 2 == 0 ? 2 : 1); }

using KernelFn = void (*)(Params);
using JoinFn = void (*)(Params, int);

// Resident CTAs per SM of an attention kernel, after allowing it its shared
// memory (once per kernel and device); 0 if it cannot run.
int resident_of(KernelFn fn, int smem) {
    static std::mutex mu;
    static struct { KernelFn fn; int dev; int n; } cache[128];
    static int used = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < used; ++i)
        if (cache[i].fn == fn && cache[i].dev == dev) return cache[i].n;
    int n = 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, kThreads, smem) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (used < 128) cache[used++] = {fn, dev, n};
    return n;
}

}  // namespace
