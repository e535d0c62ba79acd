// Decode attention for bounded caches: a sliding window with sinks, and
// attention that adds every token's weight to a running score.
//
// What it computes, for sequence s, query head h, KV head g = h / G, context
// n, with z_j = scale q_h . K_j over the tokens j the query sees:
//   out = sum_j 2^(z'_j - M) V_j / sum_j 2^(z'_j - M),  z' = z log2(e), M = max z'
// window:      j < sinks or j >= n - window.  The nv = min(n, sinks + window)
//   visible tokens are numbered v = 0 .. nv-1, token j = v below the sinks and
//   v + (n - nv) above, so the gap is skipped by one addition per row and no
//   block inside it is looked up.
// accumulate:  every j < n; then scores[s, g, j] += sum_{h in g} p_hj with
//   p_hj = 2^(z'_hj - M_h) / L_h.  p needs the whole row's M and L, so the z'
//   are written to scratch as they are computed and read back once.
//
// How: a unit is one sequence and `hw` neighbouring KV heads; its visible
// tokens go in tiles of 16 (D = 64: 32).  One warp takes one KV head of a tile:
// K and V rows come through a cp.async ring in shared memory (16-byte chunks,
// XOR swizzle by row, rows without a token zero-filled and not read), the
// group's G <= 16 query heads are the rows of m16n8k16 products on the tensor
// cores.
// Memory is the bound: 512 bytes of K and V per (token, KV head) at D = 128
// against 32 + 16 products of 16x8x16 per 8 KB tile.
//   S = Q K^T, then the online softmax on the accumulators, then O += P V with
//   P as the sum of two 16-bit numbers (its rounding and the rest): P rounded
//   once would add an error as large as the output's own rounding.  In fp16 P is in
//   units of 2^-15 (kWeightUnits).
// A CTA is four warps: hw heads times 4 / hw token splits, joined in shared
// memory.  The four read neighbouring data (4 D values of each token row, or four
// tiles of one head); a range of its own per warp was slower (window of 64 MHA
// requests 146 us against 132), a barrier to keep them together no faster.
//
// Two ways to spread the units:
//  * direct: one CTA, or one cluster of CTAs that share the unit's tokens, per
//    unit; the cluster joins its parts through distributed shared memory.  One
//    launch, no workspace traffic but z'.  For few or short units.
//  * split: the tiles of all units, in order, are cut into ranges: one large
//    range per resident CTA, then small ones that whichever CTA is done first
//    takes (cluster launch control: a running CTA cancels the launch of a
//    waiting one and does its work, keeping its plan and its full ring).  A
//    unit inside one range is finished there; a unit cut by range ends leaves
//    (M, L, unnormalised out) per piece, and a second kernel joins the pieces
//    and folds all weights into the scores.  Ranges are computed from the
//    lengths on the device by every CTA: a call needs no plan kernel, no counter
//    and no ticket, and as the cuts do not depend on who does which range,
//    every sum has a fixed order.
//
// Measured on GB300 (device time, share of the measured copy rate of 6776 GB/s):
//   window 1000 + 4 sinks, 64 requests of 128..2048, 32 heads, fp16   129 us  97 %
//   window 4093 + 7, 96 requests, 32 heads on 8, bf16                 240 us  99 %
//   accumulate, the 64 requests whole                                 186 us  92 %
//   accumulate, 8 x 32768                                             663 us  97 %
//   accumulate, 256 requests of 16..4096 (median 512), 32 heads on 8  156 us  81 %
//   window 4096 of one 32768-token context, 32 heads on 8            8.3 us  30 %
//   4 requests of at most 100 tokens, 4 heads of 64       3.0 us, with scores 3.4
// The split kernel moves each byte once (847.5 MB for 843.4) at 83 % of the DRAM
// peak with its tensor pipe 26 % busy.  About 4 us go before every ring is full
// (length -> place -> table -> rows), 3 to the last ranges; the second kernel takes
// 4 us without scores and 10 to 15 with them.  The small calls are that chain.
#include <cooperative_groups.h>

#include <climits>
#include <cmath>
#include <cstdio>
#include <mutex>

#include "bounded_place.h"
#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_mma.cuh"
#include "tc_wait.cuh"

namespace cg = cooperative_groups;

namespace {

using pkv::cp_async16_zfill;
using pkv::cp_async_commit;
using pkv::cp_async_wait;
using pkv::ldsm_x4;
using pkv::ldsm_x4_trans;
using pkv::Mma;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxRanges = 1536;   // CTAs of a split call
// Tiles of a large range at least: a range of 8 is a chain of unit ends (100
// requests of 1..64 tokens: 19.9 us with 8, 10.9 with 2; one head of a
// 30000-token window: 16.5 and 14.0).
constexpr int kMinRange = 2;
constexpr int kMinSmall = 4;       // and of a small one: a ring is at most two ranges ahead
constexpr int kMaxGroup = 16;      // query heads per KV head
constexpr int kMaxCluster = 16;    // CTAs that share a unit in a direct call
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// Tokens of a tile: 4 KB of K (or V) either way.  At D = 64 a tile of 16 had as
// many instructions in its softmax and loop as in its products: 64 requests of
// 2000 tokens and 16 heads took 90.8 us, with 32 tokens 84.8 (at D = 128 the
// registers are all taken at 16).
constexpr int tile_tokens(int D) { return D == 128 ? 16 : 32; }
template <int D>
constexpr int kTile = tile_tokens(D);
constexpr int kStages = 3;
template <int D>
constexpr int kTileBytes = kTile<D> * D * 2;  // K (or V) of one tile and head
template <int D>
constexpr int kRingBytes = kStages * 2 * kTileBytes<D>;  // one warp's ring
template <int D>
constexpr int kSmemBytes = kWarps * kRingBytes<D>;

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

// Running softmax of one warp over its tiles: rows lane/4 and lane/4 + 8 of
// the accumulators, (m, l) per row.
template <int D>
struct Acc {
    float o[D / 8][4];
    float m[2], l[2];
};

// One warp's tiles on their way through its ring: tile i of one unit after the
// other, `step` apart, each looked up one tile ahead of its copies and copied
// kStages - 1 tiles ahead of its use.  With a plan and step 1 it goes on into
// the units and ranges that follow, so that no end of one drains the ring.
template <int D>
struct Feed {
    static constexpr int NST = kStages;
    static constexpr unsigned kAllRows = kTile<D> == 32 ? 0xffffffffu : 0xffffu;
    const Params& p;
    Plan* const plan;         // null: one unit (part) at a time
    const uint32_t ring;
    const int warp, lane, hl; // hl: head of the CTA's hw that this warp takes
    const int step;
    int s, hb, n_next, i, te, left;  // the next tile to copy, and its unit; left: from its tile 0 to the range's end
    int nv, shift;
    const int32_t* bt;
    const uint16_t* k_head;
    int slot;                 // cache row of its row lane % kTile
    bool more;
    unsigned mask[NST];       // rows with a token, of the tiles in the ring
    int stage;                // of the oldest tile
    int asked, answers, pushed;  // requests made (warp 0), answers read, ranges queued

    __device__ __forceinline__ Feed(const Params& p_, Plan* plan_, uint32_t ring_, int warp_, int lane_,
                                    int hl_, int step_)
        : p(p_), plan(plan_), ring(ring_), warp(warp_), lane(lane_), hl(hl_), step(step_), asked(0),
          answers(0), pushed(0) {}

    __device__ __forceinline__ void enter(int n) {  // unit (s, hb)
        nv = visible_of(p, n);
        shift = n - nv;
        bt = p.block_tables + (int64_t)s * p.MB;
        const int kvh = hb * p.hw + hl;
        k_head = static_cast<const uint16_t*>(p.k_cache) + (int64_t)kvh * D;
        // the unit's queries are read when its first tile is used
        const char* q = static_cast<const char*>(p.q) +
                        ((int64_t)s * p.H + (int64_t)kvh * p.G) * D * 2;
        if (lane * 128 < p.G * D * 2) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + lane * 128));
    }

    // Row lane % kTile of the next tile: its cache row, or -1 where there is no
    // token (past the visible ones) or its block id is out of range.  NB * bs
    // fits an int (checked on the host).
    __device__ __forceinline__ void lookup() {
        slot = -1;
        const int v = i * kTile<D> + lane % kTile<D>;
        if (!more || v >= nv) return;
        const int tok = v < p.sinks ? v : v + shift;
        const int phys = __ldg(bt + (tok >> p.bs_log2));
        if ((unsigned)phys >= (unsigned)p.NB) {
            pkv::report(p.err, PKV_DEVERR_BLOCK_ID);
            return;
        }
        slot = (phys << p.bs_log2) | (tok & ((1 << p.bs_log2) - 1));
    }

    // Fills the ring from tile `first` of unit (s_, hb_) on, tiles below te_;
    // left_: tiles from the unit's first one to the range's end.
    __device__ __forceinline__ void begin(int s_, int hb_, int n, int first, int te_, int left_) {
        s = s_;
        hb = hb_;
        i = first;
        te = te_;
        left = left_;
        n_next = chained() && s + 1 < p.S ? context_of(p, s + 1) : 0;
        more = i < te;
        enter(n);
        lookup();
        stage = 0;
#pragma unroll
        for (int st = 0; st < NST - 1; ++st) push(st, st);
    }

    __device__ __forceinline__ bool chained() const { return plan != nullptr && step == 1; }

    // Warp 0 asks for the next range when few tiles are left of this one (not
    // earlier: a range asked for is a range no other CTA can take).
    __device__ __forceinline__ void maybe_ask(int tiles_left) {
        if (warp == 0 && tiles_left <= 3 && asked == answers) {
            if (lane == 0) ask_range(plan, asked);
            ++asked;
        }
    }
    // The next range into the queue (whole warp).
    __device__ __forceinline__ bool next() {
        maybe_ask(0);
        int k = answers;
        const bool got = next_range(p, plan, warp, lane, k, pushed);
        asked = answers = k;
        if (got) ++pushed;
        return got;
    }

    // Copies the next tile into ring stage `st` and its row mask into
    // mask[at], then looks up the one after it.
    __device__ __forceinline__ void push(int st, int at) {
        constexpr int ROWB = D * 2, CPR = ROWB / 16, CPL = kTile<D> * CPR / 32;
        mask[at] = __ballot_sync(kFull, slot >= 0) & kAllRows;
        if (more) {
            const uint32_t sk = ring + st * 2 * kTileBytes<D>, sv = sk + kTileBytes<D>;
            const int64_t row_elems = (int64_t)p.Hkv * D;
            // a split call streams more than it could find again in L2; z and the
            // pieces stay there
            const uint64_t keep_out = plan ? pkv::policy_evict_first() : pkv::policy_evict_normal();
            const int64_t to_v = static_cast<const uint16_t*>(p.v_cache) - static_cast<const uint16_t*>(p.k_cache);
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const int chunk = lane + 32 * j;
                const int row = chunk / CPR, c = chunk % CPR;
                const int sl = __shfl_sync(kFull, slot, row);
                const uint16_t* src = k_head + (int64_t)(sl < 0 ? 0 : sl) * row_elems + c * 8;
                const uint32_t dst = row * ROWB + ((c ^ (row & 7)) * 16);
                const int bytes = sl < 0 ? 0 : 16;
                cp_async16_zfill(sk + dst, src, bytes, keep_out);
                cp_async16_zfill(sv + dst, src + to_v, bytes, keep_out);
            }
            i += step;
            if (i >= te) advance();
            if (more && chained()) maybe_ask(left - i);
            lookup();
        }
        cp_async_commit();  // empty past the end: the counting stays simple
    }

    __device__ __forceinline__ void advance() {
        more = false;
        if (!chained()) return;
        left -= te;
        int n;
        if (left > 0) {  // the range's next unit
            i = 0;
            if (++hb == p.HB) {
                hb = 0;
                ++s;
                n = n_next;
                n_next = s + 1 < p.S ? context_of(p, s + 1) : 0;
            } else {
                n = context_of(p, s);
            }
        } else {         // another range
            const int at = pushed;
            if (!next()) return;
            const Range& r = plan->queue[warp][at & 3];
            s = r.s;
            hb = r.hb;
            i = r.tb;
            left = r.left + r.tb;
            n = r.n;
            n_next = s + 1 < p.S ? context_of(p, s + 1) : 0;
        }
        more = true;
        enter(n);
        te = min(tiles_of(p, n), left);
    }
};

// One warp: KV head kvh of sequence s, its tiles first, first + step, ... below
// te out of the feed.  kWide: more than 8 query heads per KV head.
template <class E, int D, bool kWide, bool kScores>
__device__ __forceinline__ void attend(const Params& p, Feed<D>& feed, int s, int kvh, int first,
                                       int te, int lane, Acc<D>& a) {
    constexpr int NK = D / 16, NO = D / 8;
    constexpr int ROWB = D * 2;
    constexpr int NST = kStages;
    constexpr int R = kWide ? 2 : 1;
    constexpr int NT = kTile<D> / 8;
    const int g = lane >> 2, t = lane & 3;

#pragma unroll
    for (int j = 0; j < NO; ++j) a.o[j][0] = a.o[j][1] = a.o[j][2] = a.o[j][3] = 0.f;
    a.m[0] = a.m[1] = -INFINITY;
    a.l[0] = a.l[1] = 0.f;
    if (first >= te) return;

    // query fragments: rows g and g + 8 are heads kvh * G + row
    uint32_t qa[NK][4];
    {
        const uint16_t* q0 = static_cast<const uint16_t*>(p.q) +
                             ((int64_t)s * p.H + (int64_t)kvh * p.G + g) * D + 2 * t;
        const bool r0 = g < p.G, r1 = kWide && g + 8 < p.G;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            qa[k][0] = r0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + 16 * k)) : 0u;
            qa[k][1] = r1 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + 8 * D + 16 * k)) : 0u;
            qa[k][2] = r0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + 16 * k + 8)) : 0u;
            qa[k][3] = r1 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + 8 * D + 16 * k + 8)) : 0u;
        }
    }

    for (int i = first; i < te; i += feed.step) {
        const int stage = feed.stage;
        feed.push(stage == 0 ? NST - 1 : stage - 1, NST - 1);
        const unsigned rows = feed.mask[0];
        cp_async_wait<NST - 1>();
        __syncwarp();
        const uint32_t sk = feed.ring + stage * 2 * kTileBytes<D>, sv = sk + kTileBytes<D>;

        // S: NT column tiles of 8 tokens
        float sc[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            const int mi = lane >> 3;
            const int row = 8 * j + (mi >> 1) * 8 + (lane & 7);
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                uint32_t b[4];
                ldsm_x4(b, sk + row * ROWB + (((2 * k + (mi & 1)) ^ (row & 7)) * 16));
                Mma<E>::run(sc[j], qa[k], b[0], b[1]);
                Mma<E>::run(sc[j + 1], qa[k], b[2], b[3]);
            }
        }
        // logits in log2 units; element e of sc[j] is row g + 8 (e / 2),
        // token 8 j + 2 t + e % 2 of the tile
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2 * R; ++e) sc[j][e] *= p.qscale;
        if (rows != Feed<D>::kAllRows) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2 * R; ++e)
                    if (!((rows >> (8 * j + 2 * t + (e & 1))) & 1u)) sc[j][e] = -INFINITY;
        }
        if constexpr (kScores) {
            float* zr = p.z + ((int64_t)s * p.H + (int64_t)kvh * p.G + g) * p.z_stride +
                        i * kTile<D> + 2 * t;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (g + 8 * r < p.G) {
                    float* zp = zr + 8 * r * p.z_stride;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        *reinterpret_cast<float2*>(zp + 8 * j) = make_float2(sc[j][2 * r], sc[j][2 * r + 1]);
                }
        }
        float corr[2] = {1.f, 1.f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float mt = fmaxf(sc[0][2 * r], sc[0][2 * r + 1]);
#pragma unroll
            for (int j = 1; j < NT; ++j) mt = fmaxf(mt, fmaxf(sc[j][2 * r], sc[j][2 * r + 1]));
            mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 1));
            mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 2));
            const float m_new = fmaxf(a.m[r], mt);
            const float m_use = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet
            corr[r] = exp2f(a.m[r] - m_use);
            a.m[r] = m_new;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int e = 0; e < 2; ++e) sc[j][2 * r + e] = exp2f(sc[j][2 * r + e] - m_use);
                sum += sc[j][2 * r] + sc[j][2 * r + 1];
            }
            a.l[r] = fmaf(a.l[r], corr[r], sum);
        }
        // most tiles leave every row's maximum as it was
        if (__any_sync(kFull, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                a.o[j][0] *= corr[0];
                a.o[j][1] *= corr[0];
                if (kWide) {
                    a.o[j][2] *= corr[1];
                    a.o[j][3] *= corr[1];
                }
            }
        }
#pragma unroll
        for (int h = 0; h < NT / 2; ++h) {  // 16 tokens each
            // P = its rounding to 16 bits + the rounding of what is left
            uint32_t ph[4] = {0u, 0u, 0u, 0u}, pl[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float x = sc[2 * h + j][2 * r] * kWeightUnits<E>, y = sc[2 * h + j][2 * r + 1] * kWeightUnits<E>;
                    const uint32_t hi = E::from_float2(x, y);
                    const float2 back = E::to_float2(hi);
                    ph[2 * j + r] = hi;
                    pl[2 * j + r] = E::from_float2(x - back.x, y - back.y);
                }
            const int mi = lane >> 3;
            const int row = 16 * h + (mi & 1) * 8 + (lane & 7);
#pragma unroll
            for (int j = 0; j < NO; j += 2) {
                uint32_t b[4];
                ldsm_x4_trans(b, sv + row * ROWB + (((j + (mi >> 1)) ^ (row & 7)) * 16));
                Mma<E>::run(a.o[j], ph, b[0], b[1]);
                Mma<E>::run(a.o[j + 1], ph, b[2], b[3]);
                Mma<E>::run(a.o[j], pl, b[0], b[1]);
                Mma<E>::run(a.o[j + 1], pl, b[2], b[3]);
            }
        }
        __syncwarp();  // this stage is filled again by the next push
#pragma unroll
        for (int st = 0; st < NST - 1; ++st) feed.mask[st] = feed.mask[st + 1];
        feed.stage = stage + 1 == NST ? 0 : stage + 1;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        a.l[r] += __shfl_xor_sync(kFull, a.l[r], 1);
        a.l[r] += __shfl_xor_sync(kFull, a.l[r], 2);
    }
}

// Joins the token splits of each head in shared memory: split 0's warp ends
// up with the whole.  Every warp's part goes into its own ring, idle here.
template <int D, bool kWide>
__device__ __forceinline__ void join_splits(const Params& p, float* ring, int warp, int lane,
                                            Acc<D>& a) {
    constexpr int NO = D / 8, R = kWide ? 2 : 1;
    constexpr int kSlice = kRingBytes<D> / 4;  // floats of one warp's ring
    __syncwarp();
    if (warp >= p.hw) {
        float* mine = ring + warp * kSlice + lane;
#pragma unroll
        for (int j = 0; j < NO; ++j)
#pragma unroll
            for (int e = 0; e < 2 * R; ++e) mine[(4 * j + e) * 32] = a.o[j][e];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mine[(4 * NO + r) * 32] = a.m[r];
            mine[(4 * NO + 2 + r) * 32] = a.l[r];
        }
    }
    __syncthreads();
    if (warp < p.hw) {
        for (int w = warp + p.hw; w < kWarps; w += p.hw) {
            const float* other = ring + w * kSlice + lane;
            float wa[2], wb[2];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float mo = other[(4 * NO + r) * 32], lo = other[(4 * NO + 2 + r) * 32];
                const float m_new = fmaxf(a.m[r], mo);
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                wa[r] = exp2f(a.m[r] - m_use);
                wb[r] = exp2f(mo - m_use);
                a.m[r] = m_new;
                a.l[r] = a.l[r] * wa[r] + lo * wb[r];
            }
#pragma unroll
            for (int j = 0; j < NO; ++j)
#pragma unroll
                for (int e = 0; e < 2 * R; ++e)
                    a.o[j][e] = a.o[j][e] * wa[e >> 1] + other[(4 * j + e) * 32] * wb[e >> 1];
        }
    }
    __syncthreads();  // the rings are filled again after this
}

// The same for a CTA with one head (direct): warp w ends up with columns
// [w, w + 1) * D / 4 of the rows, in o[.][2 r + column % 2], and with the whole m
// and l.
template <int D, bool kWide>
__device__ __forceinline__ void join_warps(float* ring, int warp, int lane, Acc<D>& a,
                                           float (&o)[D / 8 / kWarps][kWide ? 4 : 2]) {
    constexpr int NO = D / 8, R = kWide ? 2 : 1;
    constexpr int kSlice = kRingBytes<D> / 8;  // float2s of one warp's ring
    float2* all = reinterpret_cast<float2*>(ring) + lane;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int j = 0; j < NO; ++j)
            all[warp * kSlice + (R * j + r) * 32] = make_float2(a.o[j][2 * r], a.o[j][2 * r + 1]);
        all[warp * kSlice + (R * NO + r) * 32] = make_float2(a.m[r], a.l[r]);
    }
    __syncthreads();
    float2 ml[R][kWarps];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) ml[r][w] = all[w * kSlice + (R * NO + r) * 32];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float M = ml[r][0].x, L = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, ml[r][w].x);
        const float use = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            ml[r][w].x = exp2f(ml[r][w].x - use);  // the part's weight
            L = fmaf(ml[r][w].x, ml[r][w].y, L);
        }
        a.m[r] = M;
        a.l[r] = L;
    }
#pragma unroll
    for (int j = 0; j < NO / kWarps; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            o[j][2 * r] = o[j][2 * r + 1] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 x = all[w * kSlice + (R * (warp * (NO / kWarps) + j) + r) * 32];
                o[j][2 * r] = fmaf(ml[r][w].x, x.x, o[j][2 * r]);
                o[j][2 * r + 1] = fmaf(ml[r][w].x, x.y, o[j][2 * r + 1]);
            }
        }
}

// scores[s, kvh, j] += sum over the group's heads of 2^(z - M) / L for the
// tokens j0 <= j < j1 (j0 a multiple of 16) by `threads` threads.  s_m and s_inv
// hold M and 1 / L (0 for an empty row) of the G heads.  Four tokens per thread
// and round; P = 1, 2 or 4 neighbouring threads share them, four heads each, so
// that all loads of a round go out together (150 tokens, 16 heads, the call: 7.0
// us, a thread for all heads 8.5).  Every sum has a fixed order.
__device__ __forceinline__ void fold_weights(const Params& p, int s, int kvh, int j0, int j1,
                                             const float* s_m, const float* s_inv, int tid,
                                             int threads) {
    const float* z = p.z + ((int64_t)s * p.H + (int64_t)kvh * p.G) * p.z_stride;
    float* sc = p.scores + ((int64_t)s * p.Hkv + kvh) * p.score_stride;
    const bool vec = (reinterpret_cast<uintptr_t>(sc) & 15u) == 0;
    const int shift = p.G > 8 ? 2 : p.G > 4 ? 1 : 0, P = 1 << shift, part = tid & (P - 1);
    for (int base = j0; base < j1; base += 4 * (threads >> shift)) {
        const int j = base + 4 * (tid >> shift);
        const bool full = vec && j + 4 <= j1;
        float old[4];
        if (part == 0) {
            if (full) {
                const float4 x = *reinterpret_cast<const float4*>(sc + j);
                old[0] = x.x; old[1] = x.y; old[2] = x.z; old[3] = x.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) old[e] = j + e < j1 ? sc[j + e] : 0.f;
            }
        }
        float4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q * P >= p.G) break;
            const int r = part + q * P;
            v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < j1 && r < p.G) v[q] = *reinterpret_cast<const float4*>(z + r * p.z_stride + j);
        }
        float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q * P >= p.G) break;
            const int r = part + q * P;
            const float m = s_m[r], inv = r < p.G ? s_inv[r] : 0.f;
            if (inv != 0.f) {
                w[0] = fmaf(exp2f(v[q].x - m), inv, w[0]);
                w[1] = fmaf(exp2f(v[q].y - m), inv, w[1]);
                w[2] = fmaf(exp2f(v[q].z - m), inv, w[2]);
                w[3] = fmaf(exp2f(v[q].w - m), inv, w[3]);
            }
        }
        for (int x = 1; x < P; x <<= 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] += __shfl_xor_sync(kFull, w[e], x);
        if (part != 0) continue;
        if (full) {
            *reinterpret_cast<float4*>(sc + j) =
                make_float4(old[0] + w[0], old[1] + w[1], old[2] + w[2], old[3] + w[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < j1) sc[j + e] = old[e] + w[e];
        }
    }
}

// What the CTAs of a cluster send one another: 32 dims of a row ("segment") of
// every CTA to the CTA that joins it, and every row's M and L to all.
struct ClusterIn {
    float o[kMaxGroup * 4 * 32];                 // [segment / CS][CTA][32]
    float m[kMaxCluster][kMaxGroup], l[kMaxCluster][kMaxGroup];
};

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Joins the CTAs of a cluster that share a unit: every CTA writes its rows
// into the memory of the CTAs that join them, segment i to CTA
// i % CS; after one barrier each joins what it was sent, and folds its own
// tokens [tb, te) into the scores.  No CTA reads another's memory, so none has
// to stay for that.  o, m and l are as join_warps leaves them.  The caller has arrived once at the cluster's barrier: the
// wait for it says that all CTAs run.
template <class E, int D, bool kWide, bool kScores>
__device__ __forceinline__ void join_cluster(const Params& p, int s, int kvh, int n, int tb, int te,
                                             ClusterIn* in, int warp, int lane, const Acc<D>& a,
                                             const float (&mine)[D / 8 / kWarps][kWide ? 4 : 2],
                                             float* s_m, float* s_inv) {
    constexpr int NO = D / 8, R = kWide ? 2 : 1, SEGS = D / 32;
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int g = lane >> 2, t = lane & 3, tid = warp * 32 + lane;
    cluster_wait();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = g + 8 * r;
        if (row < p.G) {
#pragma unroll
            for (int i = 0; i < NO / kWarps; ++i) {
                const int j = warp * (NO / kWarps) + i, seg = row * SEGS + j / 4;
                float* to = cluster.map_shared_rank(&in->o[0], seg % CS) + (seg / CS * CS + rank) * 32 +
                            8 * (j % 4) + 2 * t;
                *reinterpret_cast<float2*>(to) = make_float2(mine[i][2 * r], mine[i][2 * r + 1]);
            }
            const int c = 4 * warp + t;  // kMaxCluster of them
            if (c < CS) {
                cluster.map_shared_rank(&in->m[rank][0], c)[row] = a.m[r];
                cluster.map_shared_rank(&in->l[rank][0], c)[row] = a.l[r];
            }
        }
    }
    cluster_arrive();
    cluster_wait();
    // M and 1 / L of a row, and the CTAs' weights 2^(m_i - M): with scores, which
    // need all rows' in every CTA, by a thread per row and before the rest (over
    // m); without, by the lanes of the warp that joins a segment (a 4096-token
    // window: 8.2 us, 8.5 the other way)
    if constexpr (kScores) {
        if (tid < p.G) {
            float m[kMaxCluster], l[kMaxCluster], M = -INFINITY, L = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxCluster; ++i) {
                m[i] = i < CS ? in->m[i][tid] : -INFINITY;
                l[i] = i < CS ? in->l[i][tid] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kMaxCluster; ++i) M = fmaxf(M, m[i]);
            const float use = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int i = 0; i < kMaxCluster; ++i) {
                m[i] = exp2f(m[i] - use);
                L = fmaf(m[i], l[i], L);
                if (i < CS) in->m[i][tid] = m[i];
            }
            s_m[tid] = M;
            s_inv[tid] = inverse_of(L);
        }
        __syncthreads();
    }
    for (int k = warp; k * CS + rank < p.G * SEGS; k += kWarps) {
        const int seg = k * CS + rank, row = seg / SEGS;
        float w, inv, o = 0.f;  // w: of CTA `lane`
        if constexpr (kScores) {
            w = lane < CS ? in->m[lane][row] : 0.f;
            inv = s_inv[row];
        } else {
            const float m = lane < CS ? in->m[lane][row] : -INFINITY;
            float M = m;
#pragma unroll
            for (int x = kMaxCluster / 2; x >= 1; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, x));
            M = __shfl_sync(kFull, M, 0);
            w = lane < CS ? exp2f(m - (M == -INFINITY ? 0.f : M)) : 0.f;
            float L = lane < CS ? w * in->l[lane][row] : 0.f;
#pragma unroll
            for (int x = kMaxCluster / 2; x >= 1; x >>= 1) L += __shfl_xor_sync(kFull, L, x);
            inv = inverse_of(__shfl_sync(kFull, L, 0));
        }
        inv *= 1.f / kWeightUnits<E>;
        for (int i = 0; i < CS; ++i) o = fmaf(__shfl_sync(kFull, w, i), in->o[(k * CS + i) * 32 + lane], o);
        o *= inv;
        const float next = __shfl_down_sync(kFull, o, 1);
        uint16_t* dst = static_cast<uint16_t*>(p.out) +
                        ((int64_t)s * p.H + (int64_t)kvh * p.G + row) * D + seg % SEGS * 32 + lane;
        if ((lane & 1) == 0) *reinterpret_cast<uint32_t*>(dst) = E::from_float2(o, next);
    }
    if constexpr (kScores)
        fold_weights(p, s, kvh, tb * kTile<D>, min(te * kTile<D>, n), s_m, s_inv, tid, kThreads);
}

// Writes the finished rows of a unit (the warp's part of the accumulators).
template <class E, int D, bool kWide>
__device__ __forceinline__ void write_rows(const Params& p, int s, int kvh, int lane, const Acc<D>& a) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < (kWide ? 2 : 1); ++r) {
        const int row = g + 8 * r;
        if (row < p.G) {
            const float inv = output_scale<E>(a.l[r]);
            uint16_t* dst = static_cast<uint16_t*>(p.out) +
                            ((int64_t)s * p.H + (int64_t)kvh * p.G + row) * D + 2 * t;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
                *reinterpret_cast<uint32_t*>(dst + 8 * j) =
                    E::from_float2(a.o[j][2 * r] * inv, a.o[j][2 * r + 1] * inv);
        }
    }
}

// Direct: cluster c / cs takes unit c / cs (hw = 1), its CTAs equal parts of
// the unit's tiles, their warps every fourth tile.
template <class E, int D, bool kWide, bool kScores>
__global__ void __launch_bounds__(kThreads, 2) direct_kernel(const __grid_constant__ Params p) {
    // inputs may come from the kernel before this one; the next may become
    // resident once every CTA is here, and waits for this grid's end
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_m[kMaxGroup], s_inv[kMaxGroup];
    __shared__ ClusterIn in;
    if (p.cs > 1) cluster_arrive();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = blockIdx.x / p.cs, rank = blockIdx.x % p.cs;
    const int s = unit / p.Hkv, kvh = unit % p.Hkv;
    const int raw = __ldg(p.context_lens + s);
    if ((raw < 0 || raw > p.max_ctx) && kvh == 0 && rank == 0 && tid == 0)
        pkv::report(p.err, PKV_DEVERR_CONTEXT);
    const int n = context_of(p, s);
    const int T = tiles_of(p, n), per = (T + p.cs - 1) / p.cs;
    const int tb = min(T, rank * per), te = min(T, tb + per);

    Feed<D> feed(p, nullptr, smem_of(smem) + warp * kRingBytes<D>, warp, lane, 0, kWarps);
    Acc<D> a;
    feed.begin(s, kvh, n, tb + warp, te, 0);
    attend<E, D, kWide, kScores>(p, feed, s, kvh, tb + warp, te, lane, a);
    cp_async_wait<0>();
    constexpr int COLS = D / 8 / kWarps;
    float o[COLS][kWide ? 4 : 2];
    join_warps<D, kWide>(reinterpret_cast<float*>(smem), warp, lane, a, o);
    if (p.cs > 1) {
        join_cluster<E, D, kWide, kScores>(p, s, kvh, n, tb, te, &in, warp, lane, a, o, s_m, s_inv);
        return;
    }
#pragma unroll
    for (int r = 0; r < (kWide ? 2 : 1); ++r) {
        const int row = (lane >> 2) + 8 * r;
        if (row < p.G) {
            const float inv = output_scale<E>(a.l[r]);
            uint16_t* dst = static_cast<uint16_t*>(p.out) +
                            ((int64_t)s * p.H + (int64_t)kvh * p.G + row) * D + 8 * COLS * warp + 2 * (lane & 3);
#pragma unroll
            for (int j = 0; j < COLS; ++j)
                *reinterpret_cast<uint32_t*>(dst + 8 * j) = E::from_float2(o[j][2 * r] * inv, o[j][2 * r + 1] * inv);
        }
    }
    if constexpr (kScores) {  // the z of this unit were written by this CTA
        if (warp == 0 && (lane & 3) == 0) {
#pragma unroll
            for (int r = 0; r < (kWide ? 2 : 1); ++r) {
                s_m[(lane >> 2) + 8 * r] = a.m[r];
                s_inv[(lane >> 2) + 8 * r] = inverse_of(a.l[r]);
            }
        }
        __syncthreads();
        fold_weights(p, s, kvh, 0, n, s_m, s_inv, tid, kThreads);
    }
}

// Split: range c = blockIdx.x, then whichever ranges this CTA can take.
template <class E, int D, bool kWide, bool kScores>
__global__ void __launch_bounds__(kThreads, 2) split_kernel(const __grid_constant__ Params p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Plan plan;
    constexpr int NO = D / 8;
    constexpr int R = kWide ? 2 : 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int hl = warp % p.hw, split = warp / p.hw;

    {  // tiles before each thread's run of sequences
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

    Feed<D> feed(p, &plan, smem_of(smem) + warp * kRingBytes<D>, warp, lane, hl, p.nsplit);
    Range r = range_at(p, plan.before, plan.map, plan.map.of_cta(blockIdx.x), lane);
    bool running = r.left > 0;  // the same for all warps of the CTA
    if (running && feed.chained())
        feed.begin(r.s, r.hb, r.n, r.tb, min(tiles_of(p, r.n), r.tb + r.left), r.left + r.tb);
    int used = 0;  // ranges taken out of the queue
    while (running) {
        // one unit (or the part of it that lies in this range)
        const int T = tiles_of(p, r.n);
        const int te = min(T, r.tb + r.left);
        const int kvh = r.hb * p.hw + hl;
        const bool last = te - r.tb == r.left;  // of the range
        Acc<D> a;
        if (!feed.chained()) feed.begin(r.s, r.hb, r.n, r.tb + split, te, 0);
        attend<E, D, kWide, kScores>(p, feed, r.s, kvh, r.tb + split, te, lane, a);
        if (!feed.chained()) {
            cp_async_wait<0>();
            join_splits<D, kWide>(p, reinterpret_cast<float*>(smem), warp, lane, a);
        }
        const bool whole = r.tb == 0 && te == T;
        if (split == 0) {
            if (whole) {
                write_rows<E, D, kWide>(p, r.s, kvh, lane, a);
                if constexpr (kScores) {
#pragma unroll
                    for (int x = 0; x < R; ++x)
                        if (t == 0 && g + 8 * x < p.G) {
                            const int64_t oh = (int64_t)r.s * p.H + (int64_t)kvh * p.G + g + 8 * x;
                            p.row_m[oh] = a.m[x];
                            p.row_l[oh] = a.l[x];
                        }
                }
            } else {
                const int64_t piece = 2 * (int64_t)r.c + (r.tb == 0 ? 1 : 0);
#pragma unroll
                for (int x = 0; x < R; ++x) {
                    const int row = g + 8 * x;
                    if (row < p.G) {
                        const int64_t at = (piece * p.hw + hl) * p.G + row;
                        float* dst = p.part_acc + at * D + 2 * t;
#pragma unroll
                        for (int j = 0; j < NO; ++j)
                            *reinterpret_cast<float2*>(dst + 8 * j) =
                                make_float2(a.o[j][2 * x], a.o[j][2 * x + 1]);
                        if (t == 0) {
                            p.part_m[at] = a.m[x];
                            p.part_l[at] = a.l[x];
                        }
                    }
                }
            }
            if (warp == 0 && lane == 0 && r.tb == 0)
                p.place[r.s * p.HB + r.hb] = make_int2(r.c, plan.map.of(r.unit0 + T - 1));
        }
        if (last) {  // the feed has gone on to the next range, if there is one
            running = used < feed.pushed;
            if (running) r = plan.queue[warp][used++ & 3];
            __syncwarp();
        } else {
            r.left -= te - r.tb;
            r.unit0 += T;
            r.tb = 0;
            if (++r.hb == p.HB) {
                r.hb = 0;
                r.n = context_of(p, ++r.s);
            }
        }
    }
    // every request has been answered: a warp stops at the answer that says no
    cp_async_wait<0>();
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

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Direct calls: visible tokens per CTA at most, and CTAs in multiples of the
// resident ones.  A wave of CTAs costs 3 us beside its bytes, a split call 6 to 9
// and with scores 10 to 20, but there it streams while units end.  Windows, direct
// and split: 100 requests of 1..64, 8 KV heads (2.6 waves) 8.2 and 10.9 us, of
// 1..1000 40.2 and 41.6, 148 of 1..500 (3.9 waves) 33.4 and 34.5; 256 of 500 (6.7)
// 90 and 86.  With scores 100 requests of 1..200 19.1 and 20.5, of 1..1000 48.4 and
// 47.1, 148 of 100..250 32.8 and 30.1.  A longer share per CTA (2048) loses where
// few CTAs run (one 32768-token context, scores: 48 us against 36).
constexpr int kDirectTokens = 1024;
constexpr int direct_waves(bool scores, int64_t most) { return !scores ? 4 : most <= 256 ? 3 : 2; }
constexpr int kJoinCtasPerSm = 3;   // of the join kernel
constexpr int kCtasPerSm = 2;       // of the attention kernels
constexpr int kMinUnits = 16;       // of a split call, else fewer KV heads per unit
// Longest context: token numbers go up to the end of a fold's 512 past it.
constexpr int kMaxContext = INT32_MAX - 1024;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
    size_t place, m, l, acc, row_m, row_l, z, total;
    int64_t z_stride;
};

int heads_per_cta(int Hkv) { return Hkv % 4 == 0 ? 4 : (Hkv % 2 == 0 ? 2 : 1); }

// scores: with the logits of contexts up to max_ctx and the rows' M and L.
Layout layout_of(int S, int H, int Hkv, int D, bool scores, int max_ctx) {
    const size_t rows = (size_t)2 * kMaxRanges * heads_per_cta(Hkv) * (H / Hkv);
    Layout L;
    size_t o = 0;
    L.place = o; o = align256(o + (size_t)S * Hkv * sizeof(int2));
    L.m = o;     o = align256(o + rows * sizeof(float));
    L.l = o;     o = align256(o + rows * sizeof(float));
    L.acc = o;   o = align256(o + rows * D * sizeof(float));
    L.row_m = L.row_l = L.z = o;
    const int tile = tile_tokens(D);
    L.z_stride = max_ctx > 0 ? ((int64_t)max_ctx + tile - 1) / tile * tile : tile;
    if (scores) {
        L.row_m = o; o = align256(o + (size_t)S * H * sizeof(float));
        L.row_l = o; o = align256(o + (size_t)S * H * sizeof(float));
        L.z = o;     o = align256(o + (size_t)S * H * L.z_stride * sizeof(float));
    }
    L.total = o;
    return L;
}

using KernelFn = void (*)(Params);
using JoinFn = void (*)(Params, int);

template <class E, bool kScores, bool kDirect>
KernelFn pick_attend(int D, bool wide) {
    if constexpr (kDirect) {
        if (D == 128) return wide ? direct_kernel<E, 128, true, kScores> : direct_kernel<E, 128, false, kScores>;
        return wide ? direct_kernel<E, 64, true, kScores> : direct_kernel<E, 64, false, kScores>;
    } else {
        if (D == 128) return wide ? split_kernel<E, 128, true, kScores> : split_kernel<E, 128, false, kScores>;
        return wide ? split_kernel<E, 64, true, kScores> : split_kernel<E, 64, false, kScores>;
    }
}
template <bool kScores, bool kDirect>
KernelFn pick_attend(pkv_dtype dtype, int D, bool wide) {
    return dtype == PKV_F16 ? pick_attend<pkv::F16, kScores, kDirect>(D, wide)
                            : pick_attend<pkv::BF16, kScores, kDirect>(D, wide);
}

template <class E, int D>
JoinFn pick_join(bool scores, bool one) {
    if (!scores) return join_kernel<E, D, false, false>;
    return one ? join_kernel<E, D, true, true> : join_kernel<E, D, true, false>;
}
JoinFn pick_join(pkv_dtype dtype, int D, bool scores, bool one) {
    if (dtype == PKV_F16) return D == 128 ? pick_join<pkv::F16, 128>(scores, one) : pick_join<pkv::F16, 64>(scores, one);
    return D == 128 ? pick_join<pkv::BF16, 128>(scores, one) : pick_join<pkv::BF16, 64>(scores, one);
}

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

pkv_status run_bounded(const char* who, void* out, const void* q, const void* k_cache,
                       const void* v_cache, const int32_t* block_tables,
                       const int32_t* context_lens, int S, int H, int Hkv, int D, int bs, int NB,
                       int MB, int max_context_len, int window, int sinks, float scale,
                       pkv_dtype dtype, bool with_scores, float* scores, int64_t score_stride,
                       void* workspace, size_t workspace_bytes, void* stream) {
    char msg[256];
    auto bad = [&](pkv_status st, const char* what) {
        snprintf(msg, sizeof msg, "%s: %s", who, what);
        return pkv::fail(st, msg);
    };
    if (S < 0 || H <= 0 || Hkv <= 0 || NB <= 0 || MB <= 0 || (dtype != PKV_F16 && dtype != PKV_BF16))
        return bad(PKV_ERR_INVALID_ARG, "bad size or dtype");
    if ((D != 64 && D != 128) || (bs != 8 && bs != 16 && bs != 32 && bs != 64))
        return bad(PKV_ERR_UNSUPPORTED, "head_dim must be 64/128, block_size 8/16/32/64");
    if (H % Hkv != 0) return bad(PKV_ERR_INVALID_ARG, "H must be a multiple of Hkv");
    if (H / Hkv > kMaxGroup) return bad(PKV_ERR_UNSUPPORTED, "at most 16 query heads per KV head");
    if (window < 1 || sinks < 0) return bad(PKV_ERR_INVALID_ARG, "window must be >= 1 and sink_tokens >= 0");
    if (!(scale == scale) || std::isinf(scale)) return bad(PKV_ERR_INVALID_ARG, "scale must be finite");
    if ((int64_t)NB * bs > INT32_MAX) return bad(PKV_ERR_INVALID_ARG, "NB * bs must fit 31 bits");
    if (S > 32767 || (int64_t)S * H > INT32_MAX / kMaxCluster)
        return bad(PKV_ERR_INVALID_ARG, "at most 32767 sequences, and 2^27 heads in all of them");
    const int64_t cap = (int64_t)MB * bs;
    const int64_t max_ctx = max_context_len == 0 ? (cap < kMaxContext ? cap : kMaxContext) : max_context_len;
    if (max_ctx < 0 || max_ctx > cap || max_ctx > kMaxContext)
        return bad(PKV_ERR_INVALID_ARG, "max_context_len must be in [0, MB*bs], below 2^31 - 1024");
    if (S == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || (with_scores && !scores))
        return bad(PKV_ERR_INVALID_ARG, "null pointer");
    if (!pkv::aligned16(out) || !pkv::aligned16(q) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache))
        return bad(PKV_ERR_INVALID_ARG, "token pointers must be 16-byte aligned");
    if (with_scores && (reinterpret_cast<uintptr_t>(scores) & 3u))
        return bad(PKV_ERR_INVALID_ARG, "scores must be 4-byte aligned");
    if (with_scores && score_stride < max_ctx)
        return bad(PKV_ERR_INVALID_ARG, "score_stride must be at least max_context_len");
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return bad(PKV_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
    const Layout L = layout_of(S, H, Hkv, D, with_scores, (int)max_ctx);
    if (workspace_bytes < L.total) return bad(PKV_ERR_WORKSPACE, "workspace too small");

    Params p;
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.S = S;
    p.H = H;
    p.Hkv = Hkv;
    p.G = H / Hkv;
    p.NB = NB;
    p.MB = MB;
    p.bs_log2 = bs == 8 ? 3 : (bs == 16 ? 4 : (bs == 32 ? 5 : 6));
    p.max_ctx = (int)max_ctx;
    p.window = window;
    p.sinks = sinks;
    p.qscale = scale * kLog2e;
    char* w = static_cast<char*>(workspace);
    p.place = reinterpret_cast<int2*>(w + L.place);
    p.part_m = reinterpret_cast<float*>(w + L.m);
    p.part_l = reinterpret_cast<float*>(w + L.l);
    p.part_acc = reinterpret_cast<float*>(w + L.acc);
    p.row_m = reinterpret_cast<float*>(w + L.row_m);
    p.row_l = reinterpret_cast<float*>(w + L.row_l);
    p.z = reinterpret_cast<float*>(w + L.z);
    p.z_stride = L.z_stride;
    p.scores = scores;
    p.score_stride = score_stride;
    p.err = pkv::device_error_word();
    const int64_t most = (int64_t)window + sinks < max_ctx ? (int64_t)window + sinks : max_ctx;
    const int tile = tile_tokens(D);
    p.tile_log2 = tile == 16 ? 4 : 5;
    const bool wide = p.G > 8;
    const int smem = D == 128 ? kSmemBytes<128> : kSmemBytes<64>;
    KernelFn direct_fn = with_scores ? pick_attend<true, true>(dtype, D, wide) : pick_attend<false, true>(dtype, D, wide);
    KernelFn split_fn = with_scores ? pick_attend<true, false>(dtype, D, wide) : pick_attend<false, false>(dtype, D, wide);
    const int sms = pkv::sm_count();
    // direct: the smallest cluster that leaves kDirectTokens per CTA; more CTAs
    // while they still fit the card at once and have a tile per warp (a cluster's
    // join costs as much as two or, of many rows, three more tiles: 150 tokens 4.4 us
    // in one CTA, 5.1 in two; 220 tokens, 8 query heads a head: 5.2 and 6.0)
    const int64_t slots = (int64_t)kCtasPerSm * sms;
    p.cs = 1;
    while (p.cs < kMaxCluster && most > (int64_t)kDirectTokens * p.cs) p.cs *= 2;
    const bool direct = most <= (int64_t)kDirectTokens * p.cs &&
                        (int64_t)S * Hkv * p.cs <= direct_waves(with_scores, most) * slots;
    if (direct)
        while (p.cs < kMaxCluster && (int64_t)S * Hkv * p.cs * 2 <= slots &&
               most > (int64_t)(p.cs > 1 ? 2 : p.G > 4 ? 4 : 3) * kWarps * tile * p.cs)
            p.cs *= 2;
    p.hw = direct ? 1 : heads_per_cta(Hkv);
    while (!direct && p.hw > 1 && (int64_t)S * Hkv / p.hw < kMinUnits) p.hw /= 2;
    p.nsplit = kWarps / p.hw;
    p.HB = Hkv / p.hw;
    const int per_sm = resident_of(direct ? direct_fn : split_fn, smem);
    if (per_sm < 1) return bad(PKV_ERR_CUDA, "the kernel cannot be resident");
    p.ranges0 = per_sm * sms;
    if (p.ranges0 > kMaxRanges / (1 + kSmallRanges)) p.ranges0 = kMaxRanges / (1 + kSmallRanges);
    // small ranges only where changing over costs nothing (a warp per head), and
    // where contexts at their bound would have some
    const int64_t most_tiles = (int64_t)S * p.HB * ((most + tile - 1) / tile);
    const bool share = p.nsplit == 1 && most_tiles / p.ranges0 * (16 - kLargeShare) / 16 / kSmallRanges >= kMinSmall;
    p.ranges = share ? p.ranges0 * (1 + kSmallRanges) : p.ranges0;

    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = pkv::as_stream(stream);
    cfg.attrs = attr;
    cfg.numAttrs = direct && p.cs > 1 ? 2 : 1;
    cfg.gridDim = dim3(direct ? (unsigned)(S * Hkv * p.cs) : (unsigned)p.ranges);
    cudaError_t e = cudaLaunchKernelEx(&cfg, direct ? direct_fn : split_fn, p);
    if (e == cudaSuccess && !direct) {
        // units of more than 8 pieces: a CTA per row
        const int wide = p.ranges > 8 * (int64_t)S * p.HB;
        cfg.dynamicSmemBytes = 0;
        cfg.numAttrs = 1;
        cfg.blockDim = dim3(kJoinThreads);
        cfg.gridDim = dim3((unsigned)(kJoinCtasPerSm * sms));
        e = cudaLaunchKernelEx(&cfg, pick_join(dtype, D, with_scores, p.G == 1), p, wide);
    }
    if (e != cudaSuccess) {
        snprintf(msg, sizeof msg, "%s launch", who);
        return pkv::cuda_fail(e, msg);
    }
    return PKV_OK;
}

bool workspace_args_ok(int S, int H, int Hkv, int D) {
    return S >= 0 && H > 0 && Hkv > 0 && H % Hkv == 0 && H / Hkv <= kMaxGroup && (D == 64 || D == 128);
}

}  // namespace

extern "C" {

size_t pkv_decode_window_workspace_size(int S, int H, int Hkv, int D) {
    if (!workspace_args_ok(S, H, Hkv, D)) return 0;
    return layout_of(S, H, Hkv, D, false, 0).total;
}

pkv_status pkv_paged_attention_decode_window(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, int S, int H, int Hkv, int D, int bs,
    int NB, int MB, int max_context_len, int window, int sink_tokens, float scale, pkv_dtype dtype,
    void* workspace, size_t workspace_bytes, void* stream) {
    PKV_TRACE("pkv_paged_attention_decode_window");
    pkv::clear_error();
    return run_bounded("paged_attention_decode_window", out, q, k_cache, v_cache, block_tables,
                       context_lens, S, H, Hkv, D, bs, NB, MB, max_context_len, window, sink_tokens,
                       scale, dtype, false, nullptr, 0, workspace, workspace_bytes, stream);
}

size_t pkv_decode_accumulate_workspace_size(int S, int H, int Hkv, int D, int max_context_len) {
    if (!workspace_args_ok(S, H, Hkv, D) || max_context_len < 1 || max_context_len > kMaxContext)
        return 0;
    return layout_of(S, H, Hkv, D, true, max_context_len).total;
}

pkv_status pkv_paged_attention_decode_accumulate(
    void* out, float* scores, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, int S, int H, int Hkv, int D, int bs,
    int NB, int MB, int max_context_len, int64_t score_stride, float scale, pkv_dtype dtype,
    void* workspace, size_t workspace_bytes, void* stream) {
    PKV_TRACE("pkv_paged_attention_decode_accumulate");
    pkv::clear_error();
    // every token is visible: a window as long as any context, no sinks
    return run_bounded("paged_attention_decode_accumulate", out, q, k_cache, v_cache, block_tables,
                       context_lens, S, H, Hkv, D, bs, NB, MB, max_context_len, INT32_MAX, 0, scale,
                       dtype, true, scores, score_stride, workspace, workspace_bytes, stream);
}

}  // extern "C"
