// Decode attention over a cache held in 4 bits (q4.cuh).
//
// For sequence s, query head h of KV head g, context n, groups r of 64 dims:
//   z_j = scale sum_r (step_jr sum_{d in r} q_d c_jd + centre_jr sum_{d in r} q_d),  c = code - 8
//   out_d = sum_j p_j (step_jr c_jd + centre_jr),  p = softmax z.
// So the codes go into the products as they are, exact in fp16, and the steps
// and centres are applied outside of them, in fp32: to the group's part of a
// logit, and to the weight, of which each group of V has its own, p_j step_jr.
//
// Units, tiles, ranges and the two ways to spread them (direct, split) are
// unit_ranges.cuh's.  A unit is one sequence and `hw` neighbouring KV heads; one
// warp takes one head of a 64-token tile: 8 runs of 8 tokens of K and of V, in one
// asynchronous bulk copy per block (a (block, head) is one run of the pool) by a
// lane of its own, an mbarrier per stage of the warp's ring.
//
// The products are m16n8k16 in fp16 with the cache as the 16 rows and the query
// heads as the 8 columns, S^T = K Q^T and O^T = V^T P^T: a group of up to 8 query
// heads fills them with half the products that heads as rows would take, and
// accumulators of half the size (more than 8 heads: two column blocks).
//  * Codes to fp16: a nibble at bits 0 or 4 of a half is, as a subnormal number,
//    2^-24 or 2^-20 times the code: 5 instructions per 8 codes.  The 8 that a code
//    is to lose comes off the sums: K's products start from -8 sum q; V's are
//    corrected every tile by a product of the same weights with -8 (not at
//    the end: sums that grow with the context would lose digits).
//  * K: ldmatrix gives a lane 8 codes of one token, 32 bits; q is loaded in the
//    order that makes of them two fragments.  A power of two per head makes q
//    fp16 with the codes' units taken out, exact but for elements below 2^-23 (fp16)
//    or 2^-26 (bf16) of the largest: what they lose is below 2^-34 of it.
//  * V: transposing ldmatrix of 16-bit pieces, 4 codes of one token each, gives a
//    lane 4 codes of two neighbouring tokens: the pairs that the product's k wants.
//  * P^T comes out of S^T's accumulators by movmatrix.  A weight times its step
//    enters the product as fp16, rounded by 2^-11 of itself: an eighth of a bf16
//    output's own rounding (a second number makes bf16 calls 8 to 20 % slower, and no
//    more exact: 1.6e-3 off 64 bits either way, which is the outputs' rounding).  For
//    fp16 outputs, whose rounding is no larger, what is left does enter as a second
//    number.  The products' units are each head's and
//    group's own and follow the largest of its products, which lies in 2^8 .. 2^15:
//    what falls below 2^-24 is 2^-32 of the largest.  (Units by the steps alone, the
//    same for all, take no vote on the products and are 1 % faster with up to 4 heads,
//    2 to 5 % with more, 10 % where 16 heads have one tile per warp.  But a group whose
//    steps are 2^30 below the other's, or a row with one such token of no weight, keeps
//    no digits in them.)
//  * The running maximum moves only when a logit passes it by more than kLazy: one
//    vote per tile instead of three exchanges per head.
//
// Measured, D = 128 (in brackets what the bytes take at a plain copy's rate, 6.80
// TB/s): 32 contexts of 4001..16384, 32 heads in fp16, 266 us (221); 32 of 32768, 8
// KV heads of 4 query heads in bf16, 204 (178), of 16384 108 (89): what a token adds
// runs at 93 % of that rate.  256 of 16..4096 60 (35); one of 32768 14.5 (6); a handful
// of short ones 3.4.  With 8 and with 16 query heads per KV head, whose products, weights
// and registers are more: 32 of 16384 126 and 184 (89), 256 of 16..4096 70 and 106 (36,
// 37), one of 32768 17.3 and 25.9 (6).  What bounds it: nothing is busy all the time.
// Long batches have DRAM at 72 % of its peak, the tensor pipe at 43 %, the ALU, which
// unpacks, at 51 %, and issue at 54 %; a warp's chain of products waits for the pipes,
// and 12 warps are what the registers hold (the forms of D = 128 spill 8 to 60 bytes
// at that).  Mixed lengths: that and the ends, 5 us until the rings are full, CTAs of
// an SM that end up to 10 us apart, as its older warps go first, and the join, 4 to 8
// us.  Few units: eight of them fill 96 SMs of 152 with twelve warps, whose next tiles
// cost 2.4 us each.  None of these gained: stages of 32 tokens (73 us where these take
// 65.5), passes of 16 tokens with a fourth CTA per SM (77 for 67), two CTAs of 255
// registers per SM (the same), three or four stages for few units (the same), ranges
// of one tile (116 for 110), ranges by a CTA's turn on its SM (113 to 119 for 110).
#include <cooperative_groups.h>

#include <climits>
#include <cmath>
#include <cstdio>
#include <mutex>
#include <type_traits>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_mma.cuh"
#include "q4.cuh"
#include "unit_ranges.cuh"

namespace cg = cooperative_groups;

namespace {

namespace q4 = pkv::q4;
using pkv::ldsm_x4;
using pkv::ldsm_x4_trans;

constexpr int kTile = 64;                    // tokens of a stage at most; short contexts go in tiles of 32
constexpr int kRuns = kTile / q4::kUnit;     // runs of 8 tokens in it
template <int D>
constexpr int kStages = D == 128 ? 2 : 3;  // what 3 (4) CTAs per SM leave room for
constexpr int kMaxRanges = 1824;  // CTAs of a split call
// log2 of what a weight may pass 1 by: it spares a scaling of every sum wherever a
// maximum creeps up.
constexpr float kLazy = 6.f;
// A weight's product with a step, in the units it enters fp16 with, stays below
// kProductMost; units that have to be new make the largest kUnits to 2 kUnits, so that
// the weights have as much room again.
constexpr float kProductMost = 0x1p15f, kUnits = 256.f;
constexpr float kUnitMost = 0x1p119f;  // of the units: the least step they are for is 2^-111

// K (or V) of one stage.
template <int D>
constexpr int kHalfBytes = kRuns * q4::kUnitBytes<D>;
template <int D>
constexpr int kRingBytes = kStages<D> * 2 * kHalfBytes<D>;  // one warp's ring
// What the 8 columns of a product are: 8 query heads, or, for groups of up to 4,
// (head, group of 64 dims): then one chain of products gives a logit's parts side
// by side, one column block carries the weights of both groups, and a lane has
// one head to take through the softmax instead of two.
template <int kPass>
struct Narrow {
    static constexpr bool kNarrow = true;
    static constexpr int X = 1, HL = 1;  // column blocks, heads per lane and block
    static constexpr int PASS = kPass;   // tokens that go through the softmax together
};
template <int kBlocks>
struct Heads {
    static constexpr bool kNarrow = false;
    static constexpr int X = kBlocks, HL = 2;
    static constexpr int PASS = 32;      // (the registers are for no more)
};

// CTAs per SM that the registers are for
template <int D, class C>
constexpr int kCtas = C::X == 2 ? 2 : (D == 64 ? 4 : 3);

// Warps of a direct call's CTAs: 4, or, for few units, half of what an SM takes, or
// (twice as many) all of it.
template <int D, class C>
constexpr int kManyWarps = C::X == 2 ? 4 : (D == 128 ? 6 : 8);

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// An 8x8 block of 16-bit elements, two of a row per lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The codes 4e and 16 + 4e bits up in x, e = 0..3, as pairs of fp16: times 2^-24
// for even e, times 2^-20 for odd.
constexpr float kEven = 0x1p-24f, kOdd = 0x1p-20f;
__device__ __forceinline__ void codes_of(uint32_t x, uint32_t (&h)[4]) {
    const uint32_t y = x >> 8;
    h[0] = x & 0x000f000fu;
    h[1] = x & 0x00f000f0u;
    h[2] = y & 0x000f000fu;
    h[3] = y & 0x00f000f0u;
}
constexpr uint32_t kMinus8Even = 0x80088008u, kMinus8Odd = 0x80808080u;  // -8 in these units

__device__ __forceinline__ void bulk_copy(uint32_t dst, const char* src, int bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// The (step, centre) pairs of a row, one per group.
template <int NG>
__device__ __forceinline__ void pairs_at(uint32_t from, uint32_t (&pair)[NG]) {
    if constexpr (NG == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(pair[0]), "=r"(pair[1]) : "r"(from) : "memory");
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(pair[0]) : "r"(from) : "memory");
}

// One warp's tiles on their way through its ring, `step` apart, each looked up one
// tile ahead of its copies and copied kStages - 1 ahead of its use.  Chained (a plan,
// and all tiles are this warp's) it goes on into the units and ranges that follow.
template <int D>
struct Feed {
    static constexpr int NST = kStages<D>;
    static constexpr int UB = q4::kUnitBytes<D>;
    const Params& p;
    Plan* const plan;          // null: one unit (part) at a time
    int* const abort;
    const uint32_t ring, bars; // bars: an mbarrier per stage
    const int warp, lane, hl;  // hl: head of the CTA's hw that this warp takes
    const int step;
    const bool chained;
    const uint64_t policy;
    const char* const cache;   // lanes 0..7 copy K's runs, 8..15 V's
    int s, hb, n_next, i, te, left;  // the next tile, and its unit; left: from its tile 0 to the range's end
    int rest, count;           // the unit's tokens from that tile on, the tile's tokens
    const int32_t* bt;
    int tok, phys;             // of the tile's run lane % 8: first token, and its block, if wanted()
    bool more;
    int has[NST];              // of the stages in the ring: runs with tokens, and tokens << 8
    int into, from;            // stages of the next copy and of the oldest one
    unsigned phase;            // bit st: parity of stage st's copy that is waited for next
    int asked, answers, pushed;

    __device__ __forceinline__ Feed(const Params& p_, Plan* plan_, int* abort_, uint32_t ring_, uint32_t bars_,
                                    int warp_, int lane_, int hl_, int step_)
        : p(p_), plan(plan_), abort(abort_), ring(ring_), bars(bars_), warp(warp_), lane(lane_), hl(hl_),
          step(step_), chained(plan_ != nullptr && step_ == 1),
          // a split call streams more than it could find again in L2
          policy(plan_ ? pkv::policy_evict_first() : pkv::policy_evict_normal()),
          cache(static_cast<const char*>(lane_ < 8 ? p_.k_cache : p_.v_cache)), into(0), from(0), phase(0),
          asked(0), answers(0), pushed(0) {
        if (lane == 0)
            for (int st = 0; st < NST; ++st) tc_mbar_init(bars + 8 * st, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    }

    __device__ __forceinline__ void enter(int n) {  // unit (s, hb), at its tile i
        rest = n - (i << p.tile_log2);
        bt = p.block_tables + (int64_t)s * p.MB;
        const char* q = static_cast<const char*>(p.q) +
                        ((int64_t)s * p.H + (int64_t)(hb * p.hw + hl) * p.G) * D * 2;
        if (lane * 128 < p.G * D * 2) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + lane * 128));
    }

    // The next tile's blocks; they are used when it is pushed.
    __device__ __forceinline__ void lookup() {
        if (!more) return;
        count = max(min(1 << p.tile_log2, rest), 0);
        tok = (i << p.tile_log2) + (lane & 7) * q4::kUnit;
        // (not touched here: whatever uses it would wait for it)
        if (wanted()) phys = __ldg(bt + (tok >> p.bs_log2));
    }
    __device__ __forceinline__ bool wanted() const { return lane < 16 && (lane & 7) * q4::kUnit < count; }

    __device__ __forceinline__ void begin(int s_, int hb_, int n, int first, int te_, int left_) {
        s = s_;
        hb = hb_;
        i = first;
        te = te_;
        left = left_;
        n_next = chained && s + 1 < p.S ? context_of(p, s + 1) : 0;
        more = i < te && !*(volatile int*)abort;
        count = tok = phys = 0;
        enter(n);
        lookup();
#pragma unroll
        for (int st = 0; st < NST - 1; ++st) push(st);
    }

    __device__ __forceinline__ void maybe_ask(int tiles_left) {
        if (warp == 0 && tiles_left <= 2 && asked == answers) {
            if (lane == 0) ask_range(plan, asked);
            ++asked;
        }
    }
    __device__ __forceinline__ bool next() {
        maybe_ask(0);
        int k = answers;
        const bool got = next_range(p, plan, warp, lane, k, pushed);
        asked = answers = k;
        if (got) ++pushed;
        return got;
    }

    // Copies the next tile into the ring, what it has into has[at], then looks up
    // the one after it.
    __device__ __forceinline__ void push(int at) {
        if (!more) return;
        const bool want = wanted(), there = want && (unsigned)phys < (unsigned)p.NB;
        if (want && !there) pkv::report(p.err, PKV_DEVERR_BLOCK_ID);
        const unsigned runs = __ballot_sync(kFull, there) & ((1u << kRuns) - 1u);
        has[at] = (int)runs | count << 8;
        const uint32_t bar = bars + 8 * into;
        if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                         "r"(__popc(runs) * 2 * UB)
                         : "memory");
        __syncwarp();
        // lanes 0..7: K's runs, 8..15: V's.  The runs of a block are one piece.
        const int units = p.bs_log2 - 3, whole = 1 << units;
        if (there && (lane & (whole - 1)) == 0) {
            // the pool's units of 8 tokens fit an int (checked on the host)
            const int unit = ((phys * p.Hkv + hb * p.hw + hl) << units) | ((tok >> 3) & ((1 << units) - 1));
            const int n = min(whole, (count - (lane & 7) * q4::kUnit + q4::kUnit - 1) / q4::kUnit);
            bulk_copy(ring + (2 * into + (lane >> 3)) * kHalfBytes<D> + (lane & 7) * UB, cache + (int64_t)unit * UB, n * UB,
                      bar, policy);
        }
        into = into + 1 == NST ? 0 : into + 1;
        i += step;
        rest -= step << p.tile_log2;
        if (i >= te) advance();
        if (more && chained) maybe_ask(left - i);
        lookup();
    }

    // The whole warp waits for stage `from`.  When that runs out it gives what else may
    // be on its way into this CTA's memory some more time.
    static __device__ __noinline__ bool wait_on(uint32_t bars, int from, unsigned phase, int* abort, int* err,
                                                uint32_t answer, uint32_t answer_parity) {
        if (__all_sync(kFull, tc_mbar_wait(bars + 8 * from, phase >> from & 1u, abort))) return true;
        pkv::report(err, PKV_DEVERR_TIMEOUT);
        *(volatile int*)abort = 1;
        auto drain = [](uint32_t bar, uint32_t parity) {
            for (int k = 0; k < 4096; ++k)
                if (tc_mbar_try(bar, parity)) return;
        };
        for (int st = 0; st < NST; ++st) drain(bars + 8 * st, phase >> st & 1u);
        if (answer) drain(answer, answer_parity);
        __syncwarp();
        return false;
    }
    // Waits for the oldest stage; false: in vain, and nothing is copied any more.
    __device__ __forceinline__ bool wait() {
        if (__all_sync(kFull, tc_mbar_try(bars + 8 * from, phase >> from & 1u))) return true;
        const uint32_t answer = plan && warp == 0 && asked != answers ? smem_of(&plan->full[answers & 1]) : 0u;
        if (wait_on(bars, from, phase, abort, p.err, answer, (answers >> 1) & 1)) return true;
        more = false;
        return false;
    }
    __device__ __forceinline__ void done() {
        phase ^= 1u << from;
        from = from + 1 == NST ? 0 : from + 1;
#pragma unroll
        for (int st = 0; st < NST - 1; ++st) has[st] = has[st + 1];
        __syncwarp();  // this stage is filled again by the next push
    }

    __device__ __forceinline__ void advance() {
        more = false;
        if (!chained) return;
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

// What a warp has of its unit: lane (g, t) = (lane / 4, lane % 4) has, of its
// heads (head_of), the dims 32 i + 4 g + e, and the heads' m and l.
template <int D, class C>
struct Acc {
    float o[C::X][D / 32][2][4];
    float m[C::X][C::HL], l[C::X][C::HL];
    __device__ __forceinline__ float& at(int x, int i, int e, int h) {
        return o[x][i][e >> 1][2 * (e & 1) + (C::kNarrow ? i / 2 : h)];
    }
    static __device__ __forceinline__ int head_of(int x, int t, int h) { return C::kNarrow ? t : 8 * x + 2 * t + h; }
};

// Sum over the lanes with the same t.
__device__ __forceinline__ float sum_rows(float x) {
    x += __shfl_xor_sync(kFull, x, 4);
    x += __shfl_xor_sync(kFull, x, 8);
    return x + __shfl_xor_sync(kFull, x, 16);
}
__device__ __forceinline__ float max_rows(float x) {
    x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
    x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
    return fmaxf(x, __shfl_xor_sync(kFull, x, 16));
}

// One warp: KV head kvh of sequence s, its tiles first, first + step, ... below
// te out of the feed.
template <class E, int D, class C>
__device__ __forceinline__ void attend(const Params& p, Feed<D>& feed, int s, int kvh, int first, int te, int lane,
                                       Acc<D, C>& a) {
    constexpr int NI = D / 32, NG = D / q4::kGroup, UB = q4::kUnitBytes<D>, UC = q4::kUnitCodes<D>;
    constexpr int SUB = C::PASS / 16, X = C::X, HL = C::HL;
    constexpr int CH = C::kNarrow ? 1 : NG;  // columns of weights per group
    constexpr bool kHalf = std::is_same<E, pkv::F16>::value;
    constexpr int PARTS = kHalf ? 2 : 1;     // numbers that make a weight
    constexpr float kProduct = 0x1p-11f;     // of a code and the largest query elements' power of two
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < X; ++x) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) a.o[x][i][0][c] = a.o[x][i][1][c] = 0.f;
#pragma unroll
        for (int h = 0; h < HL; ++h) {
            a.m[x][h] = -INFINITY;
            a.l[x][h] = 0.f;
        }
    }
    if (first >= te) return;

    // The queries as columns: lane (g, t) has column g's head, and of chunk i the
    // dims 32 i + 8 t + e and + 4, e = 0 .. 3, as the codes come.
    uint32_t qb[X][NI][4];
    float qs[X][HL], qsum[X][NG][HL];  // of the lane's heads: units of its logits, sums over the groups
#pragma unroll
    for (int x = 0; x < X; ++x) {
        const int head = C::kNarrow ? g >> 1 : 8 * x + g;
        const uint16_t* q =
            static_cast<const uint16_t*>(p.q) + ((int64_t)s * p.H + (int64_t)kvh * p.G + head) * D + 8 * t;
        float f[NI][8], top = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (head < p.G) raw = __ldg(reinterpret_cast<const uint4*>(q + 32 * i));
            pkv::unpack8<E>(raw, f[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[i][e]));
        }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // the power of two at or below the largest; its inverse times what the codes'
        // units ask for makes the query fp16, below 2^14 (it stops at 2^112: queries of
        // 2^113 are bf16's last powers, and their logits' units would not be finite); a
        // negative scale is the query's sign
        const uint32_t ex = min(max(__float_as_uint(top) & 0x7f800000u, 0x08000000u), 0x77800000u);
        const float unit = __uint_as_float(ex);
        const float down = p.qscale < 0.f ? -__uint_as_float((254u << 23) - ex) : __uint_as_float((254u << 23) - ex);
        float part[NG];  // sums over the groups, in units of the products'
#pragma unroll
        for (int r = 0; r < NG; ++r) part[r] = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool mine = !C::kNarrow || (g & 1) == i / 2;  // narrow: column g has group g % 2
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float up = down * ((e & 1 ? 0x1p20f : 0x1p24f) * kProduct);
                qb[x][i][e] = mine ? pkv::F16::from_float2(f[i][e] * up, f[i][e + 4] * up) : 0u;
                const float2 back = pkv::F16::to_float2(qb[x][i][e]);
                part[i / 2] = fmaf(back.x + back.y, e & 1 ? kOdd : kEven, part[i / 2]);
            }
        }
#pragma unroll
        for (int r = 0; r < NG; ++r) {
            part[r] += __shfl_xor_sync(kFull, part[r], 1);
            part[r] += __shfl_xor_sync(kFull, part[r], 2);
        }
        // column c is in lanes 4 c ..; no logit's unit is 0: nothing times -infinity
#pragma unroll
        for (int h = 0; h < HL; ++h) {
            qs[x][h] =
                fmaxf(__shfl_sync(kFull, unit, 4 * (2 * t + h)) * (fabsf(p.qscale) * (1.f / kProduct)), 0x1p-126f);
#pragma unroll
            for (int r = 0; r < NG; ++r)
                qsum[x][r][h] = __shfl_sync(kFull, part[r], 4 * (2 * t + (C::kNarrow ? r : h)));
        }
    }

    float centres[X][NG][HL];  // sum of p times V's centres, this lane's tokens
    float less[X][HL];         // -m, 0 for none yet
#pragma unroll
    for (int x = 0; x < X; ++x)
#pragma unroll
        for (int h = 0; h < HL; ++h) {
            less[x][h] = 0.f;
#pragma unroll
            for (int r = 0; r < NG; ++r) centres[x][r][h] = 0.f;
        }
    float wu[X][NG][HL];       // units of the weights' products with the steps: powers of two
#pragma unroll
    for (int x = 0; x < X; ++x)
#pragma unroll
        for (int r = 0; r < NG; ++r)
#pragma unroll
            for (int h = 0; h < HL; ++h) wu[x][r][h] = kUnitMost;

    // this lane's address in ldmatrix: matrix lane / 8, row lane % 8; x4 is two
    // chunks of two units
    const int mrow = lane & 7, munit = (lane >> 3) & 1, mchunk = lane >> 4;
    uint32_t at[NG];
#pragma unroll
    for (int r = 0; r < NG; ++r)
        at[r] = munit * UB + mrow * q4::code_bytes(D) + 16 * q4::chunk_place<D>(mrow, 2 * r + mchunk);
    const uint32_t pair_at = UC + g * q4::pair_bytes(D);

    for (int i = first; i < te; i += feed.step) {
        feed.push(Feed<D>::NST - 1);
        const int has = feed.has[0], count = has >> 8;
        const uint32_t stage = feed.ring + feed.from * 2 * kHalfBytes<D>;
        if (!feed.wait()) break;
        float eight[X][CH][4];  // -8 times the stage's weights in the columns: rows of even e, of odd e
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
            for (int r = 0; r < CH; ++r) eight[x][r][0] = eight[x][r][1] = eight[x][r][2] = eight[x][r][3] = 0.f;
#pragma unroll 1
      for (int pass = 0; pass == 0 || (C::PASS < kTile && pass * C::PASS < count); ++pass) {
        constexpr int RUNS = C::PASS / q4::kUnit;
        const uint32_t sk = stage + pass * RUNS * UB, sv = sk + kHalfBytes<D>;
        // tokens 8 u + g of the pass, bit u
        constexpr unsigned all = (1u << RUNS) - 1u;
        unsigned rows = (unsigned)has >> (RUNS * pass) & all;
        const bool some = rows != all || count < (pass + 1) * C::PASS;  // not all of the tokens
        if (some)
#pragma unroll
            for (int u = 0; u < RUNS; ++u)
                if (8 * u + g >= count - pass * C::PASS) rows &= ~(1u << u);

        // v[x][sub][u][h]: logit of token 16 sub + 8 u + g in units of qs
        float v[X][SUB][2][HL], dot[SUB][X][NG][4];  // dot: element 2 u + h is column 2 t + h
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int r = 0; r < NG; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h)  // the 8 that every code is to lose (narrow: column r is group r's)
                        dot[sub][x][r][h] = dot[sub][x][r][2 + h] = -8.f * qsum[x][r][h % HL];
#pragma unroll
        for (int r = 0; r < NG; ++r) {
            uint32_t k[SUB][4];  // chunks 2 r, 2 r + 1
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) ldsm_x4(k[sub], sk + at[r] + 2 * sub * UB);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t h0[SUB][4], h1[SUB][4];
#pragma unroll
                for (int sub = 0; sub < SUB; ++sub) {
                    codes_of(k[sub][2 * c], h0[sub]);      // token g
                    codes_of(k[sub][2 * c + 1], h1[sub]);  // token g + 8
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2)
#pragma unroll
                    for (int sub = 0; sub < SUB; ++sub) {
                        const uint32_t f[4] = {h0[sub][e], h1[sub][e], h0[sub][e + 1], h1[sub][e + 1]};
#pragma unroll
                        for (int x = 0; x < X; ++x)
                            pkv::Mma<pkv::F16>::run(dot[sub][x][r], f, qb[x][2 * r + c][e], qb[x][2 * r + c][e + 1]);
                    }
            }
        }
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t pair[NG];
                pairs_at<NG>(sk + pair_at + (2 * sub + u) * UB, pair);
#pragma unroll
                for (int x = 0; x < X; ++x)
#pragma unroll
                    for (int h = 0; h < HL; ++h) {
                        float sum = 0.f;
#pragma unroll
                        for (int r = 0; r < NG; ++r) {
                            const float2 sc = E::to_float2(pair[r]);
                            sum = fmaf(sc.x, dot[sub][x][r][2 * u + (C::kNarrow ? r : h)], sum);
                            sum = fmaf(sc.y, qsum[x][r][h], sum);
                        }
                        v[x][sub][u][h] = sum;
                    }
            }
        // V's steps and centres
        uint32_t vpair[SUB][2][NG];
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
            for (int u = 0; u < 2; ++u) pairs_at<NG>(sv + pair_at + (2 * sub + u) * UB, vpair[sub][u]);
        if (some) {  // nothing where there is no token
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (!((rows >> (2 * sub + u)) & 1u)) {
#pragma unroll
                        for (int x = 0; x < X; ++x)
#pragma unroll
                            for (int h = 0; h < HL; ++h) v[x][sub][u][h] = -INFINITY;
#pragma unroll
                        for (int r = 0; r < NG; ++r) vpair[sub][u][r] = 0u;
                    }
        }

        // does a maximum move?
        float top[X][HL];
        bool moves = false;
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
            for (int h = 0; h < HL; ++h) {
                float y = fmaxf(v[x][0][0][h], v[x][0][1][h]);
#pragma unroll
                for (int sub = 1; sub < SUB; ++sub) y = q4::max3(y, v[x][sub][0][h], v[x][sub][1][h]);
                top[x][h] = y * qs[x][h];
                moves = moves || top[x][h] > a.m[x][h] + kLazy;
            }
        // the sums of a head's group, and what is to come off them, by f
        auto scale_sums = [&](int x, int r, int h, float f) {
#pragma unroll
            for (int c = 2 * r; c < 2 * r + 2; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.at(x, c, e, h) *= f;
            eight[x][r % CH][C::kNarrow ? r : h] *= f;
            eight[x][r % CH][2 + (C::kNarrow ? r : h)] *= f;
        };
        if (__any_sync(kFull, moves)) {
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int h = 0; h < HL; ++h) {
                    const float y = fmaxf(max_rows(top[x][h]), a.m[x][h]);
                    const float by = y == -INFINITY ? 0.f : y - a.m[x][h], old = exp2_of(-by);
                    a.m[x][h] = y;
                    less[x][h] = y == -INFINITY ? 0.f : -y;
                    a.l[x][h] *= old;
#pragma unroll
                    for (int r = 0; r < NG; ++r) {
                        centres[x][r][h] *= old;
                        // the products so far keep their size: the units rise by as much, up to
                        // the next power of two
                        const int at = __float_as_int(wu[x][r][h]);
                        const int up = min((int)ceilf(fminf(by, 300.f)), (__float_as_int(kUnitMost) - at) >> 23);
                        wu[x][r][h] = __int_as_float(at + (up << 23));
                        scale_sums(x, r, h, exp2_of((float)up - by));
                    }
                }
        }

        // the weights, in the logits' place, and their products with V's steps, as columns
        uint32_t pb[SUB][X][CH][PARTS][2];
        auto products = [&](int sub, int x, int u, int r) {
            const float(&w)[HL] = v[x][sub][u];
            const float s0 = E::to_float2(vpair[sub][u][r]).x;
            const float w0 = w[0] * wu[x][r][0] * s0;
            const float w1 = C::kNarrow ? (NG == 2 ? w[0] * wu[x][NG - 1][0] * E::to_float2(vpair[sub][u][NG - 1]).x : 0.f)
                                        : w[HL - 1] * wu[x][r][HL - 1] * s0;
            const uint32_t hi = pkv::F16::from_float2(w0, w1);
            pb[sub][x][r][0][u] = transposed(hi);
            if (PARTS == 2) {  // and what the rounding left
                const float2 back = pkv::F16::to_float2(hi);
                pb[sub][x][r][PARTS - 1][u] = transposed(pkv::F16::from_float2(w0 - back.x, w1 - back.y));
            }
            return *reinterpret_cast<const __half2*>(&hi);
        };
        __half2 most = __float2half2_rn(0.f);
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int h = 0; h < HL; ++h) {
                        float& w = v[x][sub][u][h];
                        w = exp2_of(fmaf(w, qs[x][h], less[x][h]));
                        a.l[x][h] += w;
#pragma unroll
                        for (int r = 0; r < NG; ++r)
                            centres[x][r][h] = fmaf(w, E::to_float2(vpair[sub][u][r]).y, centres[x][r][h]);
                    }
#pragma unroll
                    for (int r = 0; r < CH; ++r) most = __hmax2(most, products(sub, x, u, r));
                }
        const float2 large = __half22float2(most);
        if (__any_sync(kFull, fmaxf(large.x, large.y) >= kProductMost)) {  // new units
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int h = 0; h < HL; ++h)
#pragma unroll
                    for (int r = 0; r < NG; ++r) {
                        float y = 0.f;
#pragma unroll
                        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                y = fmaxf(y, v[x][sub][u][h] * E::to_float2(vpair[sub][u][r]).x);
                        y = max_rows(y);
                        const uint32_t ex = min(max(__float_as_uint(y) & 0x7f800000u, 0x08000000u), 0x7e800000u);
                        const int was = __float_as_int(wu[x][r][h]);
                        const int now = y * wu[x][r][h] >= kProductMost
                                            ? __float_as_int(kUnits * __uint_as_float((254u << 23) - ex)) : was;
                        wu[x][r][h] = __int_as_float(now);
                        scale_sums(x, r, h, __int_as_float(max(now - was + (127 << 23), 0)));  // now / was
                    }
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
                for (int x = 0; x < X; ++x)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < CH; ++r) products(sub, x, u, r);
        }
        const uint32_t minus8[4] = {kMinus8Even, kMinus8Odd, kMinus8Even, kMinus8Odd};
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
#pragma unroll
            for (int r = 0; r < NG; ++r) {
                uint32_t k[4], f[4][4];
                ldsm_x4_trans(k, sv + at[r] + 2 * sub * UB);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t h0[4], h1[4];
                    codes_of(k[2 * c], h0);      // tokens 2 t, 2 t + 1
                    codes_of(k[2 * c + 1], h1);  // and 8 more
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        f[2 * c + e][0] = h0[2 * e];
                        f[2 * c + e][1] = h0[2 * e + 1];
                        f[2 * c + e][2] = h1[2 * e];
                        f[2 * c + e][3] = h1[2 * e + 1];
                    }
                }
#pragma unroll
                for (int x = 0; x < X; ++x)
#pragma unroll
                    for (int y = 0; y < PARTS; ++y) {
                        const uint32_t(&b)[2] = pb[sub][x][r % CH][y];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            pkv::Mma<pkv::F16>::run(a.o[x][2 * r + c / 2][c & 1], f[c], b[0], b[1]);
                        if (r < CH) pkv::Mma<pkv::F16>::run(eight[x][r % CH], minus8, b[0], b[1]);
                    }
            }
        }
      }
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
            for (int c = 0; c < NI; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int h = 0; h < HL; ++h)
                        a.at(x, c, e, h) += eight[x][(c / 2) % CH][2 * (e & 1) + (C::kNarrow ? c / 2 : h)];
        feed.done();
    }
#pragma unroll
    for (int x = 0; x < X; ++x)
#pragma unroll
        for (int h = 0; h < HL; ++h) {
            a.l[x][h] = sum_rows(a.l[x][h]);
#pragma unroll
            for (int r = 0; r < NG; ++r) {
                const float c = sum_rows(centres[x][r][h]), back = 1.f / wu[x][r][h];  // a power of two
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float& o = a.at(x, 2 * r + k, e, h);
                        o = fmaf(o * (e & 1 ? 0x1p20f : 0x1p24f), back, c);
                    }
            }
        }
}

// A warp's part of its unit in shared memory: rows [16][D], m and l.
template <int D>
struct Part {
    float o[kMaxGroup][D];
    float m[kMaxGroup], l[kMaxGroup];
};
static_assert(sizeof(Part<128>) <= kRingBytes<128> && sizeof(Part<64>) <= kRingBytes<64>,
              "a part takes its warp's ring");

template <int D, class C>
__device__ __forceinline__ void put_part(Part<D>* to, int lane, Acc<D, C>& a) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < C::X; ++x)
#pragma unroll
        for (int h = 0; h < C::HL; ++h) {
            const int row = a.head_of(x, t, h);
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                *reinterpret_cast<float4*>(&to->o[row][32 * i + 4 * g]) =
                    make_float4(a.at(x, i, 0, h), a.at(x, i, 1, h), a.at(x, i, 2, h), a.at(x, i, 3, h));
            if (g == 0) {
                to->m[row] = a.m[x][h];
                to->l[row] = a.l[x][h];
            }
        }
}

// The weights 2^(m - M) of a row's parts from the warps w0, w0 + step, ... of a
// CTA's N, its M and L.
template <int D, int N>
__device__ __forceinline__ float row_weights(const char* smem, int w0, int step, int row, float (&w)[N], float& L) {
    float l[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool in = w0 + i * step < N;
        const Part<D>* part = reinterpret_cast<const Part<D>*>(smem + (in ? w0 + i * step : w0) * kRingBytes<D>);
        w[i] = in ? part->m[row] : -INFINITY;
        l[i] = in ? part->l[row] : 0.f;
    }
    float M = w[0];
#pragma unroll
    for (int i = 1; i < N; ++i) M = fmaxf(M, w[i]);
    const float use = M == -INFINITY ? 0.f : M;
    L = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w[i] = exp2f(w[i] - use);
        L = fmaf(w[i], l[i], L);
    }
    return M;
}

// Four dims of a row out of those parts.
template <int D, int N>
__device__ __forceinline__ float4 row_sum(const char* smem, int w0, int step, int row, int d, const float (&w)[N]) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (w0 + i * step < N) {
            const Part<D>* part = reinterpret_cast<const Part<D>*>(smem + (w0 + i * step) * kRingBytes<D>);
            const float4 v = *reinterpret_cast<const float4*>(&part->o[row][d]);
            sum.x = fmaf(w[i], v.x, sum.x);
            sum.y = fmaf(w[i], v.y, sum.y);
            sum.z = fmaf(w[i], v.z, sum.z);
            sum.w = fmaf(w[i], v.w, sum.w);
        }
    return sum;
}

// Joins the token splits of each head (split): split 0's warp ends up with the
// whole.
template <int D, class C>
__device__ __forceinline__ void join_splits(const Params& p, char* smem, int warp, int lane, Acc<D, C>& a) {
    const int g = lane >> 2, t = lane & 3;
    __syncwarp();
    put_part<D, C>(reinterpret_cast<Part<D>*>(smem + warp * kRingBytes<D>), lane, a);
    __syncthreads();
    if (warp < p.hw) {
#pragma unroll
        for (int x = 0; x < C::X; ++x)
#pragma unroll
            for (int h = 0; h < C::HL; ++h) {
                const int row = a.head_of(x, t, h);
                float w[kWarps], L;
                a.m[x][h] = row_weights<D, kWarps>(smem, warp, p.hw, row, w, L);
                a.l[x][h] = L;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const float4 v = row_sum<D, kWarps>(smem, warp, p.hw, row, 32 * i + 4 * g, w);
                    a.at(x, i, 0, h) = v.x;
                    a.at(x, i, 1, h) = v.y;
                    a.at(x, i, 2, h) = v.z;
                    a.at(x, i, 3, h) = v.w;
                }
            }
    }
    // the rings are filled again, by the asynchronous copies, after this
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
}

template <class E>
__device__ __forceinline__ uint2 pack4(const float4& v, float f) {
    return make_uint2(E::from_float2(v.x * f, v.y * f), E::from_float2(v.z * f, v.w * f));
}

// What the CTAs of a cluster send one another: 32 dims of a row ("segment") of
// every CTA to the CTA that joins it, and every row's M and L to all.  Behind the
// rings, and only in calls with clusters: those have one CTA per SM, or few, and the
// others would lose one to it (8 query heads per KV head, 256 units of 4096 tokens, one
// CTA of six warps per SM and two: 48.8 and 35.8 us).
template <int D, class C>
struct ClusterIn {
    static constexpr int ROWS = C::kNarrow ? 4 : 8 * C::X, SEGS = ROWS * (D / 32);
    // [segment / CS][CTA][32]; the last CTAs of a cluster may have one segment less
    float o[SEGS + kMaxCluster - 1][32];
    float m[kMaxCluster][ROWS], l[kMaxCluster][ROWS];
};

// CTAs of a direct call's W warps that an SM takes, without clusters
template <int D, class C, int W>
constexpr int kDirectCtas = W == kWarps ? kCtas<D, C> : W == kManyWarps<D, C> ? 2 : 1;
constexpr int kSmemPerSm = 228 * 1024, kSmemReserved = 1024;  // the system's, per CTA

// Direct: cluster c / cs takes unit c / cs (hw = 1), its CTAs equal parts of
// the unit's tiles, their W warps a stage each in turn.
template <class E, int D, class C, int W>
__global__ void __launch_bounds__(32 * W, kDirectCtas<D, C, W>) direct_kernel(const __grid_constant__ Params p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int SEGS = D / 32;
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(8) unsigned long long full[W][kStages<D>];
    __shared__ int abort;
    static_assert(kDirectCtas<D, C, W> * (W * kRingBytes<D> + sizeof full + sizeof abort + kSmemReserved) <= kSmemPerSm,
                  "the CTAs that the registers are for");
    ClusterIn<D, C>& in = *reinterpret_cast<ClusterIn<D, C>*>(smem + W * kRingBytes<D>);  // cs > 1
    if (p.cs > 1) cluster_arrive();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) abort = 0;
    __syncthreads();
    const int unit = blockIdx.x / p.cs, rank = blockIdx.x % p.cs;
    const int s = unit / p.Hkv, kvh = unit % p.Hkv;
    const int raw = __ldg(p.context_lens + s);
    if ((raw < 0 || raw > p.max_ctx) && kvh == 0 && rank == 0 && tid == 0) pkv::report(p.err, PKV_DEVERR_CONTEXT);
    const int n = context_of(p, s);
    const int T = tiles_of(p, n), per = (T + p.cs - 1) / p.cs;
    const int tb = min(T, rank * per), te = min(T, tb + per);

    const int first = tb + warp;
    Feed<D> feed(p, nullptr, &abort, smem_of(smem) + warp * kRingBytes<D>, smem_of(&full[warp][0]), warp, lane, 0, W);
    Acc<D, C> a;
    feed.begin(s, kvh, n, first, te, 0);
    attend<E, D, C>(p, feed, s, kvh, first, te, lane, a);
    __syncwarp();
    put_part<D, C>(reinterpret_cast<Part<D>*>(smem + warp * kRingBytes<D>), lane, a);
    __syncthreads();
    uint16_t* out = static_cast<uint16_t*>(p.out) + ((int64_t)s * p.H + (int64_t)kvh * p.G) * D;
    if (p.cs == 1) {
        for (int k = tid; k < p.G * (D / 4); k += 32 * W) {
            const int row = k / (D / 4), d = k % (D / 4) * 4;
            float w[W], L;
            row_weights<D, W>(smem, 0, 1, row, w, L);
            *reinterpret_cast<uint2*>(out + row * D + d) = pack4<E>(row_sum<D, W>(smem, 0, 1, row, d, w), inverse_of(L));
        }
        return;
    }
    // every CTA sends its rows to the CTAs that join them, segment i to CTA i % CS
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks();
    cluster_wait();  // all CTAs run
    for (int seg = warp; seg < p.G * SEGS; seg += W) {
        const int row = seg / SEGS, d = seg % SEGS * 32 + lane;
        float w[W], L, sum = 0.f;
        const float M = row_weights<D, W>(smem, 0, 1, row, w, L);
#pragma unroll
        for (int i = 0; i < W; ++i)
            sum = fmaf(w[i], reinterpret_cast<const Part<D>*>(smem + i * kRingBytes<D>)->o[row][d], sum);
        cluster.map_shared_rank(&in.o[0][0], seg % CS)[(seg / CS * CS + rank) * 32 + lane] = sum;
        if (seg % SEGS == 0 && lane < CS) {
            cluster.map_shared_rank(&in.m[rank][0], lane)[row] = M;
            cluster.map_shared_rank(&in.l[rank][0], lane)[row] = L;
        }
    }
    cluster_arrive();
    cluster_wait();
    for (int k = warp; k * CS + rank < p.G * SEGS; k += W) {
        const int seg = k * CS + rank, row = seg / SEGS;
        const float m = lane < CS ? in.m[lane][row] : -INFINITY;
        float M = m;
#pragma unroll
        for (int x = kMaxCluster / 2; x >= 1; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, x));
        M = __shfl_sync(kFull, M, 0);
        const float w = lane < CS ? exp2f(m - (M == -INFINITY ? 0.f : M)) : 0.f;
        float L = lane < CS ? w * in.l[lane][row] : 0.f;
#pragma unroll
        for (int x = kMaxCluster / 2; x >= 1; x >>= 1) L += __shfl_xor_sync(kFull, L, x);
        const float inv = inverse_of(__shfl_sync(kFull, L, 0));
        float o = 0.f;
        for (int i = 0; i < CS; ++i) o = fmaf(__shfl_sync(kFull, w, i), in.o[k * CS + i][lane], o);
        o *= inv;
        const float next = __shfl_down_sync(kFull, o, 1);
        if ((lane & 1) == 0)
            *reinterpret_cast<uint32_t*>(out + row * D + seg % SEGS * 32 + lane) = E::from_float2(o, next);
    }
}

// Split: range c = blockIdx.x, then whichever ranges this CTA can take.
template <class E, int D, class C>
__global__ void __launch_bounds__(kThreads, kCtas<D, C>) split_kernel(const __grid_constant__ Params p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ __align__(128) char smem[];
    __shared__ Plan plan;
    __shared__ __align__(8) unsigned long long full[kWarps][kStages<D>];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int hl = warp % p.hw, split = warp / p.hw;
    make_plan(p, plan, tid);

    Feed<D> feed(p, &plan, &plan.abort, smem_of(smem) + warp * kRingBytes<D>, smem_of(&full[warp][0]), warp, lane, hl,
                 p.nsplit);
    Range r = range_at(p, plan.before, plan.map, plan.map.of_cta(blockIdx.x), lane);
    bool running = r.left > 0;  // the same for all warps of the CTA
    if (running && feed.chained)
        feed.begin(r.s, r.hb, r.n, r.tb, min(tiles_of(p, r.n), r.tb + r.left), r.left + r.tb);
    int used = 0;  // ranges taken out of the queue
    while (running) {
        // one unit (or the part of it that lies in this range)
        const int T = tiles_of(p, r.n);
        const int te = min(T, r.tb + r.left);
        const int kvh = r.hb * p.hw + hl;
        const bool last = te - r.tb == r.left;  // of the range
        Acc<D, C> a;
        const int first = r.tb + split;
        if (!feed.chained) feed.begin(r.s, r.hb, r.n, first, te, 0);
        attend<E, D, C>(p, feed, r.s, kvh, first, te, lane, a);
        if (!feed.chained) join_splits<D, C>(p, smem, warp, lane, a);
        const bool whole = r.tb == 0 && te == T;
        if (split == 0) {
            // finished rows, or a piece
            const int64_t piece = ((2 * (int64_t)r.c + (r.tb == 0 ? 1 : 0)) * p.hw + hl) * p.G;
            const int64_t oh = (int64_t)r.s * p.H + (int64_t)kvh * p.G;
#pragma unroll
            for (int x = 0; x < C::X; ++x)
#pragma unroll
                for (int h = 0; h < C::HL; ++h) {
                    const int row = a.head_of(x, t, h);
                    if (row >= p.G) continue;
                    const float inv = inverse_of(a.l[x][h]);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const float4 v = make_float4(a.at(x, i, 0, h), a.at(x, i, 1, h), a.at(x, i, 2, h), a.at(x, i, 3, h));
                        const int d = 32 * i + 4 * g;
                        if (whole)
                            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (oh + row) * D + d) = pack4<E>(v, inv);
                        else
                            *reinterpret_cast<float4*>(p.part_acc + (piece + row) * D + d) = v;
                    }
                    if (!whole && g == 0) {
                        p.part_m[piece + row] = a.m[x][h];
                        p.part_l[piece + row] = a.l[x][h];
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
}

// After split_kernel: the rows of units that lie in several ranges, a warp per
// row, or (`many`: units of many pieces) the warps of a CTA.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinCtasPerSm = 5;

template <class E, int D>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtasPerSm) join_kernel(const __grid_constant__ Params p, int many) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int DPL = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.hw * p.G, joins = p.S * p.HB * rows;  // = S * H
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    __shared__ __align__(16) float s_o[kJoinWarps][D];
    const int first = many ? blockIdx.x : blockIdx.x + warp * gridDim.x;  // neighbouring rows go to different SMs
    const int step = many ? gridDim.x : kJoinWarps * gridDim.x;
    for (int i = first; i < joins; i += step) {
        const int unit = i / rows;
        const int2 at = p.place[unit];
        if (pkv::pieces_of(at.x, at.y, p.ranges) < 2) continue;  // many: the same for the whole CTA
        float M, L, o[DPL];
        if (many) {
            gather_row<D, 6>(p, at.x, at.x + warp, at.y, kJoinWarps, i % rows, lane, M, L, o);
            if (lane == 0) {
                s_m[warp] = M;
                s_l[warp] = L;
            }
#pragma unroll
            for (int j = 0; j < DPL; ++j) s_o[warp][lane * DPL + j] = o[j];
            __syncthreads();
            if (warp == 0)
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
        } else {
            gather_row<D, 2>(p, at.x, at.x, at.y, 1, i % rows, lane, M, L, o);
        }
        if (!many || warp == 0) {
            const float inv = inverse_of(L);
            const int64_t oh = (int64_t)(unit / p.HB) * p.H + (int64_t)(unit % p.HB) * rows + i % rows;
            uint16_t* dst = static_cast<uint16_t*>(p.out) + oh * D + lane * DPL;
#pragma unroll
            for (int j = 0; j < DPL; j += 2)
                *reinterpret_cast<uint32_t*>(dst + j) = E::from_float2(o[j] * inv, o[j + 1] * inv);
        }
        if (many) __syncthreads();  // the parts have been read
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Direct calls.  Measured, us, 32 query heads on 8, D = 128 (with CTAs that fill an
// SM, that fill half of one, split):
//   1 context of 4096 7.0, 7.0, 12.3; of 32768 14.5, 18.4, 21.6; of 65536 23.4, 32.1,
//   25.4; of 100000 32.4, 46.5, 35.8 (131072: split 37)
//   4 of 8192 12.2, 12.5, 21.2; of 32768 32.7, 34.0, 37.1;  8 of 16384 32.6, 33.9, 38.1
//   16 of 1024 7.6, 8.0, 16.7; of 4096 17.4, 19.3, 26.1;  19 of 4096 18.2, 19.9, 28.9
//   32 (two units per SM) of 1024 -, 11.0, 21.2; of 4096 -, 33, 38
//   and with 64 query heads: 32 of 1024 -, 13.4, 23.9; of 4096 -, 37.8, 44.4; D = 64: 32 of
//   1024 -, 9.0, 22.3; of 5600 -, 30.9, 44.2
// and with four warps (split beside them): 32 of 1024 13.9, of 4096 44; 64 of 128..2048
// 26.9 (28.5); 100 of 1..500 14.0 (17.8); 220 of 1..1000 38.2 (43.5), with 64 query heads
// 45.4 (52.3); 256 of 1..200 20.9 (22.5).
// A cluster of 16 CTAs that fill an SM each finds room 7 times, of 12 8 times: eight
// units are better off with 12 (32768 tokens: 14.5 us; with 16 23.4, in two waves).
constexpr int kDirectTokens = 1024;  // the longest context that four warps take
constexpr int kDirectWaves = 4;      // of their CTAs
constexpr int kManyTokens = 704;     // per warp of the larger CTAs

struct Layout {
    size_t place, m, l, acc, total;
};

Layout layout_of(int S, int H, int Hkv, int D) {
    const size_t rows = (size_t)2 * kMaxRanges * heads_per_cta(Hkv) * (H / Hkv);
    Layout L;
    size_t o = 0;
    L.place = o; o = align256(o + (size_t)S * Hkv * sizeof(int2));
    L.m = o;     o = align256(o + rows * sizeof(float));
    L.l = o;     o = align256(o + rows * sizeof(float));
    L.acc = o;   o = align256(o + rows * D * sizeof(float));
    L.total = o;
    return L;
}

// A kernel, its warps, the shared memory of their rings, and what a cluster adds.
struct Pick {
    KernelFn fn;
    int warps, rings, more;
    int smem(int cs) const { return rings + (cs > 1 ? more : 0); }
};
// Its CTAs that an SM takes, in clusters of cs.
int resident_of(const Pick& use, int cs) {
    return resident_of(use.fn, use.smem(cs), 32 * use.warps, use.rings + use.more);
}
enum Kind { kSplit, kDirect, kDirectMany, kDirectWhole };
// Clusters of cs of its CTAs that run at once (once per kernel, size and device).
int clusters_of(const Pick& use, int cs) {
    static std::mutex mu;
    static struct { KernelFn fn; int dev, cs, n; } cache[256];
    static int used = 0;
    int dev = 0;
    if (resident_of(use, cs) < 1 || cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < used; ++i)
        if (cache[i].fn == use.fn && cache[i].dev == dev && cache[i].cs == cs) return cache[i].n;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cs;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cs);
    cfg.blockDim = dim3(32 * use.warps);
    cfg.dynamicSmemBytes = use.smem(cs);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, use.fn, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (used < 256) cache[used++] = {use.fn, dev, cs, n};
    return n;
}
template <class E, int D, class C>
Pick pick(Kind kind) {
    constexpr int ring = kRingBytes<D>, more = sizeof(ClusterIn<D, C>);
    if constexpr (C::kNarrow && C::PASS < kTile) return {direct_kernel<E, D, C, kWarps>, kWarps, kWarps * ring, more};
    else {
        constexpr int many = kManyWarps<D, C>;
        if (kind == kDirectMany) return {direct_kernel<E, D, C, many>, many, many * ring, more};
        if (kind == kDirectWhole) return {direct_kernel<E, D, C, 2 * many>, 2 * many, 2 * many * ring, more};
        if (kind == kSplit) return {split_kernel<E, D, C>, kWarps, kWarps * ring, 0};
        return {direct_kernel<E, D, C, kWarps>, kWarps, kWarps * ring, more};
    }
}
template <class E, int D>
Pick pick(Kind kind, int G, bool brief) {
    if (G <= 4) return brief ? pick<E, D, Narrow<32>>(kDirect) : pick<E, D, Narrow<64>>(kind);
    return G <= 8 ? pick<E, D, Heads<1>>(kind) : pick<E, D, Heads<2>>(kind);
}
// brief: direct, tiles of 32
Pick pick(pkv_dtype dtype, int D, Kind kind, int G, bool brief = false) {
    if (dtype == PKV_F16) return D == 128 ? pick<pkv::F16, 128>(kind, G, brief) : pick<pkv::F16, 64>(kind, G, brief);
    return D == 128 ? pick<pkv::BF16, 128>(kind, G, brief) : pick<pkv::BF16, 64>(kind, G, brief);
}
void (*pick_join(pkv_dtype dtype, int D))(Params, int) {
    if (dtype == PKV_F16) return D == 128 ? join_kernel<pkv::F16, 128> : join_kernel<pkv::F16, 64>;
    return D == 128 ? join_kernel<pkv::BF16, 128> : join_kernel<pkv::BF16, 64>;
}

bool workspace_args_ok(int S, int H, int Hkv, int D) {
    return S >= 0 && H > 0 && Hkv > 0 && H % Hkv == 0 && H / Hkv <= kMaxGroup && (D == 64 || D == 128);
}

}  // namespace

extern "C" {

size_t pkv_decode_q4_workspace_size(int S, int H, int Hkv, int D) {
    if (!workspace_args_ok(S, H, Hkv, D)) return 0;
    return layout_of(S, H, Hkv, D).total;
}

pkv_status pkv_paged_attention_decode_q4(void* out, const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* block_tables, const int32_t* context_lens, int S, int H,
                                         int Hkv, int D, int bs, int NB, int MB, int max_context_len, float scale,
                                         pkv_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    PKV_TRACE("pkv_paged_attention_decode_q4");
    pkv::clear_error();
    auto bad = [](pkv_status st, const char* what) {
        char msg[256];
        snprintf(msg, sizeof msg, "paged_attention_decode_q4: %s", what);
        return pkv::fail(st, msg);
    };
    if (S < 0 || H <= 0 || Hkv <= 0 || NB <= 0 || MB <= 0 || (dtype != PKV_F16 && dtype != PKV_BF16))
        return bad(PKV_ERR_INVALID_ARG, "bad size or dtype");
    if ((D != 64 && D != 128) || (bs != 8 && bs != 16 && bs != 32 && bs != 64))
        return bad(PKV_ERR_UNSUPPORTED, "head_dim must be 64/128, block_size 8/16/32/64");
    if (H % Hkv != 0) return bad(PKV_ERR_INVALID_ARG, "H must be a multiple of Hkv");
    if (H / Hkv > kMaxGroup) return bad(PKV_ERR_UNSUPPORTED, "at most 16 query heads per KV head");
    if (!(scale == scale) || std::isinf(scale)) return bad(PKV_ERR_INVALID_ARG, "scale must be finite");
    if ((int64_t)NB * bs > INT32_MAX) return bad(PKV_ERR_INVALID_ARG, "NB * bs must fit 31 bits");
    if ((int64_t)NB * bs / q4::kUnit * Hkv > INT32_MAX)
        return bad(PKV_ERR_INVALID_ARG, "NB * bs * Hkv must fit 34 bits");
    if (S > 32767 || (int64_t)S * H > INT32_MAX / kMaxCluster)
        return bad(PKV_ERR_INVALID_ARG, "at most 32767 sequences, and 2^27 heads in all of them");
    const int64_t cap = (int64_t)MB * bs;
    const int64_t max_ctx = max_context_len == 0 ? (cap < kMaxContext ? cap : kMaxContext) : max_context_len;
    if (max_ctx < 0 || max_ctx > cap || max_ctx > kMaxContext)
        return bad(PKV_ERR_INVALID_ARG, "max_context_len must be in [0, MB*bs], below 2^31 - 1024");
    if (S == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
        return bad(PKV_ERR_INVALID_ARG, "null pointer");
    if (!pkv::aligned16(out) || !pkv::aligned16(q) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache))
        return bad(PKV_ERR_INVALID_ARG, "token and cache pointers must be 16-byte aligned");
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return bad(PKV_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
    const Layout L = layout_of(S, H, Hkv, D);
    if (workspace_bytes < L.total) return bad(PKV_ERR_WORKSPACE, "workspace too small");

    Params p = {};
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
    p.window = INT32_MAX;  // every token is visible
    p.sinks = 0;
    p.qscale = scale * kLog2e;
    char* w = static_cast<char*>(workspace);
    p.place = reinterpret_cast<int2*>(w + L.place);
    p.part_m = reinterpret_cast<float*>(w + L.m);
    p.part_l = reinterpret_cast<float*>(w + L.l);
    p.part_acc = reinterpret_cast<float*>(w + L.acc);
    p.err = pkv::device_error_word();
    const int sms = pkv::sm_count();
    const int64_t units = (int64_t)S * Hkv;
    // Few units, of more than a few tiles: CTAs that fill an SM, or, for up to two units
    // per SM, half of one, unless their warps' shares would be longer than kManyTokens.
    // Clusters grow while every fourth of their warps has a tile (1100 tokens: 7.5 us
    // where each has one, 6.1) and all run at once.
    Pick use = pick(dtype, D, units <= sms ? kDirectWhole : kDirectMany, p.G);
    bool direct = units <= 2 * sms && max_ctx >= kDirectTokens;
    p.tile_log2 = 6;
    p.cs = 1;
    for (int cs : {2, 4, 8, 12, 16})
        if (direct && units * cs <= sms && max_ctx > (int64_t)use.warps * (kTile / 4) * p.cs &&
            clusters_of(use, cs) >= units)
            p.cs = cs;
    direct = direct && max_ctx <= (int64_t)kManyTokens * use.warps * p.cs;
    if (!direct) {
        // Short contexts: a CTA of four warps per unit, or, while they fit the card at
        // once, clusters with a tile per warp.
        const bool brief = max_ctx <= kWarps * kTile;
        use = pick(dtype, D, kDirect, p.G, brief);
        p.tile_log2 = brief ? 5 : 6;
        p.cs = 1;
        direct = max_ctx <= kDirectTokens && units <= (int64_t)kDirectWaves * resident_of(use, 1) * sms;
        const int64_t slots = (int64_t)resident_of(use, 2) * sms;
        while (direct && p.cs < kMaxCluster && units * p.cs * 2 <= slots && max_ctx > (int64_t)kWarps * kTile * p.cs)
            p.cs *= 2;
    }
    if (!direct) {
        use = pick(dtype, D, kSplit, p.G);
        p.tile_log2 = 6;
    }
    const int per_sm = resident_of(use, p.cs);
    if (per_sm < 1) return bad(PKV_ERR_CUDA, "the kernel cannot be resident");
    p.hw = direct ? 1 : heads_per_cta(Hkv);
    while (!direct && p.hw > 1 && (int64_t)S * Hkv / p.hw < kMinUnits) p.hw /= 2;
    p.nsplit = kWarps / p.hw;
    p.HB = Hkv / p.hw;
    p.ranges0 = per_sm * sms;
    if (p.ranges0 > kMaxRanges / (1 + kSmallRanges)) p.ranges0 = kMaxRanges / (1 + kSmallRanges);
    const int64_t most_tiles = (int64_t)S * p.HB * ((max_ctx + kTile - 1) / kTile);
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
    cfg.blockDim = dim3(32 * use.warps);
    cfg.dynamicSmemBytes = use.smem(p.cs);
    cfg.stream = pkv::as_stream(stream);
    cfg.attrs = attr;
    cfg.numAttrs = direct && p.cs > 1 ? 2 : 1;
    cfg.gridDim = dim3(direct ? (unsigned)(S * Hkv * p.cs) : (unsigned)p.ranges);
    cudaError_t e = cudaLaunchKernelEx(&cfg, use.fn, p);
    if (e == cudaSuccess && !direct) {
        const int many = p.ranges > 8 * (int64_t)S * p.HB;  // units of more than 8 pieces
        cfg.dynamicSmemBytes = 0;
        cfg.numAttrs = 1;
        cfg.blockDim = dim3(kJoinThreads);
        // one wave, of no more CTAs than there are rows for
        const int64_t ctas = many ? (int64_t)S * H : ((int64_t)S * H + kJoinWarps - 1) / kJoinWarps;
        cfg.gridDim = dim3((unsigned)(ctas < kJoinCtasPerSm * sms ? ctas : kJoinCtasPerSm * sms));
        e = cudaLaunchKernelEx(&cfg, pick_join(dtype, D), p, many);
    }
    return e == cudaSuccess ? PKV_OK : pkv::cuda_fail(e, "paged_attention_decode_q4 launch");
}

}  // extern "C"
