// Eviction from a paged cache by accumulated attention weight.
//
// For every (sequence s, KV head h) with n = context_lens[s] > budget:
//   pos_j  = positions[j] if stored (>= 0), else N - n + j, N = token_counts[s]
//   safe_j = pos_j < sinks or pos_j >= N - recent
//   keep the `budget` best tokens by (safe, score, lowest j)
// and close the gaps: the kept tokens at or past the budget ("movers",
// ascending) go into the evicted places below it ("holes", ascending).  Movers
// lie at >= budget and holes below, so no move overwrites what another reads:
// the moves run in any order, need no second buffer, and repeating the call
// with the same inputs writes the same bytes.  Only the moved rows are copied;
// an order-preserving compaction would copy nearly every kept row each time.
//
// Selection: scores become 32-bit keys that order as the scores do (safe =
// all ones, NaN as -inf, -0 as +0), held in shared memory; histograms of
// one digit after the other find the budget-th key (the last digits are
// skipped when a bin stays as a whole), and ties are kept from the lowest index by counting.
// All counts are integers: the result does not depend on the order of the
// atomics.
//
// One cluster of 1..8 CTAs per (s, h): each CTA holds a stretch of the row,
// histograms are summed through distributed shared memory, so few long rows
// spread over the card.
//
// Bound by memory where tokens move: 8 bytes read and written per token, and
// per move 2 x 256 bytes (D = 128) read and written, one head of one token row at
// a time.  Measured on GB300 (device time, share of the copy rate of 6776 GB/s):
//   256 requests of 16..4096 (median 512) to 500, 32 heads    220 us  83 %
//   8 x 32768 to 4096, 32 heads                               210 us  78 %
//   64 requests of 2064 to 2048, 8 heads: 16 moves a row     10.4 us  36 %
//   4 requests of 50..100 to 48, 4 heads of 64                4.9 us
// The last two are the chain length -> keys -> histogram -> counts -> lists ->
// rows, about a microsecond a link; in the steady state two or three of its sweeps of
// the row find nothing that the few keys in the first digit's bin do not say.  In the
// first, DRAM moves 1217 MB at 70 % of its peak, reads and writes of 256 bytes in
// turn.
#include <cooperative_groups.h>

#include <climits>
#include <cstdio>
#include <mutex>

#include "pagedkv.h"
#include "pkv_device.cuh"

namespace cg = cooperative_groups;

namespace {

// Threads of a CTA: 256, or
// 128 for short rows, longer ones where the rows do not all fit the card at
// once: 512 rows of 65..130 tokens 5.8 us (256 threads 6.2), 2048 8.2 (12.1), 3472
// of 303 31.7 (40.0); but 128 rows of 130..260 6.5 (6.0);
constexpr int kSmallKeys = 160;
constexpr int kSmallKeysWaiting = 320;
// 512 where there is room for it and a CTA may have this many moves: 128 rows of
// 500..1000 to 500 10.1 us (256 threads 15.7); but 128 of 484..500 to 484 5.4 (4.8).
constexpr int kManyMoves = 256;
constexpr int kMaxCluster = 8;
constexpr int kFewKeys = 2048;        // a row of fewer is one CTA's
// A row of more keys is several CTAs': 8 x 32768 to 4096, 32 heads: 213 us with
// 4096 keys per CTA, 232 with 8192; with 16384, 334: a second wave for a few rows.
constexpr int kManyKeys = 4096;
constexpr int kSmemKeys = 48 * 1024;  // keys a CTA can hold: 192 KB
constexpr int kChunk = 128;           // keys a warp takes at once, 4 per lane
constexpr unsigned kFull = 0xffffffffu;

struct Params {
    uint4* k_cache;
    uint4* v_cache;
    const float* scores;
    const int32_t* positions;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* token_counts;
    float* scores_out;
    int32_t* positions_out;
    int32_t* new_lens;
    int Hkv, NB, MB, bs_log2, max_ctx;
    int64_t stride;       // of the score and position rows
    int budget, recent, sinks;
    int seg_cap;          // keys the shared memory holds
    int vec;              // the score and position rows start on 16 bytes
    int32_t* holes;       // [S * Hkv][budget]
    int32_t* movers;      // [S * Hkv][budget]
    int* err;
};

__device__ __forceinline__ uint32_t key_of(float score, bool safe) {
    if (safe) return 0xffffffffu;
    if (score != score) return 0x007fffffu;          // as -inf
    const uint32_t u = __float_as_uint(score + 0.f);  // -0 + 0 = +0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// How many tokens of a stretch lie below the budget / past it and have a key
// above / equal to the threshold.
struct Counts {
    int gt_front, gt_back, eq_front, eq_back;
};
__device__ __forceinline__ Counts operator+(const Counts& x, const Counts& y) {
    return {x.gt_front + y.gt_front, x.gt_back + y.gt_back, x.eq_front + y.eq_front,
            x.eq_back + y.eq_back};
}

// Four consecutive entries, of which the first `count` exist (the others are
// `none`): one 16-byte load where the row allows it.
template <class T>
__device__ __forceinline__ void load4(const T* p, int count, bool vec, T none, T (&v)[4]) {
    if (vec && count >= 4) {
        const int4 x = *reinterpret_cast<const int4*>(p);
        const int w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const T*>(&w[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = e < count ? p[e] : none;
    }
}
template <class T>
__device__ __forceinline__ void store4(T* p, int count, bool vec, const T (&v)[4]) {
    if (vec && count >= 4) {
        int w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const int*>(&v[e]);
        *reinterpret_cast<int4*>(p) = make_int4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < count) p[e] = v[e];
    }
}

// kMinCtas: CTAs per SM the registers allow, of 256 threads four or five.  Five
// (48 registers) where rows wait for a place on the card: more of the moves are in
// flight (256 mixed requests: 219 us, with four 236).  Four (64) where all rows
// have one: a row is done sooner (64 requests in steady state: 12.0 us, with five
// 13.9).
template <int D, bool kCluster, int kThreads, int kMinCtas>
__global__ void __launch_bounds__(kThreads, kMinCtas) evict_kernel(Params p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ __align__(16) uint32_t s_keys[];
    constexpr int kWarps = kThreads / 32;
    // digits of 11 bits, or of 8 in a cluster, where every CTA reads every
    // histogram, and for a few keys, which a second digit mostly tells apart
    constexpr int BITS = kCluster || kThreads < 256 ? 8 : 11, PASSES = (31 + BITS) / BITS;
    constexpr int BINS = 1 << BITS, BPT = BINS > kThreads ? BINS / kThreads : 1;  // bins per thread
    __shared__ __align__(16) int s_hist[2][BINS];
    __shared__ int s_sum[kWarps];
    __shared__ int s_pick[3];
    __shared__ Counts s_warp[kWarps];
    __shared__ Counts s_cta;         // of this CTA's stretch, read by the cluster
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = kCluster ? (int)cluster.num_blocks() : 1;
    const int rank = kCluster ? (int)cluster.block_rank() : 0;
    auto sync_row = [&] {  // all the row's CTAs
        if constexpr (kCluster) cluster.sync(); else __syncthreads();
    };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool has_bins = BPT * kThreads == BINS || tid < BINS;
    const int row = blockIdx.x / CS;
    const int s = row / p.Hkv, h = row % p.Hkv;

    const int raw = __ldg(p.context_lens + s);
    int N = __ldg(p.token_counts + s);
    auto clear = [&](int which) {
#pragma unroll
        for (int i = 0; i < BPT; ++i)
            if (has_bins) s_hist[which][i * kThreads + tid] = 0;
    };
    clear(0);
    clear(1);
    const int n = raw < 0 ? 0 : (raw > p.max_ctx ? p.max_ctx : raw);
    if (rank == 0 && h == 0 && tid == 0) {
        if (raw != n || N < n) pkv::report(p.err, PKV_DEVERR_CONTEXT);
        p.new_lens[s] = min(n, p.budget);
    }
    if (N < n) N = n;
    const float* score = p.scores + (int64_t)row * p.stride;
    const int32_t* stored = p.positions + (int64_t)row * p.stride;
    float* score_out = p.scores_out + (int64_t)row * p.stride;
    int32_t* pos_out = p.positions_out + (int64_t)row * p.stride;
    const bool moved_out = score_out != score;     // results go to other arrays
    const bool moved_pos = pos_out != stored;
    const bool vec = p.vec;
    const int b = p.budget;

    if (n <= b) {  // the same in every CTA of the row
        if (!moved_out && !moved_pos) return;
        for (int j = 4 * (rank * kThreads + tid); j < n; j += 4 * CS * kThreads) {
            float sc[4];
            int q[4];
            load4(score + j, n - j, vec, 0.f, sc);
            load4(stored + j, n - j, vec, 0, q);
            if (moved_out) store4(score_out + j, n - j, vec, sc);
            if (moved_pos) store4(pos_out + j, n - j, vec, q);
        }
        return;
    }

    // this CTA's stretch [j0, j1) of the row
    const int seg = ((n + CS - 1) / CS + kChunk - 1) / kChunk * kChunk;
    const int j0 = min(n, rank * seg), j1 = min(n, j0 + seg);
    const bool in_smem = seg <= p.seg_cap;
    // safe: below the sinks, or not below N - recent
    const unsigned unsafe = max(0, N - p.recent - p.sinks);
    auto make_key = [&](float sc, int stored_pos, int j) -> uint32_t {
        const int q = stored_pos >= 0 ? stored_pos : N - n + j;
        return key_of(sc, (unsigned)(q - p.sinks) >= unsafe);
    };
    // keys of tokens j .. j + 3 (j a multiple of 4 from j0 on, below j1)
    auto keys4 = [&](int j, uint32_t (&k)[4]) {
        if (in_smem) {
            const uint4 x = *reinterpret_cast<const uint4*>(s_keys + (j - j0));
            k[0] = x.x; k[1] = x.y; k[2] = x.z; k[3] = x.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) k[e] = j + e < j1 ? make_key(score[j + e], stored[j + e], j + e) : 0u;
        }
    };
    __syncthreads();  // the histograms are empty

    // First pass over the row: keys, their first digit, and what does not
    // wait for the selection.  Entries below the budget keep their place
    // unless a mover comes (written later, over this); entries past it end as
    // 0 and -1, here where that is another array than the one movers are read
    // from.
    constexpr int U = 2;  // rounds of loads in flight
    for (int base = j0 + 4 * tid; base < j1; base += 4 * U * kThreads) {
        float sc[U][4];
        int q[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = base + 4 * u * kThreads;
            load4(score + j, j1 - j, vec, 0.f, sc[u]);
            load4(stored + j, j1 - j, vec, 0, q[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = base + 4 * u * kThreads, count = j1 - j;
            if (count <= 0) break;
            uint32_t k[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                k[e] = make_key(sc[u][e], q[u][e], j + e);
                if (e < count) atomicAdd(&s_hist[0][k[e] >> (32 - BITS)], 1);
            }
            if (in_smem) *reinterpret_cast<uint4*>(s_keys + (j - j0)) = make_uint4(k[0], k[1], k[2], k[3]);
            bool fresh = false;  // a position that was not stored yet
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                fresh |= q[u][e] < 0;
                if (j + e < b) {
                    q[u][e] = q[u][e] >= 0 ? q[u][e] : N - n + j + e;
                } else {
                    sc[u][e] = 0.f;
                    q[u][e] = -1;
                }
            }
            if (moved_out) store4(score_out + j, count, vec, sc[u]);
            if (moved_pos) store4(pos_out + j, count, vec, q[u]);
            else if (fresh && j < b) store4(pos_out + j, min(count, b - j), vec, q[u]);
        }
    }

    // the budget-th largest key T, digit by digit from the top; two histograms
    // in turn
    uint32_t T = 0;
    int want = b;        // rank still to find among the keys with the digits so far
    int drop = 32 - BITS;  // bits below the digits so far
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
        sync_row();
        // counts of the keys in higher bins: BPT bins per thread, warps, block
        int c[BPT], sum = 0;
#pragma unroll
        for (int i = 0; i < BPT; ++i) c[i] = 0;
        for (int r = 0; has_bins && r < CS; ++r) {
            const int* hist = &s_hist[pass & 1][BPT * tid];
            if constexpr (kCluster) hist = cluster.map_shared_rank(hist, r);
            if constexpr (BPT == 8) {
                const int4 x = reinterpret_cast<const int4*>(hist)[0], y = reinterpret_cast<const int4*>(hist)[1];
                c[0] += x.x; c[1] += x.y; c[2] += x.z; c[3] += x.w;
                c[4] += y.x; c[5] += y.y; c[6] += y.z; c[7] += y.w;
            } else {
#pragma unroll
                for (int i = 0; i < BPT; ++i) c[i] += hist[i];
            }
        }
#pragma unroll
        for (int i = 0; i < BPT; ++i) sum += c[i];
        int above = sum;  // keys in this lane's bins and those of higher lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_down_sync(kFull, above, o);
            if (lane + o < 32) above += y;
        }
        if (lane == 0) s_sum[warp] = above;
        __syncthreads();
        int over = above - sum;
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            if (w > warp) over += s_sum[w];
        if (over < want && over + sum >= want) {  // one thread's bins hold it
#pragma unroll
            for (int i = BPT - 1; i >= 0; --i) {
                if (over < want && over + c[i] >= want) {
                    s_pick[0] = BPT * tid + i;
                    s_pick[1] = want - over;
                    s_pick[2] = c[i];
                }
                over += c[i];
            }
        }
        __syncthreads();
        const int bits = min(BITS, 32 - BITS * pass);  // of this digit
        T = pass == 0 ? (uint32_t)s_pick[0] : (T << bits) | (uint32_t)s_pick[0];
        want = s_pick[1];
        // done, or every key with these digits stays: the rest do not matter
        if (pass == PASSES - 1 || s_pick[2] == want) break;
        const int low = max(0, drop - BITS);           // bits below the next digit
        if (pass >= 1) {  // the next digit goes where the one before last was
            clear((pass + 1) & 1);
            __syncthreads();
        }
        for (int j = j0 + 4 * tid; j < j1; j += 4 * kThreads) {
            uint32_t k[4];
            keys4(j, k);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if ((k[e] >> drop) == T && j + e < j1)
                    atomicAdd(&s_hist[(pass + 1) & 1][(k[e] >> low) & ((1 << (drop - low)) - 1)], 1);
        }
        drop = low;
    }
    // keys are compared by their digits so far; `want` of those equal to T
    // stay, lowest index first

    // count this warp's stretch [w0, w1); few instructions per key matter where all
    // rows are on the card at once (64 requests in steady state: 11.1 -> 10.5 us with
    // chunks of one kind apart)
    const int per = (seg / kChunk + kWarps - 1) / kWarps * kChunk;
    const int w0 = min(j1, j0 + warp * per), w1 = min(j1, w0 + per);
    Counts mine = {0, 0, 0, 0};
    for (int base = w0; base < w1; base += kChunk) {
        const int j = base + 4 * lane;
        uint32_t k[4] = {0u, 0u, 0u, 0u};
        if (j < w1) keys4(j, k);
        const bool full = base + kChunk <= w1;
        if (full && base + kChunk <= b) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mine.gt_front += (k[e] >> drop) > T;
                mine.eq_front += (k[e] >> drop) == T;
            }
        } else if (full && base >= b) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mine.gt_back += (k[e] >> drop) > T;
                mine.eq_back += (k[e] >> drop) == T;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = j + e < w1, front = j + e < b;
                const int gt = in && (k[e] >> drop) > T, eq = in && (k[e] >> drop) == T;
                mine.gt_front += front ? gt : 0;
                mine.gt_back += front ? 0 : gt;
                mine.eq_front += front ? eq : 0;
                mine.eq_back += front ? 0 : eq;
            }
        }
    }
    mine.gt_front = __reduce_add_sync(kFull, mine.gt_front);
    mine.gt_back = __reduce_add_sync(kFull, mine.gt_back);
    mine.eq_front = __reduce_add_sync(kFull, mine.eq_front);
    mine.eq_back = __reduce_add_sync(kFull, mine.eq_back);
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    Counts before = {0, 0, 0, 0}, all = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const Counts x = s_warp[w];
        all = all + x;
        if (w < warp) before = before + x;
    }
    if constexpr (kCluster) {
        if (tid == 0) s_cta = all;
        cluster.sync();
        for (int r = 0; r < CS; ++r) {
            if (r == rank) continue;
            const Counts x = *cluster.map_shared_rank(&s_cta, r);
            all = all + x;
            if (r < rank) before = before + x;
        }
    }
    // tokens below the budget come before those past it, so of the ties before
    // any point the kept ones are the first `want`, the front ones first
    auto kept_front = [&](int eq_front) { return min(want, eq_front); };
    const int ties0 = before.eq_front + before.eq_back;
    int hole0 = min(w0, b) - before.gt_front - kept_front(before.eq_front);
    int mover0 = before.gt_back + min(want, ties0) - kept_front(before.eq_front);
    const int all_movers = all.gt_back + min(want, all.eq_front + all.eq_back) - kept_front(all.eq_front);

    int32_t* hole_list = p.holes + (int64_t)row * b;
    int32_t* mover_list = p.movers + (int64_t)row * b;
    const unsigned lower = (1u << lane) - 1u;
    // the lane's tokens j + e with in[e] go to the list, in order over the warp
    auto append = [&](int32_t* list, int& at, int j, const bool (&in)[4]) {
        unsigned on[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) on[e] = __ballot_sync(kFull, in[e]);
        if (!(on[0] | on[1] | on[2] | on[3])) return;
        int to = at;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            to += __popc(on[e] & lower);
            at += __popc(on[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (in[e]) list[to++] = j + e;
    };
    int seen = ties0;
    for (int base = w0; base < w1; base += kChunk) {
        const int j = base + 4 * lane;
        uint32_t k[4] = {0u, 0u, 0u, 0u};
        if (j < w1) keys4(j, k);
        bool kp[4], eq[4], out[4];
        unsigned tied[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = j + e < w1;
            kp[e] = in && (k[e] >> drop) > T;
            eq[e] = in && (k[e] >> drop) == T;
            tied[e] = __ballot_sync(kFull, eq[e]);
        }
        if (seen < want && (tied[0] | tied[1] | tied[2] | tied[3])) {  // ranks of the ties, in order
            int r = seen;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                r += __popc(tied[e] & lower);
                seen += __popc(tied[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                kp[e] |= eq[e] && r < want;
                r += eq[e];
            }
        }
        if (base < b) {  // holes
#pragma unroll
            for (int e = 0; e < 4; ++e) out[e] = j + e < min(w1, b) && !kp[e];
            append(hole_list, hole0, j, out);
        }
        if (base + kChunk > b) {  // movers; the others there are evicted
            bool all = vec && j >= b && j + 4 <= w1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                out[e] = j + e >= b && j + e < w1 && !kp[e];
                kp[e] = kp[e] && j + e >= b;
                all = all && out[e];
            }
            if (!moved_out || !moved_pos) {  // nobody reads their scores and positions any more
                if (all) {
                    if (!moved_out) *reinterpret_cast<float4*>(score_out + j) = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (!moved_pos) *reinterpret_cast<int4*>(pos_out + j) = make_int4(-1, -1, -1, -1);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (out[e]) {
                            if (!moved_out) score_out[j + e] = 0.f;
                            if (!moved_pos) pos_out[j + e] = -1;
                        }
                }
            }
            append(mover_list, mover0, j, kp);
        }
    }
    sync_row();  // the lists are complete (and no CTA's memory is read after this)

    // Moves.  A warp takes up to 32 movers: lane i looks up mover i's places
    // and moves its score and position, then LPR lanes copy each K or V row.
    constexpr int LPR = D / 8;
    constexpr int PER_STEP = 32 / (2 * LPR);  // movers copied by one warp-wide load
    constexpr int M = 4;                      // loads in flight per lane (2: +21 %, 6: +9 %, 8: one CTA per SM fewer)
    const int sub = lane / (2 * LPR), part = lane % (2 * LPR);
    uint4* cache = part < LPR ? p.k_cache : p.v_cache;
    const int64_t row_vecs = (int64_t)p.Hkv * LPR;
    cache += (int64_t)h * LPR + part % LPR;
    const int32_t* bt = p.block_tables + (int64_t)s * p.MB;
    const int bs_mask = (1 << p.bs_log2) - 1;
    const int warps = CS * kWarps;
    const int chunk = min(32, max(PER_STEP, (all_movers + warps - 1) / warps));
    for (int i0 = (rank * kWarps + warp) * chunk; i0 < all_movers; i0 += warps * chunk) {
        const int count = min(chunk, all_movers - i0);
        int slot_to = -1, slot_of = -1;
        if (lane < count) {
            const int to = hole_list[i0 + lane], of = mover_list[i0 + lane];
            const int pt = __ldg(bt + (to >> p.bs_log2)), po = __ldg(bt + (of >> p.bs_log2));
            const float sv = score[of];
            const int q = stored[of];
            if ((unsigned)pt < (unsigned)p.NB && (unsigned)po < (unsigned)p.NB) {
                slot_to = (pt << p.bs_log2) | (to & bs_mask);
                slot_of = (po << p.bs_log2) | (of & bs_mask);
            } else {
                pkv::report(p.err, PKV_DEVERR_BLOCK_ID);
            }
            score_out[to] = sv;
            pos_out[to] = q >= 0 ? q : N - n + of;
            if (!moved_out) score_out[of] = 0.f;
            if (!moved_pos) pos_out[of] = -1;
        }
        for (int m = 0; m < count; m += M * PER_STEP) {
            uint4 v[M];
            int to[M];
#pragma unroll
            for (int u = 0; u < M; ++u) {
                const int i = m + u * PER_STEP + sub;
                to[u] = __shfl_sync(kFull, slot_to, i & 31);
                const int of = __shfl_sync(kFull, slot_of, i & 31);
                if (i >= count) to[u] = -1;
                if (to[u] >= 0) v[u] = cache[of * row_vecs];
            }
#pragma unroll
            for (int u = 0; u < M; ++u)
                if (to[u] >= 0) cache[to[u] * row_vecs] = v[u];
        }
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t list_bytes(int S, int Hkv, int budget) { return align256((size_t)S * Hkv * budget * sizeof(int32_t)); }

template <int D>
void (*pick(int cs, int threads, bool wait))(Params) {
    if (threads == 128) return evict_kernel<D, false, 128, 8>;
    if (threads == 512) return cs > 1 ? evict_kernel<D, true, 512, 2> : evict_kernel<D, false, 512, 2>;
    if (cs > 1) return wait ? evict_kernel<D, true, 256, 5> : evict_kernel<D, true, 256, 4>;
    return wait ? evict_kernel<D, false, 256, 5> : evict_kernel<D, false, 256, 4>;
}

// Allows the kernel its shared memory (once per device).
bool ready(void (*fn)(Params), int smem) {
    static std::mutex mu;
    static struct { void (*fn)(Params); int dev; } done[128];
    static int used = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < used; ++i)
        if (done[i].fn == fn && done[i].dev == dev) return true;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (used < 128) done[used++] = {fn, dev};
    return true;
}

}  // namespace

extern "C" {

size_t pkv_evict_workspace_size(int S, int Hkv, int budget) {
    if (S < 0 || Hkv <= 0 || budget <= 0) return 0;
    const size_t n = 2 * list_bytes(S, Hkv, budget);
    return n ? n : 256;
}

pkv_status pkv_evict_tokens(void* k_cache, void* v_cache, const float* scores,
                            const int32_t* positions, const int32_t* block_tables,
                            const int32_t* context_lens, const int32_t* token_counts,
                            float* scores_out, int32_t* positions_out, int32_t* new_context_lens,
                            int S, int Hkv, int D, int bs, int NB, int MB, int max_context_len,
                            int64_t score_stride, int budget, int recent_tokens, int sink_tokens, pkv_dtype dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
    PKV_TRACE("pkv_evict_tokens");
    pkv::clear_error();
    if (S < 0 || Hkv <= 0 || NB <= 0 || MB <= 0 || score_stride < 0 || (dtype != PKV_F16 && dtype != PKV_BF16))
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: bad size or dtype");
    if ((D != 64 && D != 128) || (bs != 8 && bs != 16 && bs != 32 && bs != 64))
        return pkv::fail(PKV_ERR_UNSUPPORTED, "evict_tokens: head_dim must be 64/128, block_size 8/16/32/64");
    if (max_context_len < 0 || max_context_len > (int64_t)MB * bs)
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: max_context_len must be in [0, MB*bs]");
    if (score_stride < (max_context_len ? max_context_len : (int64_t)MB * bs))
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: score_stride must be at least max_context_len");
    if (budget < 1 || recent_tokens < 0 || sink_tokens < 0 || (int64_t)recent_tokens + sink_tokens > budget)
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: budget must be >= 1 and hold the sinks and the recent tokens");
    if ((int64_t)NB * bs > INT32_MAX)
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: NB * bs must fit 31 bits");
    if ((int64_t)S * Hkv > INT32_MAX / kMaxCluster)
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: too many rows");
    if (S == 0) return PKV_OK;
    if (!k_cache || !v_cache || !scores || !positions || !block_tables || !context_lens ||
        !token_counts || !scores_out || !positions_out || !new_context_lens)
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: null pointer");
    if (!pkv::aligned16(k_cache) || !pkv::aligned16(v_cache))
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: cache pointers must be 16-byte aligned");
    // every head of a sequence reads its length and its count; one of them writes the new length
    auto overlap = [&](const int32_t* in) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(in), y = reinterpret_cast<uintptr_t>(new_context_lens);
        return (x < y ? y - x : x - y) < (uintptr_t)S * sizeof(int32_t);
    };
    if (overlap(context_lens) || overlap(token_counts))
        return pkv::fail(PKV_ERR_INVALID_ARG,
                         "evict_tokens: new_context_lens must not overlap context_lens or token_counts");
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: workspace must be a 256-byte aligned device pointer");
    if (workspace_bytes < pkv_evict_workspace_size(S, Hkv, budget))
        return pkv::fail(PKV_ERR_WORKSPACE, "evict_tokens: workspace too small");

    const int64_t cap = max_context_len ? max_context_len : (int64_t)MB * bs;
    Params p;
    p.k_cache = static_cast<uint4*>(k_cache);
    p.v_cache = static_cast<uint4*>(v_cache);
    p.scores = scores;
    p.positions = positions;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.token_counts = token_counts;
    p.scores_out = scores_out;
    p.positions_out = positions_out;
    p.new_lens = new_context_lens;
    p.Hkv = Hkv;
    p.NB = NB;
    p.MB = MB;
    p.bs_log2 = bs == 8 ? 3 : (bs == 16 ? 4 : (bs == 32 ? 5 : 6));
    p.max_ctx = cap < INT32_MAX / 2 ? (int)cap : INT32_MAX / 2;
    p.stride = score_stride;
    p.budget = budget;
    p.recent = recent_tokens;
    p.sinks = sink_tokens;
    p.holes = static_cast<int32_t*>(workspace);
    p.movers = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + list_bytes(S, Hkv, budget));
    p.err = pkv::device_error_word();

    p.vec = score_stride % 4 == 0 && pkv::aligned16(scores) && pkv::aligned16(positions) &&
            pkv::aligned16(scores_out) && pkv::aligned16(positions_out);
    // CTAs per row: until the card has two per SM or a CTA 2048 keys, and for
    // rows beyond a CTA's shared memory
    const int rows = S * Hkv;
    int cs = 1;
    while (cs < kMaxCluster && ((rows * cs < 2 * pkv::sm_count() && p.max_ctx / cs > kFewKeys) ||
                                p.max_ctx / cs > kManyKeys))
        cs *= 2;
    const int seg = ((p.max_ctx + cs - 1) / cs + kChunk - 1) / kChunk * kChunk;
    p.seg_cap = seg < kSmemKeys ? seg : kSmemKeys;
    const bool wait = rows * cs > 4 * pkv::sm_count();
    const int sms = pkv::sm_count();
    const int moves = p.max_ctx - budget < budget ? p.max_ctx - budget : budget;  // of a row at most
    const int threads = cs == 1 && p.max_ctx <= (rows > 5 * sms ? kSmallKeysWaiting : kSmallKeys) ? 128
                        : rows * cs <= 2 * sms && moves / cs >= kManyMoves ? 512 : 256;
    void (*fn)(Params) = D == 128 ? pick<128>(cs, threads, wait) : pick<64>(cs, threads, wait);
    if (!ready(fn, kSmemKeys * 4)) return pkv::fail(PKV_ERR_CUDA, "evict_tokens: shared memory");
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * cs));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = (size_t)p.seg_cap * 4;
    cfg.stream = pkv::as_stream(stream);
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    return e == cudaSuccess ? PKV_OK : pkv::cuda_fail(e, "evict_tokens launch");
}

}  // extern "C"
