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
// all ones, NaN as -inf, -0 as +0), held in shared memory; at most four passes
// over 8-bit digits with a 256-bin histogram find the budget-th key (fewer when
// a bin stays as a whole), and ties are kept from the lowest index by counting.
// All counts are integers: the result does not depend on the order of the
// atomics.
//
// One cluster of 1..8 CTAs per (s, h): each CTA holds a stretch of the row,
// histograms are summed through distributed shared memory, so few long rows
// spread over the card.  Bound: 8 bytes read per token for the selection and
// 2 * 2 * D * 2 bytes per moved token; see the kernel's comment for rates.
#include <cooperative_groups.h>

#include <climits>
#include <cstdio>
#include <mutex>

#include "pagedkv.h"
#include "pkv_device.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr int kPasses = 4;
constexpr int kMaxCluster = 8;
constexpr int kKeysPerCta = 4096;     // a row's CTAs: until this many keys each
constexpr int kSmemKeys = 48 * 1024;  // keys a CTA can hold: 192 KB
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
    int32_t* holes;       // [S * Hkv][budget]
    int32_t* movers;      // [S * Hkv][budget]
    int* err;
};

__device__ __forceinline__ uint32_t key_of(float score, bool safe) {
    if (safe) return 0xffffffffu;
    if (score != score) return 0x007fffffu;          // as -inf
    const uint32_t u = score == 0.f ? 0u : __float_as_uint(score);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
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

template <int D, bool kCluster>
__global__ void __launch_bounds__(kThreads) evict_kernel(Params p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ uint32_t s_keys[];
    __shared__ int s_hist[kPasses][kBins];
    __shared__ int s_pick[2];
    __shared__ Counts s_warp[kWarps];
    __shared__ Counts s_cta;         // of this CTA's stretch, read by the cluster
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = kCluster ? (int)cluster.num_blocks() : 1;
    const int rank = kCluster ? (int)cluster.block_rank() : 0;
    auto sync_row = [&] {  // all the row's CTAs
        if constexpr (kCluster) cluster.sync(); else __syncthreads();
    };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / CS;
    const int s = row / p.Hkv, h = row % p.Hkv;

    const int raw = __ldg(p.context_lens + s);
    int N = __ldg(p.token_counts + s);
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
    const int b = p.budget;

    if (n <= b) {  // the same in every CTA of the row
        for (int j = rank * kThreads + tid; j < n; j += CS * kThreads) {
            if (moved_out) score_out[j] = score[j];
            if (moved_pos) pos_out[j] = stored[j];
        }
        return;
    }

    // this CTA's stretch [j0, j1) of the row
    const int seg = ((n + CS - 1) / CS + 31) & ~31;
    const int j0 = min(n, rank * seg), j1 = min(n, j0 + seg);
    const bool in_smem = seg <= p.seg_cap;
    const int oldest_recent = N - p.recent;
    auto make_key = [&](float sc, int stored_pos, int j) -> uint32_t {
        const int q = stored_pos >= 0 ? stored_pos : N - n + j;
        return key_of(sc, q < p.sinks || q >= oldest_recent);
    };
    auto key = [&](int j) -> uint32_t {
        return in_smem ? s_keys[j - j0] : make_key(score[j], stored[j], j);
    };

    for (int i = tid; i < kPasses * kBins; i += kThreads) (&s_hist[0][0])[i] = 0;
    __syncthreads();

    // the budget-th largest key T, digit by digit from the top
    uint32_t T = 0;
    int want = b;        // rank still to find among the keys with the digits so far
    int pass = 0;
#pragma unroll 1
    for (;; ++pass) {
        const int shift = 24 - 8 * pass;
        if (pass == 0) {
            constexpr int U = 8;  // loads in flight per thread
            for (int base = j0; base < j1; base += U * kThreads) {
                float sc[U];
                int q[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int j = base + u * kThreads + tid;
                    sc[u] = j < j1 ? score[j] : 0.f;
                    q[u] = j < j1 ? stored[j] : 0;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int j = base + u * kThreads + tid;
                    if (j < j1) {
                        const uint32_t k = make_key(sc[u], q[u], j);
                        if (in_smem) s_keys[j - j0] = k;
                        atomicAdd(&s_hist[0][k >> 24], 1);
                    }
                }
            }
        } else {
            for (int j = j0 + tid; j < j1; j += kThreads) {
                const uint32_t k = key(j);
                if ((k >> (shift + 8)) == T) atomicAdd(&s_hist[pass][(k >> shift) & 255u], 1);
            }
        }
        sync_row();
        // suffix counts over the bins, 8 per lane; alone, every warp does it,
        // in a cluster warp 0 reads the others' bins and tells its CTA
        int digit = 0, rest = 0, in_bin = 0;
        if (!kCluster || warp == 0) {
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = 0;
            if constexpr (kCluster) {
                for (int r = 0; r < CS; ++r) {
                    const int4* other = reinterpret_cast<const int4*>(
                        cluster.map_shared_rank(&s_hist[pass][0], r) + 8 * lane);
                    const int4 x = other[0], y = other[1];
                    c[0] += x.x; c[1] += x.y; c[2] += x.z; c[3] += x.w;
                    c[4] += y.x; c[5] += y.y; c[6] += y.z; c[7] += y.w;
                }
            } else {
                const int4* own = reinterpret_cast<const int4*>(&s_hist[pass][8 * lane]);
                const int4 x = own[0], y = own[1];
                c[0] = x.x; c[1] = x.y; c[2] = x.z; c[3] = x.w;
                c[4] = y.x; c[5] = y.y; c[6] = y.z; c[7] = y.w;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += c[i];
            int above = sum;  // keys in this lane's bins and those of higher lanes
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_down_sync(kFull, above, o);
                if (lane + o < 32) above += y;
            }
            int over = above - sum;
            bool mine = false;
#pragma unroll
            for (int i = 7; i >= 0; --i) {
                if (over < want && over + c[i] >= want) {
                    mine = true;
                    digit = 8 * lane + i;
                    rest = want - over;
                    in_bin = c[i];
                }
                over += c[i];
            }
            const int src = __ffs(__ballot_sync(kFull, mine)) - 1;
            digit = __shfl_sync(kFull, digit, src);
            rest = __shfl_sync(kFull, rest, src);
            in_bin = __shfl_sync(kFull, in_bin, src);
            if (kCluster && lane == 0) {
                s_pick[0] = digit | (in_bin == rest ? 256 : 0);
                s_pick[1] = rest;
            }
        }
        bool whole = in_bin == rest;
        if constexpr (kCluster) {
            __syncthreads();
            digit = s_pick[0] & 255;
            whole = (s_pick[0] & 256) != 0;
            rest = s_pick[1];
        }
        T = (T << 8) | (uint32_t)digit;
        want = rest;
        // every key with these digits stays: the digits left do not matter
        if (whole || pass == kPasses - 1) break;
    }
    // keys are compared by their digits so far; `want` of those equal to T
    // stay, lowest index first
    const int drop = 24 - 8 * pass;

    // count this warp's stretch [w0, w1)
    const int per = ((seg / 32 + kWarps - 1) / kWarps) * 32;
    const int w0 = min(j1, j0 + warp * per), w1 = min(j1, w0 + per);
    Counts mine = {0, 0, 0, 0};
#pragma unroll 4
    for (int j = w0 + lane; j < w1; j += 32) {
        const uint32_t k = key(j) >> drop;
        const int gt = k > T, eq = k == T, front = j < b;
        mine.gt_front += gt & front;
        mine.gt_back += gt & (front ^ 1);
        mine.eq_front += eq & front;
        mine.eq_back += eq & (front ^ 1);
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
    int seen = ties0;
    for (int base = w0; base < w1; base += 32) {
        const int j = base + lane;
        const bool in = j < w1;
        const uint32_t k = in ? key(j) >> drop : 0u;
        const unsigned below = (1u << lane) - 1u;
        const unsigned eq = __ballot_sync(kFull, in && k == T);
        const bool kp = in && (k > T || (k == T && seen + __popc(eq & below) < want));
        seen += __popc(eq);
        const bool is_hole = in && !kp && j < b, is_mover = kp && j >= b;
        const unsigned hm = __ballot_sync(kFull, is_hole), mm = __ballot_sync(kFull, is_mover);
        if (is_hole) hole_list[hole0 + __popc(hm & below)] = j;
        if (is_mover) mover_list[mover0 + __popc(mm & below)] = j;
        hole0 += __popc(hm);
        mover0 += __popc(mm);
        if (kp && j < b) {  // stays in its place
            const int q = stored[j];
            if (moved_out) score_out[j] = score[j];
            if (moved_pos || q < 0) pos_out[j] = q >= 0 ? q : N - n + j;
        } else if (in && j >= b && !kp) {  // evicted, past the new length
            score_out[j] = 0.f;
            pos_out[j] = -1;
        }
    }
    sync_row();  // the lists are complete (and no CTA's memory is read after this)

    // Moves.  A warp takes up to 32 movers: lane i looks up mover i's places
    // and moves its score and position, then LPR lanes copy each K or V row.
    constexpr int LPR = D / 8;
    constexpr int PER_STEP = 32 / (2 * LPR);  // movers copied by one warp-wide load
    constexpr int U = 8;                      // loads in flight per lane
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
            score_out[of] = 0.f;
            pos_out[of] = -1;
        }
        for (int m = 0; m < count; m += U * PER_STEP) {
            uint4 v[U];
            int to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = m + u * PER_STEP + sub;
                to[u] = __shfl_sync(kFull, slot_to, i & 31);
                const int of = __shfl_sync(kFull, slot_of, i & 31);
                if (i >= count) to[u] = -1;
                if (to[u] >= 0) v[u] = cache[of * row_vecs];
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (to[u] >= 0) cache[to[u] * row_vecs] = v[u];
        }
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t list_bytes(int S, int Hkv, int budget) { return align256((size_t)S * Hkv * budget * sizeof(int32_t)); }

// Allows the kernel its shared memory (once per device).
bool ready(void (*fn)(Params), int smem) {
    static std::mutex mu;
    static struct { void (*fn)(Params); int dev; } done[16];
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
    if (used < 16) done[used++] = {fn, dev};
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
                            int S, int Hkv, int D, int bs, int NB, int MB, int64_t score_stride,
                            int budget, int recent_tokens, int sink_tokens, pkv_dtype dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
    PKV_TRACE("pkv_evict_tokens");
    pkv::clear_error();
    if (S < 0 || Hkv <= 0 || NB <= 0 || MB <= 0 || score_stride < 0 || (dtype != PKV_F16 && dtype != PKV_BF16))
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: bad size or dtype");
    if ((D != 64 && D != 128) || (bs != 8 && bs != 16 && bs != 32 && bs != 64))
        return pkv::fail(PKV_ERR_UNSUPPORTED, "evict_tokens: head_dim must be 64/128, block_size 8/16/32/64");
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
    // every head of a sequence reads its length
    if (new_context_lens == context_lens)
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: new_context_lens must not be context_lens");
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return pkv::fail(PKV_ERR_INVALID_ARG, "evict_tokens: workspace must be a 256-byte aligned device pointer");
    if (workspace_bytes < pkv_evict_workspace_size(S, Hkv, budget))
        return pkv::fail(PKV_ERR_WORKSPACE, "evict_tokens: workspace too small");

    const int64_t cap = (int64_t)MB * bs < score_stride ? (int64_t)MB * bs : score_stride;
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

    // CTAs per row
    const int rows = S * Hkv;
    int cs = 1;
    while (cs < kMaxCluster && p.max_ctx / cs > kKeysPerCta) cs *= 2;
    const int seg = ((p.max_ctx + cs - 1) / cs + 31) & ~31;
    p.seg_cap = seg < kSmemKeys ? seg : kSmemKeys;
    void (*fn)(Params) = cs > 1 ? (D == 128 ? evict_kernel<128, true> : evict_kernel<64, true>)
                                : (D == 128 ? evict_kernel<128, false> : evict_kernel<64, false>);
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
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)p.seg_cap * 4;
    cfg.stream = pkv::as_stream(stream);
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    return e == cudaSuccess ? PKV_OK : pkv::cuda_fail(e, "evict_tokens launch");
}

}  // extern "C"
