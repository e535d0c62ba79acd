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
// all ones, NaN as -inf, -0 as +0), held in shared memory; four passes over
// 8-bit digits with a 256-bin histogram find the budget-th key, and ties are
// kept from the lowest index by counting.  All counts are integers: the result
// does not depend on the order of the atomics.
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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr int kPasses = 4;
constexpr int kMaxCluster = 8;
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

// Sum over the block's warps of `v` below this warp, and the block's total.
__device__ __forceinline__ int warp_offset(int v, int* s_warp, int warp, int lane, int& total) {
    if (lane == 0) s_warp[warp] = v;
    __syncthreads();
    int x = lane < kWarps ? s_warp[lane] : 0;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    total = __shfl_sync(kFull, incl, kWarps - 1);
    const int before = __shfl_sync(kFull, incl - x, warp);
    __syncthreads();
    return before;
}

template <int D>
__global__ void __launch_bounds__(kThreads) evict_kernel(Params p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ uint32_t s_keys[];
    __shared__ int s_hist[kPasses][kBins];
    __shared__ int s_warp[kWarps];
    __shared__ int s_pick[2];
    __shared__ int s_counts[2];      // holes and movers of this CTA's stretch
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / CS;
    const int s = row / p.Hkv, h = row % p.Hkv;

    const int raw = __ldg(p.context_lens + s);
    const int n = raw < 0 ? 0 : (raw > p.max_ctx ? p.max_ctx : raw);
    int N = __ldg(p.token_counts + s);
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

    if (n <= b) {  // the same in every CTA of the cluster
        for (int j = rank * kThreads + tid; j < n; j += CS * kThreads) {
            if (moved_out) score_out[j] = score[j];
            if (moved_pos) pos_out[j] = stored[j];
        }
        return;
    }

    // this CTA's stretch [j0, j1), this warp's part [w0, w1)
    const int seg = ((n + CS - 1) / CS + 31) & ~31;
    const int j0 = min(n, rank * seg), j1 = min(n, j0 + seg);
    const bool in_smem = seg <= p.seg_cap;
    const int oldest_recent = N - p.recent;
    auto position = [&](int j) -> int {
        const int q = stored[j];
        return q >= 0 ? q : N - n + j;
    };
    auto make_key = [&](int j) -> uint32_t {
        const int q = position(j);
        return key_of(score[j], q < p.sinks || q >= oldest_recent);
    };
    auto key = [&](int j) -> uint32_t { return in_smem ? s_keys[j - j0] : make_key(j); };

    for (int i = tid; i < kPasses * kBins; i += kThreads) (&s_hist[0][0])[i] = 0;
    __syncthreads();

    // the budget-th largest key, digit by digit from the top
    uint32_t prefix = 0;
    int want = b;        // rank still to find among the keys with the prefix
    int ties_before = 0; // keys equal to it in the CTAs before this one
#pragma unroll 1
    for (int pass = 0; pass < kPasses; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int j = j0 + tid; j < j1; j += kThreads) {
            uint32_t k;
            if (pass == 0) {
                k = make_key(j);
                if (in_smem) s_keys[j - j0] = k;
            } else {
                k = key(j);
                if ((k >> (shift + 8)) != prefix) continue;
            }
            atomicAdd(&s_hist[pass][(k >> shift) & 255u], 1);
        }
        cluster.sync();
        // suffix counts over the bins, 8 bins per lane of warp 0
        if (warp == 0) {
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = 0;
                for (int r = 0; r < CS; ++r)
                    c[i] += cluster.map_shared_rank(&s_hist[pass][0], r)[8 * lane + i];
                sum += c[i];
            }
            int above = sum;  // keys in this lane's bins and those of higher lanes
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_down_sync(kFull, above, o);
                if (lane + o < 32) above += y;
            }
            int over = above - sum;
#pragma unroll
            for (int i = 7; i >= 0; --i) {
                if (over < want && over + c[i] >= want) {
                    s_pick[0] = 8 * lane + i;
                    s_pick[1] = want - over;
                }
                over += c[i];
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | (uint32_t)s_pick[0];
        want = s_pick[1];
    }
    const uint32_t T = prefix;
    // `want` of the keys equal to T stay, lowest index first
    for (int r = 0; r < rank; ++r)
        ties_before += cluster.map_shared_rank(&s_hist[kPasses - 1][0], r)[T & 255u];

    const int per = ((seg / 32 + kWarps - 1) / kWarps) * 32;  // this warp's stretch
    const int w0 = min(j1, j0 + warp * per), w1 = min(j1, w0 + per);
    // ties before this warp
    int ties = 0, dummy;
    for (int j = w0 + lane; j < w1; j += 32) ties += key(j) == T;
    ties = __reduce_add_sync(kFull, ties);
    const int ties0 = ties_before + warp_offset(ties, s_warp, warp, lane, dummy);

    // holes and movers: count, then list in order
    int holes = 0, movers = 0, seen = ties0;
    auto kept = [&](int j, int& seen_ties) -> bool {  // whole warp, j = base + lane
        const uint32_t k = j < w1 ? key(j) : 0u;
        const unsigned eq = __ballot_sync(kFull, j < w1 && k == T);
        const bool tie_in = seen_ties + __popc(eq & ((1u << lane) - 1u)) < want;
        seen_ties += __popc(eq);
        return j < w1 && (k > T || (k == T && tie_in));
    };
    for (int base = w0; base < w1; base += 32) {
        const int j = base + lane;
        const bool kp = kept(j, seen);
        holes += __popc(__ballot_sync(kFull, j < w1 && !kp && j < b));
        movers += __popc(__ballot_sync(kFull, kp && j >= b));
    }
    int total_holes, total_movers;
    int hole0 = warp_offset(holes, s_warp, warp, lane, total_holes);
    int mover0 = warp_offset(movers, s_warp, warp, lane, total_movers);
    if (tid == 0) {
        s_counts[0] = total_holes;
        s_counts[1] = total_movers;
    }
    cluster.sync();
    int all_movers = 0;
    for (int r = 0; r < CS; ++r) {
        const int* other = cluster.map_shared_rank(&s_counts[0], r);
        if (r < rank) {
            hole0 += other[0];
            mover0 += other[1];
        }
        all_movers += other[1];
    }
    int32_t* hole_list = p.holes + (int64_t)row * b;
    int32_t* mover_list = p.movers + (int64_t)row * b;
    seen = ties0;
    for (int base = w0; base < w1; base += 32) {
        const int j = base + lane;
        const bool kp = kept(j, seen);
        const bool is_hole = j < w1 && !kp && j < b, is_mover = kp && j >= b;
        const unsigned hm = __ballot_sync(kFull, is_hole), mm = __ballot_sync(kFull, is_mover);
        const unsigned below = (1u << lane) - 1u;
        if (is_hole) hole_list[hole0 + __popc(hm & below)] = j;
        if (is_mover) mover_list[mover0 + __popc(mm & below)] = j;
        hole0 += __popc(hm);
        mover0 += __popc(mm);
        if (kp && j < b) {  // stays in its place
            const int q = stored[j];
            if (moved_out) score_out[j] = score[j];
            if (moved_pos || q < 0) pos_out[j] = q >= 0 ? q : N - n + j;
        } else if (j < w1 && j >= b && !kp) {  // evicted, past the new length
            score_out[j] = 0.f;
            pos_out[j] = -1;
        }
    }
    cluster.sync();  // the lists are complete (and no CTA's memory is read after this)

    // moves: LPR lanes take one K or V row of D elements
    constexpr int LPR = D / 8;
    constexpr int PER_WARP = 32 / (2 * LPR);  // movers a warp takes at once
    const int sub = lane / (2 * LPR), part = lane % (2 * LPR);
    uint4* cache = part < LPR ? p.k_cache : p.v_cache;
    const int col = part % LPR;
    const int32_t* bt = p.block_tables + (int64_t)s * p.MB;
    const int bs_mask = (1 << p.bs_log2) - 1;
    const int step = CS * kWarps * PER_WARP;
    constexpr int U = 4;
    for (int i0 = (rank * kWarps + warp) * PER_WARP + sub; i0 < all_movers; i0 += U * step) {
        uint4 v[U];
        uint4* dst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * step;
            dst[u] = nullptr;
            if (i < all_movers) {
                const int to = hole_list[i], of = mover_list[i];
                const int pt = __ldg(bt + (to >> p.bs_log2)), po = __ldg(bt + (of >> p.bs_log2));
                if ((unsigned)pt < (unsigned)p.NB && (unsigned)po < (unsigned)p.NB) {
                    const int64_t rt = ((int64_t)pt << p.bs_log2) + (to & bs_mask);
                    const int64_t ro = ((int64_t)po << p.bs_log2) + (of & bs_mask);
                    dst[u] = cache + (rt * p.Hkv + h) * LPR + col;
                    v[u] = cache[(ro * p.Hkv + h) * LPR + col];
                } else if (part == 0) {
                    pkv::report(p.err, PKV_DEVERR_BLOCK_ID);
                }
                if (part == 0) {
                    const float sv = score[of];
                    const int q = position(of);
                    score_out[to] = sv;
                    pos_out[to] = q;
                    score_out[of] = 0.f;
                    pos_out[of] = -1;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (dst[u]) *dst[u] = v[u];
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

    // CTAs per row: while the card is not filled and a CTA has over 4096 keys
    const int rows = S * Hkv;
    int cs = 1;
    while (cs < kMaxCluster && rows * cs < 2 * pkv::sm_count() && p.max_ctx / cs > 4096) cs *= 2;
    const int seg = ((p.max_ctx + cs - 1) / cs + 31) & ~31;
    p.seg_cap = seg < kSmemKeys ? seg : kSmemKeys;
    void (*fn)(Params) = D == 128 ? evict_kernel<128> : evict_kernel<64>;
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
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    return e == cudaSuccess ? PKV_OK : pkv::cuda_fail(e, "evict_tokens launch");
}

}  // extern "C"
