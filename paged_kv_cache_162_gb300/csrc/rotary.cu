// Appending a step's tokens with the rotary position encoding applied on the
// way: into the 16-bit caches, or into a cache held in 4 bits (q4.cuh); and the
// way back, 4-bit rows of given slots as 16-bit values.
//
// Rotation of the first R dims of a q or K row by the angles of its position,
// pair i with cos_i and sin_i out of a table's row:
//   (a, b) -> (a cos - b sin, b cos + a sin),
// (a, b) = dims (i, i + R/2), or (2i, 2i + 1) interleaved.  In fp32, every
// product and sum rounded by itself: the same numbers wherever this is written
// with plain fp32 operations, which a value on the border between two codes
// needs to land on the same one.
//
// Memory is the bound: a row is read once and written once; a 4-bit row is
// 288 (D = 128: 576) bytes per 8 tokens.  One CTA takes a few tokens, D / 16
// neighbouring threads a row at a time; a thread holds two chunks of 8 dims that
// rotate with one another (dims 8j and R/2 + 8j, or 16 neighbouring dims when
// interleaved), so nothing is exchanged.  The next row is on its way while one is
// turned; its angles come out of L1, where the first row of the token left them.
// (Two to four rows on their way: 149 to 173 us where one takes 140; the registers
// cost more warps than the rows in flight bring.)
//
// Measured, D = 128: 16 prompts of 320..1727 tokens, 32 + 32 + 32 heads in fp16,
// interleaved: 135 us, 5.96 TB/s of what it has to move, 88 % of a plain copy's rate.
// 20 thousand tokens of 8 KV heads into 4 bits, with 32 query heads turned by 64
// dims: 98 us, 4.4 TB/s (64 us at a plain copy's rate).  It issues on 64 % of the cycles
// (8 instructions per element for the codes; half the threads wait while the other
// half's dims turn), has DRAM at 49 % of its peak, and for the rest waits for rows: one
// of 32 bytes on its way per thread is 28 KB per SM.  4-bit rows of 64 contexts back to
// fp16: 234 us, 6.25 TB/s, 92 %.  250 decoding sequences: 3.7 us, 5.0 in 4 bits; a
// handful of tokens 2.7 to 3.4: launch, position -> block -> slot, row.
#include <cmath>
#include <cstdio>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "q4.cuh"

namespace {

namespace q4 = pkv::q4;

constexpr unsigned kFull = 0xffffffffu;

struct AppendParams {
    const char *key, *value, *query;
    char* query_out;
    int64_t key_stride, value_stride, query_stride, query_out_stride;  // bytes per token
    char *k_cache, *v_cache;
    const int32_t *block_tables, *seq_idx, *pos, *rotary_pos;
    const float* table;  // [table_rows][R]: R / 2 cos, R / 2 sin
    int64_t* slots;
    int T, S, H, Hkv, bs_log2, MB, R, table_rows, interleaved;
    int per_cta;         // tokens, at most kMaxTokens
    int64_t num_slots;
    int* err;
};
// 2, 4, 8 tokens per CTA: 140, 135.5, 140 us in 16 bits, 119, 118, 126 in 4 (with
// their gather); more leave the last wave of CTAs emptier.
constexpr int kMaxTokens = 4;

// 16 bytes that are read once.  Not on the read-only path: queries may be turned in
// place.  (A store to where a load was depends on what it brought.)
__device__ __forceinline__ uint4 ld_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void st16(char* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }

// The two chunks of 8 dims that thread j of a row holds.
__device__ __forceinline__ void chunks_of(int j, int R, int interleaved, int& a, int& b) {
    const int turning = R / 16;
    if (interleaved || j >= turning) {
        a = 2 * j;
        b = a + 1;
    } else {
        a = j;
        b = j + turning;
    }
}

// Both chunks of a row by the thread's angles.
template <bool kPairs>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&cs)[8], const float (&sn)[8]) {
    auto turn = [](float& x, float& y, float c, float s) {
        const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
        y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
        x = u;
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!kPairs) turn(a[i], b[i], cs[i], sn[i]);
        else if (i < 4) turn(a[2 * i], a[2 * i + 1], cs[i], sn[i]);
        else turn(b[2 * i - 8], b[2 * i - 7], cs[i], sn[i]);
    }
}

// Least and greatest of a chunk, NaN where an element is.
__device__ __forceinline__ void bounds_of(const float (&x)[8], float& lo, float& hi) {
    lo = q4::min_nan(x[0], x[1]);
    hi = q4::max_nan(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        lo = q4::min_nan(lo, x[i], x[i + 1]);
        hi = q4::max_nan(hi, x[i], x[i + 1]);
    }
}

// The codes of a chunk.  (x - centre) / step by a product with 1 / step and one
// correction: where the quotient lies halfway between two codes, which rows of
// 16-bit values often do, a product alone would fall to either side.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float step, float centre, float inv) {
    // at 1.5 * 2^23 the numbers are whole: the sum is the nearest one (to even), and
    // its bits are kWhole + code.  What kWhole adds to the word comes off at the end.
    constexpr uint32_t kWhole = 0x4b400000u;
    uint32_t c = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        const float d = __fsub_rn(x[i], centre);
        const float t0 = __fmul_rn(d, inv);
        const float t = fminf(fmaxf(fmaf(fmaf(-t0, step, d), inv, t0), -8.f), 7.f);
        c = 16u * c + __float_as_uint(__fadd_rn(t, 12582920.f));
    }
    return c - 0x11111111u * kWhole;
}

// The 4-bit form in CTAs of 128 threads, 7 to an SM (20 thousand tokens and their
// gather: 122 us with 6, 118 with 7, 121 with 8, whose 64 registers are too few).
template <bool kQ4>
constexpr int kAppendThreads = kQ4 ? 128 : 256;

template <class E, int D, bool kQ4>
__global__ void __launch_bounds__(kAppendThreads<kQ4>, kQ4 ? 7 : 1) append_kernel(const __grid_constant__ AppendParams p) {
    // inputs may come from the kernel before this one; the next kernel may
    // become resident once every CTA is past this point
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int LPR = D / 16;  // threads per row
    __shared__ int64_t s_slot[kMaxTokens];  // negative: nothing is written for the token
    __shared__ int s_turn[kMaxTokens];
    const int tid = threadIdx.x, j = tid % LPR;
    const int64_t t0 = (int64_t)blockIdx.x * p.per_cta;
    const int tokens = (int)min((int64_t)p.per_cta, p.T - t0);

    // rows of a token: K of every KV head, V, then the queries
    const int kv = 2 * p.Hkv, rows = kv + p.H, step = blockDim.x / LPR;
    int ca, cb;
    chunks_of(j, p.R, p.interleaved, ca, cb);
    int k = 0, r = tid / LPR;  // the thread's token and row
    auto settle = [&]() {
        while (r >= rows && k < tokens) {
            r -= rows;
            ++k;
        }
    };
    settle();
    uint4 va, vb;
    auto load = [&]() {
        if (k >= tokens) return;
        const int64_t t = t0 + k;
        const char* from = r < p.Hkv ? p.key + t * p.key_stride + (int64_t)r * D * 2
                           : r < kv  ? p.value + t * p.value_stride + (int64_t)(r - p.Hkv) * D * 2
                                     : p.query + t * p.query_stride + (int64_t)(r - kv) * D * 2;
        va = ld_once(from + 16 * ca);
        vb = ld_once(from + 16 * cb);
    };
    if (tid < tokens) {
        const int64_t t = t0 + tid;
        const int place = p.pos[t], seq = p.seq_idx[t];
        const int turn_at = p.rotary_pos ? p.rotary_pos[t] : place;
        int64_t slot = pkv::slot_of(p.block_tables, seq, place, p.S, p.MB, 1 << p.bs_log2, p.err);
        if (slot >= 0 && p.R && (unsigned)turn_at >= (unsigned)p.table_rows) {
            pkv::report(p.err, PKV_DEVERR_POSITION);
            slot = -1;
        }
        p.slots[t] = slot;
        if (slot >= p.num_slots) {
            pkv::report(p.err, PKV_DEVERR_SLOT);
            slot = -1;
        }
        s_slot[tid] = slot;
        s_turn[tid] = turn_at;
    }
    load();
    __syncthreads();
    const bool turns = 16 * j < p.R;

    // whole warps go round together: the threads of a row exchange its bounds
    while (__any_sync(kFull, k < tokens)) {
        const bool in = k < tokens;
        const int64_t t = t0 + k, slot = in ? s_slot[k] : -1;
        const int row_of = r;
        uint4 xa = va, xb = vb;
        const bool rotates = turns && slot >= 0 && (r < p.Hkv || r >= kv);
        float cs[8], sn[8];
        if (rotates) {
            const float* at = p.table + (int64_t)s_turn[k] * p.R + 8 * j;
            const float4 c0 = __ldg(reinterpret_cast<const float4*>(at)), c1 = __ldg(reinterpret_cast<const float4*>(at) + 1);
            const float4 s0 = __ldg(reinterpret_cast<const float4*>(at + p.R / 2)),
                         s1 = __ldg(reinterpret_cast<const float4*>(at + p.R / 2) + 1);
            cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
            cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
            sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
            sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
        }
        r += step;
        settle();
        load();
        const bool is_kv = in && row_of < kv;
        float a[8], b[8];
        if (rotates || (kQ4 && is_kv)) {
            pkv::unpack8<E>(xa, a);
            pkv::unpack8<E>(xb, b);
        }
        if (rotates) {
            if (p.interleaved) rotate<true>(a, b, cs, sn);
            else rotate<false>(a, b, cs, sn);
        }
        if (kQ4 && __any_sync(kFull, is_kv)) {
            // bounds of the row's groups.  A chunk lies in group chunk / 8; the first half
            // of the row's threads goes on with group 0, the second with group 1.
            float lo[2], hi[2];
            bounds_of(a, lo[0], hi[0]);
            bounds_of(b, lo[1], hi[1]);
            const int mine = j / 4;  // a group is four threads' share
            const bool own[2] = {D == 64 || ca / 8 == mine, D == 64 || cb / 8 == mine};
            float l, h;
            if (D == 64) {
                l = q4::min_nan(lo[0], lo[1]);
                h = q4::max_nan(hi[0], hi[1]);
            } else {
                l = q4::min_nan(own[0] ? lo[0] : INFINITY, own[1] ? lo[1] : INFINITY);
                h = q4::max_nan(own[0] ? hi[0] : -INFINITY, own[1] ? hi[1] : -INFINITY);
                const float l1 = q4::min_nan(own[0] ? INFINITY : lo[0], own[1] ? INFINITY : lo[1]);
                const float h1 = q4::max_nan(own[0] ? -INFINITY : hi[0], own[1] ? -INFINITY : hi[1]);
                l = q4::min_nan(l, __shfl_xor_sync(kFull, l1, 4));
                h = q4::max_nan(h, __shfl_xor_sync(kFull, h1, 4));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                l = q4::min_nan(l, __shfl_xor_sync(kFull, l, o));
                h = q4::max_nan(h, __shfl_xor_sync(kFull, h, o));
            }
            const float n = fmaf(l, 0.f, h * 0.f);  // NaN where an element is not finite
            // in sixteenths, so that no sum overflows
            l *= 0.0625f;
            h *= 0.0625f;
            const float range = __fmul_rn(__fsub_rn(h, l), 1.f / 15.f) * 16.f + n;
            const float mid = __fmul_rn(__fadd_rn(8.f * h, __fmul_rn(7.f, l)), 1.f / 15.f) * 16.f + n;
            uint32_t pair = E::from_float2(range, mid);
            // a step so small that 1 / step could overflow: the group reads as its centre
            if (E::to_float2(pair).x < 0x1p-126f) pair &= 0xffff0000u;
            const float2 sm = E::to_float2(pair);  // step, centre
            const float inv = sm.x > 0.f ? q4::reciprocal(sm.x) : 0.f;
            float2 sm_of[2] = {sm, sm};
            float inv_of[2] = {inv, inv};
            if (D == 128) {
                const float2 other = E::to_float2(__shfl_xor_sync(kFull, pair, 4));
                const float inv_other = __shfl_xor_sync(kFull, inv, 4);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (!own[x]) {
                        sm_of[x] = other;
                        inv_of[x] = inv_other;
                    }
            }
            if (is_kv) {
                if (slot < 0) continue;
                const int head = row_of < p.Hkv ? row_of : row_of - p.Hkv, row = (int)(slot & 7);
                char* unit = (row_of < p.Hkv ? p.k_cache : p.v_cache) + q4::unit_at<D>((int)slot, head, p.Hkv, p.bs_log2);
                char* codes = unit + row * q4::code_bytes(D);
                *reinterpret_cast<uint32_t*>(codes + 16 * q4::chunk_place<D>(row, ca >> 2) + 4 * (ca & 3)) =
                    codes_of(a, sm_of[0].x, sm_of[0].y, inv_of[0]);
                *reinterpret_cast<uint32_t*>(codes + 16 * q4::chunk_place<D>(row, cb >> 2) + 4 * (cb & 3)) =
                    codes_of(b, sm_of[1].x, sm_of[1].y, inv_of[1]);
                if (j % 4 == 0)
                    *reinterpret_cast<uint32_t*>(unit + q4::kUnitCodes<D> + row * q4::pair_bytes(D) + j) = pair;
                continue;
            }
        }
        if (slot < 0) continue;
        if (rotates) {
            xa = pkv::pack8<E>(a);
            xb = pkv::pack8<E>(b);
        }
        char* to = row_of < p.Hkv ? p.k_cache + (slot * p.Hkv + row_of) * D * 2
                   : row_of < kv  ? p.v_cache + (slot * p.Hkv + row_of - p.Hkv) * D * 2
                                  : p.query_out + t * p.query_out_stride + (int64_t)(row_of - kv) * D * 2;
        st16(to + 16 * ca, xa);
        st16(to + 16 * cb, xb);
    }
}

struct GatherParams {
    char *key, *value;
    int64_t key_stride, value_stride;  // bytes per token
    const char *k_cache, *v_cache;
    const int64_t* slots;
    int T, Hkv, bs_log2, splits;
    int64_t num_slots;
    int* err;
};

// `splits` CTAs read 8 tokens' K and V rows of every KV head: D / 16 threads per
// row, neighbouring tokens of one head (one run of the pool when their slots are
// neighbours too) by neighbouring rows' threads.
template <class E, int D>
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ GatherParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int LPR = D / 16;
    const int j = threadIdx.x % LPR, step = blockDim.x / LPR;
    const int64_t t0 = (int64_t)(blockIdx.x / p.splits) * 8;
    const int rows = 16 * p.Hkv;
    for (int r = blockIdx.x % p.splits * step + threadIdx.x / LPR; r < rows; r += step * p.splits) {
        const int64_t t = t0 + r % 8;
        if (t >= p.T) continue;
        const int64_t slot = p.slots[t];
        if (slot < 0) continue;
        if (slot >= p.num_slots) {
            if (j == 0) pkv::report(p.err, PKV_DEVERR_SLOT);
            continue;
        }
        const int head = r / 8 % p.Hkv, row = (int)(slot & 7);
        const bool is_k = r < 8 * p.Hkv;
        const char* unit = (is_k ? p.k_cache : p.v_cache) + q4::unit_at<D>((int)slot, head, p.Hkv, p.bs_log2);
        const uint2 code = *reinterpret_cast<const uint2*>(unit + row * q4::code_bytes(D) +
                                                           16 * q4::chunk_place<D>(row, j >> 1) + 8 * (j & 1));
        const uint32_t pair = *reinterpret_cast<const uint32_t*>(unit + q4::kUnitCodes<D> + row * q4::pair_bytes(D) +
                                                                 4 * (j >> 2));
        const float2 sm = E::to_float2(pair);  // step, centre
        char* to = is_k ? p.key + t * p.key_stride : p.value + t * p.value_stride;
        to += (int64_t)head * D * 2 + 32 * j;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t c = h ? code.y : code.x;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)  // step * (code - 8) has at most 15 bits: one rounding
                f[i] = fmaf(sm.x, (float)((int)((c >> (4 * i)) & 15u) - 8), sm.y);
            st16(to + 16 * h, pkv::pack8<E>(f));
        }
    }
}

bool supported(int D, int bs) {
    return (D == 64 || D == 128) && (bs == 8 || bs == 16 || bs == 32 || bs == 64);
}
int log2_of(int bs) { return bs == 8 ? 3 : bs == 16 ? 4 : bs == 32 ? 5 : 6; }

template <class P>
cudaError_t launch(void (*fn)(P), int64_t grid, int threads, void* stream, const P& p) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = pkv::as_stream(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

// Token strides are in elements: multiples of 8 (16 bytes), a token's rows at
// least, below 2^30: its product with a token number stays in 64 bits.
bool stride_ok(int64_t stride, int heads, int D) {
    return stride >= (int64_t)heads * D && stride % 8 == 0 && stride < (int64_t)1 << 30;
}

// Whether T rows of a_wide bytes at a and of b_wide at b share a byte
// (interleaved slices of one projection do not).
bool overlap(const void* a, int64_t a_stride, int64_t a_wide, const void* b, int64_t b_stride, int64_t b_wide, int T) {
    const int64_t pa = (int64_t)reinterpret_cast<uintptr_t>(a), pb = (int64_t)reinterpret_cast<uintptr_t>(b);
    if (pa + (T - 1) * a_stride + a_wide <= pb || pb + (T - 1) * b_stride + b_wide <= pa) return false;
    if (a_stride != b_stride) return true;
    const int64_t d = ((pb - pa) % a_stride + a_stride) % a_stride;  // of a b row behind an a row
    return d < a_wide || a_stride - d < b_wide;
}

template <bool kQ4>
pkv_status append(const char* who, const void* key, int64_t key_stride, const void* value, int64_t value_stride,
                  const void* query, int64_t query_stride, void* query_out, int64_t query_out_stride, void* k_cache,
                  void* v_cache, const int32_t* block_tables, const int32_t* seq_idx, const int32_t* pos,
                  const int32_t* rotary_pos, const float* table, int table_rows, int R, int interleaved,
                  int64_t* slots, int T, int S, int H, int Hkv, int D, int bs, int NB, int MB, pkv_dtype dtype,
                  void* stream) {
    char msg[160];
    auto bad = [&](pkv_status st, const char* what) {
        snprintf(msg, sizeof msg, "%s: %s", who, what);
        return pkv::fail(st, msg);
    };
    if (T < 0 || S < 0 || (T > 0 && S == 0) || H < 0 || Hkv <= 0 || NB <= 0 || MB <= 0 ||
        (dtype != PKV_F16 && dtype != PKV_BF16))
        return bad(PKV_ERR_INVALID_ARG, "bad size or dtype");
    if (!supported(D, bs)) return bad(PKV_ERR_UNSUPPORTED, "head_dim must be 64/128, block_size 8/16/32/64");
    if (R < 0 || R > D || R % 16) return bad(PKV_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 up to head_dim");
    if ((int64_t)NB * bs > INT32_MAX) return bad(PKV_ERR_INVALID_ARG, "NB * bs must fit 31 bits");
    if (H > 1 << 20 || Hkv > 1 << 20) return bad(PKV_ERR_INVALID_ARG, "at most 2^20 heads");
    if (T == 0) return PKV_OK;
    if (!key || !value || !k_cache || !v_cache || !block_tables || !seq_idx || !pos || !slots ||
        (H > 0 && (!query || !query_out)) || (R > 0 && !table))
        return bad(PKV_ERR_INVALID_ARG, "null pointer");
    if (R > 0 && table_rows <= 0) return bad(PKV_ERR_INVALID_ARG, "the rotary table has no rows");
    if (!pkv::aligned16(key) || !pkv::aligned16(value) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache) ||
        (H > 0 && (!pkv::aligned16(query) || !pkv::aligned16(query_out))) || (R > 0 && !pkv::aligned16(table)))
        return bad(PKV_ERR_INVALID_ARG, "token, cache and table pointers must be 16-byte aligned");
    if (!stride_ok(key_stride, Hkv, D) || !stride_ok(value_stride, Hkv, D) ||
        (H > 0 && (!stride_ok(query_stride, H, D) || !stride_ok(query_out_stride, H, D))))
        return bad(PKV_ERR_INVALID_ARG, "token strides must be multiples of 8 elements, and a token's rows at least");
    if (H > 0) {
        const int64_t q = (int64_t)H * D * 2, kv = (int64_t)Hkv * D * 2, out = 2 * query_out_stride;
        const bool in_place = query_out == query && query_out_stride == query_stride;
        if ((!in_place && overlap(query, 2 * query_stride, q, query_out, out, q, T)) ||
            overlap(key, 2 * key_stride, kv, query_out, out, q, T) ||
            overlap(value, 2 * value_stride, kv, query_out, out, q, T))
            return bad(PKV_ERR_INVALID_ARG, "query_out must be query, or overlap neither it nor key nor value");
    }

    AppendParams p;
    p.key = static_cast<const char*>(key);
    p.value = static_cast<const char*>(value);
    p.query = static_cast<const char*>(query);
    p.query_out = static_cast<char*>(query_out);
    p.key_stride = 2 * key_stride;
    p.value_stride = 2 * value_stride;
    p.query_stride = 2 * query_stride;
    p.query_out_stride = 2 * query_out_stride;
    p.k_cache = static_cast<char*>(k_cache);
    p.v_cache = static_cast<char*>(v_cache);
    p.block_tables = block_tables;
    p.seq_idx = seq_idx;
    p.pos = pos;
    p.rotary_pos = rotary_pos;
    p.table = table;
    p.slots = slots;
    p.T = T;
    p.S = S;
    p.H = H;
    p.Hkv = Hkv;
    p.bs_log2 = log2_of(bs);
    p.MB = MB;
    p.R = R;
    p.table_rows = table_rows;
    p.interleaved = interleaved != 0;
    p.num_slots = (int64_t)NB * bs;
    p.err = pkv::device_error_word();
    void (*fn)(AppendParams) =
        dtype == PKV_F16 ? (D == 128 ? append_kernel<pkv::F16, 128, kQ4> : append_kernel<pkv::F16, 64, kQ4>)
                         : (D == 128 ? append_kernel<pkv::BF16, 128, kQ4> : append_kernel<pkv::BF16, 64, kQ4>);
    // few tokens: a CTA each; many: CTAs of several, so that the chain position ->
    // block -> slot is paid once for all their rows
    const int64_t want = (int64_t)(H + 2 * Hkv) * (D / 16);
    p.per_cta = 1;
    while (p.per_cta < kMaxTokens && T >= 16 * p.per_cta * pkv::sm_count()) p.per_cta *= 2;
    constexpr int most = kAppendThreads<kQ4>;
    const int threads = want * p.per_cta >= most ? most : (int)(want * p.per_cta + 31) / 32 * 32;
    const cudaError_t e = launch(fn, ((int64_t)T + p.per_cta - 1) / p.per_cta, threads, stream, p);
    if (e == cudaSuccess) return PKV_OK;
    snprintf(msg, sizeof msg, "%s launch", who);
    return pkv::cuda_fail(e, msg);
}

}  // namespace

extern "C" {

pkv_status pkv_rotate_and_cache(const void* key, int64_t key_stride, const void* value, int64_t value_stride,
                                const void* query, int64_t query_stride, void* query_out, int64_t query_out_stride,
                                void* k_cache, void* v_cache, const int32_t* block_tables, const int32_t* seq_idx,
                                const int32_t* pos, const int32_t* rotary_pos, const float* rotary_table,
                                int table_rows, int rotary_dim, int interleaved, int64_t* slot_mapping, int T, int S,
                                int H, int Hkv, int D, int bs, int NB, int MB, pkv_dtype dtype, void* stream) {
    PKV_TRACE("pkv_rotate_and_cache");
    pkv::clear_error();
    return append<false>("rotate_and_cache", key, key_stride, value, value_stride, query, query_stride, query_out,
                         query_out_stride, k_cache, v_cache, block_tables, seq_idx, pos, rotary_pos, rotary_table,
                         table_rows, rotary_dim, interleaved, slot_mapping, T, S, H, Hkv, D, bs, NB, MB, dtype, stream);
}

pkv_status pkv_rotate_and_cache_q4(const void* key, int64_t key_stride, const void* value, int64_t value_stride,
                                   const void* query, int64_t query_stride, void* query_out,
                                   int64_t query_out_stride, void* k_cache, void* v_cache,
                                   const int32_t* block_tables, const int32_t* seq_idx, const int32_t* pos,
                                   const int32_t* rotary_pos, const float* rotary_table, int table_rows,
                                   int rotary_dim, int interleaved, int64_t* slot_mapping, int T, int S, int H,
                                   int Hkv, int D, int bs, int NB, int MB, pkv_dtype dtype, void* stream) {
    PKV_TRACE("pkv_rotate_and_cache_q4");
    pkv::clear_error();
    return append<true>("rotate_and_cache_q4", key, key_stride, value, value_stride, query, query_stride, query_out,
                        query_out_stride, k_cache, v_cache, block_tables, seq_idx, pos, rotary_pos, rotary_table,
                        table_rows, rotary_dim, interleaved, slot_mapping, T, S, H, Hkv, D, bs, NB, MB, dtype, stream);
}

size_t pkv_cache_q4_row_bytes(int D) { return D == 64 || D == 128 ? (size_t)q4::row_bytes(D) : 0; }

pkv_status pkv_gather_cache_q4(void* key, int64_t key_stride, void* value, int64_t value_stride, const void* k_cache,
                               const void* v_cache, const int64_t* slot_mapping, int T, int Hkv, int D, int bs,
                               int NB, pkv_dtype dtype, void* stream) {
    PKV_TRACE("pkv_gather_cache_q4");
    pkv::clear_error();
    if (T < 0 || Hkv <= 0 || NB <= 0 || Hkv > 1 << 20 || (dtype != PKV_F16 && dtype != PKV_BF16))
        return pkv::fail(PKV_ERR_INVALID_ARG, "gather_cache_q4: bad size or dtype");
    if (!supported(D, bs))
        return pkv::fail(PKV_ERR_UNSUPPORTED, "gather_cache_q4: head_dim must be 64/128, block_size 8/16/32/64");
    if ((int64_t)NB * bs > INT32_MAX)
        return pkv::fail(PKV_ERR_INVALID_ARG, "gather_cache_q4: NB * bs must fit 31 bits");
    if (T == 0) return PKV_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping)
        return pkv::fail(PKV_ERR_INVALID_ARG, "gather_cache_q4: null pointer");
    if (!pkv::aligned16(key) || !pkv::aligned16(value) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache))
        return pkv::fail(PKV_ERR_INVALID_ARG, "gather_cache_q4: token and cache pointers must be 16-byte aligned");
    if (!stride_ok(key_stride, Hkv, D) || !stride_ok(value_stride, Hkv, D))
        return pkv::fail(PKV_ERR_INVALID_ARG,
                         "gather_cache_q4: token strides must be multiples of 8 elements, and a token's rows at least");
    const int64_t wide = (int64_t)Hkv * D * 2;
    if (overlap(key, 2 * key_stride, wide, value, 2 * value_stride, wide, T))
        return pkv::fail(PKV_ERR_INVALID_ARG, "gather_cache_q4: key and value overlap");
    GatherParams p;
    p.key = static_cast<char*>(key);
    p.value = static_cast<char*>(value);
    p.key_stride = 2 * key_stride;
    p.value_stride = 2 * value_stride;
    p.k_cache = static_cast<const char*>(k_cache);
    p.v_cache = static_cast<const char*>(v_cache);
    p.slots = slot_mapping;
    p.T = T;
    p.Hkv = Hkv;
    p.bs_log2 = log2_of(bs);
    p.num_slots = (int64_t)NB * bs;
    p.err = pkv::device_error_word();
    void (*fn)(GatherParams) = dtype == PKV_F16 ? (D == 128 ? gather_kernel<pkv::F16, 128> : gather_kernel<pkv::F16, 64>)
                                                : (D == 128 ? gather_kernel<pkv::BF16, 128> : gather_kernel<pkv::BF16, 64>);
    // few tokens: more CTAs for their heads
    const int64_t groups = ((int64_t)T + 7) / 8;
    const int passes = (16 * Hkv * (D / 16) + 255) / 256;
    p.splits = 1;
    while (p.splits * 2 <= passes && groups * p.splits * 2 <= 8 * pkv::sm_count()) p.splits *= 2;
    const cudaError_t e = launch(fn, groups * p.splits, 256, stream, p);
    return e == cudaSuccess ? PKV_OK : pkv::cuda_fail(e, "gather_cache_q4 launch");
}

}  // extern "C"
