// Decode attention over a cache held in 4 bits (q4.cuh).
//
// One CTA takes one query head of one sequence; its warps take tokens in turn,
// D / 32 elements per lane, with a running maximum and sum per warp that are
// joined at the end.
#include <climits>
#include <cmath>
#include <cstdio>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "q4.cuh"

namespace {

namespace q4 = pkv::q4;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kMaxGroup = 16;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    char* out;
    const char* q;
    const char *k_cache, *v_cache;
    const int32_t *block_tables, *context_lens;
    int S, H, Hkv, G, NB, MB, bs_log2, max_ctx;
    float qscale;  // scale * log2(e)
    int* err;
};

// D / 32 elements of row `row` of a unit, elements D / 32 * lane and up.
template <class E, int D>
__device__ __forceinline__ void row_of(const char* unit, int row, int lane, float (&x)[D / 32]) {
    constexpr int N = D / 32;
    const int d = N * lane;
    const char* code = unit + row * q4::code_bytes(D) + 16 * q4::chunk_place<D>(row, d / 32) + d % 32 / 2;
    const float2 sm = E::to_float2(*reinterpret_cast<const uint32_t*>(unit + q4::kUnitCodes<D> +
                                                                      row * q4::pair_bytes(D) + 4 * (d / 64)));
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = fmaf(sm.x, (float)((((unsigned char)code[i / 2] >> (4 * (i & 1))) & 15) - 8), sm.y);
}

template <class E, int D>
__global__ void __launch_bounds__(32 * kWarps) attend_kernel(const __grid_constant__ Params p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = blockIdx.x / p.H, h = blockIdx.x % p.H, kvh = h / p.G;
    int n = p.context_lens[s];
    if (n < 0 || n > p.max_ctx) {
        if (h == 0 && threadIdx.x == 0) pkv::report(p.err, PKV_DEVERR_CONTEXT);
        n = n < 0 ? 0 : p.max_ctx;
    }
    const int64_t oh = ((int64_t)s * p.H + h) * D;
    float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 x = E::to_float2(*reinterpret_cast<const uint32_t*>(p.q + 2 * (oh + N * lane + i)));
        q[i] = x.x;
        q[i + 1] = x.y;
        o[i] = o[i + 1] = 0.f;
    }
    for (int j = warp; j < n; j += kWarps) {
        const int phys = p.block_tables[(int64_t)s * p.MB + (j >> p.bs_log2)];
        if ((unsigned)phys >= (unsigned)p.NB) {
            if (lane == 0) pkv::report(p.err, PKV_DEVERR_BLOCK_ID);
            continue;
        }
        const int slot = (phys << p.bs_log2) | (j & ((1 << p.bs_log2) - 1));
        const int64_t unit = q4::unit_at<D>(slot, kvh, p.Hkv, p.bs_log2);
        float k[N], v[N], z = 0.f;
        row_of<E, D>(p.k_cache + unit, slot & 7, lane, k);
        row_of<E, D>(p.v_cache + unit, slot & 7, lane, v);
#pragma unroll
        for (int i = 0; i < N; ++i) z = fmaf(q[i], k[i], z);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) z += __shfl_xor_sync(kFull, z, x);
        z *= p.qscale;
        const float m_new = fmaxf(m, z), use = m_new == -INFINITY ? 0.f : m_new;
        const float old = exp2f(m - use), w = exp2f(z - use);
        m = m_new;
        l = fmaf(l, old, w);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(w, v[i], o[i] * old);
    }
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
    s_m[warp] = m;
    s_l[warp] = l;
#pragma unroll
    for (int i = 0; i < N; ++i) s_o[warp][N * lane + i] = o[i];
    __syncthreads();
    if (warp != 0) return;
    float M = s_m[0];
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    const float use = M == -INFINITY ? 0.f : M;
    float L = 0.f, r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = 0.f;
    for (int w = 0; w < kWarps; ++w) {
        const float x = exp2f(s_m[w] - use);
        L = fmaf(x, s_l[w], L);
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = fmaf(x, s_o[w][N * lane + i], r[i]);
    }
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2)
        *reinterpret_cast<uint32_t*>(p.out + 2 * (oh + N * lane + i)) = E::from_float2(r[i] * inv, r[i + 1] * inv);
}

constexpr int kMaxContext = INT32_MAX - 1024;

bool workspace_args_ok(int S, int H, int Hkv, int D) {
    return S >= 0 && H > 0 && Hkv > 0 && H % Hkv == 0 && H / Hkv <= kMaxGroup && (D == 64 || D == 128);
}

}  // namespace

extern "C" {

size_t pkv_decode_q4_workspace_size(int S, int H, int Hkv, int D) {
    if (!workspace_args_ok(S, H, Hkv, D)) return 0;
    return 256;
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
    if (S > 32767 || (int64_t)S * H > INT32_MAX / 16)
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
    if (workspace_bytes < pkv_decode_q4_workspace_size(S, H, Hkv, D))
        return bad(PKV_ERR_WORKSPACE, "workspace too small");
    Params p;
    p.out = static_cast<char*>(out);
    p.q = static_cast<const char*>(q);
    p.k_cache = static_cast<const char*>(k_cache);
    p.v_cache = static_cast<const char*>(v_cache);
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
    p.qscale = scale * kLog2e;
    p.err = pkv::device_error_word();
    void (*fn)(Params) = dtype == PKV_F16 ? (D == 128 ? attend_kernel<pkv::F16, 128> : attend_kernel<pkv::F16, 64>)
                                          : (D == 128 ? attend_kernel<pkv::BF16, 128> : attend_kernel<pkv::BF16, 64>);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(S * H));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = pkv::as_stream(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    return e == cudaSuccess ? PKV_OK : pkv::cuda_fail(e, "paged_attention_decode_q4 launch");
}

}  // extern "C"
