// The cache held in 4 bits: what its writer (rotary.cu) and its readers
// (rotary.cu, q4_decode.cu) share.
//
// Element i of a row's group of 64 stands for centre + step * (code - 8), code
// 0..15, with step = (max - min) / 15 and centre = (8 max + 7 min) / 15 of the
// group, each rounded once to the model's 16-bit type: the 16 values run from
// min to max.  A group of 64 costs half a bit per element (step and centre).
//
// A pool is [NB][Hkv][bs][RB] bytes, RB = D/2 + D/16, K and V apart: all tokens
// of a (block, head) are one run, so that a reader that takes one head copies it
// in one piece.  It is made of units of 8 tokens:
//   8 rows of D/2 code bytes: byte j of a row holds elements 2j (low nibble) and
//     2j + 1; the row's 16-byte chunks (32 elements) are permuted by
//     chunk_place, so that eight rows' chunk c lie in different banks of shared
//     memory when a unit is copied there as it is;
//   8 rows of D/64 pairs (step, centre).
// A unit is 288 or 576 bytes, a multiple of 16: what the asynchronous bulk copy
// wants.
#pragma once

#include <cstdint>

#include "pkv_device.cuh"

namespace pkv {
namespace q4 {

constexpr int kGroup = 64;  // elements that share a step and a centre
constexpr int kUnit = 8;    // tokens of a unit

__host__ __device__ constexpr int code_bytes(int D) { return D / 2; }  // of one row
__host__ __device__ constexpr int pair_bytes(int D) { return D / kGroup * 4; }
__host__ __device__ constexpr int row_bytes(int D) { return code_bytes(D) + pair_bytes(D); }
template <int D>
constexpr int kUnitBytes = kUnit * row_bytes(D);
template <int D>
constexpr int kUnitCodes = kUnit * code_bytes(D);

// The greatest of three (a NaN only where all are).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// The least and the greatest; NaN where one is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float d;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// 1 / x to an ulp.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Where row r (0..7) of a unit has its 16-byte chunk c.
template <int D>
__device__ __forceinline__ int chunk_place(int r, int c) {
    return D == 128 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1);
}

// First byte of the unit with token `slot` of head h.  slot = block * bs +
// offset < 2^31.
template <int D>
__device__ __forceinline__ int64_t unit_at(int slot, int h, int Hkv, int bs_log2) {
    const int block = slot >> bs_log2, off = slot & ((1 << bs_log2) - 1);
    return ((((int64_t)block * Hkv + h) << (bs_log2 - 3)) + (off >> 3)) * kUnitBytes<D>;
}

}  // namespace q4
}  // namespace pkv
