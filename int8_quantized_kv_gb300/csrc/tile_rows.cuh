// tile_rows.cuh -- what the kernels over tiles of query rows (prompts, shared
// prefixes) have in common: the reference of a row's weights, the groups of a
// shared batch, rows of the three types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq8_device.cuh"
#include "kvq8_internal.cuh"
#include "kvq8_ptx.cuh"

namespace kvq8 {

// The four bf16 (or fp16) values in two words.
__device__ __forceinline__ float4 widen(uint32_t a, uint32_t b, int dtype) {
    if (dtype == KVQ8_DTYPE_BF16)
        return make_float4(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u), __uint_as_float(b << 16),
                           __uint_as_float(b & 0xffff0000u));
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    return make_float4(x.x, x.y, y.x, y.y);
}

// Brings the 128 values of a row from element i on into L2.
__device__ __forceinline__ void prefetch_l2(const void *base, int dtype, int64_t i) {
    const int size = dtype == KVQ8_DTYPE_F32 ? 4 : 2;
    bulk_prefetch_l2(static_cast<const char *>(base) + i * size, kHD * size);
}

__device__ __forceinline__ void store1(void *base, int dtype, int64_t i, float x) {
    if (dtype == KVQ8_DTYPE_F32) static_cast<float *>(base)[i] = x;
    else if (dtype == KVQ8_DTYPE_BF16) static_cast<__nv_bfloat16 *>(base)[i] = __float2bfloat16_rn(x);
    else static_cast<__half *>(base)[i] = __float2half_rn(x);
}

// A row's reference M: its operand P = 2^(s - M) * V scale has its maximum put between 2^7 and 2^9 when M is set; M moves
// (up, by a whole number) when P might pass 2^15.9 (fp16 ends below 2^16).  (A V scale counts as the next power of two.)
constexpr float kPTopLog2 = 9.0f, kPMaxLog2 = 15.9f;
// V scales below count as this (rows of zeros do).  Not lower: weights of up to 2^(15.9 + 90) still add up, a million of them.
// (Where V scales reach 2^x, weights below 2^-(134 - x) of a row's largest are lost: below fp32's normal numbers.)
constexpr int kTinyScaleLog2 = -90;

// The least whole number above log2 of a V scale (kTinyScaleLog2 at least), by its exponent bits.
__device__ __forceinline__ float exponent_above(float scale) {
    return __int_as_float(max(__float_as_int(scale) >> 23, kTinyScaleLog2 + 126) | 0x4b000000) - (0x1p23f + 126.0f);
}

// 2^d (d <= 0) as two factors, each a normal number where 2^d alone need not be: the sums of weights that it is for reach
// 2^126, and what is left of them after a move by more than 2^-126 still counts.
__device__ __forceinline__ float2 pow2_parts(float d) {
    const float whole = floorf(0.5f * fmaxf(d, -252.0f));
    return make_float2(ex2_approx(whole), ex2_approx(d - whole));   // (0 for d = -inf)
}

// Whether group entry g (0 .. n_groups) may be part of a cut of the batch.
__device__ __forceinline__ bool group_entry_ok(const TileParams &p, int g) {
    const int s = p.group_starts[g];
    if (g == 0) return s == 0;
    return s >= p.group_starts[g - 1] && (g < p.n_groups || s == p.batch);
}

// Tokens of row b that it shares with its group of `shared` tokens.
__device__ __forceinline__ int row_shared(const TileParams &p, int b, int shared, int cap) {
    const int L = max(0, min(p.ctx_lens[b], cap));
    return max(0, min(shared, p.step ? L - 1 : L));
}

}  // namespace kvq8
