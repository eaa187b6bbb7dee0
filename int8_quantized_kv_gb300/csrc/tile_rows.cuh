// tile_rows.cuh -- what the kernels over tiles of query rows (prompts, shared
// prefixes) have in common: where a row's query lies, the groups of a shared
// batch, rows of the three types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq8_device.cuh"
#include "kvq8_internal.cuh"

namespace kvq8 {

// Four consecutive values of a row of `dtype` from element i (a multiple of 4).
__device__ __forceinline__ float4 load4(const void *base, int dtype, int64_t i) {
    if (dtype == KVQ8_DTYPE_F32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + i);
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + i);
    if (dtype == KVQ8_DTYPE_BF16)
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                           __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void store1(void *base, int dtype, int64_t i, float x) {
    if (dtype == KVQ8_DTYPE_F32) static_cast<float *>(base)[i] = x;
    else if (dtype == KVQ8_DTYPE_BF16) static_cast<__nv_bfloat16 *>(base)[i] = __float2bfloat16_rn(x);
    else static_cast<__half *>(base)[i] = __float2half_rn(x);
}

// The group of row b: the last g with group_starts[g] <= b (of groups that are
// known to cut the batch).
__device__ __forceinline__ int group_of_row(const int32_t *starts, int n_groups, int b) {
    int lo = 0, hi = n_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= b) lo = mid;
        else hi = mid;
    }
    return lo;
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
