// read.cu -- the K and V rows of given positions as the values their codes
// stand for: code * scale in fp32, rounded once to the output's type.
//
// Traffic bounds it: 264 B of cache and 2 * 128 values of output per (token, kv
// head); 8 x 4096 tokens x 8 heads to fp32 in 55.8 us (6.0 TB/s, 49.8 at the copy
// rate), 18000 tokens to bf16 in 22.3 (16.5).  A warp takes the 16 slots of a tile that one 16-byte access of a V
// row (dim-major per 64 slots) covers: lane l holds the codes of dims 4l..4l+3
// of all 16 tokens, V as one 16-byte load per dim turned by byte permutes, K as
// one word per token (the row's chunk j stands at j ^ (slot & 7)), so that every
// store of a token is a whole row of 128 values side by side.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq8_device.cuh"
#include "kvq8_internal.cuh"
#include "kvq8_ptx.cuh"

namespace kvq8 {
namespace {

constexpr int kReadSlots = 16;
constexpr int kReadWarps = 8;

// The codes in a word's four bytes as floats, times s.
__device__ __forceinline__ float4 code_values(uint32_t w, float s) {
    return make_float4((float)(int8_t)(w & 0xff) * s, (float)(int8_t)((w >> 8) & 0xff) * s,
                       (float)(int8_t)((w >> 16) & 0xff) * s, (float)(int8_t)(w >> 24) * s);
}

template <typename T>
__device__ __forceinline__ void put4(T *dst, float4 x);
template <>
__device__ __forceinline__ void put4<float>(float *dst, float4 x) {
    __stcs(reinterpret_cast<float4 *>(dst), x);
}
template <>
__device__ __forceinline__ void put4<__nv_bfloat16>(__nv_bfloat16 *dst, float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    __stcs(reinterpret_cast<uint2 *>(dst),
           make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b)));
}
template <>
__device__ __forceinline__ void put4<__half>(__half *dst, float4 x) {
    const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
    __stcs(reinterpret_cast<uint2 *>(dst),
           make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b)));
}

// Task = (sequence, 16-slot group, kv head), heads fastest.
template <typename T>
__global__ void __launch_bounds__(kReadWarps * 32)
read_kernel(ReadParams p, int groups) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t task = (int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5);
    const int h = (int)(task % p.nkv);
    const int64_t rest = task / p.nkv;
    const int b = (int)(rest / groups);
    if (b >= p.batch) return;
    const int n = p.n_tokens ? min(p.n_new, p.n_tokens[b]) : p.n_new;
    const int64_t start = p.start_pos[b], cap = (int64_t)p.max_blocks * kBS;
    // the group's slots are positions t0 .. t0 + 15, of which [lo, hi) are wanted
    const int64_t t0 = (start >> 4 << 4) + (rest % groups) * kReadSlots;
    int64_t lo = max(t0, start), hi = min(t0 + kReadSlots, start + n);
    if (lo >= hi) return;
    if (lo < 0 || hi > cap) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
        lo = max(lo, (int64_t)0);
        hi = min(hi, cap);
        if (lo >= hi) return;
    }
    const int phys = p.block_table[(size_t)b * p.max_blocks + t0 / kBS];
    if (phys < 0 || phys >= p.num_blocks) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
        return;
    }
    const size_t tile = (size_t)phys * p.nkv + h;
    const int slot0 = (int)(t0 % kBS);
    const int first = (int)(lo - t0), last = (int)(hi - t0);   // wanted: slots slot0 + [first, last)
    // element of the first wanted token's row, heads side by side
    const int64_t row0 = (int64_t)b * p.n_new + (lo - start);
    uint4 v[4];
    uint32_t k[kReadSlots];
    float scale = 0.0f;   // lane r: K scale of slot r; lane 16 + r: V scale
    if (p.v_out) {
        const int8_t *src = p.v_pool + tile * kHD * kBS + (size_t)(slot0 / kStageTok) * kTileVQuarter + slot0 % kStageTok;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __ldg(reinterpret_cast<const uint4 *>(src + (size_t)(4 * lane + i) * kStageTok));
        if (lane >= 16) scale = __ldg(p.v_scale + tile * kBS + slot0 + lane - 16);
    }
    if (p.k_out) {
        const int8_t *src = p.k_pool + (tile * kBS + slot0) * kHD;
#pragma unroll
        for (int r = 0; r < kReadSlots; ++r)
            k[r] = __ldg(reinterpret_cast<const uint32_t *>(src + r * kHD + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4));
        if (lane < 16) scale = __ldg(p.k_scale + tile * kBS + slot0 + lane);
    }
    if (p.k_out) {
        T *dst = static_cast<T *>(p.k_out) + row0 * p.k_stride + (size_t)h * kHD + 4 * lane;
#pragma unroll
        for (int r = 0; r < kReadSlots; ++r) {
            const float s = __shfl_sync(0xffffffffu, scale, r);
            if (r >= first && r < last) put4<T>(dst + (int64_t)(r - first) * p.k_stride, code_values(k[r], s));
        }
    }
    if (p.v_out) {
        T *dst = static_cast<T *>(p.v_out) + row0 * p.v_stride + (size_t)h * kHD + 4 * lane;
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // tokens 4q .. 4q + 3: a 4 x 4 block of bytes, turned
            const uint32_t w0 = q == 0 ? v[0].x : q == 1 ? v[0].y : q == 2 ? v[0].z : v[0].w;
            const uint32_t w1 = q == 0 ? v[1].x : q == 1 ? v[1].y : q == 2 ? v[1].z : v[1].w;
            const uint32_t w2 = q == 0 ? v[2].x : q == 1 ? v[2].y : q == 2 ? v[2].z : v[2].w;
            const uint32_t w3 = q == 0 ? v[3].x : q == 1 ? v[3].y : q == 2 ? v[3].z : v[3].w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t sel = (uint32_t)(i | ((4 + i) << 4));
                const uint32_t lo2 = __byte_perm(w0, w1, sel), hi2 = __byte_perm(w2, w3, sel);
                const int r = 4 * q + i;
                const float s = __shfl_sync(0xffffffffu, scale, 16 + r);
                if (r >= first && r < last)
                    put4<T>(dst + (int64_t)(r - first) * p.v_stride, code_values(__byte_perm(lo2, hi2, 0x5410), s));
            }
        }
    }
}

// 16-slot groups that n_new tokens may touch, wherever the first position lies in its group.
int64_t read_groups(int n_new) { return ((int64_t)n_new + 2 * kReadSlots - 2) / kReadSlots; }

int64_t read_blocks(const ReadParams &p) {
    // (at most 65535 * 65535 rows of 2^27 groups: below 2^63)
    const int64_t rows = (int64_t)p.batch * p.nkv, groups = read_groups(p.n_new);
    return (rows * groups + kReadWarps - 1) / kReadWarps;
}

template <typename T>
cudaError_t launch_read_t(const ReadParams &p, cudaStream_t s) {
    const int groups = (int)read_groups(p.n_new);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)read_blocks(p));
    cfg.blockDim = dim3(kReadWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, read_kernel<T>, p, groups);
}

}  // namespace

bool read_fits(const ReadParams &p) { return read_blocks(p) <= 2147483647; }

cudaError_t launch_read(const ReadParams &p, cudaStream_t s) {
    switch (p.dtype) {
        case KVQ8_DTYPE_F32: return launch_read_t<float>(p, s);
        case KVQ8_DTYPE_BF16: return launch_read_t<__nv_bfloat16>(p, s);
        default: return launch_read_t<__half>(p, s);
    }
}

}  // namespace kvq8
