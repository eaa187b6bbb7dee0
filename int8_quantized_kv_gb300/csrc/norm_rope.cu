// norm_rope.cu -- per-head norm of queries and keys, position rotation and
// quantise-append of K and V in one pass, and the rotation's table.
//
// A row x of 128 values (one token, one head) becomes
//   r = 1 / sqrt(mean(x^2) + eps), u = x * r * w (u = x without a weight),
//   y_a = u_a cos - u_b sin, y_b = u_b cos + u_a sin
// for the pairs (a, b) = (i, i + 64) or (2i, 2i + 1).  A query row is written
// in fp32; a key row goes to the int8 cache with scale = max|y| * (1/127) and code
// = round_half_even(127 y / max|y|).  The code is that of the exact values: r
// is common to the row and cancels, and where fp32 cannot tell on which side
// of a border 127 y / max|y| lies, 64 bits decide.  A value row is quantised
// by the append's own rule, but that both scales are the product with the
// rounded 1/127 (as the query blocks'), not a division.
#include "kvq8_device.cuh"
#include "kvq8_internal.cuh"
#include "kvq8_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace kvq8 {
namespace {

constexpr int kRowWarps = 8;   // warps per CTA, one row each

// Largest |x| of a row held as a float4 per lane; a row with a NaN or an
// infinity is cleared and flagged, and its maximum is 0.
__device__ __forceinline__ float row_max_checked(float4 &x, uint32_t *status) {
    const uint32_t a = max(max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu),
                           max(__float_as_uint(x.z) & 0x7fffffffu, __float_as_uint(x.w) & 0x7fffffffu));
    const uint32_t m = __reduce_max_sync(0xffffffffu, a);
    if (m >= 0x7f800000u) {   // warp-uniform
        x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if ((threadIdx.x & 31) == 0) flag_status(status, KVQ8_DEV_NONFINITE);
        return 0.0f;
    }
    return __uint_as_float(m);
}

// Four consecutive values of a row.
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __half *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);   // a bf16 is the high half of an fp32
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}

__device__ __forceinline__ float4 scaled(float4 x, float f) {
    return make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
}
__device__ __forceinline__ float4 times(float4 x, float4 w) {
    return make_float4(x.x * w.x, x.y * w.y, x.z * w.z, x.w * w.w);
}

// x * r for the row's r = 1 / sqrt(mean(x^2) + eps).  Squares that overflow
// (|x| above about 2^60) are taken of x * 2^-64 instead.
__device__ __forceinline__ float4 normed(float4 x, float eps) {
    float f = 1.0f;
    float ss = warp_sum(fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w))));
    if (ss > 0x1p120f) {   // warp-uniform
        f = 0x1p-64f;
        x = scaled(x, f);
        ss = warp_sum(fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w))));
    }
    return scaled(x, rsqrtf(fmaf(ss, 1.0f / kHD, eps * f * f)));
}

// The rotation of a row held as dims 4l..4l+3 in lane l.  Halves: lane l and
// lane l ^ 16 hold the two ends of the same pairs; pairs: both ends are in the
// lane.  cs, sn: cosines and sines of the lane's values (see load_turn).
template <bool kPairs>
__device__ __forceinline__ float4 rotated(float4 u, float4 cs, float4 sn, int lane) {
    if (kPairs)
        return make_float4(u.x * cs.x - u.y * sn.x, u.y * cs.x + u.x * sn.x,
                           u.z * cs.y - u.w * sn.y, u.w * cs.y + u.z * sn.y);
    float4 o;
    o.x = __shfl_xor_sync(0xffffffffu, u.x, 16);
    o.y = __shfl_xor_sync(0xffffffffu, u.y, 16);
    o.z = __shfl_xor_sync(0xffffffffu, u.z, 16);
    o.w = __shfl_xor_sync(0xffffffffu, u.w, 16);
    const float f = lane < 16 ? -1.0f : 1.0f;
    return make_float4(u.x * cs.x + o.x * (f * sn.x), u.y * cs.y + o.y * (f * sn.y),
                       u.z * cs.z + o.z * (f * sn.z), u.w * cs.w + o.w * (f * sn.w));
}

// The same in 64 bits, of x * w.
template <bool kPairs>
__device__ __forceinline__ void rotated64(float4 x, float4 w, float4 cs, float4 sn, int lane, double (&z)[4]) {
    double u[4] = {(double)x.x * w.x, (double)x.y * w.y, (double)x.z * w.z, (double)x.w * w.w};
    if (kPairs) {
        z[0] = u[0] * cs.x - u[1] * sn.x;
        z[1] = u[1] * cs.x + u[0] * sn.x;
        z[2] = u[2] * cs.y - u[3] * sn.y;
        z[3] = u[3] * cs.y + u[2] * sn.y;
        return;
    }
    const double f = lane < 16 ? -1.0 : 1.0;
    const float c[4] = {cs.x, cs.y, cs.z, cs.w}, s[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double o = __shfl_xor_sync(0xffffffffu, u[i], 16);
        z[i] = u[i] * c[i] + o * (f * s[i]);
    }
}

// Cosines and sines of the lane's values from a table row [cos 64 | sin 64].
template <bool kPairs>
__device__ __forceinline__ void load_turn(const float *row, int lane, float4 &cs, float4 &sn) {
    if (kPairs) {
        const float2 c = reinterpret_cast<const float2 *>(row)[lane];
        const float2 s = reinterpret_cast<const float2 *>(row + kHD / 2)[lane];
        cs = make_float4(c.x, c.y, 0.0f, 0.0f);
        sn = make_float4(s.x, s.y, 0.0f, 0.0f);
    } else {
        cs = reinterpret_cast<const float4 *>(row)[lane & 15];
        sn = reinterpret_cast<const float4 *>(row + kHD / 2)[lane & 15];
    }
}

// One warp per (new token, head): query heads, then key heads, then value heads.
template <typename T, bool kPairs>
__global__ void __launch_bounds__(kRowWarps * 32)
norm_rope_append_kernel(NormRopeParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int heads = p.nqh + 2 * p.nkv;
    const int64_t task = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (task >= (int64_t)p.batch * p.n_new * heads) return;
    const int64_t row = task / heads;
    int head = (int)(task % heads);
    const int b = (int)(row / p.n_new), i = (int)(row % p.n_new);
    if (p.n_tokens && i >= p.n_tokens[b]) return;   // padding
    const int64_t slot_pos = (int64_t)p.start_pos[b] + i;
    const int64_t pos = p.positions ? p.positions[row] : slot_pos;
    if (pos < 0 || pos >= p.n_pos) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
        return;
    }
    const bool is_q = head < p.nqh, is_k = !is_q && head < p.nqh + p.nkv;
    const T *src = reinterpret_cast<const T *>(is_q ? p.q : is_k ? p.k : p.v) +
                   row * (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride);
    if (!is_q) head -= is_k ? p.nqh : p.nqh + p.nkv;
    float4 x = load4(src + (size_t)head * kHD + 4 * lane);

    float4 y, w = make_float4(1.0f, 1.0f, 1.0f, 1.0f), cs, sn;
    if (is_q || is_k) {
        const float *weight = is_q ? p.q_weight : p.k_weight;
        load_turn<kPairs>(p.rope + (size_t)pos * kHD, lane, cs, sn);
        y = x;
        if (weight) {
            w = load4(weight + 4 * lane);
            y = times(normed(x, p.eps), w);
        }
        y = rotated<kPairs>(y, cs, sn, lane);
        if (is_q) {
            *reinterpret_cast<float4 *>(p.q_out + (row * p.nqh + head) * kHD + 4 * lane) = y;
            return;
        }
    }
    if (slot_pos < 0 || slot_pos >= (int64_t)p.max_blocks * kBS) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
        return;
    }
    const int phys = p.block_table[(size_t)b * p.max_blocks + slot_pos / kBS];
    if (phys < 0 || phys >= p.num_blocks) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
        return;
    }
    const int slot = (int)(slot_pos % kBS);
    const size_t tile = (size_t)phys * p.nkv + head;
    if (is_k) {
        const float s = __fmul_rn(row_max_checked(y, p.dev_status), KVQ8_INV127);
        int code[4] = {0, 0, 0, 0};
        if (s > 0.0f) {   // warp-uniform
            double z[4];
            rotated64<kPairs>(x, w, cs, sn, lane, z);
            double top = fmax(fmax(fabs(z[0]), fabs(z[1])), fmax(fabs(z[2]), fabs(z[3])));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
            for (int k = 0; k < 4; ++k) code[k] = __double2int_rn(127.0 * z[k] / top);
        }
        unsigned char *dst = reinterpret_cast<unsigned char *>(p.k_pool) + (tile * kBS + slot) * kHD;
        reinterpret_cast<uint32_t *>(dst + (((lane >> 2) ^ (slot & 7)) << 4))[lane & 3] =
            low_bytes4(make_uint4(code[0], code[1], code[2], code[3]));
        if (lane == 0) {
            p.k_scale[tile * kBS + slot] = s;
            if (p.weight_sum) p.weight_sum[tile * kBS + slot] = 0.0f;
        }
    } else {
        const float s = __fmul_rn(row_max_checked(x, p.dev_status), KVQ8_INV127);
        const uint4 c = kv_code_bytes4(x, s);
        int8_t *vg = p.v_pool + tile * kHD * kBS + (size_t)(slot / kStageTok) * kTileVQuarter + slot % kStageTok;
        vg[(size_t)(4 * lane + 0) * kStageTok] = (int8_t)c.x;
        vg[(size_t)(4 * lane + 1) * kStageTok] = (int8_t)c.y;
        vg[(size_t)(4 * lane + 2) * kStageTok] = (int8_t)c.z;
        vg[(size_t)(4 * lane + 3) * kStageTok] = (int8_t)c.w;
        if (lane == 0) p.v_scale[tile * kBS + slot] = s;
    }
}

// Table row of position t: cos(t f_i) and sin(t f_i) of the 64 frequencies,
// computed in 64 bits (an angle of 10^5 radians keeps 11 digits) and rounded
// once.
__global__ void __launch_bounds__(256)
rope_table_kernel(const double *inv_freq, int64_t n, float *table) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t t = i / (kHD / 2);
    const int f = (int)(i % (kHD / 2));
    double s, c;
    sincos((double)t * inv_freq[f], &s, &c);
    table[t * kHD + f] = (float)c;
    table[t * kHD + kHD / 2 + f] = (float)s;
}

template <typename T, bool kPairs>
cudaError_t launch_rows(const NormRopeParams &p, cudaStream_t s) {
    const int64_t tasks = (int64_t)p.batch * p.n_new * (p.nqh + 2 * p.nkv);
    const int64_t blocks = (tasks + kRowWarps - 1) / kRowWarps;
    if (blocks > 2147483647) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kRowWarps * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_append_kernel<T, kPairs>, p);
}

template <typename T>
cudaError_t launch_t(const NormRopeParams &p, cudaStream_t s) {
    return p.pairs ? launch_rows<T, true>(p, s) : launch_rows<T, false>(p, s);
}

}  // namespace

cudaError_t launch_norm_rope_append(const NormRopeParams &p, cudaStream_t s) {
    switch (p.dtype) {
        case KVQ8_DTYPE_F32: return launch_t<float>(p, s);
        case KVQ8_DTYPE_BF16: return launch_t<__nv_bfloat16>(p, s);
        case KVQ8_DTYPE_F16: return launch_t<__half>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_rope_table(const double *inv_freq, int64_t n_pos, float *table, cudaStream_t s) {
    const int64_t n = n_pos * (kHD / 2);
    rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(inv_freq, n, table);
    return cudaGetLastError();
}

}  // namespace kvq8
