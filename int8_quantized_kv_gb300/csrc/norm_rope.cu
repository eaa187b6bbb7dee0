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

constexpr int kTaskWarps = 4;             // warps per CTA, one task each
constexpr int kRunTok = 16;               // tokens per key/value task
constexpr int kGroupTok = 4;              // tokens of it loaded at once
constexpr int kQUnroll = 4;               // query heads of a task loaded at once
constexpr int kQueryTasks = 152 * 32;     // query tasks that fill the GPU

// A row x is held two ways.  Turned rows (queries, keys): lane l holds dims
// 2l, 2l + 1 (x, y) and 64 + 2l, 65 + 2l (z, w), so that both kinds of pairs,
// (i, i + 64) and (2i, 2i + 1), lie within a lane and turning needs no
// exchange.  Value rows: dims 4l..4l+3, as the append holds them.
__device__ __forceinline__ float2 load2(const float *p) { return __ldcs(reinterpret_cast<const float2 *>(p)); }
__device__ __forceinline__ float2 load2(const __half *p) {
    const uint32_t v = __ldcs(reinterpret_cast<const unsigned int *>(p));
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *p) {
    const uint32_t v = __ldcs(reinterpret_cast<const unsigned int *>(p));   // a bf16 is the high half of an fp32
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const float *p) { return __ldcs(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 load4(const __half *p) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ float4 load_turned(const T *row, int lane) {
    const float2 lo = load2(row + 2 * lane), hi = load2(row + kHD / 2 + 2 * lane);
    return make_float4(lo.x, lo.y, hi.x, hi.y);
}
// The weights of a lane's dims (1 without a norm).
__device__ __forceinline__ float4 load_weight(const float *w, int lane) {
    if (!w) return make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    const float2 lo = reinterpret_cast<const float2 *>(w)[lane], hi = reinterpret_cast<const float2 *>(w + kHD / 2)[lane];
    return make_float4(lo.x, lo.y, hi.x, hi.y);
}
// Cosine and sine of a lane's two pairs from a table row [cos 64 | sin 64]:
// (c.x, s.x) turns the first pair, (c.y, s.y) the second.
struct Turn {
    float2 c, s;
};
template <bool kPairs>
__device__ __forceinline__ Turn load_turn(const float *row, int lane) {
    if (kPairs) return {make_float2(row[lane], row[32 + lane]), make_float2(row[64 + lane], row[96 + lane])};
    return {reinterpret_cast<const float2 *>(row)[lane], reinterpret_cast<const float2 *>(row + kHD / 2)[lane]};
}
template <bool kPairs>
__device__ __forceinline__ float4 turned(float4 u, const Turn &t) {
    if (kPairs)
        return make_float4(u.x * t.c.x - u.y * t.s.x, u.y * t.c.x + u.x * t.s.x,
                           u.z * t.c.y - u.w * t.s.y, u.w * t.c.y + u.z * t.s.y);
    return make_float4(u.x * t.c.x - u.z * t.s.x, u.y * t.c.y - u.w * t.s.y,
                       u.z * t.c.x + u.x * t.s.x, u.w * t.c.y + u.y * t.s.y);
}

__device__ __forceinline__ float4 scaled(float4 x, float f) {
    return make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
}
__device__ __forceinline__ float sum_squares(float4 x) {
    return warp_sum(fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w))));
}

// x * r * w for the row's r = 1 / sqrt(mean(x^2) + eps).  Squares that
// overflow (|x| above about 2^60) are taken of x * 2^-64 instead.
__device__ __forceinline__ float4 normed(float4 x, float4 w, float eps) {
    float f = 1.0f;
    float ss = sum_squares(x);
    if (ss > 0x1p120f) {   // warp-uniform
        f = 0x1p-64f;
        x = scaled(x, f);
        ss = sum_squares(x);
    }
    x = scaled(x, rsqrtf(fmaf(ss, 1.0f / kHD, eps * f * f)));
    return make_float4(x.x * w.x, x.y * w.y, x.z * w.z, x.w * w.w);
}

// Largest |x| of a row held as four values per lane; a row with a NaN or an
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

// The codes of a key row from its inputs in 64 bits, for the values of `mask`
// (bit k: the lane's value k); x * w is exact there.
template <bool kPairs>
__device__ __noinline__ uint4 exact_codes(float4 x, float4 w, Turn t, uint4 codes, int mask) {
    const double ux = (double)x.x * w.x, uy = (double)x.y * w.y, uz = (double)x.z * w.z, uw = (double)x.w * w.w;
    double z[4];
    if (kPairs) {
        z[0] = ux * t.c.x - uy * t.s.x;
        z[1] = uy * t.c.x + ux * t.s.x;
        z[2] = uz * t.c.y - uw * t.s.y;
        z[3] = uw * t.c.y + uz * t.s.y;
    } else {
        z[0] = ux * t.c.x - uz * t.s.x;
        z[1] = uy * t.c.y - uw * t.s.y;
        z[2] = uz * t.c.x + ux * t.s.x;
        z[3] = uw * t.c.y + uy * t.s.y;
    }
    double top = fmax(fmax(fabs(z[0]), fabs(z[1])), fmax(fabs(z[2]), fabs(z[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (mask >> k & 1) c[k] = (uint32_t)__double2int_rn(127.0 * z[k] / top);
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// Codes (low bytes) of a key row y = turned x * r * w with maximum m > 0 and
// scale s: round_half_even(127 y* / max|y*|) of the exact values y*, whose
// common factor r cancels.  In units of eps = 2^-24 and Z = max|y*|: u = x r w
// carries two roundings (r's own cancels), the turn one of a product and one of
// the sum, and |u_a c| + |u_b s| <= |(u_a, u_b)| |(c, s)| <= sqrt(2) Z, so that
// y is within (3 sqrt(2) + 1) eps Z of y* and so is m of Z; 127 * rcp(m) adds 3
// eps.  127 y / m is then within 127 * 13.5 eps < 2^-13.2 of 127 y* / Z, and
// where its distance to the rounded value is at most 1/2 - 2^-13 that value is
// the code (t = fl(y * inv + 1.5 * 2^23) holds it in its low mantissa bits, as
// in kv_code_bytes4).  The others, 2^-12 of values and a value in 3 % of rows,
// are decided in 64 bits, as are rows whose range leaves the products' errors
// unbounded.
template <bool kPairs>
__device__ __forceinline__ uint4 key_codes(float4 y, float m, float s, float4 x, float4 w, const Turn &t) {
    if (s == 0.0f) return make_uint4(0u, 0u, 0u, 0u);   // warp-uniform
    constexpr float kShift = 0x1.8p23f;
    constexpr float kLim = 0.5f - 0x1p-13f;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(m));
    inv *= 127.0f;
    const float t0 = __fmaf_rn(y.x, inv, kShift), t1 = __fmaf_rn(y.y, inv, kShift);
    const float t2 = __fmaf_rn(y.z, inv, kShift), t3 = __fmaf_rn(y.w, inv, kShift);
    const float e0 = __fmaf_rn(y.x, inv, -__fsub_rn(t0, kShift)), e1 = __fmaf_rn(y.y, inv, -__fsub_rn(t1, kShift));
    const float e2 = __fmaf_rn(y.z, inv, -__fsub_rn(t2, kShift)), e3 = __fmaf_rn(y.w, inv, -__fsub_rn(t3, kShift));
    uint4 c = make_uint4(__float_as_uint(t0), __float_as_uint(t1), __float_as_uint(t2), __float_as_uint(t3));
    const bool wide = !(m >= 0x1p-100f && m <= 0x1p120f);
    const bool near = !((fabsf(e0) <= kLim) & (fabsf(e1) <= kLim) & (fabsf(e2) <= kLim) & (fabsf(e3) <= kLim));
    if (__any_sync(0xffffffffu, wide | near)) {
        const int mask = wide ? 15 : !(fabsf(e0) <= kLim) | !(fabsf(e1) <= kLim) << 1 | !(fabsf(e2) <= kLim) << 2 |
                                         !(fabsf(e3) <= kLim) << 3;
        c = exact_codes<kPairs>(x, w, t, c, mask);
    }
    return c;
}

// Writes a key row's codes, held as a turned row, to the row at dst of a slot.
__device__ __forceinline__ void store_key_codes(unsigned char *dst, int slot, int lane, uint4 c) {
    const int j = lane >> 3, at = 2 * (lane & 7);
    *reinterpret_cast<uint16_t *>(dst + ((j ^ (slot & 7)) << 4) + at) = (uint16_t)__byte_perm(c.x, c.y, 0x0040);
    *reinterpret_cast<uint16_t *>(dst + (((4 + j) ^ (slot & 7)) << 4) + at) = (uint16_t)__byte_perm(c.z, c.w, 0x0040);
}

// New tokens of sequence b (the rest of its n_new rows is padding).
__device__ __forceinline__ int token_count(const NormRopeParams &p, int b) {
    return p.n_tokens ? min(p.n_new, p.n_tokens[b]) : p.n_new;
}

// Key/value task w = (b * runs + x) * nkv + h: the new tokens of sequence b in
// run x of 16 cache slots, counted from the run of the first, of kv head h.
template <typename T, bool kPairs>
__device__ __forceinline__ void append_run(const NormRopeParams &p, int64_t w, int runs, int lane) {
    const int h = (int)(w % p.nkv);
    w /= p.nkv;
    const int b = (int)(w / runs);
    const int64_t cap = (int64_t)p.max_blocks * kBS;
    const int64_t start = p.start_pos[b];
    const int nt = token_count(p, b);
    // slots [r0, r0 + 16), of which tokens with positions in [lo, hi) are written
    const int64_t r0 = (start >= 0 ? start / kRunTok : -((-start + kRunTok - 1) / kRunTok)) * kRunTok +
                       (w % runs) * kRunTok;
    int64_t lo = max(start, r0), hi = min(start + nt, r0 + kRunTok);
    if (lo >= hi) return;
    if (lo < 0 || hi > cap) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
        lo = max(lo, (int64_t)0);
        hi = min(hi, cap);
        if (lo >= hi) return;
    }
    const int phys = p.block_table[(size_t)b * p.max_blocks + r0 / kBS];
    // lane r: the rotation position of the token in slot r0 + r
    const int64_t row0 = (int64_t)b * p.n_new + (r0 - start);   // row of the token in slot r0 (may precede the tensor)
    const bool mine = lane < kRunTok && r0 + lane >= lo && r0 + lane < hi;
    int64_t pos = 0;
    if (mine) pos = p.positions ? p.positions[row0 + lane] : r0 + lane;
    const bool good = mine && pos >= 0 && pos < p.n_pos;
    if (mine && !good) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
    if (phys < 0 || phys >= p.num_blocks) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
        return;
    }
    const unsigned todo = __ballot_sync(0xffffffffu, good);
    const size_t tile = (size_t)phys * p.nkv + h;
    const int slot0 = (int)(r0 % kBS);
    unsigned char *krow = reinterpret_cast<unsigned char *>(p.k_pool) + (tile * kBS + slot0) * kHD;
    int8_t *vrun = p.v_pool + tile * kHD * kBS + (size_t)(slot0 / kStageTok) * kTileVQuarter + slot0 % kStageTok;
    const T *ksrc = reinterpret_cast<const T *>(p.k) + (size_t)h * kHD;
    const T *vsrc = reinterpret_cast<const T *>(p.v) + (size_t)h * kHD + 4 * lane;
    const float4 weight = load_weight(p.k_weight, lane);
    const bool norm = p.k_weight != nullptr;

    if (todo == 0xffffu) {
        // the whole run, four tokens at a time
        uint32_t vw[4][kRunTok / 4];   // after group g, vw[i][3]: the codes of its tokens of dim 4 * lane + i
        float sc_keep = 0.0f;          // lane r < 16: K scale of row r; lane 16 + r: V scale
#pragma unroll 1
        for (int g = 0; g < kRunTok / kGroupTok; ++g) {
            float4 xk[kGroupTok], xv[kGroupTok];
            Turn tn[kGroupTok];
#pragma unroll
            for (int u = 0; u < kGroupTok; ++u) {
                const int r = kGroupTok * g + u;
                xk[u] = load_turned(ksrc + (row0 + r) * p.k_stride, lane);
                xv[u] = load4(vsrc + (row0 + r) * p.v_stride);
                tn[u] = load_turn<kPairs>(p.rope + (size_t)__shfl_sync(0xffffffffu, (int)pos, r) * kHD, lane);
            }
            uint32_t wg[4];
#pragma unroll
            for (int u = 0; u < kGroupTok; ++u) {
                const int r = kGroupTok * g + u;
                float4 y = turned<kPairs>(norm ? normed(xk[u], weight, p.eps) : xk[u], tn[u]);
                const float mk = row_max_checked(y, p.dev_status), sk = __fmul_rn(mk, KVQ8_INV127);
                store_key_codes(krow + r * kHD, r, lane, key_codes<kPairs>(y, mk, sk, xk[u], weight, tn[u]));
                const float sv = __fmul_rn(row_max_checked(xv[u], p.dev_status), KVQ8_INV127);
                const uint4 cv = kv_code_bytes4(xv[u], sv);
                if (lane == r) sc_keep = sk;
                if (lane == 16 + r) sc_keep = sv;
                constexpr uint32_t kIns[4] = {0x3210, 0x3240, 0x3410, 0x4210};
                if (u == 0) {
                    wg[0] = cv.x; wg[1] = cv.y; wg[2] = cv.z; wg[3] = cv.w;
                } else {
                    wg[0] = __byte_perm(wg[0], cv.x, kIns[u]);
                    wg[1] = __byte_perm(wg[1], cv.y, kIns[u]);
                    wg[2] = __byte_perm(wg[2], cv.z, kIns[u]);
                    wg[3] = __byte_perm(wg[3], cv.w, kIns[u]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                vw[i][0] = vw[i][1];
                vw[i][1] = vw[i][2];
                vw[i][2] = vw[i][3];
                vw[i][3] = wg[i];
            }
        }
        (lane < 16 ? p.k_scale : p.v_scale)[tile * kBS + slot0 + (lane & 15)] = sc_keep;
        if (p.weight_sum && lane < 16) p.weight_sum[tile * kBS + slot0 + lane] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4 *>(vrun + (size_t)(4 * lane + i) * kStageTok) =
                make_uint4(vw[i][0], vw[i][1], vw[i][2], vw[i][3]);
        return;
    }
    // part of a run: row by row
    for (unsigned left = todo; left; left &= left - 1) {
        const int r = __ffs(left) - 1;
        const float4 xk = load_turned(ksrc + (row0 + r) * p.k_stride, lane);
        float4 xv = load4(vsrc + (row0 + r) * p.v_stride);
        const Turn tn = load_turn<kPairs>(p.rope + (size_t)__shfl_sync(0xffffffffu, (int)pos, r) * kHD, lane);
        float4 y = turned<kPairs>(norm ? normed(xk, weight, p.eps) : xk, tn);
        const float mk = row_max_checked(y, p.dev_status), sk = __fmul_rn(mk, KVQ8_INV127);
        store_key_codes(krow + r * kHD, r, lane, key_codes<kPairs>(y, mk, sk, xk, weight, tn));
        const float sv = __fmul_rn(row_max_checked(xv, p.dev_status), KVQ8_INV127);
        const uint4 c = kv_code_bytes4(xv, sv);
        vrun[(size_t)(4 * lane + 0) * kStageTok + r] = (int8_t)c.x;
        vrun[(size_t)(4 * lane + 1) * kStageTok + r] = (int8_t)c.y;
        vrun[(size_t)(4 * lane + 2) * kStageTok + r] = (int8_t)c.z;
        vrun[(size_t)(4 * lane + 3) * kStageTok + r] = (int8_t)c.w;
        if (lane == 0) {
            p.k_scale[tile * kBS + slot0 + r] = sk;
            p.v_scale[tile * kBS + slot0 + r] = sv;
            if (p.weight_sum) p.weight_sum[tile * kBS + slot0 + r] = 0.0f;
        }
    }
}

// Query task w = row * parts + c: heads [c * hp, (c + 1) * hp) of a token.
template <typename T, bool kPairs>
__device__ __forceinline__ void turn_queries(const NormRopeParams &p, int64_t w, int hp, int lane) {
    const int parts = (p.nqh + hp - 1) / hp;
    const int64_t row = w / parts;
    const int h0 = (int)(w % parts) * hp, h1 = min(p.nqh, h0 + hp);
    const int b = (int)(row / p.n_new), i = (int)(row % p.n_new);
    if (p.n_tokens && i >= p.n_tokens[b]) return;   // padding
    const int64_t pos = p.positions ? p.positions[row] : (int64_t)p.start_pos[b] + i;
    if (pos < 0 || pos >= p.n_pos) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
        return;
    }
    const T *src = reinterpret_cast<const T *>(p.q) + row * p.q_stride;
    float *dst = p.q_out + row * p.nqh * kHD;
    const float4 weight = load_weight(p.q_weight, lane);
    const bool norm = p.q_weight != nullptr;
    const Turn tn = load_turn<kPairs>(p.rope + (size_t)pos * kHD, lane);
    for (int h = h0; h < h1; h += kQUnroll) {
        float4 x[kQUnroll];
#pragma unroll
        for (int u = 0; u < kQUnroll; ++u)
            if (h + u < h1) x[u] = load_turned(src + (size_t)(h + u) * kHD, lane);
#pragma unroll
        for (int u = 0; u < kQUnroll; ++u) {
            if (h + u < h1) {
                const float4 y = turned<kPairs>(norm ? normed(x[u], weight, p.eps) : x[u], tn);
                float *d = dst + (size_t)(h + u) * kHD + 2 * lane;
                *reinterpret_cast<float2 *>(d) = make_float2(y.x, y.y);
                *reinterpret_cast<float2 *>(d + kHD / 2) = make_float2(y.z, y.w);
            }
        }
    }
}

// One task per warp: first the key/value tasks, which are longer, then the
// query tasks.
template <typename T, bool kPairs>
__global__ void __launch_bounds__(kTaskWarps * 32)
norm_rope_append_kernel(NormRopeParams p, int runs, int hp) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t task = (int64_t)blockIdx.x * kTaskWarps + (threadIdx.x >> 5);
    const int64_t kv = (int64_t)p.batch * runs * p.nkv;
    if (task < kv) {
        append_run<T, kPairs>(p, task, runs, lane);
    } else if (task - kv < (int64_t)p.batch * p.n_new * ((p.nqh + hp - 1) / hp)) {
        turn_queries<T, kPairs>(p, task - kv, hp, lane);
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
    // runs of 16 slots that n_new consecutive positions touch, at most
    const int runs = (int)(((int64_t)p.n_new + kRunTok - 2) / kRunTok + 1);
    const int64_t rows = (int64_t)p.batch * p.n_new;
    // A query task takes one head while that leaves the GPU short of warps, and
    // up to 8 (which then share one turn and weight) when there are many.
    int hp = 1;
    while (hp < 8 && rows * p.nqh >= (int64_t)hp * 2 * kQueryTasks) hp *= 2;
    const int64_t tasks = (int64_t)p.batch * runs * p.nkv + rows * ((p.nqh + hp - 1) / hp);
    const int64_t blocks = (tasks + kTaskWarps - 1) / kTaskWarps;
    if (blocks > 2147483647) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kTaskWarps * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_append_kernel<T, kPairs>, p, runs, hp);
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
