// norm_rope.cu -- per-head norm of queries and keys, position rotation and
// quantise-append of K and V in one pass, and the rotation's table.
//
// A row x of 128 values (one token, one head) becomes
//   r = 1 / sqrt(mean(x^2) + eps), u = x * r * w (u = x without a weight),
//   y_a = u_a cos - u_b sin, y_b = u_b cos + u_a sin
// for the pairs (a, b) = (i, i + 64) or (2i, 2i + 1).  A query row is written
// in fp32; a key row goes to the int8 cache with scale = max|y| * (1/127) and
// code = round_half_even(127 y / max|y|).  The code is that of the exact
// values: r is common to the row and cancels, and where fp32 cannot tell on
// which side of a border 127 y / max|y| lies, 64 bits decide.  A value row is
// quantised by the append's own rule, but that both scales are the product
// with the rounded 1/127 (as the query blocks'), not a division.
//
// Two kinds of warp tasks, the first kind before the second in the grid (which
// measured 2 % faster than the two mixed evenly, and than the other order):
//  * turn tasks: up to four heads at a time of one token, eight lanes to a
//    row.  With 16 values a lane, a row's sum and maximum take three exchanges
//    instead of five, shared by four rows, and the table row is loaded once
//    for all heads of the task.
//  * value tasks: the new tokens of a run of 16 (or 4) cache slots of one kv
//    head, a warp to a row, since V is stored with 64 tokens of a dim side by
//    side: lane l gathers the codes of its 4 dims over the run and writes them
//    as one 16-byte (4-byte) piece each.
#include "kvq8_device.cuh"
#include "kvq8_internal.cuh"
#include "kvq8_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace kvq8 {
namespace {

constexpr int kTaskWarps = 4;             // warps per CTA, one task each
constexpr int kMinCtas = 6;               // CTAs per SM
constexpr int kDepth = 3;                 // stages of a warp's ring
// Tasks from which on the GPU counts as full: a threshold that was measured, 4/3
// of the 24 warps that each of 152 SMs holds of this kernel.
constexpr int kFullTasks = 152 * 32;
constexpr int kMostGroups = 8;            // groups of four heads per turn task
// Value tasks of 16 slots from which on they are used, without and with
// padding (which leaves some of them empty): 6 x 1111 tokens of bf16 take 41 us
// with them and 46 with tasks of 4 slots, 8 x 4096 of fp32 134 and 180, but 6
// padded prompts of 1 to 1111 tokens 31 and 27.  Below, the four times shorter
// tasks have the lower latency.
constexpr int kLongRuns = kFullTasks / 3, kLongRunsPadded = kFullTasks;

// ------------------------------------------------------------- conversion --
__device__ __forceinline__ float2 pair_of(uint32_t v, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
__device__ __forceinline__ float2 pair_of(uint32_t v, __nv_bfloat16) {   // a bf16 is the high half of an fp32
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 load2(const float *p) { return *reinterpret_cast<const float2 *>(p); }
template <typename T>
__device__ __forceinline__ float2 load2(const T *p) { return pair_of(*reinterpret_cast<const uint32_t *>(p), T()); }
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <typename T>
__device__ __forceinline__ float4 load4(const T *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const float2 a = pair_of(v.x, T()), b = pair_of(v.y, T());
    return make_float4(a.x, a.y, b.x, b.y);
}

// ------------------------------------------------------------- turn tasks --
// Eight lanes to a row: lane j (of 8) holds dims 32c + 4j + i in x[4c + i] (i <
// 4, c < 4).  Both kinds of pairs lie within a lane, and the eight lanes read
// or write whole sectors of the row at a time.  (With 8 consecutive values a
// lane every access touches half a sector, and the ring below made 8 x 4096
// tokens slower, 165 -> 190 us, where it now takes 155 to 137.)
template <typename T>
__device__ __forceinline__ void load_row(const T *row, int j, float (&x)[16]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float4 v = load4(row + 32 * c + 4 * j);
        x[4 * c] = v.x;
        x[4 * c + 1] = v.y;
        x[4 * c + 2] = v.z;
        x[4 * c + 3] = v.w;
    }
}
// The rows of a turn task (four at a time, one stage) and of a value task (four
// rows, one stage) pass through a ring of kDepth stages in shared memory, of
// which kDepth - 1 are in flight: what bounds the turn tasks is how many bytes
// 24 warps keep in flight (2 KiB a warp: 79 % of the copy peak; 4 KiB: 96 %).
// A lane copies the pieces that it reads back itself, [piece][lane], so that
// its own copy groups order everything and the warp needs no barrier.
template <typename T>
__host__ __device__ constexpr int stage_bytes() {
    return 4 * kHD * (int)sizeof(T);
}
__device__ __forceinline__ void copy4(void *dst, const float *src) { cp_async16_cg(dst, src); }
template <typename T>
__device__ __forceinline__ void copy4(void *dst, const T *src) { cp_async8(dst, src); }
template <typename T>
__device__ __forceinline__ void fetch_row(unsigned char *stage, const T *row, int j, int lane) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        copy4(stage + (c * 32 + lane) * 4 * (int)sizeof(T), row + 32 * c + 4 * j);
}
template <typename T>
__device__ __forceinline__ void read_row(const unsigned char *stage, int lane, float (&x)[16]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float4 v = load4(reinterpret_cast<const T *>(stage) + (c * 32 + lane) * 4);
        x[4 * c] = v.x;
        x[4 * c + 1] = v.y;
        x[4 * c + 2] = v.z;
        x[4 * c + 3] = v.w;
    }
}
// Cosines and sines of the lane's eight pairs from a table row [cos 64 | sin
// 64]: pairs (x[e], x[8+e]), or (x[2e], x[2e+1]) for e < 8.
template <bool kPairs>
__device__ __forceinline__ void load_turn(const float *row, int j, float (&c)[8], float (&s)[8]) {
    if (kPairs) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 a = *reinterpret_cast<const float2 *>(row + 16 * q + 2 * j);
            const float2 b = *reinterpret_cast<const float2 *>(row + kHD / 2 + 16 * q + 2 * j);
            c[2 * q] = a.x; c[2 * q + 1] = a.y;
            s[2 * q] = b.x; s[2 * q + 1] = b.y;
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const float4 a = *reinterpret_cast<const float4 *>(row + 32 * q + 4 * j);
        const float4 b = *reinterpret_cast<const float4 *>(row + kHD / 2 + 32 * q + 4 * j);
        c[4 * q] = a.x; c[4 * q + 1] = a.y; c[4 * q + 2] = a.z; c[4 * q + 3] = a.w;
        s[4 * q] = b.x; s[4 * q + 1] = b.y; s[4 * q + 2] = b.z; s[4 * q + 3] = b.w;
    }
}
template <bool kPairs>
__device__ __forceinline__ void turn(float (&u)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float &a = u[kPairs ? 2 * e : e], &b = u[kPairs ? 2 * e + 1 : 8 + e];
        const float ya = fmaf(a, c[e], -(b * s[e])), yb = fmaf(b, c[e], a * s[e]);
        a = ya;
        b = yb;
    }
}
__device__ __forceinline__ void weighted(float (&x)[16], const float *w, int j) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float4 v = *reinterpret_cast<const float4 *>(w + 32 * c + 4 * j);
        x[4 * c] *= v.x;
        x[4 * c + 1] *= v.y;
        x[4 * c + 2] *= v.z;
        x[4 * c + 3] *= v.w;
    }
}
// Over the eight lanes of a row.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_squares(const float (&x)[16]) {
    float a = x[0] * x[0], b = x[1] * x[1];
#pragma unroll
    for (int e = 2; e < 16; e += 2) {
        a = fmaf(x[e], x[e], a);
        b = fmaf(x[e + 1], x[e + 1], b);
    }
    return row_sum(a + b);
}
// The same of x * f.
__device__ __forceinline__ float row_squares(const float (&x)[16], float f) {
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        a = fmaf(x[e] * f, x[e] * f, a);
        b = fmaf(x[e + 1] * f, x[e + 1] * f, b);
    }
    return row_sum(a + b);
}
constexpr float kMostSquares = 0x1p120f;

// Where a token's keys go: the tile of kv head 0 and the slot; tile < 0: nowhere.
struct KeyPlace {
    int64_t tile;
    int slot;
};
__device__ __forceinline__ KeyPlace key_place(const NormRopeParams &p, int b, int64_t at, int lane) {
    KeyPlace k = {-1, 0};
    if (at < 0 || at >= (int64_t)p.max_blocks * kBS) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
        return k;
    }
    const int phys = p.block_table[(size_t)b * p.max_blocks + at / kBS];
    if (phys < 0 || phys >= p.num_blocks) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
        return k;
    }
    k.tile = (int64_t)phys * p.nkv;
    k.slot = (int)(at % kBS);
    return k;
}

// round_half_even(127 z / top) for |z| <= top without a division: the nearest
// integer by fp32, which is at most one off, moved by the exact remainder.
__device__ __forceinline__ uint32_t exact_code(double z, double top, float inv) {
    const double v = 127.0 * z;
    int k = __float2int_rn((float)v * inv);
    const double d = fma(-(double)k, top, v), half = 0.5 * top;
    if (d > half || (d == half && (k & 1))) ++k;
    else if (d < -half || (d == -half && (k & 1))) --k;
    return (uint32_t)k;
}

// A key row of kv head h by the whole warp in 64 bits (x * w is exact there),
// lane l holding dims 2l, 2l + 1, 64 + 2l, 65 + 2l.  sc: the row's scale, or
// negative: the scale is found here too, for rows that fp32 cannot hold
// (squares or products beyond its range, a NaN or an infinity: stored as zeros
// and flagged).
template <typename T, bool kPairs>
__device__ __noinline__ void exact_key_row(const NormRopeParams &p, int64_t row, int64_t pos, int h, KeyPlace at,
                                           float sc, int lane) {
    const T *src = reinterpret_cast<const T *>(p.k) + row * p.k_stride + (size_t)h * kHD;
    const float2 x0 = load2(src + 2 * lane), x1 = load2(src + kHD / 2 + 2 * lane);
    const double x[4] = {x0.x, x0.y, x1.x, x1.y};
    double u[4] = {x[0], x[1], x[2], x[3]};
    if (p.k_weight) {
        const float2 w0 = load2(p.k_weight + 2 * lane), w1 = load2(p.k_weight + kHD / 2 + 2 * lane);
        u[0] *= w0.x;
        u[1] *= w0.y;
        u[2] *= w1.x;
        u[3] *= w1.y;
    }
    const float *t = p.rope + (size_t)pos * kHD;
    double z[4];
    if (kPairs) {
        const double c0 = t[lane], c1 = t[32 + lane], s0 = t[64 + lane], s1 = t[96 + lane];
        z[0] = u[0] * c0 - u[1] * s0;
        z[1] = u[1] * c0 + u[0] * s0;
        z[2] = u[2] * c1 - u[3] * s1;
        z[3] = u[3] * c1 + u[2] * s1;
    } else {
        const float2 c = load2(t + 2 * lane), s = load2(t + kHD / 2 + 2 * lane);
        z[0] = u[0] * c.x - u[2] * s.x;
        z[1] = u[1] * c.y - u[3] * s.y;
        z[2] = u[2] * c.x + u[0] * s.x;
        z[3] = u[3] * c.y + u[1] * s.y;
    }
    double top = fmax(fmax(fabs(z[0]), fabs(z[1])), fmax(fabs(z[2]), fabs(z[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (sc < 0.0f && top == 0.0) {   // warp-uniform: a row of zeros (or of NaN, see below)
        sc = 0.0f;
    } else if (sc < 0.0f) {
        double r = 1.0;
        if (p.k_weight) {
            double ss = x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = 1.0 / sqrt(ss / kHD + (double)p.eps);
        }
        sc = __fmul_rn((float)(top * r), KVQ8_INV127);
    }
    // a NaN or an infinity among the inputs, or a value beyond fp32
    bool bad = !(sc < INFINITY);
#pragma unroll
    for (int k = 0; k < 4; ++k) bad |= !isfinite(z[k]);
    if (__any_sync(0xffffffffu, bad)) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_NONFINITE);
        sc = 0.0f;
    }
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    if (sc > 0.0f) {
        // z and top brought near 1 by a power of two (top's exponent), which fp32 needs for its candidate
        const double f = __hiloint2double((2046 << 20) - (__double2hiint(top) & 0x7ff00000), 0);
        const float inv = 1.0f / (float)(top * f);
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = exact_code(z[k] * f, top * f, inv);
    }
    const size_t place = (size_t)(at.tile + h) * kBS + at.slot;
    unsigned char *dst = reinterpret_cast<unsigned char *>(p.k_pool) + place * kHD;
    const int chunk = lane >> 3, byte = 2 * (lane & 7);
    *reinterpret_cast<uint16_t *>(dst + ((chunk ^ (at.slot & 7)) << 4) + byte) = (uint16_t)__byte_perm(c[0], c[1], 0x0040);
    *reinterpret_cast<uint16_t *>(dst + (((4 + chunk) ^ (at.slot & 7)) << 4) + byte) =
        (uint16_t)__byte_perm(c[2], c[3], 0x0040);
    if (lane == 0) {
        p.k_scale[place] = sc;
        if (p.weight_sum) p.weight_sum[place] = 0.0f;
    }
}

// Stores the codes t[16] (low bytes) and the scale of a lane's part of a key row.
__device__ __forceinline__ void store_codes(const NormRopeParams &p, const uint32_t (&t)[16], float sc, int h,
                                            KeyPlace at, int j) {
    const size_t place = (size_t)(at.tile + h) * kBS + at.slot;
    unsigned char *dst = reinterpret_cast<unsigned char *>(p.k_pool) + place * kHD + 4 * (j & 3);
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint32_t *>(dst + (((2 * c + (j >> 2)) ^ (at.slot & 7)) << 4)) =
            low_bytes4(make_uint4(t[4 * c], t[4 * c + 1], t[4 * c + 2], t[4 * c + 3]));
    if (j == 0) {
        p.k_scale[place] = sc;
        if (p.weight_sum) p.weight_sum[place] = 0.0f;
    }
}

// a + b = sum + err exactly.
__device__ __forceinline__ float2 two_sum(float a, float b) {
    const float t = __fadd_rn(a, b), v = __fsub_rn(t, a);
    return make_float2(t, __fadd_rn(__fsub_rn(a, __fsub_rn(t, v)), __fsub_rn(b, v)));
}

// (h + l) * g, and a + b, as pairs hi + lo of fp32.
__device__ __forceinline__ float2 pair_times(float h, float l, float g) {
    const float t = __fmul_rn(h, g);
    return make_float2(t, __fmaf_rn(l, g, __fmaf_rn(h, g, -t)));
}
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
    const float2 t = two_sum(a.x, b.x);
    return two_sum(t.x, __fadd_rn(t.y, __fadd_rn(a.y, b.y)));
}

// round_half_even(127 z / m) of pairs z = zh + zl and m = mh + ml >= |z|, inv
// near 127 / m; `open` is set where 127 z / m is within 2^-34 of a border.
// With z and m within 12 * 2^-48 m of the exact values the others are theirs.
__device__ __forceinline__ uint32_t pair_code(float zh, float zl, float mh, float ml, float inv, bool &open) {
    // k = the nearest integer or next to it; d = 127 z - k m
    float k = rintf(__fmul_rn(zh, inv));
    const float p1 = __fmul_rn(127.0f, zh), e1 = __fmaf_rn(127.0f, zh, -p1);
    const float p2 = __fmul_rn(k, mh), e2 = __fmaf_rn(k, mh, -p2);
    const float2 d = two_sum(p1, -p2);
    const float dl = __fadd_rn(__fadd_rn(d.y, __fsub_rn(e1, e2)), __fsub_rn(__fmul_rn(127.0f, zl), __fmul_rn(k, ml)));
    // its distances above m/2 and above -m/2
    const float up = __fadd_rn(__fsub_rn(d.x, 0.5f * mh), __fsub_rn(dl, 0.5f * ml));
    const float dn = __fadd_rn(__fadd_rn(d.x, 0.5f * mh), __fadd_rn(dl, 0.5f * ml));
    if (up > 0.0f) k += 1.0f;
    else if (dn < 0.0f) k -= 1.0f;
    open |= !(fminf(fabsf(up), fabsf(dn)) >= 0x1p-34f * mh);
    return (uint32_t)__float2int_rn(k);
}

// One value (dim `dim`) of turned x * w as a pair, from memory.
template <typename T, bool kPairs>
__device__ __forceinline__ float2 pair_value(const NormRopeParams &p, const T *x, const float *turn, int dim) {
    const int other = kPairs ? dim ^ 1 : dim ^ (kHD / 2), i = kPairs ? dim >> 1 : dim & (kHD / 2 - 1);
    const bool second = kPairs ? dim & 1 : dim >= kHD / 2;
    const float c = turn[i], s = turn[kHD / 2 + i];
    const float xa = load1(x + dim), xb = load1(x + other);
    float wa = 1.0f, wb = 1.0f;
    if (p.k_weight) {
        wa = p.k_weight[dim];
        wb = second ? p.k_weight[other] : -p.k_weight[other];
    } else if (!second) {
        wb = -1.0f;
    }
    const float ah = __fmul_rn(xa, wa), al = __fmaf_rn(xa, wa, -ah);
    const float bh = __fmul_rn(xb, wb), bl = __fmaf_rn(xb, wb, -bh);
    return pair_add(pair_times(ah, al, c), pair_times(bh, bl, s));
}

// Key rows with one value next to a border (dim `near` in one or more of the
// row's lanes, -1 in the others) and one that can be the maximum (dim `peak`
// in one lane): only these are computed as pairs.  Returns the code at `near`;
// `open` as pair_code.
template <typename T, bool kPairs>
__device__ __noinline__ uint32_t near_code(const NormRopeParams &p, int64_t row, int64_t pos, int h, int near, int peak,
                                           float inv, bool &open, int lane) {
    const T *x = reinterpret_cast<const T *>(p.k) + row * p.k_stride + (size_t)h * kHD;
    const float *turn = p.rope + (size_t)pos * kHD;
    float2 top = make_float2(0.0f, 0.0f), z = top;
    if (near >= 0) z = pair_value<T, kPairs>(p, x, turn, near);
    if (peak >= 0) top = pair_value<T, kPairs>(p, x, turn, peak);
    if (top.x < 0.0f) top = make_float2(-top.x, -top.y);
    const int src = (lane & 24) + __ffs((__ballot_sync(0xffffffffu, peak >= 0) >> (lane & 24)) & 0xffu) - 1;
    top.x = __shfl_sync(0xffffffffu, top.x, src & 31);
    top.y = __shfl_sync(0xffffffffu, top.y, src & 31);
    open = false;
    return pair_code(z.x, z.y, top.x, top.y, inv, open);
}

// Key rows of which more than one value is next to a border, every value held
// as a pair of fp32.  mask: the lanes of these rows (eight to a row); the rows
// are stored.  Returns the lanes that find a value undecided (or a NaN): their
// rows are left to exact_key_row.
template <typename T, bool kPairs>
__device__ __noinline__ unsigned near_key_rows(const NormRopeParams &p, int64_t row, int64_t pos, int h0, KeyPlace at,
                                               float sc, unsigned mask, int lane) {
    const int j = lane & 7, h = min(h0 + (lane >> 3), p.nkv - 1);
    float x[16], w[16], c[8], s[8], zl[16];
    load_row(reinterpret_cast<const T *>(p.k) + row * p.k_stride + (size_t)h * kHD, j, x);
    load_turn<kPairs>(p.rope + (size_t)pos * kHD, j, c, s);
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = 1.0f;
    if (p.k_weight) load_row(p.k_weight, j, w);
    float mh = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int ia = kPairs ? 2 * e : e, ib = kPairs ? 2 * e + 1 : 8 + e;
        const float ah = __fmul_rn(x[ia], w[ia]), al = __fmaf_rn(x[ia], w[ia], -ah);
        const float bh = __fmul_rn(x[ib], w[ib]), bl = __fmaf_rn(x[ib], w[ib], -bh);
        const float2 za = pair_add(pair_times(ah, al, c[e]), pair_times(-bh, -bl, s[e]));
        const float2 zb = pair_add(pair_times(bh, bl, c[e]), pair_times(ah, al, s[e]));
        x[ia] = za.x;
        zl[ia] = za.y;
        x[ib] = zb.x;
        zl[ib] = zb.y;
        mh = fmaxf(mh, fmaxf(fabsf(za.x), fabsf(zb.x)));
    }
    mh = row_max(mh);
    float ml = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (fabsf(x[e]) == mh) ml = fmaxf(ml, x[e] < 0.0f ? -zl[e] : zl[e]);
    ml = row_max(ml);
    const float inv = __fdividef(127.0f, mh);
    bool open = false;
    uint32_t t[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        t[e] = pair_code(x[e], zl[e], mh, ml, inv, open);
    }
    const bool mine = (mask >> (lane & 24)) & 0xffu;
    const unsigned rest = __ballot_sync(0xffffffffu, open && mine);
    if (mine && !((rest >> (lane & 24)) & 0xffu)) store_codes(p, t, sc, h, at, j);
    return rest;
}

// Keys of kv heads h0 .. h0 + 3 (below nkv) of a token; x: the rows, one per
// eight lanes.
//
// Codes in fp32: z = turned x * w (r left out).  In units of eps = 2^-24 and Z
// = max|z*| of the exact values: x * w carries one rounding, the turn one of a
// product and one of the sum, and |u_a c| + |u_b s| <= |(u_a, u_b)| |(c, s)|
// <= sqrt(2) Z, so that z is within (2 sqrt(2) + 1) eps Z of z*, and so is m =
// max|z| of Z; 127 * rcp(m) adds 3 eps.  127 z / m is then within 127 * 10.7
// eps of 127 z* / Z, and where its distance to the rounded value is at most 1/2
// - 1408 eps that value is the code (t = fl(z * inv + 1.5 * 2^23) holds it in
// its low mantissa bits, as in kv_code_bytes4).  Of the others (1.7e-4 of
// values, one in 2 % of rows) and of the row's largest, z is computed again as a
// pair of fp32 (near_code); a row with several of either goes to
// near_key_rows, one out of the range in which these errors are relative ones,
// or within 2^-34 of a border, to exact_key_row.  (64-bit arithmetic has a
// hundredth of fp32's rate: with it for all of these a call of 64 tokens takes
// 8.6 us instead of 5.1.)
template <typename T, bool kPairs>
__device__ __forceinline__ void store_keys(const NormRopeParams &p, float (&x)[16], const float (&c)[8],
                                           const float (&s)[8], int64_t row, int64_t pos, int h0, KeyPlace at,
                                           int lane) {
    constexpr float kShift = 0x1.8p23f;
    constexpr float kLim = 0.5f - 1408.0f * 0x1p-24f;
    const int j = lane & 7, h = h0 + (lane >> 3);
    const float ss = row_squares(x);
    if (p.k_weight) weighted(x, p.k_weight, j);
    turn<kPairs>(x, c, s);
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
    m = row_max(m);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(m));
    inv *= 127.0f;
    const float r = p.k_weight ? rsqrtf(fmaf(ss, 1.0f / kHD, p.eps)) : 1.0f;
    const float sc = __fmul_rn(m * r, KVQ8_INV127);
    const bool wide = !(m >= 0x1p-60f && m <= 0x1p60f && ss < kMostSquares && sc >= 0x1p-100f);   // the whole row
    bool odd = wide;
    uint32_t t[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float f = __fmaf_rn(x[e], inv, kShift);
        odd |= !(fabsf(__fmaf_rn(x[e], inv, -__fsub_rn(f, kShift))) <= kLim);
        t[e] = __float_as_uint(f);
    }
    const bool live = h < p.nkv;
    const unsigned who = __ballot_sync(0xffffffffu, odd && live);
    const bool mine = (who >> (lane & 24)) & 0xffu;   // this row has such a value
    if (live && !mine) store_codes(p, t, sc, h, at, j);
    if (who) {   // warp-uniform
        int near = -1, peak = -1, several = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int dim = 32 * (e / 4) + 4 * j + e % 4;
            const float f = __uint_as_float(t[e]);
            if (!(fabsf(__fmaf_rn(x[e], inv, -__fsub_rn(f, kShift))) <= kLim)) {
                several |= near >= 0;
                near = dim;
            }
            if (fabsf(x[e]) >= m * (1.0f - 0x1p-21f)) {   // z's error is below 2^-22 m
                several |= peak >= 0;
                peak = dim;
            }
        }
        const unsigned peaks = __ballot_sync(0xffffffffu, peak >= 0) >> (lane & 24) & 0xffu;
        several |= (peaks & (peaks - 1)) != 0 || peaks == 0 || wide;
        unsigned hard = __ballot_sync(0xffffffffu, mine && several);   // by lanes, then by rows
        bool open;
        const uint32_t code = near_code<T, kPairs>(p, row, pos, min(h, p.nkv - 1), near, peak, inv, open, lane);
        hard |= __ballot_sync(0xffffffffu, mine && near >= 0 && open);
        if (live && mine && !((hard >> (lane & 24)) & 0xffu)) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (near == 32 * (e / 4) + 4 * j + e % 4) t[e] = code;
            store_codes(p, t, sc, h, at, j);
        }
        unsigned left = __ballot_sync(0xffffffffu, wide && live);
        const unsigned pairs = __ballot_sync(0xffffffffu, live && mine && !wide && ((hard >> (lane & 24)) & 0xffu));
        if (pairs) left |= near_key_rows<T, kPairs>(p, row, pos, h0, at, sc, pairs, lane);
        while (left) {
            const int g = (__ffs(left) - 1) >> 3;
            left &= ~(0xffu << (8 * g));
            // (a negative scale asks for it to be found too)
            exact_key_row<T, kPairs>(p, row, pos, h0 + g, at, __shfl_sync(0xffffffffu, wide ? -1.0f : sc, 8 * g), lane);
        }
    }
}

// Queries of heads h0 .. h0 + 3 (below nqh) of a token.  Where the squares' sum
// is beyond 2^120 it is taken again of x * 2^-68, of which 128 squares stay
// below 2^7 (2^128 2^-68)^2 = 2^127 whatever the row; x itself is multiplied by
// the scaled row's root, at most 2^12 there, and then by 2^-68 (exact).
template <bool kPairs>
__device__ __forceinline__ void store_queries(const NormRopeParams &p, float (&x)[16], const float (&c)[8],
                                              const float (&s)[8], int64_t row, int h0, int lane) {
    const int j = lane & 7, h = h0 + (lane >> 3);
    if (p.q_weight) {
        float ss = row_squares(x), f = 1.0f;
        const bool wide = __any_sync(0xffffffffu, ss > kMostSquares);
        if (wide) {
            if (ss > kMostSquares) f = 0x1p-68f;
            ss = row_squares(x, f);
        }
        const float r = rsqrtf(fmaf(ss, 1.0f / kHD, p.eps * f * f));
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= r;
        if (wide) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= f;
        }
        weighted(x, p.q_weight, j);
    }
    turn<kPairs>(x, c, s);
    if (h < p.nqh) {
        float *d = p.q_out + (row * p.nqh + h) * kHD + 4 * j;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(d + 32 * i) = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
}

// Turn task w = row * parts + c: groups [c * gp, (c + 1) * gp) of four heads
// of a token, the query heads' groups before the kv heads'.
template <typename T, bool kPairs>
__device__ __forceinline__ void turn_heads(const NormRopeParams &p, int w, int parts, int gp, int lane,
                                           unsigned char *ring) {
    const int row = w / parts;
    const int b = row / p.n_new, i = row - b * p.n_new;
    if (p.n_tokens && i >= p.n_tokens[b]) return;   // padding
    const int64_t at = (int64_t)p.start_pos[b] + i;
    const int64_t pos = p.positions ? p.positions[row] : at;
    const int j = lane & 7, g = lane >> 3;
    const int qg = (p.nqh + 3) / 4, groups = qg + (p.nkv + 3) / 4;
    const int g0 = (w - row * parts) * gp, g1 = min(groups, g0 + gp);
    // a lane whose head is beyond the last loads the last
    auto fetch = [&](int gi) {
        if (gi < g1) {
            const bool is_q = gi < qg;
            const int h = min((is_q ? gi : gi - qg) * 4 + g, (is_q ? p.nqh : p.nkv) - 1);
            fetch_row(ring + (gi - g0) % kDepth * stage_bytes<T>(),
                      reinterpret_cast<const T *>(is_q ? p.q : p.k) + (int64_t)row * (is_q ? p.q_stride : p.k_stride) +
                          (size_t)h * kHD, j, lane);
        }
        cp_async_commit();   // possibly empty: one group per stage
    };
#pragma unroll
    for (int d = 0; d < kDepth - 1; ++d) fetch(g0 + d);
    if (pos < 0 || pos >= p.n_pos) {
        if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
        cp_async_wait<0>();
        return;
    }
    KeyPlace place = {-1, 0};
    if (g1 > qg) place = key_place(p, b, at, lane);
#pragma unroll 1
    for (int gi = g0; gi < g1; ++gi) {
        cp_async_wait<kDepth - 2>();
        float x[16];
        read_row<T>(ring + (gi - g0) % kDepth * stage_bytes<T>(), lane, x);
        fetch(gi + kDepth - 1);   // into the stage read before this one
        // the table row comes from L1 again for each group: kept, its 16
        // registers push others out
        float c[8], s[8];
        load_turn<kPairs>(p.rope + (size_t)pos * kHD, j, c, s);
        if (gi < qg) store_queries<kPairs>(p, x, c, s, row, 4 * gi, lane);
        else if (place.tile >= 0) store_keys<T, kPairs>(p, x, c, s, row, pos, 4 * (gi - qg), place, lane);
    }
}

// ------------------------------------------------------------ value tasks --
// Value task w = (b * runs + x) * nkv + h: the new tokens of sequence b in run
// x of kRun cache slots, counted from the run of the first, of kv head h.
// Places outside the table or the pool are flagged by the turn tasks.
template <typename T, int kRun>
__device__ __forceinline__ void append_values(const NormRopeParams &p, int w, int runs, int lane,
                                              unsigned char *ring) {
    const int bx = w / p.nkv, h = w - bx * p.nkv;
    const int b = bx / runs;
    const int64_t cap = (int64_t)p.max_blocks * kBS;
    const int64_t start = p.start_pos[b];
    const int nt = p.n_tokens ? min(p.n_new, p.n_tokens[b]) : p.n_new;   // the rest is padding
    // slots [r0, r0 + kRun), of which tokens with positions in [lo, hi) are written
    const int64_t r0 = (start >= 0 ? start / kRun : -((-start + kRun - 1) / kRun)) * kRun +
                       (int64_t)(bx - b * runs) * kRun;
    const int64_t lo = max(max(start, r0), (int64_t)0), hi = min(min(start + nt, r0 + kRun), cap);
    if (lo >= hi) return;
    const int phys = p.block_table[(size_t)b * p.max_blocks + r0 / kBS];
    // lane r: whether the token in slot r0 + r is appended
    const int64_t row0 = (int64_t)b * p.n_new + (r0 - start);   // row of the token in slot r0 (may precede the tensor)
    bool good = lane < kRun && r0 + lane >= lo && r0 + lane < hi;
    if (good) {
        const int64_t pos = p.positions ? p.positions[row0 + lane] : r0 + lane;
        good = pos >= 0 && pos < p.n_pos;
    }
    if (phys < 0 || phys >= p.num_blocks) return;
    const unsigned todo = __ballot_sync(0xffffffffu, good);
    const size_t tile = (size_t)phys * p.nkv + h;
    const int slot0 = (int)(r0 % kBS);
    int8_t *vrun = p.v_pool + tile * kHD * kBS + (size_t)(slot0 / kStageTok) * kTileVQuarter + slot0 % kStageTok;
    const T *src = reinterpret_cast<const T *>(p.v) + (size_t)h * kHD + 4 * lane;

    if (todo == (1u << kRun) - 1) {
        // the whole run, four tokens at a time through the ring (a lane reads what it copied)
        auto fetch = [&](int g) {
            if (g < kRun / 4) {
                unsigned char *st = ring + g % kDepth * stage_bytes<T>();
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    copy4(st + (u * 32 + lane) * 4 * (int)sizeof(T), src + (row0 + 4 * g + u) * p.v_stride);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int g = 0; g < kDepth - 1; ++g) fetch(g);
        uint32_t vw[4][kRun / 4];        // codes of dim 4 * lane + i
        float sc_keep = 0.0f;            // lane r: scale of row r
#pragma unroll
        for (int g = 0; g < kRun / 4; ++g) {
            cp_async_wait<kDepth - 2>();
            float4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[u] = load4(reinterpret_cast<const T *>(ring + g % kDepth * stage_bytes<T>()) + (u * 32 + lane) * 4);
            fetch(g + kDepth - 1);
            uint4 cv[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float sc = kv_row_scale_checked<true>(v[u], p.dev_status);
                cv[u] = kv_code_bytes4(v[u], sc);
                if (lane == 4 * g + u) sc_keep = sc;
            }
            vw[0][g] = low_bytes4(make_uint4(cv[0].x, cv[1].x, cv[2].x, cv[3].x));
            vw[1][g] = low_bytes4(make_uint4(cv[0].y, cv[1].y, cv[2].y, cv[3].y));
            vw[2][g] = low_bytes4(make_uint4(cv[0].z, cv[1].z, cv[2].z, cv[3].z));
            vw[3][g] = low_bytes4(make_uint4(cv[0].w, cv[1].w, cv[2].w, cv[3].w));
        }
        if (lane < kRun) p.v_scale[tile * kBS + slot0 + lane] = sc_keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int8_t *d = vrun + (size_t)(4 * lane + i) * kStageTok;
            if constexpr (kRun == 16)
                *reinterpret_cast<uint4 *>(d) = make_uint4(vw[i][0], vw[i][1], vw[i][2], vw[i][3]);
            else
                *reinterpret_cast<uint32_t *>(d) = vw[i][0];
        }
        return;
    }
    // part of a run: row by row
    for (unsigned left = todo; left; left &= left - 1) {
        const int r = __ffs(left) - 1;
        float4 v = load4(src + (row0 + r) * p.v_stride);
        const float sc = kv_row_scale_checked<true>(v, p.dev_status);
        const uint4 c = kv_code_bytes4(v, sc);
        vrun[(size_t)(4 * lane + 0) * kStageTok + r] = (int8_t)c.x;
        vrun[(size_t)(4 * lane + 1) * kStageTok + r] = (int8_t)c.y;
        vrun[(size_t)(4 * lane + 2) * kStageTok + r] = (int8_t)c.z;
        vrun[(size_t)(4 * lane + 3) * kStageTok + r] = (int8_t)c.w;
        if (lane == 0) p.v_scale[tile * kBS + slot0 + r] = sc;
    }
}

// How the two kinds of tasks are laid out over the grid: the turn tasks' CTAs,
// then the value tasks'.
struct TaskPlan {
    int turn_tasks, parts, gp;    // groups of four heads per turn task, such parts per token
    int value_tasks, runs;
    unsigned turn_ctas;
};

template <typename T, bool kPairs, int kRun>
__global__ void __launch_bounds__(kTaskWarps * 32, kMinCtas)
norm_rope_append_kernel(NormRopeParams p, TaskPlan plan) {
    __shared__ __align__(16) unsigned char rings[kTaskWarps][kDepth * stage_bytes<T>()];
    // (the next kernel starts only when those before this one are done: a step
    // with the cache declared ready reads what they wrote without waiting)
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= plan.turn_ctas) {
        const int64_t w = (int64_t)(blockIdx.x - plan.turn_ctas) * kTaskWarps + warp;
        if (w < plan.value_tasks) append_values<T, kRun>(p, (int)w, plan.runs, lane, rings[warp]);
    } else {
        const int64_t w = (int64_t)blockIdx.x * kTaskWarps + warp;
        if (w < plan.turn_tasks) turn_heads<T, kPairs>(p, (int)w, plan.parts, plan.gp, lane, rings[warp]);
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

template <typename T, bool kPairs, int kRun>
cudaError_t launch_runs(const NormRopeParams &p, cudaStream_t s) {
    TaskPlan plan;
    // runs of kRun slots that n_new consecutive positions touch, at most
    plan.runs = (int)(((int64_t)p.n_new + kRun - 2) / kRun + 1);
    const int64_t rows = (int64_t)p.batch * p.n_new;
    // A turn task takes one group of four heads while that leaves the GPU short
    // of warps, and several (which share one turn) when there are many.
    const int groups = (p.nqh + 3) / 4 + (p.nkv + 3) / 4;
    plan.gp = (int)max((int64_t)1, min((int64_t)kMostGroups, rows * groups / kFullTasks));
    plan.parts = (groups + plan.gp - 1) / plan.gp;
    const int64_t values = (int64_t)p.batch * plan.runs * p.nkv, turns = rows * plan.parts;
    const int64_t vb = (values + kTaskWarps - 1) / kTaskWarps, tb = (turns + kTaskWarps - 1) / kTaskWarps;
    if (values > 2147483647 || turns > 2147483647 || vb + tb > 2147483647) return cudaErrorInvalidConfiguration;
    plan.value_tasks = (int)values;
    plan.turn_tasks = (int)turns;
    plan.turn_ctas = (unsigned)tb;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(vb + tb));
    cfg.blockDim = dim3(kTaskWarps * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_append_kernel<T, kPairs, kRun>, p, plan);
}

// A value task takes 16 slots (its V pieces are then 16 bytes) when there are
// enough of them, else 4 (a quarter of the latency).
template <typename T, bool kPairs>
cudaError_t launch_rows(const NormRopeParams &p, cudaStream_t s) {
    const int64_t runs = (int64_t)p.batch * p.nkv * ((p.n_new + 15) / 16);
    if (runs >= (p.n_tokens ? kLongRunsPadded : kLongRuns)) return launch_runs<T, kPairs, 16>(p, s);
    return launch_runs<T, kPairs, 4>(p, s);
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
