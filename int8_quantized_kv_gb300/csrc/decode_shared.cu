// decode_shared.cu -- the decode of a batch whose rows share their first tokens
// in groups: the split over each row's own tokens (decode_tail.cuh) and the merge
// of its partial results with those of the shared tokens.
#include "decode_tail.cuh"
#include "tile_rows.cuh"

namespace kvq8 {
namespace {

// Merge of one (row, query head) by a warp, four dims to a lane: the records of
// the shared tokens (one per CTA of the tile that the row lies in) and of the
// row's own tokens, by the rule of decode_combine_kernel, in this order, four
// records' loads at a time.
constexpr int kMergeHeads = 4;
__global__ void __launch_bounds__(kMergeHeads * 32)
shared_merge_kernel(DecodeParams d, TileParams t, int G) {
    pdl_wait();
    pdl_launch_dependents();
    const int qh = blockIdx.x * kMergeHeads + (threadIdx.x >> 5), b = blockIdx.y, lane = threadIdx.x & 31;
    if (qh >= d.nqh) return;
    const int h = qh / G, g = qh % G;
    const int own = t.ws_tail[b], b0 = t.ws_first[b];   // own <= the context's length
    const size_t u = (size_t)b * d.nkv + h;
    const int2 meta = d.ws_meta[u];                     // (not written for a row without tokens of its own)
    const int L = clamp_len(d.ctx_lens[b], d.max_blocks * kBS);
    const int n = (b - b0) * G + g;                     // row of the (kv head, group)
    const int64_t x0 = ((int64_t)h * t.batch + b0) * G;
    const int4 dir = own > 0 ? t.ws_dir[x0 + n / t.tile_rows * t.tile_rows] : make_int4(0, 0, 0, 0);
    const int shared = dir.y, count = shared + (own < L ? meta.y : 0);
    const int64_t r1 = x0 + n + (int64_t)dir.x * t.tile_rows, r2 = ((int64_t)meta.x + u) * G + g;
    float m = -INFINITY, s_sum = 0.0f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAtOnce = 4;
    for (int i0 = 0; i0 < count; i0 += kAtOnce) {
        float2 ml[kAtOnce];
        float4 x[kAtOnce];
        float top = m;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = i0 + k;
            ml[k] = make_float2(-INFINITY, 0.0f);
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < count) {
                const bool s = i < shared;
                const int64_t r = s ? r1 + (int64_t)i * t.tile_rows : r2 + (int64_t)(i - shared) * G;
                ml[k] = *reinterpret_cast<const float2 *>((s ? t.ws_ml : d.ws_ml) + r * 2);
                x[k] = *reinterpret_cast<const float4 *>((s ? t.ws_acc : d.ws_acc) + r * kHD + 4 * lane);
            }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);
        if (top == -INFINITY) continue;
        const float2 old = pow2_parts(m - top);   // 0 while m is -inf
        const float f_old = old.x * old.y;
        s_sum = s_sum * old.x * old.y;
        a = make_float4(a.x * f_old, a.y * f_old, a.z * f_old, a.w * f_old);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const float2 part = pow2_parts(ml[k].x - top);
            const float f = part.x * part.y;
            s_sum = fmaf(ml[k].y * part.x, part.y, s_sum);
            a.x = fmaf(x[k].x, f, a.x);
            a.y = fmaf(x[k].y, f, a.y);
            a.z = fmaf(x[k].z, f, a.z);
            a.w = fmaf(x[k].w, f, a.w);
        }
        m = top;
    }
    const float inv = s_sum > 0.0f ? 1.0f / s_sum : 0.0f;
    *reinterpret_cast<float4 *>(d.out + ((size_t)b * d.nqh + qh) * kHD + 4 * lane) =
        make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
}

}  // namespace

cudaError_t launch_decode_tail_split(const DecodeParams &p, int group, cudaStream_t s) {
    switch (group) {
        case 1: return launch_tail_g<1>(p, s);
        case 2: return launch_tail_g<2>(p, s);
        case 4: return launch_tail_g<4>(p, s);
        case 8: return launch_tail_g<8>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_shared_merge(const DecodeParams &d, const TileParams &p, int group, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((d.nqh + kMergeHeads - 1) / kMergeHeads, d.batch);
    cfg.blockDim = dim3(kMergeHeads * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, shared_merge_kernel, d, p, group);
}

}  // namespace kvq8
