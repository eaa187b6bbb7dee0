// decode_shared.cu -- the decode of a batch whose rows share their first tokens
// in groups: the split over each row's own tokens (decode_split.cuh, kTail) and
// the merge of its partial results with those of the shared tokens.
#include "decode_split.cuh"
#include "tile_rows.cuh"

namespace kvq8 {
namespace {

// Merge of one (row, query head), thread = dim: the records of the shared tokens
// (one per CTA of the tile that the row lies in) and of the row's own tokens, by
// the rule of decode_combine_kernel, in this order.
__global__ void __launch_bounds__(kHD)
shared_merge_kernel(DecodeParams d, TileParams t, int G) {
    pdl_wait();
    pdl_launch_dependents();
    const int qh = blockIdx.x, b = blockIdx.y, dim = threadIdx.x;
    const int h = qh / G, g = qh % G;
    const int L = clamp_len(d.ctx_lens[b], d.max_blocks * kBS);
    const int own = t.ws_tail[b];   // <= L
    float m = -INFINITY, s_sum = 0.0f, a = 0.0f;
    auto add = [&](float2 ml, float x) {
        const float m_new = fmaxf(m, ml.x);
        if (m_new == -INFINITY) return;
        const float f_old = ex2_approx(m - m_new), f = ex2_approx(ml.x - m_new);
        s_sum = fmaf(ml.y, f, s_sum * f_old);
        a = fmaf(x, f, a * f_old);
        m = m_new;
    };
    if (own > 0) {
        const int grp = group_of_row(t.group_starts, t.n_groups, b);
        const int b0 = t.group_starts[grp];
        const int n = (b - b0) * G + g;                                     // row of the (kv head, group)
        const int64_t x0 = ((int64_t)h * t.batch + b0) * G;
        const int4 dir = t.ws_dir[x0 + n / t.tile_rows * t.tile_rows];
        for (int c = 0; c < dir.y; ++c) {
            const int64_t r = x0 + n + (int64_t)(dir.x + c) * kTileRows;
            add(*reinterpret_cast<const float2 *>(t.ws_ml + r * 2), t.ws_acc[r * kHD + dim]);
        }
    }
    if (own < L) {
        const size_t u = (size_t)b * d.nkv + h;
        const int2 meta = d.ws_meta[u];
        for (int c = 0; c < meta.y; ++c) {
            const size_t r = ((size_t)meta.x + u + c) * G + g;
            add(*reinterpret_cast<const float2 *>(d.ws_ml + r * 2), d.ws_acc[r * kHD + dim]);
        }
    }
    d.out[((size_t)b * d.nqh + qh) * kHD + dim] = s_sum > 0.0f ? __fdividef(a, s_sum) : 0.0f;
}

}  // namespace

cudaError_t launch_decode_tail_split(const DecodeParams &p, int group, cudaStream_t s) {
    switch (group) {
        case 1: return launch_split_gm<1, false, 1, kTail>(p, s);
        case 2: return launch_split_two<kTail>(p, s);
        case 4: return launch_split_gm<4, false, 1, kTail>(p, s);
        case 8: return launch_split_gm<8, false, 1, kTail>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_shared_merge(const DecodeParams &d, const TileParams &p, int group, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(d.nqh, d.batch);
    cfg.blockDim = dim3(kHD);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, shared_merge_kernel, d, p, group);
}

}  // namespace kvq8
