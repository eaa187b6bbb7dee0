// decode_weights.cu -- decode attention that also adds up the attention weight
// of every cached token: the scored split kernel and the merge that turns the
// scores into weights.
//
// weight_sum[t] += sum over the group's heads g of p_{g,t}, p_{g,t} =
// 2^(s_{g,t} - M_g) / S_g with the maximum M and sum S of the whole softmax,
// which are known only when every split is done.  The split kernel therefore
// writes the scores it computes anyway (4 G bytes per token beside the
// 2 * 128 + 8 bytes that it reads), and the merge reads them back, mostly from
// L2, in the launch that merges the output.
#include "decode_combine.cuh"

namespace kvq8 {
namespace {

constexpr int kTokThread = 4;                    // tokens per thread of a weights block
constexpr int kChunkTok = kTokThread * kHD;      // tokens per weights block

// Blocks [0, batch * nqh): the output row of one (sequence, query head), as
// decode_combine_kernel.  The others: kChunkTok tokens of one unit.
template <int G>
__global__ void __launch_bounds__(kHD)
weights_merge_kernel(DecodeParams p, int chunks) {
    pdl_launch_dependents();
    pdl_wait();
    const int rows = p.batch * p.nqh;
    if (blockIdx.x < rows) {
        combine_row(p, G, blockIdx.x % p.nqh, blockIdx.x / p.nqh, threadIdx.x);
        return;
    }
    __shared__ float sm_m[G], sm_inv[G];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int w = blockIdx.x - rows;
    const int u = w / chunks, b = u / p.nkv, h = u % p.nkv;
    const int cap = p.max_blocks * kBS;
    const int t0 = (w % chunks) * kChunkTok;
    const int Lraw = p.ctx_lens[b];
    const int L = clamp_len(Lraw, cap);
    if (t0 >= L) return;
    // the softmax's maximum and sum over the unit's records
    const int2 meta = p.ws_meta[u];
    for (int g = warp; g < G; g += kHD / 32) {
        float m = -INFINITY, s = 0.0f;
        for (int j = lane; j < meta.y; j += 32) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.ws_ml + (((size_t)meta.x + u + j) * G + g) * 2);
            if (ml.x == -INFINITY) continue;
            const float mn = fmaxf(m, ml.x);
            s = s * ex2_approx(m - mn) + ml.y * ex2_approx(ml.x - mn);
            m = mn;
        }
        const float top = redux_max_f32(m);
        s = warp_sum(m == -INFINITY ? 0.0f : s * ex2_approx(m - top));
        if (lane == 0) {
            sm_m[g] = top;
            sm_inv[g] = s > 0.0f ? 1.0f / s : 0.0f;
        }
    }
    __syncthreads();
    const int t = t0 + kTokThread * tid;
    if (t >= L) return;
    const int phys = p.block_table[(size_t)b * p.max_blocks + t / kBS];
    if (phys < 0 || phys >= p.num_blocks) return;   // flagged by the split
    float4 w4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float *sc = p.ws_scores + (size_t)u * G * cap + t;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float4 s = *reinterpret_cast<const float4 *>(sc + (size_t)g * cap);
        const float m = sm_m[g], inv = sm_inv[g];
        if (inv > 0.0f) {
            w4.x = fmaf(ex2_approx(s.x - m), inv, w4.x);
            w4.y = fmaf(ex2_approx(s.y - m), inv, w4.y);
            w4.z = fmaf(ex2_approx(s.z - m), inv, w4.z);
            w4.w = fmaf(ex2_approx(s.w - m), inv, w4.w);
        }
    }
    float *dst = p.weight_sum + ((size_t)phys * p.nkv + h) * kBS + t % kBS;
    // a step's new token starts its sum here (none for a length beyond the table)
    const int fresh = p.k_new && Lraw == L ? L - 1 : -1;
    if (t + kTokThread <= L && (fresh < t || fresh >= t + kTokThread)) {
        const float4 o = *reinterpret_cast<const float4 *>(dst);
        *reinterpret_cast<float4 *>(dst) = make_float4(o.x + w4.x, o.y + w4.y, o.z + w4.z, o.w + w4.w);
    } else {
        const float v[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int i = 0; i < kTokThread; ++i)
            if (t + i < L) dst[i] = t + i == fresh ? v[i] : dst[i] + v[i];
    }
}

template <int G>
cudaError_t launch_merge_g(const DecodeParams &p, int chunks, unsigned grid, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kHD);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weights_merge_kernel<G>, p, chunks);
}

int weights_chunks(int max_blocks) {
    return (int)(((int64_t)max_blocks * kBS + kChunkTok - 1) / kChunkTok);
}

}  // namespace

int64_t weights_merge_blocks(int batch, int nqh, int nkv, int max_blocks) {
    return (int64_t)batch * nqh + (int64_t)batch * nkv * weights_chunks(max_blocks);
}

cudaError_t launch_decode_weights_split(const DecodeParams &p, int group, cudaStream_t s) {
    switch (group) {
        case 1: return launch_split_gm<1, false, 1, kScored>(p, s);
        case 2: return launch_split_gm<2, false, 1, kScored>(p, s);
        case 4: return launch_split_gm<4, false, 1, kScored>(p, s);
        case 8: return launch_split_gm<8, false, 1, kScored>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_weights_merge(const DecodeParams &p, int group, cudaStream_t s) {
    const int chunks = weights_chunks(p.max_blocks);
    const int64_t blocks = weights_merge_blocks(p.batch, p.nqh, p.nkv, p.max_blocks);
    if (blocks > 2147483647) return cudaErrorInvalidConfiguration;
    switch (group) {
        case 1: return launch_merge_g<1>(p, chunks, (unsigned)blocks, s);
        case 2: return launch_merge_g<2>(p, chunks, (unsigned)blocks, s);
        case 4: return launch_merge_g<4>(p, chunks, (unsigned)blocks, s);
        case 8: return launch_merge_g<8>(p, chunks, (unsigned)blocks, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvq8
