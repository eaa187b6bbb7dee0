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
#include "decode_split.cuh"

namespace kvq8 {
namespace {

constexpr int kTokThread = 4;                    // tokens per thread of a weights block
constexpr int kChunkTok = kTokThread * kHD;      // tokens per weights block

// The output of one (sequence, query head), thread = dim: the merge rule of
// decode_combine_kernel with the records' (M, S) spread over the lanes, so that
// any 32 records take two load rounds and few registers (the weights blocks of
// the same kernel need the occupancy).
__device__ __forceinline__ void combine_row_lanes(const DecodeParams &p, int G, int qh, int b, int d) {
    const int h = qh / G, g = qh % G, lane = d & 31;
    const size_t u = (size_t)b * p.nkv + h;
    const int2 meta = p.ws_meta[u];
    const int L = clamp_len(p.ctx_lens[b], p.max_blocks * kBS);
    const int n = L > 0 ? meta.y : 0;   // (an empty unit's entry is not written)
    float m = -INFINITY, s = 0.0f, a = 0.0f;
    for (int j0 = 0; j0 < n; j0 += 32) {
        const size_t r0 = (size_t)meta.x + u + j0;
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (j0 + lane < n) ml = *reinterpret_cast<const float2 *>(p.ws_ml + ((r0 + lane) * G + g) * 2);
        const int count = min(32, n - j0);
        float acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = j < count ? p.ws_acc[((r0 + j) * G + g) * kHD + d] : 0.0f;
        const float top = redux_max_f32(ml.x);
        if (top == -INFINITY) continue;
        const float m_new = fmaxf(m, top), f_old = ex2_approx(m - m_new);   // 0 while m is -inf
        const float f = ex2_approx(ml.x - m_new);
        s = s * f_old + warp_sum(ml.y * f);
        a *= f_old;
        m = m_new;
        for (int j = 0; j < count; j += 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, (j + k) & 31);
                if (j + k < count) a = fmaf(acc[k], fk, a);
                acc[k] = j + 8 + k < count ? p.ws_acc[((r0 + j + 8 + k) * G + g) * kHD + d] : 0.0f;
            }
        }
    }
    p.out[((size_t)b * p.nqh + qh) * kHD + d] = s > 0.0f ? __fdividef(a, s) : 0.0f;
}

// Blocks [0, batch * nqh): the output row of one (sequence, query head).  The
// others: kChunkTok tokens of one unit, whose scores and sums are loaded
// before the softmax's maximum and sum are known.
template <int G>
__global__ void __launch_bounds__(kHD, 8)
weights_merge_kernel(DecodeParams p, int chunks) {
    pdl_launch_dependents();
    pdl_wait();
    const int rows = p.batch * p.nqh;
    if (blockIdx.x < rows) {
        combine_row_lanes(p, G, blockIdx.x % p.nqh, blockIdx.x / p.nqh, threadIdx.x);
        return;
    }
    __shared__ float sm_m[G], sm_inv[G];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int w = blockIdx.x - rows;
    const int u = w / chunks, b = u / p.nkv, h = u % p.nkv;
    const int cap = p.max_blocks * kBS;
    const int t = (w % chunks) * kChunkTok + kTokThread * tid;
    const int Lraw = p.ctx_lens[b];
    const int2 meta = p.ws_meta[u];
    const int L = clamp_len(Lraw, cap);
    if (t - kTokThread * tid >= L) return;
    int phys = -1;
    float4 sc[G], old = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float *dst = p.weight_sum;
    if (t < L) {
        phys = p.block_table[(size_t)b * p.max_blocks + t / kBS];
        const float *src = p.ws_scores + (size_t)u * G * cap + t;
#pragma unroll
        for (int g = 0; g < G; ++g) sc[g] = __ldcs(reinterpret_cast<const float4 *>(src + (size_t)g * cap));
        if (phys >= p.num_blocks) phys = -1;   // (flagged by the split)
        if (phys >= 0) {
            dst += ((size_t)phys * p.nkv + h) * kBS + t % kBS;
            old = *reinterpret_cast<const float4 *>(dst);
        }
    }
    // the softmax's maximum and sum over the unit's records
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
    if (phys < 0) return;
    float4 w4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float m = sm_m[g], inv = sm_inv[g];
        if (inv > 0.0f) {
            w4.x = fmaf(ex2_approx(sc[g].x - m), inv, w4.x);
            w4.y = fmaf(ex2_approx(sc[g].y - m), inv, w4.y);
            w4.z = fmaf(ex2_approx(sc[g].z - m), inv, w4.z);
            w4.w = fmaf(ex2_approx(sc[g].w - m), inv, w4.w);
        }
    }
    // a step's new token starts its sum here (none for a length beyond the table)
    const int fresh = p.k_new && Lraw == L ? L - 1 : -1;
    const float v[4] = {w4.x, w4.y, w4.z, w4.w};
    const float o[4] = {old.x, old.y, old.z, old.w};
    if (t + kTokThread <= L) {
        *reinterpret_cast<float4 *>(dst) =
            make_float4(t == fresh ? v[0] : o[0] + v[0], t + 1 == fresh ? v[1] : o[1] + v[1],
                        t + 2 == fresh ? v[2] : o[2] + v[2], t + 3 == fresh ? v[3] : o[3] + v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kTokThread; ++i)
            if (t + i < L) dst[i] = t + i == fresh ? v[i] : o[i] + v[i];
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
        case 2: return launch_split_two<kScored>(p, s);
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
