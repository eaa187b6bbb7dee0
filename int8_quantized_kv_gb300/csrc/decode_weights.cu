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

constexpr int kRowTok = 4 * kHD;                 // tokens that a block takes at once, four per thread
// Times that a weights block does so: twice, so that half as many blocks look
// for the softmax's maximum and sum (28 layers at 8K: 87.6 -> 86.2 us; 4 x
// 128K, G = 4: 195.9 -> 193.7 us; four times spills).  G = 8 has no registers
// for it.
constexpr int block_rows(int G) { return G >= 8 ? 1 : 2; }

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
// others: block_rows(G) * kRowTok tokens of one unit, whose scores and sums are loaded
// before the softmax's maximum and sum are known.
template <int G>
__global__ void __launch_bounds__(kHD, 8)
weights_merge_kernel(DecodeParams p, int chunks) {
    pdl_wait();
    pdl_launch_dependents();   // (released before the wait: the same times)
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
    constexpr int kRows = block_rows(G);
    const int t_lo = (w % chunks) * (kRows * kRowTok) + 4 * tid;
    const int Lraw = p.ctx_lens[b];
    const int2 meta = p.ws_meta[u];
    const int L = clamp_len(Lraw, cap);
    if (t_lo - 4 * tid >= L) return;
    float4 sc[kRows][G], old[kRows];
    float *dst[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int t = t_lo + r * kRowTok;
        dst[r] = nullptr;
        if (t < L) {
            const int phys = p.block_table[(size_t)b * p.max_blocks + t / kBS];
            const float *src = p.ws_scores + (size_t)u * G * cap + t;
#pragma unroll
            for (int g = 0; g < G; ++g) sc[r][g] = __ldcs(reinterpret_cast<const float4 *>(src + (size_t)g * cap));
            if (phys >= 0 && phys < p.num_blocks) {   // (else flagged by the split)
                dst[r] = p.weight_sum + ((size_t)phys * p.nkv + h) * kBS + t % kBS;
                old[r] = *reinterpret_cast<const float4 *>(dst[r]);
            }
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
    // a step's new token starts its sum here (none for a length beyond the table)
    const int fresh = p.k_new && Lraw == L ? L - 1 : -1;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (!dst[r]) continue;
        const int t = t_lo + r * kRowTok;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float m = sm_m[g], inv = sm_inv[g];
            if (inv > 0.0f) {
                v[0] = fmaf(ex2_approx(sc[r][g].x - m), inv, v[0]);
                v[1] = fmaf(ex2_approx(sc[r][g].y - m), inv, v[1]);
                v[2] = fmaf(ex2_approx(sc[r][g].z - m), inv, v[2]);
                v[3] = fmaf(ex2_approx(sc[r][g].w - m), inv, v[3]);
            }
        }
        const float o[4] = {old[r].x, old[r].y, old[r].z, old[r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t + i != fresh) v[i] += o[i];
        if (t + 4 <= L) {
            *reinterpret_cast<float4 *>(dst[r]) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t + i < L) dst[r][i] = v[i];
        }
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

int weights_chunks(int max_blocks, int group) {
    const int64_t tokens = block_rows(group) * kRowTok;
    return (int)(((int64_t)max_blocks * kBS + tokens - 1) / tokens);
}

}  // namespace

int64_t weights_merge_blocks(int batch, int nqh, int nkv, int max_blocks) {
    return (int64_t)batch * nqh + (int64_t)batch * nkv * weights_chunks(max_blocks, nqh / nkv);
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
    const int chunks = weights_chunks(p.max_blocks, group);
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
