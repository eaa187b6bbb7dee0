// tiles.cu -- attention of many query rows over a cached stretch: prompts and
// shared prefixes.
#include <math.h>

#include "kvq8_ptx.cuh"
#include "tile_rows.cuh"

namespace kvq8 {
namespace {

constexpr int kWarps = 4;

// One warp per query row: codes of the row in shared memory, 32 tokens at a time
// (lane = token) scored by dp4a, weights passed on by shuffles to lanes that hold
// four dims each.  table: the block-table row; lim: tokens [0, lim).
__device__ void attend_row(const TileParams &p, float4 x, int h, const int32_t *table, int lim, int8_t *codes,
                           float *scales, float4 &acc, float &M, float &S) {
    const int lane = threadIdx.x & 31;
    float *stage = reinterpret_cast<float *>(codes);
    *reinterpret_cast<float4 *>(stage + 4 * lane) = x;
    __syncwarp();
    float xs[4];
    for (int k = 0; k < 4; ++k) xs[k] = stage[32 * k + lane];
    __syncwarp();
    quantize_q_vals_warp(xs, lane, codes, scales, p.dev_status);
    __syncwarp();
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    M = -INFINITY;
    S = 0.f;
    for (int t0 = 0; t0 < lim; t0 += 32) {
        const int phys = table[t0 / kBS];
        if (phys < 0 || phys >= p.num_blocks) {
            if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
            continue;
        }
        const size_t tile = (size_t)phys * p.nkv + h;
        const int slot = t0 % kBS + lane;
        const bool ok = t0 + lane < lim;
        float s = -INFINITY, vs = 0.f;
        if (ok) {
            float d = 0.f;
            for (int k = 0; k < 4; ++k) {
                int a = 0;
                for (int c = 2 * k; c < 2 * k + 2; ++c) {
                    const int4 kw = *reinterpret_cast<const int4 *>(p.k_pool + (tile * kBS + slot) * kHD + ((c ^ (slot & 7)) << 4));
                    const int4 qw = *reinterpret_cast<const int4 *>(codes + 16 * c);
                    a = __dp4a(kw.x, qw.x, a);
                    a = __dp4a(kw.y, qw.y, a);
                    a = __dp4a(kw.z, qw.z, a);
                    a = __dp4a(kw.w, qw.w, a);
                }
                d = fmaf((float)a, scales[k], d);
            }
            s = d * p.k_scale[tile * kBS + slot] * p.sm_scale_log2;
            vs = p.v_scale[tile * kBS + slot];
        }
        const float m = fmaxf(M, warp_max(s));
        const float al = exp2f(M - m), w = ok ? exp2f(s - m) : 0.f;
        M = m;
        S = fmaf(S, al, warp_sum(w));
        acc.x *= al; acc.y *= al; acc.z *= al; acc.w *= al;
        const float wv = w * vs;
        const int8_t *v = p.v_pool + tile * kHD * kBS + (size_t)(t0 % kBS / kStageTok) * kTileVQuarter + t0 % kStageTok;
        for (int r = 0; r < 32 && t0 + r < lim; ++r) {
            const float a = __shfl_sync(0xffffffffu, wv, r);
            acc.x = fmaf((float)v[(4 * lane + 0) * kStageTok + r], a, acc.x);
            acc.y = fmaf((float)v[(4 * lane + 1) * kStageTok + r], a, acc.y);
            acc.z = fmaf((float)v[(4 * lane + 2) * kStageTok + r], a, acc.z);
            acc.w = fmaf((float)v[(4 * lane + 3) * kStageTok + r], a, acc.w);
        }
    }
}

template <bool kShared>
__global__ void __launch_bounds__(kWarps * 32)
tile_rows_kernel(TileParams p, int G) {
    __shared__ __align__(16) int8_t codes[kWarps][512];
    __shared__ __align__(16) float scales[kWarps][4];
    __shared__ int bad;
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cap = p.max_blocks * kBS;
    if (kShared) {
        if (threadIdx.x == 0) bad = 0;
        __syncthreads();
        for (int g = threadIdx.x; g <= p.n_groups; g += blockDim.x)
            if (!group_entry_ok(p, g)) bad = 1;
        __syncthreads();
    }
    const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t tok = row / p.nqh;
    const int j = (int)(row % p.nqh), h = j / G;
    int b, lim;
    const int32_t *table;
    int64_t rec = 0;
    if (kShared) {
        if (tok >= p.batch) return;
        b = (int)tok;
        if (bad) {
            if (lane == 0) {
                flag_status(p.dev_status, KVQ8_DEV_BAD_GROUPS);
                p.ws_tail[b] = 0;
            }
            return;
        }
        const int g = group_of_row(p.group_starts, p.n_groups, b);
        const int b0 = p.group_starts[g], m = p.group_starts[g + 1] - b0;
        if (p.shared_lens[g] < 0) flag_status(p.dev_status, KVQ8_DEV_BAD_CTX_LEN);
        lim = row_shared(p, b, p.shared_lens[g], cap);
        int lead = b0;
        for (int r = b0; r < b0 + m; ++r)
            if (row_shared(p, r, p.shared_lens[g], cap) > row_shared(p, lead, p.shared_lens[g], cap)) lead = r;
        table = p.block_table + (size_t)lead * p.max_blocks;
        if (lane == 0) p.ws_tail[b] = lim;
        rec = (int64_t)b0 * p.nqh + (int64_t)h * m * G + (b - b0) * G + j % G;
        const int n = (int)(rec - (int64_t)b0 * p.nqh - (int64_t)h * m * G);
        if (lane == 0 && n % kTileRows == 0) p.ws_dir[rec] = make_int4(0, 1, 0, 0);
    } else {
        b = (int)(tok / p.n_new);
        if (b >= p.batch) return;
        const int i = (int)(tok % p.n_new);
        if (p.n_tokens && i >= p.n_tokens[b]) return;
        const int64_t pos = (int64_t)p.start_pos[b] + i;
        if (pos < 0 || pos >= cap) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
        lim = (int)max((int64_t)0, min((int64_t)cap, pos + 1));
        table = p.block_table + (size_t)b * p.max_blocks;
    }
    float4 acc;
    float M, S;
    attend_row(p, load4(p.q, p.q_dtype, tok * p.q_stride + (int64_t)j * kHD + 4 * lane), h, table, lim, codes[warp],
               scales[warp], acc, M, S);
    if (kShared) {
        *reinterpret_cast<float4 *>(p.ws_acc + rec * kHD + 4 * lane) = acc;
        if (lane == 0) {
            p.ws_ml[rec * 2] = M;
            p.ws_ml[rec * 2 + 1] = S;
        }
    } else {
        const float inv = S > 0.f ? 1.f / S : 0.f;
        const int64_t o = tok * p.out_stride + (int64_t)j * kHD + 4 * lane;
        store1(p.out, p.out_dtype, o + 0, acc.x * inv);
        store1(p.out, p.out_dtype, o + 1, acc.y * inv);
        store1(p.out, p.out_dtype, o + 2, acc.z * inv);
        store1(p.out, p.out_dtype, o + 3, acc.w * inv);
    }
}

template <bool kShared>
cudaError_t launch_rows(const TileParams &p, int group, cudaStream_t s) {
    const int64_t rows = (int64_t)p.batch * p.n_new * p.nqh;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + kWarps - 1) / kWarps));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tile_rows_kernel<kShared>, p, group);
}

}  // namespace

cudaError_t launch_prompt(const TileParams &p, int group, cudaStream_t s) { return launch_rows<false>(p, group, s); }
cudaError_t launch_shared_prefix(const TileParams &p, int group, cudaStream_t s) { return launch_rows<true>(p, group, s); }

}  // namespace kvq8
