// evict.cu -- eviction from the int8 cache by accumulated attention weight.
//
// Per unit (sequence, kv head) of L tokens the m = min(L, keep) tokens to keep
// are: the first n_first, the last n_recent, and of the others those of
// largest weight (equal weights: the lower index first).  A radix selection
// over the weights' ordered bit patterns finds the m-th largest, a scan in
// order of position writes the list of kept tokens, and a copy brings codes,
// scales and weights of these tokens, in that order, into the destination
// blocks.
#include "kvq8_device.cuh"
#include "kvq8_internal.cuh"
#include "kvq8_ptx.cuh"

namespace kvq8 {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kCopyWarps = 8;

// Order of a weight as an unsigned number: larger weights above smaller ones,
// -0 equal to 0, a NaN below everything.  Nothing maps to 0xffffffff, which
// marks a token that is kept whatever its weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t x = __float_as_uint(w);
    if ((x & 0x7fffffffu) > 0x7f800000u) return 0u;
    if ((x & 0x7fffffffu) == 0u) return 0x80000000u;
    return (x >> 31) ? ~x : (x | 0x80000000u);
}

__device__ __forceinline__ uint32_t token_key(const EvictParams &p, const int32_t *row, int h, int t, int L) {
    if (t < p.n_first || t >= L - p.n_recent) return 0xffffffffu;
    return weight_key(p.weight_sum[((size_t)row[t / kBS] * p.nkv + h) * kBS + t % kBS]);
}

// One CTA per unit.
__global__ void __launch_bounds__(kSelectThreads)
evict_select_kernel(EvictParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int hist[256];
    __shared__ int warp_gt[kSelectWarps], warp_eq[kSelectWarps];
    __shared__ int sh_digit, sh_need, sh_bad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int u = blockIdx.x, b = u / p.nkv, h = u % p.nkv;
    const int cap = p.max_blocks * kBS;
    const int Lraw = p.ctx_lens[b];
    const int L = max(0, min(Lraw, cap));
    const int m = min(L, p.keep);
    int32_t *kept = p.kept + (size_t)u * p.keep;
    const int32_t *row = p.block_table + (size_t)b * p.max_blocks;
    const int32_t *dst = p.dst_table + (size_t)b * p.dst_max_blocks;
    if (tid == 0) {
        sh_bad = 0;
        if (Lraw != L && h == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_CTX_LEN);
    }
    __syncthreads();

    // every block id must lie in the pool, and a destination must be neither a
    // source of the sequence nor listed twice
    const int n_src = (L + kBS - 1) / kBS, n_dst = (m + kBS - 1) / kBS;
    bool bad = false;
    for (int i = tid; i < n_src; i += kSelectThreads) bad |= row[i] < 0 || row[i] >= p.num_blocks;
    for (int64_t i = tid; i < (int64_t)n_dst * (n_src + n_dst); i += kSelectThreads) {
        const int d = (int)(i / (n_src + n_dst)), j = (int)(i % (n_src + n_dst));
        const int id = dst[d];
        if (j < n_src) bad |= id == row[j];
        else bad |= j - n_src == d ? (id < 0 || id >= p.num_blocks) : id == dst[j - n_src];
    }
    if (bad) sh_bad = 1;
    __syncthreads();
    if (sh_bad) {   // the sequence is left out
        for (int j = tid; j < p.keep; j += kSelectThreads) kept[j] = -1;
        if (tid == 0) {
            flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
            if (h == 0) p.new_lens[b] = 0;
        }
        return;
    }
    if (tid == 0 && h == 0) p.new_lens[b] = m;

    // the m-th largest key, digit by digit from the top: `prefix` holds the
    // digits found, `need` how many tokens with exactly this prefix are kept
    uint32_t prefix = 0;
    int need = m;
    for (int shift = 24; shift >= 0 && m < L; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int t = tid; t < L; t += kSelectThreads) {
            const uint32_t k = token_key(p, row, h, t, L);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, d = 255;
            while (d > 0 && hist[d] < left) left -= hist[d--];
            sh_digit = d;
            sh_need = left;
        }
        __syncthreads();
        prefix |= (uint32_t)sh_digit << shift;
        need = sh_need;
        __syncthreads();
    }

    // tokens above the m-th largest are kept, and the first `need` equal to it
    int base_gt = 0, base_eq = 0;
    for (int t0 = 0; t0 < L; t0 += kSelectThreads) {
        const int t = t0 + tid;
        const uint32_t k = t < L ? (m < L ? token_key(p, row, h, t, L) : 1u) : 0u;
        const bool gt = t < L && k > prefix, eq = t < L && k == prefix;
        const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            warp_gt[warp] = __popc(bg);
            warp_eq[warp] = __popc(be);
        }
        __syncthreads();
        int g = base_gt, e = base_eq;
        for (int w = 0; w < kSelectWarps; ++w) {
            if (w == warp) {
                const unsigned below = (1u << lane) - 1;
                const int ng = g + __popc(bg & below), ne = e + __popc(be & below);
                if (gt) kept[ng + min(ne, need)] = t;
                else if (eq && ne < need) kept[ng + ne] = t;
            }
            g += warp_gt[w];
            e += warp_eq[w];
        }
        base_gt = g;
        base_eq = e;
        __syncthreads();
    }
    for (int j = m + tid; j < p.keep; j += kSelectThreads) kept[j] = -1;
}

// One warp per kept token of a unit.
__global__ void __launch_bounds__(kCopyWarps * 32)
evict_copy_kernel(EvictParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t task = (int64_t)blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
    if (task >= (int64_t)p.batch * p.nkv * p.keep) return;
    const int u = (int)(task / p.keep), j = (int)(task % p.keep);
    const int b = u / p.nkv, h = u % p.nkv;
    const int t = p.kept[task];
    if (t < 0) return;
    const size_t src = (size_t)p.block_table[(size_t)b * p.max_blocks + t / kBS] * p.nkv + h;
    const size_t dst = (size_t)p.dst_table[(size_t)b * p.dst_max_blocks + j / kBS] * p.nkv + h;
    const int s = t % kBS, d = j % kBS;
    const int c = lane >> 2, w = lane & 3;
    const uint32_t *ks = reinterpret_cast<const uint32_t *>(p.k_pool + (src * kBS + s) * kHD);
    uint32_t *kd = reinterpret_cast<uint32_t *>(p.k_pool + (dst * kBS + d) * kHD);
    kd[((c ^ (d & 7)) << 2) + w] = ks[((c ^ (s & 7)) << 2) + w];
    const int8_t *vs = p.v_pool + src * kBS * kHD + (size_t)(s / kStageTok) * kTileVQuarter + s % kStageTok;
    int8_t *vd = p.v_pool + dst * kBS * kHD + (size_t)(d / kStageTok) * kTileVQuarter + d % kStageTok;
#pragma unroll
    for (int i = 0; i < 4; ++i) vd[(size_t)(lane + 32 * i) * kStageTok] = vs[(size_t)(lane + 32 * i) * kStageTok];
    if (lane == 0) p.k_scale[dst * kBS + d] = p.k_scale[src * kBS + s];
    if (lane == 1) p.v_scale[dst * kBS + d] = p.v_scale[src * kBS + s];
    if (lane == 2) p.weight_sum[dst * kBS + d] = p.weight_sum[src * kBS + s];
}

cudaError_t launch_pdl(void (*kernel)(EvictParams), unsigned grid, unsigned block, const EvictParams &p,
                       cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t s) {
    const int64_t tokens = (int64_t)p.batch * p.nkv * p.keep;
    const int64_t blocks = (tokens + kCopyWarps - 1) / kCopyWarps;
    if (blocks > 2147483647) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_pdl(evict_select_kernel, (unsigned)(p.batch * p.nkv), kSelectThreads, p, s);
    if (e != cudaSuccess) return e;
    return launch_pdl(evict_copy_kernel, (unsigned)blocks, kCopyWarps * 32, p, s);
}

}  // namespace kvq8
