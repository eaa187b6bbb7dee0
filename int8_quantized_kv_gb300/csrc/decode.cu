// decode.cu -- single-query decode attention over the paged INT8 cache:
// the launches of the split-KV kernel (decode_split.cuh) and the merge of its
// partial results.
#include "decode_combine.cuh"

namespace kvq8 {
namespace {

__global__ void __launch_bounds__(kHD)
decode_combine_kernel(DecodeParams p, int G) {
    // The next kernel of the stream may be scheduled at once: every kernel of
    // this library waits for the grid before it to complete before it reads
    // what that grid writes (a decode step's split kernel, with the cache
    // declared ready, reads only the cache before that), and its CTAs take the
    // SMs that the split kernel before this one leaves.
    pdl_launch_dependents();
    pdl_wait();  // the split kernel's records are visible after this
    combine_row(p, G, blockIdx.x, blockIdx.y, threadIdx.x);
}

// The merge of the 4-bit decode, whose split writes unit u's records at
// u * nsplit + j: the records are loaded beside the unit's length (one load
// round, no record directory), and the length says how many of them this call
// wrote (int4_split_count); merged in the order of decode_combine_kernel.
__global__ void __launch_bounds__(kHD)
decode_combine_fixed_kernel(DecodeParams p, int G, int ns) {
    pdl_launch_dependents();   // as in decode_combine_kernel
    pdl_wait();
    const int qh = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
    const int h = qh / G, g = qh % G;
    const size_t u = (size_t)b * p.nkv + h;
    const int L = clamp_len(p.ctx_lens[b], p.max_blocks * kBS);
    float mr[kCombineRegs], sr[kCombineRegs], ar[kCombineRegs];
#pragma unroll
    for (int j = 0; j < kCombineRegs; ++j) {
        if (j < ns) {
            const size_t r = (u * ns + j) * G + g;
            const float2 ml = *reinterpret_cast<const float2 *>(p.ws_ml + r * 2);
            mr[j] = ml.x;
            sr[j] = ml.y;
            ar[j] = p.ws_acc[r * kHD + d];
        }
    }
    float *o = p.out + ((size_t)b * p.nqh + qh) * kHD + d;
    if (L == 0) { *o = 0.0f; return; }
    const int n1 = int4_split_count(L, ns);
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kCombineRegs; ++j)
        if (j < n1) m = fmaxf(m, mr[j]);
    float s_sum = 0.0f, a = 0.0f;
    if (m != -INFINITY) {
#pragma unroll
        for (int j = 0; j < kCombineRegs; ++j) {
            if (j < n1) {
                const float f = ex2_approx(mr[j] - m);
                s_sum = fmaf(sr[j], f, s_sum);
                a = fmaf(ar[j], f, a);
            }
        }
    }
    *o = s_sum > 0.0f ? __fdividef(a, s_sum) : 0.0f;
}

template <int G>
cudaError_t launch_split_g(const DecodeParams &p, cudaStream_t s) {
    if (p.first_q8_block) {
        if constexpr (G == 2) return launch_split_gm<G, true, 2>(p, s);
        return launch_split_gm<G, true, 1>(p, s);
    }
    if constexpr (G == 2) {
        const int64_t units = (int64_t)p.batch * p.nkv;
        const int64_t stages_max = units * p.max_blocks * (kBS / kStageTok);
        const int sms = device_sm_count();
        if (units >= kTwoPerSmMinUnits && stages_max >= (int64_t)kTwoPerSmMinStages * 2 * sms)
            return launch_split_gm<G, false, 2>(p, s);
    }
    return launch_split_gm<G, false, 1>(p, s);
}

}  // namespace

bool make_decode_plan(int batch, int nqh, int nkv, int max_blocks, DecodePlan *plan) {
    if (batch < 0 || nqh <= 0 || nkv <= 0 || max_blocks <= 0 || nqh % nkv) return false;
    const int G = nqh / nkv;
    auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
    plan->group = G;
    plan->units = (int64_t)batch * nkv;
    plan->records = kMaxCtas + plan->units;
    plan->meta_offset = 0;
    plan->ml_offset = align((size_t)plan->units * sizeof(int2));
    plan->acc_offset = plan->ml_offset + align((size_t)plan->records * G * 2 * sizeof(float));
    plan->bytes = plan->acc_offset + align((size_t)plan->records * G * kHD * sizeof(float));
    return true;
}

cudaError_t launch_decode_split(const DecodeParams &p, int group, cudaStream_t s) {
    switch (group) {
        case 1: return launch_split_g<1>(p, s);
        case 2: return launch_split_g<2>(p, s);
        case 4: return launch_split_g<4>(p, s);
        case 8: return launch_split_g<8>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_decode_combine_fixed(const DecodeParams &p, int group, int nsplit, cudaStream_t s) {
    if (nsplit < 1 || nsplit > kCombineRegs) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.nqh, p.batch);
    cfg.blockDim = dim3(kHD);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_combine_fixed_kernel, p, group, nsplit);
}

cudaError_t launch_decode_combine(const DecodeParams &p, int group, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.nqh, p.batch);
    cfg.blockDim = dim3(kHD);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_combine_kernel, p, group);
}

}  // namespace kvq8
