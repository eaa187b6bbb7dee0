// decode.cu -- single-query decode attention over the paged INT8 cache:
// the launches of the split-KV kernel (decode_split.cuh) and the merge of its
// partial results.
#include "decode_split.cuh"

namespace kvq8 {
namespace {

// Merge of the partial records of one (sequence, query head); thread = dim.
// [Day 9-2] §2 segment 3 generalised to several partial states:
// M = max_i M_i, S = sum_i S_i 2^(M_i - M), out = sum_i acc_i 2^(M_i - M) / S,
// the factors 2^(M_i - M) <= 1 by the approximate base-2 exponential, as the
// split kernel's weights, and the final division by the fast approximate one
// (S >= 1 and far below 2^126, where it is within 2 ulp; the library's exact
// exp2f and division cost this short kernel about 0.6 us of its critical
// path).  The records come from one split kernel,
// or from two (mixed precision by token age: the 4-bit split over [0, x) and
// the int8 split over [x, L)).
constexpr int kCombineRegs = 8;   // records merged from registers (more: the loop below)
constexpr int kCombineWide = 32;  // records of one source merged after one load round

template <bool kEarly>
__global__ void __launch_bounds__(kHD)
decode_combine_kernel(DecodeParams p, int G) {
    // The merge of a whole call releases the next kernel of the stream at once,
    // so that its CTAs take the SMs that the split before this one leaves: every
    // kernel of this library waits for the grid before it before it reads what
    // that grid writes, and what a decode step with the cache declared ready
    // reads before its wait is not written by the call ahead of it.  (All
    // before the split is done when this kernel starts.)  With the release
    // behind the wait 28 one-layer steps in a graph take 244 us instead of 217.
    // A merge called on its own waits first: anything may lie ahead of it.
    if (kEarly) pdl_launch_dependents();
    pdl_wait();  // the split kernel's records are visible after this
    if (!kEarly) pdl_launch_dependents();
    const int qh = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
    const int h = qh / G, g = qh % G;
    const int cap = p.max_blocks * kBS;
    const size_t u = (size_t)b * p.nkv + h;
    // the unit's record directories are loaded beside its length (one load
    // round); an entry is used only when the length says the unit has records
    // in that source (an empty unit's entry is not written by the split)
    const int2 meta0_raw = p.ws_meta[u];
    const int2 meta1_raw = p.ws_meta2 ? p.ws_meta2[u] : make_int2(0, 0);
    const SeqSpan sp = seq_span(p, b, cap);
    float *o = p.out + ((size_t)b * p.nqh + qh) * kHD + d;
    if (sp.y == 0) { *o = 0.0f; return; }
    // source 0: this decode's records over [x, L); source 1: the 4-bit split's over [0, x)
    const bool has0 = sp.y > sp.x, has1 = p.ws_meta2 != nullptr && sp.x > 0;
    const int2 meta0 = has0 ? meta0_raw : make_int2(0, 0);
    const int2 meta1 = has1 ? meta1_raw : make_int2(0, 0);
    const size_t r00 = (size_t)meta0.x + u, r10 = (size_t)meta1.x + u;
    // the records of one source (both single-source paths below read these, so
    // that a call whose records all come from one split kernel gives the same
    // bits whichever source slot holds them)
    const bool one = meta0.y == 0 || meta1.y == 0;
    const float *ml1 = meta0.y ? p.ws_ml : p.ws_ml2, *acc1 = meta0.y ? p.ws_acc : p.ws_acc2;
    const size_t r01 = meta0.y ? r00 : r10;
    const int n1 = meta0.y ? meta0.y : meta1.y;
    if (one && n1 <= kCombineRegs) {
        // the usual case: every record's (M, S) and accumulator loaded at once,
        // then merged in the same order as below
        float mr[kCombineRegs], sr[kCombineRegs], ar[kCombineRegs];
#pragma unroll
        for (int j = 0; j < kCombineRegs; ++j) {
            if (j < n1) {
                const size_t r = (r01 + j) * G + g;
                const float2 ml = *reinterpret_cast<const float2 *>(ml1 + r * 2);
                mr[j] = ml.x;
                sr[j] = ml.y;
                ar[j] = acc1[r * kHD + d];
            }
        }
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
        return;
    }
    if (one && n1 <= kCombineWide) {
        // up to 32 records of one source (a call of few long units): one load
        // round, then the same merge
        float2 mlr[kCombineWide];
        float ar[kCombineWide];
#pragma unroll
        for (int j = 0; j < kCombineWide; ++j) {
            if (j < n1) {
                const size_t r = (r01 + j) * G + g;
                mlr[j] = *reinterpret_cast<const float2 *>(ml1 + r * 2);
                ar[j] = acc1[r * kHD + d];
            }
        }
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < kCombineWide; ++j)
            if (j < n1) m = fmaxf(m, mlr[j].x);
        float s_sum = 0.0f, a = 0.0f;
        if (m != -INFINITY) {
#pragma unroll
            for (int j = 0; j < kCombineWide; ++j) {
                if (j < n1) {
                    const float f = ex2_approx(mlr[j].x - m);
                    s_sum = fmaf(mlr[j].y, f, s_sum);
                    a = fmaf(ar[j], f, a);
                }
            }
        }
        *o = s_sum > 0.0f ? __fdividef(a, s_sum) : 0.0f;
        return;
    }
    if (!one && meta0.y + meta1.y <= kCombineRegs) {
        // two sources, few records (a mixed-precision call of long units): both
        // sources' records loaded in one round (source 0's first), then merged
        float mr[kCombineRegs], sr[kCombineRegs], ar[kCombineRegs];
#pragma unroll
        for (int j = 0; j < kCombineRegs; ++j) {
            if (j < meta0.y + meta1.y) {
                const bool s0 = j < meta0.y;
                const size_t r = ((s0 ? r00 + j : r10 + (j - meta0.y))) * G + g;
                const float2 ml = *reinterpret_cast<const float2 *>((s0 ? p.ws_ml : p.ws_ml2) + r * 2);
                mr[j] = ml.x;
                sr[j] = ml.y;
                ar[j] = (s0 ? p.ws_acc : p.ws_acc2)[r * kHD + d];
            }
        }
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < kCombineRegs; ++j)
            if (j < meta0.y + meta1.y) m = fmaxf(m, mr[j]);
        float s_sum = 0.0f, a = 0.0f;
        if (m != -INFINITY) {
#pragma unroll
            for (int j = 0; j < kCombineRegs; ++j) {
                if (j < meta0.y + meta1.y) {
                    const float f = ex2_approx(mr[j] - m);
                    s_sum = fmaf(sr[j], f, s_sum);
                    a = fmaf(ar[j], f, a);
                }
            }
        }
        *o = s_sum > 0.0f ? __fdividef(a, s_sum) : 0.0f;
        return;
    }
    // more records: groups of kCombineRegs records, each group loaded at once
    // and merged into the running state with the same rescaling rule
    float m = -INFINITY, s_sum = 0.0f, a = 0.0f;
    auto merge_group = [&](const float *ml, const float *accp, size_t r0, int n) {
        float mr[kCombineRegs], sr[kCombineRegs], ar[kCombineRegs];
        float mg = -INFINITY;
#pragma unroll
        for (int j = 0; j < kCombineRegs; ++j) {
            if (j < n) {
                const size_t r = (r0 + j) * G + g;
                const float2 v = *reinterpret_cast<const float2 *>(ml + r * 2);
                mr[j] = v.x;
                sr[j] = v.y;
                ar[j] = accp[r * kHD + d];
                mg = fmaxf(mg, v.x);
            }
        }
        if (mg == -INFINITY) return;
        const float m_new = fmaxf(m, mg);
        const float f_old = ex2_approx(m - m_new);   // 0 while m is -inf
        s_sum *= f_old;
        a *= f_old;
#pragma unroll
        for (int j = 0; j < kCombineRegs; ++j) {
            if (j < n) {
                const float f = ex2_approx(mr[j] - m_new);
                s_sum = fmaf(sr[j], f, s_sum);
                a = fmaf(ar[j], f, a);
            }
        }
        m = m_new;
    };
    for (int j0 = 0; j0 < meta0.y; j0 += kCombineRegs)
        merge_group(p.ws_ml, p.ws_acc, r00 + j0, min(kCombineRegs, meta0.y - j0));
    for (int j0 = 0; j0 < meta1.y; j0 += kCombineRegs)
        merge_group(p.ws_ml2, p.ws_acc2, r10 + j0, min(kCombineRegs, meta1.y - j0));
    *o = s_sum > 0.0f ? __fdividef(a, s_sum) : 0.0f;
}

// The merge of the 4-bit decode, whose split writes unit u's records at
// u * nsplit + j: the records are loaded beside the unit's length (one load
// round, no record directory), and the length says how many of them this call
// wrote (int4_split_count); merged in the order of decode_combine_kernel.
__global__ void __launch_bounds__(kHD)
decode_combine_fixed_kernel(DecodeParams p, int G, int ns) {
    pdl_launch_dependents();   // (the 4-bit split releases this kernel by its end)
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
    return cudaLaunchKernelEx(&cfg, p.release_early ? decode_combine_kernel<true> : decode_combine_kernel<false>, p, group);
}

}  // namespace kvq8
