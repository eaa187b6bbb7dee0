// decode_tail.cuh -- the split over each row's own tokens, behind those that it
// shares: many units (sequence, kv head) of few 64-token stages.
//
// decode_split.cuh's kernel gives a unit to the seven consumer warps of a CTA,
// which pays for long contexts: of a unit of six stages each warp has one, and
// the queries, the meeting of the warps' states and the record are paid per
// unit and CTA (224 rows x 8 heads of 100 to 700 tokens: 80 us for what can be
// read in 28; here 48).  Here every warp is a worker by itself: it takes an equal,
// contiguous share of the sequence of all units' stages, keeps the state of its
// unit in registers and writes the unit's record from there.  A stage takes a
// lone warp some 7000 clocks, so warps count, not stages in flight: each has
// room for one stage, whose K is overwritten with the next one's when the dot
// products are done and whose V when the sums are, so that each copy has half a
// stage's time (12 warps an SM with one stage each against 6 with two: 48 us
// against 56).  Queries, block ids and a step's new token are loaded when the
// unit's first stage is asked for.  The dot products of a stage are
// decode_split.cuh's; the softmax goes by one reference per head for scores and V
// scales together, as in the tile kernel, so that a token of small V scale keeps
// its bits beside one of large V scale and little weight.  The kernel starts on
// the SMs that the tile kernel ahead has left and waits for it at its own end (28
// layers' step 119.7 -> 110.7 us).  Spilled are 196 to 224 bytes a thread with G =
// 1, 84 with 8, 8 to 52 with 2 and 4.
#pragma once

#include "decode_split.cuh"
#include "tile_rows.cuh"

namespace kvq8 {
namespace {

template <int G>
struct TailLay {
    static constexpr int kWarps = G == 8 ? 8 : 12;                     // (255 or 170 registers a thread)
    static constexpr int kP = (G * 2 * kPRowHalves * 2 + 15) / 16 * 16;
    static constexpr int oStage = 0;                                   // [warp]
    static constexpr int oP = kWarps * kStageBytes;                    // [warp]
    static constexpr int oQCodes = oP + kWarps * kP;
    static constexpr int oQScale = oQCodes + kWarps * G * kHD;
    static constexpr int oFull = oQScale + kWarps * G * kNQB * 4;
    static constexpr int oMisc = oFull + kWarps * 2 * 8;
    static constexpr int kBytes = oMisc + 320;
    static_assert(oQScale % 16 == 0 && oFull % 8 == 0 && oMisc % 16 == 0, "alignment");
    static_assert(kBytes <= kSmemLimit, "shared memory budget");
};

struct TailMisc {
    long long warp_tot[12];
    long long base[12];   // worker: stages ahead of its first sequence
    int b0[12];           // worker: that sequence
};
static_assert(sizeof(TailMisc) <= 320, "misc");

// Base-2 scores of a staged stage's tokens lane and lane + 32 (-inf where not va, vb) for the G query heads of a unit.
template <int G>
__device__ __forceinline__ void tail_scores(const unsigned char *st, const int8_t *q_codes, const float *q_scale, int lane,
                                            bool va, bool vb, float sm_scale_log2, float (&sa)[G], float (&sb)[G]) {
    const int8_t *kst = reinterpret_cast<const int8_t *>(st);
    const float *ks_st = reinterpret_cast<const float *>(st + kStageKBytes + kStageVBytes);
    const int ta = lane, tb = lane + 32;
    // ---- segment 2a: int32 block dots, lane = token ----
    int da[G][kNQB], db[G][kNQB];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int q = 0; q < kNQB; ++q) { da[g][q] = 0; db[g][q] = 0; }
#pragma unroll
    for (int cc = 0; cc < 8; ++cc) {
        const int4 ka = lds128(kst + ta * kHD + ((cc ^ (ta & 7)) << 4));
        const int4 kb = lds128(kst + tb * kHD + ((cc ^ (tb & 7)) << 4));
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int4 qw = lds128(q_codes + g * kHD + cc * 16);
            int x = da[g][cc >> 1], y = db[g][cc >> 1];
            x = __dp4a(ka.x, qw.x, x); y = __dp4a(kb.x, qw.x, y);
            x = __dp4a(ka.y, qw.y, x); y = __dp4a(kb.y, qw.y, y);
            x = __dp4a(ka.z, qw.z, x); y = __dp4a(kb.z, qw.z, y);
            x = __dp4a(ka.w, qw.w, x); y = __dp4a(kb.w, qw.w, y);
            da[g][cc >> 1] = x;
            db[g][cc >> 1] = y;
        }
    }
    const float ksa = ks_st[ta], ksb = ks_st[tb];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float4 qs = *reinterpret_cast<const float4 *>(q_scale + g * kNQB);
        float a = (float)da[g][0] * qs.x;
        a = fmaf((float)da[g][1], qs.y, a);
        a = fmaf((float)da[g][2], qs.z, a);
        a = fmaf((float)da[g][3], qs.w, a);
        float bb = (float)db[g][0] * qs.x;
        bb = fmaf((float)db[g][1], qs.y, bb);
        bb = fmaf((float)db[g][2], qs.z, bb);
        bb = fmaf((float)db[g][3], qs.w, bb);
        sa[g] = va ? a * ksa * sm_scale_log2 : -INFINITY;
        sb[g] = vb ? bb * ksb * sm_scale_log2 : -INFINITY;
    }
}

// The state takes these tokens in, vsa and vsb their V scales (0 where masked): Sl and acc are relative to the reference R;
// fresh says that there is none yet.  sa, sb: the scores, here made relative to it.  p_hi, p_lo: the warp's room for P.
template <int G>
__device__ __forceinline__ void tail_sums(const unsigned char *st, __half *p_hi, __half *p_lo, int lane, int n, int t4,
                                          float vsa, float vsb, float (&sa)[G], float (&sb)[G], bool fresh,
                                          float (&R)[G], float (&Sl)[G], float (&acc)[8][4]) {
    const int8_t *vst = reinterpret_cast<const int8_t *>(st) + kStageKBytes;
    const int ta = lane, tb = lane + 32;
    // n, t4: MMA fragment coordinates (lane / 4, lane % 4).
    // P.V for G <= 4 packs P's high fp16 parts into columns 0..G-1 and its
    // low parts into G..2G-1 of one MMA (half the MMAs); the columns' sums
    // are added at the segment's end.  Accumulator columns 2*t4, 2*t4 + 1
    // then belong to heads col_head0, col_head1 (for their rescaling).
    constexpr bool kPackPV = G <= 4;
    const int col_head0 = kPackPV ? (2 * t4) % G : 2 * t4;
    const int col_head1 = kPackPV ? (2 * t4 + 1) % G : 2 * t4 + 1;
    // ---- segment 2b: online softmax ----
    const float ea = exponent_above(vsa), eb = exponent_above(vsb);
    const float most_a = kPMaxLog2 - ea, most_b = kPMaxLog2 - eb;
    bool grow = fresh;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        sa[g] -= R[g];
        sb[g] -= R[g];
        grow |= sa[g] > most_a || sb[g] > most_b;
    }
    if (__any_sync(0xffffffffu, grow)) {
        float f0 = 0.0f, f1 = 0.0f;
        uint32_t leapt = 0;   // (by head)
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float top = redux_max_f32(fmaxf(sa[g] + ea, sb[g] + eb));
            float f = 1.0f;
            if (fresh || top > kPMaxLog2) {
                const float by = ceilf(top) - kPTopLog2;
                const float2 part = fresh ? make_float2(0.0f, 0.0f) : pow2_parts(-by);
                Sl[g] = Sl[g] * part.x * part.y;
                f = part.x * part.y;
                sa[g] -= by;
                sb[g] -= by;
                R[g] += by;
                if (fabsf(by) > 0x1p20f) leapt |= 1u << g;
            }
            if (g == col_head0) f0 = f;
            if (g == col_head1) f1 = f;
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            acc[mt][0] *= f0; acc[mt][1] *= f1;
            acc[mt][2] *= f0; acc[mt][3] *= f1;
        }
        if (__builtin_expect(leapt != 0, 0)) {
            // scores whose own rounding takes the distances that P depends on: now that they are small, they move once
            // more, exactly (what such a head held is 0)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (leapt >> g & 1) {
                    const float by = ceilf(redux_max_f32(fmaxf(sa[g] + ea, sb[g] + eb))) - kPTopLog2;
                    sa[g] -= by;
                    sb[g] -= by;
                    R[g] += by;
                }
            }
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float wa = ex2_approx(sa[g]), wb = ex2_approx(sb[g]);   // (masked: 0)
        Sl[g] += wa + wb;
        const float pa = wa * vsa, pb = wb * vsb;
        const __half ha = __float2half_rn(pa), hb = __float2half_rn(pb);
        p_hi[g * kPRowHalves + ta] = ha;
        p_hi[g * kPRowHalves + tb] = hb;
        p_lo[g * kPRowHalves + ta] = __float2half_rn(pa - __half2float(ha));
        p_lo[g * kPRowHalves + tb] = __float2half_rn(pb - __half2float(hb));
    }
    __syncwarp();

    // ---- segment 2c: acc += V . P on the tensor cores ----
    // B columns: kPackPV, head n's high part (n < G) or head n - G's
    // low part (G <= n < 2G); else the high part of head n in
    // bh and its low part in bl (two MMAs)
    uint32_t bh[8], bl[8];
    const __half *rh = kPackPV ? (n < G ? p_hi + n * kPRowHalves
                                        : (n < 2 * G ? p_lo + (n - G) * kPRowHalves : nullptr))
                               : (n < G ? p_hi + n * kPRowHalves : nullptr);
    if (rh) {
        const int4 h0 = lds128(rh + t4 * 16);
        const int4 h1 = lds128(rh + t4 * 16 + 8);
        bh[0] = h0.x; bh[1] = h0.y; bh[2] = h0.z; bh[3] = h0.w;
        bh[4] = h1.x; bh[5] = h1.y; bh[6] = h1.z; bh[7] = h1.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) bh[i] = 0u;
    }
    if (!kPackPV && n < G) {
        const int4 l0 = lds128(p_lo + n * kPRowHalves + t4 * 16);
        const int4 l1 = lds128(p_lo + n * kPRowHalves + t4 * 16 + 8);
        bl[0] = l0.x; bl[1] = l0.y; bl[2] = l0.z; bl[3] = l0.w;
        bl[4] = l1.x; bl[5] = l1.y; bl[6] = l1.z; bl[7] = l1.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) bl[i] = 0u;
    }
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
        const int d = mt * 16 + n;
        const int4 v0 = lds128(vst + d * kStageTok + t4 * 16);
        const int4 v1 = lds128(vst + (d + 8) * kStageTok + t4 * 16);
        const uint32_t w0[4] = {(uint32_t)v0.x, (uint32_t)v0.y, (uint32_t)v0.z, (uint32_t)v0.w};
        const uint32_t w1[4] = {(uint32_t)v1.x, (uint32_t)v1.y, (uint32_t)v1.z, (uint32_t)v1.w};
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint32_t a0, a2, a1, a3;
            codes_to_sub2(w0[s], a0, a2);
            codes_to_sub2(w1[s], a1, a3);
            a0 = sub2_signed(a0); a1 = sub2_signed(a1);
            a2 = sub2_signed(a2); a3 = sub2_signed(a3);
            mma_f16_16816(part, a0, a1, a2, a3, bh[2 * s], bh[2 * s + 1]);
            if (!kPackPV) mma_f16_16816(part, a0, a1, a2, a3, bl[2 * s], bl[2 * s + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][i] += part[i];
    }
}

// Where a warp is in the sequence of stages: stage j of unit (b, h), which has nb of the span sp.
struct TailCursor {
    int b, h, j, nb;
    SeqSpan sp;
    __device__ __forceinline__ void load(const DecodeParams &p, int cap) {   // the sequence b, or the next that has stages
        for (; b < p.batch; ++b, h = 0) {
            sp = seq_span<false, kTail>(p, b, cap);
            nb = span_stages(sp);
            if (nb > 0) return;
        }
    }
    __device__ __forceinline__ void next_unit(const DecodeParams &p, int cap) {
        j = 0;
        if (++h < p.nkv) return;
        h = 0;
        ++b;
        load(p, cap);
    }
};

template <int G>
__global__ void __launch_bounds__((TailLay<G>::kWarps * 32), 1)
decode_tail_kernel(DecodeParams p) {
    using Lay = TailLay<G>;
    constexpr int kTailWarps = Lay::kWarps;
    extern __shared__ __align__(1024) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cap = p.max_blocks * kBS;
    TailMisc *ms = reinterpret_cast<TailMisc *>(smem + Lay::oMisc);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Lay::oFull) + warp * 2;   // of K and scales, of V
    if (lane < 2) {
        mbar_init(smem_addr(full + lane), 1);
        fence_mbar_init();
    }
    // No wait here: nothing below reads what the tile kernel ahead writes, and what is ahead of that kernel (the plan's
    // ws_tail among it) was done when its CTAs let this kernel start.  The CTAs begin on the SMs that it has left, and
    // each waits for it before it leaves itself, so that the merge behind finds both done.  What the wait would order is
    // ordered here: a word of the plan read at GPU scope, then a fence, so that no load below takes a line that an earlier
    // call left in this SM's L1.
    acquire_gpu(p.windows);
    // ---- the workers' shares of all units' stages ----
    const int per = (p.batch + kTailWarps * 32 - 1) / (kTailWarps * 32);
    const int b_lo = min(p.batch, tid * per), b_hi = min(p.batch, b_lo + per);
    long long mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int L = p.ctx_lens[b];
        if (blockIdx.x == 0 && (L < 0 || L > cap)) flag_status(p.dev_status, KVQ8_DEV_BAD_CTX_LEN);
        mine += (long long)p.nkv * span_stages(seq_span<false, kTail>(p, b, cap));
    }
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) ms->warp_tot[warp] = before;
    __syncthreads();
    before -= mine;
    long long T = 0;
    for (int k = 0; k < kTailWarps; ++k) {
        if (k < warp) before += ms->warp_tot[k];
        T += ms->warp_tot[k];
    }
    // consecutive workers lie on different SMs
    const int W = (int)min((long long)gridDim.x * kTailWarps, T);
    auto share = [&](int worker) {   // its first stage
        const long long q = T / W;
        const int r = (int)(T - q * W);
        return (long long)worker * q + ((long long)worker * r) / W;
    };
    if (mine > 0) {
        for (int k = 0; k < kTailWarps; ++k) {
            const int worker = k * gridDim.x + blockIdx.x;
            if (worker >= W) break;
            const long long lo = share(worker);
            if (lo < before || lo >= before + mine) continue;
            long long acc = before;
            for (int b = b_lo; b < b_hi; ++b) {
                const long long n = (long long)p.nkv * span_stages(seq_span<false, kTail>(p, b, cap));
                if (lo < acc + n) {
                    ms->b0[k] = b;
                    ms->base[k] = acc;
                    break;
                }
                acc += n;
            }
        }
    }
    __syncthreads();
    const int worker = warp * gridDim.x + blockIdx.x;
    if (worker >= W) {
        pdl_wait();
        return;
    }
    const long long lo = share(worker);
    const int total = (int)(share(worker + 1) - lo);

    unsigned char *st = smem + Lay::oStage + warp * kStageBytes;
    const float *vs_st = reinterpret_cast<const float *>(st + kStageKBytes + kStageVBytes) + kStageTok;
    __half *p_hi = reinterpret_cast<__half *>(smem + Lay::oP + warp * Lay::kP), *p_lo = p_hi + G * kPRowHalves;
    int8_t *q_codes = reinterpret_cast<int8_t *>(smem + Lay::oQCodes) + warp * G * kHD;
    float *q_scale = reinterpret_cast<float *>(smem + Lay::oQScale) + warp * G * kNQB;
    const int n = lane >> 2, t4 = lane & 3;   // MMA fragment coordinates

    TailCursor at;   // the stage that is decoded
    at.b = ms->b0[warp];
    at.load(p, cap);
    {
        const long long rel = lo - ms->base[warp];
        at.h = (int)(rel / at.nb);
        at.j = (int)(rel - (long long)at.h * at.nb);
    }
    TailCursor ask = at;   // the stage that is copied next
    // of the unit that is asked for: queries, new token, block ids
    float qx[G][4];
    float4 nxk = make_float4(0.f, 0.f, 0.f, 0.f), nxv = nxk;
    int blk = -1, phys = -1, phys_next = -1, new_phys = -1;
    auto enter = [&]() {
        const float *q = p.q + ((size_t)ask.b * p.nqh + (size_t)ask.h * G) * kHD;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k) qx[g][k] = q[g * kHD + 32 * k + lane];
        if (p.k_new) {
            const size_t src = ((size_t)ask.b * p.nkv + ask.h) * kHD;
            nxk = reinterpret_cast<const float4 *>(p.k_new + src)[lane];
            nxv = reinterpret_cast<const float4 *>(p.v_new + src)[lane];
            new_phys = p.block_table[(size_t)ask.b * p.max_blocks + (ask.sp.y - 1) / kBS];
        }
        blk = -1;
    };
    const uint64_t pol = l2_evict_first_policy();
    bool skip = false, skip_next = false;   // the stage's block id is outside the pool
    size_t tile = 0;
    int quarter = 0;
    auto copy_k = [&]() {   // K and the scales of the stage that is asked for
        const int t0 = ask.sp.x + ask.j * kStageTok, lb = t0 / kBS;
        quarter = (t0 / kStageTok) & 3;
        if (lb != blk) {
            const int32_t *row = p.block_table + (size_t)ask.b * p.max_blocks;
            phys = blk >= 0 ? phys_next : row[lb];
            phys_next = lb + 1 < p.max_blocks ? row[lb + 1] : -1;   // (in time for the next block)
            blk = lb;
        }
        skip_next = phys < 0 || phys >= p.num_blocks;
        tile = skip_next ? 0 : (size_t)phys * p.nkv + ask.h;
        if (lane == 0) {
            const uint32_t bar = smem_addr(full), dst = smem_addr(st);
            if (!skip_next) {
                mbar_arrive_expect_tx(bar, kStageKBytes + 2 * kStageSBytes);
                bulk_copy_g2s(dst, p.k_pool + (tile * kBS + quarter * kStageTok) * kHD, kStageKBytes, bar, pol);
                bulk_copy_g2s(dst + kStageKBytes + kStageVBytes, p.k_scale + tile * kBS + quarter * kStageTok, kStageSBytes, bar, pol);
                bulk_copy_g2s(dst + kStageKBytes + kStageVBytes + kStageSBytes, p.v_scale + tile * kBS + quarter * kStageTok,
                              kStageSBytes, bar, pol);
            } else {
                flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
                mbar_arrive(bar);
            }
        }
    };
    auto copy_v = [&]() {   // V of the same stage
        if (lane == 0) {
            const uint32_t bar = smem_addr(full + 1);
            if (!skip_next) {
                mbar_arrive_expect_tx(bar, kStageVBytes);
                bulk_copy_g2s(smem_addr(st + kStageKBytes), p.v_pool + tile * kHD * kBS + quarter * kTileVQuarter, kStageVBytes, bar, pol);
            } else {
                mbar_arrive(bar);
            }
        }
    };
    float R[G], Sl[G], acc[8][4];
    bool begin = true, fresh = true, gave_up = false;
    auto wait = [&](int which, int k) {
        if (!gave_up && !mbar_wait_tries(smem_addr(full + which), k & 1)) {
            gave_up = true;
            if (lane == 0) flag_status(p.dev_status, KVQ8_DEV_TIMEOUT);
        }
        gave_up = __any_sync(0xffffffffu, gave_up);
    };
    enter();
    copy_k();
    copy_v();
    int copied = 1;   // stages asked for
#pragma unroll 1
    for (int k = 0; k < total && !gave_up; ++k) {
        if (begin) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                quantize_q_vals_warp(qx[g], lane, q_codes + g * kHD, q_scale + g * kNQB, p.dev_status);
                R[g] = Sl[g] = 0.0f;
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][i] = 0.0f;
            fresh = true;
            __syncwarp();
        }
        skip = skip_next;
        const int t0 = at.sp.x + at.j * kStageTok, pos = at.sp.y - 1;
        const bool va = t0 + lane >= at.sp.lo && t0 + lane < at.sp.y;
        const bool vb = t0 + lane + 32 >= at.sp.lo && t0 + lane + 32 < at.sp.y;
        wait(0, k);
        // (a step's token: at the end of a context that the table holds)
        const bool append = p.k_new && pos - t0 < kStageTok && !skip && p.ctx_lens[at.b] == at.sp.y;
        if (append) {
            wait(1, k);
            append_new_token<false>(p, at.b, at.h, pos, pos - t0, lane, st, nxk, nxv, new_phys);
            fence_async_smem();   // (the next copies overwrite what it wrote)
            __syncwarp();
        }
        float sa[G], sb[G], vsa = 0.0f, vsb = 0.0f;
        if (!skip) {
            tail_scores<G>(st, q_codes, q_scale, lane, va, vb, p.sm_scale_log2, sa, sb);
            if (va) vsa = vs_st[lane];
            if (vb) vsb = vs_st[lane + 32];
        }
        __syncwarp();
        if (k + 1 < total && !gave_up) {   // K's room is free
            if (++ask.j == ask.nb) {
                ask.next_unit(p, cap);
                enter();
            }
            copy_k();
            ++copied;
        }
        if (!append) wait(1, k);
        if (!skip) {
            tail_sums<G>(st, p_hi, p_lo, lane, n, t4, vsa, vsb, sa, sb, fresh, R, Sl, acc);
            fresh = false;
        }
        __syncwarp();
        if (copied == k + 2) copy_v();
        begin = ++at.j == at.nb;
        if (begin || k + 1 == total) {
            // ---- the record of this worker's part of the unit ----
            const size_t u = (size_t)at.b * p.nkv + at.h, rec = worker + u;
            if (G <= 4) {
#pragma unroll
                for (int mt = 0; mt < 8; ++mt) {
                    if (G == 1) {
                        acc[mt][0] += acc[mt][1];
                        acc[mt][2] += acc[mt][3];
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[mt][i] += __shfl_xor_sync(0xffffffffu, acc[mt][i], G / 2);
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float s = warp_sum(Sl[g]);
                if (lane == 0) *reinterpret_cast<float2 *>(p.ws_ml + (rec * G + g) * 2) = make_float2(s > 0.0f ? R[g] : -INFINITY, s);
            }
            float *out = p.ws_acc + rec * G * kHD + n;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int g = 2 * t4 + i;
                    if (g < G) {
                        out[g * kHD + mt * 16] = acc[mt][i] * kCodeUnit;
                        out[g * kHD + mt * 16 + 8] = acc[mt][2 + i] * kCodeUnit;
                    }
                }
            }
            const int first = k + 1 - at.j;   // the unit's first stage, as a stage of this worker's
            if (lane == 0 && first >= 0)
                p.ws_meta[u] = make_int2(worker, (int)(((lo + first + at.nb) * W + T - 1) / T) - worker);
            if (begin) at.next_unit(p, cap);
        }
    }
    // no copy may still be in flight when the warp leaves (after a wait that gave up)
    if (gave_up && lane == 0) {
        for (int i = 0; i < 2; ++i) mbar_wait_bounded(smem_addr(full + i), (copied - 1) & 1, kWaitTimeoutNs);
    }
    pdl_wait();
    pdl_launch_dependents();
}

template <int G>
cudaError_t launch_tail_g(const DecodeParams &p, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(min(sms, kMaxTailWorkers / TailLay<G>::kWarps));   // (a record per worker)
    cfg.blockDim = dim3(TailLay<G>::kWarps * 32);
    cfg.dynamicSmemBytes = TailLay<G>::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_after_setting(
        configured,
        [] {
            return cudaFuncSetAttribute(decode_tail_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, TailLay<G>::kBytes);
        },
        [&] { return cudaLaunchKernelEx(&cfg, decode_tail_kernel<G>, p); });
}

}  // namespace
}  // namespace kvq8
