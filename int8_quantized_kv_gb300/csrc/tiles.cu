// tiles.cu -- attention of many query rows over a cached stretch on the
// 5th-generation tensor cores: prompts, and the prefixes that batch rows share.
//
// The mathematics is the decode's: the query in 32-blocks of int8 codes, s_t =
// (sum_b dot_b qscale_b) kscale_t sm_scale, a softmax in base 2 with a running
// maximum, V entering as code * (weight * vscale).  Here up to 128 query rows
// that share a kv head (a tile) meet 128 cached tokens at a time, as two
// products whose left operand is the cache:
//   S^T [tokens x rows] = K [tokens x 128] Q^T,   O^T [128 x rows] += V^T [128 x tokens] P^T
// The cache's own order is what a left operand in tensor memory wants: a lane
// per token for K (token-major rows), a lane per dim for V (dim-major), so the
// codes go from the bulk-copied stage through registers (int8 -> fp16, exact)
// into tensor memory with neither a transpose nor a second pass through shared
// memory, and the right operands' row count is the tile's own (a multiple of
// 16), so that few rows cost little softmax work.
//
// fp32-class results from fp16 operands: the codes are exact; a query row's
// values code * scale and the weights P enter as a high and a low fp16 part
// (22 bits).  Of a tile of up to 64 rows both parts are columns of one product
// (A from tensor memory feeds at most 128 columns per 64 cycles, so the second
// part is free); of up to 128 rows they are two products into one accumulator.
// bf16 outputs take P's high part alone: 11 bits of each weight, an eighth of
// the output's own rounding.
//
// A persistent CTA per SM takes an equal share of the (tile, 128-token stage)
// sequence.  Warp 0 copies the stages (bulk copies into a ring), warp 1 issues
// the MMAs, warps 4..7 turn the codes into operands and, per tile, the queries,
// warps 8..15 take the softmax: the score tile is S^T, so a thread holds one
// token of half the tile's rows, whose row sums it keeps for itself until the
// tile ends.  A row's weights 2^(s - M) need no exact maximum: M is set so that
// the row's largest weight * V scale fills fp16's range, and moved only when one
// would leave it (a factor of 2^7 or more later), which a comparison per score
// and one barrier over the eight warps find out; maxima across lanes are formed
// only then.  (With M from the scores alone a row that leans on tokens of small
// V would lose P's low bits next to one large V scale.)
#include <math.h>

#include "kvq8_ptx.cuh"
#include "tile_rows.cuh"

namespace kvq8 {
namespace {

constexpr int kTok = 128;                       // tokens per stage
constexpr int kThreads = 512;
constexpr int kCodeBytes = kTok * kHD;          // 16 KiB of K or V codes
constexpr int kSlotBytes = kCodeBytes + 2 * kTok * 4;   // K codes with both scales, or V codes
constexpr int kCoreRow = 2048;                  // bytes between cores along the rows (16 cores of 128 B along k)
constexpr uint64_t kLimitNs = 2000000000ull;
// A row's reference M: P = 2^(s - M) * V scale, whose maximum is put between 2^8 and 2^9 when M is set; M moves
// when P would pass 2^15.9 (fp16 ends below 2^16).
constexpr float kPTopLog2 = 9.0f, kPMaxLog2 = 15.9f;
constexpr float kTinyScaleLog2 = -60.0f;        // V scales below count as this when M is set (rows of zeros do)
// registers per thread of the four warpgroups: copies and MMAs, operands, softmax (2); their sum is what the
// launch holds (4 * 128)
constexpr int kRegsIssue = 64, kRegsOperand = 96, kRegsSoftmax = 176;
static_assert(kRegsIssue + kRegsOperand + 2 * kRegsSoftmax == 4 * 128, "the launch's registers");
// columns of tensor memory
constexpr int kColK = 0, kColV = 128, kColS = 256, kColO = 384;

// Rows per tile and shared memory: Q (high, low), P (high, low), the ring.
template <bool kWide, bool kLow>
struct Lay {
    static constexpr int kRows = kWide ? 128 : 64;
    static constexpr int kQ = kRows * 2 * kHD * 2;
    static constexpr int kP = kRows * (kLow ? 2 : 1) * kTok * 2;
    static constexpr int oQ = 0;
    static constexpr int oP = kQ;
    static constexpr int oMisc = oP + kP;
    static constexpr int kMisc = 12288;
    static constexpr int oRing = oMisc + kMisc;
    static constexpr int kSlots = (232448 - oRing) / kSlotBytes < 8 ? (232448 - oRing) / kSlotBytes : 8;
    static constexpr int kBytes = oRing + kSlots * kSlotBytes;
    static_assert(kSlots >= 4, "ring too shallow");
};

struct Misc {
    uint64_t full[8], empty[8];                 // ring slots
    uint64_t k_ready[2], k_free[2], v_ready[2], v_free[2], sc_ready[4];
    // (two, since the operand warps may be two tiles ahead of the softmax's)
    uint64_t q_ready[2];
    uint64_t s_full, s_free, p_ready, pv_done, q_free, o_free, all_done;
    long long warp_tot[kThreads / 32];
    long long base, end;
    int s0, r0;
    volatile int abort;
    uint32_t tmem;
    int skip[8];                                // slot: its block id is outside the pool
    int bad[4];                                 // stage (mod 4): the same
    int lim_min[2];
    alignas(16) float2 scale[4][kTok];          // stage (mod 4): (K scale * sm_scale, V scale)
    alignas(16) float2 col[2 * kTileRows];      // per row: (score factor, -M)
    alignas(16) int lim[kTileRows];             // per row: tokens below
    alignas(16) float alpha[kTileRows];
    alignas(16) float wave[4][kTileRows];       // per warp and row: maxima, sums
    float factor[2][kTileRows];                 // per tile (mod 2) and row: power of two of the query's operand
};
static_assert(sizeof(Misc) <= 12288, "misc");

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Misc *ms, uint32_t *status) {
    const uint32_t a = smem_addr(bar);
    if (mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(a, parity)) {
        if (ms->abort) return false;
        if (global_timer_ns() - t0 > kLimitNs) {
            ms->abort = 1;
            flag_status(status, KVQ8_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}

// The same by all lanes of a warp, together again behind it.
__device__ __forceinline__ void wait_warp(uint64_t *bar, uint32_t parity, Misc *ms, uint32_t *status) {
    wait_bar(bar, parity, ms, status);
    __syncwarp();
}

// The tiles in their order: (sequence or group, kv head, rows).
template <bool kShared>
struct Walk {
    const TileParams &p;
    const int lg, rows_per_tile, cap;
    int s = 0, h = 0, r = 0;
    int rows = 0;          // of the sequence or group, per kv head
    int first = 0;         // shared: first batch row; prompt: unused
    int lead = 0, span = 0;
    long long start = 0;   // prompt: position of the first query token

    __device__ Walk(const TileParams &p_, int lg_, int rows_) : p(p_), lg(lg_), rows_per_tile(rows_), cap(p_.max_blocks * kBS) {}
    __device__ void load(int s_) {
        s = s_;
        if (kShared) {
            const int4 g = p.ws_group[s];
            first = g.x;
            lead = g.z;
            span = g.w;
            rows = span > 0 ? g.y << lg : 0;
        } else {
            const int n = p.n_tokens ? max(0, min(p.n_new, p.n_tokens[s])) : p.n_new;
            rows = n << lg;
            start = p.start_pos[s];
            lead = s;
        }
    }
    __device__ int tiles() const { return (rows + rows_per_tile - 1) / rows_per_tile; }
    __device__ int tile_rows(int r_) const { return min(rows_per_tile, rows - r_ * rows_per_tile); }
    // Tokens that the tile's rows look at: [0, end)
    __device__ int end(int r_) const {
        if (kShared) return span;
        const long long e = start + (((long long)r_ * rows_per_tile + tile_rows(r_)) >> lg);
        return (int)max(0ll, min((long long)cap, e));
    }
    __device__ int stages(int r_) const { return max(1, (end(r_) + kTok - 1) / kTok); }
    // Tokens that row n of tile r_ looks at; bad: its position is outside the table.
    __device__ int limit(int r_, int n, bool &bad) const {
        const int i = (r_ * rows_per_tile + n) >> lg;
        if (kShared) {
            bad = false;
            return p.ws_tail[first + i];
        }
        const long long e = start + i + 1;
        bad = e < 1 || e > cap;
        return (int)max(0ll, min((long long)cap, e));
    }
    __device__ long long token(int r_, int n) const {   // row of q and out that row n belongs to
        const int i = (r_ * rows_per_tile + n) >> lg;
        return kShared ? first + i : (long long)s * p.n_new + i;
    }
    __device__ int head(int n) const { return (h << lg) + (n & ((1 << lg) - 1)); }
    __device__ void next(int count) {
        if (++r < tiles()) return;
        r = 0;
        if (++h < p.nkv) return;
        h = 0;
        for (++s; s < count; ++s) {
            load(s);
            if (rows > 0) return;
        }
    }
};

// int8 codes of four consecutive contraction elements -> two fp16 pairs, exact:
// a byte below 0x64 is the half 1024 + (code + 128).
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t x = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// 32 bytes of codes (two 16-byte chunks) into 16 columns of this lane.
__device__ __forceinline__ void put_codes(uint32_t tmem, uint4 x, uint4 y) {
    uint32_t v[8];
    codes_to_half2(x.x, v[0], v[1]);
    codes_to_half2(x.y, v[2], v[3]);
    codes_to_half2(x.z, v[4], v[5]);
    codes_to_half2(x.w, v[6], v[7]);
    tmem_st8(tmem, v);
    codes_to_half2(y.x, v[0], v[1]);
    codes_to_half2(y.y, v[2], v[3]);
    codes_to_half2(y.z, v[4], v[5]);
    codes_to_half2(y.w, v[6], v[7]);
    tmem_st8(tmem + 8, v);
}

__device__ __forceinline__ uint32_t half2_bits(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }   // -126 .. 127

// Floats as integers of the same order, so that one redux gives a maximum.
__device__ __forceinline__ float warp_top(float x) {
    int k = __float_as_int(x);
    k ^= (k >> 31) & 0x7fffffff;
    k = __reduce_max_sync(0xffffffffu, k);
    k ^= (k >> 31) & 0x7fffffff;
    return __int_as_float(k);
}

template <bool kShared, bool kWide, bool kLow>
__global__ void __launch_bounds__(kThreads, 1)
tile_kernel(TileParams p, int lg) {
    using L = Lay<kWide, kLow>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Misc *ms = reinterpret_cast<Misc *>(smem + L::oMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x;
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(smem_addr(&ms->full[i]), 1);
            mbar_init(smem_addr(&ms->empty[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ms->q_ready[i]), 4);
            mbar_init(smem_addr(&ms->k_ready[i]), 4);
            mbar_init(smem_addr(&ms->k_free[i]), 1);
            mbar_init(smem_addr(&ms->v_ready[i]), 4);
            mbar_init(smem_addr(&ms->v_free[i]), 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(smem_addr(&ms->sc_ready[i]), 4);
        mbar_init(smem_addr(&ms->s_full), 1);
        mbar_init(smem_addr(&ms->s_free), 8);
        mbar_init(smem_addr(&ms->p_ready), 8);
        mbar_init(smem_addr(&ms->pv_done), 1);
        mbar_init(smem_addr(&ms->q_free), 1);
        mbar_init(smem_addr(&ms->o_free), 8);
        mbar_init(smem_addr(&ms->all_done), 1);
        fence_mbar_init();
        ms->abort = 0;
        ms->s0 = 0;
        ms->r0 = 0;
        ms->lim_min[0] = ms->lim_min[1] = 0x7fffffff;
    }
    if (warp == 1) tmem_alloc(smem_addr(&ms->tmem), 512);
    pdl_wait();
    pdl_launch_dependents();   // (the next kernel's CTAs find no registers here before this one leaves)
    // ---- this CTA's share: stages [lo, hi) of the sequence of all tiles' stages ----
    Walk<kShared> w(p, lg, L::kRows);
    const int per_seq = kShared ? 1 : (int)((((long long)p.n_new << lg) + L::kRows - 1) / L::kRows);
    const int seqs = kShared ? p.n_groups : p.batch;
    const long long items = (long long)seqs * per_seq;   // (sequence, tile of one kv head), or group
    const long long per = (items + kThreads - 1) / kThreads;
    const long long i_lo = min(items, tid * per), i_hi = min(items, i_lo + per);
    auto item = [&](long long i, int &s, int &r) {
        s = (int)(i / per_seq);
        r = (int)(i % per_seq);
        w.load(s);
        if (kShared) return (long long)w.tiles() * w.stages(0) * (w.rows > 0);
        return r < w.tiles() ? (long long)w.stages(r) : 0ll;
    };
    long long mine = 0;
    int s, r;
    for (long long i = i_lo; i < i_hi; ++i) mine += item(i, s, r);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) ms->warp_tot[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long excl = incl - mine, total = 0;
    for (int k = 0; k < kThreads / 32; ++k) {
        if (k < warp) excl += ms->warp_tot[k];
        total += ms->warp_tot[k];
    }
    const long long T = total * p.nkv;
    const int C = (int)min((long long)gridDim.x, T);
    long long lo = 0, hi = 0;
    if (c < C) {
        const long long Tq = T / C;
        const int Tr = (int)(T - Tq * C);
        lo = (long long)c * Tq + ((long long)c * Tr) / C;
        hi = (long long)(c + 1) * Tq + ((long long)(c + 1) * Tr) / C;
    }
    if (!kShared && tid == 0) p.ws_dir[c] = make_int4(0, 0, 0, 0);
    const uint32_t tmem = ms->tmem;
    int off = 0;
    if (hi > lo) {   // (uniform over the CTA)
        long long acc = excl;
        for (long long i = i_lo; i < i_hi; ++i) {
            const long long v = item(i, s, r);
            if (r == 0 && acc * p.nkv <= lo) atomicMax(&ms->s0, s);
            acc += v;
        }
        if (tid == 0) ms->end = total;
        __syncthreads();
        const int s0 = ms->s0;
        acc = excl;
        for (long long i = i_lo; i < i_hi; ++i) {
            const long long v = item(i, s, r);
            if (r == 0 && s == s0) ms->base = acc;
            if (r == 0 && s == s0 + 1) ms->end = acc;
            acc += v;
        }
        __syncthreads();
        const long long base = ms->base, W = ms->end - base;
        long long rem = lo - base * p.nkv;
        const int h0 = (int)(rem / W);
        rem -= h0 * W;
        if (kShared) {
            w.load(s0);
            w.r = (int)(rem / w.stages(0));
            off = (int)(rem % w.stages(0));
        } else {
            acc = excl;
            for (long long i = i_lo; i < i_hi; ++i) {
                const long long v = item(i, s, r);
                if (s == s0 && v > 0 && acc - base <= rem) atomicMax(&ms->r0, r);
                acc += v;
            }
            __syncthreads();
            w.r = ms->r0;
            acc = excl;
            for (long long i = i_lo; i < i_hi; ++i) {
                const long long v = item(i, s, r);
                if (s == s0 && r == w.r) ms->end = rem - (acc - base);
                acc += v;
            }
            __syncthreads();
            off = (int)ms->end;
            w.load(s0);
        }
        w.h = h0;
    }
    long long left = hi - lo;
    // `part` stages of tile (w.s, w.h, w.r) from stage `off` on are this CTA's
#define KVQ8_FOR_TILES                                                                                    \
    for (int part = 0, seg = 0; left > 0 && !(seg > 0 && w.s >= seqs);                                   \
         left -= part, off = 0, ++seg, w.next(seqs))                                                       \
        if (part = (int)min(left, (long long)(w.stages(w.r) - off)), true)

    if (warp < 4) {
        regs_shrink<kRegsIssue>();
        if (warp == 0) {
            // ============================ copies ============================
            int g = 0;   // granules so far: K and V of every stage
            bool stop = false;
            KVQ8_FOR_TILES {
                const int end = w.end(w.r);
                const int32_t *row = p.block_table + (size_t)w.lead * p.max_blocks;
                int tbl_base = -1, tbl = -1;
                for (int j = 0; j < part && !stop; ++j, g += 2) {
                    const int t0 = (off + j) * kTok, lb = t0 / kBS;
                    if (tbl_base < 0 || lb >= tbl_base + 32) {
                        tbl_base = lb;
                        tbl = lb + lane < p.max_blocks ? row[lb + lane] : -1;
                    }
                    const int phys = __shfl_sync(0xffffffffu, tbl, lb - tbl_base);
                    if (lane == 0) {
                        const bool any = t0 < end, ok = any && phys >= 0 && phys < p.num_blocks;
                        if (any && !ok) flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
                        const size_t tile = ok ? (size_t)phys * p.nkv + w.h : 0;
                        const int slot0 = t0 % kBS;
                        for (int v = 0; v < 2 && !stop; ++v) {
                            const int at = (g + v) % L::kSlots;
                            if (!wait_bar(&ms->empty[at], (((g + v) / L::kSlots) & 1) ^ 1, ms, p.dev_status)) {
                                stop = true;
                                break;
                            }
                            const uint32_t bar = smem_addr(&ms->full[at]);
                            const uint32_t dst = smem_addr(smem + L::oRing + at * kSlotBytes);
                            ms->skip[at] = !ok;
                            if (!ok) {
                                mbar_arrive(bar);
                            } else if (v == 0) {
                                mbar_arrive_expect_tx(bar, kCodeBytes + 2 * kTok * 4);
                                bulk_copy_g2s_plain(dst, p.k_pool + (tile * kBS + slot0) * kHD, kCodeBytes, bar);
                                bulk_copy_g2s_plain(dst + kCodeBytes, p.k_scale + tile * kBS + slot0, kTok * 4, bar);
                                bulk_copy_g2s_plain(dst + kCodeBytes + kTok * 4, p.v_scale + tile * kBS + slot0, kTok * 4, bar);
                            } else {
                                mbar_arrive_expect_tx(bar, kCodeBytes);
                                bulk_copy_g2s_plain(dst, p.v_pool + tile * kBS * kHD + (size_t)slot0 * kHD, kCodeBytes, bar);
                            }
                        }
                    }
                    stop = __shfl_sync(0xffffffffu, (int)stop, 0) != 0;
                }
                if (stop) break;
            }
            // no copy may still be in flight when the CTA exits (a stopped ring: whichever the slots were given last)
            if (lane == 0) {
                for (int k = max(0, g - L::kSlots); k < g; ++k)
                    mbar_wait_bounded(smem_addr(&ms->full[k % L::kSlots]), (k / L::kSlots) & 1, kLimitNs);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ============================= MMAs =============================
            if (lane == 0) {
                const uint32_t q0 = smem_addr(smem + L::oQ), p0 = smem_addr(smem + L::oP);
                int j = 0;   // stages so far
                KVQ8_FOR_TILES {
                    const int n = (w.tile_rows(w.r) + 15) & ~15;
                    const uint32_t word_q = mma_word(kWide ? n : 2 * n, false);
                    const uint32_t word_p = mma_word(kWide || !kLow ? n : 2 * n, true);
                    wait_bar(&ms->q_ready[seg & 1], (seg >> 1) & 1, ms, p.dev_status);
                    for (int i = 0; i <= part; ++i) {
                        if (i < part) {
                            const int x = j + i;
                            wait_bar(&ms->k_ready[x & 1], (x >> 1) & 1, ms, p.dev_status);
                            wait_bar(&ms->s_free, (x & 1) ^ 1, ms, p.dev_status);
                            tc_fence_after();
                            const uint32_t a = tmem + kColK + (x & 1) * 64;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mma_tmem_a(tmem + kColS, a + 8 * k, core_desc(q0 + k * 256, 128, kCoreRow), word_q, k > 0);
                            if (kWide) {
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    mma_tmem_a(tmem + kColS, a + 8 * k,
                                               core_desc(q0 + L::kRows / 8 * kCoreRow + k * 256, 128, kCoreRow), word_q, true);
                            }
                            mma_commit(smem_addr(&ms->k_free[x & 1]));
                            mma_commit(smem_addr(&ms->s_full));
                            if (i == part - 1) mma_commit(smem_addr(&ms->q_free));
                        }
                        if (i > 0) {
                            const int x = j + i - 1;
                            wait_bar(&ms->v_ready[x & 1], (x >> 1) & 1, ms, p.dev_status);
                            if (i == 1) wait_bar(&ms->o_free, (seg & 1) ^ 1, ms, p.dev_status);
                            wait_bar(&ms->p_ready, x & 1, ms, p.dev_status);
                            tc_fence_after();
                            const uint32_t a = tmem + kColV + (x & 1) * 64;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mma_tmem_a(tmem + kColO, a + 8 * k, core_desc(p0 + k * 256, 128, kCoreRow), word_p, i > 1 || k > 0);
                            if (kWide && kLow) {
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    mma_tmem_a(tmem + kColO, a + 8 * k,
                                               core_desc(p0 + L::kRows / 8 * kCoreRow + k * 256, 128, kCoreRow), word_p, true);
                            }
                            mma_commit(smem_addr(&ms->v_free[x & 1]));
                            mma_commit(smem_addr(&ms->pv_done));
                        }
                    }
                    j += part;
                }
                mma_commit(smem_addr(&ms->all_done));
                mbar_wait_bounded(smem_addr(&ms->all_done), 0, kLimitNs);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        regs_shrink<kRegsOperand>();
        // ========================= operands =========================
        const int quad = warp & 3, row = 32 * quad + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        int j = 0;
        KVQ8_FOR_TILES {
            // the tile's queries: high and low parts of code * scale, in units of a power of two per row
            const int rows = w.tile_rows(w.r), n = (rows + 15) & ~15;
            wait_warp(&ms->q_free, (seg & 1) ^ 1, ms, p.dev_status);
            for (int i = quad; i < n; i += 4) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < rows) x = load4(p.q, p.q_dtype, w.token(w.r, i) * p.q_stride + (int64_t)w.head(i) * kHD + 4 * lane);
                // lane l: dims 4l .. 4l + 3, a 32-block is eight lanes; the rule of quantize_q_vals_warp
                uint32_t m = max(max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu),
                                 max(__float_as_uint(x.z) & 0x7fffffffu, __float_as_uint(x.w) & 0x7fffffffu));
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (m >= 0x7f800000u) {
                    x = make_float4(0.f, 0.f, 0.f, 0.f);
                    m = 0;
                    if ((lane & 7) == 0) flag_status(p.dev_status, KVQ8_DEV_NONFINITE);
                }
                float qm = __uint_as_float(m);
                if (qm < 1e-6f) qm = 1.0f;
                const float iq = __fdiv_rn(127.0f, qm), qs = __fmul_rn(qm, KVQ8_INV127);
                auto value = [&](float v) { return __fmul_rn((float)max(-128, min(127, __float2int_rn(__fmul_rn(v, iq)))), qs); };
                x = make_float4(value(x.x), value(x.y), value(x.z), value(x.w));
                // exponent of the row's largest value: the row is scaled to below 2^11
                int e = max(max(__float_as_int(x.x) & 0x7fffffff, __float_as_int(x.y) & 0x7fffffff),
                            max(__float_as_int(x.z) & 0x7fffffff, __float_as_int(x.w) & 0x7fffffff));
                e = max(-100, (__reduce_max_sync(0xffffffffu, e) >> 23) - 127 - 10);
                const float down = exp2_int(-e);
                x = make_float4(x.x * down, x.y * down, x.z * down, x.w * down);
                const __half2 h0 = __floats2half2_rn(x.x, x.y), h1 = __floats2half2_rn(x.z, x.w);
                const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
                const __half2 l0 = __floats2half2_rn(x.x - f0.x, x.y - f0.y), l1 = __floats2half2_rn(x.z - f1.x, x.w - f1.y);
                unsigned char *at = smem + L::oQ + (lane >> 1) * 128 + (lane & 1) * 8;
                auto put = [&](int k, __half2 a, __half2 b) {
                    *reinterpret_cast<uint2 *>(at + (k >> 3) * kCoreRow + (k & 7) * 16) = make_uint2(half2_bits(a), half2_bits(b));
                };
                put(i, h0, h1);
                put(i + (kWide ? L::kRows : n), l0, l1);
                if (lane == 0) ms->factor[seg & 1][i] = exp2_int(e);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ms->q_ready[seg & 1]));
            const int end = w.end(w.r);
            for (int i = 0; i < part; ++i, ++j) {
                const uint32_t par = (j >> 1) & 1;
                // K: lane = token, the row's chunk c stands at c ^ (token & 7)
                int g = 2 * j, at = g % L::kSlots;
                const unsigned char *st = smem + L::oRing + at * kSlotBytes;
                wait_warp(&ms->full[at], (g / L::kSlots) & 1, ms, p.dev_status);
                const int skip = ms->skip[at];
                const int t = (off + i) * kTok + row;
                const float *scales = reinterpret_cast<const float *>(st + kCodeBytes);
                const bool real = !skip && t < end;
                const float ks = real ? scales[row] * p.sm_scale_log2 : 0.0f, vs = real ? scales[kTok + row] : 0.0f;
                ms->scale[j & 3][row] = make_float2(ks, vs);
                if (lane == 0 && quad == 0) ms->bad[j & 3] = skip;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ms->sc_ready[j & 3]));
                wait_warp(&ms->k_free[j & 1], par ^ 1, ms, p.dev_status);
                tc_fence_after();
                const uint4 *kr = reinterpret_cast<const uint4 *>(st + row * kHD);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    put_codes(lanes + kColK + (j & 1) * 64 + 16 * k, kr[(2 * k) ^ (lane & 7)], kr[(2 * k + 1) ^ (lane & 7)]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&ms->empty[at]));
                    mbar_arrive(smem_addr(&ms->k_ready[j & 1]));
                }
                // V: lane = dim; two 64-token quarters of 64 bytes.  Lanes 2 apart start at
                // another chunk, so that eight lanes' 16-byte reads hit all banks, and turn
                // the four chunks back into order
                ++g;
                at = g % L::kSlots;
                st = smem + L::oRing + at * kSlotBytes;
                wait_warp(&ms->full[at], (g / L::kSlots) & 1, ms, p.dev_status);
                wait_warp(&ms->v_free[j & 1], par ^ 1, ms, p.dev_status);
                tc_fence_after();
                const int turn = (lane >> 1) & 3;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint4 *vr = reinterpret_cast<const uint4 *>(st + q * kTileVQuarter + row * kStageTok);
                    uint4 a[4], b[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) a[k] = vr[(k + turn) & 3];
#pragma unroll
                    for (int k = 0; k < 4; ++k) b[k] = (turn & 1) ? a[(k + 3) & 3] : a[k];
#pragma unroll
                    for (int k = 0; k < 4; ++k) a[k] = (turn & 2) ? b[(k + 2) & 3] : b[k];
                    put_codes(lanes + kColV + (j & 1) * 64 + 32 * q, a[0], a[1]);
                    put_codes(lanes + kColV + (j & 1) * 64 + 32 * q + 16, a[2], a[3]);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&ms->empty[at]));
                    mbar_arrive(smem_addr(&ms->v_ready[j & 1]));
                }
            }
        }
    } else {
        regs_grow<kRegsSoftmax>();
        // ========================== softmax ==========================
        constexpr int kCols = L::kRows / 2;   // a warp's share of the rows
        constexpr int kBar = 1, kN = 256;
        const int quad = warp & 3, half = (warp - 8) >> 2, st = tid - 256;
        const int row = 32 * quad + lane;     // token of the stage (scores), dim (output)
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        unsigned char *prow = smem + L::oP + row * 16;
        int j = 0;
        KVQ8_FOR_TILES {
            const int rows = w.tile_rows(w.r), n = (rows + 15) & ~15;
            const int nh = n / 2, c0 = half * nh;   // this warp: rows c0 .. c0 + nh - 1
            wait_warp(&ms->q_ready[seg & 1], (seg >> 1) & 1, ms, p.dev_status);
            if (st < n) {
                int lim = 0x7fffffff;
                if (st < rows) {
                    bool bad;
                    lim = w.limit(w.r, st, bad);
                    if (bad) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
                    atomicMin(&ms->lim_min[seg & 1], lim);
                }
                ms->lim[st] = lim;
                ms->col[st] = make_float2(ms->factor[seg & 1][st], INFINITY);
            }
            named_barrier_sync(kBar, kN);
            const int lim_min = ms->lim_min[seg & 1];
            if (st == 0) ms->lim_min[(seg & 1) ^ 1] = 0x7fffffff;
            float sum[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) sum[i] = 0.0f;
            for (int i = 0; i < part; ++i, ++j) {
                const int buf = j & 3;
                wait_warp(&ms->sc_ready[buf], (j >> 2) & 1, ms, p.dev_status);
                const float2 sc = ms->scale[buf][row];
                const bool bad = ms->bad[buf] != 0;
                const int t0 = (off + i) * kTok;
                const int tok = bad ? 0x7fffffff : t0 + row;
                const bool masked = bad || t0 + kTok > lim_min;   // some row does not see all of the stage
                const float vs_log2 = fmaxf(__log2f(sc.y), kTinyScaleLog2);
                wait_warp(&ms->s_full, j & 1, ms, p.dev_status);
                tc_fence_after();
                float t[kCols];
                // scores of this thread's token, relative to the running maxima
                auto scores = [&](bool relative) {
#pragma unroll
                    for (int k = 0; k < kCols / 8; ++k) {
                        if (8 * k < nh) {
                            float x[8], y[8];
                            tmem_ld8(lanes + kColS + c0 + 8 * k, x);
                            if (!kWide) tmem_ld8(lanes + kColS + n + c0 + 8 * k, y);
#pragma unroll
                            for (int q = 0; q < 8; ++q) t[8 * k + q] = x[q];
                            if (!kWide) {
                                tmem_wait_ld();
#pragma unroll
                                for (int q = 0; q < 8; ++q) {
                                    asm volatile("" : "+f"(t[8 * k + q]), "+f"(y[q]));
                                    t[8 * k + q] += y[q];
                                }
                            }
                        }
                    }
                    if (kWide) {
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < kCols; ++q) asm volatile("" : "+f"(t[q]));
                    }
#pragma unroll
                    for (int k = 0; k < kCols / 2; ++k) {
                        if (2 * k < nh) {
                            const float4 f = *reinterpret_cast<const float4 *>(&ms->col[c0 + 2 * k]);
                            t[2 * k] = fmaf(t[2 * k] * sc.x, f.x, relative ? f.y : 0.0f);
                            t[2 * k + 1] = fmaf(t[2 * k + 1] * sc.x, f.z, relative ? f.w : 0.0f);
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < kCols / 4; ++k) {
                            if (4 * k < nh) {
                                const int4 f = *reinterpret_cast<const int4 *>(&ms->lim[c0 + 4 * k]);
                                if (tok >= f.x) t[4 * k] = -INFINITY;
                                if (tok >= f.y) t[4 * k + 1] = -INFINITY;
                                if (tok >= f.z) t[4 * k + 2] = -INFINITY;
                                if (tok >= f.w) t[4 * k + 3] = -INFINITY;
                            }
                        }
                    }
                };
                scores(true);
                const float most = kPMaxLog2 - vs_log2;
                bool raise = false;
#pragma unroll
                for (int k = 0; k < kCols / 8; ++k) {
                    if (8 * k < nh) {
                        float top = t[8 * k];
#pragma unroll
                        for (int q = 1; q < 8; ++q) top = fmaxf(top, t[8 * k + q]);
                        raise |= top > most;
                    }
                }
                bool p_free = i == 0;   // the product before this one is done
                if (barrier_any(kBar, kN, raise)) {
                    // move the references that are too low, by whole numbers
                    scores(false);
#pragma unroll
                    for (int k = 0; k < kCols; ++k) {
                        if (k < nh) {
                            const float top = warp_top(t[k] + vs_log2);
                            if (lane == (k & 31)) ms->wave[quad][c0 + k] = top;
                        }
                    }
                    named_barrier_sync(kBar, kN);
                    if (st < n) {
                        const float top = fmaxf(fmaxf(ms->wave[0][st], ms->wave[1][st]), fmaxf(ms->wave[2][st], ms->wave[3][st]));
                        const float old = -ms->col[st].y;
                        float now = old;
                        if (top > old + kPMaxLog2) now = ceilf(top) - kPTopLog2;   // (also the first time: old is -inf)
                        ms->col[st].y = -now;
                        ms->alpha[st] = old == -INFINITY ? 0.0f : ex2_approx(old - now);
                    }
                    named_barrier_sync(kBar, kN);
                    if (!p_free) {
                        wait_warp(&ms->pv_done, (j & 1) ^ 1, ms, p.dev_status);
                        tc_fence_after();
                        p_free = true;
#pragma unroll 1
                        for (int part_lo = 0; part_lo < (!kWide && kLow ? 2 : 1); ++part_lo) {
#pragma unroll 1
                            for (int k = 0; k < nh; k += 8) {
                                const uint32_t at = lanes + kColO + part_lo * n + c0 + k;
                                float x[8];
                                uint32_t v[8];
                                tmem_ld8(at, x);
                                tmem_wait_ld();
#pragma unroll
                                for (int q = 0; q < 8; ++q) {
                                    asm volatile("" : "+f"(x[q]));
                                    v[q] = __float_as_uint(x[q] * ms->alpha[c0 + k + q]);
                                }
                                tmem_st8(at, v);
                            }
                        }
                        tmem_wait_st();
                    }
#pragma unroll
                    for (int k = 0; k < kCols; ++k)
                        if (k < nh) sum[k] *= ms->alpha[c0 + k];
                    scores(true);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ms->s_free));
                // weights, and P = weight * V scale in high and low parts
                const float pvs = sc.y;
                uint32_t hi[kCols / 2], lo[kLow ? kCols / 2 : 1];
#pragma unroll
                for (int k = 0; k < kCols / 2; ++k) {
                    if (2 * k < nh) {
                        const float w0 = ex2_approx(t[2 * k]), w1 = ex2_approx(t[2 * k + 1]);
                        sum[2 * k] += w0;
                        sum[2 * k + 1] += w1;
                        const float x0 = w0 * pvs, x1 = w1 * pvs;
                        const __half2 a = __floats2half2_rn(x0, x1);
                        hi[k] = half2_bits(a);
                        if (kLow) {
                            const float2 f = __half22float2(a);
                            lo[k] = half2_bits(__floats2half2_rn(x0 - f.x, x1 - f.y));
                        }
                    }
                }
                if (!p_free) wait_warp(&ms->pv_done, (j & 1) ^ 1, ms, p.dev_status);
#pragma unroll
                for (int k = 0; k < kCols / 8; ++k) {
                    if (8 * k < nh) {
                        const int core = (c0 >> 3) + k;
                        *reinterpret_cast<uint4 *>(prow + core * kCoreRow) =
                            make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
                        if (kLow)
                            *reinterpret_cast<uint4 *>(prow + (core + (kWide ? L::kRows / 8 : n / 8)) * kCoreRow) =
                                make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ms->p_ready));
            }
            // ---- the tile's end: row sums over the tokens, then the output or a record ----
            // (each step adds the halves of the rows that a lane keeps and gives away: lane l ends with rows
            // l * kCols / 32 ..)
#pragma unroll
            for (int o = 16, cnt = kCols / 2; o > 0; o >>= 1, cnt >>= 1) {
#pragma unroll
                for (int k = 0; k < cnt; ++k) {
                    const bool up = lane & o;
                    const float give = up ? sum[k] : sum[k + cnt], keep = up ? sum[k + cnt] : sum[k];
                    sum[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
#pragma unroll
            for (int k = 0; k < kCols / 32; ++k) {
                const int x = lane * (kCols / 32) + k;
                if (x < nh) ms->wave[quad][c0 + x] = sum[k];
            }
            named_barrier_sync(kBar, kN);
            const bool whole = off == 0 && part == w.stages(w.r);
            const bool direct = !kShared && whole;
            // first record row of this part
            long long rec;
            if (kShared) rec = (long long)w.first * p.nqh + (long long)w.h * w.rows + (long long)w.r * L::kRows + (long long)c * kTileRows;
            else rec = ((long long)c * 2 + (off == 0 ? 1 : 0)) * kTileRows;
            if (st < n) {
                const float S = ms->wave[0][st] + ms->wave[1][st] + ms->wave[2][st] + ms->wave[3][st];
                ms->alpha[st] = direct ? (S > 0.0f ? 1.0f / S : 0.0f) : 1.0f;
                if (!direct && st < rows) {
                    const float2 ml = make_float2(-ms->col[st].y, S);
                    *reinterpret_cast<float2 *>(p.ws_ml + (rec + st) * 2) = ml;
                }
            }
            if (st == 0 && !whole && off == 0) {
                // the CTAs c .. that hold this tile's records
                const int cnt = (int)(((hi - left + w.stages(w.r)) * C + T - 1) / T) - c;
                if (!kShared) p.ws_dir[c] = make_int4(cnt, w.s, w.h, w.r);
                else p.ws_dir[rec - (long long)c * kTileRows] = make_int4(c, cnt, 0, 0);
            } else if (kShared && st == 0 && whole) {
                p.ws_dir[rec - (long long)c * kTileRows] = make_int4(c, 1, 0, 0);
            }
            named_barrier_sync(kBar, kN);
            wait_warp(&ms->pv_done, (j & 1) ^ 1, ms, p.dev_status);
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < nh; k += 8) {
                float x[8], y[8];
                tmem_ld8(lanes + kColO + c0 + k, x);
                if (!kWide && kLow) tmem_ld8(lanes + kColO + n + c0 + k, y);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    asm volatile("" : "+f"(x[q]));
                    if (!kWide && kLow) {
                        asm volatile("" : "+f"(y[q]));
                        x[q] += y[q];
                    }
                    const int i = c0 + k + q;
                    if (i >= rows) continue;
                    const float v = x[q] * ms->alpha[i];
                    if (direct) store1(p.out, p.out_dtype, w.token(w.r, i) * p.out_stride + (int64_t)w.head(i) * kHD + row, v);
                    else p.ws_acc[(rec + i) * kHD + row] = v;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ms->o_free));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
#undef KVQ8_FOR_TILES
}

// What the tile kernel needs to know of the groups: (first row, rows, the row
// whose block-table row the shared tokens are read through, tokens), and of
// every row the tokens that it shares.  A warp per group.
constexpr int kPlanWarps = 8;
__global__ void __launch_bounds__(kPlanWarps * 32)
shared_plan_kernel(TileParams p) {
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    for (int g = threadIdx.x; g <= p.n_groups; g += blockDim.x)
        if (!group_entry_ok(p, g)) bad = 1;
    __syncthreads();
    const int cap = p.max_blocks * kBS, lane = threadIdx.x & 31;
    const int stride = gridDim.x * kPlanWarps;
    if (bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_GROUPS);
        for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < p.batch; b += gridDim.x * blockDim.x) p.ws_tail[b] = 0;
        for (int g = blockIdx.x * blockDim.x + threadIdx.x; g < p.n_groups; g += gridDim.x * blockDim.x)
            p.ws_group[g] = make_int4(0, 0, 0, 0);
        return;
    }
    for (int g = blockIdx.x * kPlanWarps + (threadIdx.x >> 5); g < p.n_groups; g += stride) {
        const int b0 = p.group_starts[g], b1 = p.group_starts[g + 1], shared = p.shared_lens[g];
        if (shared < 0 && lane == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_CTX_LEN);
        int most = 0, lead = b0;   // the lane's first row of most shared tokens
        for (int b = b0 + lane; b < b1; b += 32) {
            const int x = row_shared(p, b, shared, cap);
            p.ws_tail[b] = x;
            if (x > most) {
                most = x;
                lead = b;
            }
        }
        const int top = __reduce_max_sync(0xffffffffu, most);
        lead = __reduce_min_sync(0xffffffffu, most == top ? lead : 0x7fffffff);
        if (lane == 0) p.ws_group[g] = make_int4(b0, b1 - b0, lead, top);
    }
}

// Merge of the prompt tiles that several CTAs share, by the rule of
// decode_combine_kernel: the tile that CTA blockIdx.x began, a warp per row.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(kMergeWarps * 32)
prompt_merge_kernel(TileParams p, int lg, int rows_per_tile) {
    pdl_wait();
    pdl_launch_dependents();
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const int4 dir = p.ws_dir[c];
    if (dir.x == 0) return;
    Walk<false> w(p, lg, rows_per_tile);
    w.load(dir.y);
    w.h = dir.z;
    w.r = dir.w;
    const int i = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
    if (i >= w.tile_rows(w.r)) return;
    // record k: of CTA c + k; the first one is c's own second place
    auto at = [&](int k) { return ((long long)(c + k) * 2 + (k == 0 ? 1 : 0)) * kTileRows + i; };
    float m = -INFINITY;
    for (int k = lane; k < dir.x; k += 32) m = fmaxf(m, p.ws_ml[at(k) * 2]);
    m = warp_max(m);
    float S = 0.0f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (m != -INFINITY) {
#pragma unroll 4
        for (int k = 0; k < dir.x; ++k) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.ws_ml + at(k) * 2);
            const float4 x = *reinterpret_cast<const float4 *>(p.ws_acc + at(k) * kHD + 4 * lane);
            const float f = ex2_approx(ml.x - m);
            S = fmaf(ml.y, f, S);
            a.x = fmaf(x.x, f, a.x);
            a.y = fmaf(x.y, f, a.y);
            a.z = fmaf(x.z, f, a.z);
            a.w = fmaf(x.w, f, a.w);
        }
    }
    const float inv = S > 0.0f ? 1.0f / S : 0.0f;
    const int64_t o = w.token(w.r, i) * p.out_stride + (int64_t)w.head(i) * kHD + 4 * lane;
    store1(p.out, p.out_dtype, o, a.x * inv);
    store1(p.out, p.out_dtype, o + 1, a.y * inv);
    store1(p.out, p.out_dtype, o + 2, a.z * inv);
    store1(p.out, p.out_dtype, o + 3, a.w * inv);
}

// A launch as a programmatic dependent of the kernel before it.
template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int tile_ctas() { return min(device_sm_count(), kMaxTileCtas); }

template <bool kShared, bool kWide, bool kLow>
cudaError_t launch_tiles(const TileParams &p, int lg, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};
    const int ctas = tile_ctas();
    if (ctas <= 0) return cudaErrorInvalidDevice;
    return launch_after_setting(
        configured,
        [] {
            // the warpgroups trade registers within the launch's own: it must hold what they come to
            cudaFuncAttributes a;
            cudaError_t e = cudaFuncGetAttributes(&a, tile_kernel<kShared, kWide, kLow>);
            if (e != cudaSuccess) return e;
            if (a.numRegs != 128) return cudaErrorInvalidConfiguration;
            return cudaFuncSetAttribute(tile_kernel<kShared, kWide, kLow>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        Lay<kWide, kLow>::kBytes);
        },
        [&] {
            return launch_dependent(tile_kernel<kShared, kWide, kLow>, dim3(ctas), kThreads, Lay<kWide, kLow>::kBytes, s, p, lg);
        });
}

int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

}  // namespace

// Tiles of 128 rows where a sequence (or, on average, a group) has more than 64.
cudaError_t launch_prompt(const TileParams &p, int group, cudaStream_t s) {
    const int lg = log2_of(group);
    const bool wide = ((int64_t)p.n_new << lg) > 64, low = p.out_dtype != KVQ8_DTYPE_BF16;
    const cudaError_t e = wide ? (low ? launch_tiles<false, true, true>(p, lg, s) : launch_tiles<false, true, false>(p, lg, s))
                               : (low ? launch_tiles<false, false, true>(p, lg, s) : launch_tiles<false, false, false>(p, lg, s));
    if (e != cudaSuccess) return e;
    const int rows = wide ? 128 : 64;
    return launch_dependent(prompt_merge_kernel, dim3(tile_ctas(), rows / kMergeWarps), kMergeWarps * 32, 0, s, p, lg, rows);
}

cudaError_t launch_shared_prefix(TileParams &p, int group, cudaStream_t s) {
    const int lg = log2_of(group);
    const bool wide = ((int64_t)p.batch << lg) > 64 * (int64_t)p.n_groups;
    p.tile_rows = wide ? 128 : 64;
    const int blocks = min((p.n_groups + kPlanWarps - 1) / kPlanWarps, 304);
    const cudaError_t e = launch_dependent(shared_plan_kernel, dim3(blocks), kPlanWarps * 32, 0, s, p);
    if (e != cudaSuccess) return e;
    return wide ? launch_tiles<true, true, true>(p, lg, s) : launch_tiles<true, false, true>(p, lg, s);
}

}  // namespace kvq8
