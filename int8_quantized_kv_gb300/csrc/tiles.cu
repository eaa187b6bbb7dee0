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
// memory, and the right operands are as narrow as the tile's height (16, 32, 64
// or 128 rows: rows that a tile does not have are computed and dropped), so that
// few rows cost little softmax work.
//
// fp32-class results from fp16 operands: the codes are exact; a query row's
// values code * scale and the weights P enter as a high and a low fp16 part
// (22 bits).  Of a tile of up to 64 rows both parts are columns of one product
// (A from tensor memory feeds at most 128 columns per 64 cycles, so the second
// part is free); of up to 128 rows they are two products into one accumulator.
// (The query's low part counts 2^-11 of itself, in the addition of the columns
// or as the first product's result enters the second.)
// bf16 outputs take P's high part alone: 11 bits of each weight, an eighth of
// the output's own rounding.
//
// A persistent CTA per SM takes an equal share of the (tile, 128-token stage)
// sequence.  Warp 0 copies the stages (bulk copies into a ring, K and V apart),
// warps 1 and 3 issue the MMAs of scores and output, warp 2 says which tiles,
// warps 4..7 turn K's codes into operands and 8..11 V's, the others (16; 8 for
// tiles of 32 rows, 4 for 16) take the softmax, four warps to an equal share of the rows,
// and prepare the next tile's queries behind their last stage.  S^T and P^T move
// as MMA fragments (tcgen05.ld 16x256b, stmatrix), so that a thread holds tokens
// of few rows, whose references and sums stay in its registers.  A row's weights
// 2^(s - M) need no exact maximum: M is set so that the row's largest weight * V
// scale fills fp16's range, and moved only when one would leave it (a factor of
// 2^7 or more later), which a comparison per token and one barrier over the four
// warps find out; maxima across lanes are formed only then.  (With M from the
// scores alone a row that leans on tokens of small V would lose P's low bits next
// to one large V scale.)
//
// What bounds it.  Of 128 rows and fp32 outputs a stage has 32 MMAs of 128 x 128
// x 16, 64 clocks each: 2048 clocks.  The codes' conversion (8 warps) and the
// softmax of 16384 scores (16 warps, about 15 instructions for two scores) make
// them 3600 to 3700: the four schedulers issue in 64 % of all cycles, the tensor
// cores run in 55 %.  512 tokens x 32 heads behind 130560: 1.80 ms, 610 TFLOP/s
// of the operator's own arithmetic (each product counted once), with 4.7 GB of
// DRAM traffic for 0.28 GB of cache (16 tiles of a kv head at different places of
// it at a time; 36 % of DRAM's rate, which bounds nothing yet); 4096 tokens x 16
// heads in bf16, without P's low part: 119 us, 578 TFLOP/s.  Tiles of 32 rows
// take some 2100 clocks a stage, of 16 rows 1900, of which the MMAs are 512 (272)
// and the bytes 1400 (at the copy rate; 28 layers x 8 heads of 4096 tokens, 16
// rows: 57 us, 36 at that rate): the warps of seven roles draw on the instruction
// caches, so that longer loops (unrolled operands) and more warps (16 for the
// operands, two groups of softmax warps in turn, two CTAs per SM) all came out
// slower, and fewer (four of softmax for 16 rows) faster.
#include <math.h>

#include "kvq8_ptx.cuh"
#include "tile_rows.cuh"

namespace kvq8 {
namespace {

constexpr int kTok = 128;                       // tokens per stage
// What a tile costs beside its stages (queries, first references, output), in stages: the CTAs' shares count it, or
// one that gets many short tiles ends long after the others (4096 tokens x 16 heads: 131 us counting 3, 125 counting 4,
// 128 counting 5).
constexpr int kTileCost = 4;
constexpr int kCodeBytes = kTok * kHD;          // 16 KiB of K or V codes
constexpr int kSlotBytes = kCodeBytes + 2 * kTok * 4;   // K codes with both scales, or V codes
constexpr int kCoreRow = 2048;                  // bytes between cores along the rows (16 cores of 128 B along k)
constexpr int kLimit = 232448;                  // bytes of shared memory
constexpr int kColumns = 512;                   // of tensor memory: all
constexpr int kSoftmaxWarp0 = 12;               // warps before: 4 for copies, MMAs and order, 4 for K's operands, 4 for V's
constexpr uint64_t kLimitNs = 2000000000ull;    // bound of the waits at the end: two seconds
// The query's low parts are held 2^11 times as large as they are: at half a step of the high part at most, they end
// below fp16's largest, and parts of small values keep their bits.
constexpr int kQLowBits = 11;
// Shared memory for tiles of kRows rows: Q (high, low), P (high, low), the ring.
template <int kRows, bool kLow>
struct Lay {
    static constexpr bool kWide = kRows > 64;   // the parts are two products; else columns of one
    static constexpr int kQ = kRows * 2 * kHD * 2;
    static constexpr int kP = kRows * (kLow ? 2 : 1) * kTok * 2;
    static constexpr int oQ = 0;
    static constexpr int oP = kQ;
    static constexpr int oMisc = oP + kP;
    static constexpr int kMisc = 13824;
    static constexpr int oRing = oMisc + kMisc;
    static constexpr int kSlots = (kLimit - oRing) / kSlotBytes < 8 ? (kLimit - oRing) / kSlotBytes : 8;
    static constexpr int kBytes = oRing + kSlots * kSlotBytes;
    static_assert(kSlots >= 4, "ring too shallow");
    // columns of tensor memory: two of K's operand and of V's, scores, output
    static constexpr int kColK = 0, kColV = 128, kColS = 256, kColO = kColS + (kWide ? kRows : 2 * kRows);
    static_assert(kColO + (kWide ? kRows : 2 * kRows) <= kColumns, "tensor memory");
    // Softmax warps: as many as fill the SM's registers, but for tiles of up to 32 rows, where a warp of sixteen would
    // have 8 rows or fewer (8 prompts of 5 tokens x 32 heads, 20 rows: 33.1 us with sixteen, 32.2 us with eight; later
    // 31.0 with eight, 32.9 with four).
    static constexpr int kSoftmaxWarps = kRows == 16 ? 4 : kRows == 32 ? 8 : 16;
    static constexpr int kThreads = (kSoftmaxWarp0 + kSoftmaxWarps) * 32;
    // Stages whose outputs add up in tensor memory.  The tensor cores cut off what leaves an accumulator's 24 bits, always
    // downwards in size, so that a long sum shrinks (2e-4 of the output over 130560 tokens): after a run of stages it is
    // added, in fp32 and rounded, to a total in the workspace, and begins anew.  The shorter the run, the nearer to the
    // 64-bit result and the more often 64 KB per tile of 128 rows go out.  bf16 outputs need none of it: over 256 stages
    // the cut is a thirtieth of their rounding.
    static constexpr int kRun = !kLow ? 256 : kWide ? 12 : 8;
    // Registers per thread: what the launch holds, and, for wide tiles, what the warpgroups (copies, MMAs and order;
    // K's operands; V's; four of softmax) trade them for.  Local memory costs more here than elsewhere, since shared memory
    // leaves it no L1: 56 to 72 bytes a thread are spilled with 128 rows, 12 to 20 with 64.  (The build checks the count.)
    static constexpr int kLaunchRegs = 72, kRegsOther = 40, kRegsSoftmax = 96;
    static_assert(!kWide || kSoftmaxWarp0 / 4 * kRegsOther + kSoftmaxWarps / 4 * kRegsSoftmax <= kThreads / 128 * kLaunchRegs,
                  "registers");
};

// One tile's stages of one CTA.
struct Part {
    int stages, off, end, rows;                 // (stages 0: no more)
    int lead, head, token, direct;              // block-table row, kv head, first token, whether out is written
    long long rec;                              // first record row
};

struct Misc {
    uint64_t full[8], empty[8];                 // ring slots
    uint64_t k_ready[2], k_free[2], v_ready[2], v_free[2];
    uint64_t part_ready[4], part_free[4];
    uint64_t s_full, s_free, p_ready, pv_done, q_ready, q_free, o_free, all_done[2];
    long long warp_tot[32];
    int4 at0, of0;                              // the first tile: sequence, rows' tile, rows, its cost ahead of this CTA; its Walk
    volatile int abort;
    uint32_t tmem;                              // address of the columns
    int skip[8];                                // slot: its block id is outside the pool
    int bad[4];                                 // stage (mod 4): the same
    int lim_min[4];                             // tile (mod 4)
    alignas(16) Part part[4];
    alignas(16) int lim[4][kTileRows];          // tile (mod 4), row: tokens below
    alignas(16) float gain[4][kTileRows];       // tile (mod 4), row: power of two of the query's operand
    float common[4][4];                         // tile (mod 4), share of a wide tile: its rows' gain, 0 where they differ
    int2 spread[16];                            // warp: largest and smallest exponent of its rows' queries
    alignas(16) float2 scale[4][kTok];          // stage (mod 4): (K scale * sm_scale, V scale)
    alignas(16) float ref[kTileRows];           // per row: -M
    alignas(16) float shift[kTileRows];         // per row: M before - M now, or the output's factor
    alignas(16) float wave[4][kTileRows];       // per warp and row: maxima, sums
    char *dst[kTileRows];                       // per row: where its output or record starts (null: nowhere)
};
static_assert(sizeof(Misc) <= 13824, "misc");

// Bounded like every wait here: a try sleeps up to two microseconds, and after 2^20 of them (two seconds at most) the
// CTA gives up, its other waits with it.  Short, since the loops of all roles share the SM's instruction cache.  kTest:
// asks once before it may sleep, which takes 100 clocks less where the phase is complete already, as it often is for the
// softmax and in tiles of up to 64 rows (8 x 5-token prompts 31.4 -> 29.5 us); in all roles of wide tiles the longer
// code costs more (4096 tokens x 16 heads 123 -> 129 us).
template <bool kTest>
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Misc *ms) {
    const uint32_t a = smem_addr(bar);
    if (kTest && mbar_test(a, parity)) return true;
    int left = 1 << 20;
#pragma unroll 1
    while (!mbar_try_wait_for(a, parity, 2000u)) {
        if (--left == 0) ms->abort = 1;
        if (ms->abort) return false;
    }
    return true;
}

// The same by all lanes of a warp, together again behind it.
template <bool kTest>
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Misc *ms) {
    const bool ok = wait_bar<kTest>(bar, parity, ms);
    return __all_sync(0xffffffffu, ok);
}

// The tiles in their order: (kv head, sequence or group, rows).
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
    __device__ int cost(int r_) const { return kTileCost + stages(r_); }
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
    // (there is one behind: the caller counts)
    __device__ void next(int count) {
        if (++r < tiles()) return;
        r = 0;
        do {
            if (++s == count) {
                s = 0;
                ++h;
            }
            load(s);
        } while (rows == 0);
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
    uint32_t v[16];
    codes_to_half2(x.x, v[0], v[1]);
    codes_to_half2(x.y, v[2], v[3]);
    codes_to_half2(x.z, v[4], v[5]);
    codes_to_half2(x.w, v[6], v[7]);
    codes_to_half2(y.x, v[8], v[9]);
    codes_to_half2(y.y, v[10], v[11]);
    codes_to_half2(y.z, v[12], v[13]);
    codes_to_half2(y.w, v[14], v[15]);
    tmem_st16(tmem, v);
}

__device__ __forceinline__ uint32_t half2_bits(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }   // -126 .. 127

// Combines 2 * kCount values per lane over the lanes that differ in the bits from kLanes down to 4: each step combines
// the half of the values that a lane keeps with the other lane's, then (one value left) the lanes that share it.  Of
// `count` values that the first step (16 lanes apart) began with, lane l ends with value l / (32 / count).
template <int kCount, int kLanes, typename Op>
__device__ __forceinline__ void halve(float *v, int lane, Op op) {
    if constexpr (kLanes >= 4) {
        if constexpr (kCount > 0) {
#pragma unroll
            for (int k = 0; k < kCount; ++k) {
                const bool up = lane & kLanes;
                const float give = up ? v[k] : v[k + kCount], keep = up ? v[k + kCount] : v[k];
                v[k] = op(keep, __shfl_xor_sync(0xffffffffu, give, kLanes));
            }
        } else {
            v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], kLanes));
        }
        halve<kCount / 2, kLanes / 2>(v, lane, op);
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A total's element, which one thread alone has to do with: what it asks for in turn happens in turn.
__device__ __forceinline__ void store_relaxed(float *at, float x) {
    asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(at), "f"(x) : "memory");
}
__device__ __forceinline__ void add_relaxed(float *at, float x) {
    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(at), "f"(x) : "memory");
}
__device__ __forceinline__ float load_relaxed(const float *at) {
    float x;
    asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(x) : "l"(at) : "memory");
    return x;
}

// a / b for positive b; in 32 bits where that does.
__device__ __forceinline__ long long divide(long long a, long long b) {
    if (((a | b) >> 31) == 0) return (int)a / (int)b;
    return a / b;
}

// The exponent of the unit in which a positive value lies in [2^14, 2^15).
__device__ __forceinline__ int unit_exponent(float x) { return (__float_as_int(x) >> 23) - 127 - 14; }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// a - b, b in fp16
__device__ __forceinline__ float minus(float a, __half b) {
    float d;
    asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d) : "h"(__half_as_ushort(b)), "h"((unsigned short)0xbc00), "f"(a));
    return d;
}

template <bool kShared, int kRows, bool kLow>
__global__ void __launch_bounds__((Lay<kRows, kLow>::kThreads), 1)
tile_kernel(TileParams p, int lg) {
    using L = Lay<kRows, kLow>;
    constexpr int kThreads = L::kThreads, kSoftmaxWarps = L::kSoftmaxWarps;
    constexpr bool kWide = L::kWide;
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
            mbar_init(smem_addr(&ms->k_ready[i]), 4);
            mbar_init(smem_addr(&ms->k_free[i]), 1);
            mbar_init(smem_addr(&ms->v_ready[i]), 4);
            mbar_init(smem_addr(&ms->v_free[i]), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&ms->part_ready[i]), 1);
            mbar_init(smem_addr(&ms->part_free[i]), kSoftmaxWarps);
        }
        mbar_init(smem_addr(&ms->s_full), 1);
        mbar_init(smem_addr(&ms->s_free), kSoftmaxWarps);
        mbar_init(smem_addr(&ms->p_ready), kSoftmaxWarps);
        mbar_init(smem_addr(&ms->pv_done), 1);
        mbar_init(smem_addr(&ms->q_ready), kSoftmaxWarps);
        mbar_init(smem_addr(&ms->q_free), 1);
        mbar_init(smem_addr(&ms->o_free), kSoftmaxWarps);
        mbar_init(smem_addr(&ms->all_done[0]), 1);
        mbar_init(smem_addr(&ms->all_done[1]), 1);
        fence_mbar_init();
        ms->abort = 0;
    }
    if (warp == 1) tmem_alloc(smem_addr(&ms->tmem), kColumns);
    pdl_wait();
    pdl_launch_dependents();   // (the tails find no room here before this CTA leaves; what does just waits)
    // ---- this CTA's share: [lo, hi) of the sequence of all tiles, each as long as it costs ----
    Walk<kShared> w(p, lg, kRows);
    const int per_seq = kShared ? 1 : (int)((((long long)p.n_new << lg) + kRows - 1) / kRows);
    const int seqs = kShared ? p.n_groups : p.batch;
    const int items = seqs * per_seq;   // (sequence, tile of one kv head), or group
    const int per = (items + kThreads - 1) / kThreads;
    const int i_lo = min(items, tid * per), i_hi = min(items, i_lo + per);
    auto item = [&](int i) {   // its cost, for one kv head
        const int s = i / per_seq, r = i - s * per_seq;
        w.load(s);
        w.r = r;
        return kShared ? (w.rows > 0 ? (long long)w.tiles() * w.cost(0) : 0) : r < w.tiles() ? w.cost(r) : 0;
    };
    long long mine = 0;
#pragma unroll 1
    for (int i = i_lo; i < i_hi; ++i) mine += item(i);
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) ms->warp_tot[warp] = before;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;   // (who has all columns has them from 0 on)
    const long long of_warp = lane < kThreads / 32 ? ms->warp_tot[lane] : 0;
    long long upto = of_warp;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    const long long total = __shfl_sync(0xffffffffu, upto, 31);   // cost of one kv head
    before += __shfl_sync(0xffffffffu, upto - of_warp, warp) - mine;
    const long long T = total * p.nkv;
    const int C = (int)min((long long)gridDim.x, T);
    if (!kShared && tid == 0) p.ws_dir[c] = make_int4(0, 0, 0, 0);
    long long lo = 0, hi = 0;
    int off = 0;   // of the first tile: cost that lies ahead of this CTA
    if (c < C) {   // (uniform over the CTA)
        const long long Tq = divide(T, C);
        const int Tr = (int)(T - Tq * C);
        lo = (long long)c * Tq + (c * Tr) / C;
        hi = (long long)(c + 1) * Tq + ((c + 1) * Tr) / C;
        const int h = (int)divide(lo, total);
        const long long rem = lo - h * total;
        // the thread whose item holds lo says so (one item to a thread: what it loaded still stands)
#pragma unroll 1
        for (int i = i_lo; i < i_hi && before <= rem; ++i) {
            const long long v = per == 1 ? mine : item(i);
            if (rem < before + v) {
                long long at = rem - before;   // (of a group's tiles together, which may pass 31 bits)
                if (kShared) {
                    const int n = w.cost(0);
                    w.r = (int)divide(at, n);
                    at -= (long long)w.r * n;
                }
                ms->at0 = make_int4(w.s, w.r, w.rows, (int)at);
                ms->of0 = make_int4(w.first, w.lead, w.span, (int)w.start);
            }
            before += v;
        }
        __syncthreads();
        const int4 at0 = ms->at0, of0 = ms->of0;
        w.s = at0.x;
        w.h = h;
        w.r = at0.y;
        w.rows = at0.z;
        off = at0.w;
        w.first = of0.x;
        w.lead = of0.y;
        w.span = of0.z;
        w.start = of0.w;
    }

    if (warp < 4) {
        if constexpr (kWide) regs_shrink<L::kRegsOther>();
        if (warp == 0) {
            // ============================ copies ============================
            int g = 0;   // granules so far: K and V of every stage
            bool stop = false;
#pragma unroll 1
            for (int seg = 0; !stop; ++seg) {
                if (!wait_warp<!kWide>(&ms->part_ready[seg & 3], (seg >> 2) & 1, ms)) break;
                const Part &part = ms->part[seg & 3];
                const int n = part.stages, first = part.off, end = part.end, h = part.head;
                if (n == 0) break;
                const int32_t *row = p.block_table + (size_t)part.lead * p.max_blocks;
                int tbl_base = -1, tbl = -1;
#pragma unroll 1
                for (int j = 0; j < n && !stop; ++j, g += 2) {
                    const int t0 = (first + j) * kTok, lb = t0 / kBS;
                    if (tbl_base < 0 || lb >= tbl_base + 32) {
                        tbl_base = lb;
                        tbl = lb + lane < p.max_blocks ? row[lb + lane] : -1;
                    }
                    const int phys = __shfl_sync(0xffffffffu, tbl, lb - tbl_base);
                    if (lane == 0) {
                        const bool any = t0 < end, ok = any && phys >= 0 && phys < p.num_blocks;
                        if (any && !ok) flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
                        const size_t tile = ok ? (size_t)phys * p.nkv + h : 0;
                        const int slot0 = t0 % kBS;
#pragma unroll 1
                        for (int v = 0; v < 2; ++v) {
                            const int at = (g + v) % L::kSlots;
                            if (!wait_bar<!kWide>(&ms->empty[at], (((g + v) / L::kSlots) & 1) ^ 1, ms)) {
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
            }
            // no copy may still be in flight when the CTA exits (a stopped ring: whichever the slots were given last)
            if (lane == 0) {
                for (int k = max(0, g - L::kSlots); k < g; ++k)
                    mbar_wait_bounded(smem_addr(&ms->full[k % L::kSlots]), (k / L::kSlots) & 1, kLimitNs);
            }
            __syncwarp();
        } else if (warp != 2) {
            // ============================= MMAs =============================
            // warp 1: scores, warp 3: output (a warp for both leaves the tensor cores waiting for its own waits)
            const bool scores = warp == 1;
            const uint64_t b = core_desc(smem_addr(smem + (scores ? L::oQ : L::oP)), 128, kCoreRow);
            constexpr uint64_t kLowPart = kRows / 8 * kCoreRow / 16;
            int x = 0;   // stages so far
#pragma unroll 1
            for (int seg = 0;; ++seg) {
                if (!wait_warp<!kWide>(&ms->part_ready[seg & 3], (seg >> 2) & 1, ms)) break;
                const int n = ms->part[seg & 3].stages;
                if (n == 0) break;
                if (scores) {
                    wait_warp<!kWide>(&ms->q_ready, seg & 1, ms);
#pragma unroll 1
                    for (int i = 0; i < n; ++i, ++x) {
                        constexpr uint32_t kWord = mma_word(kWide ? kRows : 2 * kRows, false);
                        const int buf = x & 1;
                        const uint32_t d = tmem + L::kColS, a = tmem + L::kColK + buf * 64;
                        wait_warp<!kWide>(&ms->k_ready[buf], (x >> 1) & 1, ms);
                        wait_warp<!kWide>(&ms->s_free, (x & 1) ^ 1, ms);
                        tc_fence_after();
                        // (low parts first: what they add to is small yet, and little is cut off)
                        if constexpr (kWide) {
                            mma_k128(d, a, b + kLowPart, kWord, false);
                            mma_k128<kQLowBits>(d, a, b, kWord, true);
                        } else {
                            mma_k128(d, a, b, kWord, false);
                        }
                        mma_commit(smem_addr(&ms->s_full));
                        mma_commit(smem_addr(&ms->k_free[buf]));
                    }
                    mma_commit(smem_addr(&ms->q_free));
                } else {
                    wait_warp<!kWide>(&ms->o_free, (seg & 1) ^ 1, ms);
#pragma unroll 1
                    for (int i = 0; i < n; ++i, ++x) {
                        constexpr uint32_t kWord = mma_word(kWide || !kLow ? kRows : 2 * kRows, true);
                        const int buf = x & 1;
                        const uint32_t d = tmem + L::kColO, a = tmem + L::kColV + buf * 64;
                        wait_warp<!kWide>(&ms->v_ready[buf], (x >> 1) & 1, ms);
                        wait_warp<!kWide>(&ms->p_ready, x & 1, ms);
                        tc_fence_after();
                        mma_k128(d, a, b, kWord, i % L::kRun != 0);
                        if (kWide && kLow) mma_k128(d, a, b + kLowPart, kWord, true);
                        mma_commit(smem_addr(&ms->pv_done));
                        mma_commit(smem_addr(&ms->v_free[buf]));
                    }
                }
            }
            // none may still run when the CTA gives its tensor memory back
            uint64_t *done = &ms->all_done[scores ? 0 : 1];
            mma_commit(smem_addr(done));
            mbar_wait_bounded(smem_addr(done), 0, kLimitNs);
            __syncwarp();
        } else if (warp == 2) {
            // ======================= the tiles' order =======================
            // a tile's cost is kTileCost, then one for each stage: a share that ends in the former has none of it
            long long left = hi - lo;
#pragma unroll 1
            for (int seg = 0;; ++seg) {
                int n = 0, stages = 0, from = 0;
                while (left > 0) {
                    stages = w.stages(w.r);
                    const int until = (int)min((long long)(kTileCost + stages), off + left);   // of the tile's cost
                    from = max(0, off - kTileCost);
                    n = max(0, until - kTileCost) - from;
                    if (n > 0) break;
                    left = 0;   // (only the last tile)
                }
                if (!wait_warp<!kWide>(&ms->part_free[seg & 3], ((seg >> 2) & 1) ^ 1, ms)) break;
                Part &part = ms->part[seg & 3];
                if (n > 0) {
                    const int rows = w.tile_rows(w.r);
                    int least = 0x7fffffff;
#pragma unroll 1
                    for (int i = lane; i < kRows; i += 32) {
                        int lim = 0x7fffffff;
                        if (i < rows) {
                            bool bad;
                            lim = w.limit(w.r, i, bad);
                            if (bad) flag_status(p.dev_status, KVQ8_DEV_BAD_POSITION);
                            // the row's query, soon to be read
                            prefetch_l2(p.q, p.q_dtype, w.token(w.r, i) * p.q_stride + (int64_t)w.head(i) * kHD);
                        }
                        ms->lim[seg & 3][i] = lim;
                        least = min(least, lim);
                    }
                    least = __reduce_min_sync(0xffffffffu, least);
                    if (lane == 0) {
                        const bool whole = n == stages;
                        const long long x = (((long long)w.h * p.batch + w.first) << lg) + (long long)w.r * kRows;
                        ms->lim_min[seg & 3] = least;
                        part.off = from;
                        part.end = w.end(w.r);
                        part.rows = rows;
                        part.lead = w.lead;
                        part.head = w.h;
                        part.token = (int)w.token(w.r, 0);
                        part.direct = !kShared && whole;
                        part.rec = kShared ? x + (long long)c * kRows : ((long long)c * 3 + (whole ? 2 : from == 0 ? 1 : 0)) * kRows;
                        if (from == 0) {   // the CTAs c .. that hold this tile's records
                            const long long end = hi - left - off + kTileCost + stages;
                            const int cnt = (int)divide(end * C + T - 1, T) - c;
                            if (kShared) p.ws_dir[x] = make_int4(c, whole ? 1 : cnt, 0, 0);
                            else if (!whole) p.ws_dir[c] = make_int4(cnt, w.s, w.h, w.r);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    part.stages = n;
                    mbar_arrive(smem_addr(&ms->part_ready[seg & 3]));
                }
                if (n == 0) break;
                left -= kTileCost + stages - off;
                off = 0;
                if (left > 0) w.next(seqs);
            }
        }
    } else if (warp < kSoftmaxWarp0) {
        if constexpr (kWide) regs_shrink<L::kRegsOther>();
        // ========================= operands =========================
        const int quad = warp & 3, row = 32 * quad + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        int j = 0;
#pragma unroll 1
        for (int seg = 0;; ++seg) {
            if (!wait_warp<!kWide>(&ms->part_ready[seg & 3], (seg >> 2) & 1, ms)) break;
            const Part &part = ms->part[seg & 3];
            const int n = part.stages;
            if (n == 0) break;
            // tokens of the tile behind this lane's in its first stage
            int behind = part.end - part.off * kTok - row;
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++j, behind -= kTok) {
                const int buf = j & 1;
                const uint32_t par = (j >> 1) & 1;
                if (warp < 8) {
                    // K: lane = token, the row's chunk c stands at c ^ (token & 7)
                    const int g = 2 * j, at = g % L::kSlots;
                    const unsigned char *st = smem + L::oRing + at * kSlotBytes;
                    wait_warp<!kWide>(&ms->full[at], (g / L::kSlots) & 1, ms);
                    const int skip = ms->skip[at];
                    const float *scales = reinterpret_cast<const float *>(st + kCodeBytes);
                    const bool real = !skip && behind > 0;
                    ms->scale[j & 3][row] = make_float2(real ? scales[row] * p.sm_scale_log2 : 0.0f, real ? scales[kTok + row] : 0.0f);
                    if (lane == 0 && quad == 0) ms->bad[j & 3] = skip;
                    wait_warp<!kWide>(&ms->k_free[buf], par ^ 1, ms);
                    tc_fence_after();
                    const uint4 *kr = reinterpret_cast<const uint4 *>(st + row * kHD);
#pragma unroll 1
                    for (int k = 0; k < 4; ++k)
                        put_codes(lanes + L::kColK + buf * 64 + 16 * k, kr[(2 * k) ^ (lane & 7)], kr[(2 * k + 1) ^ (lane & 7)]);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_addr(&ms->k_ready[buf]));
                        mbar_arrive(smem_addr(&ms->empty[at]));
                    }
                } else {
                    // V: lane = dim; two 64-token quarters of 64 bytes.  Lanes 2 apart start at
                    // another chunk, so that eight lanes' 16-byte reads hit all banks, and turn
                    // the four chunks back into order
                    const int g = 2 * j + 1, at = g % L::kSlots;
                    const unsigned char *st = smem + L::oRing + at * kSlotBytes;
                    wait_warp<!kWide>(&ms->full[at], (g / L::kSlots) & 1, ms);
                    wait_warp<!kWide>(&ms->v_free[buf], par ^ 1, ms);
                    tc_fence_after();
                    const int turn = (lane >> 1) & 3;
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        const uint4 *vr = reinterpret_cast<const uint4 *>(st + q * kTileVQuarter + row * kStageTok);
                        uint4 a[4], b[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) a[k] = vr[(k + turn) & 3];
#pragma unroll
                        for (int k = 0; k < 4; ++k) b[k] = (turn & 1) ? a[(k + 3) & 3] : a[k];
#pragma unroll
                        for (int k = 0; k < 4; ++k) a[k] = (turn & 2) ? b[(k + 2) & 3] : b[k];
                        put_codes(lanes + L::kColV + buf * 64 + 32 * q, a[0], a[1]);
                        put_codes(lanes + L::kColV + buf * 64 + 32 * q + 16, a[2], a[3]);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_addr(&ms->v_ready[buf]));
                        mbar_arrive(smem_addr(&ms->empty[at]));
                    }
                }
            }
        }
    } else {
        if constexpr (kWide) regs_grow<L::kRegsSoftmax>();
        // ========================== softmax ==========================
        constexpr int kCols = kRows / (kSoftmaxWarps / 4);   // a warp's rows
        // the four warps of a share of the rows see to it by themselves
        const int quad = warp & 3, share = (warp - kSoftmaxWarp0) >> 2, c0 = share * kCols, st = tid & 127;
        const int bar = 1 + share;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        // Scores and P are held as MMA fragments: a thread has the tokens 32 quad + 8 m + lane / 4 (m < 4) of the
        // stage and the rows c0 + 8 g + 2 (lane % 4) + {0, 1} (g < kGroups) of the tile, so that what concerns a
        // row stays in registers (with a token per thread each row's reference and gain come from shared memory
        // for every stage, which keeps the MMAs' operands waiting) and P's cores are stored as matrices.
        constexpr int kGroups = kCols / 8, kVals = 2 * kGroups;
        const int col = c0 + 2 * (lane & 3);                                      // + 8 g
        const int folded = lane / (32 / kVals);                                   // of kVals values, halve() leaves this one
        const int folded_row = c0 + 8 * (folded >> 1) + 2 * (lane & 3) + (folded & 1);
        const uint32_t pout = smem_addr(smem + L::oP) + (c0 >> 3) * kCoreRow + quad * 512 + lane * 16;
        // Tile seg's queries: high and low parts of code * scale, in units of a power of two per row.  False when
        // there is no such tile (or a wait gave up: the four warps of a share go by one answer, or a barrier
        // would wait for the one that left).
        auto queries = [&](int seg) {
            const bool ok = wait_warp<!kWide>(&ms->part_ready[seg & 3], (seg >> 2) & 1, ms);
            if (barrier_any(bar, 128, !ok)) return false;
            const Part &part = ms->part[seg & 3];
            if (part.stages == 0) return false;
            if (warp - kSoftmaxWarp0 < kRows / 8) {
                // eight rows to a warp: lane l has row l % 8, and of every 32-block the dims 8 (l / 8) .. + 7, a
                // 16-byte line of an operand's core, so that eight lanes fill a core
                const int i = (warp - kSoftmaxWarp0) * 8 + (lane & 7);
                float4 x[8];
                const bool real = i < part.rows;
                const int64_t src = real ? ((long long)part.token + (i >> lg)) * p.q_stride +
                                               (int64_t)((part.head << lg) + (i & ((1 << lg) - 1))) * kHD + 8 * (lane >> 3)
                                         : 0;
                // (one test of the type around all loads: with a test in each they wait for one another)
                if (!real) {
#pragma unroll
                    for (int b = 0; b < 8; ++b) x[b] = make_float4(0.f, 0.f, 0.f, 0.f);
                } else if (p.q_dtype == KVQ8_DTYPE_F32) {
                    const float *row = static_cast<const float *>(p.q) + src;
#pragma unroll
                    for (int b = 0; b < 8; ++b) x[b] = *reinterpret_cast<const float4 *>(row + 32 * (b >> 1) + 4 * (b & 1));
                } else {
                    const uint16_t *row = static_cast<const uint16_t *>(p.q) + src;
                    uint4 y[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) y[b] = *reinterpret_cast<const uint4 *>(row + 32 * b);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        x[2 * b] = widen(y[b].x, y[b].y, p.q_dtype);
                        x[2 * b + 1] = widen(y[b].z, y[b].w, p.q_dtype);
                    }
                }
                // the rule of quantize_q_vals_warp; |x| as bits orders as |x| does, a NaN or infinity above all
                float top[4];
                float most = 0.0f, least = INFINITY;   // of the blocks that are not zeros
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t m = 0;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float4 y = x[2 * b + k];
                        m = max(max(m, max(__float_as_uint(y.x) & 0x7fffffffu, __float_as_uint(y.y) & 0x7fffffffu)),
                                max(__float_as_uint(y.z) & 0x7fffffffu, __float_as_uint(y.w) & 0x7fffffffu));
                    }
                    m = max(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    if (m >= 0x7f800000u) {
                        x[2 * b] = x[2 * b + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
                        m = 0;
                        flag_status(p.dev_status, KVQ8_DEV_NONFINITE);
                    }
                    top[b] = __uint_as_float(m);
                    if (top[b] < 1e-6f) top[b] = 1.0f;   // (codes 0)
                    else {
                        most = fmaxf(most, top[b]);
                        least = fminf(least, top[b]);
                    }
                }
                // A row's values lie below 2^15 in units of 2^e (fp16 ends below 2^16).  The low parts, in units 2^11 times
                // smaller, leave out 2^-36 at most: 2^-22 of a block's largest up to blocks 2^28 times smaller than the row's
                // largest.  (A block's own size counts, not the row's: keys may be zeros everywhere else.)
                int e = max(-100, unit_exponent(most));
                if constexpr (kWide) {
                    // one unit for the share's rows (prepared by its four warps) where their largest block is at most 2^28 times
                    // the smallest, by the same bound: a multiplication less per pair of scores (4096 tokens x 16 heads in bf16 127 -> 117 us;
                    // fp32 outputs as before)
                    const int most_e = __reduce_max_sync(0xffffffffu, e);
                    const int least_e = __reduce_min_sync(0xffffffffu, most > 0.0f ? unit_exponent(least) : 127);
                    if (lane == 0) ms->spread[4 * share + quad] = make_int2(most_e, least_e);
                    named_barrier_sync(bar, 128);
                    int2 all = ms->spread[4 * share];
#pragma unroll
                    for (int k = 1; k < 4; ++k) {
                        const int2 y = ms->spread[4 * share + k];
                        all = make_int2(max(all.x, y.x), min(all.y, y.y));
                    }
                    const bool even = all.x - all.y <= 27;   // (by exponents: a ratio below 2^28)
                    if (even) e = all.x;
                    if (st == 0) ms->common[seg & 3][share] = even ? exp2_int(all.x) : 0.0f;
                }
                const float down = exp2_int(-e);
                wait_warp<!kWide>(&ms->q_free, (seg & 1) ^ 1, ms);
                unsigned char *at = smem + L::oQ + (warp - kSoftmaxWarp0) * kCoreRow + (lane >> 3) * 128 + (lane & 7) * 16;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float iq = __fdiv_rn(127.0f, top[b]), unit = __fmul_rn(top[b], KVQ8_INV127) * down;
                    const float2 unit2 = make_float2(unit, unit);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 y = x[2 * b + (k >> 1)];
                        // round_half_even(fl(x * iq)) by a sum whose spacing is 1; |x * iq| < 127.5, so no clamp.
                        // (The product apart: a packed product and the packed sum behind it are made one
                        // operation of one rounding, which moves a code now and then)
                        float2 v = k & 1 ? make_float2(__fmul_rn(y.z, iq), __fmul_rn(y.w, iq))
                                         : make_float2(__fmul_rn(y.x, iq), __fmul_rn(y.y, iq));
                        v = add2(add2(v, make_float2(0x1.8p23f, 0x1.8p23f)), make_float2(-0x1.8p23f, -0x1.8p23f));
                        v = mul2(v, unit2);
                        const __half2 h = __floats2half2_rn(v.x, v.y);
                        hi[k] = half2_bits(h);
                        constexpr float kUp = 1 << kQLowBits;
                        v = mul2(fma2(__half22float2(h), make_float2(-1.f, -1.f), v), make_float2(kUp, kUp));
                        lo[k] = half2_bits(__floats2half2_rn(v.x, v.y));
                    }
                    *reinterpret_cast<uint4 *>(at + b * 512) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(at + b * 512 + kRows / 8 * kCoreRow) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                if (lane < 8) ms->gain[seg & 3][i] = exp2_int(e);
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ms->q_ready));
            return true;
        };
        // the outputs of eight rows from c0 + k on, dim 32 quad + lane
        auto read_output = [&](int k, float (&x)[8]) {
            float y[8];
            tmem_ld8(lanes + L::kColO + c0 + k, x);
            if (!kWide && kLow) tmem_ld8(lanes + L::kColO + kRows + c0 + k, y);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                asm volatile("" : "+f"(x[q]));
                if (!kWide && kLow) {
                    asm volatile("" : "+f"(y[q]));
                    x[q] += y[q];
                }
            }
        };
        int j = 0;
        bool more = queries(0);
#pragma unroll 1
        for (int seg = 0; more; ++seg) {
            const int n = ms->part[seg & 3].stages;
            wait_warp<!kWide>(&ms->q_ready, seg & 1, ms);
            if (st < kCols) ms->ref[c0 + st] = 0.0f;
            const int lim_min = ms->lim_min[seg & 3];
            named_barrier_sync(bar, 128);
            float2 ref[kGroups], sum[kGroups];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) ref[g] = sum[g] = make_float2(0.0f, 0.0f);
            bool fresh = true;   // no row has a reference yet
            const float common = kWide ? ms->common[seg & 3][share] : 0.0f;
            int t0 = ms->part[seg & 3].off * kTok;
            // where the totals of tiles of more than one run are kept, the record's place: of row c0, this thread's dim
            // (asked for when needed: a register less in the stages)
            auto totals = [&] { return p.ws_acc + (ms->part[seg & 3].rec + c0) * kHD + 32 * quad + lane; };
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++j, t0 += kTok) {
                wait_warp<true>(&ms->s_full, j & 1, ms);   // (the scales were there before the scores' operand)
                tc_fence_after();
                float2 sc[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) sc[m] = ms->scale[j & 3][32 * quad + 8 * m + (lane >> 2)];
                const bool bad = ms->bad[j & 3] != 0;
                // scores relative to the references: [pair of matrices][group][matrix of the pair][row of two]
                float t[2][kGroups][2][2];
                tmem_ld_fragments<kGroups>(lanes + L::kColS + c0, &t[0][0][0][0]);
                tmem_ld_fragments<kGroups>(lanes + (16u << 16) + L::kColS + c0, &t[1][0][0][0]);
                if constexpr (kWide) {
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < kVals * 4; ++k) asm volatile("" : "+f"((&t[0][0][0][0])[k]));
                } else {
                    float low[kVals * 4];
                    tmem_ld_fragments<kGroups>(lanes + L::kColS + kRows + c0, low);
                    tmem_ld_fragments<kGroups>(lanes + (16u << 16) + L::kColS + kRows + c0, low + kVals * 2);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < kVals * 4; ++k) {
                        asm volatile("" : "+f"((&t[0][0][0][0])[k]), "+f"(low[k]));
                        (&t[0][0][0][0])[k] = fmaf(low[k], 1.0f / (1 << kQLowBits), (&t[0][0][0][0])[k]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ms->s_free));
                if constexpr (kWide) {
                    if (__builtin_expect(common == 0.0f, 0)) {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) {
                            const float2 gain = *reinterpret_cast<const float2 *>(&ms->gain[seg & 3][col + 8 * g]);
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                t[m >> 1][g][m & 1][0] *= gain.x;
                                t[m >> 1][g][m & 1][1] *= gain.y;
                            }
                        }
                    } else {
#pragma unroll
                        for (int m = 0; m < 4; ++m) sc[m].x *= common;
                    }
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            float *x = t[m >> 1][g][m & 1];
                            const float2 y = fma2(make_float2(x[0], x[1]), make_float2(sc[m].x, sc[m].x), ref[g]);
                            x[0] = y.x;
                            x[1] = y.y;
                        }
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const float2 gain = *reinterpret_cast<const float2 *>(&ms->gain[seg & 3][col + 8 * g]);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            float *x = t[m >> 1][g][m & 1];
                            const float2 y = fma2(mul2(make_float2(x[0], x[1]), make_float2(sc[m].x, sc[m].x)), gain, ref[g]);
                            x[0] = y.x;
                            x[1] = y.y;
                        }
                    }
                }
                if (__builtin_expect(bad || t0 + kTok > lim_min, 0)) {   // some row does not see all of the stage
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const int2 lim = *reinterpret_cast<const int2 *>(&ms->lim[seg & 3][col + 8 * g]);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const int tok = bad ? 0x7fffffff : t0 + 32 * quad + 8 * m + (lane >> 2);
                            float *x = t[m >> 1][g][m & 1];
                            if (tok >= lim.x) x[0] = -INFINITY;
                            if (tok >= lim.y) x[1] = -INFINITY;
                        }
                    }
                }
                bool raise = fresh;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    float top = -INFINITY;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) top = max3(top, t[m >> 1][g][m & 1][0], t[m >> 1][g][m & 1][1]);
                    raise |= top > kPMaxLog2 - exponent_above(sc[m].y);
                }
                bool rest = i == 0;   // the product before is done: P's room is free, the accumulator at rest
                if (__builtin_expect(barrier_any(bar, 128, raise), 0)) {
                    // move the references of rows whose P would leave fp16's range (at first: of all), by whole
                    // numbers.  A row that a stage hides is hidden in all stages behind, but for bad blocks: a
                    // stage of one leaves the rows fresh
                    float vs_log2[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) vs_log2[m] = exponent_above(sc[m].y);
                    // the largest score + log2 V scale of row c0 + st, for the threads st < kCols
                    auto row_tops = [&] {
                        float top[kVals];
#pragma unroll
                        for (int g = 0; g < kGroups; ++g)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                top[2 * g + k] = fmaxf(fmaxf(t[0][g][0][k] + vs_log2[0], t[0][g][1][k] + vs_log2[1]),
                                                       fmaxf(t[1][g][0][k] + vs_log2[2], t[1][g][1][k] + vs_log2[3]));
                        halve<kVals / 2, 16>(top, lane, [](float a, float b) { return fmaxf(a, b); });
                        ms->wave[quad][folded_row] = top[0];
                        named_barrier_sync(bar, 128);
                        const int x = c0 + (st & (kCols - 1));
                        return fmaxf(fmaxf(ms->wave[0][x], ms->wave[1][x]), fmaxf(ms->wave[2][x], ms->wave[3][x]));
                    };
                    // the references move by ms->shift, and what is held with them
                    auto move = [&] {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) {
                            const float2 by = *reinterpret_cast<const float2 *>(&ms->shift[col + 8 * g]);
                            ref[g] = add2(ref[g], by);
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                t[m >> 1][g][m & 1][0] += by.x;
                                t[m >> 1][g][m & 1][1] += by.y;
                            }
                        }
                    };
                    float most = row_tops();
                    if (st < kCols) {
                        const float by = (fresh ? most > -INFINITY : most > kPMaxLog2) ? kPTopLog2 - ceilf(most) : 0.0f;
                        ms->ref[c0 + st] += by;
                        ms->shift[c0 + st] = by;
                    }
                    named_barrier_sync(bar, 128);
                    if (!rest && !fresh) {
                        wait_warp<!kWide>(&ms->pv_done, (j & 1) ^ 1, ms);
                        tc_fence_after();
                        rest = true;
#pragma unroll 1
                        for (int x = 0; x < (!kWide && kLow ? 2 : 1); ++x) {
#pragma unroll 1
                            for (int k = 0; k < kCols; k += 8) {
                                const uint32_t at = lanes + L::kColO + x * kRows + c0 + k;
                                float o[8];
                                uint32_t v[8];
                                tmem_ld8(at, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int q = 0; q < 8; ++q) {
                                    asm volatile("" : "+f"(o[q]));
                                    v[q] = __float_as_uint(o[q] * ex2_approx(ms->shift[c0 + k + q]));
                                }
                                tmem_st8(at, v);
                            }
                        }
                        tmem_wait_st();
                    }
                    if (i > L::kRun && !fresh) {
                        float *const total = totals();
                        const int rows = ms->part[seg & 3].rows;
#pragma unroll 1
                        for (int k = 0; k < kCols && c0 + k < rows; ++k)
                            if (ms->shift[c0 + k] != 0.0f)
                                store_relaxed(total + k * kHD, load_relaxed(total + k * kHD) * ex2_approx(ms->shift[c0 + k]));
                    }
                    bool far = false;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const float2 by = *reinterpret_cast<const float2 *>(&ms->shift[col + 8 * g]);
                        far |= fmaxf(fabsf(by.x), fabsf(by.y)) > 0x1p20f;
                        if (!fresh) {
                            const float2 fx = pow2_parts(by.x), fy = pow2_parts(by.y);
                            sum[g] = mul2(mul2(sum[g], make_float2(fx.x, fy.x)), make_float2(fx.y, fy.y));
                        }
                    }
                    move();
                    if (__builtin_expect(barrier_any(bar, 128, far), 0)) {
                        // Scores beyond 2^20: the distances that P depends on were lost in their rounding (from 2^26 on
                        // P would leave fp16's range).  Now that they are small, they move once more, exactly.  (What
                        // such a row held is 0.)
                        most = row_tops();
                        if (st < kCols) {
                            const float by = fabsf(ms->shift[c0 + st]) > 0x1p20f ? kPTopLog2 - ceilf(most) : 0.0f;
                            ms->ref[c0 + st] += by;
                            ms->shift[c0 + st] = by;
                        }
                        named_barrier_sync(bar, 128);
                        move();
                    }
                    fresh = fresh && bad;
                }
                // weights, and P = weight * V scale in high and low parts, kept until the product before is done
                // (which this overlaps)
                uint32_t hi[kGroups][4], lo[kGroups][4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float2 vs = make_float2(sc[m].y, sc[m].y);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const float *x = t[m >> 1][g][m & 1];
                        const float2 e = make_float2(ex2_approx(x[0]), ex2_approx(x[1]));
                        sum[g] = add2(sum[g], e);
                        const float2 v = mul2(e, vs);
                        const __half2 a = __floats2half2_rn(v.x, v.y);
                        hi[g][m] = half2_bits(a);
                        if (kLow) {
                            lo[g][m] = half2_bits(__floats2half2_rn(minus(v.x, __low2half(a)), minus(v.y, __high2half(a))));
                        }
                    }
                }
                if (!rest) wait_warp<true>(&ms->pv_done, (j & 1) ^ 1, ms);
                if (i % L::kRun == 0 && i > 0) {   // a run's end
                    tc_fence_after();
                    float *const total = totals();
                    const int rows = ms->part[seg & 3].rows - c0;
#pragma unroll 1
                    for (int k = 0; k < kCols; k += 8) {
                        float o[8];
                        read_output(k, o);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            if (k + q >= rows) continue;
                            if (i > L::kRun) add_relaxed(total + (k + q) * kHD, o[q]);
                            else store_relaxed(total + (k + q) * kHD, o[q]);
                        }
                    }
                }
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    store_matrices(pout + g * kCoreRow, hi[g][0], hi[g][1], hi[g][2], hi[g][3]);
                    if (kLow) store_matrices(pout + (g + kRows / 8) * kCoreRow, lo[g][0], lo[g][1], lo[g][2], lo[g][3]);
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ms->p_ready));
            }
            // ---- the tile's end: row sums over the tokens, then the output or a record ----
            halve<kVals / 2, 16>(&sum[0].x, lane, [](float a, float b) { return a + b; });
            ms->wave[quad][folded_row] = sum[0].x;
            more = queries(seg + 1);   // (while the last product runs)
            const Part &part = ms->part[seg & 3];
            const bool direct = part.direct != 0;
            const int row = 32 * quad + lane;   // dim
            named_barrier_sync(bar, 128);
            if (st < kCols) {
                const int x = c0 + st;
                const float S = ms->wave[0][x] + ms->wave[1][x] + ms->wave[2][x] + ms->wave[3][x];
                ms->shift[x] = direct ? (S > 0.0f ? 1.0f / S : 0.0f) : 1.0f;
                char *dst = nullptr;
                if (x < part.rows) {
                    if (direct) {
                        dst = static_cast<char *>(p.out) + (p.out_dtype == KVQ8_DTYPE_F32 ? 4 : 2) *
                                  (((long long)part.token + (x >> lg)) * p.out_stride +
                                   (long long)((part.head << lg) + (x & ((1 << lg) - 1))) * kHD);
                    } else {
                        dst = reinterpret_cast<char *>(p.ws_acc + (part.rec + x) * kHD);
                        // (a row that sees none of these tokens has no reference: the merge must not go by its 0)
                        *reinterpret_cast<float2 *>(p.ws_ml + (part.rec + x) * 2) =
                            make_float2(S > 0.0f ? -ms->ref[x] : -INFINITY, S);
                    }
                }
                ms->dst[x] = dst;
            }
            named_barrier_sync(bar, 128);
            wait_warp<!kWide>(&ms->pv_done, (j & 1) ^ 1, ms);
            tc_fence_after();
            const int type = direct ? p.out_dtype : KVQ8_DTYPE_F32;
            float *const total = totals();
#pragma unroll(kWide ? 2 : 1)
            for (int k = 0; k < kCols; k += 8) {
                float x[8];
                read_output(k, x);
                if (direct && n > L::kRun) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (c0 + k + q < part.rows) x[q] += load_relaxed(total + (k + q) * kHD);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) x[q] *= ms->shift[c0 + k + q];
                if (!direct && n > L::kRun) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (c0 + k + q < part.rows) add_relaxed(total + (k + q) * kHD, x[q]);
                } else if (type == KVQ8_DTYPE_F32) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (char *dst = ms->dst[c0 + k + q]) reinterpret_cast<float *>(dst)[row] = x[q];
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const uint16_t v = !kLow ? __bfloat16_as_ushort(__float2bfloat16_rn(x[q])) : __half_as_ushort(__float2half_rn(x[q]));
                        if (char *dst = ms->dst[c0 + k + q]) reinterpret_cast<uint16_t *>(dst)[row] = v;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_addr(&ms->o_free));
                mbar_arrive(smem_addr(&ms->part_free[seg & 3]));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kColumns);
    if (tid == 0 && ms->abort) flag_status(p.dev_status, KVQ8_DEV_TIMEOUT);
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
        for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < p.batch; b += gridDim.x * blockDim.x) p.ws_tail[b] = p.ws_first[b] = 0;
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
            p.ws_first[b] = b0;
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
    // record k: of CTA c + k; the first one is c's own second place
    auto at = [&](int k) { return ((long long)(c + k) * 3 + (k == 0 ? 1 : 0)) * rows_per_tile + i; };
    // four at a time, and asked for before the tile's rows are known (rows behind them are anything, and go nowhere)
    float m = -INFINITY, S = 0.0f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAtOnce = 4;
    for (int k0 = 0; k0 < dir.x; k0 += kAtOnce) {
        float2 ml[kAtOnce];
        float4 x[kAtOnce];
        float top = m;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            ml[k] = make_float2(-INFINITY, 0.0f);
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 + k < dir.x) {
                ml[k] = *reinterpret_cast<const float2 *>(p.ws_ml + at(k0 + k) * 2);
                x[k] = *reinterpret_cast<const float4 *>(p.ws_acc + at(k0 + k) * kHD + 4 * lane);
            }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);
        if (top == -INFINITY) continue;
        const float2 old = pow2_parts(m - top);   // 0 while m is -inf
        const float f_old = old.x * old.y;
        S = S * old.x * old.y;
        a = make_float4(a.x * f_old, a.y * f_old, a.z * f_old, a.w * f_old);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const float2 part = pow2_parts(ml[k].x - top);
            const float f = part.x * part.y;
            S = fmaf(ml[k].y * part.x, part.y, S);
            a.x = fmaf(x[k].x, f, a.x);
            a.y = fmaf(x[k].y, f, a.y);
            a.z = fmaf(x[k].z, f, a.z);
            a.w = fmaf(x[k].w, f, a.w);
        }
        m = top;
    }
    if (i >= w.tile_rows(w.r)) return;
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

// CTAs of a launch: one to an SM.
int tile_ctas() { return min(device_sm_count(), kMaxTileCtas); }

template <bool kShared, int kRows, bool kLow>
cudaError_t launch_tiles(const TileParams &p, int lg, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};
    const int ctas = tile_ctas();
    if (ctas <= 0) return cudaErrorInvalidDevice;
    return launch_after_setting(
        configured,
        [] {
            // the warpgroups trade registers within the launch's own: it must hold what they come to
            cudaFuncAttributes a;
            cudaError_t e = cudaFuncGetAttributes(&a, tile_kernel<kShared, kRows, kLow>);
            if (e != cudaSuccess) return e;
            if (Lay<kRows, kLow>::kWide && a.numRegs != Lay<kRows, kLow>::kLaunchRegs) return cudaErrorInvalidConfiguration;
            return cudaFuncSetAttribute(tile_kernel<kShared, kRows, kLow>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        Lay<kRows, kLow>::kBytes);
        },
        [&] {
            return launch_dependent(tile_kernel<kShared, kRows, kLow>, dim3(ctas), Lay<kRows, kLow>::kThreads, Lay<kRows, kLow>::kBytes, s, p, lg);
        });
}

int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

}  // namespace

// Rows per tile: the most that a sequence (on average, a group) has, up to 128, since a stage's time grows with its
// tile's rows, and each further tile turns the same codes into operands again.  8 sequences behind 4000 tokens, G = 4,
// with tiles of 32, 64 and 128 rows: 20 rows 29, 35, 45 us; 64 rows 46, 36, 47 us; 128 rows 74, 55, 52 us; of 16 and
// 32 rows: 8 rows 23.8, 26.7 us.  The counts that a tile really has are device data, which the rule does not see, so
// sequences or groups of very unequal counts are faster in calls of their own: a prompt of 2000 tokens beside 60 single
// tokens behind 4000 (G = 4, 8 kv heads) 349 us in one call, 110 + 107 in two; a group of 200 rows behind 8192 beside
// 199 groups of one row behind 1024 297 us, 84 + 130 in two.
static int rows_of(int64_t rows) { return rows > 64 ? 128 : rows > 32 ? 64 : rows > 16 ? 32 : 16; }

cudaError_t launch_prompt(const TileParams &p, int group, cudaStream_t s) {
    const int lg = log2_of(group), rows = rows_of((int64_t)p.n_new << lg);
    cudaError_t e;
    // (without P's low part, which bf16 outputs would not show: 4096 tokens x 16 heads 130 us, with it 150)
    if (p.out_dtype == KVQ8_DTYPE_BF16)
        e = rows == 128 ? launch_tiles<false, 128, false>(p, lg, s)
            : rows == 64 ? launch_tiles<false, 64, false>(p, lg, s) : rows == 32 ? launch_tiles<false, 32, false>(p, lg, s) : launch_tiles<false, 16, false>(p, lg, s);
    else
        e = rows == 128 ? launch_tiles<false, 128, true>(p, lg, s)
            : rows == 64 ? launch_tiles<false, 64, true>(p, lg, s) : rows == 32 ? launch_tiles<false, 32, true>(p, lg, s) : launch_tiles<false, 16, true>(p, lg, s);
    if (e != cudaSuccess) return e;
    return launch_dependent(prompt_merge_kernel, dim3(tile_ctas(), rows / kMergeWarps), kMergeWarps * 32, 0, s, p, lg, rows);
}

cudaError_t launch_shared_prefix(TileParams &p, int group, cudaStream_t s) {
    const int lg = log2_of(group);
    p.tile_rows = rows_of((((int64_t)p.batch << lg) + p.n_groups - 1) / p.n_groups);
    const int blocks = min((p.n_groups + kPlanWarps - 1) / kPlanWarps, 304);
    const cudaError_t e = launch_dependent(shared_plan_kernel, dim3(blocks), kPlanWarps * 32, 0, s, p);
    if (e != cudaSuccess) return e;
    return p.tile_rows == 128 ? launch_tiles<true, 128, true>(p, lg, s)
           : p.tile_rows == 64 ? launch_tiles<true, 64, true>(p, lg, s) : p.tile_rows == 32 ? launch_tiles<true, 32, true>(p, lg, s) : launch_tiles<true, 16, true>(p, lg, s);
}

}  // namespace kvq8
