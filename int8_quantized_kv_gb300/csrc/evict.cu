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

constexpr int kDigitBits = 11;                  // three digits of 11, 11 and 10 bits
constexpr int kBins = 1 << kDigitBits;
// Tokens whose keys a CTA keeps in shared memory: 80 KiB, so that two CTAs share
// an SM even where the table is wide (the keys of the others are made again
// from L2).
constexpr int kMostCached = 20 * 1024;
constexpr int kMostCtas = 8;                    // of a unit's cluster

// Order of a weight as an unsigned number: larger weights above smaller ones,
// -0 equal to 0, a NaN below everything.  Nothing maps to 0xffffffff, which
// marks a token that is kept whatever its weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t x = __float_as_uint(w);
    if ((x & 0x7fffffffu) > 0x7f800000u) return 0u;
    if ((x & 0x7fffffffu) == 0u) return 0x80000000u;
    return (x >> 31) ? ~x : (x | 0x80000000u);
}

// A CTA's share [lo, hi) of a unit's tokens, in the order that decides what is
// kept.  The keys of its first n_cached tokens are kept in shared memory, the
// others' made again.
struct Keys {
    const int32_t *row;
    const float *weight_sum;
    int nkv, h, lo, hi;
    int first, recent0;              // tokens below first and from recent0 on are kept
    uint32_t *cache;
    int n_cached;                    // a multiple of 4, as lo
    __device__ __forceinline__ uint32_t key(int t, float w) const {
        return t < first || t >= recent0 ? 0xffffffffu : weight_key(w);
    }
    __device__ __forceinline__ const float *at(int t) const {
        return weight_sum + ((size_t)row[t / kBS] * nkv + h) * kBS + t % kBS;
    }
    // Keys of the four tokens from t on, a multiple of 4 (w: their weights).
    __device__ __forceinline__ uint4 four(int t, float4 w) const {
        return make_uint4(key(t, w.x), key(t + 1, w.y), key(t + 2, w.z), key(t + 3, w.w));
    }
    __device__ __forceinline__ uint4 get4(int t) const {
        if (t - lo < n_cached) return *reinterpret_cast<const uint4 *>(cache + (t - lo));
        return four(t, *reinterpret_cast<const float4 *>(at(t)));
    }
};

// Inclusive sum over the warp's lanes from lane on to the last.
__device__ __forceinline__ int warp_suffix(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_down_sync(0xffffffffu, v, o);
        if (lane + o < 32) v += x;
    }
    return v;
}

// One CTA per unit, or a cluster of n_ctas (kCluster): each CTA takes a share of
// the unit's tokens, the digits' counts are added up through distributed shared
// memory, and every CTA finds the same digit.  A radix selection over the keys,
// then the list of kept tokens in order of position.  What the CTAs of a
// cluster branch on is read from one of them or from all of them, so that all
// take the same barriers.
template <int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 2 : 8)
evict_select_kernel(EvictParams p, int cache_tokens, int n_ctas) {
    constexpr int kWarps = kThreads / 32;
    constexpr int kThreadBins = kBins / kThreads;   // consecutive bins of a thread
    extern __shared__ __align__(16) uint32_t sm_keys[];
    __shared__ __align__(16) int hist[3][kBins];
    __shared__ int warp_a[kWarps], warp_b[kWarps];
    __shared__ int sh_digit, sh_need, sh_bad, sh_len;
    __shared__ __align__(8) int2 sh_total;
    // (in this order in every kernel that is not a split's merge: the next one then
    // starts only when those before this one are done, as a step with the cache
    // declared ready needs it)
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kCluster ? cluster_rank() : 0;
    if (!kCluster) n_ctas = 1;
    auto sync_all = [&] {
        if (kCluster) cluster_sync();
        else __syncthreads();
    };
    const int u = blockIdx.x / n_ctas, b = u / p.nkv, h = u % p.nkv;
    const int cap = p.max_blocks * kBS;
    int32_t *kept = p.kept + (size_t)u * p.keep;
    const int32_t *row = p.block_table + (size_t)b * p.max_blocks;
    const int32_t *dst = p.dst_table + (size_t)b * p.dst_max_blocks;
    if (tid == 0) {
        sh_bad = 0;
        if (rank == 0) {
            const int Lraw = p.ctx_lens[b];
            sh_len = max(0, min(Lraw, cap));
            if (Lraw != sh_len && h == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_CTX_LEN);
        }
    }
    for (int i = tid; i < 3 * kBins / 4; i += kThreads) reinterpret_cast<int4 *>(hist)[i] = make_int4(0, 0, 0, 0);
    sync_all();
    const int L = kCluster ? load_cluster_int(&sh_len, 0) : sh_len;
    const int m = min(L, p.keep);

    // every block id must lie in the pool, and a destination must be neither a
    // source of the sequence nor listed twice
    const int n_src = (L + kBS - 1) / kBS, n_dst = (m + kBS - 1) / kBS;
    bool bad = false;
    for (int i = rank * kThreads + tid; i < n_src; i += n_ctas * kThreads) bad |= row[i] < 0 || row[i] >= p.num_blocks;
    for (int d = rank * kWarps + warp; d < n_dst; d += n_ctas * kWarps) {
        const int id = dst[d];
        bad |= id < 0 || id >= p.num_blocks;
        for (int j = lane; j < n_src; j += 32) bad |= row[j] == id;
        for (int j = lane; j < d; j += 32) bad |= dst[j] == id;
    }
    if (bad) sh_bad = 1;
    sync_all();
    int any_bad = sh_bad;
    if (kCluster) any_bad = __any_sync(0xffffffffu, lane < n_ctas && load_cluster_int(&sh_bad, lane) != 0);
    if (any_bad && rank == 0 && tid == 0) flag_status(p.dev_status, KVQ8_DEV_BAD_BLOCK_ID);
    // a sequence with a bad id is left out; behind the last kept token -1; all tokens kept: no selection
    for (int j = (any_bad ? 0 : m) + rank * kThreads + tid; j < p.keep; j += n_ctas * kThreads) kept[j] = -1;
    if (any_bad || m == L) {
        if (!any_bad)
            for (int t = rank * kThreads + tid; t < L; t += n_ctas * kThreads) kept[t] = t;
        if (kCluster) cluster_sync();   // (no CTA leaves while another reads its shared memory)
        return;
    }

    // this CTA's share of the tokens
    const int cta_share = ((L + n_ctas - 1) / n_ctas + 127) / 128 * 128;
    const int c_lo = min(L, rank * cta_share), c_hi = min(L, c_lo + cta_share);
    const Keys keys = {row, p.weight_sum, p.nkv, h, c_lo, c_hi, p.n_first, L - p.n_recent, sm_keys,
                       min((c_hi - c_lo + 3) / 4 * 4, cache_tokens)};
    // the m-th largest key, digit by digit from the top: `prefix` holds the
    // digits found, `need` how many tokens with exactly this prefix are kept.
    // The first digit is counted as the weights are loaded.
    constexpr int kAhead = 4;   // weights loaded at once, in fours per thread
    for (int t0 = c_lo + 4 * tid; t0 < c_hi; t0 += kAhead * 4 * kThreads) {
        float4 w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = t0 + i * 4 * kThreads;
            if (t < c_hi) w[i] = *reinterpret_cast<const float4 *>(keys.at(t));   // (t % 4 == 0: within the block)
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = t0 + i * 4 * kThreads;
            if (t < c_hi) {
                const uint4 k = keys.four(t, w[i]);
                if (t - c_lo < keys.n_cached) *reinterpret_cast<uint4 *>(sm_keys + (t - c_lo)) = k;
                atomicAdd(&hist[0][k.x >> 21], 1);
                if (t + 1 < c_hi) atomicAdd(&hist[0][k.y >> 21], 1);
                if (t + 2 < c_hi) atomicAdd(&hist[0][k.z >> 21], 1);
                if (t + 3 < c_hi) atomicAdd(&hist[0][k.w >> 21], 1);
            }
        }
    }
    uint32_t prefix = 0;
    int need = m;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        if (pass > 0) {
            const int above = pass == 1 ? 21 : 10;
            for (int t = c_lo + 4 * tid; t < c_hi; t += 4 * kThreads) {
                const uint4 k4 = keys.get4(t);
                const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t + i < c_hi && (k[i] >> above) == (prefix >> above))
                        atomicAdd(&hist[pass][(k[i] >> shift) & (pass == 1 ? kBins - 1 : 1023)], 1);
            }
        }
        sync_all();
        // thread i: bins kThreadBins * i and on; the bin in which the need-th token from the top lies
        int bin[kThreadBins], sum = 0;
#pragma unroll
        for (int i = 0; i < kThreadBins / 4; ++i) {
            const int4 *mine = reinterpret_cast<const int4 *>(hist[pass]) + tid * (kThreadBins / 4) + i;
            int4 c = make_int4(0, 0, 0, 0);
            if (kCluster) {
                int4 x[kMostCtas];   // (all loads in flight at once)
#pragma unroll
                for (int r = 0; r < kMostCtas; ++r)
                    x[r] = r < n_ctas ? load_cluster_int4(mine, r) : make_int4(0, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < kMostCtas; ++r) {
                    c.x += x[r].x; c.y += x[r].y; c.z += x[r].z; c.w += x[r].w;
                }
            } else {
                c = *mine;
            }
            bin[4 * i] = c.x; bin[4 * i + 1] = c.y; bin[4 * i + 2] = c.z; bin[4 * i + 3] = c.w;
            sum += c.x + c.y + c.z + c.w;
        }
        const int suffix = warp_suffix(sum, lane);
        if (lane == 0) warp_a[warp] = suffix;
        __syncthreads();
        int above = __reduce_add_sync(0xffffffffu, lane > warp && lane < kWarps ? warp_a[lane] : 0) + suffix - sum;
        if (above < need && need <= above + sum) {   // (tokens above this thread's bins)
#pragma unroll
            for (int i = kThreadBins - 1; i >= 0; --i) {
                if (above < need && need <= above + bin[i]) {
                    sh_digit = kThreadBins * tid + i;
                    sh_need = need - above;
                }
                above += bin[i];
            }
        }
        __syncthreads();
        prefix |= (uint32_t)sh_digit << shift;
        need = sh_need;
        // (the next pass's first barrier keeps these reads before the next writes)
    }

    // tokens above the m-th largest are kept, and the first `need` equal to it:
    // each warp counts both in its share of the tokens, and writes them behind
    // those of the warps and CTAs before it
    const int share = ((c_hi - c_lo + kWarps - 1) / kWarps + 127) / 128 * 128;
    const int t_lo = min(c_hi, c_lo + warp * share), t_hi = min(c_hi, t_lo + share);
    // (tokens above, tokens equal) of the four tokens from t on
    auto count4 = [&](uint4 k4, int t, bool (&gt)[4], bool (&eq)[4]) {
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        int n_gt = 0, n_eq = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            gt[i] = t + i < t_hi && k[i] > prefix;
            eq[i] = t + i < t_hi && k[i] == prefix;
            n_gt += gt[i];
            n_eq += eq[i];
        }
        return make_int2(n_gt, n_eq);
    };
    bool is_gt[4], is_eq[4];
    int gt = 0, eq = 0;
    for (int t = t_lo + 4 * lane; t < t_hi; t += 128) {
        const int2 c = count4(keys.get4(t), t, is_gt, is_eq);
        gt += c.x;
        eq += c.y;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        warp_a[warp] = gt;
        warp_b[warp] = eq;
    }
    __syncthreads();
    if (kCluster) {
        if (warp == 0) {
            const int a = __reduce_add_sync(0xffffffffu, lane < kWarps ? warp_a[lane] : 0);
            const int c = __reduce_add_sync(0xffffffffu, lane < kWarps ? warp_b[lane] : 0);
            if (lane == 0) sh_total = make_int2(a, c);
        }
        cluster_sync();
    }
    gt = lane < warp ? warp_a[lane] : 0;   // (warp < kWarps <= 32)
    eq = lane < warp ? warp_b[lane] : 0;
    if (kCluster && lane < rank) {
        gt += load_cluster_int(&sh_total.x, lane);
        eq += load_cluster_int(&sh_total.y, lane);
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    for (int t0 = t_lo; t0 < t_hi; t0 += 128) {
        const int t = t0 + 4 * lane;
        const int2 c = count4(t < t_hi ? keys.get4(t) : make_uint4(0u, 0u, 0u, 0u), t, is_gt, is_eq);
        int run = c.x | c.y << 16, incl = run;   // both at most 128
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const int all = __shfl_sync(0xffffffffu, incl, 31);
        run = incl - run;
        int ng = gt + (run & 0xffff), ne = eq + (run >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (is_gt[i] || (is_eq[i] && ne < need)) kept[ng + min(ne, need)] = t + i;
            ng += is_gt[i];
            ne += is_eq[i];
        }
        gt += all & 0xffff;
        eq += all >> 16;
    }
    if (kCluster) cluster_sync();   // (as above)
}

// One CTA per 64 kept tokens of a unit (a quarter of a destination tile).  K
// rows are copied 16 bytes at a time into their new chunk order.  V is stored
// with the 64 tokens of a quarter side by side per dim, so a token is a byte
// of every 64-byte row: the source quarters that hold one of the tokens are
// copied into shared memory, kSrcQuarters at a time, only the 32-byte halves
// of their rows that hold one, and each thread collects the 16 bytes of (dim,
// 16 tokens) from there.  Which bytes these are is the same for every dim: four
// tokens' bytes come from at most four aligned words of the row, and a byte
// permutation per word, made once per CTA, puts them in place.
constexpr int kCopyThreads = 128;
constexpr int kSrcQuarters = 3;   // half of the tokens kept: two or three source quarters
constexpr int kVStage = kTileVQuarter;

// Where byte s (0..63) of dim d's row is in a staged quarter: its 16-byte
// pieces are permuted so that eight rows' same word lies in different banks.
__device__ __forceinline__ int staged_byte(int d, int s) { return d * kStageTok + (s ^ (((d >> 1) & 3) << 4)); }

__global__ void __launch_bounds__(kCopyThreads, 9)
evict_copy_kernel(EvictParams p, int quarters) {
    __shared__ __align__(16) unsigned char stage[kSrcQuarters * kVStage];
    __shared__ int src_tok[kStageTok];          // source position of each token, -1 behind the last
    __shared__ int src_tile[kStageTok];         // its (block, kv head) tile
    __shared__ int src_off[kStageTok];          // its byte in the staged rows: quarter's place in the list * kVStage + slot
    __shared__ int2 moves[kStageTok / 4][4];    // per four tokens: (aligned word of the staged row, permutation), or -1
    __shared__ int list_q[kStageTok];           // the distinct source quarters: tile * 4 + quarter
    __shared__ unsigned list_half[kStageTok];   // which halves of them
    __shared__ int n_list;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int u = blockIdx.x / quarters, qd = blockIdx.x % quarters;
    const int b = u / p.nkv, h = u % p.nkv;
    const int32_t *kept = p.kept + (size_t)u * p.keep + qd * kStageTok;
    const int most = min(kStageTok, p.keep - qd * kStageTok);
    const int32_t *row = p.block_table + (size_t)b * p.max_blocks;
    const size_t dst = (size_t)p.dst_table[(size_t)b * p.dst_max_blocks + qd / 4] * p.nkv + h;
    // the CTA of the sequence's last kept token knows how many there are (written
    // here and not in the selection, so that new_lens may be ctx_lens itself)
    const bool more = h == 0 && tid == 0 && p.keep - qd * kStageTok > kStageTok && kept[kStageTok] >= 0;
    if (tid < kStageTok) {
        const int t = tid < most ? kept[tid] : -1;
        src_tok[tid] = t;
        src_tile[tid] = t >= 0 ? row[t / kBS] * p.nkv + h : 0;
        list_half[tid] = 0u;
    }
    __syncthreads();
    if (warp == 0 && h == 0) {
        const int count = __popc(__ballot_sync(0xffffffffu, src_tok[lane] >= 0)) +
                          __popc(__ballot_sync(0xffffffffu, src_tok[32 + lane] >= 0));
        if (lane == 0 && !more && (count > 0 || qd == 0)) p.new_lens[b] = qd * kStageTok + count;
    }
    if (src_tok[0] < 0) return;
    const int slot0 = (qd % 4) * kStageTok;     // slot of the first token

    // warp 0: the distinct source quarters, in order (the positions increase)
    if (warp == 0) {
        int before = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i, t = src_tok[j];
            const bool fresh = t >= 0 && (j == 0 || src_tok[j - 1] / kStageTok != t / kStageTok);
            const unsigned f = __ballot_sync(0xffffffffu, fresh);
            const int at = before + __popc(f & ((2u << lane) - 1)) - 1;
            if (fresh) list_q[at] = src_tile[j] * 4 + (t / kStageTok) % 4;
            src_off[j] = t >= 0 ? at * kVStage + t % kStageTok : -1;
            if (t >= 0) atomicOr(&list_half[at], 1u << ((t % kStageTok) / 32));
            before += __popc(f);
        }
        if (lane == 0) n_list = before;
        __syncwarp();
        if (lane < kStageTok / 4) {
            int word = -1, count = 0;
            unsigned sel = 0x3210u;   // keep the four bytes as they are
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int off = src_off[4 * lane + i];
                if (off < 0) break;
                if (word >= 0 && (off & ~3) != word) {
                    moves[lane][count++] = make_int2(word, (int)sel);
                    sel = 0x3210u;
                }
                word = off & ~3;
                sel = (sel & ~(0xfu << (4 * i))) | ((4u + (off & 3)) << (4 * i));   // byte i: byte off % 4 of the word
            }
            if (word >= 0) moves[lane][count++] = make_int2(word, (int)sel);
            for (; count < 4; ++count) moves[lane][count] = make_int2(-1, 0);
        }
    }
    // K: eight threads to a row
    uint4 k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = (tid >> 3) + 16 * i, t = src_tok[j];
        if (t >= 0)
            k[i] = reinterpret_cast<const uint4 *>(p.k_pool + ((size_t)src_tile[j] * kBS + t % kBS) * kHD)[(tid & 7) ^ (t & 7)];
    }
    __syncthreads();
    // copies of the source quarters q0 .. q0 + kSrcQuarters - 1 into the stage
    const int n = n_list;
    auto fetch = [&](int q0) {
#pragma unroll
        for (int q = 0; q < kSrcQuarters; ++q) {
            if (q0 + q < n) {
                const unsigned half = list_half[q0 + q];
                const int at = list_q[q0 + q];
                const int8_t *src = p.v_pool + (size_t)(at >> 2) * kBS * kHD + (size_t)(at & 3) * kTileVQuarter;
                if (half >> ((tid & 3) >> 1) & 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // thread: piece tid & 3 of rows tid >> 2, + 32, + 64, + 96
                        const int d = (tid >> 2) + 32 * i;
                        cp_async16_cg(stage + q * kVStage + staged_byte(d, (tid & 3) * 16), src + d * kStageTok + (tid & 3) * 16);
                    }
                }
            }
        }
        cp_async_commit();
    };
    fetch(0);
    // scales and weights meanwhile, and K's rows
    float sw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = tid + kCopyThreads * i, j = x % kStageTok, t = src_tok[j];
        const float *a = x < kStageTok ? p.k_scale : x < 2 * kStageTok ? p.v_scale : p.weight_sum;
        if (x < 3 * kStageTok && t >= 0) sw[i] = a[(size_t)src_tile[j] * kBS + t % kBS];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = (tid >> 3) + 16 * i;
        if (src_tok[j] >= 0)
            reinterpret_cast<uint4 *>(p.k_pool + (dst * kBS + slot0 + j) * kHD)[(tid & 7) ^ (j & 7)] = k[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = tid + kCopyThreads * i, j = x % kStageTok;
        float *a = x < kStageTok ? p.k_scale : x < 2 * kStageTok ? p.v_scale : p.weight_sum;
        if (x < 3 * kStageTok && src_tok[j] >= 0) a[dst * kBS + slot0 + j] = sw[i];
    }
    // V: thread (r, g): the 16 tokens 16g.. of dims r, r + 32, r + 64, r + 96
    const int g = tid & 3, r = tid >> 2;
    uint32_t out[4][4] = {};
    for (int q0 = 0; q0 < n; q0 += kSrcQuarters) {
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 4; ++w) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int2 mv = moves[4 * g + w][e];
                const int from = mv.x - q0 * kVStage;
                if (mv.x >= 0 && from >= 0 && from < kSrcQuarters * kVStage) {
                    // (rows r, r + 32, ... have their pieces permuted alike)
                    const unsigned char *x = stage + (from & ~(kStageTok - 1)) + staged_byte(r, from & (kStageTok - 1));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        out[i][w] = __byte_perm(out[i][w], *reinterpret_cast<const uint32_t *>(x + 32 * i * kStageTok), mv.y);
                }
            }
        }
        if (q0 + kSrcQuarters < n) {
            __syncthreads();
            fetch(q0 + kSrcQuarters);
        }
    }
    // 16 tokens of a dim are 16 contiguous bytes; behind the last token nothing is written
    int live = 16;
    if (src_tok[kStageTok - 1] < 0)
        live = min(16, max(0, __popc(__ballot_sync(0xffffffffu, src_tok[lane] >= 0)) +
                                  __popc(__ballot_sync(0xffffffffu, src_tok[32 + lane] >= 0)) - 16 * g));
    int8_t *vd = p.v_pool + dst * kBS * kHD + (size_t)(qd % 4) * kTileVQuarter + 16 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int8_t *d = vd + (r + 32 * i) * kStageTok;
        if (live == 16) {
            *reinterpret_cast<uint4 *>(d) = make_uint4(out[i][0], out[i][1], out[i][2], out[i][3]);
        } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (4 * w + 4 <= live) {
                    reinterpret_cast<uint32_t *>(d)[w] = out[i][w];
                } else {
#pragma unroll
                    for (int c = 0; c < 3; ++c)
                        if (4 * w + c < live) d[4 * w + c] = (int8_t)(out[i][w] >> (8 * c));
                }
            }
        }
    }
}

cudaError_t launch_copy(const EvictParams &p, int quarters, unsigned blocks, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_copy_kernel, p, quarters);
}

template <int kThreads, bool kCluster>
cudaError_t launch_select(const EvictParams &p, int n_ctas, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};
    // keys of as many tokens as a CTA's share of the table, up to kMostCached
    const int64_t share = ((int64_t)p.max_blocks * kBS + n_ctas - 1) / n_ctas;
    const int cached = (int)min((share + 127) / 128 * 128, (int64_t)kMostCached);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.batch * p.nkv * n_ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = cached * sizeof(uint32_t);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = n_ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster ? 2 : 1;
    return launch_after_setting(
        configured,
        [] {
            return cudaFuncSetAttribute(evict_select_kernel<kThreads, kCluster>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, kMostCached * (int)sizeof(uint32_t));
        },
        [&] { return cudaLaunchKernelEx(&cfg, evict_select_kernel<kThreads, kCluster>, p, cached, n_ctas); });
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t s) {
    const int quarters = (p.keep + kStageTok - 1) / kStageTok;
    const int64_t units = (int64_t)p.batch * p.nkv, blocks = units * quarters;
    const int64_t tokens = (int64_t)p.max_blocks * kBS;   // most tokens of a unit
    if (blocks > 2147483647 || units > 2147483647 / 8) return cudaErrorInvalidConfiguration;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Small tables: CTAs of 128 threads, eight to an SM up to 768 tokens and six
    // at 2048 (24 KiB of counts and the keys each).  Else 512 threads, two
    // to an SM (1024 leave room for one: 224 units of 8192 tokens then took two
    // rounds), and where that leaves SMs idle, clusters of up to eight CTAs per
    // unit with at least 8192 tokens each, the table's width taken for the
    // lengths, which the host does not know.  (Whole calls: 32 units of 131072
    // tokens 363 -> 202 us, 32 of 32768 91 -> 66, 18 of 24000 53 -> 45; with
    // 2048 tokens per CTA the cluster's barriers cost more than they save: 64
    // units of 8192 44 -> 49, 32 of 32768 76.)
    int n_ctas = 1;
    while (n_ctas < kMostCtas && units * n_ctas <= sms && tokens / (2 * n_ctas) >= 8192) n_ctas *= 2;
    cudaError_t e;
    if (tokens <= 2048) e = launch_select<128, false>(p, 1, s);
    else if (n_ctas > 1) e = launch_select<512, true>(p, n_ctas, s);
    else e = launch_select<512, false>(p, 1, s);
    if (e != cudaSuccess) return e;
    return launch_copy(p, quarters, (unsigned)blocks, s);
}

}  // namespace kvq8
