// The next token of each row of logits, from given random numbers.
//
// Per row: the tokens in order of falling logit (lowest index first on ties,
// the router's own rule); the first top_k of them; of those the shortest
// prefix that holds top_p of their mass, with masses e_i = exp((l_i - max) /
// temperature); of those the ones with e_i >= min_p; and then, in the order of
// the tokens, the first whose running mass exceeds u times the kept mass.
//
// Masses are held as integers in units of 2^-45 of the largest one (one unit at
// least: u = 0 is the first token that takes part), each within 3e-9 of the true
// one, so sums do not depend on the order of the atomics.  Three roundings remain,
// the same on every run:
//   - The whole mass that top_p is taken of counts the tokens far below the largest
//     (less than 1/64 of the largest mass together) by an approximate 2^x, summed in
//     fp32 per thread: off by less than 2^-23 of the largest mass (Softmax::
//     approximate).  Whether one of them itself is kept goes by its integer mass.
//   - A histogram's bin drops what is below one unit once for all its tokens, a list
//     or a pass once for each token: 2^-32 of the largest mass in all.
//   - Running sums are compared with top_p of the whole as doubles, 2^-53 of a sum.
//
// A row belongs to a cluster of thread blocks that keep it in their shared
// memory: the logits are read from memory once, the later passes read shared
// memory, and the blocks exchange histograms, sums and lists over distributed
// shared memory.  The whole row is never sorted:
//   - Tokens fall into bins of 1/32 of a power of two of mass.  A histogram (of
//     the threads' largest tokens, which bounds the top_k from below, or of all
//     tokens that the top_p could reach, with their masses) names the bin where
//     a prefix ends.
//   - If the tokens down to that bin are few (2048), the first block of the
//     cluster gets them as a list and finishes the row alone.
//   - Else it gets the tokens of that bin alone and finds the cut inside; the
//     blocks then add up what lies above the cut, in the order of the tokens.
//   - Where a bin holds more than a list takes (many equal logits), the cut is
//     found by selecting 11, 11 and 10 bits of the logits' ordered integers.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kSaThreads = 512;
constexpr int kSaWarps = kSaThreads / 32;
constexpr int kSaMaxCluster = 8;
constexpr int kMassBits = 45;
constexpr int kList = 2048;               // tokens of a list
constexpr int kMassBins = 1024;           // bins of 1/32 of a power of two
constexpr int kKeyBins = 2048;            // bins of the selection by key bits
// a block's scratch: a list of its own tokens and, in the first block, the row's
// (or the 3 x kKeyBins words of the selection by key bits); then the histogram
constexpr int kScratchWords = 2 * 2 * kList;
constexpr int kHistWords = 2 * kMassBins;
static_assert(kScratchWords >= 3 * kKeyBins, "scratch");
constexpr float kMagic = 12582912.0f;     // 1.5 x 2^23: adding it rounds to an integer in the low bits

// Ordered integers of logits: the sign bit set for values >= 0, all bits
// inverted below.  (Logits are kept with -0 as +0; what may not be chosen and
// NaN as -infinity.)
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xff800000u); }

// Masses 2^x, x = (l - max) c, c = log2(e) / temperature.  32 l c is rounded to an
// integer k_l by one fused multiply-add; r = l c - k_l / 32 is another, exact but
// for one rounding of a number below 1/64; with k_m and r_m of the largest logit,
// 2^x = 2^(floor(k / 32)) T[k mod 32] (1 + q), k = k_l - k_m, T[j] = 2^(j / 32) in
// 31 bits and q = 2^(r - r_m) - 1 by its Taylor polynomial to degree 4 (remainder
// 4e-11): within 3e-9 of the true value, in fp32 and integer instructions.  (With
// fp64 and a polynomial of degree 9, 256 x 131072 tokens took 4 times as long.)
// Where |max c| is too large for k_l, l - max takes the place of l; it is exact
// for every token whose mass is not far below the smallest unit.
struct Softmax {
    float max_logit, shift, c, c32, c_lo, rm, t_max;   // t_max: kMagic + k_m
    double m, cd;
    const uint32_t* tab;                    // shared: round(2^(30 + j / 32))
    __device__ __forceinline__ void init(float largest, float temperature, const uint32_t* table) {
        max_logit = largest;
        m = (double)largest;
        cd = 1.4426950408889634074 / (double)temperature;
        c = (float)cd;
        c_lo = (float)(cd - (double)c);
        c32 = c * 32.0f;
        shift = fabs(m * cd) > 65536.0 ? max_logit : 0.0f;
        t_max = place(max_logit);
        rm = (float)((m - (double)shift) * cd - (double)(t_max - kMagic) / 32.0);
        tab = table;
    }
    // kMagic + k_l: falls with the logit, -infinity for tokens that take no part
    __device__ __forceinline__ float place(float l) const { return __fmaf_rn(__fsub_rn(l, shift), c32, kMagic); }
    __device__ __forceinline__ int bin(float t) const { return (int)__fsub_rn(t_max, t); }
    // the 31-bit mantissa (units of 2^-30) of a token at place t, at least t_max - 2^15
    __device__ __forceinline__ uint32_t mantissa(float l, float t) const {
        const float lr = __fsub_rn(l, shift);
        float r = __fmaf_rn(lr, c, __fmul_rn(__fsub_rn(t, kMagic), -0.03125f));
        r = __fsub_rn(__fmaf_rn(lr, c_lo, r), rm);
        float p = __fmaf_rn(r, 0.00961812910763f, 0.0555041086648f);   // ln2^4 / 24, ln2^3 / 6
        p = __fmaf_rn(p, r, 0.240226506959f);                          // ln2^2 / 2
        p = __fmaf_rn(p, r, 0.693147180560f);
        p = __fmul_rn(p, r);
        const uint32_t T = tab[(__float_as_int(t) - __float_as_int(t_max)) & 31];
        const int q = __float2int_rn(__fmul_rn(p, 4294967296.0f));
        return T + (uint32_t)(int)(((int64_t)(uint64_t)T * q) >> 32);
    }
    // The places and mantissas of four tokens, by pairs of operations.
    __device__ __forceinline__ void place4(const float4& l, Pair (&lr)[2], Pair (&t)[2]) const {
        const Pair less(-shift, -shift), scale(c32, c32), magic(kMagic, kMagic);
        lr[0] = Pair(l.x, l.y) + less;
        lr[1] = Pair(l.z, l.w) + less;
        t[0] = fma2(lr[0], scale, magic);
        t[1] = fma2(lr[1], scale, magic);
    }
    __device__ __forceinline__ void mantissa4(const Pair (&lr)[2], const Pair (&t)[2], uint32_t (&M)[4]) const {
        auto two = [](float v) { return Pair(v, v); };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            Pair r = fma2(lr[i], two(c), (t[i] + two(-kMagic)) * two(-0.03125f));
            r = fma2(lr[i], two(c_lo), r) + two(-rm);
            Pair p = fma2(r, two(0.00961812910763f), two(0.0555041086648f));
            p = fma2(p, r, two(0.240226506959f));
            p = fma2(p, r, two(0.693147180560f));
            p = p * r * two(4294967296.0f);
            float q[2], at[2];
            p.get(q[0], q[1]);
            t[i].get(at[0], at[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t T = tab[(__float_as_int(at[j]) - __float_as_int(t_max)) & 31];
                M[2 * i + j] = T + (uint32_t)(int)(((int64_t)(uint64_t)T * __float2int_rn(q[j])) >> 32);
            }
        }
    }
    // in units of 2^-45, for a token `below` places under the largest
    static __device__ __forceinline__ uint64_t fixed(uint32_t M, int below) {
        return ((uint64_t)M << (kMassBits - 30)) >> ((below + 31) >> 5);
    }
    __device__ __forceinline__ uint64_t mass(float l) const {
        const float t = place(l);
        if (!(t >= t_max - 46.0f * 32)) return t >= t_max - 32000.0f ? 1 : 0;
        return max(fixed(mantissa(l, t), bin(t)), (uint64_t)1);
    }
    // The mass 2^x as a fraction of the largest, for the tokens far below it.  l - max, c
    // and their product are rounded to fp32, 3 |x| ln 2 < 2.1 |x| units of 2^-24 of the
    // mass; ex2.approx adds 4, and a thread's sum over up to 64 tokens 64 more.  Masses are
    // at most 2^-x0, x0 = 6.5 + log2(vocab), so all of them together are off by at most
    // vocab 2^-x0 (2.1 x0 + 68) < 1.4 of these units.
    __device__ __forceinline__ float approximate(float l) const {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(__fsub_rn(l, max_logit), c)));
        return e;
    }
    // the mass in 64 bits, for the chosen token's probability
    __device__ __forceinline__ double exact(float l) const { return exp2(((double)l - m) * cd); }
};

// The two halves of a cluster barrier: a block's shared memory may be accessed from
// another one only when it is known to have started.  (Not .aligned: a warp's lanes
// need not have come back together.)  Announcing the start orders nothing before it.
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

__device__ __forceinline__ uint64_t warp_sum_u64(uint64_t v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ uint64_t warp_scan_u64(uint64_t v, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

struct SaShared {
    uint64_t slots[2][kSaMaxCluster];     // per reduction, alternating: one value per block
    uint64_t warp_sum[kSaWarps];
    uint64_t coarse[32], total;           // this block's histogram by powers of two, and its mass
    uint64_t gather[2][kSaMaxCluster][32], gather_total[kSaMaxCluster];
    uint64_t found_above, found_entry;
    uint64_t block_above[kSaMaxCluster];  // in the first block: each block's mass over the bin of the cut
    uint64_t pick_target, pick_total;
    int32_t pick_block;
    uint32_t found;
    float cut_value;
    int32_t cut_index;
    uint32_t list_base, list_count[2];    // list_count: of the row's lists, in the first block
    uint32_t own_count;
    uint32_t tab[32];
};

// The tokens still in the running: logit above K, or equal to K and index below I.
struct Cut {
    float K;
    int I;
    __device__ __forceinline__ bool in(float l, int index) const { return l > K || (l == K && index < I); }
};

// One row of a cluster.
struct Row {
    cg::cluster_group cl;
    int nb, rank;                // blocks of the cluster, this one
    SaShared* sh;
    float* logits;               // this block's tokens [lo, lo + n), -infinity up to a multiple of 4
    uint32_t* scratch;
    uint32_t* hist;
    int lo, n, per_warp;         // a warp owns tokens [warp * per_warp, + per_warp) of the block's
    int turn;
    int tid, lane, warp;

    // Sum of v over the cluster, and over the blocks before this one.
    __device__ uint64_t sum(uint64_t v, uint64_t& before) {
        v = warp_sum_u64(v);
        __syncthreads();
        if (lane == 0) sh->warp_sum[warp] = v;
        __syncthreads();
        if (warp == 0) {
            v = warp_sum_u64(lane < kSaWarps ? sh->warp_sum[lane] : 0);
            if (lane < nb) *cl.map_shared_rank(&sh->slots[turn][rank], lane) = v;
        }
        cl.sync();
        uint64_t total = 0;
        before = 0;
        for (int i = 0; i < nb; ++i) {
            const uint64_t s = sh->slots[turn][i];
            if (i < rank) before += s;
            total += s;
        }
        turn ^= 1;
        return total;
    }
    // The largest of v over the cluster: its first exchange.  Every thread has arrived
    // at the cluster's barrier when its block started; waiting here, after the row has
    // been read, costs nothing.
    __device__ float max_logit(float v) {
        uint32_t k = __reduce_max_sync(0xffffffffu, key_of(v));
        if (lane == 0) sh->warp_sum[warp] = k;
        __syncthreads();
        cluster_wait();
        if (warp == 0) {
            k = __reduce_max_sync(0xffffffffu, lane < kSaWarps ? (uint32_t)sh->warp_sum[lane] : 0u);
            if (lane < nb) *cl.map_shared_rank(&sh->slots[turn][rank], lane) = k;
        }
        cl.sync();
        k = 0;
        for (int i = 0; i < nb; ++i) k = max(k, (uint32_t)sh->slots[turn][i]);
        turn ^= 1;
        return value_of(k);
    }
    // Sum over the threads of the block.
    __device__ uint64_t block_sum(uint64_t v) {
        v = warp_sum_u64(v);
        __syncthreads();
        if (lane == 0) sh->warp_sum[warp] = v;
        __syncthreads();
        return warp_sum_u64(lane < kSaWarps ? sh->warp_sum[lane] : 0);
    }
    // Inclusive scan of v over the threads of the block, and the sum of all.
    __device__ uint64_t block_scan(uint64_t v, uint64_t& total) {
        v = warp_scan_u64(v, lane);
        __syncthreads();
        if (lane == 31) sh->warp_sum[warp] = v;
        __syncthreads();
        uint64_t s = lane < kSaWarps ? sh->warp_sum[lane] : 0;
        total = warp_sum_u64(s);
        return v + warp_sum_u64(lane < warp ? s : 0);
    }
    // A block's last step: the others leave, the first one when none of them
    // reads its shared memory any more.
    __device__ void leave() {
        cluster_arrive();
        if (rank == 0) cluster_wait();
    }
};

// ------------------------------------------------------------------ selection by key bits

// Among the tokens inside `cut`, in order of falling logit: the one at which
// the running count (or mass) reaches `need`, and how much lies strictly above
// it.  False when the whole set does not reach it.
template <bool MASS>
__device__ __noinline__ bool select_key(Row& r, const Softmax& sm, const Cut& cut, double need, float& value_out,
                                        uint64_t& above_out) {
    constexpr int kPer = kKeyBins / kSaThreads;
    uint32_t prefix = 0, mask = 0;
    uint64_t above = 0;
    uint32_t* h = r.scratch;
    for (int lv = 0; lv < 3; ++lv) {
        const int shift = lv == 0 ? 21 : lv == 1 ? 10 : 0, bins = lv == 2 ? 1024 : 2048;
        r.cl.sync();   // nobody reads the last histogram any more
        for (int i = r.tid; i < (MASS ? 3 : 1) * kKeyBins; i += kSaThreads) h[i] = 0;
        __syncthreads();
        for (int i = r.tid; i < r.n; i += kSaThreads) {
            const float l = r.logits[i];
            const uint32_t k = key_of(l);
            if ((k & mask) != prefix || !cut.in(l, r.lo + i)) continue;
            const int bin = (k >> shift) & (bins - 1);
            if constexpr (MASS) {
                // 15 bits at a time: 2^15 tokens of a block cannot overflow a sum
                const uint64_t m = sm.mass(l);
                if (m & 0x7fffu) atomicAdd(&h[bin], (uint32_t)(m & 0x7fffu));
                if ((m >> 15) & 0x7fffu) atomicAdd(&h[kKeyBins + bin], (uint32_t)((m >> 15) & 0x7fffu));
                if (m >> 30) atomicAdd(&h[2 * kKeyBins + bin], (uint32_t)(m >> 30));
            } else {
                atomicAdd(&h[bin], 1u);
            }
        }
        r.cl.sync();
        // thread t: bins from the top, [bins - 1 - t * kPer .. - (kPer - 1)]
        uint64_t v[kPer];
        uint64_t mine = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int bin = bins - 1 - (r.tid * kPer + j);
            uint64_t s = 0;
            if (bin >= 0)
                for (int b = 0; b < r.nb; ++b) {
                    const uint32_t* hb = r.cl.map_shared_rank(h, b);
                    s += hb[bin];
                    if constexpr (MASS) s += ((uint64_t)hb[kKeyBins + bin] << 15) + ((uint64_t)hb[2 * kKeyBins + bin] << 30);
                }
            v[j] = s;
            mine += s;
        }
        if (r.tid == 0) r.sh->found = 0xffffffffu;
        uint64_t all;
        uint64_t before = above + r.block_scan(mine, all) - mine;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if ((double)before < need && (double)(before + v[j]) >= need) {
                r.sh->found = (uint32_t)(bins - 1 - (r.tid * kPer + j));
                r.sh->found_above = before;
            }
            before += v[j];
        }
        __syncthreads();
        const uint32_t bin = r.sh->found;
        if (bin == 0xffffffffu) return false;   // the same in every block: they see the same sums
        above = r.sh->found_above;
        prefix |= bin << shift;
        mask |= (uint32_t)(bins - 1) << shift;
    }
    value_out = value_of(prefix);
    above_out = above;
    return true;
}

// The index of the tie number `keep` (from 0, in the order of the tokens) among
// the tokens inside `cut` whose logit is K: the first one left out; `none` when
// there are not that many.
__device__ __noinline__ int tie_limit(Row& r, const Cut& cut, float K, uint64_t keep, int none) {
    const int w0 = r.warp * r.per_warp, w1 = min(r.n, w0 + r.per_warp);
    uint32_t c = 0;
    for (int i = w0 + r.lane; i < w1; i += 32) c += r.logits[i] == K && cut.in(K, r.lo + i);
    const uint64_t mine = warp_sum_u64(c);
    uint64_t before;
    if (r.sum(c, before) <= keep) return none;
    __syncthreads();
    if (r.lane == 0) r.sh->warp_sum[r.warp] = mine;
    if (r.tid == 0) r.sh->cut_index = 0;
    __syncthreads();
    for (int w = 0; w < r.warp; ++w) before += r.sh->warp_sum[w];
    if (before <= keep && keep < before + mine) {
        uint64_t at = before;
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const int i = i0 + r.lane;
            const bool is = i < w1 && r.logits[i] == K && cut.in(K, r.lo + i);
            const uint32_t m = __ballot_sync(0xffffffffu, is);
            if (keep < at + __popc(m)) {
                if (is && __popc(m & ((1u << r.lane) - 1)) == (int)(keep - at)) r.sh->cut_index = r.lo + i;
                break;
            }
            at += __popc(m);
        }
    }
    __syncthreads();
    uint64_t unused;
    const int local = r.sh->cut_index;   // 0 in every block but one
    return (int)r.sum(r.tid == 0 ? (uint64_t)local : 0, unused);
}

// The first top_k tokens inside `cut`, by key bits.
__device__ __noinline__ void cut_count(Row& r, const Softmax& sm, Cut& cut, int top_k, int vocab) {
    float K = 0;
    uint64_t above = 0;
    if (!select_key<false>(r, sm, cut, (double)top_k, K, above)) return;
    cut = Cut{K, tie_limit(r, cut, K, (uint64_t)top_k - above, vocab)};
}

// The shortest prefix of the tokens inside `cut` whose mass reaches `need`, by key bits.
__device__ __noinline__ void cut_mass(Row& r, const Softmax& sm, Cut& cut, double need, int vocab) {
    float K = 0;
    uint64_t above = 0;
    if (!select_key<true>(r, sm, cut, need, K, above)) return;
    const uint64_t ties = (uint64_t)fmax(1.0, ceil((need - (double)above) / (double)sm.mass(K)));
    const int I = tie_limit(r, cut, K, ties, vocab);
    cut = Cut{K, K == cut.K ? min(I, cut.I) : I};
}

// ------------------------------------------------------------------ lists

// Entries order by falling logit, then rising index.
__device__ __forceinline__ uint64_t entry_of(float l, int index) { return ((uint64_t)key_of(l) << 32) | (uint32_t)~index; }
__device__ __forceinline__ float entry_logit(uint64_t e) { return value_of((uint32_t)(e >> 32)); }
__device__ __forceinline__ int entry_index(uint64_t e) { return (int)~(uint32_t)e; }

// The row's tokens at places [t0, t1] as list number `which` in the first
// block's scratch (second half).  Returns how many there are; more than kList:
// the list is incomplete.
__device__ uint32_t make_list(Row& r, const Softmax& sm, float t0, float t1, int which) {
    uint64_t* own = reinterpret_cast<uint64_t*>(r.scratch);
    __syncthreads();
    if (r.tid == 0) r.sh->own_count = 0;
    __syncthreads();
#pragma unroll 2
    for (int i = r.tid * 4; i < r.n; i += kSaThreads * 4) {
        const float4 q = *reinterpret_cast<const float4*>(r.logits + i);
        const float l[4] = {q.x, q.y, q.z, q.w};
        bool in[4], any = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float t = sm.place(l[j]);
            in[j] = t >= t0 && t <= t1;
            any |= in[j];
        }
        if (any) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in[j] && l[j] > minus_inf()) {
                    const uint32_t at = atomicAdd(&r.sh->own_count, 1u);
                    if (at < kList) own[at] = entry_of(l[j], r.lo + i + j);
                }
        }
    }
    __syncthreads();
    const uint32_t count = r.sh->own_count;
    uint32_t* row_count = r.cl.map_shared_rank(&r.sh->list_count[which], 0);
    if (r.tid == 0) r.sh->list_base = count ? atomicAdd(row_count, count) : 0;
    __syncthreads();
    uint64_t* list = r.cl.map_shared_rank(own + kList, 0);
    const uint32_t base = r.sh->list_base;
    for (uint32_t i = r.tid; i < min(count, (uint32_t)kList) && base + i < kList; i += kSaThreads) list[base + i] = own[i];
    r.cl.sync();
    return *row_count;
}

__device__ __forceinline__ int pow2_at_least(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

// Sort n entries (a power of two up to kSaThreads), falling: thread t holds entry
// t of the order.  Bitonic; neighbours of a warp exchange by shuffles, the others
// through `buf` (2 x kSaThreads words, used in turn).
__device__ void sort_falling(uint64_t& v, uint64_t* buf, int n, int tid) {
    int turn = 0;
    for (int size = 2; size <= n; size <<= 1)
        for (int step = size >> 1; step > 0; step >>= 1) {
            uint64_t* b = buf + turn * kSaThreads;
            if (step >= 32) {
                b[tid] = v;
                __syncthreads();
                turn ^= 1;
            }
            const uint64_t y = step >= 32 ? b[tid ^ step] : __shfl_xor_sync(0xffffffffu, v, step);
            const bool larger = ((tid & size) == 0) == ((tid & step) == 0);   // this place keeps the larger one
            v = (v > y) == larger ? v : y;
        }
}

// Bring n entries (list[0 .. n), at most kSaThreads, in any order) into falling
// order of the entries, or of the entries with their halves exchanged (rising
// index), with run[i] the mass up to and with entry i.  By one block; list and run
// are the two halves of its scratch.
template <bool BY_INDEX>
__device__ void order_by_sort(Row& r, const Softmax& sm, uint64_t* list, uint64_t* run, int n) {
    const int i = r.tid;
    uint64_t v = i < n ? list[i] : 0;
    if (BY_INDEX) v = (v << 32) | (v >> 32);
    __syncthreads();   // the list is in registers: its place serves the sort
    sort_falling(v, run, pow2_at_least(n), i);
    __syncthreads();
    if (BY_INDEX) v = (v << 32) | (v >> 32);
    uint64_t total;
    const uint64_t inc = r.block_scan(i < n ? sm.mass(entry_logit(v)) : 0, total);
    if (i < n) {
        list[i] = v;
        run[i] = inc;
    }
    __syncthreads();
}

// The same for at most kCounted entries, by counting: `parts` neighbouring
// threads per entry add up what precedes it.  (The sort's 28 steps for 128
// entries took 3 us.)
constexpr int kCounted = 128;

template <bool BY_INDEX>
__device__ __noinline__ void order_by_count(Row& r, const Softmax& sm, uint64_t* list, uint64_t* run, int n) {
    uint64_t* order = run + 512;      // what the entries are ordered by, and their masses
    uint64_t* mass = run + 1024;
    const int parts = min(32, kSaThreads / pow2_at_least(n));
    const int i = r.tid / parts, part = r.tid % parts;
    uint64_t e = 0, mine = 0, m = 0;
    if (i < n) {
        e = list[i];
        mine = BY_INDEX ? (e << 32) | (e >> 32) : e;
        m = sm.mass(entry_logit(e));
        if (part == 0) {
            order[i] = mine;
            mass[i] = m;
        }
    }
    __syncthreads();
    uint64_t before = 0;
    int place = 0;
    if (i < n) {
#pragma unroll 4
        for (int j = part; j < n; j += parts) {
            const bool over = order[j] > mine;
            before += over ? mass[j] : 0;
            place += over;
        }
    }
    for (int o = parts >> 1; o >= 1; o >>= 1) {
        place += __shfl_xor_sync(0xffffffffu, place, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (i < n && part == 0) {         // every entry of the list has been read
        list[place] = e;
        run[place] = before + m;
    }
    __syncthreads();
}

template <bool BY_INDEX>
__device__ __forceinline__ void order_list(Row& r, const Softmax& sm, uint64_t* list, uint64_t* run, int n) {
    if (n <= kCounted)
        order_by_count<BY_INDEX>(r, sm, list, run, n);
    else
        order_by_sort<BY_INDEX>(r, sm, list, run, n);
}

// In a longer list no order is formed.  Among the entries e[0 .. n) that are at
// least `least`, in falling order: the one at which the running value (their
// masses, or with COUNT their number) reaches `need`, at most the sum of all.  By
// one block; e and mass lie in its shared memory.  Each round spreads the range
// that is left over 512 bins, until one holds at most 32 entries (they are
// distinct).
template <bool COUNT>
__device__ __noinline__ uint64_t select_entry(Row& r, const uint64_t* e, const uint64_t* mass, int n, uint64_t least,
                                              uint64_t need) {
    uint64_t* bins = reinterpret_cast<uint64_t*>(r.hist);
    uint32_t* counts = r.hist + 2 * kSaThreads;
    uint64_t* few = r.sh->gather[0][0];   // up to 32 entries, then their values
    uint64_t lo = least, hi = ~(uint64_t)0, above = 0;
    uint32_t left = (uint32_t)n;
    bool ranged = false;
    while (left > 32) {
        if (!ranged) {   // the smallest and largest high words
            uint32_t k0 = 0xffffffffu, k1 = 0;
            for (int i = r.tid; i < n; i += kSaThreads)
                if (e[i] >= least) {
                    k0 = min(k0, (uint32_t)(e[i] >> 32));
                    k1 = max(k1, (uint32_t)(e[i] >> 32));
                }
            k0 = __reduce_min_sync(0xffffffffu, k0);
            k1 = __reduce_max_sync(0xffffffffu, k1);
            __syncthreads();
            if (r.lane == 0) r.sh->warp_sum[r.warp] = ((uint64_t)k1 << 32) | k0;
            __syncthreads();
            const uint64_t w = r.sh->warp_sum[r.lane % kSaWarps];
            lo = max(lo, (uint64_t)__reduce_min_sync(0xffffffffu, (uint32_t)w) << 32);
            hi = ((uint64_t)__reduce_max_sync(0xffffffffu, (uint32_t)(w >> 32)) << 32) | 0xffffffffu;
            ranged = true;
        }
        const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 9);
        bins[r.tid] = 0;
        counts[r.tid] = 0;
        __syncthreads();
        for (int i = r.tid; i < n; i += kSaThreads) {
            const uint64_t x = e[i];
            if (x < lo || x > hi) continue;
            const int b = (int)((hi - x) >> shift);
            atomicAdd(&counts[b], 1u);
            if (!COUNT) atomicAdd((unsigned long long*)&bins[b], (unsigned long long)mass[i]);
        }
        __syncthreads();
        const uint64_t v = COUNT ? counts[r.tid] : bins[r.tid];
        uint64_t all;
        const uint64_t inc = above + r.block_scan(v, all);
        if (inc - v < need && inc >= need) {
            r.sh->found = (uint32_t)r.tid;
            r.sh->found_above = inc - v;
        }
        __syncthreads();
        const uint32_t b = r.sh->found;
        above = r.sh->found_above;
        left = counts[b];
        hi -= (uint64_t)b << shift;
        lo = max(lo, hi - (((uint64_t)1 << shift) - 1));
        __syncthreads();
    }
    if (r.tid == 0) r.sh->own_count = 0;
    __syncthreads();
    for (int i = r.tid; i < n; i += kSaThreads)
        if (e[i] >= lo && e[i] <= hi) {
            const uint32_t at = atomicAdd(&r.sh->own_count, 1u);
            few[at] = e[i];
            few[32 + at] = COUNT ? 1 : mass[i];
        }
    __syncthreads();
    if (r.warp == 0) {
        const int c = (int)r.sh->own_count;
        const uint64_t mine = r.lane < c ? few[r.lane] : 0;
        uint64_t before = above;
#pragma unroll 4
        for (int j = 0; j < c; ++j) before += few[j] > mine ? few[32 + j] : 0;
        if (r.lane < c && before < need && before + few[32 + r.lane] >= need) r.sh->found_entry = mine;
    }
    __syncthreads();
    return r.sh->found_entry;
}

// The masses of the list's n entries, to the first half of the scratch.
__device__ void list_masses(Row& r, const Softmax& sm, const uint64_t* list, uint64_t* mass, int n) {
    for (int i = r.tid; i < n; i += kSaThreads) mass[i] = sm.mass(entry_logit(list[i]));
    __syncthreads();
}

// The mass of the entries that are at least `least`.
__device__ uint64_t mass_from(Row& r, const uint64_t* e, const uint64_t* mass, int n, uint64_t least) {
    uint64_t s = 0;
    for (int i = r.tid; i < n; i += kSaThreads) s += e[i] >= least ? mass[i] : 0;
    return r.block_sum(s);
}

// The whole number that a sum of masses reaches when it reaches `need`, at most `total`.
__device__ __forceinline__ uint64_t whole_need(double need, uint64_t total) {
    return min((uint64_t)fmax(ceil(need), 1.0), total);
}

// The first of n places where `at` holds (it holds from there on), by one warp;
// n if there is none.
template <class Pred>
__device__ __forceinline__ int first_where(int n, int lane, Pred at) {
    int lo = 0, len = n;
    while (len > 0) {
        const int step = (len + 31) / 32, i = min(len, (lane + 1) * step) - 1;
        const uint32_t b = __ballot_sync(0xffffffffu, at(lo + i));
        if (!b) return lo + len;
        const int f = __ffs(b) - 1;
        if (step == 1) return lo + f;
        len = min(step, len - f * step) - 1;   // its last place holds: among the others, or that one
        lo += f * step;
    }
    return lo;
}

__device__ __forceinline__ uint64_t target_of(float u, uint64_t total) {
    const uint64_t t = u > 0.0f ? (uint64_t)floor((double)u * (double)total) : 0;
    return min(t, total - 1);
}

__device__ void choose(const SampleParams& p, const Softmax& sm, int row, int index, float l, uint64_t total) {
    p.token[row] = index;
    if (p.prob) p.prob[row] = (float)(sm.exact(l) * (double)(1ull << kMassBits) / (double)total);
}

// Finish a row whose n tokens in the running are all in the list, by the first
// block alone; every warp follows the steps that are not the whole block's.
// top_p < 1: the prefix reaches `need`, or (top_k > 0) top_p of the mass of the
// first top_k.
__device__ void finish_list(Row& r, const SampleParams& p, const Softmax& sm, int row, int n, int top_k, float top_p,
                            double need, float min_logit) {
    uint64_t* run = reinterpret_cast<uint64_t*>(r.scratch);
    uint64_t* list = run + kList;
    if (n > kSaThreads) {
        uint64_t* mass = run;
        list_masses(r, sm, list, mass, n);
        uint64_t least = 0;
        if (top_k > 0 && top_k < n) least = select_entry<true>(r, list, mass, n, 0, (uint64_t)top_k);
        if (top_p < 1.0f) {
            const uint64_t z = mass_from(r, list, mass, n, least);
            if (top_k > 0) need = (double)top_p * (double)z;
            least = select_entry<false>(r, list, mass, n, least, whole_need(need, z));
        }
        least = max(least, (uint64_t)key_of(min_logit) << 32);
        uint64_t kept = 0;
        for (int i = r.tid; i < n; i += kSaThreads) {
            const uint64_t e = list[i];
            const bool in = e >= least;
            kept += in ? mass[i] : 0;
            list[i] = in ? (e << 32) | (e >> 32) : 0;   // ~index on top: it falls as the index rises
        }
        const uint64_t total = r.block_sum(kept);
        uint64_t e = select_entry<false>(r, list, mass, n, 1, target_of(p.u[row], total) + 1);
        e = (e << 32) | (e >> 32);
        if (r.tid == 0) choose(p, sm, row, entry_index(e), entry_logit(e), total);
        return;
    }
    order_list<false>(r, sm, list, run, n);
    if (top_k > 0) n = min(n, top_k);
    if (top_p < 1.0f) {
        if (top_k > 0) need = fmax((double)top_p * (double)run[n - 1], 1.0);
        n = min(n, first_where(n, r.lane, [&](int i) { return (double)run[i] >= need; }) + 1);
    }
    n = max(1, first_where(n, r.lane, [&](int i) { return entry_logit(list[i]) < min_logit; }));
    const uint64_t total = run[n - 1];
    const uint64_t target = target_of(p.u[row], total);
    __syncthreads();
    order_list<true>(r, sm, list, run, n);
    if (r.warp == 0) {
        const int at = first_where(n, r.lane, [&](int i) { return run[i] > target; });
        if (r.lane == 0) choose(p, sm, row, entry_index(list[at]), entry_logit(list[at]), total);
    }
}

// Of a list of n tokens of one bin, `above` being the mass over it (block_above:
// each block's): the last one of the prefix that reaches `need`, and, if no other
// cut follows, the block that holds the token to choose and what is left of the
// target there.  Written to every block of the cluster.
__device__ void cut_in_list(Row& r, const SampleParams& p, const Softmax& sm, int row, int n, uint64_t above, double need) {
    uint64_t* run = reinterpret_cast<uint64_t*>(r.scratch);
    uint64_t* list = run + kList;
    uint64_t last, total;
    if (n <= kCounted) {
        order_list<false>(r, sm, list, run, n);
        const int at = min(n - 1, first_where(n, r.lane, [&](int i) { return (double)(above + run[i]) >= need; }));
        for (int i = r.tid; i <= at; i += kSaThreads)
            atomicAdd((unsigned long long*)&r.sh->block_above[entry_index(list[i]) / p.per_block],
                      (unsigned long long)(run[i] - (i ? run[i - 1] : 0)));
        last = list[at];
        total = above + run[at];
    } else {
        list_masses(r, sm, list, run, n);
        last = select_entry<false>(r, list, run, n, 0, whole_need(need - (double)above, mass_from(r, list, run, n, 0)));
        uint64_t kept = 0;
        for (int i = r.tid; i < n; i += kSaThreads)
            if (list[i] >= last) {
                kept += run[i];
                atomicAdd((unsigned long long*)&r.sh->block_above[entry_index(list[i]) / p.per_block],
                          (unsigned long long)run[i]);
            }
        total = above + r.block_sum(kept);
    }
    const uint64_t target = target_of(p.u[row], total);
    __syncthreads();
    if (r.tid < r.nb) {
        uint64_t before = 0;
        int b = 0;
        while (b + 1 < r.nb && before + r.sh->block_above[b] <= target) before += r.sh->block_above[b++];
        SaShared* to = r.cl.map_shared_rank(r.sh, r.tid);
        to->cut_value = entry_logit(last);
        to->cut_index = entry_index(last) + 1;
        to->pick_block = b;
        to->pick_target = target - before;
        to->pick_total = total;
    }
}

// ------------------------------------------------------------------ the histogram

// What a block's histogram holds of one bin: its count, or its mass.
template <bool MASS>
__device__ __forceinline__ uint64_t bin_value(const uint32_t* h, int bin) {
    if constexpr (!MASS) return h[bin];
    // sums of mantissas below 2^31 of at most 2^15 tokens, of masses 2^-n
    const uint64_t s = (uint64_t)h[bin] + ((uint64_t)h[kMassBins + bin] << 16);
    return (s << (kMassBits - 30)) >> ((bin + 31) >> 5);
}

// The bin at which the running count (or mass) of the row reaches `need`, and
// what lies above it; kMassBins when it does not.  `own`: this thread's part of
// the mass that is in no bin; `total`: all of it.  need is top_p of it, or given.  Two
// levels, so that a block reads 64 words of each other one's shared memory: the
// sums over powers of two, then the 32 bins of one of them.
template <bool MASS>
__device__ int find_bin(Row& r, uint64_t own, float top_p, double& need, uint64_t& total, uint64_t& above) {
    const uint64_t mine = r.block_sum(own);   // (its barriers complete the histogram)
    for (int g = r.warp; g < 32; g += kSaWarps) {
        const uint64_t s = warp_sum_u64(bin_value<MASS>(r.hist, g * 32 + r.lane));
        if (r.lane == 0) r.sh->coarse[g] = s;
    }
    if (r.tid == 0) r.sh->total = mine;
    r.cl.sync();
    if (r.warp < r.nb) {
        const SaShared* from = r.cl.map_shared_rank(r.sh, r.warp);
        r.sh->gather[0][r.warp][r.lane] = from->coarse[r.lane];
        if (r.lane == 0) r.sh->gather_total[r.warp] = from->total;
    }
    __syncthreads();
    uint64_t s = 0;
    total = 0;
    for (int b = 0; b < r.nb; ++b) {
        s += r.sh->gather[0][b][r.lane];
        total += r.sh->gather_total[b];
    }
    total += warp_sum_u64(s);
    if (MASS) need = fmax((double)top_p * (double)total, 1.0);
    uint64_t inc = warp_scan_u64(s, r.lane);
    uint32_t at = __ballot_sync(0xffffffffu, (double)inc >= need);
    if (!at) return kMassBins;
    const int g = __ffs(at) - 1;
    above = __shfl_sync(0xffffffffu, inc - s, g);
    if (r.warp < r.nb)
        r.sh->gather[1][r.warp][r.lane] = bin_value<MASS>(r.cl.map_shared_rank(r.hist, r.warp), g * 32 + r.lane);
    __syncthreads();
    s = 0;
    for (int b = 0; b < r.nb; ++b) s += r.sh->gather[1][b][r.lane];
    inc = above + warp_scan_u64(s, r.lane);
    at = __ballot_sync(0xffffffffu, (double)inc >= need);
    const int j = __ffs(at) - 1;   // the bins of g add up to its sum: one is found
    above = __shfl_sync(0xffffffffu, inc - s, j);
    if (MASS && r.warp < r.nb) {
        const uint64_t own_above = warp_sum_u64((r.lane < g ? r.sh->gather[0][r.warp][r.lane] : 0) +
                                                (r.lane < j ? r.sh->gather[1][r.warp][r.lane] : 0));
        if (r.lane == 0) r.sh->block_above[r.warp] = own_above;
    }
    return g * 32 + j;
}

// A logit as it is kept: -0 as +0, a NaN or what may not be chosen as -infinity.
__device__ __forceinline__ float clean(float v) { return __fadd_rn(fmaxf(v, minus_inf()), 0.0f); }

__device__ __forceinline__ uint64_t kept_mass(const Row& r, const Softmax& sm, const Cut& cut, int i) {
    const float l = r.logits[i];
    return cut.in(l, r.lo + i) ? sm.mass(l) : 0;
}

// The token of this block at which the running mass of those inside `cut`, in
// their order, exceeds `target` (the last one, should a sum of rounded masses
// fall short of it).
__device__ void pick_in_block(Row& r, const SampleParams& p, const Softmax& sm, int row, const Cut& cut, uint64_t target,
                              uint64_t total) {
    // a lane owns `run` neighbouring tokens, read in turn from a place of its own so
    // that the lanes' reads fall into different banks
    const int run = r.per_warp / 32, l0 = (r.warp * 32 + r.lane) * run;
    uint64_t z = 0;
#pragma unroll 2
    for (int j = 0; j < run; ++j) {
        int o = j + r.lane;
        o -= o >= run ? o / run * run : 0;
        if (l0 + o < r.n) z += kept_mass(r, sm, cut, l0 + o);
    }
    const uint64_t inc = warp_scan_u64(z, r.lane);
    __syncthreads();
    if (r.lane == 31) r.sh->warp_sum[r.warp] = inc;
    __syncthreads();
    const uint64_t s = r.lane < kSaWarps ? r.sh->warp_sum[r.lane] : 0;
    target = min(target, warp_sum_u64(s) - 1);
    const uint64_t at = warp_sum_u64(r.lane < r.warp ? s : 0);
    const uint32_t holds = __ballot_sync(0xffffffffu, at + inc - z <= target && target < at + inc);
    if (!holds) return;
    const int owner = __ffs(holds) - 1;
    uint64_t before = at + __shfl_sync(0xffffffffu, inc - z, owner);
    for (int j0 = 0; j0 < run; j0 += 32) {
        const int i = (r.warp * 32 + owner) * run + j0 + r.lane;
        const uint64_t m = warp_scan_u64(j0 + r.lane < run && i < r.n ? kept_mass(r, sm, cut, i) : 0, r.lane);
        const uint32_t over = __ballot_sync(0xffffffffu, before + m > target);
        if (over) {
            if (r.lane == __ffs(over) - 1) choose(p, sm, row, r.lo + i, r.logits[i], total);
            return;
        }
        before += __shfl_sync(0xffffffffu, m, 31);
    }
}

template <bool VEC>
__global__ void __launch_bounds__(kSaThreads, 2) sample_kernel(const SampleParams p) {
    pdl_trigger();
    extern __shared__ __align__(16) uint32_t sa_smem[];
    __shared__ SaShared shared;
    Row r{cg::this_cluster()};
    r.nb = (int)r.cl.num_blocks();
    r.rank = (int)r.cl.block_rank();
    r.sh = &shared;
    r.scratch = sa_smem;
    r.hist = sa_smem + kScratchWords;
    r.logits = reinterpret_cast<float*>(sa_smem + kScratchWords + kHistWords);
    r.tid = threadIdx.x;
    r.lane = threadIdx.x & 31;
    r.warp = threadIdx.x >> 5;
    r.turn = 0;
    const int row = blockIdx.x / r.nb;
    r.lo = min(p.vocab, r.rank * p.per_block);
    r.n = min(p.vocab, r.lo + p.per_block) - r.lo;
    r.per_warp = p.per_block / kSaWarps;
    if (r.tid < 32) shared.tab[r.tid] = (uint32_t)rint(exp2(30.0 + r.tid / 32.0));
    if (r.tid < 2) shared.list_count[r.tid] = 0;
    for (int i = r.tid; i < kHistWords; i += kSaThreads) r.hist[i] = 0;
    cluster_started();   // this block has started; waited for before the first exchange (max_logit)
    pdl_wait();

    // the row's logits into shared memory
    const int64_t base = (int64_t)row * p.ld + r.lo;
    const uint32_t* allowed = p.allowed ? p.allowed + (int64_t)row * p.ld_allowed : nullptr;
    float own_max = minus_inf();
    if constexpr (VEC) {
#pragma unroll 4
        for (int g = r.tid; g < (r.n + 7) / 8; g += kSaThreads) {
            float v[8];
            if (g * 8 + 8 <= r.n) {
                load8_act(p.logits, base + g * 8, p.dtype, v);
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[c] = g * 8 + c < r.n
                               ? (p.dtype == MOE_BF16
                                      ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p.logits)[base + g * 8 + c])
                                      : reinterpret_cast<const float*>(p.logits)[base + g * 8 + c])
                               : minus_inf();
            }
            if (allowed) {
                const int i0 = r.lo + g * 8;   // a multiple of 8
                const uint32_t bits = allowed[i0 >> 5] >> (i0 & 31);
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = (bits >> c) & 1u ? v[c] : minus_inf();
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                v[c] = clean(v[c]);
                own_max = fmaxf(own_max, v[c]);
            }
            reinterpret_cast<float4*>(r.logits)[2 * g] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(r.logits)[2 * g + 1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll 4
        for (int i = r.tid; i < r.n; i += kSaThreads) {
            const float v = p.dtype == MOE_BF16 ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p.logits)[base + i])
                                                : reinterpret_cast<const float*>(p.logits)[base + i];
            const bool may = !allowed || ((allowed[(r.lo + i) >> 5] >> ((r.lo + i) & 31)) & 1u);
            r.logits[i] = may ? clean(v) : minus_inf();
            own_max = fmaxf(own_max, r.logits[i]);
        }
        if (r.tid < (-r.n & 3)) r.logits[r.n + r.tid] = minus_inf();
    }
    const float given = p.temperature ? p.temperature[row] : 1.0f;
    const float temp = given > 3e38f ? 3e38f : given;   // (a NaN stays one: greedy)
    const int top_k = p.top_k ? p.top_k[row] : 0;
    const float top_p = p.top_p && p.top_p[row] < 1.0f ? p.top_p[row] : 1.0f;   // (a NaN is off)
    const float min_p = p.min_p ? p.min_p[row] : 0.0f;
    float top = r.max_logit(own_max);
    const bool writer = r.rank == 0 && r.tid == 0;
    if (top == minus_inf()) {   // nothing may be chosen
        if (writer) {
            p.token[row] = -1;
            if (p.prob) p.prob[row] = 0.0f;
        }
        r.cl.sync();
        return;
    }
    if (!(temp > kSampleMinTemperature)) {   // greedy: the lowest index among the largest
        const int at = tie_limit(r, Cut{minus_inf(), 0}, top, 0, 0);
        if (writer) {
            p.token[row] = at;
            if (p.prob) p.prob[row] = 1.0f;
        }
        r.cl.sync();
        return;
    }
    if (top == -minus_inf()) {   // infinities share the mass, nothing else has any
        __syncthreads();
        for (int i = r.tid; i < (r.n + 3) / 4 * 4; i += kSaThreads) r.logits[i] = r.logits[i] == top ? 0.0f : minus_inf();
        own_max = own_max == top ? 0.0f : minus_inf();
        top = 0.0f;
        __syncthreads();
    }
    Softmax sm;
    sm.init(top, temp, shared.tab);
    // e >= min_p as a bound on the logit (half a step of 1 in 64 bits counts as equal)
    const float min_logit =
        min_p > 0.0f ? fminf(top, __double2float_ru(sm.m + (double)temp * (log(fmin((double)min_p, 1.0)) - 1.2e-16)))
                     : minus_inf();
    Cut cut{minus_inf(), 0};   // every token that may be chosen

    if (top_k > 0) {
        // a bin that the top_k tokens do not go below: from the threads' largest tokens
        // while these are at least four times as many, else from all tokens
        auto count = [&](float l) {
            const float t = sm.place(l);
            if (t > sm.t_max - (float)kMassBins) atomicAdd(&r.hist[sm.bin(t)], 1u);
        };
        if (top_k <= r.nb * kSaThreads / 4) {
            count(own_max);
        } else {
            for (int i = r.tid; i < r.n; i += kSaThreads) count(r.logits[i]);
        }
        uint64_t total, above;
        double need = (double)top_k;
        const int b = find_bin<false>(r, 0, 1.0f, need, total, above);
        // (tokens below all bins are in the list too when the bins do not reach top_k)
        const float t0 = b < kMassBins ? sm.t_max - (float)b : minus_inf();
        const uint32_t n = make_list(r, sm, t0, sm.t_max, 0);
        if (n <= kList) {
            if (r.rank == 0) finish_list(r, p, sm, row, (int)n, top_k, top_p, 0.0, min_logit);
            r.leave();
            return;
        }
        cut_count(r, sm, cut, top_k, p.vocab);
        if (top_p < 1.0f) {
            uint64_t z = 0, none;
            for (int i = r.tid; i < r.n; i += kSaThreads)
                if (cut.in(r.logits[i], r.lo + i)) z += sm.mass(r.logits[i]);
            total = r.sum(z, none);
            cut_mass(r, sm, cut, fmax((double)top_p * (double)total, 1.0), p.vocab);
        }
    } else if (top_p < 1.0f) {
        // masses of all tokens; those below tail / vocab of the largest mass hold less than
        // tail <= 1 - top_p together, so the prefix ends above them
        const float tail = log2f(fminf(1.0f - top_p, 0.015625f) / (float)p.vocab) - 0.5f;
        const float t_last = sm.t_max - fminf(fmaxf(floorf(-32.0f * tail), 0.0f), (float)(kMassBins - 1));
        float zt = 0.0f;   // the tail's part, less than 1/64 in all, by the approximate 2^x
        const int steps = (r.n + kSaThreads * 4 - 1) / (kSaThreads * 4);
        for (int k = 0; k < steps; ++k) {   // whole warps: the vote below
            const int i = (k * kSaThreads + r.tid) * 4;
            const float4 l = i < r.n ? *reinterpret_cast<const float4*>(r.logits + i)
                                     : make_float4(minus_inf(), minus_inf(), minus_inf(), minus_inf());
            Pair lr[2], at[2];
            sm.place4(l, lr, at);
            float t[4];
            at[0].get(t[0], t[1]);
            at[1].get(t[2], t[3]);
            const float lv[4] = {l.x, l.y, l.z, l.w};
            if (__any_sync(0xffffffffu, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) >= t_last)) {
                uint32_t M[4];
                sm.mantissa4(lr, at, M);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (t[j] >= t_last) {
                        const int bin = sm.bin(t[j]);
                        atomicAdd(&r.hist[bin], M[j] & 0xffffu);
                        atomicAdd(&r.hist[kMassBins + bin], M[j] >> 16);
                    } else {
                        zt += sm.approximate(lv[j]);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) zt += sm.approximate(lv[j]);
            }
        }
        const uint64_t z = (uint64_t)((double)zt * (double)(1ull << kMassBits));
        uint64_t total = 0, above = 0;
        double need = 0.0;
        const int b = find_bin<true>(r, z, top_p, need, total, above);
        if (b >= kMassBins) {
            cut_mass(r, sm, cut, need, p.vocab);   // the prefix ends below the last bin
        } else {
            // every token has at most the largest mass: need / 2^45 tokens at least
            const float t = sm.t_max - (float)b;
            if (need < (double)kList * (double)(1ull << kMassBits)) {
                const uint32_t n = make_list(r, sm, t, sm.t_max, 0);
                if (n <= kList) {
                    if (r.rank == 0) finish_list(r, p, sm, row, (int)n, 0, top_p, need, min_logit);
                    r.leave();
                    return;
                }
            }
            const uint32_t n = make_list(r, sm, t, t, 1);
            if (n <= kList) {
                if (r.rank == 0) cut_in_list(r, p, sm, row, (int)n, above, need);
                r.cl.sync();
                cut = Cut{r.sh->cut_value, r.sh->cut_index};
                if (!(min_logit > cut.K)) {
                    // the histograms tell which block holds the token: the others are done
                    if (r.rank == r.sh->pick_block) pick_in_block(r, p, sm, row, cut, r.sh->pick_target, r.sh->pick_total);
                    return;
                }
            } else {
                cut_mass(r, sm, cut, need, p.vocab);
            }
        }
    }
    if (min_logit > cut.K) cut = Cut{min_logit, p.vocab};
    // the kept mass, by block and cluster
    uint64_t z = 0, before;
#pragma unroll 2
    for (int i = r.tid; i < r.n; i += kSaThreads) z += kept_mass(r, sm, cut, i);
    const uint64_t mine = r.block_sum(z);
    const uint64_t total = r.sum(z, before);
    const uint64_t target = target_of(p.u[row], total);
    if (before <= target && target < before + mine) pick_in_block(r, p, sm, row, cut, target - before, total);
    r.cl.sync();   // no block leaves while another may still write to its slots
}

}  // namespace

cudaError_t launch_sample(const SampleParams& in, cudaStream_t s) {
    SampleParams p = in;
    int nb = 1;
    while (nb < kSaMaxCluster && p.vocab > nb * 8192) nb *= 2;
    const int unit = kSaWarps * 32;
    p.per_block = ((p.vocab + nb - 1) / nb + unit - 1) / unit * unit;
    constexpr int kFixed = kScratchWords + kHistWords;
    const size_t smem = (size_t)(kFixed + p.per_block) * 4;
    const size_t esz = p.dtype == MOE_BF16 ? 2 : 4;
    const bool vec = ((uintptr_t)p.logits & 15) == 0 && (p.ld * (int64_t)esz) % 16 == 0;
    static std::atomic<uint64_t> attr[2];
    auto kern = vec ? sample_kernel<true> : sample_kernel<false>;
    cudaError_t e = smem_attr_once(kern, (size_t)(kFixed + kSampleMaxVocab / kSaMaxCluster) * 4, attr[vec]);
    if (e != cudaSuccess) return e;
    return launch_cluster(kern, dim3((unsigned)(p.rows * nb)), dim3(kSaThreads), nb, smem, s, p);
}

}  // namespace moe
