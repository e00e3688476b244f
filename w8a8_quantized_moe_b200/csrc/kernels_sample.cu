// The next token of each row of logits, from given random numbers.
//
// Per row: the tokens in order of falling logit (lowest index first on ties,
// the router's own rule); the first top_k of them; of those the shortest
// prefix that holds top_p of their mass, with masses e_i = exp((l_i - max) /
// temperature); of those the ones with e_i >= min_p; and then, in the order of
// the tokens, the first whose running mass exceeds u times the kept mass.
//
// Masses are held as integers in units of 2^-45 of the largest one (one unit at
// least: u = 0 is the first token that takes part), so sums do not depend on
// the order of the atomics and every comparison is exact.
//
// A row belongs to a cluster of thread blocks that keep it in their shared
// memory: the logits are read from memory once, the later passes read shared
// memory, and the blocks exchange histograms, sums and lists over distributed
// shared memory.  The whole row is never sorted:
//   - Tokens fall into bins of 1/32 of a power of two of mass.  A histogram (of
//     the threads' largest tokens, which bounds the top_k from below, or of all
//     tokens that the top_p could reach, with their masses) names the bin where
//     a prefix ends.
//   - If the tokens down to that bin are few, the first block of the cluster
//     gets them as a list, sorts it and finishes the row alone.
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
constexpr uint32_t kNone = 0x007fffffu;   // ordered key of -infinity: a token that may not be chosen
constexpr int kList = 2048;               // tokens of a list
constexpr int kMassBins = 1024;           // bins of 1/32 of a power of two, the last one open
constexpr int kKeyBins = 2048;            // bins of the selection by key bits
// scratch of a block: the histograms (3 x kKeyBins words, or counts, low and high
// sums of kMassBins), or a list of its own tokens and, in the first block, the row's
constexpr int kScratchWords = 2 * 2 * kList;
static_assert(kScratchWords >= 3 * kKeyBins && kScratchWords >= 3 * kMassBins, "scratch");

// Keys order like the logits: the sign bit set for values >= 0, all bits
// inverted below.  -0 becomes +0, a NaN counts as -infinity.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (!(v == v)) return kNone;
    const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// Masses 2^x, x = (l - max) log2(e) / temperature.  x is formed in two fp32
// parts (the difference and the product each with its rounding error), x = k /
// 32 + r, and 2^x = 2^(k >> 5) T[k & 31] (1 + q) with a table of 2^(j / 32) in
// 32 bits and q = e^(r ln 2) - 1 by its Taylor polynomial to degree 4 (|r ln 2|
// < 0.011, remainder 2e-12): within 2e-9 of the true value, in integer and fp32
// instructions alone.  (In fp64, with a polynomial of degree 9, a pass over 256
// x 131072 tokens took several times as long.)
struct Softmax {
    uint32_t kmax;
    float m, c, c_lo;
    double cd;
    const uint32_t* tab;   // shared: round(2^(31 + j / 32))
    __device__ __forceinline__ void init(uint32_t key_max, float temperature, const uint32_t* table) {
        kmax = key_max;
        m = value_of(key_max);
        cd = 1.4426950408889634074 / (double)temperature;
        c = (float)fmin(cd, 3e38);
        c_lo = (float)(fmin(cd, 3e38) - (double)c);
        tab = table;
    }
    // k and the 32-bit mantissa M (in units of 2^-31): mass M 2^(k >> 5); false
    // below 2^-1000.
    __device__ __forceinline__ bool parts(uint32_t key, int& k, uint32_t& M) const {
        const float l = value_of(key);
        const float s = __fsub_rn(l, m), b = __fsub_rn(s, l);
        const float err = __fadd_rn(__fsub_rn(l, __fsub_rn(s, b)), __fsub_rn(-m, b));
        const float xh = __fmul_rn(s, c);
        if (key == kmax) {
            k = 0;
            M = 1u << 31;
            return true;
        }
        if (!(xh > -1000.0f)) return false;
        const float xl = __fadd_rn(__fmaf_rn(s, c, -xh), __fmaf_rn(s, c_lo, __fmul_rn(err, c)));
        const float t = __fmaf_rn(xh, 32.0f, 12582912.0f);   // 1.5 x 2^23: rounds to an integer in the low bits
        k = __float_as_int(t) - 0x4b400000;
        const float r = __fadd_rn(__fmaf_rn(__fsub_rn(t, 12582912.0f), -0.03125f, xh), xl);
        const float y = __fmul_rn(r, 0.693147180559945f);
        float p = __fmaf_rn(y, 1.0f / 24, 1.0f / 6);
        p = __fmaf_rn(p, y, 0.5f);
        p = __fmaf_rn(__fmul_rn(p, y), y, y);
        const uint32_t T = tab[k & 31];
        const int q = __float2int_rn(__fmul_rn(p, 4294967296.0f));
        M = T + (uint32_t)(((int64_t)(uint64_t)T * q) >> 32);
        return true;
    }
    static __device__ __forceinline__ uint64_t fixed(int k, uint32_t M) {
        const int n = -(k >> 5);
        const uint64_t v = n < 64 ? ((uint64_t)M << (kMassBits - 31)) >> n : 0;
        return v ? v : 1;
    }
    __device__ __forceinline__ uint64_t mass(uint32_t key) const {
        int k;
        uint32_t M;
        return parts(key, k, M) ? fixed(k, M) : 0;
    }
    // the bin of a token: tokens of a lower bin have a larger logit
    __device__ __forceinline__ int bin(uint32_t key) const {
        if (key == kmax) return 0;
        const float xh = __fmul_rn(__fsub_rn(value_of(key), m), c);
        if (!(xh > -1000.0f)) return kMassBins - 1;
        const int k = __float_as_int(__fmaf_rn(xh, 32.0f, 12582912.0f)) - 0x4b400000;
        return min(-k, kMassBins - 1);
    }
    // the mass in 64 bits, for the chosen token's probability
    __device__ __forceinline__ double exact(uint32_t key) const {
        if (key == kmax) return 1.0;
        return exp2(((double)value_of(key) - (double)m) * cd);
    }
};

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
    uint64_t slots[2][kSaMaxCluster];   // per reduction, alternating: one value per block
    uint64_t warp_sum[kSaWarps];
    uint64_t found_above, found_need;
    uint32_t found, cut_key;
    int32_t cut_index;
    uint32_t list_base, list_count;     // list_count: of the row, in the first block
    uint32_t own_count;
    uint32_t tab[32];
};

// The tokens still in the running: key above K, or equal to K and below index I.
struct Cut {
    uint32_t K;
    int I;
    __device__ __forceinline__ bool in(uint32_t key, int index) const { return key > K || (key == K && index < I); }
};

// One row of a cluster.
struct Row {
    cg::cluster_group cl;
    int nb, rank;                // blocks of the cluster, this one
    SaShared* sh;
    uint32_t* keys;              // this block's tokens [lo, lo + n), kNone up to a multiple of 4
    uint32_t* scratch;
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
    __device__ uint32_t max_key(uint32_t k) {
        k = __reduce_max_sync(0xffffffffu, k);
        if (lane == 0) sh->warp_sum[warp] = k;
        __syncthreads();
        if (warp == 0) {
            k = __reduce_max_sync(0xffffffffu, lane < kSaWarps ? (uint32_t)sh->warp_sum[lane] : 0u);
            if (lane < nb) *cl.map_shared_rank(&sh->slots[turn][rank], lane) = k;
        }
        cl.sync();
        k = 0;
        for (int i = 0; i < nb; ++i) k = max(k, (uint32_t)sh->slots[turn][i]);
        turn ^= 1;
        return k;
    }
    // A block's last step: the others leave, the first one when none of them
    // reads its shared memory any more.
    __device__ void leave() {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        if (rank == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    // Inclusive scan of v over the threads of the block.
    __device__ uint64_t block_scan(uint64_t v) {
        v = warp_scan_u64(v, lane);
        __syncthreads();
        if (lane == 31) sh->warp_sum[warp] = v;
        __syncthreads();
        for (int w = 0; w < warp; ++w) v += sh->warp_sum[w];
        return v;
    }
};

// ------------------------------------------------------------------ selection by key bits

// Among the tokens inside `cut`, in order of falling key: the key at which the
// running count (or mass) reaches `need`, and how much lies strictly above it.
// False when the whole set does not reach it.
template <bool MASS>
__device__ __noinline__ bool select_key(Row& r, const Softmax& sm, const Cut& cut, double need, uint32_t& key_out,
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
            const uint32_t k = r.keys[i];
            if ((k & mask) != prefix || !cut.in(k, r.lo + i)) continue;
            const int bin = (k >> shift) & (bins - 1);
            if constexpr (MASS) {
                // 15 bits at a time: 2^15 tokens of a block cannot overflow a sum
                const uint64_t m = sm.mass(k);
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
        uint64_t before = above + r.block_scan(mine) - mine;
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
    key_out = prefix;
    above_out = above;
    return true;
}

// The index of the tie number `keep` (from 0, in the order of the tokens) among
// the tokens inside `cut` whose key is K: the first one left out; `none` when
// there are not that many.
__device__ __noinline__ int tie_limit(Row& r, const Cut& cut, uint32_t K, uint64_t keep, int none) {
    const int w0 = r.warp * r.per_warp, w1 = min(r.n, w0 + r.per_warp);
    uint32_t c = 0;
    for (int i = w0 + r.lane; i < w1; i += 32) c += r.keys[i] == K && cut.in(K, r.lo + i);
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
            const bool is = i < w1 && r.keys[i] == K && cut.in(K, r.lo + i);
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
    uint32_t K = 0;
    uint64_t above = 0;
    if (!select_key<false>(r, sm, cut, (double)top_k, K, above)) return;
    cut = Cut{K, tie_limit(r, cut, K, (uint64_t)top_k - above, vocab)};
}

// The shortest prefix of the tokens inside `cut` whose mass reaches `need`, by key bits.
__device__ __noinline__ void cut_mass(Row& r, const Softmax& sm, Cut& cut, double need, int vocab) {
    uint32_t K = 0;
    uint64_t above = 0;
    if (!select_key<true>(r, sm, cut, need, K, above)) return;
    const uint64_t ties = (uint64_t)fmax(1.0, ceil((need - (double)above) / (double)sm.mass(K)));
    const int I = tie_limit(r, cut, K, ties, vocab);
    cut = Cut{K, K == cut.K ? min(I, cut.I) : I};
}

// ------------------------------------------------------------------ lists

// Entries order by falling logit, then rising index.
__device__ __forceinline__ uint64_t entry_of(uint32_t key, int index) { return ((uint64_t)key << 32) | (uint32_t)~index; }
__device__ __forceinline__ uint32_t entry_key(uint64_t e) { return (uint32_t)(e >> 32); }
__device__ __forceinline__ int entry_index(uint64_t e) { return (int)~(uint32_t)e; }

// The row's tokens of bins [b0, b1] as a list in the first block's scratch
// (second half).  Returns how many there are; more than kList: the list is
// incomplete.  Every block calls it; `list_count` was cleared before the last
// cluster barrier.
__device__ uint32_t make_list(Row& r, const Softmax& sm, int b0, int b1) {
    uint64_t* own = reinterpret_cast<uint64_t*>(r.scratch);
    if (r.tid == 0) r.sh->own_count = 0;
    __syncthreads();
    for (int i = r.tid * 4; i < r.n; i += kSaThreads * 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(r.keys + i);
        const uint32_t k[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (k[j] <= kNone) continue;
            const int b = sm.bin(k[j]);
            if (b < b0 || b > b1) continue;
            const uint32_t at = atomicAdd(&r.sh->own_count, 1u);
            if (at < kList) own[at] = entry_of(k[j], r.lo + i + j);
        }
    }
    __syncthreads();
    const uint32_t count = r.sh->own_count;
    uint32_t* row_count = r.cl.map_shared_rank(&r.sh->list_count, 0);
    if (r.tid == 0) r.sh->list_base = count ? atomicAdd(row_count, count) : 0;
    __syncthreads();
    uint64_t* list = r.cl.map_shared_rank(own + kList, 0);
    const uint32_t base = r.sh->list_base;
    for (uint32_t i = r.tid; i < min(count, (uint32_t)kList) && base + i < kList; i += kSaThreads) list[base + i] = own[i];
    r.cl.sync();
    return *row_count;
}

// Sort n entries (a power of two), falling, by the threads of one block.
__device__ void sort_falling(uint64_t* a, int n, int tid) {
    for (int size = 2; size <= n; size <<= 1)
        for (int step = size >> 1; step > 0; step >>= 1) {
            __syncthreads();
            for (int t = tid; t < n / 2; t += kSaThreads) {
                const int i = ((t & -step) << 1) | (t & (step - 1)), j = i + step;
                const bool falling = (i & size) == 0;
                const uint64_t x = a[i], y = a[j];
                if ((x < y) == falling) {
                    a[i] = y;
                    a[j] = x;
                }
            }
        }
    __syncthreads();
}

__device__ int pow2_at_least(int n) { return n <= 2 ? 2 : 1 << (32 - __clz(n - 1)); }

// Sort the row's list of `count` entries; the first block only.
__device__ uint64_t* sorted_list(Row& r, int count) {
    uint64_t* list = reinterpret_cast<uint64_t*>(r.scratch) + kList;
    const int n = pow2_at_least(count);
    for (int i = count + r.tid; i < n; i += kSaThreads) list[i] = 0;
    sort_falling(list, n, r.tid);
    return list;
}

// Of the list's first `count` entries, in order: the running mass (plus
// `above`) after entry i to run[i].  The first block only.
__device__ void running_mass(Row& r, const Softmax& sm, const uint64_t* list, int count, uint64_t above, uint64_t* run) {
    constexpr int kPer = kList / kSaThreads;
    uint64_t v[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = r.tid * kPer + j;
        v[j] = i < count ? sm.mass(entry_key(list[i])) : 0;
        mine += v[j];
    }
    uint64_t at = above + r.block_scan(mine) - mine;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        at += v[j];
        if (r.tid * kPer + j < count) run[r.tid * kPer + j] = at;
    }
    __syncthreads();
}

// Number of entries whose running mass, without themselves, is below `need`
// (at least one).  The first block only.
__device__ int prefix_reaching(Row& r, const uint64_t* run, int count, double need) {
    if (r.tid == 0) r.sh->found = count;
    __syncthreads();
    for (int i = r.tid; i < count; i += kSaThreads)
        if ((double)run[i] >= need) atomicMin(&r.sh->found, (uint32_t)(i + 1));
    __syncthreads();
    return (int)r.sh->found;
}

__device__ __forceinline__ uint64_t target_of(float u, uint64_t total) {
    const uint64_t t = u > 0.0f ? (uint64_t)floor((double)u * (double)total) : 0;
    return min(t, total - 1);
}

__device__ void choose(const SampleParams& p, const Softmax& sm, int row, int index, uint32_t key, uint64_t total) {
    p.token[row] = index;
    if (p.prob) p.prob[row] = (float)(sm.exact(key) * (double)(1ull << kMassBits) / (double)total);
}

// Finish a row whose tokens in the running are all in the list, by the first block alone.
__device__ void finish_list(Row& r, const SampleParams& p, const Softmax& sm, int row, int count, int top_k, float top_p,
                            double min_mass) {
    uint64_t* list = sorted_list(r, count);
    uint64_t* run = reinterpret_cast<uint64_t*>(r.scratch);
    int n = top_k > 0 ? min(count, top_k) : count;
    running_mass(r, sm, list, n, 0, run);
    // need: given, or (by the list alone) top_p of its mass
    if (top_p < 1.0f) {
        const double need = top_k > 0 ? fmax((double)top_p * (double)run[n - 1], 1.0) : __longlong_as_double(r.sh->found_need);
        n = prefix_reaching(r, run, n, need);
    }
    if (min_mass > 0.0) {
        if (r.tid == 0) r.sh->found = n;
        __syncthreads();
        for (int i = r.tid; i < n; i += kSaThreads)
            if ((double)sm.mass(entry_key(list[i])) < min_mass) atomicMin(&r.sh->found, (uint32_t)i);
        __syncthreads();
        n = max(1, (int)r.sh->found);
    }
    const uint64_t total = run[n - 1];
    const uint64_t target = target_of(p.u[row], total);
    // in the order of the tokens: entries with the index on top, sorted again
    __syncthreads();
    const int m = pow2_at_least(n);
    for (int i = r.tid; i < m; i += kSaThreads) {
        const uint64_t e = list[i];
        list[i] = i < n ? (e << 32) | (e >> 32) : 0;   // ~index falls as the index rises
    }
    sort_falling(list, m, r.tid);
    for (int i = r.tid; i < n; i += kSaThreads) list[i] = (list[i] << 32) | (list[i] >> 32);
    __syncthreads();
    running_mass(r, sm, list, n, 0, run);
    for (int i = r.tid; i < n; i += kSaThreads)
        if (run[i] > target && (i == 0 || run[i - 1] <= target))
            choose(p, sm, row, entry_index(list[i]), entry_key(list[i]), total);
}

// ------------------------------------------------------------------ the histogram of masses

// The first bin at which the running count (or mass) of the row's histogram
// reaches `need`, what lies above it, or kMassBins when it does not.  All
// blocks; the histograms are complete (a cluster barrier has passed).
template <bool MASS>
__device__ int find_bin(Row& r, double need, uint64_t& above) {
    constexpr int kPer = kMassBins / kSaThreads;
    uint64_t v[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int bin = r.tid * kPer + j;
        uint64_t s = 0;
        for (int b = 0; b < r.nb; ++b) {
            const uint32_t* h = r.cl.map_shared_rank(r.scratch, b);
            s += h[bin];
            if constexpr (MASS) s += (uint64_t)h[kMassBins + bin] << 16;
        }
        if constexpr (MASS) {
            // sums of mantissas of masses 2^-n: at most 2^50, or 2^49 where n = 0
            const int n = (bin + 31) >> 5;
            s = (s << (kMassBits - 31)) >> n;
        }
        v[j] = s;
        mine += s;
    }
    if (r.tid == 0) r.sh->found = kMassBins;
    uint64_t before = r.block_scan(mine) - mine;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if ((double)before < need && (double)(before + v[j]) >= need) {
            r.sh->found = (uint32_t)(r.tid * kPer + j);
            r.sh->found_above = before;
        }
        before += v[j];
    }
    __syncthreads();
    above = r.sh->found_above;
    return (int)r.sh->found;
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
    r.keys = sa_smem + kScratchWords;
    r.tid = threadIdx.x;
    r.lane = threadIdx.x & 31;
    r.warp = threadIdx.x >> 5;
    r.turn = 0;
    const int row = blockIdx.x / r.nb;
    r.lo = min(p.vocab, r.rank * p.per_block);
    r.n = min(p.vocab, r.lo + p.per_block) - r.lo;
    r.per_warp = p.per_block / kSaWarps;
    if (r.tid < 32) shared.tab[r.tid] = (uint32_t)rint(exp2(31.0 + r.tid / 32.0));
    if (r.tid == 0) shared.list_count = 0;
    for (int i = r.tid; i < 3 * kMassBins; i += kSaThreads) r.scratch[i] = 0;
    pdl_wait();

    // the row's logits, as keys, into shared memory
    const int64_t base = (int64_t)row * p.ld + r.lo;
    const uint32_t* allowed = p.allowed ? p.allowed + (int64_t)row * p.ld_allowed : nullptr;
    uint32_t own_max = 0;
    if constexpr (VEC) {
#pragma unroll 4
        for (int g = r.tid; g < (r.n + 7) / 8; g += kSaThreads) {
            uint32_t k[8];
            if (g * 8 + 8 <= r.n) {
                float v[8];
                load8_act(p.logits, base + g * 8, p.dtype, v);
#pragma unroll
                for (int c = 0; c < 8; ++c) k[c] = key_of(v[c]);
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    k[c] = g * 8 + c < r.n
                               ? key_of(p.dtype == MOE_BF16
                                            ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p.logits)[base + g * 8 + c])
                                            : reinterpret_cast<const float*>(p.logits)[base + g * 8 + c])
                               : kNone;
            }
            const int i0 = r.lo + g * 8;   // a multiple of 8
            const uint32_t bits = allowed ? allowed[i0 >> 5] >> (i0 & 31) : 0xffu;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                k[c] = (bits >> c) & 1u ? k[c] : kNone;
                own_max = max(own_max, k[c]);
            }
            reinterpret_cast<uint4*>(r.keys)[2 * g] = make_uint4(k[0], k[1], k[2], k[3]);
            reinterpret_cast<uint4*>(r.keys)[2 * g + 1] = make_uint4(k[4], k[5], k[6], k[7]);
        }
    } else {
#pragma unroll 4
        for (int i = r.tid; i < r.n; i += kSaThreads) {
            uint32_t k = key_of(p.dtype == MOE_BF16 ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p.logits)[base + i])
                                                    : reinterpret_cast<const float*>(p.logits)[base + i]);
            if (allowed && !((allowed[(r.lo + i) >> 5] >> ((r.lo + i) & 31)) & 1u)) k = kNone;
            r.keys[i] = k;
            own_max = max(own_max, k);
        }
        if (r.tid < (-r.n & 3)) r.keys[r.n + r.tid] = kNone;
    }
    const float temp = p.temperature ? p.temperature[row] : 1.0f;
    const int top_k = p.top_k ? p.top_k[row] : 0;
    const float top_p = p.top_p ? p.top_p[row] : 1.0f;
    const float mp = p.min_p ? p.min_p[row] : 0.0f;
    const uint32_t kmax = r.max_key(own_max);
    const bool writer = r.rank == 0 && r.tid == 0;
    if (kmax <= kNone) {   // nothing may be chosen
        if (writer) {
            p.token[row] = -1;
            if (p.prob) p.prob[row] = 0.0f;
        }
        r.cl.sync();
        return;
    }
    if (!(temp > 0.0f)) {   // greedy: the lowest index among the largest
        const int at = tie_limit(r, Cut{kNone, 0}, kmax, 0, 0);
        if (writer) {
            p.token[row] = at;
            if (p.prob) p.prob[row] = 1.0f;
        }
        r.cl.sync();
        return;
    }
    Softmax sm;
    sm.init(kmax, temp, shared.tab);
    const double min_mass = mp > 0.0f ? fmin((double)mp, 1.0) * (double)(1ull << kMassBits) : 0.0;
    Cut cut{kNone, 0};   // every token that may be chosen
    uint32_t* hist = r.scratch;
    bool cut_p = top_p < 1.0f;

    if (top_k > 0) {
        // a bin that the top_k tokens do not go below: from the threads' largest tokens
        // while these are at least four times as many, else from all tokens
        const bool by_thread = top_k <= r.nb * kSaThreads / 4;
        if (by_thread) {
            if (own_max > kNone) atomicAdd(&hist[sm.bin(own_max)], 1u);
        } else {
            for (int i = r.tid; i < r.n; i += kSaThreads)
                if (r.keys[i] > kNone) atomicAdd(&hist[sm.bin(r.keys[i])], 1u);
        }
        r.cl.sync();
        uint64_t above;
        const int b = min(find_bin<false>(r, (double)top_k, above), kMassBins - 1);
        r.cl.sync();   // the histograms have been read: the scratch is free
        const uint32_t count = make_list(r, sm, 0, b);
        if (count <= kList) {
            if (r.rank == 0) finish_list(r, p, sm, row, (int)count, top_k, top_p, min_mass);
            r.leave();
            return;
        }
        cut_count(r, sm, cut, top_k, p.vocab);
        if (cut_p) {
            uint64_t z = 0, none;
            for (int i = r.tid; i < r.n; i += kSaThreads)
                if (cut.in(r.keys[i], r.lo + i)) z += sm.mass(r.keys[i]);
            const uint64_t total = r.sum(z, none);
            cut_mass(r, sm, cut, fmax((double)top_p * (double)total, 1.0), p.vocab);
        }
    } else if (cut_p) {
        // masses of all tokens; those below (1 - top_p) / vocab of the largest mass hold
        // less than 1 - top_p together, so the prefix ends above them
        const float tail = log2f((1.0f - top_p) / (float)p.vocab) - 0.5f;
        const int last = tail > -31.0f ? (int)(-32.0f * tail) : kMassBins - 1;
        uint64_t z = 0, none;
        for (int i = r.tid * 4; i < r.n; i += kSaThreads * 4) {
            const uint4 q = *reinterpret_cast<const uint4*>(r.keys + i);
            const uint32_t key[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                int k;
                uint32_t M;
                if (key[j] <= kNone || !sm.parts(key[j], k, M)) continue;
                z += Softmax::fixed(k, M);
                if (-k <= last && -k < kMassBins - 1) {
                    atomicAdd(&hist[-k], M & 0xffffu);
                    atomicAdd(&hist[kMassBins - k], M >> 16);
                }
            }
        }
        const uint64_t total = r.sum(z, none);
        const double need = fmax((double)top_p * (double)total, 1.0);
        uint64_t above = 0;
        const int b = find_bin<true>(r, need, above);
        r.cl.sync();   // the histograms have been read: the scratch is free
        if (b >= kMassBins) {
            cut_mass(r, sm, cut, need, p.vocab);   // the prefix ends below the last bin
        } else {
            // every token has at most the largest mass: need / 2^45 tokens at least
            if (need < (double)kList * (double)(1ull << kMassBits)) {
                const uint32_t count = make_list(r, sm, 0, b);
                if (count <= kList) {
                    if (r.rank == 0) {
                        if (r.tid == 0) r.sh->found_need = (uint64_t)__double_as_longlong(need);
                        finish_list(r, p, sm, row, (int)count, 0, top_p, min_mass);
                    }
                    r.leave();
                    return;
                }
                r.cl.sync();
                if (writer) r.sh->list_count = 0;
                r.cl.sync();
            }
            const uint32_t count = make_list(r, sm, b, b);
            if (count <= kList) {
                if (r.rank == 0) {
                    uint64_t* run = reinterpret_cast<uint64_t*>(r.scratch);
                    const uint64_t* list = sorted_list(r, (int)count);
                    running_mass(r, sm, list, (int)count, above, run);
                    const int n = prefix_reaching(r, run, (int)count, need);
                    if (r.tid < r.nb) {
                        SaShared* to = r.cl.map_shared_rank(r.sh, r.tid);
                        to->cut_key = entry_key(list[n - 1]);
                        to->cut_index = entry_index(list[n - 1]) + 1;
                    }
                }
                r.cl.sync();
                cut = Cut{r.sh->cut_key, r.sh->cut_index};
            } else {
                cut_mass(r, sm, cut, need, p.vocab);
            }
        }
    }
    // the kept mass, by warp (the tokens of a warp are neighbours), block and cluster
    const int w0 = r.warp * r.per_warp, w1 = min(r.n, w0 + r.per_warp);
    auto kept = [&](int i) -> uint64_t {
        const uint32_t k = r.keys[i];
        if (!cut.in(k, r.lo + i)) return 0;
        const uint64_t m = sm.mass(k);
        return (double)m < min_mass ? 0 : m;
    };
    uint64_t z = 0, before;
    for (int i = w0 + r.lane; i < w1; i += 32) z += kept(i);
    const uint64_t mine = warp_sum_u64(z);
    const uint64_t total = r.sum(z, before);
    const uint64_t target = target_of(p.u[row], total);
    __syncthreads();
    if (r.lane == 0) r.sh->warp_sum[r.warp] = mine;
    __syncthreads();
    for (int w = 0; w < r.warp; ++w) before += r.sh->warp_sum[w];
    if (before <= target && target < before + mine) {
        uint64_t at = before;
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const int i = i0 + r.lane;
            const uint64_t m = i < w1 ? kept(i) : 0;
            const uint64_t inc = at + warp_scan_u64(m, r.lane);
            const uint32_t over = __ballot_sync(0xffffffffu, inc > target);
            if (over) {
                if (r.lane == __ffs(over) - 1) choose(p, sm, row, r.lo + i, r.keys[i], total);
                break;
            }
            at = __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    r.cl.sync();   // no block leaves while another may still write to its slots
}

}  // namespace

cudaError_t launch_sample(const SampleParams& in, cudaStream_t s) {
    SampleParams p = in;
    int nb = 1;
    while (nb < kSaMaxCluster && p.vocab > nb * 8192) nb *= 2;
    const int unit = kSaWarps * 32;
    p.per_block = ((p.vocab + nb - 1) / nb + unit - 1) / unit * unit;
    const size_t smem = (size_t)(kScratchWords + p.per_block) * 4;
    const size_t esz = p.dtype == MOE_BF16 ? 2 : 4;
    const bool vec = ((uintptr_t)p.logits & 15) == 0 && (p.ld * (int64_t)esz) % 16 == 0;
    static std::atomic<uint64_t> attr[2];
    auto kern = vec ? sample_kernel<true> : sample_kernel<false>;
    cudaError_t e = smem_attr_once(kern, (size_t)(kScratchWords + kSampleMaxVocab / kSaMaxCluster) * 4, attr[vec]);
    if (e != cudaSuccess) return e;
    return launch_cluster(kern, dim3((unsigned)(p.rows * nb)), dim3(kSaThreads), nb, smem, s, p);
}

}  // namespace moe
