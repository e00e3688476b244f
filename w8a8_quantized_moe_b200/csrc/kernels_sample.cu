// The next token of each row of logits, from given random numbers.
//
// Per row: the tokens in order of falling logit (lowest index first on ties,
// the router's own rule); the first top_k of them; of those the shortest
// prefix that holds top_p of their mass, with masses e_i = exp((l_i - max) /
// temperature); of those the ones with e_i >= min_p; and then, in the order of
// the tokens, the first whose running mass exceeds u times the kept mass.
//
// No order is ever formed: "the first top_k" and "the shortest prefix" are
// each a key K (a logit as an ordered 32-bit integer) and a first excluded
// index among the tokens that equal K, found by selecting 11, 11 and 10 bits
// of the key at a time from a histogram of counts, or of masses.  Masses are
// held as integers in units of 2^-45 of the largest one (one unit at least: u =
// 0 is the first token that takes part), so sums do not depend on the order of
// the atomics and every comparison is exact.
//
// A row belongs to a cluster of thread blocks that keep it in their shared
// memory: the logits are read from memory once, the later passes read shared
// memory, and the blocks exchange histograms and sums over distributed shared
// memory.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kSaThreads = 512;
constexpr int kSaWarps = kSaThreads / 32;
constexpr int kSaMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kBinsPerThread = kBins / kSaThreads;
constexpr uint32_t kNone = 0x007fffffu;   // ordered key of -infinity: a token that may not be chosen
constexpr int kMassBits = 45;

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

// exp((l - max) / temperature) in 64 bits: 2^x, x = (l - max) log2(e) / t = n +
// f with |f| <= 1/2, and the Taylor polynomial of e^(f ln 2) to degree 9, whose
// remainder is below 0.35^10 / 10! = 8e-12.
struct Softmax {
    uint32_t kmax;
    double vmax, c;   // c = log2(e) / temperature
    __device__ __forceinline__ double e(uint32_t key) const {
        if (key == kmax) return 1.0;
        const double x = ((double)value_of(key) - vmax) * c;
        if (!(x > -1000.0)) return 0.0;
        const double n = rint(x);
        const double y = (x - n) * 0.69314718055994530942;
        double p = 1.0 / 362880;
        p = fma(p, y, 1.0 / 40320);
        p = fma(p, y, 1.0 / 5040);
        p = fma(p, y, 1.0 / 720);
        p = fma(p, y, 1.0 / 120);
        p = fma(p, y, 1.0 / 24);
        p = fma(p, y, 1.0 / 6);
        p = fma(p, y, 0.5);
        p = fma(p, y, 1.0);
        p = fma(p, y, 1.0);
        return p * __hiloint2double((1023 + (int)n) << 20, 0);
    }
    __device__ __forceinline__ uint64_t mass(uint32_t key) const {
        const double v = e(key);
        return v > 0.0 ? max(__double2ull_rn(v * (double)(1ull << kMassBits)), 1ull) : 0ull;
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
    uint64_t slots[2][kSaMaxCluster][2];   // per reduction, alternating: one pair of sums per block
    uint64_t warp_a[kSaWarps], warp_b[kSaWarps];
    uint64_t found_above;
    uint32_t found_bin;
    int32_t out_index;
};

// One row of a cluster.
struct Row {
    cg::cluster_group cl;
    int nb, rank;                // blocks of the cluster, this one
    SaShared* sh;
    uint32_t* keys;              // this block's tokens [lo, lo + n)
    uint32_t* hist;              // [2][3][kBins]
    int lo, n, per_warp;         // a warp owns tokens [warp * per_warp, + per_warp) of the block's
    int turn, level;
    int tid, lane, warp;

    // Sums of a and b over the cluster, and the sums over the blocks before this one.
    __device__ void sum2(uint64_t a, uint64_t b, uint64_t& ta, uint64_t& tb, uint64_t& pa, uint64_t& pb) {
        a = warp_sum_u64(a);
        b = warp_sum_u64(b);
        __syncthreads();
        if (lane == 0) {
            sh->warp_a[warp] = a;
            sh->warp_b[warp] = b;
        }
        __syncthreads();
        if (warp == 0) {
            a = warp_sum_u64(lane < kSaWarps ? sh->warp_a[lane] : 0);
            b = warp_sum_u64(lane < kSaWarps ? sh->warp_b[lane] : 0);
            if (lane < nb) {
                uint64_t* dst = cl.map_shared_rank(&sh->slots[turn][rank][0], lane);
                dst[0] = a;
                dst[1] = b;
            }
        }
        cl.sync();
        ta = tb = pa = pb = 0;
        for (int i = 0; i < nb; ++i) {
            const uint64_t va = sh->slots[turn][i][0], vb = sh->slots[turn][i][1];
            if (i < rank) pa += va, pb += vb;
            ta += va, tb += vb;
        }
        turn ^= 1;
    }
    __device__ uint32_t max_key(uint32_t k) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
        __syncthreads();
        if (lane == 0) sh->warp_a[warp] = k;
        __syncthreads();
        if (warp == 0) {
            k = lane < kSaWarps ? (uint32_t)sh->warp_a[lane] : 0u;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
            if (lane < nb) *cl.map_shared_rank(&sh->slots[turn][rank][0], lane) = k;
        }
        cl.sync();
        for (int i = 0; i < nb; ++i) k = i == 0 ? (uint32_t)sh->slots[turn][0][0] : max(k, (uint32_t)sh->slots[turn][i][0]);
        turn ^= 1;
        return k;
    }
};

// The tokens still in the running: key above K, or equal to K and below index I.
struct Cut {
    uint32_t K;
    int I;
    __device__ __forceinline__ bool in(uint32_t key, int index) const { return key > K || (key == K && index < I); }
};

// Among the tokens inside `cut`, in order of falling key: the key at which the
// running count (or mass) reaches `need`, and how much lies strictly above it.
// False when the whole set does not reach it.
template <bool MASS>
__device__ bool select_key(Row& r, const Softmax& sm, const Cut& cut, double need, uint32_t& key_out, uint64_t& above_out) {
    uint32_t prefix = 0, mask = 0;
    uint64_t above = 0;
    for (int lv = 0; lv < 3; ++lv) {
        const int shift = lv == 0 ? 21 : lv == 1 ? 10 : 0, bins = lv == 2 ? 1024 : 2048;
        uint32_t* h = r.hist + (r.level & 1) * 3 * kBins;
        for (int i = r.tid; i < (MASS ? 3 : 1) * kBins; i += kSaThreads) h[i] = 0;
        __syncthreads();
        for (int i = r.tid; i < r.n; i += kSaThreads) {
            const uint32_t k = r.keys[i];
            if ((k & mask) != prefix || !cut.in(k, r.lo + i)) continue;
            const int bin = (k >> shift) & (bins - 1);
            if constexpr (MASS) {
                const uint64_t m = sm.mass(k);
                if (m & 0x7fffu) atomicAdd(&h[bin], (uint32_t)(m & 0x7fffu));
                if ((m >> 15) & 0x7fffu) atomicAdd(&h[kBins + bin], (uint32_t)((m >> 15) & 0x7fffu));
                if (m >> 30) atomicAdd(&h[2 * kBins + bin], (uint32_t)(m >> 30));
            } else {
                atomicAdd(&h[bin], 1u);
            }
        }
        r.cl.sync();
        // thread t: bins from the top, [bins - 1 - t * 4 .. - 3]
        uint64_t v[kBinsPerThread];
        uint64_t mine = 0;
#pragma unroll
        for (int j = 0; j < kBinsPerThread; ++j) {
            const int bin = bins - 1 - (r.tid * kBinsPerThread + j);
            uint64_t s = 0;
            if (bin >= 0)
                for (int b = 0; b < r.nb; ++b) {
                    const uint32_t* hb = r.cl.map_shared_rank(h, b);
                    s += hb[bin];
                    if constexpr (MASS) s += ((uint64_t)hb[kBins + bin] << 15) + ((uint64_t)hb[2 * kBins + bin] << 30);
                }
            v[j] = s;
            mine += s;
        }
        // prefix over the threads: each knows what lies above its bins
        const uint64_t inc = warp_scan_u64(mine, r.lane);
        __syncthreads();
        if (r.lane == 31) r.sh->warp_a[r.warp] = inc;
        if (r.tid == 0) r.sh->found_bin = 0xffffffffu;
        __syncthreads();
        uint64_t before = above + inc - mine;
        for (int w = 0; w < r.warp; ++w) before += r.sh->warp_a[w];
#pragma unroll
        for (int j = 0; j < kBinsPerThread; ++j) {
            if ((double)before < need && (double)(before + v[j]) >= need) {
                r.sh->found_bin = (uint32_t)(bins - 1 - (r.tid * kBinsPerThread + j));
                r.sh->found_above = before;
            }
            before += v[j];
        }
        __syncthreads();
        const uint32_t bin = r.sh->found_bin;
        if (bin == 0xffffffffu) return false;   // the same in every block: they see the same sums
        above = r.sh->found_above;
        prefix |= bin << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        ++r.level;
    }
    key_out = prefix;
    above_out = above;
    return true;
}

// The index of the tie number `keep` (from 0, in the order of the tokens) among
// the tokens inside `cut` whose key is K: the first one left out.
__device__ int tie_limit(Row& r, const Cut& cut, uint32_t K, uint64_t keep, int vocab) {
    const int w0 = r.warp * r.per_warp, w1 = min(r.n, w0 + r.per_warp);
    uint32_t c = 0;
    for (int i = w0 + r.lane; i < w1; i += 32) c += r.keys[i] == K && cut.in(K, r.lo + i);
    uint64_t total, none, before, none2;
    const uint64_t mine = warp_sum_u64(c);
    r.sum2(c, 0, total, none, before, none2);
    if (total <= keep) return vocab;
    __syncthreads();
    if (r.lane == 0) r.sh->warp_b[r.warp] = mine;
    if (r.tid == 0) r.sh->out_index = -1;
    __syncthreads();
    for (int w = 0; w < r.warp; ++w) before += r.sh->warp_b[w];
    if (before <= keep && keep < before + mine) {
        uint64_t at = before;
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const int i = i0 + r.lane;
            const bool is = i < w1 && r.keys[i] == K && cut.in(K, r.lo + i);
            const uint32_t m = __ballot_sync(0xffffffffu, is);
            if (keep < at + __popc(m)) {
                const int nth = (int)(keep - at);
                if (is && __popc(m & ((1u << r.lane) - 1)) == nth) r.sh->out_index = r.lo + i;
                break;
            }
            at += __popc(m);
        }
    }
    __syncthreads();
    const int local = r.sh->out_index;
    uint64_t a, b, pa, pb;
    r.sum2(r.tid == 0 && local >= 0 ? (uint64_t)local : 0, 0, a, b, pa, pb);
    return (int)a;
}

template <bool VEC>
__global__ void __launch_bounds__(kSaThreads) sample_kernel(const SampleParams p) {
    pdl_trigger();
    extern __shared__ __align__(16) uint32_t sa_smem[];
    __shared__ SaShared shared;
    Row r{cg::this_cluster()};
    r.nb = (int)r.cl.num_blocks();
    r.rank = (int)r.cl.block_rank();
    r.sh = &shared;
    r.hist = sa_smem;
    r.keys = sa_smem + 2 * 3 * kBins;
    r.tid = threadIdx.x;
    r.lane = threadIdx.x & 31;
    r.warp = threadIdx.x >> 5;
    r.turn = r.level = 0;
    const int row = blockIdx.x / r.nb;
    r.lo = min(p.vocab, r.rank * p.per_block);
    r.n = min(p.vocab, r.lo + p.per_block) - r.lo;
    r.per_warp = p.per_block / kSaWarps;
    pdl_wait();

    // the row's logits, as keys, into shared memory
    const int64_t base = (int64_t)row * p.ld + r.lo;
    const uint32_t* allowed = p.allowed ? p.allowed + (int64_t)row * p.ld_allowed : nullptr;
    uint32_t kmax = 0;
    uint64_t valid = 0;
    if constexpr (VEC) {
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
                kmax = max(kmax, k[c]);
                valid += k[c] > kNone;
            }
            reinterpret_cast<uint4*>(r.keys)[2 * g] = make_uint4(k[0], k[1], k[2], k[3]);
            reinterpret_cast<uint4*>(r.keys)[2 * g + 1] = make_uint4(k[4], k[5], k[6], k[7]);
        }
    } else {
        for (int i = r.tid; i < r.n; i += kSaThreads) {
            uint32_t k = key_of(p.dtype == MOE_BF16 ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p.logits)[base + i])
                                                    : reinterpret_cast<const float*>(p.logits)[base + i]);
            if (allowed && !((allowed[(r.lo + i) >> 5] >> ((r.lo + i) & 31)) & 1u)) k = kNone;
            r.keys[i] = k;
            kmax = max(kmax, k);
            valid += k > kNone;
        }
    }
    kmax = r.max_key(kmax);
    uint64_t n_valid, t0, t1, t2;
    r.sum2(valid, 0, n_valid, t0, t1, t2);
    const bool writer = r.rank == 0 && r.tid == 0;
    if (n_valid == 0) {
        if (writer) {
            p.token[row] = -1;
            if (p.prob) p.prob[row] = 0.0f;
        }
        r.cl.sync();
        return;
    }
    const float temp = p.temperature ? p.temperature[row] : 1.0f;
    if (!(temp > 0.0f)) {   // greedy: the lowest index among the largest
        const int at = tie_limit(r, Cut{kNone, 0}, kmax, 0, 0);
        if (writer) {
            p.token[row] = at;
            if (p.prob) p.prob[row] = 1.0f;
        }
        r.cl.sync();
        return;
    }
    Softmax sm{kmax, (double)value_of(kmax), 1.4426950408889634074 / (double)temp};
    Cut cut{kNone, 0};   // every token that may be chosen
    const int top_k = p.top_k ? p.top_k[row] : 0;
    if (top_k > 0 && (uint64_t)top_k < n_valid) {
        uint32_t K = 0;
        uint64_t above = 0;
        if (select_key<false>(r, sm, cut, (double)top_k, K, above)) {
            const int I = tie_limit(r, cut, K, (uint64_t)top_k - above, p.vocab);
            cut = Cut{K, I};
        }
    }
    const float top_p = p.top_p ? p.top_p[row] : 1.0f;
    if (top_p < 1.0f) {
        uint64_t z = 0, total;
        for (int i = r.tid; i < r.n; i += kSaThreads) {
            const uint32_t k = r.keys[i];
            if (cut.in(k, r.lo + i)) z += sm.mass(k);
        }
        r.sum2(z, 0, total, t0, t1, t2);
        // the least mass that reaches the prefix; at least the first token's
        const double need = fmax((double)top_p * (double)total, 1.0);
        uint32_t K = 0;
        uint64_t above = 0;
        if (select_key<true>(r, sm, cut, need, K, above)) {
            const double m = (double)sm.mass(K);
            const uint64_t ties = (uint64_t)fmax(1.0, ceil((need - (double)above) / m));
            const int I = tie_limit(r, cut, K, ties, p.vocab);
            cut = Cut{K, K == cut.K ? min(I, cut.I) : I};
        }
    }
    const float mp = p.min_p ? p.min_p[row] : 0.0f;
    const double min_p = mp > 0.0f ? fmin((double)mp, 1.0) : 0.0;
    // the kept mass, by warp (the tokens of a warp are neighbours), block and cluster
    const int w0 = r.warp * r.per_warp, w1 = min(r.n, w0 + r.per_warp);
    auto kept = [&](int i) -> uint64_t {
        const uint32_t k = r.keys[i];
        if (!cut.in(k, r.lo + i)) return 0;
        if (min_p > 0.0 && sm.e(k) < min_p) return 0;
        return sm.mass(k);
    };
    uint64_t z = 0, total, before;
    for (int i = w0 + r.lane; i < w1; i += 32) z += kept(i);
    const uint64_t mine = warp_sum_u64(z);
    r.sum2(z, 0, total, t0, before, t1);
    const float u = p.u[row];
    uint64_t target = u > 0.0f ? (uint64_t)floor((double)u * (double)total) : 0;
    target = min(target, total - 1);
    __syncthreads();
    if (r.lane == 0) r.sh->warp_b[r.warp] = mine;
    __syncthreads();
    for (int w = 0; w < r.warp; ++w) before += r.sh->warp_b[w];
    if (before <= target && target < before + mine) {
        uint64_t at = before;
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const int i = i0 + r.lane;
            const uint64_t m = i < w1 ? kept(i) : 0;
            const uint64_t inc = at + warp_scan_u64(m, r.lane);
            const uint32_t over = __ballot_sync(0xffffffffu, inc > target);
            if (over) {
                if (r.lane == __ffs(over) - 1) {
                    p.token[row] = r.lo + i;
                    if (p.prob) p.prob[row] = (float)(sm.e(r.keys[i]) * (double)(1ull << kMassBits) / (double)total);
                }
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
    const size_t smem = (size_t)(2 * 3 * kBins + p.per_block) * 4;
    const size_t esz = p.dtype == MOE_BF16 ? 2 : 4;
    const bool vec = ((uintptr_t)p.logits & 15) == 0 && (p.ld * (int64_t)esz) % 16 == 0;
    static std::atomic<uint64_t> attr[2];
    auto kern = vec ? sample_kernel<true> : sample_kernel<false>;
    cudaError_t e = smem_attr_once(kern, (size_t)(2 * 3 * kBins + kSampleMaxVocab / kSaMaxCluster) * 4, attr[vec]);
    if (e != cudaSuccess) return e;
    return launch_cluster(kern, dim3((unsigned)(p.rows * nb)), dim3(kSaThreads), nb, smem, s, p);
}

}  // namespace moe
