// Dense products in 8-bit integers with one scale per token and one per output
// channel ("MiniMax-M3 W8A8 on K100AI", s1.2: INT8 x INT8 with integer
// accumulation and dequantisation at the end; s3.2: activations per token,
// weights per output channel):
//
//   y[t][n] = (sum_j xq[t][j] wq[n][j]) sx[t] sw[n] + bias[n]
//
// on tcgen05 tensor cores (kind::i8, INT32 accumulators, so the sums are exact
// whatever their order).
//
// Two kernels.  A few tokens are bound by reading the weights once: the
// weights are the MMA's 128-row operand and the tokens its N columns, and the
// input dimension is split over the blocks of a cluster so that every SM
// reads; the blocks add their INT32 accumulators over distributed shared
// memory.  Many tokens are bound by the tensor cores: pairs of SMs compute
// 256 x 256 tiles with cta_group::2 MMAs, with the epilogue of one tile under
// the main loop of the next.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kTile = 128;                        // channels and inputs of a weight tile
constexpr int kTileBytes = kTile * kTile;

// ------------------------------------------------------------------ preparation

// aw[j] = max_n |w[j][n]|, one block per input.
__global__ void linear_input_absmax_kernel(const float* __restrict__ w, int n, float* __restrict__ aw) {
    __shared__ float red[32];
    const float* row = w + (int64_t)blockIdx.x * n;
    float m = 0.0f;
    for (int i = threadIdx.x; i < n; i += blockDim.x) m = fmaxf(m, fabsf(row[i]));
    m = block_max_nonneg(m, red);
    if (threadIdx.x == 0) aw[blockIdx.x] = m;
}

// sw[n] = max_j |s_j w[j][n]| / 127 (0 past the last channel), 32 channels per block.
// A channel that holds a NaN gets that scale, so that its outputs are NaN; an infinite
// one does so by itself (codes 0 times an infinite scale).
__global__ void __launch_bounds__(256) linear_scales_kernel(const float* __restrict__ w, const float* __restrict__ smooth,
                                                            int k, int n, float* __restrict__ sw) {
    __shared__ float red[8][32];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
    float m = 0.0f;
    if (c < n)
        for (int j = ty; j < k; j += 8) {
            float v = w[(int64_t)j * n + c];
            if (smooth) v = __fmul_rn(smooth[j], v);
            m = max_abs_nan(m, v);
        }
    red[ty][tx] = m;
    __syncthreads();
    if (ty == 0) {
        for (int i = 1; i < 8; ++i) m = max_abs_nan(m, red[i][tx]);
        sw[c] = m == 0.0f ? 0.0f : __fdiv_rn(m, 127.0f);
    }
}

// One weight tile per block: codes rint(s_j w[j][n] / sw[n]), zeros past the edges.
__global__ void __launch_bounds__(256) linear_codes_kernel(const float* __restrict__ w, const float* __restrict__ smooth,
                                                           int k, int n, const float* __restrict__ sw,
                                                           int8_t* __restrict__ out) {
    __shared__ __align__(16) int8_t tile[kTile][kTile + 16];
    const int c = threadIdx.x & 127, half = threadIdx.x >> 7;
    const int64_t ch = (int64_t)blockIdx.y * kTile + c;
    const float s = sw[ch];
    for (int jj = half; jj < kTile; jj += 2) {
        const int j = blockIdx.x * kTile + jj;
        int q = 0;
        if (j < k && ch < n && s > 0.0f) {
            float v = w[(int64_t)j * n + ch];
            if (smooth) v = __fmul_rn(smooth[j], v);
            q = quant_code(v, s);
        }
        tile[c][jj] = (int8_t)q;
    }
    __syncthreads();
    int8_t* dst = out + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kTileBytes;
    for (int i = threadIdx.x; i < kTileBytes / 16; i += 256)
        reinterpret_cast<int4*>(dst)[i] = *reinterpret_cast<const int4*>(&tile[i >> 3][(i & 7) * 16]);
}

// One weight tile per block, from or to codes [n][k].
template <bool TO_TILES>
__global__ void __launch_bounds__(256) linear_tile_kernel(const int8_t* __restrict__ src, int k, int n,
                                                          int8_t* __restrict__ dst) {
    const int64_t t0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kTileBytes;
    for (int i = threadIdx.x; i < kTileBytes; i += 256) {
        const int64_t ch = (int64_t)blockIdx.y * kTile + (i >> 7);
        const int j = blockIdx.x * kTile + (i & 127);
        const bool in = ch < n && j < k;
        if (TO_TILES)
            dst[t0 + i] = in ? src[ch * k + j] : (int8_t)0;
        else if (in)
            dst[ch * k + j] = src[t0 + i];
    }
}

// ------------------------------------------------------------------ shared parts

__host__ __device__ constexpr uint32_t idesc_i8(int m, int n) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <uint32_t ID>
__device__ __forceinline__ void mma_i8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(ID), "r"(accum));
}

template <uint32_t ID>
__device__ __forceinline__ void mma_i8_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(ID), "r"(accum));
}

struct LinearParams {
    int n, k, T, kb;          // channels, inputs, tokens, input tiles
    int stages;               // small kernel: ring stages
    const void* x;            // small kernel, quantising: the activations
    const float* inv_s;
    int64_t ldx;
    int in_dtype;
    int n_tiles, m_tiles;     // pair kernel: 256-channel and 256-token tiles
    const float *sw, *bias, *sx;
    void* y;
    int64_t ldy;
    int out_bf16, vec;        // vec: y and its rows are aligned for 16-byte stores
    int32_t* status;
};

// ------------------------------------------------------------------ a few tokens

// TN tokens per block, the weights' 128 channels as the MMA's M.  Block (x, y)
// of the grid: channel tile x / S of cluster rank x % S, tokens [y TN, + TN).
// The S blocks of a cluster take contiguous parts of the input tiles.
//   warp 0   TMA producer: weight tiles (and, from codes, the tokens' 128 codes)
//            into a ring.  The weights are constants of the handle, so their
//            first copies are issued before the previous kernel's results are
//            waited for.
//   warp 1   tensor memory and the MMAs
//   all 8    accumulators (lane = channel) to shared memory as [token][channel]
//            words; then each block of the cluster adds the S partial tiles of
//            its part of the tokens and writes whole rows.
// QUANT: from the activations of at most kLinearQuantTokens tokens.  Each block
// finds the tokens' scales itself and quantises its own part of the inputs while
// its weights are on their way: one launch instead of two, at the price of every
// block reading the tokens.
constexpr int kSmallThreads = 256;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallMaxStages = 4;
constexpr int kSmallMaxSplit = 8;
constexpr size_t kSmallMaxSmem = 220 * 1024;   // beside the static part

struct SmallCtl {
    uint64_t full[kSmallMaxStages], empty[kSmallMaxStages], acc;
    uint32_t tmem_base;
    int abort;
    uint32_t amax[kSmallWarps][kLinearQuantTokens];   // QUANT: the warps' largest values (bits), then ...
    float scale[128];                                 // the tokens' scales
};

template <int TN, bool QUANT>
__host__ __device__ constexpr int small_stage_bytes() { return kTileBytes + (QUANT ? 0 : TN * kTile); }
// Shared memory of a block with `stages` ring stages and (QUANT) nkb input tiles
// of codes; the partial tile reuses it from its start.
template <int TN, bool QUANT>
constexpr size_t small_smem(int stages, int nkb) {
    const size_t operands = (size_t)stages * small_stage_bytes<TN, QUANT>() + (QUANT ? (size_t)nkb * TN * kTile : 0);
    const size_t part = (size_t)TN * kTile * 4;
    return (operands > part ? operands : part) + 1024;
}

// QUANT: the codes of this block's part of the inputs, [input tile][token][128
// codes] in the 128-byte swizzle (16-byte chunks XOR the row), and the tokens'
// scales.  The part's values are loaded first and stay in registers.
constexpr int kOwnGroups = 4;   // groups of 8 values of the part per thread

__device__ __forceinline__ void small_load(const LinearParams& p, int t, int j, float (&v)[8]) {
    load8_act(p.x, (int64_t)t * p.ldx + j, p.in_dtype, v);
    if (p.inv_s) {
        const float4 a = *reinterpret_cast<const float4*>(p.inv_s + j), b = *reinterpret_cast<const float4*>(p.inv_s + j + 4);
        const float s[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = __fmul_rn(v[c], s[c]);
    }
}

template <int TN>
__device__ __forceinline__ void small_quantize(const LinearParams& p, SmallCtl* ctl, uint8_t* codes, int kb0, int nkb) {
    const int groups = nkb * (kTile / 8);
    float own[kOwnGroups][8];
#pragma unroll
    for (int i = 0; i < kOwnGroups; ++i) {
        const int at = threadIdx.x + i * kSmallThreads, t = at / groups, j = kb0 * kTile + at % groups * 8;
        if (t < p.T && j < p.k) {
            small_load(p, t, j, own[i]);
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) own[i][c] = 0.0f;   // inputs past the last one
        }
    }
    for (int t = 0; t < p.T; ++t) {
        uint32_t m = 0;
#pragma unroll 4
        for (int j = threadIdx.x * 8; j < p.k; j += kSmallThreads * 8) {
            float v[8];
            small_load(p, t, j, v);
#pragma unroll
            for (int c = 0; c < 8; ++c) m = max(m, __float_as_uint(fabsf(v[c])));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if ((threadIdx.x & 31) == 0) ctl->amax[threadIdx.x >> 5][t] = m;
    }
    __syncthreads();
    if (threadIdx.x < p.T) {
        uint32_t m = 0;
        for (int w = 0; w < kSmallWarps; ++w) m = max(m, ctl->amax[w][threadIdx.x]);
        // a token that holds an infinity or a NaN gets codes 0 and the scale NaN
        ctl->scale[threadIdx.x] = m < 0x7f800000u ? __fdiv_rn(__uint_as_float(m), 127.0f) : __int_as_float(0x7fc00000);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOwnGroups; ++i) {
        const int at = threadIdx.x + i * kSmallThreads, t = at / groups, g = at % groups;
        if (t >= p.T) break;
        const float s = ctl->scale[t];
        uint2 q = make_uint2(0u, 0u);
        if (s > 0.0f) {
            const float inv = __frcp_rn(s);
            q = make_uint2(fmt_codes4<FMT_INT8>(own[i][0], own[i][1], own[i][2], own[i][3], s, inv),
                           fmt_codes4<FMT_INT8>(own[i][4], own[i][5], own[i][6], own[i][7], s, inv));
        }
        const int chunk = (g >> 1) & 7;
        *reinterpret_cast<uint2*>(codes + (size_t)(g >> 4) * TN * kTile + t * kTile + ((chunk ^ (t & 7)) << 4) + (g & 1) * 8) = q;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
}

template <int TN, bool QUANT>
__global__ void __launch_bounds__(kSmallThreads) linear_small_kernel(const __grid_constant__ CUtensorMap tm_w,
                                                                     const __grid_constant__ CUtensorMap tm_x,
                                                                     const LinearParams p) {
    constexpr int kStageBytes = small_stage_bytes<TN, QUANT>();
    constexpr uint32_t kCols = TN < 32 ? 32 : TN;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ SmallCtl shared_ctl;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    SmallCtl* ctl = &shared_ctl;
    cg::cluster_group cl = cg::this_cluster();
    const int S = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nt = blockIdx.x / S, t0 = blockIdx.y * TN, tn = min(TN, p.T - t0);
    const int kb0 = (int)((int64_t)p.kb * rank / S), kb1 = (int)((int64_t)p.kb * (rank + 1) / S);
    const int nkb = kb1 - kb0, stages = p.stages;
    uint8_t* codes = smem + stages * kStageBytes;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        mbar_init(&ctl->acc, 1);
        ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem_base)),
                     "r"(kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // only now: the next kernel's blocks must not hold tensor memory that this block
    // still asks for, since they wait for this kernel to end before they free it
    pdl_trigger();
    const uint32_t tmem = ctl->tmem_base;
    volatile int* abort = &ctl->abort;

    auto load_w = [&](int i) {
        const int s = i % stages;
        mbar_arrive_expect_tx(&ctl->full[s], kStageBytes);
        tma_load_2d(smem + s * kStageBytes, &tm_w, &ctl->full[s], 0, (nt * p.kb + kb0 + i) * kTile);
    };
    const int first = min(nkb, stages);
    if (threadIdx.x == 0)
        for (int i = 0; i < first; ++i) load_w(i);
    __syncwarp();
    if (QUANT) {
        pdl_wait();
        small_quantize<TN>(p, ctl, codes, kb0, nkb);
    }
    if (warp == 0) {
        if (lane == 0) {
            auto load_x = [&](int i) {
                const int s = i % stages;
                tma_load_2d(smem + s * kStageBytes + kTileBytes, &tm_x, &ctl->full[s], (kb0 + i) * kTile, t0);
            };
            if (!QUANT) {
                pdl_wait();
                for (int i = 0; i < first; ++i) load_x(i);
            }
            int issued = first;
            for (int i = first; i < nkb; ++i) {
                if (!mbar_wait(&ctl->empty[i % stages], ((i / stages) - 1) & 1, abort, p.status, 1, i)) break;
                load_w(i);
                if (!QUANT) load_x(i);
                ++issued;
            }
            // every copy has landed before the stages are reused or the block ends (bounded)
            for (int i = max(0, issued - stages); i < issued; ++i) {
                const uint64_t b = global_timer();
                while (!mbar_try_wait(&ctl->full[i % stages], (i / stages) & 1) && global_timer() - b < kWaitBudgetNs) {}
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int i = 0; i < nkb; ++i) {
                const int s = i % stages;
                if (!mbar_wait(&ctl->full[s], (i / stages) & 1, abort, p.status, 3, i)) break;
                tc_fence_after();
                const uint32_t a = smem_u32(smem + s * kStageBytes);
                const uint32_t b = QUANT ? smem_u32(codes + (size_t)i * TN * kTile) : a + kTileBytes;
#pragma unroll
                for (int kk = 0; kk < kTile / 32; ++kk)
                    mma_i8<idesc_i8(kTile, TN)>(tmem, desc_sw128(a + kk * 32), desc_sw128(b + kk * 32), (i | kk) != 0);
                mma_commit(&ctl->empty[s]);
            }
            mma_commit(&ctl->acc);
        }
    }
    __syncwarp();
    // what the output needs besides the sums, while these are formed: four neighbouring
    // channels per thread where whole words can be stored, else every 32nd, so that a
    // warp's stores are neighbours
    const int n0 = nt * kTile + (p.vec ? lane * 4 : lane), dn = p.vec ? 1 : 32;
    float sw[4], bs[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        sw[c] = p.sw[n0 + c * dn];
        bs[c] = p.bias ? p.bias[n0 + c * dn] : 0.0f;
    }
    pdl_wait();
    if (!QUANT && threadIdx.x < tn) ctl->scale[threadIdx.x] = p.sx[t0 + threadIdx.x];
    const bool ok = nkb == 0 || mbar_wait(&ctl->acc, 0, abort, p.status, 4, 0);
    __syncthreads();   // the stages are free: every copy and MMA is done
    tc_fence_after();

    // partial tile [token][channel], 128 words per row; two warps share a lane quarter
    int32_t* part = reinterpret_cast<int32_t*>(smem);
    const int quad = warp & 3, half = warp >> 2, ch = quad * 32 + lane;
    constexpr int kHalf = TN < 32 ? TN : TN / 2, kChunk = kHalf < 32 ? kHalf : 32;
    if (TN >= 32 || half == 0) {
#pragma unroll
        for (int c = 0; c < kHalf / kChunk; ++c) {
            uint32_t v[kChunk];
            const int col = half * kHalf + c * kChunk;
            const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + col;
            if constexpr (kChunk == 16)
                tmem_ld16(at, v);
            else
                tmem_ld32(at, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kChunk; ++j) part[(col + j) * kTile + ch] = ok && nkb > 0 ? (int)v[j] : 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
    }
    if (S > 1) cl.sync();
    // this block's part of the tokens
    const int r0 = tn * rank / S, r1 = tn * (rank + 1) / S;
#pragma unroll 4
    for (int r = r0 + warp; r < r1; r += kSmallWarps) {
        int acc[4] = {0, 0, 0, 0};
        for (int b = 0; b < S; ++b) {
            const int32_t* from = cl.map_shared_rank(part, b) + r * kTile;
            if (p.vec) {
                const int4 q = reinterpret_cast<const int4*>(from)[lane];
                acc[0] += q.x, acc[1] += q.y, acc[2] += q.z, acc[3] += q.w;
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] += from[lane + 32 * c];
            }
        }
        const int64_t t = t0 + r;
        const float sx = ctl->scale[r];
        float y[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(acc[c]), sx), sw[c]), bs[c]);
        if (p.out_bf16) {
            uint16_t* dst = reinterpret_cast<uint16_t*>(p.y) + t * p.ldy + n0;
            if (p.vec && n0 + 4 <= p.n) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(
                    (uint32_t)f32_to_bf16_bits(y[0]) | ((uint32_t)f32_to_bf16_bits(y[1]) << 16),
                    (uint32_t)f32_to_bf16_bits(y[2]) | ((uint32_t)f32_to_bf16_bits(y[3]) << 16));
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (n0 + c * dn < p.n) dst[c * dn] = f32_to_bf16_bits(y[c]);
            }
        } else {
            float* dst = reinterpret_cast<float*>(p.y) + t * p.ldy + n0;
            if (p.vec && n0 + 4 <= p.n) {
                *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (n0 + c * dn < p.n) dst[c * dn] = y[c];
            }
        }
    }
    if (S > 1) cl.sync();   // no block leaves while another reads its partial tile
}

// ------------------------------------------------------------------ many tokens

// 256 tokens x 256 channels per pair of SMs: each block holds its 128 tokens
// and half of the channels in shared memory, the pair's MMA (M = 256, N = 256)
// leaves each block its own 128 rows of the accumulator.  Roles as in the
// grouped pair kernel: warp 0 copies, warp 1 of the leader issues MMAs, warps
// 2..9 are the epilogue of the previous tile under the next one's main loop.
constexpr int kPStages = 6;
constexpr int kPStageBytes = 2 * kTileBytes;
constexpr int kPEpiWarps = 8;
constexpr int kPThreads = 64 + kPEpiWarps * 32;
constexpr int kPEpiBytes = 32 * 33 * 4;          // a warp's 32 x 32 words, one word of padding per row
constexpr size_t kPSmem = (size_t)kPStages * kPStageBytes + (size_t)kPEpiWarps * kPEpiBytes + 1024 + 256;

struct PairCtl {
    uint64_t full[kPStages], empty[kPStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base;
    int abort;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                       const LinearParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float* epi_stage = reinterpret_cast<float*>(smem + kPStages * kPStageBytes);
    PairCtl* ctl = reinterpret_cast<PairCtl*>(smem + kPStages * kPStageBytes + kPEpiWarps * kPEpiBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPStages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->acc_full[b], 1);
            mbar_init(&ctl->acc_empty[b], 2 * kPEpiWarps);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem_base)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int* abort = &ctl->abort;
    pdl_wait();
    pdl_trigger();
    const int num_tiles = p.n_tiles * p.m_tiles;
    const int cid = (int)cluster_index(), ncl = (int)cluster_count();
    const int nkb = p.kb;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            uint32_t issued_par[kPStages];
            bool issued[kPStages];
            for (int i = 0; i < kPStages; ++i) issued[i] = false;
            bool ok = true;
            for (int t = cid; t < num_tiles && ok; t += ncl) {
                const int mt = t % p.m_tiles, nt = t / p.m_tiles;
                const int row0 = mt * 256 + rank * kTile, wrow = (nt * 2 + rank) * nkb * kTile;
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait(&ctl->empty[s], ph ^ 1, abort, p.status, 1, t)) { ok = false; break; }
                    if (leader) mbar_arrive_expect_tx(&ctl->full[s], 2 * kPStageBytes);
                    const uint32_t bar = leader_addr(&ctl->full[s]);
                    uint8_t* sa = smem + s * kPStageBytes;
                    tma_load_2d_pair(sa, &tm_x, bar, kb * kTile, row0);
                    tma_load_2d_pair(sa + kTileBytes, &tm_w, bar, 0, wrow + kb * kTile);
                    issued[s] = true;
                    issued_par[s] = ph;
                    if (++s == kPStages) { s = 0; ph ^= 1; }
                }
            }
            if (leader) {
                for (int i = 0; i < kPStages; ++i) {
                    if (!issued[i]) continue;
                    const uint64_t b = global_timer();
                    while (!mbar_try_wait(&ctl->full[i], issued_par[i]) && global_timer() - b < kWaitBudgetNs) {}
                }
            }
            if (!ok) {
                // after a timeout this block's copies may be in flight, counted on the
                // other block's barrier only: time to land before the block can end
                const uint64_t b = global_timer();
                while (global_timer() - b < 200000ull) {}
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            int s = 0, buf = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int t = cid; t < num_tiles && ok; t += ncl) {
                if (!mbar_wait_cluster(&ctl->acc_empty[buf], aph ^ 1, abort, p.status, 2, t)) break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * 256);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait(&ctl->full[s], ph, abort, p.status, 3, t)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + s * kPStageBytes), b = a + kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < kTile / 32; ++kk)
                        mma_i8_pair<idesc_i8(256, 256)>(d, desc_sw128(a + kk * 32), desc_sw128(b + kk * 32), (kb | kk) != 0);
                    mma_commit_pair(&ctl->empty[s], 0x3);
                    if (++s == kPStages) { s = 0; ph ^= 1; }
                }
                if (!ok) break;
                mma_commit_pair(&ctl->acc_full[buf], 0x3);
                buf ^= 1;
                if (buf == 0) aph ^= 1;
            }
            mma_commit_pair(&ctl->drain, 0x1);
            const uint64_t b = global_timer();
            while (!mbar_try_wait(&ctl->drain, 0) && global_timer() - b < kWaitBudgetNs) {}
        }
    } else {
        // epilogue: a warp owns 32 tokens (its tensor-memory lanes) and 128 channels, 32 at a time
        const int ew = warp - 2, quad = warp & 3, half = ew >> 2;
        float* stage = epi_stage + ew * (kPEpiBytes / 4);
        int buf = 0;
        uint32_t aph = 0;
        for (int t = cid; t < num_tiles; t += ncl) {
            const int mt = t % p.m_tiles, nt = t / p.m_tiles;
            const int64_t row0 = (int64_t)mt * 256 + rank * kTile + quad * 32;
            const int nvalid = (int)max((int64_t)0, min((int64_t)32, p.T - row0));
            const float sx = lane < nvalid ? p.sx[row0 + lane] : 0.0f;
            if (!mbar_wait(&ctl->acc_full[buf], aph, abort, p.status, 4, t)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * 256 + half * 128);
            for (int c = 0; c < 4; ++c) {
                uint32_t v[32];
                tmem_ld32(taddr + c * 32, v);
                tmem_ld_wait();
                if (c == 3) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(&ctl->acc_empty[buf]))
                                     : "memory");
                    }
                }
                const int n0 = nt * 256 + half * 128 + c * 32;
                const float sw = p.sw[n0 + lane], bs = p.bias ? p.bias[n0 + lane] : 0.0f;
#pragma unroll
                for (int j = 0; j < 32; ++j) stage[lane * 33 + j] = __fmul_rn(__int2float_rn((int)v[j]), sx);
                __syncwarp();
                const bool in = n0 + lane < p.n;
                for (int r = 0; r < nvalid; ++r) {
                    const float y = __fadd_rn(__fmul_rn(stage[r * 33 + lane], sw), bs);
                    if (!in) continue;
                    if (p.out_bf16)
                        reinterpret_cast<uint16_t*>(p.y)[(row0 + r) * p.ldy + n0 + lane] = f32_to_bf16_bits(y);
                    else
                        reinterpret_cast<float*>(p.y)[(row0 + r) * p.ldy + n0 + lane] = y;
                }
                __syncwarp();
            }
            buf ^= 1;
            if (buf == 0) aph ^= 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// ------------------------------------------------------------------ host side

// Map over rows of 8-bit codes, boxes of `box_rows` rows x 128 bytes with the
// 128-byte swizzle the MMA descriptors expect; bytes past `cols` read as zero.
bool make_codes_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t ld, uint64_t rows, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {ld};
    const cuuint32_t box[2] = {(cuuint32_t)kTile, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TN, bool QUANT>
cudaError_t launch_small_as(const LinearTiles& t, const CUtensorMap& tx, LinearParams& p, int split, cudaStream_t s) {
    // the ring: what the block reads, four stages at most, fewer where two blocks would
    // not fit on an SM (64 x 4096 x 32000 took 25.3 us with four, 34.6 with six)
    const int nkb = (t.kb + split - 1) / split;
    p.stages = std::min(nkb, kSmallMaxStages);
    while (p.stages > 2 && small_smem<TN, QUANT>(p.stages, nkb) > kSmallMaxSmem / 2) --p.stages;
    const size_t smem = small_smem<TN, QUANT>(p.stages, nkb);
    static std::atomic<uint64_t> attr{0};
    cudaError_t e = smem_attr_once(linear_small_kernel<TN, QUANT>, kSmallMaxSmem, attr);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((t.n + kTile - 1) / kTile * split), (unsigned)(((int64_t)p.T + TN - 1) / TN));
    return launch_cluster(linear_small_kernel<TN, QUANT>, grid, dim3(kSmallThreads), split, smem, s, t.tm_w, tx, p);
}

cudaError_t launch_small(const LinearTiles& t, const CUtensorMap& tx, LinearParams& p, int tokens, int split,
                         cudaStream_t s) {
    switch (tokens) {
        case 16: return launch_small_as<16, false>(t, tx, p, split, s);
        case 32: return launch_small_as<32, false>(t, tx, p, split, s);
        case 64: return launch_small_as<64, false>(t, tx, p, split, s);
        default: return launch_small_as<128, false>(t, tx, p, split, s);
    }
}

cudaError_t pair_clusters(int* out) {
    static std::atomic<int> clusters[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = clusters[dev & 63].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(2);
        q.blockDim = dim3(kPThreads);
        q.dynamicSmemBytes = kPSmem;
        cudaLaunchAttribute a[1];
        a[0].id = cudaLaunchAttributeClusterDimension;
        a[0].val.clusterDim.x = 2;
        a[0].val.clusterDim.y = 1;
        a[0].val.clusterDim.z = 1;
        q.attrs = a;
        q.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, (const void*)linear_pair_kernel, &q);
        if (e != cudaSuccess) return e;
        if (n <= 0) return cudaErrorInvalidConfiguration;
        clusters[dev & 63].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return cudaSuccess;
}

}  // namespace

bool linear_make_map(LinearTiles* t) {
    const uint64_t rows = (uint64_t)t->nb * t->kb * kTile;
    return make_codes_map(&t->tm_w, t->w, kTile, kTile, rows, kTile);
}

cudaError_t launch_linear_input_absmax(const float* w, int k, int n, float* aw, cudaStream_t s) {
    linear_input_absmax_kernel<<<k, 256, 0, s>>>(w, n, aw);
    return cudaGetLastError();
}

cudaError_t launch_linear_quantize(const float* w, const float* smooth, const LinearTiles& t, int8_t* out, float* sw,
                                   cudaStream_t s) {
    linear_scales_kernel<<<t.nb * kTile / 32, 256, 0, s>>>(w, smooth, t.k, t.n, sw);
    linear_codes_kernel<<<dim3(t.kb, t.nb), 256, 0, s>>>(w, smooth, t.k, t.n, sw, out);
    return cudaGetLastError();
}

cudaError_t launch_linear_tile(const int8_t* wq, const LinearTiles& t, int8_t* out, cudaStream_t s) {
    linear_tile_kernel<true><<<dim3(t.kb, t.nb), 256, 0, s>>>(wq, t.k, t.n, out);
    return cudaGetLastError();
}

cudaError_t launch_linear_untile(const LinearTiles& t, int8_t* wq, cudaStream_t s) {
    linear_tile_kernel<false><<<dim3(t.kb, t.nb), 256, 0, s>>>(t.w, t.k, t.n, wq);
    return cudaGetLastError();
}

namespace {

// How a call runs: tokens per block and parts of the inputs for the kernel of a few
// tokens, or (tokens = 0) the pair kernel.
struct LinearPlan {
    int tokens, split;
};

// The plan that a model of the kernels' times, in ns, finds the shortest.  A block
// of the small kernel takes a fixed time that grows with its tokens (its set-up and
// its output), 700 more if the inputs are split (two cluster barriers), and 350 per
// input tile (16 KB at the 50 GB/s that a block takes in), 420 where two blocks
// share an SM; more than two per SM wait for another round.  A pair of SMs takes 8
// us and 450 ns per input tile and round.  The measured times that the numbers come
// from (us, model in brackets): 517 x 1000 x 1111 with 32 tokens per block 6.8 (7.2),
// with 64 in two parts 7.2 (7.4), with 128 11.0 (10.3); 256 x 4096 x 4096 with 64 in
// two parts 12.1 (12.4), with 128 in four 11.7 (11.6), in two 13.6 (13.8); 1024 x
// 4096 x 4096 with 128 20.6 (20.9); 32 x 4096 x 6144 with 32 in four parts 7.2
// (7.9); 4096 x 4096 x 4096 on pairs 56 to 77 (66).  It has no term for memory: 64 x
// 4096 x 32000 is 18 in it, its bytes alone take 21 and the launch takes 25.
LinearPlan linear_plan(const LinearTiles& t, int T, bool quantize) {
    LinearPlan best{0, 1};
    const int64_t channels = (t.n + kTile - 1) / kTile;
    const int64_t pairs = (int64_t)((t.n + 255) / 256) * (((int64_t)T + 255) / 256), at_once = std::max(1, t.num_sms / 2);
    int64_t least = quantize || T <= 64 ? INT64_MAX : 8000 + (pairs + at_once - 1) / at_once * t.kb * 450;
    const int fixed[4] = {3800, 3800, 5000, 7500};
    for (int i = 0; i < 4; ++i) {
        const int tokens = 16 << i;
        if ((quantize && tokens > 16) || (i > 0 && tokens / 2 >= T)) break;
        if (((int64_t)T + tokens - 1) / tokens > 65535) continue;   // the grid's second dimension
        for (int split = 1; split <= kSmallMaxSplit && (split == 1 || t.kb / split >= 4); split *= 2) {
            const int64_t blocks = channels * (((int64_t)T + tokens - 1) / tokens) * split;
            const int64_t rounds = (blocks + 2 * t.num_sms - 1) / (2 * t.num_sms);
            const int64_t tiles = (t.kb + split - 1) / split;
            const int64_t ns = rounds * (fixed[i] + (split > 1 ? 700 : 0) + tiles * (blocks > t.num_sms ? 420 : 350));
            if (ns < least) {
                least = ns;
                best = LinearPlan{tokens, split};
            }
        }
    }
    return best;
}

LinearParams linear_params(const LinearTiles& t, int T, void* y, int64_t ldy, int out_dtype) {
    LinearParams p{};
    p.n = t.n;
    p.k = t.k;
    p.T = T;
    p.kb = t.kb;
    p.sw = t.sw;
    p.bias = t.bias;
    p.y = y;
    p.ldy = ldy;
    p.out_bf16 = out_dtype == MOE_BF16;
    p.vec = ((uintptr_t)y & 15) == 0 && (ldy * (p.out_bf16 ? 2 : 4)) % 16 == 0;
    p.status = t.status;
    p.n_tiles = (t.n + 255) / 256;
    p.m_tiles = (int)(((int64_t)T + 255) / 256);
    return p;
}

}  // namespace

bool linear_quantizes(const LinearTiles& t, const void* x, int64_t ldx, int T, int in_dtype) {
    const int64_t esz = in_dtype == MOE_BF16 ? 2 : 4;
    if (t.k % 8 || ((uintptr_t)x & 15) || (ldx * esz) % 16 || T > kLinearQuantTokens) return false;
    const int split = linear_plan(t, T, true).split, nkb = (t.kb + split - 1) / split;
    return T * nkb * (kTile / 8) <= kOwnGroups * kSmallThreads;   // the part's values fit the threads' registers
}

cudaError_t launch_linear_quantizing(const LinearTiles& t, const void* x, int64_t ldx, int in_dtype, const float* inv_s,
                                     int T, void* y, int64_t ldy, int out_dtype, cudaStream_t s) {
    LinearParams p = linear_params(t, T, y, ldy, out_dtype);
    p.x = x;
    p.ldx = ldx;
    p.in_dtype = in_dtype;
    p.inv_s = inv_s;
    return launch_small_as<16, true>(t, t.tm_w, p, linear_plan(t, T, true).split, s);   // (no map of x)
}

cudaError_t launch_linear(const LinearTiles& t, const int8_t* xq, int64_t ldq, const float* sx, int T, void* y, int64_t ldy,
                          int out_dtype, cudaStream_t s) {
    LinearParams p = linear_params(t, T, y, ldy, out_dtype);
    p.sx = sx;
    const LinearPlan plan = linear_plan(t, T, false);
    CUtensorMap tx;
    if (!make_codes_map(&tx, xq, t.k, ldq, T, plan.tokens ? plan.tokens : kTile)) return cudaErrorInvalidValue;
    if (plan.tokens == 0) {
        static std::atomic<uint64_t> attr{0};
        cudaError_t e = smem_attr_once(linear_pair_kernel, kPSmem, attr);
        if (e != cudaSuccess) return e;
        int nc = 0;
        e = pair_clusters(&nc);
        if (e != cudaSuccess) return e;
        const int grid = 2 * (int)std::min<int64_t>(nc, (int64_t)p.n_tiles * p.m_tiles);
        return launch_pdl(linear_pair_kernel, dim3(grid), dim3(kPThreads), kPSmem, s, t.tm_w, tx, p);
    }
    return launch_small(t, tx, p, plan.tokens, plan.split, s);
}

}  // namespace moe
