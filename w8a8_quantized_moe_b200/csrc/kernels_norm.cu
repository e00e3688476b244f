// The norms around a block and what lies between them, one pass per row:
//
//   p = b                       or  b / rms(b) * (w_post + offset)   (norm after the block)
//   r = residual_scale x + branch_scale g p, rounded to the stream's type
//   n = r / rms(r) * (w_pre + offset)                                (norm before the next block)
//   q = rint(v / s'), s' = max|v| / 127, v = r (w_pre + offset) inv_s, s = s' / rms(r)
//
// with rms(v) = sqrt(mean v^2 + eps), so that q s inv_s^-1 stands for n: the
// 8-bit codes and scale of the next product's input ("MiniMax-M3 W8A8 on
// K100AI", s3.2: activations per token, smoothed).  The row's rms cancels in
// v / s', so the codes do not depend on the order of the sum of squares; it
// enters the scale alone.
//
// Bound by memory: every value is read once and written once, and a row stays
// in registers between its two norms.  Two kernels: block_norm_rows_kernel for
// rows on 16-byte boundaries whose stream and branch have one type (16-byte
// accesses; the blocks stay and load their next row before they work on the
// current one), block_norm_kernel for everything else.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

// W consecutive values from index i of a row (W = 8: 16-byte accesses).
template <int W>
__device__ __forceinline__ void load_vals(const void* p, int64_t i, int dtype, float (&v)[W]) {
    if constexpr (W == 8) {
        load8_act(p, i, dtype, v);
    } else {
        v[0] = dtype == MOE_BF16 ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p)[i])
                                 : reinterpret_cast<const float*>(p)[i];
    }
}

// Round to the stored type and store; v keeps the rounded values.
template <int W>
__device__ __forceinline__ void round_vals(int dtype, float (&v)[W]) {
    if (dtype == MOE_BF16) {
#pragma unroll
        for (int c = 0; c < W; ++c) v[c] = __bfloat162float(__float2bfloat16_rn(v[c]));
    }
}

template <int W>
__device__ __forceinline__ void store_vals(void* p, int64_t i, int dtype, const float (&v)[W]) {
    if constexpr (W == 8) {
        if (dtype == MOE_BF16) {
            uint32_t w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * c], v[2 * c + 1]);
                w[c] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
        if (dtype == MOE_BF16)
            reinterpret_cast<uint16_t*>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        else
            reinterpret_cast<float*>(p)[i] = v[0];
    }
}

// Sum and unsigned maximum over the TPR threads of a row.  `red`: 2 words per
// warp of the block, used by one call at a time (the caller alternates halves).
template <int TPR>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& mx, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) {
            red[warp] = sum;
            red[NW + warp] = __uint_as_float(mx);
        }
        __syncthreads();
        float s = lane < NW ? red[lane] : 0.0f;
        uint32_t m = lane < NW ? __float_as_uint(red[NW + lane]) : 0u;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        }
        sum = s;
        mx = m;
    }
}

// The codes of four values for scale s > 0 (inv = fp32(1 / s)): identical to
// quant_code of each.  t = v inv is within 2.3e-5 of the IEEE quotient where that
// is below 128 (quant_code_fast), so unless t lies within 3e-5 of a half-integer
// both round to the same integer, which the sum with 1.5 x 2^23 leaves in its low
// byte; the largest value has the quotient 127 and a rounding, so no clamp is
// needed.  Otherwise (or when 1 / s overflowed: the comparison fails) the
// quotients are formed.
__device__ __forceinline__ uint32_t int8_codes4(float v0, float v1, float v2, float v3, float s, float inv) {
    const float v[4] = {v0, v1, v2, v3};
    float a[4];
    bool fast = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float t = __fmul_rn(v[i], inv);
        a[i] = __fadd_rn(t, 12582912.0f);
        fast = fast && fabsf(__fsub_rn(t, __fsub_rn(a[i], 12582912.0f))) < 0.49997f;
    }
    if (fast)
        return __byte_perm(__byte_perm(__float_as_uint(a[0]), __float_as_uint(a[1]), 0x0040),
                           __byte_perm(__float_as_uint(a[2]), __float_as_uint(a[3]), 0x0040), 0x5410);
    return pack4(quant_code(v0, s), quant_code(v1, s), quant_code(v2, s), quant_code(v3, s));
}

// TPR threads per row, each with G groups of W values: group g of thread t is
// values [(t + TPR g) W, ... + W).  Rows per block: 8 when a warp owns a row,
// else one.
template <int TPR, int G, int W>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR) block_norm_kernel(const NormParams p) {
    pdl_trigger();
    __shared__ float red[2][TPR > 32 ? 2 * TPR / 32 : 2];
    const int tid = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    pdl_wait();
    if (row >= p.T) return;   // a whole warp, or nobody
    const int ng = p.d / W;
    float r[G][W], b[G][W];
    if (p.x) {
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (tid + TPR * g < ng) load_vals<W>(p.x, row * p.ldx + (int64_t)(tid + TPR * g) * W, p.res_dtype, r[g]);
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int c = 0; c < W; ++c) r[g][c] = 0.0f;
    }
    if (p.b) {
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (tid + TPR * g < ng) load_vals<W>(p.b, row * p.ldb + (int64_t)(tid + TPR * g) * W, p.in_dtype, b[g]);
    }
    uint32_t mx = 0;
    if (p.b) {
        float scale = p.branch_scale;
        if (p.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (tid + TPR * g < ng)
#pragma unroll
                    for (int c = 0; c < W; ++c) ss = fmaf(b[g][c], b[g][c], ss);
            row_reduce<TPR>(ss, mx, red[0]);
            const float rb = __frsqrt_rn(ss / (float)p.d + p.eps);
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (tid + TPR * g < ng) {
                    float w[W];
                    load_vals<W>(p.w_post, (int64_t)(tid + TPR * g) * W, MOE_F32, w);
#pragma unroll
                    for (int c = 0; c < W; ++c) b[g][c] = b[g][c] * rb * (w[c] + p.weight_offset);
                }
        }
        float gt = 1.0f;
        if (p.gate_kind == MOE_GATE_TOKEN) {
            gt = reinterpret_cast<const float*>(p.gate)[row];
            if (p.gate_sigmoid) gt = 1.0f / (1.0f + expf(-gt));
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (tid + TPR * g < ng) {
                const int64_t at = (int64_t)(tid + TPR * g) * W;
                float gv[W];
                if (p.gate_kind == MOE_GATE_CHANNEL || p.gate_kind == MOE_GATE_ELEMENT) {
                    if (p.gate_kind == MOE_GATE_CHANNEL)
                        load_vals<W>(p.gate, at, MOE_F32, gv);
                    else
                        load_vals<W>(p.gate, row * p.ldg + at, p.in_dtype, gv);
                    if (p.gate_sigmoid) {
#pragma unroll
                        for (int c = 0; c < W; ++c) gv[c] = 1.0f / (1.0f + expf(-gv[c]));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < W; ++c) gv[c] = gt;
                }
#pragma unroll
                for (int c = 0; c < W; ++c)
                    r[g][c] = __fadd_rn(__fmul_rn(p.residual_scale, r[g][c]), __fmul_rn(scale, b[g][c] * gv[c]));
            }
    } else if (p.residual_scale != 1.0f) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int c = 0; c < W; ++c) r[g][c] = __fmul_rn(p.residual_scale, r[g][c]);
    }
    // the new stream, as it is kept; v = r (w_pre + offset) for the norm and, smoothed, for the codes
    float ss = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g)
        if (tid + TPR * g < ng) {
            const int64_t at = (int64_t)(tid + TPR * g) * W;
            round_vals<W>(p.res_dtype, r[g]);
            if (p.x_out) store_vals<W>(p.x_out, row * p.ldxo + at, p.res_dtype, r[g]);
            if (p.w_pre) {
                float w[W];
                load_vals<W>(p.w_pre, at, MOE_F32, w);
#pragma unroll
                for (int c = 0; c < W; ++c) {
                    ss = fmaf(r[g][c], r[g][c], ss);
                    r[g][c] = __fmul_rn(r[g][c], __fadd_rn(w[c], p.weight_offset));
                }
            }
            if (p.xq) {
                float w[W];
                if (p.inv_s) load_vals<W>(p.inv_s, at, MOE_F32, w);
#pragma unroll
                for (int c = 0; c < W; ++c) {
                    b[g][c] = p.inv_s ? __fmul_rn(r[g][c], w[c]) : r[g][c];
                    mx = max(mx, __float_as_uint(fabsf(b[g][c])));
                }
            }
        }
    if (!p.w_pre && !p.xq) return;
    mx = p.xq ? mx : 0u;
    row_reduce<TPR>(ss, mx, red[1]);
    const float rs = p.w_pre ? __frsqrt_rn(ss / (float)p.d + p.eps) : 1.0f;
    // codes: a row that holds an infinity or a NaN gets codes 0 and the scale NaN
    const bool finite = mx < 0x7f800000u;
    const float s = finite ? __fdiv_rn(__uint_as_float(mx), 127.0f) : 0.0f;
    const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
    if (p.xq && tid == 0) p.sx[row] = finite ? __fmul_rn(s, rs) : __int_as_float(0x7fc00000);
#pragma unroll
    for (int g = 0; g < G; ++g)
        if (tid + TPR * g < ng) {
            const int64_t at = (int64_t)(tid + TPR * g) * W;
            if (p.xq) {
                int8_t* dst = p.xq + row * p.ldq + at;
                if constexpr (W == 8) {
                    *reinterpret_cast<uint2*>(dst) =
                        s > 0.0f ? make_uint2(int8_codes4(b[g][0], b[g][1], b[g][2], b[g][3], s, inv),
                                              int8_codes4(b[g][4], b[g][5], b[g][6], b[g][7], s, inv))
                                 : make_uint2(0u, 0u);
                } else {
                    *dst = s > 0.0f ? (int8_t)quant_code_fast(b[g][0], s, inv) : (int8_t)0;
                }
            }
            if (p.n_out) {
#pragma unroll
                for (int c = 0; c < W; ++c) r[g][c] *= rs;
                store_vals<W>(p.n_out, row * p.ldn + at, p.out_dtype, r[g]);
            }
        }
}

// 8 values of a row as they are stored.
template <bool BF16>
struct Raw8;
template <>
struct Raw8<true> {
    uint4 q;
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Raw8<false> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
        a = q[0];
        b = q[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

__device__ __forceinline__ float gate_value(const NormParams& p, float g) {
    return p.gate_sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
}

// Rows on 16-byte boundaries.  A block (a warp for TPR = 32) takes every
// gridDim-th row; the loads of its next row are in flight while it works on the
// current one.  Thread t owns values [(t + TPR g) 8, + 8), g < G.
// BRANCH, POST, GATED, CODES: b, w_post, a gate and xq are given.  Measured against one block
// per row without the early loads, and 16 instead of 9 instructions per code:
// 16384 x 8192 bf16 with residual add and norm 299 -> %NL% us, the quantisation of
// 16384 x 4096 in front of a product %QB% -> %QA% us.
template <int TPR, int G, bool BF16, bool BRANCH, bool POST, bool GATED, bool CODES>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR, TPR == 32 ? 4 : 1024 / TPR)
    block_norm_rows_kernel(const NormParams p) {
    pdl_trigger();
    constexpr int NW = TPR / 32;
    __shared__ float red[TPR > 32 ? 2 : 1][TPR > 32 ? 2 * NW : 1], red_post[TPR > 32 ? NW : 1];
    const int tid = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t step = TPR == 32 ? (int64_t)gridDim.x * 8 : gridDim.x;
    const int ng = p.d / 8;
    const float rd = 1.0f / (float)p.d;
    int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 8 + warp : blockIdx.x;
    pdl_wait();
    Raw8<BF16> nx[G], nb[BRANCH ? G : 1];
    auto fetch = [&](int64_t r) {
        if (r >= p.T) return;
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (tid + TPR * g < ng) {
                if (p.x) nx[g].load(p.x, r * p.ldx + (tid + TPR * g) * 8);
                if (BRANCH) nb[g].load(p.b, r * p.ldb + (tid + TPR * g) * 8);
            }
    };
    fetch(row);
    for (int turn = 0; row < p.T; row += step, turn ^= 1) {   // the same number of rows for every thread of a row
        float r[G][8], b[BRANCH ? G : 1][8];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (p.x) {
                nx[g].get(r[g]);
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c) r[g][c] = 0.0f;
            }
            if (BRANCH) nb[g].get(b[g]);
        }
        fetch(row + step);
        if (BRANCH) {
            float rb = 1.0f;
            if (POST) {
                float ss = 0.0f;
#pragma unroll
                for (int g = 0; g < G; ++g)
                    if (tid + TPR * g < ng)
#pragma unroll
                        for (int c = 0; c < 8; ++c) ss = fmaf(b[g][c], b[g][c], ss);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if constexpr (TPR > 32) {
                    if (lane == 0) red_post[warp] = ss;
                    __syncthreads();
                    ss = 0.0f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) ss += red_post[w];
                }
                rb = __frsqrt_rn(ss * rd + p.eps);
            }
            float gt = 1.0f;
            if (GATED && p.gate_kind == MOE_GATE_TOKEN) gt = gate_value(p, reinterpret_cast<const float*>(p.gate)[row]);
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (tid + TPR * g < ng) {
                    const int at = (tid + TPR * g) * 8;
                    if (POST) {
                        float w[8];
                        load_vals<8>(p.w_post, at, MOE_F32, w);
#pragma unroll
                        for (int c = 0; c < 8; ++c) b[g][c] = b[g][c] * rb * (w[c] + p.weight_offset);
                    }
                    if (GATED && p.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) b[g][c] *= gt;
                    } else if (GATED) {
                        float gv[8];
                        if (p.gate_kind == MOE_GATE_CHANNEL)
                            load_vals<8>(p.gate, at, MOE_F32, gv);
                        else
                            load_vals<8>(p.gate, row * p.ldg + at, p.in_dtype, gv);
#pragma unroll
                        for (int c = 0; c < 8; ++c) b[g][c] *= gate_value(p, gv[c]);
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        r[g][c] = __fadd_rn(__fmul_rn(p.residual_scale, r[g][c]), __fmul_rn(p.branch_scale, b[g][c]));
                }
        } else if (p.residual_scale != 1.0f) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int c = 0; c < 8; ++c) r[g][c] = __fmul_rn(p.residual_scale, r[g][c]);
        }
        // the new stream, as it is kept; then v = r (w_pre + offset), its sum of squares and,
        // for the codes, the largest smoothed value
        float ss = 0.0f;
        uint32_t mx = 0;
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (tid + TPR * g < ng) {
                const int at = (tid + TPR * g) * 8;
                if (BRANCH || p.residual_scale != 1.0f) round_vals<8>(p.res_dtype, r[g]);
                if (p.x_out) store_vals<8>(p.x_out, row * p.ldxo + at, p.res_dtype, r[g]);
                if (p.w_pre) {
                    float w[8];
                    load_vals<8>(p.w_pre, at, MOE_F32, w);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        ss = fmaf(r[g][c], r[g][c], ss);
                        r[g][c] = __fmul_rn(r[g][c], __fadd_rn(w[c], p.weight_offset));
                    }
                }
                if (CODES) {
                    float w[8];
                    if (p.inv_s) load_vals<8>(p.inv_s, at, MOE_F32, w);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        mx = max(mx, __float_as_uint(fabsf(p.inv_s ? __fmul_rn(r[g][c], w[c]) : r[g][c])));
                }
            }
        if (!p.w_pre && !CODES) continue;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (CODES) mx = __reduce_max_sync(0xffffffffu, mx);
        if constexpr (TPR > 32) {
            // (the buffer of two rows ago: everybody has read it before the last row's barrier)
            if (lane == 0) {
                red[turn][warp] = ss;
                red[turn][NW + warp] = __uint_as_float(mx);
            }
            __syncthreads();
            ss = 0.0f;
            mx = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                ss += red[turn][w];
                if (CODES) mx = max(mx, __float_as_uint(red[turn][NW + w]));
            }
        }
        const float rs = p.w_pre ? __frsqrt_rn(ss * rd + p.eps) : 1.0f;
        // codes: a row that holds an infinity or a NaN gets codes 0 and the scale NaN
        const bool finite = mx < 0x7f800000u;
        const float s = CODES && finite ? __fdiv_rn(__uint_as_float(mx), 127.0f) : 0.0f;
        const float inv = CODES && s > 0.0f ? __frcp_rn(s) : 0.0f;
        if (CODES && tid == 0) p.sx[row] = finite ? __fmul_rn(s, rs) : __int_as_float(0x7fc00000);
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (tid + TPR * g < ng) {
                const int at = (tid + TPR * g) * 8;
                if (CODES) {
                    float v[8];
                    if (p.inv_s) load_vals<8>(p.inv_s, at, MOE_F32, v);
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = p.inv_s ? __fmul_rn(r[g][c], v[c]) : r[g][c];
                    *reinterpret_cast<uint2*>(p.xq + row * p.ldq + at) =
                        s > 0.0f ? make_uint2(int8_codes4(v[0], v[1], v[2], v[3], s, inv),
                                              int8_codes4(v[4], v[5], v[6], v[7], s, inv))
                                 : make_uint2(0u, 0u);
                }
                if (p.n_out) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) r[g][c] *= rs;
                    store_vals<8>(p.n_out, row * p.ldn + at, p.out_dtype, r[g]);
                }
            }
    }
}

template <int TPR, int G, int W>
cudaError_t run(const NormParams& p, cudaStream_t s) {
    const int64_t blocks = TPR == 32 ? (p.T + 7) / 8 : p.T;
    return launch_pdl(block_norm_kernel<TPR, G, W>, dim3((unsigned)blocks), dim3(TPR == 32 ? 256 : TPR), 0, s, p);
}

template <int TPR, int G, bool BF16, bool BRANCH, bool POST, bool GATED, bool CODES>
cudaError_t run_rows_as(const NormParams& p, cudaStream_t s) {
    auto kern = block_norm_rows_kernel<TPR, G, BF16, BRANCH, POST, GATED, CODES>;
    constexpr int kThreads = TPR == 32 ? 256 : TPR;
    // as many blocks as can be resident, by device
    static std::atomic<int> resident[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int most = resident[dev & 63].load(std::memory_order_relaxed);
    if (most == 0) {
        int per_sm = 0, sms = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, 0);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        most = per_sm > 0 ? per_sm * sms : sms;
        resident[dev & 63].store(most, std::memory_order_relaxed);
    }
    const int64_t blocks = TPR == 32 ? (p.T + 7) / 8 : p.T;
    return launch_pdl(kern, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, s, p);
}

template <int TPR, int G, bool BF16, bool BRANCH, bool POST, bool GATED>
cudaError_t run_rows_codes(const NormParams& p, cudaStream_t s) {
    return p.xq ? run_rows_as<TPR, G, BF16, BRANCH, POST, GATED, true>(p, s)
                : run_rows_as<TPR, G, BF16, BRANCH, POST, GATED, false>(p, s);
}

template <int TPR, int G, bool BF16>
cudaError_t run_rows(const NormParams& p, cudaStream_t s) {
    const bool gated = p.gate_kind != MOE_GATE_NONE;
    if (!p.b) return run_rows_codes<TPR, G, BF16, false, false, false>(p, s);
    if (!p.w_post)
        return gated ? run_rows_codes<TPR, G, BF16, true, false, true>(p, s)
                     : run_rows_codes<TPR, G, BF16, true, false, false>(p, s);
    return gated ? run_rows_codes<TPR, G, BF16, true, true, true>(p, s)
                 : run_rows_codes<TPR, G, BF16, true, true, false>(p, s);
}

template <bool BF16>
cudaError_t run_rows_by_size(const NormParams& p, cudaStream_t s) {
    const int d = p.d;
    if (d <= 256) return run_rows<32, 1, BF16>(p, s);
    if (d <= 1024) return run_rows<128, 1, BF16>(p, s);
    if (d <= 2048) return run_rows<256, 1, BF16>(p, s);
    if (d <= 4096) return run_rows<512, 1, BF16>(p, s);
    if (d <= 8192) return run_rows<1024, 1, BF16>(p, s);
    return run_rows<1024, 2, BF16>(p, s);
}

bool aligned(const void* p, int64_t ld, size_t esz) {
    return !p || (((uintptr_t)p & 15) == 0 && (ld * (int64_t)esz) % 16 == 0);
}

}  // namespace

cudaError_t launch_block_norm(const NormParams& p, cudaStream_t s) {
    const size_t eb = p.in_dtype == MOE_BF16 ? 2 : 4, er = p.res_dtype == MOE_BF16 ? 2 : 4,
                 eo = p.out_dtype == MOE_BF16 ? 2 : 4;
    const bool vec = p.d % 8 == 0 && aligned(p.b, p.ldb, eb) && aligned(p.x, p.ldx, er) &&
                     aligned(p.x_out, p.ldxo, er) && aligned(p.n_out, p.ldn, eo) && aligned(p.w_post, 0, 4) &&
                     aligned(p.w_pre, 0, 4) && aligned(p.inv_s, 0, 4) && aligned(p.xq, p.ldq, 1) &&
                     (p.gate_kind != MOE_GATE_ELEMENT || aligned(p.gate, p.ldg, eb)) &&
                     (p.gate_kind != MOE_GATE_CHANNEL || aligned(p.gate, 0, 4));
    const int d = p.d;
    if (vec) {
        const bool both = p.b && p.x;
        const int type = p.x ? p.res_dtype : p.in_dtype;
        if (!both || p.in_dtype == p.res_dtype)
            return type == MOE_BF16 ? run_rows_by_size<true>(p, s) : run_rows_by_size<false>(p, s);
        // a stream and a branch of different types
        if (d <= 512) return run<32, 2, 8>(p, s);
        if (d <= 2048) return run<256, 1, 8>(p, s);
        if (d <= 8192) return run<512, 2, 8>(p, s);
        return run<1024, 2, 8>(p, s);
    }
    if (d <= 256) return run<32, 8, 1>(p, s);
    if (d <= 1024) return run<256, 4, 1>(p, s);
    if (d <= 4096) return run<512, 8, 1>(p, s);
    return run<1024, 16, 1>(p, s);
}

}  // namespace moe
