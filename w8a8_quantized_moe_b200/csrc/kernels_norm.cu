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
// in registers between its two norms (a group of 8 values per 16-byte load).
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
                        s > 0.0f ? make_uint2(fmt_codes4<FMT_INT8>(b[g][0], b[g][1], b[g][2], b[g][3], s, inv),
                                              fmt_codes4<FMT_INT8>(b[g][4], b[g][5], b[g][6], b[g][7], s, inv))
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

template <int TPR, int G, int W>
cudaError_t run(const NormParams& p, cudaStream_t s) {
    const int64_t blocks = TPR == 32 ? (p.T + 7) / 8 : p.T;
    return launch_pdl(block_norm_kernel<TPR, G, W>, dim3((unsigned)blocks), dim3(TPR == 32 ? 256 : TPR), 0, s, p);
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
        if (d <= 512) return run<32, 2, 8>(p, s);
        if (d <= 1024) return run<128, 1, 8>(p, s);
        if (d <= 2048) return run<256, 1, 8>(p, s);
        if (d <= 4096) return run<256, 2, 8>(p, s);
        if (d <= 8192) return run<512, 2, 8>(p, s);
        return run<1024, 2, 8>(p, s);
    }
    if (d <= 256) return run<32, 8, 1>(p, s);
    if (d <= 1024) return run<256, 4, 1>(p, s);
    if (d <= 4096) return run<512, 8, 1>(p, s);
    return run<1024, 16, 1>(p, s);
}

}  // namespace moe
