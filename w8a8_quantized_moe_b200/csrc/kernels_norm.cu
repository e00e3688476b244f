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
// many rows on 16-byte boundaries, bound by memory and instructions, with few
// threads per row; block_norm_kernel for a few rows, bound by latency, with many,
// and for every type, stride and size.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

// W consecutive values from index i of a row, in one access (W = 8 in fp32: two).
template <int W>
__device__ __forceinline__ void load_vals(const void* p, int64_t i, int dtype, float (&v)[W]) {
    if constexpr (W == 8) {
        load8_act(p, i, dtype, v);
    } else if (dtype == MOE_BF16) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + i;
        if constexpr (W == 1) {
            v[0] = bf16_bits_to_f32(*q);
        } else {
            uint32_t w[W / 2];
            if constexpr (W == 4) {
                const uint2 u = *reinterpret_cast<const uint2*>(q);
                w[0] = u.x, w[W / 2 - 1] = u.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t*>(q);
            }
#pragma unroll
            for (int c = 0; c < W / 2; ++c) {
                v[2 * c] = __uint_as_float(w[c] << 16);
                v[2 * c + 1] = __uint_as_float(w[c] & 0xffff0000u);
            }
        }
    } else {
        const float* q = reinterpret_cast<const float*>(p) + i;
        if constexpr (W == 4) {
            const float4 u = *reinterpret_cast<const float4*>(q);
            v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
        } else if constexpr (W == 2) {
            const float2 u = *reinterpret_cast<const float2*>(q);
            v[0] = u.x, v[1] = u.y;
        } else {
            v[0] = *q;
        }
    }
}

// Round to the stored type; v keeps the rounded values.
template <int W>
__device__ __forceinline__ void round_vals(int dtype, float (&v)[W]) {
    if (dtype == MOE_BF16) {
#pragma unroll
        for (int c = 0; c < W; ++c) v[c] = __bfloat162float(__float2bfloat16_rn(v[c]));
    }
}

template <int W>
__device__ __forceinline__ void store_vals(void* p, int64_t i, int dtype, const float (&v)[W]) {
    if (dtype == MOE_BF16) {
        uint16_t* q = reinterpret_cast<uint16_t*>(p) + i;
        if constexpr (W == 1) {
            *q = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        } else {
            uint32_t w[W / 2];
#pragma unroll
            for (int c = 0; c < W / 2; ++c) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * c], v[2 * c + 1]);
                w[c] = *reinterpret_cast<const uint32_t*>(&h);
            }
            if constexpr (W == 8)
                *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
            else if constexpr (W == 4)
                *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t*>(q) = w[0];
        }
    } else {
        float* q = reinterpret_cast<float*>(p) + i;
        if constexpr (W >= 4) {
#pragma unroll
            for (int c = 0; c < W; c += 4)
                reinterpret_cast<float4*>(q)[c / 4] = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        } else if constexpr (W == 2) {
            *reinterpret_cast<float2*>(q) = make_float2(v[0], v[1]);
        } else {
            *q = v[0];
        }
    }
}

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
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

// The codes of eight values for scale s > 0 (inv = fp32(1 / s)): identical to
// quant_code of each.  t = v inv is within 2.3e-5 of the IEEE quotient where that
// is below 128 (quant_code_fast), so unless t lies within 3e-5 of a half-integer
// both round to the same integer, which the sum with 1.5 x 2^23 leaves in its low
// byte; the largest value has the quotient 127 and a rounding, so no clamp is
// needed.  Otherwise (or when 1 / s overflowed: the comparison fails) the
// quotients are formed.
__device__ __forceinline__ uint2 int8_codes8(const Pair (&v)[4], float s, float inv) {
    const Pair magic(12582912.0f, 12582912.0f), minus(-12582912.0f, -12582912.0f), one(-1.0f, -1.0f), r(inv, inv);
    float a[8];
    float off = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Pair t = v[i] * r;
        const Pair sum = t + magic;
        float d0, d1;
        fma2(sum + minus, one, t).get(d0, d1);   // t less the integer next to it
        off = max_abs_nan(max_abs_nan(off, d0), d1);
        sum.get(a[2 * i], a[2 * i + 1]);
    }
    uint32_t q[2];
    if (off < 0.49997f) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            q[i] = __byte_perm(__byte_perm(__float_as_uint(a[4 * i]), __float_as_uint(a[4 * i + 1]), 0x0040),
                               __byte_perm(__float_as_uint(a[4 * i + 2]), __float_as_uint(a[4 * i + 3]), 0x0040), 0x5410);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float e[4];
            v[2 * i].get(e[0], e[1]);
            v[2 * i + 1].get(e[2], e[3]);
            q[i] = pack4(quant_code(e[0], s), quant_code(e[1], s), quant_code(e[2], s), quant_code(e[3], s));
        }
    }
    return make_uint2(q[0], q[1]);
}

__device__ __forceinline__ float gate_value(const NormParams& p, float g) {
    return p.gate_sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
}

// TPR threads per row, each with G groups of W values: group g of thread t is
// values [(t + TPR g) W, ... + W).  Rows per block: 8 when a warp owns a row,
// else one.  TYPE: the one type of the branch, the stream and n_out, or -1 (each
// as the parameters say).  What a call asks for is decided between the passes over
// a thread's groups, not inside them: with single values (rows off every boundary)
// a decision per value cost more than the value (16384 x 4095 bf16 with codes and
// n_out: 320 us, 147 instructions per value; now 231).
template <int TPR, int G, int W, int TYPE>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR, TPR == 32 ? 4 : W == 1 && TPR < 1024 ? 1536 / TPR : 1024 / TPR)
    block_norm_kernel(const NormParams p) {
    const int in_dtype = TYPE < 0 ? p.in_dtype : TYPE, res_dtype = TYPE < 0 ? p.res_dtype : TYPE,
              out_dtype = TYPE < 0 ? p.out_dtype : TYPE;
    pdl_trigger();
    __shared__ float red[2][TPR > 32 ? 2 * TPR / 32 : 2];
    const int tid = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    pdl_wait();
    if (row >= p.T) return;   // a whole warp, or nobody
    const int ng = p.d / W;
    float r[G][W], b[G][W];
    // f(group, index of its first value) for the thread's groups.  Past the row's end a
    // group stands for the row's last one when it loads and holds zeros, so that the
    // passes between loads and stores are free of branches.
    auto all = [&](auto f) {
#pragma unroll
        for (int g = 0; g < G; ++g) f(g, min((tid + TPR * g) * W, p.d - W));
    };
    auto each = [&](auto f) {
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (tid + TPR * g < ng) f(g, (tid + TPR * g) * W);
    };
    auto load = [&](float (&v)[G][W], const void* from, int64_t ld, int dtype) {
        all([&](int g, int at) {
            load_vals<W>(from, row * ld + at, dtype, v[g]);
            if (tid + TPR * g >= ng) {
#pragma unroll
                for (int c = 0; c < W; ++c) v[g][c] = 0.0f;
            }
        });
    };
    auto times = [&](float (&v)[G][W], const float* weights, float offset) {
        all([&](int g, int at) {
            float w[W];
            load_vals<W>(weights, at, MOE_F32, w);
#pragma unroll
            for (int c = 0; c < W; ++c) v[g][c] = __fmul_rn(v[g][c], offset != 0.0f ? __fadd_rn(w[c], offset) : w[c]);
        });
    };
    if (p.x) {
        load(r, p.x, p.ldx, res_dtype);
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int c = 0; c < W; ++c) r[g][c] = 0.0f;
    }
    if (p.b) load(b, p.b, p.ldb, in_dtype);
    uint32_t mx = 0;
    if (p.b) {
        if (p.w_post) {
            float ss = 0.0f;
            all([&](int g, int) {
#pragma unroll
                for (int c = 0; c < W; ++c) ss = fmaf(b[g][c], b[g][c], ss);
            });
            row_reduce<TPR>(ss, mx, red[0]);
            const float rb = __frsqrt_rn(ss / (float)p.d + p.eps);
            all([&](int g, int) {
#pragma unroll
                for (int c = 0; c < W; ++c) b[g][c] *= rb;
            });
            times(b, p.w_post, p.weight_offset);
        }
        if (p.gate_kind == MOE_GATE_TOKEN) {
            const float gt = gate_value(p, reinterpret_cast<const float*>(p.gate)[row]);
            all([&](int g, int) {
#pragma unroll
                for (int c = 0; c < W; ++c) b[g][c] *= gt;
            });
        } else if (p.gate_kind != MOE_GATE_NONE) {
            const bool element = p.gate_kind == MOE_GATE_ELEMENT;
            all([&](int g, int at) {
                float gv[W];
                if (element)
                    load_vals<W>(p.gate, row * p.ldg + at, in_dtype, gv);
                else
                    load_vals<W>(p.gate, at, MOE_F32, gv);
#pragma unroll
                for (int c = 0; c < W; ++c) b[g][c] *= gate_value(p, gv[c]);
            });
        }
        all([&](int g, int) {
#pragma unroll
            for (int c = 0; c < W; ++c)
                r[g][c] = __fadd_rn(__fmul_rn(p.residual_scale, r[g][c]), __fmul_rn(p.branch_scale, b[g][c]));
        });
    } else if (p.residual_scale != 1.0f) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int c = 0; c < W; ++c) r[g][c] = __fmul_rn(p.residual_scale, r[g][c]);
    }
    // the new stream, as it is kept; v = r (w_pre + offset) for the norm and, smoothed, for the codes
    all([&](int g, int) { round_vals<W>(res_dtype, r[g]); });
    if (p.x_out) each([&](int g, int at) { store_vals<W>(p.x_out, row * p.ldxo + at, res_dtype, r[g]); });
    if (!p.w_pre && !p.xq) return;
    float ss = 0.0f, big = 0.0f;
    if (p.w_pre) {
        all([&](int g, int) {
#pragma unroll
            for (int c = 0; c < W; ++c) ss = fmaf(r[g][c], r[g][c], ss);
        });
        // past the row's end an infinite weight or gate of its last values has made 0 a NaN, which is not
        // the row's (rare, so asked once: zeros kept there by a pass of their own cost 3 to 5%)
        if (isnan(ss)) {
            ss = 0.0f;
            each([&](int g, int) {
#pragma unroll
                for (int c = 0; c < W; ++c) ss = fmaf(r[g][c], r[g][c], ss);
            });
        }
        times(r, p.w_pre, p.weight_offset);
    }
    if (p.xq) {
        all([&](int g, int) {
#pragma unroll
            for (int c = 0; c < W; ++c) b[g][c] = r[g][c];
        });
        if (p.inv_s) times(b, p.inv_s, 0.0f);
        all([&](int g, int) {
#pragma unroll
            for (int c = 0; c < W; ++c) big = max_abs_nan(big, b[g][c]);
        });
    }
    mx = __float_as_uint(big);
    row_reduce<TPR>(ss, mx, red[1]);
    const float rs = p.w_pre ? __frsqrt_rn(ss / (float)p.d + p.eps) : 1.0f;
    if (p.xq) {
        // a row that holds an infinity or a NaN gets codes 0 and the scale NaN
        const bool finite = mx < 0x7f800000u;
        const float s = finite ? __fdiv_rn(__uint_as_float(mx), 127.0f) : 0.0f;
        if (tid == 0) p.sx[row] = finite ? __fmul_rn(s, rs) : __int_as_float(0x7fc00000);
        int8_t* dst = p.xq + row * p.ldq;
        uint32_t q[G][W == 8 ? 2 : 1];
        if (s > 0.0f) {
            const float inv = __frcp_rn(s);
            if constexpr (W == 8) {
                all([&](int g, int) {
                    const Pair v[4] = {Pair(b[g][0], b[g][1]), Pair(b[g][2], b[g][3]), Pair(b[g][4], b[g][5]),
                                       Pair(b[g][6], b[g][7])};
                    const uint2 two = int8_codes8(v, s, inv);
                    q[g][0] = two.x, q[g][W == 8 ? 1 : 0] = two.y;
                });
            } else {
                // as in int8_codes8, with one look at how near any of the thread's values is to a half-integer
                float off = 0.0f;
                all([&](int g, int) {
                    uint32_t word = 0;
#pragma unroll
                    for (int c = 0; c < W; ++c) {
                        const float t = __fmul_rn(b[g][c], inv), a = __fadd_rn(t, 12582912.0f);
                        off = max_abs_nan(off, __fsub_rn(t, __fsub_rn(a, 12582912.0f)));
                        word |= (__float_as_uint(a) & 0xffu) << (8 * c);
                    }
                    q[g][0] = word;
                });
                if (!(off < 0.49997f))
                    all([&](int g, int) {
                        uint32_t word = 0;
#pragma unroll
                        for (int c = 0; c < W; ++c) word |= ((uint32_t)quant_code(b[g][c], s) & 0xffu) << (8 * c);
                        q[g][0] = word;
                    });
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g) q[g][0] = q[g][W == 8 ? 1 : 0] = 0u;
        }
        each([&](int g, int at) {
            if constexpr (W == 8)
                *reinterpret_cast<uint2*>(dst + at) = make_uint2(q[g][0], q[g][W == 8 ? 1 : 0]);
            else if constexpr (W == 4)
                *reinterpret_cast<uint32_t*>(dst + at) = q[g][0];
            else if constexpr (W == 2)
                *reinterpret_cast<uint16_t*>(dst + at) = (uint16_t)q[g][0];
            else
                dst[at] = (int8_t)q[g][0];
        });
    }
    if (p.n_out)
        each([&](int g, int at) {
#pragma unroll
            for (int c = 0; c < W; ++c) r[g][c] *= rs;
            store_vals<W>(p.n_out, row * p.ldn + at, out_dtype, r[g]);
        });
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
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = q;
    }
    __device__ __forceinline__ void get(Pair (&v)[4]) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = Pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    __device__ __forceinline__ void set(const Pair (&v)[4]) {   // rounds
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            v[i].get(a, b);
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        q = make_uint4(w[0], w[1], w[2], w[3]);
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
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
        q[0] = a;
        q[1] = b;
    }
    __device__ __forceinline__ void get(Pair (&v)[4]) const {
        v[0] = Pair(a.x, a.y);
        v[1] = Pair(a.z, a.w);
        v[2] = Pair(b.x, b.y);
        v[3] = Pair(b.z, b.w);
    }
    __device__ __forceinline__ void set(const Pair (&v)[4]) {
        v[0].get(a.x, a.y);
        v[1].get(a.z, a.w);
        v[2].get(b.x, b.y);
        v[3].get(b.z, b.w);
    }
};

// 8 fp32 weights (plus `offset`).
__device__ __forceinline__ void load_weights(const float* p, int at, float offset, Pair (&w)[4]) {
    Raw8<false> q;
    q.load(p, at);
    q.get(w);
    if (offset != 0.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = w[i] + Pair(offset, offset);
    }
}

// Many rows on 16-byte boundaries, stream and branch of one type.  TPR threads
// per row (a warp, or a block of that many), G groups of 8 values each: thread t
// owns values [(t + TPR g) 8, + 8).  Few threads with many values each, so that a
// row's fixed work (two reductions, a division) is shared by many values; the row
// is kept as it is stored (the new stream is rounded to its type anyway), twice
// unpacked, so that it takes 4 registers per 8 values of bf16.  Measured, 16384 x
// 4096 bf16, us: residual add and norm 80 (6.7 TB/s), with both norms and a gate
// 92, codes alone 51 to 55 (instructions: 20 per value, issue slots 63% used), codes
// of a norm 60, smoothed 79 (each weight vector is read again for each row); blocks
// that stay and take every n-th row 97, 101 and 56; twice the values per thread 100,
// 130 and 63 (registers); 512 threads per row, the next row's loads early, 88, 144
// and 87 (a row's fixed work).
// BRANCH, POST, CODES: b, w_post and xq are given.
template <int TPR, int G, bool BF16, bool BRANCH, bool POST, bool CODES>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) block_norm_rows_kernel(const NormParams p) {
    pdl_trigger();
    constexpr int NW = TPR / 32;
    __shared__ float red[TPR > 32 ? 2 * NW : 1], red_post[TPR > 32 ? NW : 1];
    const int tid = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 4 + warp : blockIdx.x;
    const int ng = p.d / 8;
    const float rd = 1.0f / (float)p.d;
    pdl_wait();
    if (row >= p.T) return;   // a whole warp, or nobody
    Raw8<BF16> r[G], b[BRANCH ? G : 1];
    float gt = 1.0f, rb = 1.0f;
#pragma unroll
    for (int g = 0; g < G; ++g)
        if (tid + TPR * g < ng) {
            const int at = (tid + TPR * g) * 8;
            if (BRANCH) b[g].load(p.b, row * p.ldb + at);
            if (p.x) r[g].load(p.x, row * p.ldx + at);
        }
    if (BRANCH && p.gate_kind == MOE_GATE_TOKEN) gt = gate_value(p, reinterpret_cast<const float*>(p.gate)[row]);
    if (POST) {
        Pair sum(0.0f, 0.0f);
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (tid + TPR * g < ng) {
                Pair v[4];
                b[g].get(v);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum = fma2(v[i], v[i], sum);
            }
        float s0, s1;
        sum.get(s0, s1);
        float ss = warp_sum_f(s0 + s1);
        if constexpr (TPR > 32) {
            if (lane == 0) red_post[warp] = ss;
            __syncthreads();
            ss = warp_sum_f(lane < NW ? red_post[lane] : 0.0f);
        }
        rb = __frsqrt_rn(ss * rd + p.eps);
    }
    // the new stream, as it is kept; its sum of squares and, for the codes, the
    // largest value of r (w_pre + offset) inv_s
    Pair sum(0.0f, 0.0f);
    float big = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g)
        if (tid + TPR * g < ng) {
            const int at = (tid + TPR * g) * 8;
            Pair v[4];
            if (p.x) {
                r[g].get(v);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = Pair(p.residual_scale, p.residual_scale) * v[i];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = Pair(0.0f, 0.0f);
            }
            if (BRANCH) {
                Pair u[4];
                b[g].get(u);
                if (POST) {
                    Pair w[4];
                    load_weights(p.w_post, at, p.weight_offset, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = u[i] * Pair(rb, rb) * w[i];
                }
                if (p.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = u[i] * Pair(gt, gt);
                } else if (p.gate_kind != MOE_GATE_NONE) {
                    Pair gv[4];
                    if (p.gate_kind == MOE_GATE_CHANNEL) {
                        load_weights(reinterpret_cast<const float*>(p.gate), at, 0.0f, gv);
                    } else {
                        Raw8<BF16> q;
                        q.load(p.gate, row * p.ldg + at);
                        q.get(gv);
                    }
                    if (p.gate_sigmoid) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float a, c;
                            gv[i].get(a, c);
                            gv[i] = Pair(gate_value(p, a), gate_value(p, c));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = u[i] * gv[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = v[i] + Pair(p.branch_scale, p.branch_scale) * u[i];
            }
            r[g].set(v);
            if (p.x_out) r[g].store(p.x_out, row * p.ldxo + at);
            if (BF16) r[g].get(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = fma2(v[i], v[i], sum);
            if (CODES) {
                Pair w[4];
                if (p.w_pre) {
                    load_weights(p.w_pre, at, p.weight_offset, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = v[i] * w[i];
                }
                if (p.inv_s) {
                    load_weights(p.inv_s, at, 0.0f, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = v[i] * w[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a, c;
                    v[i].get(a, c);
                    big = max_abs_nan(max_abs_nan(big, a), c);
                }
            }
        }
    if (!p.w_pre && !CODES) return;
    float s0, s1;
    sum.get(s0, s1);
    float ss = p.w_pre ? warp_sum_f(s0 + s1) : 0.0f;
    uint32_t mx = CODES ? __reduce_max_sync(0xffffffffu, __float_as_uint(big)) : 0u;
    if constexpr (TPR > 32) {
        if (lane == 0) {
            red[warp] = ss;
            if (CODES) red[NW + warp] = __uint_as_float(mx);
        }
        __syncthreads();
        if (p.w_pre) ss = warp_sum_f(lane < NW ? red[lane] : 0.0f);
        if (CODES) mx = __reduce_max_sync(0xffffffffu, lane < NW ? __float_as_uint(red[NW + lane]) : 0u);
    }
    const float rs = p.w_pre ? __frsqrt_rn(ss * rd + p.eps) : 1.0f;
    // codes: a row that holds an infinity or a NaN gets codes 0 and the scale NaN
    const bool finite = mx < 0x7f800000u;
    const float s = CODES && finite ? __fdiv_rn(__uint_as_float(mx), 127.0f) : 0.0f;
    const float inv = CODES && s > 0.0f ? __frcp_rn(s) : 0.0f;
    if (CODES && tid == 0) p.sx[row] = finite ? __fmul_rn(s, rs) : __int_as_float(0x7fc00000);
    if (!CODES && !p.n_out) return;
#pragma unroll
    for (int g = 0; g < G; ++g)
        if (tid + TPR * g < ng) {
            const int at = (tid + TPR * g) * 8;
            Pair v[4], w[4];
            r[g].get(v);
            if (p.w_pre) {
                load_weights(p.w_pre, at, p.weight_offset, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = v[i] * w[i];
            }
            if (p.n_out) {
                Pair n[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) n[i] = v[i] * Pair(rs, rs);
                if (p.out_dtype == MOE_BF16) {
                    Raw8<true> o;
                    o.set(n);
                    o.store(p.n_out, row * p.ldn + at);
                } else {
                    Raw8<false> o;
                    o.set(n);
                    o.store(p.n_out, row * p.ldn + at);
                }
            }
            if (CODES) {
                if (p.inv_s) {
                    load_weights(p.inv_s, at, 0.0f, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = v[i] * w[i];
                }
                *reinterpret_cast<uint2*>(p.xq + row * p.ldq + at) =
                    s > 0.0f ? int8_codes8(v, s, inv) : make_uint2(0u, 0u);
            }
        }
}

template <int TPR, int G, int W, int TYPE>
cudaError_t run_as(const NormParams& p, cudaStream_t s) {
    const int64_t blocks = TPR == 32 ? (p.T + 7) / 8 : p.T;
    return launch_pdl(block_norm_kernel<TPR, G, W, TYPE>, dim3((unsigned)blocks), dim3(TPR == 32 ? 256 : TPR), 0, s, p);
}

template <int TPR, int G, int W>
cudaError_t run(const NormParams& p, cudaStream_t s) {
    const int type = p.res_dtype;   // the new stream's, also where there is no x
    if ((p.b && p.in_dtype != type) || (p.n_out && p.out_dtype != type)) return run_as<TPR, G, W, -1>(p, s);
    return type == MOE_BF16 ? run_as<TPR, G, W, MOE_BF16>(p, s) : run_as<TPR, G, W, MOE_F32>(p, s);
}

template <int TPR, int G, bool BF16, bool BRANCH, bool POST, bool CODES>
cudaError_t run_rows_as(const NormParams& p, cudaStream_t s) {
    auto kern = block_norm_rows_kernel<TPR, G, BF16, BRANCH, POST, CODES>;
    constexpr int kThreads = TPR == 32 ? 128 : TPR;
    const int64_t blocks = TPR == 32 ? (p.T + 3) / 4 : p.T;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, s, p);
}

template <int TPR, int G, bool BF16, bool BRANCH, bool POST>
cudaError_t run_rows_codes(const NormParams& p, cudaStream_t s) {
    return p.xq ? run_rows_as<TPR, G, BF16, BRANCH, POST, true>(p, s) : run_rows_as<TPR, G, BF16, BRANCH, POST, false>(p, s);
}

template <int TPR, int G, bool BF16>
cudaError_t run_rows(const NormParams& p, cudaStream_t s) {
    if (!p.b) return run_rows_codes<TPR, G, BF16, false, false>(p, s);
    return p.w_post ? run_rows_codes<TPR, G, BF16, true, true>(p, s) : run_rows_codes<TPR, G, BF16, true, false>(p, s);
}

template <bool BF16>
cudaError_t run_rows_by_size(const NormParams& p, cudaStream_t s) {
    const int d = p.d;
    if (d <= 256) return run_rows<32, 1, BF16>(p, s);
    if (d <= 512) return run_rows<32, 2, BF16>(p, s);
    if (d <= 1024) return run_rows<32, 4, BF16>(p, s);
    if (d <= 2048) return run_rows<64, 4, BF16>(p, s);
    if (d <= 4096) return run_rows<128, 4, BF16>(p, s);
    if (d <= 8192) return run_rows<256, 4, BF16>(p, s);
    return run_rows<512, 4, BF16>(p, s);
}

// Rows of W values (times the size of one) stay on their boundaries.
bool aligned(const void* p, int64_t ld, size_t esz, int W) {
    return !p || (((uintptr_t)p % (esz * W)) == 0 && ld % W == 0);
}

bool in_groups(const NormParams& p, int W) {
    auto size = [](int dtype) -> size_t { return dtype == MOE_BF16 ? 2 : 4; };
    // (fp32 groups of 8 are two accesses of 16 bytes)
    auto ok = [&](const void* q, int64_t ld, size_t esz) { return aligned(q, ld, esz, std::min(W, (int)(16 / esz))); };
    return p.d % W == 0 && ok(p.b, p.ldb, size(p.in_dtype)) && ok(p.x, p.ldx, size(p.res_dtype)) &&
           ok(p.x_out, p.ldxo, size(p.res_dtype)) && ok(p.n_out, p.ldn, size(p.out_dtype)) && ok(p.w_post, 0, 4) &&
           ok(p.w_pre, 0, 4) && ok(p.inv_s, 0, 4) &&
           (p.gate_kind != MOE_GATE_ELEMENT || ok(p.gate, p.ldg, size(p.in_dtype))) &&
           (p.gate_kind != MOE_GATE_CHANNEL || ok(p.gate, 0, 4));   // (xq is on 16 bytes with its rows)
}

// Rows from which few threads per row take over: one count for every width.  Measured
// around it, residual add and norm of bf16, us a launch with many threads per row / with
// few: 200 x 1024 2.4 / 3.3, 200 x 4096 3.3 / 3.8, 200 x 8192 5.9 / 4.9, 200 x 16384 8.3 /
// 5.9; 600 x 1024 3.3 / 3.6, 600 x 4096 6.8 / 5.3, 600 x 8192 12.7 / 7.8; 64 x 8192 3.5 /
// 3.6.  (Rows of at most 512 values do better with few threads at any count, 1 x 512 2.3 /
// 2.1, rows of 1024 with many up to 1200; both by less than a call takes on the host.)
constexpr int64_t kManyRows = 200;

}  // namespace

cudaError_t launch_block_norm(const NormParams& p, cudaStream_t s) {
    const int d = p.d;
    // For a few rows, the block whose threads hold the row in one group of 8 each (a warp
    // up to 512 values, 1024 threads at most).  Half the threads with two groups each: 64 x
    // 1024 2.6 us instead of 2.2, 64 x 4096 2.9 instead of 2.8, 64 x 8192 3.7 instead of
    // 3.5 (but 199 x 8192 4.6 instead of 5.9).  Narrower groups: as many threads, more
    // groups each.
    if (in_groups(p, 8)) {
        if (p.T >= kManyRows && (!p.b || p.in_dtype == p.res_dtype))
            return p.res_dtype == MOE_BF16 ? run_rows_by_size<true>(p, s) : run_rows_by_size<false>(p, s);
        if (d <= 512) return run<32, 2, 8>(p, s);
        if (d <= 1024) return run<128, 1, 8>(p, s);
        if (d <= 2048) return run<256, 1, 8>(p, s);
        if (d <= 4096) return run<512, 1, 8>(p, s);
        if (d <= 8192) return run<1024, 1, 8>(p, s);
        return run<1024, 2, 8>(p, s);
    }
    if (in_groups(p, 4)) {
        if (d <= 512) return run<32, 4, 4>(p, s);
        if (d <= 1024) return run<128, 2, 4>(p, s);
        if (d <= 4096) return run<256, 4, 4>(p, s);
        return run<1024, 4, 4>(p, s);
    }
    if (in_groups(p, 2)) {
        if (d <= 512) return run<32, 8, 2>(p, s);
        if (d <= 1024) return run<128, 4, 2>(p, s);
        if (d <= 4096) return run<512, 4, 2>(p, s);
        return run<1024, 8, 2>(p, s);
    }
    if (d <= 256) return run<32, 8, 1>(p, s);
    if (d <= 1024) return run<256, 4, 1>(p, s);
    if (d <= 4096) return run<512, 8, 1>(p, s);
    return run<1024, 16, 1>(p, s);
}

}  // namespace moe
