// C ABI of the operators around the MoE layer: dense products in 8-bit
// integers, the norms around a block, and token sampling.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdlib>
#include <new>

#include "internal.h"

using namespace moe;

struct moe_w8a8_linear {
    moe_w8a8_linear_config cfg;
    int device;
    LinearTiles tiles;
    int8_t* w;          // tiles.w
    float* sw;          // tiles.sw
    float* bias;        // tiles.bias, or null
    float* inv_s;       // [k], or null: no smoothing
};

namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool dtype_ok(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
size_t dtype_bytes(int32_t t) { return t == MOE_BF16 ? 2 : 4; }
bool misaligned(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

// A row-major matrix argument: rows `ld` elements apart, each of d elements.
bool bad_rows(const void* p, int64_t ld, int64_t d, size_t esz) {
    return !p || ld < d || ld > ((int64_t)1 << 40) || misaligned(p, esz);
}

moe_status check_linear_config(const moe_w8a8_linear_config* c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (!(c->alpha >= 0.0f && c->alpha <= 1.0f)) return MOE_ERR_INVALID_ARG;
    if (!dtype_ok(c->in_dtype) || !dtype_ok(c->out_dtype)) return MOE_ERR_INVALID_ARG;
    if (c->n <= 0 || c->n > MOE_LINEAR_MAX_N || c->k <= 0 || c->k > MOE_LINEAR_MAX_K) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

void free_linear(moe_w8a8_linear* l) {
    if (!l) return;
    cudaFree(l->w);
    cudaFree(l->sw);
    cudaFree(l->bias);
    cudaFree(l->inv_s);
    cudaFree(l->tiles.status);
    delete l;
}

// A handle with its device memory, scales and bias cleared past the edges.
moe_status new_linear(const moe_w8a8_linear_config* cfg, const float* bias, bool smooth, cudaStream_t s,
                      moe_w8a8_linear** out) {
    moe_w8a8_linear* l = new (std::nothrow) moe_w8a8_linear();
    if (!l) return MOE_ERR_OOM;
    l->cfg = *cfg;
    LinearTiles& t = l->tiles;
    t.n = cfg->n;
    t.k = cfg->k;
    t.nb = (cfg->n + 255) / 256 * 2;
    t.kb = (cfg->k + 127) / 128;
    if (cudaGetDevice(&l->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&t.num_sms, cudaDevAttrMultiProcessorCount, l->device) != cudaSuccess) {
        free_linear(l);
        return MOE_ERR_CUDA;
    }
    const size_t chans = (size_t)t.nb * 128;
    if (cudaMalloc(&l->w, chans * t.kb * 128) != cudaSuccess || cudaMalloc(&l->sw, chans * 4) != cudaSuccess ||
        (bias && cudaMalloc(&l->bias, chans * 4) != cudaSuccess) ||
        (smooth && cudaMalloc(&l->inv_s, (size_t)cfg->k * 4) != cudaSuccess) ||
        cudaMalloc(&t.status, 64) != cudaSuccess) {
        cudaGetLastError();
        free_linear(l);
        return MOE_ERR_OOM;
    }
    t.w = l->w;
    t.sw = l->sw;
    t.bias = l->bias;
    if (cudaMemsetAsync(t.status, 0, 64, s) != cudaSuccess || cudaMemsetAsync(l->sw, 0, chans * 4, s) != cudaSuccess ||
        (bias && (cudaMemsetAsync(l->bias, 0, chans * 4, s) != cudaSuccess ||
                  cudaMemcpyAsync(l->bias, bias, (size_t)cfg->n * 4, cudaMemcpyDeviceToDevice, s) != cudaSuccess)) ||
        !linear_make_map(&t)) {
        cudaGetLastError();
        free_linear(l);
        return MOE_ERR_CUDA;
    }
    *out = l;
    return MOE_OK;
}

bool on_device(const moe_w8a8_linear* l) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == l->device;
}

// The codes of T tokens in the workspace: rows of k padded to 16 bytes, then the scales.
int64_t codes_ld(const moe_w8a8_linear* l) { return ((int64_t)l->cfg.k + 15) / 16 * 16; }
size_t scales_at(const moe_w8a8_linear* l, int32_t T) { return align_up((size_t)codes_ld(l) * T); }

}  // namespace

extern "C" {

moe_status moe_w8a8_linear_prepare(const moe_w8a8_linear_config* cfg, const float* w, const float* bias,
                                   const float* act_absmax, moe_stream_t stream, moe_w8a8_linear** out) {
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    const moe_status st = check_linear_config(cfg);
    if (st != MOE_OK) return st;
    if (!w || misaligned(w, 4) || misaligned(bias, 4) || misaligned(act_absmax, 4)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    moe_w8a8_linear* l = nullptr;
    const moe_status made = new_linear(cfg, bias, act_absmax != nullptr, s, &l);
    if (made != MOE_OK) return made;
    const int k = cfg->k, n = cfg->n;
    float *dev = nullptr, *host = nullptr;   // aw then s on the device; aw, ax, s, 1 / s on the host
    moe_status err = MOE_OK;
    if (act_absmax) {
        host = (float*)std::malloc((size_t)4 * k * 4);
        if (!host || cudaMalloc(&dev, (size_t)2 * k * 4) != cudaSuccess) err = MOE_ERR_OOM;
        if (err == MOE_OK && (launch_linear_input_absmax(w, k, n, dev, s) != cudaSuccess ||
                              cudaMemcpyAsync(host, dev, (size_t)k * 4, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
                              cudaMemcpyAsync(host + k, act_absmax, (size_t)k * 4, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
                              cudaStreamSynchronize(s) != cudaSuccess))
            err = MOE_ERR_CUDA;
        if (err == MOE_OK) {
            // s_j = ax^alpha / aw^(1 - alpha) in fp64, both statistics floored at 1e-5, as for the experts
            const double a = (double)cfg->alpha, floor_v = (double)1e-5f;
            for (int j = 0; j < k; ++j) {
                const double xv = host[k + j] > 1e-5f ? (double)host[k + j] : floor_v;
                const double wv = host[j] > 1e-5f ? (double)host[j] : floor_v;
                host[2 * k + j] = (float)(std::pow(xv, a) / std::pow(wv, 1.0 - a));
                host[3 * k + j] = (float)(1.0 / (double)host[2 * k + j]);
            }
            if (cudaMemcpyAsync(dev + k, host + 2 * k, (size_t)k * 4, cudaMemcpyHostToDevice, s) != cudaSuccess ||
                cudaMemcpyAsync(l->inv_s, host + 3 * k, (size_t)k * 4, cudaMemcpyHostToDevice, s) != cudaSuccess)
                err = MOE_ERR_CUDA;
        }
    }
    if (err == MOE_OK && launch_linear_quantize(w, act_absmax ? dev + k : nullptr, l->tiles, l->w, l->sw, s) != cudaSuccess)
        err = MOE_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess && err == MOE_OK) err = MOE_ERR_CUDA;
    cudaFree(dev);
    std::free(host);
    if (err != MOE_OK) {
        cudaGetLastError();
        free_linear(l);
        return err;
    }
    *out = l;
    return MOE_OK;
}

moe_status moe_w8a8_linear_prepare_codes(const moe_w8a8_linear_config* cfg, const int8_t* wq, const float* sw,
                                         const float* bias, const float* inv_s, moe_stream_t stream,
                                         moe_w8a8_linear** out) {
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    const moe_status st = check_linear_config(cfg);
    if (st != MOE_OK) return st;
    if (!wq || !sw || misaligned(sw, 4) || misaligned(bias, 4) || misaligned(inv_s, 4)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    moe_w8a8_linear* l = nullptr;
    const moe_status made = new_linear(cfg, bias, inv_s != nullptr, s, &l);
    if (made != MOE_OK) return made;
    if (launch_linear_tile(wq, l->tiles, l->w, s) != cudaSuccess ||
        cudaMemcpyAsync(l->sw, sw, (size_t)cfg->n * 4, cudaMemcpyDeviceToDevice, s) != cudaSuccess ||
        (inv_s && cudaMemcpyAsync(l->inv_s, inv_s, (size_t)cfg->k * 4, cudaMemcpyDeviceToDevice, s) != cudaSuccess) ||
        cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        free_linear(l);
        return MOE_ERR_CUDA;
    }
    *out = l;
    return MOE_OK;
}

size_t moe_w8a8_linear_workspace_size(const moe_w8a8_linear* l, int32_t max_tokens) {
    if (!l || max_tokens < 0) return 0;
    return align_up(scales_at(l, max_tokens) + (size_t)max_tokens * 4);
}

moe_status moe_w8a8_linear_forward_codes(const moe_w8a8_linear* l, const int8_t* xq, int64_t ldq, const float* sx,
                                         int32_t T, void* y, int64_t ldy, moe_stream_t stream) {
    if (!l || T < 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const moe_w8a8_linear_config& c = l->cfg;
    if (bad_rows(xq, ldq, c.k, 16) || ldq % 16 || !sx || misaligned(sx, 4) ||
        bad_rows(y, ldy, c.n, dtype_bytes(c.out_dtype)) || !on_device(l))
        return MOE_ERR_INVALID_ARG;
    return launch_linear(l->tiles, xq, ldq, sx, T, y, ldy, c.out_dtype, (cudaStream_t)stream) == cudaSuccess ? MOE_OK
                                                                                                         : MOE_ERR_CUDA;
}

moe_status moe_w8a8_linear_forward(const moe_w8a8_linear* l, const void* x, int64_t ldx, int32_t T, void* y, int64_t ldy,
                                   void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    if (!l || T < 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const moe_w8a8_linear_config& c = l->cfg;
    if (bad_rows(x, ldx, c.k, dtype_bytes(c.in_dtype)) || bad_rows(y, ldy, c.n, dtype_bytes(c.out_dtype)) || !workspace ||
        misaligned(workspace, kAlign) || !on_device(l))
        return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_w8a8_linear_workspace_size(l, T)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (linear_quantizes(l->tiles, x, ldx, T, c.in_dtype))
        return launch_linear_quantizing(l->tiles, x, ldx, c.in_dtype, l->inv_s, T, y, ldy, c.out_dtype,
                                        (cudaStream_t)stream) == cudaSuccess
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    NormParams q{};
    q.T = T;
    q.d = c.k;
    q.in_dtype = q.res_dtype = q.out_dtype = c.in_dtype;
    q.residual_scale = q.branch_scale = 1.0f;
    q.x = x;
    q.ldx = ldx;
    q.inv_s = l->inv_s;
    q.xq = (int8_t*)workspace;
    q.ldq = codes_ld(l);
    q.sx = (float*)((char*)workspace + scales_at(l, T));
    if (launch_block_norm(q, (cudaStream_t)stream) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_linear(l->tiles, q.xq, q.ldq, q.sx, T, y, ldy, c.out_dtype, (cudaStream_t)stream) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

moe_status moe_w8a8_linear_export(const moe_w8a8_linear* l, int8_t* wq, float* sw, float* inv_s, moe_stream_t stream) {
    if (!l || !on_device(l)) return MOE_ERR_INVALID_ARG;
    if (inv_s && !l->inv_s) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if ((wq && launch_linear_untile(l->tiles, wq, s) != cudaSuccess) ||
        (sw && cudaMemcpyAsync(sw, l->sw, (size_t)l->cfg.n * 4, cudaMemcpyDeviceToDevice, s) != cudaSuccess) ||
        (inv_s && cudaMemcpyAsync(inv_s, l->inv_s, (size_t)l->cfg.k * 4, cudaMemcpyDeviceToDevice, s) != cudaSuccess))
        return MOE_ERR_CUDA;
    return MOE_OK;
}

moe_status moe_w8a8_linear_check_status(const moe_w8a8_linear* l, moe_stream_t stream) {
    if (!l || !on_device(l)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    int32_t word = 0;
    if (cudaMemcpyAsync(&word, l->tiles.status, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (word != 0 && (cudaMemsetAsync(l->tiles.status, 0, 64, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess))
        return MOE_ERR_CUDA;
    return (moe_status)word;
}

void moe_w8a8_linear_destroy(moe_w8a8_linear* l) { free_linear(l); }

moe_status moe_w8a8_block_norm(const moe_w8a8_norm_config* c, const moe_w8a8_norm_io* io, int32_t T, moe_stream_t stream) {
    if (!c || !io || T < 0) return MOE_ERR_INVALID_ARG;
    if (!dtype_ok(c->in_dtype) || !dtype_ok(c->res_dtype) || !dtype_ok(c->out_dtype)) return MOE_ERR_INVALID_ARG;
    if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_ELEMENT || (c->gate_sigmoid != 0 && c->gate_sigmoid != 1))
        return MOE_ERR_INVALID_ARG;
    if (!(c->eps > 0.0f) || !std::isfinite(c->eps) || !std::isfinite(c->residual_scale) ||
        !std::isfinite(c->branch_scale) || !std::isfinite(c->weight_offset))
        return MOE_ERR_INVALID_ARG;
    if (c->d <= 0 || c->d > MOE_NORM_MAX_D) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    const int64_t d = c->d;
    const size_t eb = dtype_bytes(c->in_dtype), er = dtype_bytes(c->res_dtype), eo = dtype_bytes(c->out_dtype);
    if (!io->b && !io->x) return MOE_ERR_INVALID_ARG;
    if (io->b && bad_rows(io->b, io->ldb, d, eb)) return MOE_ERR_INVALID_ARG;
    if (io->x && bad_rows(io->x, io->ldx, d, er)) return MOE_ERR_INVALID_ARG;
    if (!io->b && (io->w_post || c->gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if ((c->gate != MOE_GATE_NONE) != (io->gate != nullptr)) return MOE_ERR_INVALID_ARG;
    if (c->gate == MOE_GATE_ELEMENT && bad_rows(io->gate, io->ldg, d, eb)) return MOE_ERR_INVALID_ARG;
    if (c->gate != MOE_GATE_ELEMENT && misaligned(io->gate, 4)) return MOE_ERR_INVALID_ARG;
    if (misaligned(io->w_post, 4) || misaligned(io->w_pre, 4) || misaligned(io->inv_s, 4) || misaligned(io->sx, 4))
        return MOE_ERR_INVALID_ARG;
    if (!io->x_out && !io->n_out && !io->xq) return MOE_ERR_INVALID_ARG;
    if (io->x_out && bad_rows(io->x_out, io->ldxo, d, er)) return MOE_ERR_INVALID_ARG;
    if (io->n_out && (!io->w_pre || bad_rows(io->n_out, io->ldn, d, eo))) return MOE_ERR_INVALID_ARG;
    if ((io->xq != nullptr) != (io->sx != nullptr) || (io->inv_s && !io->xq)) return MOE_ERR_INVALID_ARG;
    if (io->xq && (bad_rows(io->xq, io->ldq, d, 16) || io->ldq % 16)) return MOE_ERR_INVALID_ARG;
    NormParams p{};
    p.T = T;
    p.d = c->d;
    p.in_dtype = c->in_dtype;
    p.res_dtype = c->res_dtype;
    p.out_dtype = c->out_dtype;
    p.gate_kind = c->gate;
    p.gate_sigmoid = c->gate_sigmoid;
    p.eps = c->eps;
    p.residual_scale = c->residual_scale;
    p.branch_scale = c->branch_scale;
    p.weight_offset = c->weight_offset;
    p.b = io->b;
    p.x = io->x;
    p.gate = io->gate;
    p.w_post = io->w_post;
    p.w_pre = io->w_pre;
    p.inv_s = io->inv_s;
    p.x_out = io->x_out;
    p.n_out = io->n_out;
    p.xq = io->xq;
    p.sx = io->sx;
    p.ldb = io->ldb;
    p.ldx = io->ldx;
    p.ldg = io->ldg;
    p.ldxo = io->ldxo;
    p.ldn = io->ldn;
    p.ldq = io->ldq;
    return launch_block_norm(p, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_w8a8_sample(const moe_w8a8_sample_io* io, int32_t rows, int32_t vocab, int32_t dtype, moe_stream_t stream) {
    if (!io || rows < 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
    if (vocab <= 0 || vocab > kSampleMaxVocab || rows > MOE_SAMPLE_MAX_ROWS) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return MOE_OK;
    if (bad_rows(io->logits, io->ld, vocab, dtype_bytes(dtype)) || !io->u || misaligned(io->u, 4) || !io->token ||
        misaligned(io->token, 4) || misaligned(io->prob, 4) || misaligned(io->temperature, 4) || misaligned(io->top_k, 4) ||
        misaligned(io->top_p, 4) || misaligned(io->min_p, 4))
        return MOE_ERR_INVALID_ARG;
    if (io->allowed && bad_rows(io->allowed, io->ld_allowed, (vocab + 31) / 32, 4)) return MOE_ERR_INVALID_ARG;
    SampleParams p{};
    p.logits = io->logits;
    p.ld = io->ld;
    p.ld_allowed = io->ld_allowed;
    p.rows = rows;
    p.vocab = vocab;
    p.dtype = dtype;
    p.allowed = (const uint32_t*)io->allowed;
    p.temperature = io->temperature;
    p.top_k = io->top_k;
    p.top_p = io->top_p;
    p.min_p = io->min_p;
    p.u = io->u;
    p.token = io->token;
    p.prob = io->prob;
    return launch_sample(p, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
