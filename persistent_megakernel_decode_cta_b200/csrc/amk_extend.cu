// amk_extend.cu -- the multi-token step: the decoder's layers over several
// tokens, by amk_linear and amk_attention, and the small kernels between them.
//
// The residual stream is fp32, as in the single-token step; what a matrix
// product takes (normed x, rotated q, attention and SwiGLU outputs) is rounded
// to bf16, the type that the tensor cores multiply, where the single-token
// step keeps fp32 (or 15 bits).  K and V are rounded once, into the cache.
#include <math.h>

#include "amk_extend.h"
#include "amk_ops.cuh"

namespace amk {
namespace {

using namespace ops;

// Cosine and sine of pos * theta^(-2 e / hd), the angle reduced in fp64.
__global__ void rope_table(float2 *out, int n, int pos, int half, double theta)
{
    pdl_wait();
    pdl_launch();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n * half)
        return;
    const double a = (pos + i / half) * pow(theta, -(double)(i % half) / half);
    const double turns = a * 0.15915494309189533577;
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    out[i] = make_float2(c, s);
}

// Sum over the CTA's 256 threads in a fixed order.
__device__ float block_sum(float v)
{
    __shared__ float part[8];
#pragma unroll
    for (int off = 16; off; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w)
        s += part[w];
    return s;
}

// xn = bf16(x / sqrt(mean x^2 + eps) * gain), one token to a CTA.  EMBED: x is
// first set to the token's embedding row.
template <bool EMBED>
__global__ void __launch_bounds__(256) norm_rows(float *x, const uint16_t *embed,
                                                 const int32_t *tokens, const uint16_t *gain,
                                                 uint16_t *xn, int hidden, float eps)
{
    pdl_wait();
    pdl_launch();
    const int t = blockIdx.x;
    float *xr = x + (int64_t)t * hidden;
    const uint16_t *er = EMBED ? embed + (int64_t)tokens[t] * hidden : nullptr;
    float s = 0.f;
    if (!EMBED && hidden % 4 == 0 && hidden <= 4096 && ((uintptr_t)gain & 7) == 0) {
        // a row in registers: one latency for its loads
        const int quads = hidden / 4;
        float4 v[4];
        uint2 gn[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = threadIdx.x + j * 256;
            v[j] = i < quads ? reinterpret_cast<const float4 *>(xr)[i] : make_float4(0, 0, 0, 0);
            gn[j] = i < quads ? reinterpret_cast<const uint2 *>(gain)[i] : make_uint2(0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s = fmaf(v[j].x, v[j].x, s);
            s = fmaf(v[j].y, v[j].y, s);
            s = fmaf(v[j].z, v[j].z, s);
            s = fmaf(v[j].w, v[j].w, s);
        }
        const float r = rsqrtf(block_sum(s) / (float)hidden + eps);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = threadIdx.x + j * 256;
            if (i < quads) {
                uint2 o;
                o.x = f_bf16(v[j].x * r * bf16f((uint16_t)gn[j].x)) |
                      (uint32_t)f_bf16(v[j].y * r * bf16f((uint16_t)(gn[j].x >> 16))) << 16;
                o.y = f_bf16(v[j].z * r * bf16f((uint16_t)gn[j].y)) |
                      (uint32_t)f_bf16(v[j].w * r * bf16f((uint16_t)(gn[j].y >> 16))) << 16;
                reinterpret_cast<uint2 *>(xn + (int64_t)t * hidden)[i] = o;
            }
        }
        return;
    }
    for (int i = threadIdx.x; i < hidden; i += 256) {
        float v;
        if (EMBED) {
            v = bf16f(er[i]);
            xr[i] = v;
        } else {
            v = xr[i];
        }
        s = fmaf(v, v, s);
    }
    const float r = rsqrtf(block_sum(s) / (float)hidden + eps);
    for (int i = threadIdx.x; i < hidden; i += 256)  // each thread's own elements again
        xn[(int64_t)t * hidden + i] = f_bf16(xr[i] * r * bf16f(gain[i]));
}

// Rotates q and k (pairs i, i + hd / 2), and writes q, and k and v into the
// cache rows pos + t: a thread to a pair of a token, so that each has one
// latency; parts CTAs to a token.
__global__ void __launch_bounds__(256) rope_append(const float *qkv, const float2 *rope,
                                                   uint16_t *q, uint16_t *kc, uint16_t *vc, int nh,
                                                   int nkv, int hd, int pos, int max_ctx,
                                                   int parts)
{
    pdl_wait();
    pdl_launch();
    const int t = blockIdx.x / parts, half = hd / 2;
    const int i = blockIdx.x % parts * 256 + threadIdx.x;
    const float *src = qkv + (int64_t)t * (nh + 2 * nkv) * hd;
    const float2 *cs = rope + (int64_t)t * half;
    const int h = i / half, e = i - h * half;
    if (h < nh + nkv) {
        const float a = src[h * hd + e], b = src[h * hd + e + half];
        const float2 r = cs[e];
        uint16_t *dst = h < nh ? q + ((int64_t)t * nh + h) * hd
                               : kc + ((int64_t)(h - nh) * max_ctx + pos + t) * hd;
        dst[e] = f_bf16(a * r.x - b * r.y);
        dst[e + half] = f_bf16(b * r.x + a * r.y);
    } else if (h < nh + 2 * nkv) {
        uint16_t *dst = vc + ((int64_t)(h - nh - nkv) * max_ctx + pos + t) * hd;
        dst[e] = f_bf16(src[h * hd + e]);
        dst[e + half] = f_bf16(src[h * hd + e + half]);
    }
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

template <typename... P, typename... A>
int launch(void (*kernel)(P...), int grid, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, P(args)...), "amk_extend");
}

}  // namespace

size_t extend_bytes(const amk_config &c, int32_t chunk)
{
    const size_t n = (size_t)chunk, qo = (size_t)c.n_heads * c.head_dim;
    const size_t qkv = qo + 2 * (size_t)c.n_kv_heads * c.head_dim;
    return up256(4 * n) + up256(8 * n * (c.head_dim / 2)) + up256(4 * n * c.hidden) +
           up256(2 * n * c.hidden) + up256(4 * n * qkv) + 2 * up256(2 * n * qo) +
           up256(2 * n * c.ffn);
}

ExtendBuffers extend_buffers(const amk_config &c, int32_t chunk, void *block)
{
    const size_t n = (size_t)chunk, qo = (size_t)c.n_heads * c.head_dim;
    const size_t qkv = qo + 2 * (size_t)c.n_kv_heads * c.head_dim;
    uint8_t *p = static_cast<uint8_t *>(block);
    auto take = [&p](size_t bytes) {
        void *at = p;
        p += up256(bytes);
        return at;
    };
    ExtendBuffers b;
    b.chunk = chunk;
    b.tokens = static_cast<int32_t *>(take(4 * n));
    b.rope = static_cast<float2 *>(take(8 * n * (c.head_dim / 2)));
    b.x = static_cast<float *>(take(4 * n * c.hidden));
    b.xn = static_cast<uint16_t *>(take(2 * n * c.hidden));
    b.qkv = static_cast<float *>(take(4 * n * qkv));
    b.q = static_cast<uint16_t *>(take(2 * n * qo));
    b.attn = static_cast<uint16_t *>(take(2 * n * qo));
    b.act = static_cast<uint16_t *>(take(2 * n * c.ffn));
    return b;
}

int extend_chunk(const amk_config &c, const ModelWeights &w, const ExtendBuffers &b, uint16_t *kv,
                 int32_t n, int32_t pos, int32_t window, int32_t sinks, int32_t n_logits,
                 float *logits, cudaStream_t stream)
{
    const int hd = c.head_dim, half = hd / 2, qo = c.n_heads * hd, ko = c.n_kv_heads * hd;
    const int qkv = qo + 2 * ko, parts = (qkv / 2 + 255) / 256;
    const size_t block = (size_t)c.n_kv_heads * c.max_ctx * hd;  // K or V of a layer
    auto gain = [](const void *p) { return static_cast<const uint16_t *>(p); };
    auto linear = [&](const uint16_t *x, int k, const void *mat, const void *scale, int out,
                      float *y, int ldy, const float *residual) {
        amk_linear_args a{};
        a.x = x;
        a.w = mat;
        a.w_scale = scale;
        a.residual = residual;
        a.y = y;
        a.ldx = k;
        a.ldr = a.ldy = ldy;
        a.m = n;
        a.n = out;
        a.k = k;
        a.quant = c.quant;
        a.residual_type = a.y_type = AMK_DT_F32;
        return amk_linear(&a, stream);
    };
    auto sc = [&](int m, int l) { return w.scale[m].empty() ? nullptr : w.scale[m][l]; };
    int rc = launch(rope_table, (n * half + 255) / 256, stream, b.rope, n, pos, half,
                    (double)c.rope_theta);
    if (rc == AMK_OK)
        rc = launch(norm_rows<true>, n, stream, b.x, gain(w.embed), b.tokens, gain(w.norm[0][0]),
                    b.xn, c.hidden, c.rms_eps);
    for (int l = 0; l < c.n_layers && rc == AMK_OK; ++l) {
        uint16_t *kc = kv + (size_t)l * 2 * block, *vc = kc + block;
        if ((rc = linear(b.xn, c.hidden, w.mat[W_Q][l], sc(W_Q, l), qo, b.qkv, qkv, nullptr)) ||
            (rc = linear(b.xn, c.hidden, w.mat[W_K][l], sc(W_K, l), ko, b.qkv + qo, qkv, nullptr)) ||
            (rc = linear(b.xn, c.hidden, w.mat[W_V][l], sc(W_V, l), ko, b.qkv + qo + ko, qkv,
                         nullptr)) ||
            (rc = launch(rope_append, n * parts, stream, b.qkv, b.rope, b.q, kc, vc, c.n_heads,
                         c.n_kv_heads, hd, pos, c.max_ctx, parts)))
            break;
        amk_attention_args a{};
        a.q = b.q;
        a.k = kc;
        a.v = vc;
        a.out = b.attn;
        a.q_token_stride = a.out_token_stride = qo;
        a.q_head_stride = a.out_head_stride = a.k_row_stride = a.v_row_stride = hd;
        a.k_head_stride = a.v_head_stride = (int64_t)c.max_ctx * hd;
        a.n_tokens = n;
        a.pos = pos;
        a.n_heads = c.n_heads;
        a.n_kv_heads = c.n_kv_heads;
        a.head_dim = hd;
        a.kv_rows = c.max_ctx;
        a.window = window;
        a.sinks = sinks;
        if ((rc = amk_attention(&a, stream)) ||
            (rc = linear(b.attn, qo, w.mat[W_O][l], sc(W_O, l), c.hidden, b.x, c.hidden, b.x)) ||
            (rc = launch(norm_rows<false>, n, stream, b.x, nullptr, nullptr, gain(w.norm[1][l]),
                         b.xn, c.hidden, c.rms_eps)))
            break;
        amk_linear_args f{};
        f.x = b.xn;
        f.w = w.mat[W_GATE][l];
        f.w_scale = sc(W_GATE, l);
        f.up = w.mat[W_UP][l];
        f.up_scale = sc(W_UP, l);
        f.y = b.act;
        f.ldx = c.hidden;
        f.ldy = c.ffn;
        f.m = n;
        f.n = c.ffn;
        f.k = c.hidden;
        f.quant = c.quant;
        f.act = AMK_ACT_SILU;
        f.y_type = AMK_DT_BF16;
        const void *next = l + 1 < c.n_layers ? w.norm[0][l + 1] : w.final_norm;
        if ((rc = amk_linear(&f, stream)) ||
            (rc = linear(b.act, c.ffn, w.mat[W_DOWN][l], sc(W_DOWN, l), c.hidden, b.x, c.hidden,
                         b.x)) ||
            (rc = launch(norm_rows<false>, n, stream, b.x, nullptr, nullptr, gain(next), b.xn,
                         c.hidden, c.rms_eps)))
            break;
    }
    if (rc != AMK_OK || n_logits == 0)
        return rc;
    amk_linear_args h{};
    h.x = b.xn + (size_t)(n - n_logits) * c.hidden;
    h.w = c.tied_embeddings ? w.embed : w.lm_head;
    h.quant = c.tied_embeddings ? (int)AMK_QUANT_BF16 : c.quant;
    h.w_scale = h.quant == AMK_QUANT_BF16 ? nullptr : w.lm_head_scale;
    h.y = logits;
    h.ldx = c.hidden;
    h.ldy = c.vocab;
    h.m = n_logits;
    h.n = c.vocab;
    h.k = c.hidden;
    h.y_type = AMK_DT_F32;
    return amk_linear(&h, stream);
}

}  // namespace amk
