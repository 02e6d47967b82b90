// amk_op_attention.cu -- amk_attention: causal attention with a sliding window
// and sinks over KV-cache rows.
#include <math.h>

#include "amk_ops.h"

namespace amk {
namespace {

struct AttnParams {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    int64_t q_ts, q_hs, o_ts, o_hs, k_hs, k_rs, v_hs, v_rs;
    int32_t T, pos, n_heads, group, hd, window, sinks;
    float scale_log2;  // scale * log2(e): weights are 2^(s - m)
};

__device__ __forceinline__ float bf16f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f_bf16(float f)
{
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The visible rows of position p: [0, s) and [lo, p].
__device__ __forceinline__ void visible(const AttnParams &a, int p, int &s, int &lo)
{
    lo = a.window && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    s = min(a.sinks, lo);
}

// ---- one output row by one warp -----------------------------------------------
// Any head size, stride and alignment: 32 rows at a time, lane j scores row j,
// then the lanes hold the output's elements and take the rows one after the
// other.  Rows outside the mask are not touched, so nothing they hold can
// reach the result.  qs: the warp's query in shared memory, pre-scaled, [hd].
constexpr int kMaxHd = 256;

__device__ void attend_row(const AttnParams &a, int t, int h, const float *qs)
{
    const int lane = threadIdx.x & 31;
    const int p = a.pos + t, hd = a.hd;
    int s, lo;
    visible(a, p, s, lo);
    const int n = s + (p - lo + 1);  // visible rows, the i-th being i < s ? i : i - s + lo
    const uint16_t *kb = a.k + (h / a.group) * a.k_hs, *vb = a.v + (h / a.group) * a.v_hs;
    float m = -INFINITY, l = 0.f, o[kMaxHd / 32] = {};
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        float sc = -INFINITY;
        if (i < n) {
            const uint16_t *kr = kb + (int64_t)(i < s ? i : i - s + lo) * a.k_rs;
            sc = 0.f;
            for (int d = 0; d < hd; ++d)
                sc = fmaf(qs[d], bf16f(kr[d]), sc);
        }
        float mx = sc;
        bool nan = i < n && sc != sc;  // a NaN among the visible rows is the row's result
        for (int off = 16; off; off >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        nan = __any_sync(0xffffffffu, nan);
        const float mn = nan ? NAN : fmaxf(m, mx);
        // -inf scores alone so far: weights of 0 and nothing to rescale
        const float base = mn == -INFINITY ? 0.f : mn;
        const float pr = i < n ? exp2_fast(sc - base) : 0.f;
        const float corr = exp2_fast(m - base);
        float sum = pr;
        for (int off = 16; off; off >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * corr + sum;
        m = mn;
#pragma unroll
        for (int e = 0; e < kMaxHd / 32; ++e)
            o[e] *= corr;
        const int nb = min(32, n - i0);
        for (int j = 0; j < nb; ++j) {
            const float w = __shfl_sync(0xffffffffu, pr, j);
            const int r = i0 + j;
            const uint16_t *vr = vb + (int64_t)(r < s ? r : r - s + lo) * a.v_rs;
#pragma unroll
            for (int e = 0; e < kMaxHd / 32; ++e)
                if (lane + 32 * e < hd)
                    o[e] = fmaf(w, bf16f(vr[lane + 32 * e]), o[e]);
        }
    }
    uint16_t *out = a.out + t * a.o_ts + h * a.o_hs;
#pragma unroll
    for (int e = 0; e < kMaxHd / 32; ++e)
        if (lane + 32 * e < hd)
            out[lane + 32 * e] = f_bf16(o[e] / l);
}

__global__ void __launch_bounds__(128) attn_rows(const AttnParams a)
{
    __shared__ float qs[4][kMaxHd];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.T * a.n_heads;
    for (int64_t r = (int64_t)blockIdx.x * 4 + warp; r < rows; r += (int64_t)gridDim.x * 4) {
        const int t = (int)(r / a.n_heads), h = (int)(r % a.n_heads);
        const uint16_t *q = a.q + t * a.q_ts + h * a.q_hs;
        for (int d = lane; d < a.hd; d += 32)
            qs[warp][d] = bf16f(q[d]) * a.scale_log2;
        __syncwarp();
        attend_row(a, t, h, qs[warp]);
        __syncwarp();
    }
}

int check_attention(const amk_attention_args *a)
{
    auto bad = [](const char *what) {
        return amk_set_error(AMK_ERR_INVALID_ARG, "amk_attention: %s", what);
    };
    if (!a)
        return bad("NULL arguments");
    if (a->n_tokens < 0 || a->n_heads < 1 || a->n_kv_heads < 1 || a->head_dim < 1)
        return bad("n_tokens < 0, or a head count or size < 1");
    if (a->n_heads % a->n_kv_heads)
        return bad("n_heads is not a multiple of n_kv_heads");
    if (a->head_dim > kMaxHd)
        return amk_set_error(AMK_ERR_UNSUPPORTED, "amk_attention: head_dim %d above %d",
                             a->head_dim, kMaxHd);
    if (a->window < 0 || a->sinks < 0)
        return bad("window or sinks < 0");
    if (a->pos < 0 || (int64_t)a->pos + a->n_tokens > a->kv_rows)
        return amk_set_error(AMK_ERR_POS_RANGE, "amk_attention: positions %d .. %lld outside the "
                             "%d rows", a->pos, (long long)a->pos + a->n_tokens - 1, a->kv_rows);
    if (!(a->scale >= 0.f) || isinf(a->scale))
        return bad("scale is negative or not finite");
    if (!a->q || !a->k || !a->v || !a->out)
        return bad("q, k, v or out is NULL");
    if (!aligned(a->q, 2) || !aligned(a->k, 2) || !aligned(a->v, 2) || !aligned(a->out, 2))
        return bad("a pointer is not aligned to its element");
    if (a->q_token_stride < 0 || a->q_head_stride < 0 || a->k_head_stride < 0 ||
        a->v_head_stride < 0 || a->k_row_stride < 0 || a->v_row_stride < 0)
        return bad("a stride is negative");
    // no two rows of out may overlap: tokens outside heads, or heads outside tokens
    const int64_t ts = a->out_token_stride, hs = a->out_head_stride, hd = a->head_dim;
    const bool th = (hs >= hd || a->n_heads == 1) &&
                    (ts >= (a->n_heads - 1) * hs + hd || a->n_tokens <= 1);
    const bool ht = (ts >= hd || a->n_tokens <= 1) &&
                    (hs >= (a->n_tokens - 1) * ts + hd || a->n_heads == 1);
    if (ts < 0 || hs < 0 || (!th && !ht))
        return bad("the rows of out overlap");
    return AMK_OK;
}

}  // namespace
}  // namespace amk

extern "C" int amk_attention(const amk_attention_args *a, void *cuda_stream)
{
    using namespace amk;
    const int rc = check_attention(a);
    if (rc != AMK_OK || a->n_tokens == 0)
        return rc;
    AttnParams p{};
    p.q = static_cast<const uint16_t *>(a->q);
    p.k = static_cast<const uint16_t *>(a->k);
    p.v = static_cast<const uint16_t *>(a->v);
    p.out = static_cast<uint16_t *>(a->out);
    p.q_ts = a->q_token_stride;
    p.q_hs = a->q_head_stride;
    p.o_ts = a->out_token_stride;
    p.o_hs = a->out_head_stride;
    p.k_hs = a->k_head_stride;
    p.k_rs = a->k_row_stride;
    p.v_hs = a->v_head_stride;
    p.v_rs = a->v_row_stride;
    p.T = a->n_tokens;
    p.pos = a->pos;
    p.n_heads = a->n_heads;
    p.group = a->n_heads / a->n_kv_heads;
    p.hd = a->head_dim;
    p.window = a->window;
    p.sinks = a->sinks;
    p.scale_log2 = (a->scale > 0.f ? a->scale : 1.f / sqrtf((float)a->head_dim)) * 1.4426950408889634f;
    const int64_t rows = (int64_t)a->n_tokens * a->n_heads;
    const unsigned grid = (unsigned)((rows + 3) / 4 < (1 << 20) ? (rows + 3) / 4 : (1 << 20));
    attn_rows<<<grid, 128, 0, static_cast<cudaStream_t>(cuda_stream)>>>(p);
    return launch_status(cudaGetLastError(), "amk_attention");
}
