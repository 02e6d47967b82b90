// amk_op_linear.cu -- amk_linear: the matrix product with its epilogue.
#include <cuda_fp16.h>
#include <math.h>

#include "amk_ops.h"

namespace amk {
namespace {

constexpr int kQ4GroupLog2 = 7;

__device__ __forceinline__ float bf16f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
// round to nearest even; the cast of a NaN stays a NaN
__device__ __forceinline__ uint16_t f_bf16(float f)
{
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
    return r;
}

// The epilogue of one output: act(a + bias) [* (u + up_bias)] [+ residual].
struct Epilogue {
    const uint16_t *bias, *up_bias;
    const uint16_t *w_scale, *up_scale;  // fp16 row scales (W8A16), or null
    const void *residual;
    void *y;
    int64_t ldr, ldy;
    int32_t m, n, act, gated, res_f32, y_f32;
};

__device__ __forceinline__ float activate(int act, float v)
{
    if (act == AMK_ACT_SILU)
        return v / (1.f + __expf(-v));
    if (act == AMK_ACT_GELU)
        return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    if (act == AMK_ACT_RELU)
        return v < 0.f ? 0.f : v;  // a NaN stays
    return v;
}

__device__ __forceinline__ void store_out(const Epilogue &e, int row, int col, float a, float u)
{
    if (row >= e.m || col >= e.n)
        return;
    if (e.w_scale)
        a *= __half2float(__ushort_as_half(e.w_scale[col]));
    if (e.bias)
        a += bf16f(e.bias[col]);
    a = activate(e.act, a);
    if (e.gated) {
        if (e.up_scale)
            u *= __half2float(__ushort_as_half(e.up_scale[col]));
        if (e.up_bias)
            u += bf16f(e.up_bias[col]);
        a *= u;
    }
    if (e.residual) {
        const int64_t i = row * e.ldr + col;
        a += e.res_f32 ? static_cast<const float *>(e.residual)[i]
                       : bf16f(static_cast<const uint16_t *>(e.residual)[i]);
    }
    const int64_t o = row * e.ldy + col;
    if (e.y_f32)
        static_cast<float *>(e.y)[o] = a;
    else
        static_cast<uint16_t *>(e.y)[o] = f_bf16(a);
}

// ---- the kernel for any alignment ---------------------------------------------
// A 64 x 64 tile of y per CTA, K in blocks of 32, bf16 mma.sync with fp32
// accumulators.  Every element is loaded by itself, so no address needs more
// than its element's alignment.  Codes enter the product as the integers they
// are (exact in bf16); int8 row scales are applied to the sums, and the sums
// of each group of 128 inputs of an int4 row are scaled by themselves.
constexpr int kGM = 64, kGN = 64, kGK = 32, kGS = kGK + 8;  // kGS: padded row (elements)

struct GenericParams {
    const uint16_t *x;
    const void *w, *up;
    const uint16_t *w_gs, *up_gs;  // int4 group scales [n][groups]
    int64_t ldx;
    int32_t k, groups;
    Epilogue e;
};

template <int QUANT>
__device__ __forceinline__ uint16_t weight_bf16(const void *w, int64_t row, int k, int64_t K)
{
    if (QUANT == AMK_QUANT_BF16)
        return static_cast<const uint16_t *>(w)[row * K + k];
    int q;
    if (QUANT == AMK_QUANT_W8A16) {
        q = static_cast<const int8_t *>(w)[row * K + k];
    } else {
        const int b = static_cast<const uint8_t *>(w)[row * (K / 2) + (k >> 1)];
        q = (int)((unsigned)((k & 1) ? b >> 4 : b & 15) << 28) >> 28;
    }
    return f_bf16((float)q);
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4],
                                            const uint32_t (&b)[2])
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

template <int QUANT, int MATS>
__global__ void __launch_bounds__(128) linear_generic(const GenericParams p)
{
    __shared__ __align__(16) uint16_t xs[kGM * kGS];
    __shared__ __align__(16) uint16_t ws[MATS][kGN * kGS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * kGN;
    const int wm = (warp & 1) * 32, wn = (warp >> 1) * 32;
    for (int m0 = blockIdx.y * kGM; m0 < p.e.m; m0 += gridDim.y * kGM) {
        float acc[MATS][2][4][4] = {};
        float part[QUANT == AMK_QUANT_W4A16 ? MATS : 1][2][4][4] = {};
        for (int k0 = 0; k0 < p.k; k0 += kGK) {
            uint16_t xr[kGM * kGK / 128], wr[MATS][kGN * kGK / 128];
#pragma unroll
            for (int i = 0; i < kGM * kGK / 128; ++i) {
                const int r = i * 4 + warp, k = k0 + lane;
                xr[i] = m0 + r < p.e.m && k < p.k ? p.x[(m0 + r) * p.ldx + k] : (uint16_t)0;
#pragma unroll
                for (int b = 0; b < MATS; ++b)
                    wr[b][i] = n0 + r < p.e.n && k < p.k
                                   ? weight_bf16<QUANT>(b ? p.up : p.w, n0 + r, k, p.k)
                                   : (uint16_t)0;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kGM * kGK / 128; ++i) {
                const int r = i * 4 + warp;
                xs[r * kGS + lane] = xr[i];
#pragma unroll
                for (int b = 0; b < MATS; ++b)
                    ws[b][r * kGS + lane] = wr[b][i];
            }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < kGK; kk += 16) {
                uint32_t a[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        a[i][r] = *reinterpret_cast<const uint32_t *>(
                            &xs[(wm + i * 16 + g + (r & 1) * 8) * kGS + kk + 2 * t + (r >> 1) * 8]);
#pragma unroll
                for (int b = 0; b < MATS; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t f[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            f[r] = *reinterpret_cast<const uint32_t *>(
                                &ws[b][(wn + j * 8 + g) * kGS + kk + 2 * t + r * 8]);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            mma_16x8x16(QUANT == AMK_QUANT_W4A16 ? part[b][i][j] : acc[b][i][j],
                                        a[i], f);
                    }
            }
            if constexpr (QUANT == AMK_QUANT_W4A16) {
                if (((k0 + kGK) & (kQ4Group - 1)) == 0 || k0 + kGK >= p.k) {
                    const int grp = k0 >> kQ4GroupLog2;
#pragma unroll
                    for (int b = 0; b < MATS; ++b)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int n = n0 + wn + j * 8 + 2 * t + c;
                                const float s =
                                    n < p.e.n ? __half2float(__ushort_as_half(
                                                    (b ? p.up_gs : p.w_gs)[(int64_t)n * p.groups + grp]))
                                              : 0.f;
#pragma unroll
                                for (int i = 0; i < 2; ++i)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        acc[b][i][j][c + 2 * h] += s * part[b][i][j][c + 2 * h];
                                        part[b][i][j][c + 2 * h] = 0.f;
                                    }
                            }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    store_out(p.e, m0 + wm + i * 16 + g + (r >> 1) * 8,
                              n0 + wn + j * 8 + 2 * t + (r & 1), acc[0][i][j][r],
                              MATS == 2 ? acc[MATS - 1][i][j][r] : 0.f);
    }
}

template <int QUANT>
cudaError_t launch_generic(const GenericParams &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)((p.e.n + kGN - 1) / kGN),
                    (unsigned)min((p.e.m + kGM - 1) / kGM, 65535));
    if (p.e.gated)
        linear_generic<QUANT, 2><<<grid, 128, 0, stream>>>(p);
    else
        linear_generic<QUANT, 1><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

int check_linear(const amk_linear_args *a)
{
    auto bad = [](const char *what) {
        return amk_set_error(AMK_ERR_INVALID_ARG, "amk_linear: %s", what);
    };
    if (!a)
        return bad("NULL arguments");
    if (a->m < 0 || a->n < 1 || a->k < 1)
        return bad("m < 0, n < 1 or k < 1");
    if (a->quant < AMK_QUANT_BF16 || a->quant > AMK_QUANT_W4A16)
        return bad("unknown weight format");
    if (a->quant == AMK_QUANT_W4A16 && a->k % 2)
        return bad("int4 rows need an even number of inputs");
    if (a->act < AMK_ACT_NONE || a->act > AMK_ACT_RELU)
        return bad("unknown activation");
    if (a->y_type < AMK_DT_BF16 || a->y_type > AMK_DT_F32 || a->residual_type < AMK_DT_BF16 ||
        a->residual_type > AMK_DT_F32)
        return bad("unknown type of y or residual");
    if (!a->x || !a->w || !a->y)
        return bad("x, w or y is NULL");
    if (a->ldx < a->k || a->ldy < a->n || (a->residual && a->ldr < a->n))
        return bad("a row stride is less than the row");
    if (a->quant != AMK_QUANT_BF16 && (!a->w_scale || (a->up && !a->up_scale)))
        return bad("int8 and int4 weights need their scales");
    if (!a->up && a->up_bias)
        return bad("up_bias without up");
    const uintptr_t yb = a->y_type == AMK_DT_F32 ? 4 : 2, rb = a->residual_type == AMK_DT_F32 ? 4 : 2;
    if (!aligned(a->x, 2) || !aligned(a->y, yb) || !aligned(a->residual, rb) ||
        !aligned(a->bias, 2) || !aligned(a->up_bias, 2) || !aligned(a->w_scale, 2) ||
        !aligned(a->up_scale, 2) ||
        (a->quant == AMK_QUANT_BF16 && (!aligned(a->w, 2) || !aligned(a->up, 2))))
        return bad("a pointer is not aligned to its element");
    return AMK_OK;
}

}  // namespace
}  // namespace amk

extern "C" int amk_linear(const amk_linear_args *a, void *cuda_stream)
{
    using namespace amk;
    const int rc = check_linear(a);
    if (rc != AMK_OK || a->m == 0)
        return rc;
    GenericParams p{};
    p.x = static_cast<const uint16_t *>(a->x);
    p.w = a->w;
    p.up = a->up;
    p.ldx = a->ldx;
    p.k = a->k;
    p.groups = (a->k + kQ4Group - 1) / kQ4Group;
    p.e.bias = static_cast<const uint16_t *>(a->bias);
    p.e.up_bias = static_cast<const uint16_t *>(a->up_bias);
    if (a->quant == AMK_QUANT_W8A16) {
        p.e.w_scale = static_cast<const uint16_t *>(a->w_scale);
        p.e.up_scale = static_cast<const uint16_t *>(a->up_scale);
    } else if (a->quant == AMK_QUANT_W4A16) {
        p.w_gs = static_cast<const uint16_t *>(a->w_scale);
        p.up_gs = static_cast<const uint16_t *>(a->up_scale);
    }
    p.e.residual = a->residual;
    p.e.y = a->y;
    p.e.ldr = a->ldr;
    p.e.ldy = a->ldy;
    p.e.m = a->m;
    p.e.n = a->n;
    p.e.act = a->act;
    p.e.gated = a->up != nullptr;
    p.e.res_f32 = a->residual_type == AMK_DT_F32;
    p.e.y_f32 = a->y_type == AMK_DT_F32;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    cudaError_t e;
    if (a->quant == AMK_QUANT_W8A16)
        e = launch_generic<AMK_QUANT_W8A16>(p, st);
    else if (a->quant == AMK_QUANT_W4A16)
        e = launch_generic<AMK_QUANT_W4A16>(p, st);
    else
        e = launch_generic<AMK_QUANT_BF16>(p, st);
    return launch_status(e, "amk_linear");
}
