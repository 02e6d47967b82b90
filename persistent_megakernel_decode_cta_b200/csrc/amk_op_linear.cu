// amk_op_linear.cu -- amk_linear: argument checks, the choice of a kernel, and
// the kernel for any alignment.
#include <atomic>
#include <math.h>

#include "amk_op_linear.cuh"

namespace amk {
namespace linear {
namespace {

constexpr int kQ4GroupLog2 = 7;
// The kernels count n and k in 32 bits, up to a tile or eight stages (of 128
// inputs) and a share's last steps beyond them: less than 4096 in all.
constexpr int kMaxSide = INT32_MAX - 4095;

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
    for (int64_t m0 = (int64_t)blockIdx.y * kGM; m0 < p.e.m; m0 += (int64_t)gridDim.y * kGM) {
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
                                    n < p.e.n ? fp16f((b ? p.up_gs : p.w_gs)[(int64_t)n * p.groups + grp])
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
                {
                    const int64_t m = m0 + wm + i * 16 + g + (r >> 1) * 8;
                    const int n = n0 + wn + j * 8 + 2 * t + (r & 1);
                    if (m < p.e.m && n < p.e.n)
                        emit(p.e, row_const(p.e, n), (int)m, n, acc[0][i][j][r],
                             MATS == 2 ? acc[MATS - 1][i][j][r] : 0.f);
                }
    }
}

template <int QUANT>
cudaError_t launch_generic(const GenericParams &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)((p.e.n + kGN - 1) / kGN),
                    (unsigned)min(((int64_t)p.e.m + kGM - 1) / kGM, (int64_t)65535));
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
    if (a->n > kMaxSide || a->k > kMaxSide)
        return amk_set_error(AMK_ERR_UNSUPPORTED, "amk_linear: n %d, k %d: at most %d", a->n, a->k,
                             kMaxSide);
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

// ---- the tensor-core kernel ----------------------------------------------------

bool fits_tensor_cores(const amk_linear_args *a)
{
    const int64_t row = a->quant == AMK_QUANT_BF16    ? 2 * (int64_t)a->k
                        : a->quant == AMK_QUANT_W8A16 ? a->k
                        : a->k % 2                    ? 1
                                                      : a->k / 2;
    return aligned(a->x, 16) && aligned(a->w, 16) && aligned(a->up, 16) && row % 16 == 0 &&
           (a->m == 1 || a->ldx % 8 == 0);
}

// The variant, the CTAs of a cluster that share a tile, and the grid.
struct Choice {
    Variant v;
    int split, grid;
};

// What a variant's CTA costs, in us (fitted to some 1100 calls of 60 shapes on
// B200, 17 .. 2000 tokens; the choices made by it take 2 % longer than the
// fastest variant of each, 26 % at worst): its start and end, each block of 64
// inputs, each CTA of its cluster, and how much of a block's time a second CTA
// on the same SM adds.
struct Cost {
    float fixed, block, member, shared;
};
constexpr Cost kSplitCost[3][4] = {  // weight format; 16, 32, 64, 128 tokens
    {{4.9f, 0.20f, 0.12f, 0.28f}, {5.8f, 0.30f, 0.04f, 0.20f},
     {6.5f, 0.31f, 0.10f, 0.27f}, {9.9f, 0.26f, 0.02f, 0.f}},
    {{5.3f, 0.21f, 0.32f, 0.62f}, {7.4f, 0.19f, 0.50f, 0.f},
     {8.6f, 0.20f, 0.59f, 0.f}, {10.5f, 0.26f, 0.87f, 0.f}},
    {{5.0f, 0.23f, 0.30f, 0.52f}, {6.9f, 0.22f, 0.50f, 0.f},
     {8.0f, 0.25f, 0.61f, 0.f}, {10.3f, 0.31f, 0.80f, 0.f}}};
constexpr Cost kWalkCost[3][2] = {  // weight format; sums left to the tensor cores, or promoted
    {{6.1f, 0.36f}, {6.1f, 0.40f}}, {{5.4f, 0.36f}, {4.9f, 0.27f}}, {{3.8f, 0.36f}, {3.8f, 0.36f}}};

Choice choose(const amk_linear_args *a, int sms)
{
    const int rows = a->up ? 64 : 128;
    const int64_t tn = ((int64_t)a->n + rows - 1) / rows;
    const bool codes = a->quant != AMK_QUANT_BF16;
    const int blocks = (a->k + 63) / 64;
    Choice best{};
    double least = 1e300;
    auto consider = [&](const Variant &v, int split, int64_t tiles, int64_t room, double us) {
        if (us < least && tiles * split <= INT32_MAX) {
            least = us;
            best.v = v;
            best.split = split;
            best.grid = (int)(v.split ? tiles * split : tiles < room ? tiles : room);
        }
    };
    for (int i = 0; i < 4; ++i) {
        const int nt = 16 << i, per_sm = nt <= (codes ? 16 : 64) ? 2 : 1;
        const int64_t tiles = tn * (((int64_t)a->m + nt - 1) / nt);
        const Cost &c = kSplitCost[a->quant][i];
        for (int split = 1; split <= 8 && split <= (a->k + 127) / 128; split *= 2) {
            // clusters of four and of eight leave some SMs of each GPC over
            const int64_t room = (int64_t)per_sm * (split <= 2 ? sms : split == 4 ? sms - 4 : sms * 7 / 8);
            const int64_t ctas = tiles * split, waves = (ctas + room - 1) / room;
            const double block = c.block * (per_sm == 2 && ctas > sms ? 1 + c.shared : 1.0);
            consider({nt, true, true}, split, tiles, room,
                     waves * (c.fixed + (blocks + split - 1) / split * block) + split * c.member);
        }
    }
    // a wide tile's gate and up meet after its last sum (40 tokens, int8: 8192 x
    // 2048 with a gate 21.7 us walking, 16384 x 2048 without 18.3 us)
    const double gate = a->up ? 4. : 0.;
    const bool must = a->y_type == AMK_DT_F32 || a->quant == AMK_QUANT_W4A16;
    for (int promote = must; promote <= (must || codes); ++promote) {
        const int nt = !codes ? 256 : promote ? 128 : 192;
        const int64_t tiles = tn * (((int64_t)a->m + nt - 1) / nt);
        const Cost &c = kWalkCost[a->quant][promote];
        consider({nt, false, promote != 0}, 1, tiles, sms,
                 c.fixed + gate + (tiles + sms - 1) / sms * (double)blocks * c.block);
    }
    return best;
}

int launch_few(const amk_linear_args *a, const Epilogue &e, cudaStream_t stream)
{
    SkinnyParams p{};
    p.x = static_cast<const uint16_t *>(a->x);
    p.w = a->w;
    p.up = a->up;
    p.w_gs = static_cast<const uint16_t *>(a->w_scale);
    p.up_gs = static_cast<const uint16_t *>(a->up_scale);
    p.ldx = a->ldx;
    p.k = a->k;
    p.groups = (a->k + kQ4Group - 1) / kQ4Group;
    p.row_bytes = a->quant == AMK_QUANT_BF16    ? 2 * (int64_t)a->k
                  : a->quant == AMK_QUANT_W8A16 ? a->k
                                                : a->k / 2;
    p.e = e;
    const int rows = a->up ? kSkinnyRows / 2 : kSkinnyRows;
    const int64_t tiles = ((int64_t)a->n + rows - 1) / rows;
    // more CTAs to a tile as long as they all run at once and a warp keeps some
    // steps (64 bytes of a row); fewer steps only where the CTAs are few
    p.split = 1;
    while (p.split < 8 && tiles * p.split * 2 <= 2 * sm_count() &&
           p.row_bytes / 64 >= kSkinnyKG * 2 * p.split * (tiles * p.split < 64 ? 3 : 8))
        p.split *= 2;
    cudaError_t err;
    if (a->quant == AMK_QUANT_W8A16)
        err = skinny_int8(p, stream);
    else if (a->quant == AMK_QUANT_W4A16)
        err = skinny_int4(p, stream);
    else
        err = skinny_bf16(p, stream);
    return launch_status(err, "amk_linear");
}

int launch_tc(const amk_linear_args *a, const Epilogue &e, cudaStream_t stream)
{
    const int sms = sm_count();
    if (!sms)
        return no_device("amk_linear");
    const Choice c = choose(a, sms);
    if (!c.v.nt)
        return amk_set_error(AMK_ERR_UNSUPPORTED, "amk_linear: more tiles than a grid holds");
    TcParams p;
    p.e = e;
    const int ksub = a->quant != AMK_QUANT_BF16 || c.v.split ? 2 : 1;
    const int rows = a->up ? 64 : 128;
    p.groups = (a->k + kQ4Group - 1) / kQ4Group;
    p.w_gs = static_cast<const uint16_t *>(a->w_scale);
    p.up_gs = static_cast<const uint16_t *>(a->up_scale);
    p.blocks = (a->k + ksub * 64 - 1) / (ksub * 64);
    // int4: a sum for each group of 128 inputs, to be scaled by itself; fp32
    // outputs: 512 inputs; bf16 outputs round away more than is cut off
    p.seg = a->quant == AMK_QUANT_W4A16 ? 1
            : a->y_type == AMK_DT_F32   ? 8 / ksub
                                        : p.blocks;
    p.tiles_m = (int)(((int64_t)a->m + c.v.nt - 1) / c.v.nt);
    p.tiles = (int)(((int64_t)a->n + rows - 1) / rows) * p.tiles_m;
    p.split = c.split;
    bool ok = encode_2d(&p.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a->x, a->k, a->m,
                     a->m == 1 ? (2 * (int64_t)a->k + 15) & ~(int64_t)15 : 2 * a->ldx, 64, c.v.nt,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    for (int i = 0; i < (a->up ? 2 : 1) && ok; ++i) {
        CUtensorMap *map = i ? &p.up : &p.w;
        const void *w = i ? a->up : a->w;
        if (a->quant == AMK_QUANT_BF16)
            ok = encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w, a->k, a->n, 2 * (int64_t)a->k, 64,
                        rows, CU_TENSOR_MAP_SWIZZLE_128B);
        else {
            const int per = a->quant == AMK_QUANT_W8A16 ? 1 : 2;  // codes to a byte
            ok = encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, a->k / per, a->n, a->k / per,
                           ksub * 64 / per, rows,
                           per == 1 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
        }
    }
    if (!ok)
        return amk_set_error(AMK_ERR_CUDA, "amk_linear: a tensor map was refused");
    cudaError_t err;
    if (a->quant == AMK_QUANT_W8A16)
        err = launch_int8(c.v, p, c.grid, stream);
    else if (a->quant == AMK_QUANT_W4A16)
        err = launch_int4(c.v, p, c.grid, stream);
    else
        err = launch_bf16(c.v, p, c.grid, stream);
    return launch_status(err, "amk_linear");
}

}  // namespace
}  // namespace linear
}  // namespace amk

extern "C" int amk_linear(const amk_linear_args *a, void *cuda_stream)
{
    using namespace amk;
    using namespace amk::linear;
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
    if (fits_tensor_cores(a))
        return a->m <= kSkinnyTokens ? launch_few(a, p.e, st) : launch_tc(a, p.e, st);
    cudaError_t e;
    if (a->quant == AMK_QUANT_W8A16)
        e = launch_generic<AMK_QUANT_W8A16>(p, st);
    else if (a->quant == AMK_QUANT_W4A16)
        e = launch_generic<AMK_QUANT_W4A16>(p, st);
    else
        e = launch_generic<AMK_QUANT_BF16>(p, st);
    return launch_status(e, "amk_linear");
}
