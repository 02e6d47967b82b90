// amk_op_linear_skinny.cuh -- amk_linear for up to 16 tokens.
//
// The product then costs what reading the weights costs.  They go from HBM
// into registers: every lane loads 16 bytes of a row at a time, several loads
// ahead, turns codes into bf16 integers there, and feeds them to mma.sync as
// the A operand (16 rows of w), x being B (8 tokens).  An MMA sums over its K
// in any order, so a lane's 16 consecutive bytes serve as its K positions of
// two (bf16), four (int8) or eight (int4) MMAs, x being read by the same
// order; no shuffle, no shared memory.  tcgen05 has nothing to add here: its
// operands would first have to be written to shared memory, which cost more
// than the rest of the call (one token, 4096 x 11008 int4 gate and up: 35 us).
//
// A warp takes 32 rows (16 of w and 16 of up when gated) so that a read of x
// serves two MMAs.  K is shared by four warps of a CTA and by the CTAs of a
// cluster, whose sums are added in a fixed order.  Sums leave the tensor
// cores every 512 inputs (every scale group for int4) and are added in fp32.
//
// Measured: one token, 4096 x 4096 bf16 9.1 us (reading the weights takes 5.2 at
// the copy rate: start, cluster sums and end are the rest), 32000 x 4096 42.9 us
// (6.1 TB/s); 5 tokens, 8192 x 2048 int8 gate and up 9.3 us and 11008 x 4096
// 23.5; one token, 11008 x 4096 int4 gate and up 19.3.  Codes wait for their
// loads first (int8 4.5 warps to an issue, int4 2.3, two steps being all that the
// registers hold), then for the instructions that convert them, three and a
// subtraction to two (the ALU is busy for 50 % of the active cycles); and 344
// CTAs of 11008 rows on 296 places leave the SMs active for 23 to 36 thousand
// cycles, 27 on average (int4).
#ifndef AMK_OP_LINEAR_SKINNY_CUH
#define AMK_OP_LINEAR_SKINNY_CUH

#include "amk_op_linear.cuh"

namespace amk {
namespace linear {
namespace {

constexpr int kSkinnyThreads = 256;

__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The bf16 pairs of one MMA from a lane's 16 bytes of a row: pair 0 and pair 1
// of its MMA j.
template <int QUANT>
__device__ __forceinline__ uint32_t pair_of(const uint4 &v, int j, int h)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (QUANT == AMK_QUANT_BF16)
        return w[2 * j + h];
    if (QUANT == AMK_QUANT_W8A16)
        return i8_pair(w[j], h ? 0x4342 : 0x4140);
    // codes 0 and 2 of a word's four, then 1 and 3: as bytes (code + 8), which lie
    // under an exponent of 0x43 as 128 + 8 + code
    const uint32_t c = ((h ? w[j >> 1] >> 4 : w[j >> 1]) & 0x0f0f0f0fu) ^ 0x08080808u;
    const uint32_t b = __byte_perm(c, 0x43434343u, j & 1 ? 0x4342 : 0x4140);
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(b), "r"(0x43084308u));
    return r;
}

// T8: tokens / 8.  A lane holds AHEAD steps of its weights (64 bytes each), two
// CTAs to an SM: 64 KB of weights and more on their way.  Measured (us, AHEAD
// 2 / 3 / 4): 1 x 32000 x 4096 bf16 45.7 / 43.6 / 43.0, 5 x 8192 x 2048 int8
// gated 9.3 / 11.2 / 9.9, 1 x 11008 x 4096 int4 gated 19.3 / 21.7 / 22.7 (the
// registers of codes spill at 3 and 4); three or four CTAs to an SM were slower
// throughout.  The 3 of bf16 with 9 to 16 tokens is not the best of them: 13 x
// 11008 x 4096 20.7 / 26.5 / 27.4.
template <int QUANT, int T8>
struct SkinnyCfg {
    static constexpr int KL = QUANT == AMK_QUANT_BF16 ? 8 : QUANT == AMK_QUANT_W8A16 ? 16 : 32;
    static constexpr int AHEAD = QUANT == AMK_QUANT_BF16 ? (T8 == 1 ? 4 : 3) : 2;
};
template <int QUANT, int T8>
__global__ void __launch_bounds__(kSkinnyThreads, 2)
    linear_skinny(const SkinnyParams p)
{
    constexpr int KL = SkinnyCfg<QUANT, T8>::KL, AHEAD = SkinnyCfg<QUANT, T8>::AHEAD;
    constexpr int STEP = 4 * KL, MMAS = KL / 4;  // inputs and MMAs of a step
    constexpr int PROMOTE = 512 / STEP;          // steps of a sum (int4: every step)
    constexpr int NT = 8 * T8;
    __shared__ float red[kSkinnyKG][NT][kSkinnyRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rg = warp & 1, kg = warp >> 1;
    const bool gated = p.e.gated;
    const int rows_out = gated ? kSkinnyRows / 2 : kSkinnyRows;
    const int split = p.split, rank = blockIdx.x % split;
    const int n0 = (int)(blockIdx.x / split) * rows_out;
    // the lane's rows: g and g + 8 of two tiles of 16 (a row behind the last
    // one is read as the last, and its result dropped)
    const uint8_t *wp[4];
    const uint16_t *sp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tile = i >> 1, r = g + 8 * (i & 1);
        const int n = min(n0 + (gated ? rg * 16 + r : rg * 32 + tile * 16 + r), p.e.n - 1);
        const bool up = gated && tile;
        wp[i] = static_cast<const uint8_t *>(up ? p.up : p.w) + n * p.row_bytes + t * 16;
        sp[i] = QUANT == AMK_QUANT_W4A16 ? (up ? p.up_gs : p.w_gs) + (int64_t)n * p.groups : nullptr;
    }
    const int steps = (p.k + STEP - 1) / STEP, unit = rank * kSkinnyKG + kg;
    const int s0 = (int)((int64_t)steps * unit / (split * kSkinnyKG));
    const int s1 = (int)((int64_t)steps * (unit + 1) / (split * kSkinnyKG));
    // a column of x to a lane's token (one behind the last is read as the last:
    // columns of a product do not mix)
    const uint16_t *xp[T8];
#pragma unroll
    for (int c = 0; c < T8; ++c)
        xp[c] = p.x + min(c * 8 + g, p.e.m - 1) * p.ldx + t * KL;
    pdl_wait();
    pdl_launch();
    uint4 w[AHEAD][4];
    uint16_t sc[AHEAD][4];
    float acc[2][T8][4] = {}, part[2][T8][4] = {};
    // the products of a step's weights w and x
    auto products = [&](const uint4(&w)[4], const uint16_t(&sc)[4], const uint4(&xv)[T8][KL / 8]) {
#pragma unroll
        for (int j = 0; j < MMAS; ++j) {
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
                const uint32_t a0 = pair_of<QUANT>(w[2 * tile], j, 0);
                const uint32_t a1 = pair_of<QUANT>(w[2 * tile + 1], j, 0);
                const uint32_t a2 = pair_of<QUANT>(w[2 * tile], j, 1);
                const uint32_t a3 = pair_of<QUANT>(w[2 * tile + 1], j, 1);
#pragma unroll
                for (int c = 0; c < T8; ++c) {
                    const uint4 q = xv[c][j >> 1];
                    uint32_t b0 = (j & 1) ? q.z : q.x, b1 = (j & 1) ? q.w : q.y;
                    if (QUANT == AMK_QUANT_W4A16) {  // in the codes' order
                        const uint32_t x = b0;
                        b0 = __byte_perm(x, b1, 0x5410);
                        b1 = __byte_perm(x, b1, 0x7632);
                    }
                    mma_bf16(part[tile][c], a0, a1, a2, a3, b0, b1);
                }
            }
        }
        if (QUANT == AMK_QUANT_W4A16) {
#pragma unroll
            for (int tile = 0; tile < 2; ++tile)
#pragma unroll
                for (int c = 0; c < T8; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[tile][c][i] =
                            fmaf(part[tile][c][i], fp16f(sc[2 * tile + (i >> 1)]), acc[tile][c][i]);
                        part[tile][c][i] = 0.f;
                    }
        }
    };
    auto promote = [&] {
#pragma unroll
        for (int tile = 0; tile < 2; ++tile)
#pragma unroll
            for (int c = 0; c < T8; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[tile][c][i] += part[tile][c][i];
                    part[tile][c][i] = 0.f;
                }
    };
    // a step's weights, zeros behind the end of the share and of the row
    auto load = [&](uint4(&v)[4], uint16_t(&sv)[4], int step) {
        const bool in = step < s1 && step * STEP + t * KL < p.k;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = in ? ldg_stream(wp[i] + (int64_t)step * 64) : make_uint4(0, 0, 0, 0);
            if (QUANT == AMK_QUANT_W4A16)
                sv[i] = step < s1 ? __ldg(sp[i] + step) : (uint16_t)0;
        }
    };
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
        load(w[a], sc[a], s0 + a);
    int since = 0, s = s0;
    // While neither these steps nor those that are loaded reach the end, nothing
    // is looked at and offsets are constants (5 tokens, 4096 x 11008 int8 gate and
    // up 27.5 us, all by the loop behind 28.7; 13 tokens, 4096 x 4096 int8 9.2 and
    // 10.6).  bf16 does not take it: its registers spill, 35.6 us instead of 33.0.
    const int whole = min(s1, p.k / STEP);
    if (QUANT != AMK_QUANT_BF16 && s + 2 * AHEAD <= whole) {
        const uint8_t *wq[4];
        const uint16_t *sq[4], *xq[T8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wq[i] = wp[i] + (int64_t)(s + AHEAD) * 64;
            if (QUANT == AMK_QUANT_W4A16)
                sq[i] = sp[i] + s + AHEAD;
        }
#pragma unroll
        for (int c = 0; c < T8; ++c)
            xq[c] = xp[c] + s * STEP;
        for (; s + 2 * AHEAD <= whole; s += AHEAD) {
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                uint4 xv[T8][KL / 8];
#pragma unroll
                for (int c = 0; c < T8; ++c)
#pragma unroll
                    for (int i = 0; i < KL / 8; ++i)
                        xv[c][i] = __ldg(reinterpret_cast<const uint4 *>(xq[c] + a * STEP) + i);
                products(w[a], sc[a], xv);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[a][i] = ldg_stream(wq[i] + a * 64);
                    if (QUANT == AMK_QUANT_W4A16)
                        sc[a][i] = __ldg(sq[i] + a);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wq[i] += AHEAD * 64;
                if (QUANT == AMK_QUANT_W4A16)
                    sq[i] += AHEAD;
            }
#pragma unroll
            for (int c = 0; c < T8; ++c)
                xq[c] += AHEAD * STEP;
            since += AHEAD;
            if (QUANT != AMK_QUANT_W4A16 && since >= PROMOTE) {
                since = 0;
                promote();
            }
        }
    }
    for (; s < s1; s += AHEAD) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int k = (s + a) * STEP;
            const bool in = s + a < s1 && k + t * KL < p.k;
            uint4 xv[T8][KL / 8];
#pragma unroll
            for (int c = 0; c < T8; ++c)
#pragma unroll
                for (int i = 0; i < KL / 8; ++i)
                    xv[c][i] = in && c * 8 + g < p.e.m
                                   ? __ldg(reinterpret_cast<const uint4 *>(xp[c] + k) + i)
                                   : make_uint4(0, 0, 0, 0);
            products(w[a], sc[a], xv);
            load(w[a], sc[a], s + a + AHEAD);
        }
        since += AHEAD;
        if (QUANT != AMK_QUANT_W4A16 && since >= PROMOTE) {
            since = 0;
            promote();
        }
    }
    if (QUANT != AMK_QUANT_W4A16)
        promote();
    // c[0], c[1]: row g of tokens 2 t, 2 t + 1; c[2], c[3]: row g + 8
#pragma unroll
    for (int tile = 0; tile < 2; ++tile)
#pragma unroll
        for (int c = 0; c < T8; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[kg][c * 8 + 2 * t + (i & 1)][rg * 32 + tile * 16 + g + 8 * (i >> 1)] =
                    acc[tile][c][i];
    __syncthreads();
    const int m = p.e.m;
    if (split == 1) {
        for (int i = tid; i < rows_out * m; i += kSkinnyThreads) {
            const int r = i % rows_out, c = i / rows_out, n = n0 + r;
            const int slot = gated ? (r >> 4) * 32 + (r & 15) : r;
            float a = 0.f, u = 0.f;
#pragma unroll
            for (int k = 0; k < kSkinnyKG; ++k) {
                a += red[k][c][slot];
                if (gated)
                    u += red[k][c][slot + 16];
            }
            if (n < p.e.n)
                emit(p.e, row_const(p.e, n), c, n, a, u);
        }
        return;
    }
    for (int i = tid; i < kSkinnyRows * m; i += kSkinnyThreads) {
        const int r = i % kSkinnyRows, c = i / kSkinnyRows;
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < kSkinnyKG; ++k)
            a += red[k][c][r];
        red[0][c][r] = a;
    }
    cluster_sync();
    const int rows = rows_out / split;  // this rank's rows
    const uint32_t base = smem_u32(&red[0][0][0]);
    for (int i = tid; i < rows * m; i += kSkinnyThreads) {
        const int r = rank * rows + i % rows, c = i / rows, n = n0 + r;
        const int slot = gated ? (r >> 4) * 32 + (r & 15) : r;
        float a[8], u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < split) {
                const uint32_t at = map_rank(base, k) + (uint32_t)(c * kSkinnyRows + slot) * 4;
                a[k] = ld_cluster(at);
                u[k] = gated ? ld_cluster(at + 64) : 0.f;
            }
        float as = 0.f, us = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < split) {
                as += a[k];
                us += u[k];
            }
        if (n < p.e.n)
            emit(p.e, row_const(p.e, n), c, n, as, us);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
}

template <int QUANT>
cudaError_t launch_skinny_of(const SkinnyParams &p, cudaStream_t stream)
{
    const int rows = p.e.gated ? kSkinnyRows / 2 : kSkinnyRows;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(((p.e.n + rows - 1) / rows) * p.split));
    cfg.blockDim = dim3(kSkinnyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return p.e.m <= 8 ? cudaLaunchKernelEx(&cfg, linear_skinny<QUANT, 1>, p)
                      : cudaLaunchKernelEx(&cfg, linear_skinny<QUANT, 2>, p);
}

}  // namespace
}  // namespace linear
}  // namespace amk

#endif
