// amk_op_linear.cuh -- the tensor-core kernel of amk_linear, and the epilogue
// that it shares with the kernel for any alignment.
//
// y = x w^T is taken as its transpose: the 128 rows of the tcgen05 tile are
// rows of w (or 64 of w and 64 of up), its NT columns are tokens.  So the
// tile has 128 rows however few tokens there are, the weights stream through
// shared memory once for up to NT tokens, and a thread of the epilogue holds
// one row of w: its scale and bias are two registers, and a warp's stores of a
// token are 32 consecutive outputs.
//
// Warps: 0 fetches K blocks with TMA into a ring of stages, 1 issues the MMAs,
// 2 owns the TMEM, 4.. drain the accumulators (several buffers, so that the next
// sum runs meanwhile); with int8 and int4 weights eight more turn the codes into
// the bf16 integers they are (exact) and write them to TMEM, from where the MMA
// takes its A: shared memory, which bounds these kernels, then carries the codes
// and x alone (2048 tokens, 4096 x 11008 int8 gate and up: 390 us with A in
// shared memory, 313 to 337 us so; bf16 weights 272 us, the tensor cores busy for
// 81 % of the cycles).  int8 row scales are applied to the sums.  The sums of an
// int4 row's 128-input groups are scaled apart: each group is a sum of its own
// (`seg`), which the draining warps scale and add in fp32 registers, and which
// costs the time between the two (same call: 522 us).  So weights are never
// rounded.
//
// Few tiles of codes are bound by latency: at 77 tokens, 4096 x 11008 int4 (23.7
// us) and 300 tokens, 4096 x 4096 int8 (22.8) no pipe is busy for more than 41 %
// of the active cycles, tensor cores and ALU included.  A stage's chain of
// wait, load, convert, TMEM store, store wait and arrive sets the pace, two of
// them at a time (a TMEM buffer each).
//
// Tensor cores cut off what falls below their accumulators when they align
// the terms of a sum, always downward in magnitude: over K = 4096 an fp32
// output lost 3e-6 of its size.  fp32 outputs are therefore summed in segments
// too (`promote`).
#ifndef AMK_OP_LINEAR_CUH
#define AMK_OP_LINEAR_CUH

#include "amk_op_linear.h"
#include "amk_ops.cuh"

namespace amk {
namespace linear {
namespace {

using namespace ops;

__device__ __forceinline__ float activate(int act, float v)
{
    // __expf is off by (2 + 1.2 |v|) 2^-23 of its value at most, as in the decode
    // step's SwiGLU; the rest of a SiLU adds three roundings
    if (act == AMK_ACT_SILU)
        return v / (1.f + __expf(-v));
    if (act == AMK_ACT_GELU)
        return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    if (act == AMK_ACT_RELU)
        return v < 0.f ? 0.f : v;  // a NaN stays
    return v;
}

// What an output row of w brings to the epilogue: scales and biases.
struct RowConst {
    float ws, bias, us, ubias;
};
__device__ __forceinline__ RowConst row_const(const Epilogue &e, int n)
{
    RowConst c = {1.f, 0.f, 1.f, 0.f};
    if (n < e.n) {
        if (e.w_scale)
            c.ws = fp16f(e.w_scale[n]);
        if (e.bias)
            c.bias = bf16f(e.bias[n]);
        if (e.up_scale)
            c.us = fp16f(e.up_scale[n]);
        if (e.up_bias)
            c.ubias = bf16f(e.up_bias[n]);
    }
    return c;
}
__device__ __forceinline__ float residual_at(const Epilogue &e, int64_t m, int n)
{
    return e.res_f32 ? static_cast<const float *>(e.residual)[m * e.ldr + n]
                     : bf16f(static_cast<const uint16_t *>(e.residual)[m * e.ldr + n]);
}
__device__ __forceinline__ void store_at(const Epilogue &e, int64_t m, int n, float v)
{
    if (e.y_f32)
        static_cast<float *>(e.y)[m * e.ldy + n] = v;
    else
        static_cast<uint16_t *>(e.y)[m * e.ldy + n] = f_bf16(v);
}
// 16 tokens of a row at once: nc of them are there.
__device__ __forceinline__ void activate16(int act, float (&v)[16])
{
    if (act == AMK_ACT_SILU) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
            v[c] = activate(AMK_ACT_SILU, v[c]);
    } else if (act == AMK_ACT_RELU) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
            v[c] = activate(AMK_ACT_RELU, v[c]);
    } else {
#pragma unroll
        for (int c = 0; c < 16; ++c)
            v[c] = activate(AMK_ACT_GELU, v[c]);
    }
}
__device__ __forceinline__ void residual16(const Epilogue &e, int64_t m, int n, int nc,
                                           float (&v)[16])
{
    const int64_t at = m * e.ldr + n;
    if (e.res_f32) {
        const float *r = static_cast<const float *>(e.residual) + at;
#pragma unroll
        for (int c = 0; c < 16; ++c)
            v[c] = c < nc ? r[c * e.ldr] : 0.f;
    } else {
        const uint16_t *r = static_cast<const uint16_t *>(e.residual) + at;
#pragma unroll
        for (int c = 0; c < 16; ++c)
            v[c] = c < nc ? bf16f(r[c * e.ldr]) : 0.f;
    }
}
__device__ __forceinline__ void store16(const Epilogue &e, int64_t m, int n, int nc,
                                        const float (&v)[16])
{
    const int64_t at = m * e.ldy + n;
    if (e.y_f32) {
        float *y = static_cast<float *>(e.y) + at;
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < nc)
                y[c * e.ldy] = v[c];
    } else {
        uint16_t *y = static_cast<uint16_t *>(e.y) + at;
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < nc)
                y[c * e.ldy] = f_bf16(v[c]);
    }
}
// One output from its sums.
__device__ __forceinline__ void emit(const Epilogue &e, const RowConst &c, int m, int n, float a,
                                     float u)
{
    float v = activate(e.act, fmaf(a, c.ws, c.bias));
    if (e.gated)
        v *= fmaf(u, c.us, c.ubias);
    if (e.residual)
        v += residual_at(e, m, n);
    store_at(e, m, n, v);
}

// Exact bf16 pairs of int8 codes: 128 + the low seven bits, less 256 or 128 by
// the sign.  The bytes of w that sel picks, 0x4140 or 0x4342, are the mantissas
// under an exponent of 0x43, whose last bit is then the sign.
__device__ __forceinline__ uint32_t i8_pair(uint32_t w, uint32_t sel)
{
    const uint32_t b = __byte_perm(w, 0x43434343u, sel);
    const uint32_t a = b & 0xff7fff7fu, s = b & 0xff80ff80u;
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(s));
    return r;
}
// Exact bf16 pairs of a word's eight int4 codes, in order: 128 + (code + 8),
// less 136.
__device__ __forceinline__ void i4_pairs(uint32_t w, uint32_t *d)
{
    const uint32_t u = w ^ 0x88888888u, lo = u & 0x0f0f0f0fu, hi = (u >> 4) & 0x0f0f0f0fu;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t four = __byte_perm(lo, hi, e ? 0x7362 : 0x5140);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t b = __byte_perm(four, 0x43434343u, h ? 0x4342 : 0x4140);
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d[2 * e + h]) : "r"(b), "r"(0x43084308u));
        }
    }
}

template <int QUANT, int NT, bool SPLIT, bool PROMOTE>
struct Cfg {
    // K elements of a stage, in blocks of 64 (one swizzled row of bf16): two
    // for codes (one to each of two converting groups) and where the weights
    // only stream through
    static constexpr int KSUB = QUANT != AMK_QUANT_BF16 || SPLIT ? 2 : 1;
    static constexpr int BLK = 128 * 128;  // a block of 128 rows of 64 bf16
    static constexpr int A = KSUB * BLK, X = KSUB * NT * 128;
    static constexpr int RAW = QUANT == AMK_QUANT_W8A16   ? KSUB * 64 * 128
                               : QUANT == AMK_QUANT_W4A16 ? KSUB * 32 * 128
                                                          : 0;
    static constexpr int STAGE = X + (RAW ? RAW : A);
    static constexpr int ASTAGES = RAW ? 2 : 0;                   // converted stages, in TMEM
    static constexpr int ACOLS = KSUB * 32;                       // TMEM columns of one
    static constexpr int CW = RAW ? 8 : 0;       // converting warps
    static constexpr int NB = NT <= 64 ? 4 : RAW && NT == 128 ? 3 : 2;  // accumulators
    static constexpr int XCH = SPLIT ? 0 : 2 * 2 * 16 * 64 * 4;
    static constexpr int CTAS = SPLIT && NT <= (RAW ? 16 : 64) ? 2 : 1;  // to an SM
    // of an SM's 227 KB: half for a CTA where weights stream (two CTAs to an SM
    // keep the stream going while one starts or ends), else all of it
    static constexpr int ROOM = (CTAS == 2 ? 112 * 1024 : 224 * 1024) - 2048 - XCH;
    static constexpr int FIT = ROOM / STAGE;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    // Barriers of landed stages.  Two groups of converting warps take the stages
    // by turns, and each waits for its own alone, by the parity of the barrier's
    // phase: the use before must have been its own too, or it could take a still
    // older phase for this one (copies land in any order).  An odd ring's uses of
    // a stage alternate between the groups and take two barriers in turn.
    static constexpr int FULLS = RAW && STAGES % 2 ? 2 * STAGES : STAGES;
    static_assert(!RAW || FULLS % 2 == 0, "a barrier of landed stages belongs to one group");
    static constexpr int SMEM = STAGES * STAGE + XCH + 1024;
    static constexpr int EW = NT >= 64 ? 2 : 1;  // draining warpgroups
    static constexpr int NC = NT / EW;           // columns of each
    static constexpr int THREADS = 128 + EW * 128 + CW * 32;
    // 640 threads are launched with 96 registers each: 128 x 40 + 256 x DRAIN +
    // 256 x CONVERT of them are no more than that
    static constexpr int REGS = CW && EW == 2 ? 96 : 0;
    static constexpr int DRAIN = 136, CONVERT = 80;
    static_assert(!REGS || 128 * 40 + 256 * (DRAIN + CONVERT) <= THREADS * REGS, "register split");
    static constexpr int USED = NB * NT + ASTAGES * ACOLS;  // TMEM columns: sums, codes
    static constexpr int COLS = USED <= 32    ? 32
                                : USED <= 64  ? 64
                                : USED <= 128 ? 128
                                : USED <= 256 ? 256
                                              : 512;
    static_assert(STAGES >= 2, "a ring needs two stages");
    static_assert(!SPLIT || NT * 512 <= STAGES * STAGE, "the sums reuse the ring");
    static_assert(NB * NT + ASTAGES * ACOLS <= 512 && CTAS * COLS <= 512, "TMEM columns");
};

__device__ unsigned int g_timeouts;  // CTAs that gave up a wait

// A warpgroup's registers from FROM, with which it was launched, to TO a thread.
template <int FROM, int TO>
__device__ __forceinline__ void setmaxnreg_to()
{
    if constexpr (TO > FROM)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TO));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TO));
}

template <int QUANT, int NT, bool SPLIT, bool PROMOTE>
__global__ void __launch_bounds__(Cfg<QUANT, NT, SPLIT, PROMOTE>::THREADS,
                                  Cfg<QUANT, NT, SPLIT, PROMOTE>::CTAS)
    linear_tc(const __grid_constant__ TcParams p)
{
    using C = Cfg<QUANT, NT, SPLIT, PROMOTE>;
    constexpr bool CODES = QUANT != AMK_QUANT_BF16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[C::FULLS + C::STAGES + 2 * C::ASTAGES + 2 * C::NB];
    __shared__ uint32_t tmem_slot;
    __shared__ int fail_flag;
    volatile int *fail = &fail_flag;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t xch = ring + C::STAGES * C::STAGE;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8 * s; };
    constexpr int RING = C::FULLS + C::STAGES;
    auto empty = [&](int s) { return bar0 + 8 * (C::FULLS + s); };
    auto afull = [&](int s) { return bar0 + 8 * (RING + s); };
    auto aempty = [&](int s) { return bar0 + 8 * (RING + C::ASTAGES + s); };
    auto accf = [&](int b) { return bar0 + 8 * (RING + 2 * C::ASTAGES + b); };
    auto acce = [&](int b) { return bar0 + 8 * (RING + 2 * C::ASTAGES + C::NB + b); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        fail_flag = 0;
        for (int s = 0; s < C::FULLS; ++s)
            mbar_init(full(s), 1);
        for (int s = 0; s < C::STAGES; ++s)
            mbar_init(empty(s), 1 + C::CW / 2);  // the MMAs, and the stage's converting warps
        for (int s = 0; s < C::ASTAGES; ++s) {
            mbar_init(afull(s), C::CW / 2);
            mbar_init(aempty(s), 1);
        }
        for (int b = 0; b < C::NB; ++b) {
            mbar_init(accf(b), 1);
            mbar_init(acce(b), 4 * C::EW);
        }
        mbar_init_fence();
        prefetch_map(&p.x);
        prefetch_map(&p.w);
        if (p.e.gated)
            prefetch_map(&p.up);
    }
    if (warp == 2)
        tmem_alloc<C::COLS>(smem_u32(&tmem_slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const bool gated = p.e.gated;
    const int rows_out = gated ? 64 : 128;
    const int split = SPLIT ? p.split : 1, rank = SPLIT ? (int)(blockIdx.x % split) : 0;
    const int first = SPLIT ? blockIdx.x / split : blockIdx.x;
    const int step = SPLIT ? p.tiles : gridDim.x;  // a split tile is the cluster's only one
    const int kb0 = (int)((int64_t)p.blocks * rank / split);
    const int kb1 = (int)((int64_t)p.blocks * (rank + 1) / split);
    if (warp == 0 && lane < min(kb1 - kb0, C::STAGES)) {  // the first stages' weights
        // (17 tokens, 11008 x 4096 int4 gate and up 41.0 us without, 40.1 with)
        const int n0 = (first / p.tiles_m) * rows_out, k = (kb0 + lane) * C::KSUB * 64;
        for (int j = 0; j < (CODES ? 1 : C::KSUB); ++j) {
            const int kx = QUANT == AMK_QUANT_W4A16 ? k / 2 : k + j * 64;
            prefetch_2d(&p.w, kx, n0);
            if (gated)
                prefetch_2d(&p.up, kx, n0);
        }
    }
    pdl_wait();    // nothing above reads or writes global memory
    pdl_launch();  // the next kernel's CTAs may take the room that ending CTAs leave

    // the wide kernels for codes: the draining warps hold the sums, and take the
    // registers that the others give up
    if (warp < 4) {
        if constexpr (C::REGS != 0)
            setmaxnreg_to<C::REGS, 40>();
        if (warp == 0) {
            uint32_t it = 0, ph = 1;
            int s = 0, turn = 0;  // turn: STAGES on an odd ring's second barriers
            bool ok = true;
            for (int tile = first; tile < p.tiles && ok; tile += step) {
                const int n0 = (tile / p.tiles_m) * rows_out, m0 = (tile % p.tiles_m) * NT;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    if (!warp_wait(empty(s), ph, fail)) {
                        ok = false;
                        break;
                    }
                    const uint32_t xs = ring + s * C::STAGE, ws = xs + C::X;
                    const uint32_t landed = full(s + turn);
                    const int k = kb * C::KSUB * 64;
                    if (elect_one()) {
                        mbar_expect_tx(landed, C::STAGE);
                        if (CODES) {
                            const int kx = QUANT == AMK_QUANT_W8A16 ? k : k / 2;
                            tma_2d(ws, &p.w, kx, n0, landed);
                            if (gated)
                                tma_2d(ws + C::RAW / 2, &p.up, kx, n0, landed);
                        }
#pragma unroll
                        for (int j = 0; j < C::KSUB; ++j) {
                            if (!CODES) {
                                tma_2d(ws + j * C::BLK, &p.w, k + j * 64, n0, landed);
                                if (gated)
                                    tma_2d(ws + j * C::BLK + C::BLK / 2, &p.up, k + j * 64, n0,
                                           landed);
                            }
                            tma_2d(xs + j * NT * 128, &p.x, k + j * 64, m0, landed);
                        }
                    }
                    __syncwarp();
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1;
                        if (C::FULLS != C::STAGES)
                            turn ^= C::STAGES;
                    }
                }
            }
            if (!ok && lane == 0)  // no copy may land after the CTA has gone
                for (uint32_t j = it > C::STAGES ? it - C::STAGES : 0; j < it; ++j) {
                    const long long t0 = clock64();
                    while (!mbar_try_wait(full(j % C::FULLS), (j / C::FULLS) & 1) &&
                           clock64() - t0 < 2000000000ll) {
                    }
                }
        } else if (warp == 1) {
            constexpr uint32_t idesc = tc_idesc(128, NT);
            uint32_t sc = 0, ph = 0, aph = 0;
            int s = 0, as = 0;
            bool ok = true;
            for (int tile = first; tile < p.tiles && ok; tile += step) {
                for (int kb = kb0; kb < kb1 && ok; ++sc) {
                    const int b = sc % C::NB, end = min(kb + p.seg, kb1);
                    if (!warp_wait(acce(b), ((sc / C::NB) & 1) ^ 1, fail)) {
                        ok = false;
                        break;
                    }
                    uint32_t accumulate = 0;
                    for (; kb < end; ++kb) {
                        // converted weights come after their stage, and so after its x
                        if (!(CODES ? warp_wait(afull(as), aph, fail)
                                    : warp_wait(full(s), ph, fail))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t xs = ring + s * C::STAGE;
                        const uint64_t ad = tc_desc(xs + C::X), bd = tc_desc(xs);
                        const uint32_t at = tmem + C::NB * NT + as * C::ACOLS;
                        if (elect_one()) {
#pragma unroll
                            for (int j = 0; j < C::KSUB; ++j)
#pragma unroll
                                for (int k16 = 0; k16 < 4; ++k16) {  // 32 bytes of a row each
                                    const uint64_t bk = bd + j * (NT * 128 >> 4) + 2 * k16;
                                    const uint32_t add = j + k16 ? 1u : accumulate;
                                    if (CODES)
                                        tc_mma_ta(tmem + b * NT, at + j * 32 + k16 * 8, bk, idesc, add);
                                    else
                                        tc_mma(tmem + b * NT, ad + j * (C::BLK >> 4) + 2 * k16, bk,
                                               idesc, add);
                                }
                            if (CODES)
                                tc_commit(aempty(as));
                            tc_commit(empty(s));
                            if (kb + 1 == end)
                                tc_commit(accf(b));
                        }
                        __syncwarp();
                        accumulate = 1;
                        if (CODES && ++as == C::ASTAGES) {
                            as = 0;
                            aph ^= 1;
                        }
                        if (++s == C::STAGES) {
                            s = 0;
                            ph ^= 1;
                        }
                    }
                }
            }
        }
    } else if (warp < 4 + 4 * C::EW) {
        if constexpr (C::REGS != 0)
            setmaxnreg_to<C::REGS, C::DRAIN>();
        const int wg = (warp - 4) >> 2, q = warp & 3, r = q * 32 + lane;  // row of the tile
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + wg * C::NC;
        uint32_t sc = 0;
        bool ok = true;
        for (int tile = first; tile < p.tiles && ok; tile += step) {
            const int n0 = (tile / p.tiles_m) * rows_out, m0 = (tile % p.tiles_m) * NT;
            const bool is_up = gated && r >= 64;
            const int n = n0 + (is_up ? r - 64 : r);
            const uint16_t *gs = nullptr;  // the row's group scales
            if (QUANT == AMK_QUANT_W4A16 && n < p.e.n)
                gs = (is_up ? p.up_gs : p.w_gs) + (int64_t)n * p.groups;
            float acc[PROMOTE ? C::NC : 1];
            if constexpr (PROMOTE) {
#pragma unroll
                for (int c = 0; c < C::NC; ++c)
                    acc[c] = 0.f;
                uint16_t next = gs ? gs[kb0] : (uint16_t)0;  // seg = a group of 128 = a block
                for (int kb = kb0; kb < kb1; kb += p.seg, ++sc) {
                    const int b = sc % C::NB;
                    float scale = 1.f;
                    if (QUANT == AMK_QUANT_W4A16) {
                        scale = fp16f(next);
                        if (gs && kb + p.seg < kb1)
                            next = gs[kb + p.seg];
                    }
                    if (!warp_wait(accf(b), (sc / C::NB) & 1, fail)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    float v[2][16];
                    tmem_ld16(taddr + b * NT, v[0]);
#pragma unroll
                    for (int c0 = 0; c0 < C::NC; c0 += 16) {
                        float(&w)[16] = v[(c0 >> 4) & 1];
                        tmem_ld_wait(w);
                        if (c0 + 16 < C::NC)  // the next columns come meanwhile
                            tmem_ld16(taddr + b * NT + c0 + 16, v[(c0 >> 4) & 1 ^ 1]);
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            acc[c0 + c] = QUANT == AMK_QUANT_W4A16
                                              ? fmaf(w[c], scale, acc[c0 + c])
                                              : acc[c0 + c] + w[c];
                    }
                    if (!SPLIT && kb + p.seg >= kb1) {
                        // the tile's sums go back into the last buffer, from where
                        // the loop below takes them a few columns at a time
#pragma unroll
                        for (int c0 = 0; c0 < C::NC; c0 += 16) {
                            float v[16];
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                v[c] = acc[c0 + c];
                            tmem_st16(taddr + b * NT + c0, v);
                        }
                        tmem_st_wait();
                        break;
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(acce(b));
                }
            }
            if constexpr (!SPLIT && !PROMOTE) {
                ok = warp_wait(accf(sc % C::NB), (sc / C::NB) & 1, fail);
                tc_fence_after();
            }
            // a gated tile's warps meet at barriers below: all of them, or, when a
            // wait ran out in one, none.  Also, every warp has read both buffers
            // of the tile before.
            if (!SPLIT && gated)
                ok = named_bar_and(1 + wg, 128, ok);
            if (!ok)
                break;
            if constexpr (SPLIT) {
                static_assert(PROMOTE, "a split tile's sums are held in registers");
                // the ring is idle: every MMA that read it has finished
#pragma unroll
                for (int c = 0; c < C::NC; ++c)
                    sts32f(ring + (uint32_t)((wg * C::NC + c) * 128 + r) * 4, acc[c]);
            } else {
                const int b = sc % C::NB;
                const RowConst rc = row_const(p.e, n);
                const int cols = min(C::NC, p.e.m - m0 - wg * C::NC);  // tokens there are
                const bool mine = n < p.e.n && !is_up;
                // rolled: unrolled, the loop would not fit the instruction cache
#pragma unroll 1
                for (int c0 = 0; c0 < cols; c0 += 16) {
                    float v[16];
                    tmem_ld16(taddr + b * NT + c0, v);
                    const int64_t mc = (int64_t)m0 + wg * C::NC + c0;
                    const int nc = mine ? cols - c0 : 0;
                    float res[16];
                    if (p.e.residual)
                        residual16(p.e, mc, n, nc, res);
                    tmem_ld_wait(v);
                    if (!is_up) {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            v[c] = fmaf(v[c], rc.ws, rc.bias);
                        if (p.e.act != AMK_ACT_NONE)
                            activate16(p.e.act, v);
                    }
                    // a gated row's other half sits 64 lanes on: through shared memory,
                    // in two buffers by turns so that one barrier a round suffices
                    if (gated) {
                        const uint32_t xb =
                            xch + (uint32_t)((wg * 2 + ((c0 >> 4) & 1)) * 16 * 64 + (r & 63)) * 4;
                        if (is_up) {
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                sts32f(xb + c * 256, fmaf(v[c], rc.us, rc.ubias));
                        }
                        named_bar(1 + wg, 128);
                        if (!is_up) {
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                v[c] *= lds32f(xb + c * 256);
                        }
                    }
                    if (p.e.residual) {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            v[c] += res[c];
                    }
                    store16(p.e, mc, n, nc, v);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(acce(b));
                ++sc;
            }
        }
    } else if constexpr (CODES) {
        if constexpr (C::REGS != 0)
            setmaxnreg_to<C::REGS, C::CONVERT>();
        // the two groups of four warps take the stages by turns, a warp 32 rows
        const int grp = (warp - 4 - 4 * C::EW) >> 2, row = (warp & 3) * 32 + lane;
        static_assert(C::ASTAGES == 2 && C::CW == 8 && C::KSUB == 2, "a group to a stage");
        const uint32_t dst =
            tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::NB * NT + grp * C::ACOLS;
        uint32_t it = 0, ph = 0, aph = 1;
        int s = 0, turn = 0;  // as the copies' warp counts them
        bool ok = true;
        for (int tile = first; tile < p.tiles && ok; tile += step)
            for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
                if ((it & 1) == grp) {
                    if (!warp_wait(full(s + turn), ph, fail)) {
                        ok = false;
                        break;
                    }
                    const uint32_t src = ring + s * C::STAGE + C::X;
                    // a lane takes a row's 128 codes: 16-byte pieces that lie swizzled
                    // by row, so that eight lanes' loads share no bank
                    constexpr int NV = C::RAW / 2048, PITCH = C::RAW / 128;
                    const int sw = QUANT == AMK_QUANT_W8A16 ? row & 7 : (row >> 1) & 3;
                    // (both blocks before the wait took 2 % longer)
#pragma unroll
                    for (int j = 0; j < C::KSUB; ++j) {
                        uint32_t o[32];
#pragma unroll
                        for (int i = 0; i < NV / 2; ++i) {
                            const int piece = j * NV / 2 + i;
                            const uint4 v = lds128(src + row * PITCH + ((piece ^ sw) << 4));
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                            uint32_t *d = o + i * (64 / NV);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (QUANT == AMK_QUANT_W8A16) {
                                    d[2 * e] = i8_pair(w[e], 0x4140);
                                    d[2 * e + 1] = i8_pair(w[e], 0x4342);
                                } else {
                                    i4_pairs(w[e], d + 4 * e);
                            }
                            }
                        }
                        if (j == 0) {
                            ok = warp_wait(aempty(grp), aph, fail);
                            tc_fence_after();
                        }
                        tmem_st32(dst + j * 32, o);
                    }
                    if (!ok)
                        break;
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(afull(grp));
                        mbar_arrive(empty(s));
                    }
                    aph ^= 1;
                }
                if (++s == C::STAGES) {
                    s = 0;
                    if (C::FULLS != C::STAGES)
                        turn ^= C::STAGES;
                    if (turn == 0)
                        ph ^= 1;
                }
            }
    }
    __syncwarp();
    if (SPLIT) {
        // every rank's sums are in its shared memory, unless one gave up a wait
        if (split == 1)
            __syncthreads();
        else
            cluster_sync_failed(fail, split);
        const int et = tid - 128;
        if (et >= 0 && et < C::EW * 128 && !*fail) {
            const int tile = first;
            const int n0 = (tile / p.tiles_m) * rows_out, m0 = (tile % p.tiles_m) * NT;
            const int rows = rows_out / split;  // this rank's rows of the tile
            const int cols = min(NT, p.e.m - m0);
            const int r = rank * rows + et % rows, n = n0 + r, dc = C::EW * 128 / rows;
            const RowConst rc = row_const(p.e, n);
            uint32_t at[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                at[k] = split == 1 ? ring + (uint32_t)r * 4
                                   : map_rank(ring + (uint32_t)r * 4, k < split ? k : 0);
            // added in the ranks' order: the same bits every time.  Several tokens at
            // a time: one by one, a load's latency each was a third of a short call.
            if (split == 1) {
                for (int c = et / rows; c < cols && n < p.e.n; c += 8 * dc) {
                    float s[8], u[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {  // a token behind the last: the last again
                        const uint32_t o = at[0] + (uint32_t)min(c + i * dc, cols - 1) * 512;
                        s[i] = lds32f(o);
                        u[i] = gated ? lds32f(o + 64 * 4) : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c + i * dc < cols)
                            emit(p.e, rc, m0 + c + i * dc, n, s[i], u[i]);
                }
            } else {
                for (int c = et / rows; c < cols && n < p.e.n; c += 4 * dc) {
                    float s[4] = {}, u[4] = {};
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < split) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t o = at[k] + (uint32_t)min(c + i * dc, cols - 1) * 512;
                                s[i] += ld_cluster(o);
                                if (gated)
                                    u[i] += ld_cluster(o + 64 * 4);
                            }
                        }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i * dc < cols)
                            emit(p.e, rc, m0 + c + i * dc, n, s[i], u[i]);
                }
            }
        }
        if (split == 1)
            __syncthreads();
        else
            cluster_sync();  // no CTA leaves while another reads its shared memory
    } else {
        __syncthreads();
    }
    if (tid == 0 && *fail)
        atomicAdd(&g_timeouts, 1u);
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc<C::COLS>(tmem);
    }
}

template <int QUANT, int NT, bool SPLIT, bool PROMOTE>
cudaError_t launch_one(const TcParams &p, int grid, cudaStream_t stream)
{
    using C = Cfg<QUANT, NT, SPLIT, PROMOTE>;
    auto kernel = linear_tc<QUANT, NT, SPLIT, PROMOTE>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_once(allowed, reinterpret_cast<const void *>(kernel), C::SMEM);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int QUANT>
cudaError_t launch_variant(const Variant &v, const TcParams &p, int grid, cudaStream_t stream)
{
    if (v.split)
        switch (v.nt) {
        case 16: return launch_one<QUANT, 16, true, true>(p, grid, stream);
        case 32: return launch_one<QUANT, 32, true, true>(p, grid, stream);
        case 64: return launch_one<QUANT, 64, true, true>(p, grid, stream);
        default: return launch_one<QUANT, 128, true, true>(p, grid, stream);
        }
    // eight draining warps hold 256 columns of 128 sums in registers; beside
    // the converting warps there is room for half of them.  Two buffers of 192
    // columns and the codes fill the TMEM
    constexpr int WIDE = QUANT == AMK_QUANT_BF16 ? 256 : 128;
    if (v.promote || QUANT == AMK_QUANT_W4A16)
        return launch_one<QUANT, WIDE, false, true>(p, grid, stream);
    if constexpr (QUANT != AMK_QUANT_W4A16)
        return launch_one<QUANT, QUANT == AMK_QUANT_BF16 ? 256 : 192, false, false>(p, grid,
                                                                                    stream);
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace linear
}  // namespace amk

#endif
