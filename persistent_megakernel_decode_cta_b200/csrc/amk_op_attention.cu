// amk_op_attention.cu -- amk_attention: causal attention with a sliding window
// and sinks over KV-cache rows.
#include <atomic>
#include <math.h>

#include "amk_ops.cuh"
#include "amk_ops.h"

namespace amk {
namespace {

using namespace ops;

struct AttnParams {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    int64_t q_ts, q_hs, o_ts, o_hs, k_hs, k_rs, v_hs, v_rs;
    int32_t T, pos, n_heads, group, hd, window, sinks;
    int32_t q_pairs;   // q can be read two elements at a time
    float scale_log2;  // scale * log2(e): weights are 2^(s - m)
};

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
// Writes the elements d for which mine(d).
constexpr int kMaxHd = kAttentionMaxHd, kMaxRows = kAttentionMaxRows;

template <typename Mine>
__device__ void attend_row(const AttnParams &a, int t, int h, const float *qs, Mine mine)
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
        const float pr = i < n ? ex2(sc - base) : 0.f;
        const float corr = ex2(m - base);
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
        if (lane + 32 * e < hd && mine(lane + 32 * e))
            out[lane + 32 * e] = f_bf16(o[e] / l);
}

__global__ void __launch_bounds__(128) attn_rows(const AttnParams a)
{
    pdl_wait();
    pdl_launch();
    __shared__ float qs[4][kMaxHd];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.T * a.n_heads;
    for (int64_t r = (int64_t)blockIdx.x * 4 + warp; r < rows; r += (int64_t)gridDim.x * 4) {
        const int t = (int)(r / a.n_heads), h = (int)(r % a.n_heads);
        const uint16_t *q = a.q + t * a.q_ts + h * a.q_hs;
        for (int d = lane; d < a.hd; d += 32)
            qs[warp][d] = bf16f(q[d]) * a.scale_log2;
        __syncwarp();
        attend_row(a, t, h, qs[warp], [](int) { return true; });
        __syncwarp();
    }
}

__device__ unsigned int g_timeouts;  // CTAs that gave up a wait

// ---- tiles of rows ---------------------------------------------------------------
// The (token, head) pairs of a KV head are the rows of tiles of 16: a group's
// heads and neighbouring tokens share every K and V row that is read.  A
// producer warp streams the visible K and V rows, 64 at a time, through a ring
// of stages with TMA (swizzled; rows behind the last token and elements behind
// head_dim read as 0); GR groups of WK warps take the stages by turns, a warp
// the tile's 16 rows and a WK-th of the stage's keys: scores, the running
// maximum and sum of the softmax (Milakov and Gimelshein, Online normalizer
// calculation for softmax, 2018), and the weighted sum of V, all in registers.
// Weights are rounded to bf16 for the product with V; their sum is taken before.
// An MMA's operands have one type: weights of more bits would take V as tf32, in
// twice the shared memory at half the rate.  The rounding is at most 2^-8 of each
// weight, of either sign, and so no more in their sum than what the output loses
// when it is rounded to bf16 itself.  The warps merge through shared memory, the CTAs of a cluster that share the keys of a tile through
// distributed shared memory, in a fixed order.
//
// A step of a warp is a chain of dependent instructions (0.4 us for 16 keys),
// so what counts is how many of them run at once: tiles of 32 or 64 rows, with
// as many warps, took 28 and 30 us where these take 19 (5 tokens, 32 heads on
// 4, 32000 rows of 64).
//
// A masked weight is 0, and 0 times a NaN or infinity in a masked V row is
// NaN.  So where a result is not finite its row is computed again by
// attend_row, which touches visible rows alone.
constexpr int kKeys = 64;  // of a stage

struct TileParams {
    CUtensorMap k, v;
    AttnParams a;
    int32_t rows;    // T * group
    int32_t tiles, n_kv, split;
};

__device__ __forceinline__ float weigh(float m, float M)
{
    return m == -INFINITY ? 0.f : ex2(m - M);
}
// Element d of a tile's row r, unless it is not finite: the row is then noted.
__device__ __forceinline__ void put(const TileParams &p, int r0, int kvh, int r, int d, float v,
                                    int *redo)
{
    if (!(fabsf(v) < INFINITY)) {
        redo[r] = 1;
        return;
    }
    const AttnParams &a = p.a;
    const int row = r0 + r;
    a.out[(row / a.group) * a.o_ts + (kvh * a.group + row % a.group) * a.o_hs + d] = f_bf16(v);
}
// Merges the sums os [rows][OS] and their (maximum, sum) ml [rows][2] of a
// cluster's CTAs, in the ranks' order; this rank's share of the elements, four
// at a time, by thread idx of nt.  A cluster barrier before and after.
template <int OS>
__device__ __forceinline__ void merge_cluster(const TileParams &p, uint32_t os, uint32_t ml, int r0,
                                              int nrows, int kvh, int rank, int idx, int nt,
                                              int *redo)
{
    const int hd = p.a.hd, split = p.split, quads = (hd + 3) / 4;
    for (int i = rank * nt + idx; i < nrows * quads; i += split * nt) {
        const int r = i / quads, d = (i - r * quads) * 4;
        float M = -INFINITY, L = 0.f, O[4] = {};
        for (int k0 = 0; k0 < split; k0 += 4) {  // four CTAs' partials at a time
            float2 w[4];
            float4 o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int kk = min(k0 + k, split - 1);
                w[k] = ld_cluster2(map_rank(ml + r * 8, kk));
                o[k] = ld_cluster4(map_rank(os + (r * OS + d) * 4, kk));
            }
            float Mn = M;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                Mn = fmaxf(Mn, w[k].x);  // the last one twice does no harm here
            const float c = weigh(M, Mn);
            L *= c;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                O[e] *= c;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float f = k0 + k < split ? weigh(w[k].x, Mn) : 0.f;
                if (k0 + k < split) {
                    L = fmaf(w[k].y, f, L);
                    O[0] = fmaf(o[k].x, f, O[0]);
                    O[1] = fmaf(o[k].y, f, O[1]);
                    O[2] = fmaf(o[k].z, f, O[2]);
                    O[3] = fmaf(o[k].w, f, O[3]);
                }
            }
            M = Mn;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < hd)
                put(p, r0, kvh, r, d + e, O[e] / L, redo);
    }
}
// The noted rows again, by warps first, first + n, ...: this rank's share of
// their elements.  qs: the warp's own kMaxHd floats.
__device__ __forceinline__ void redo_rows(const TileParams &p, const int *redo, int r0, int nrows,
                                          int kvh, int rank, int nt, int first, int n, float *qs)
{
    const AttnParams &a = p.a;
    const int lane = threadIdx.x & 31;
    for (int r = first; r < nrows; r += n)
        if (redo[r]) {
            const int row = r0 + r, tok = row / a.group, h = kvh * a.group + row % a.group;
            const uint16_t *q = a.q + tok * a.q_ts + h * a.q_hs;
            for (int d = lane; d < a.hd; d += 32)
                qs[d] = bf16f(q[d]) * a.scale_log2;
            __syncwarp();
            attend_row(a, tok, h, qs, [&](int d) {
                return (r * ((a.hd + 3) / 4) + d / 4) / nt % p.split == rank;
            });
            __syncwarp();
        }
}
// The stages of a tile's keys that this rank of its cluster takes: [t0, t1).
__device__ __forceinline__ void share(int stages, int rank, int split, int &t0, int &t1)
{
    t0 = (int)((int64_t)stages * rank / split);
    t1 = (int)((int64_t)stages * (rank + 1) / split);
}

template <int HD, int WK, int GR>
struct TileCfg {
    static constexpr int ROWS = 16, KW = kKeys / WK;
    static constexpr int WARPS = WK * GR, THREADS = 32 * (WARPS + 1);
    static constexpr int STAGE = 2 * kKeys * HD * 2;
    // two CTAs to an SM where their registers fit (168 a thread of the wide
    // heads, 112 else)
    static constexpr int CTAS = THREADS * (HD == 128 ? 168 : 112) * 2 <= 65536 ? 2 : 1;
    static constexpr int STAGES = (CTAS == 1 ? 192 : 96) * 1024 / STAGE;
    // a group waits for its next use of a stage by that use's parity: the one
    // before must have been its own, or it could take an older phase for it
    static_assert(STAGES % GR == 0, "a stage belongs to one group");
    static constexpr int OS = HD + 8;  // floats of a row of sums (padded)
    static constexpr int SMEM = STAGES * STAGE + 1024;
    static_assert(WARPS * ROWS * (OS + 2) * 4 + ROWS * 8 + WARPS * kMaxHd * 4 <= STAGES * STAGE,
                  "the sums reuse the ring");
};

template <int HD, int WK, int GR>
__global__ void __launch_bounds__(TileCfg<HD, WK, GR>::THREADS, (TileCfg<HD, WK, GR>::CTAS))
    attn_tiles(const __grid_constant__ TileParams p)
{
    using C = TileCfg<HD, WK, GR>;
    constexpr int KW = C::KW;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * C::STAGES];
    __shared__ int fail_flag, redo[C::ROWS];
    volatile int *fail = &fail_flag;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8 * s; };
    auto empty = [&](int s) { return bar0 + 8 * (C::STAGES + s); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        fail_flag = 0;
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), WK);
        }
        mbar_init_fence();
        prefetch_map(&p.k);
        prefetch_map(&p.v);
    }
    for (int r = tid; r < C::ROWS; r += C::THREADS)
        redo[r] = 0;
    __syncthreads();
    const AttnParams &a = p.a;
    const int split = p.split, rank = blockIdx.x % split;
    const int rest = blockIdx.x / split, kvh = rest % p.n_kv;
    const int tile = p.tiles - 1 - rest / p.n_kv;  // the longest rows start first
    const int r0 = tile * C::ROWS, nrows = min(C::ROWS, p.rows - r0);
    const int pmin = a.pos + r0 / a.group, pmax = a.pos + (r0 + nrows - 1) / a.group;
    // the keys that some row sees: [0, na) and [lo, pmax]
    int na, lo;
    visible(a, pmin, na, lo);
    const int ta = (na + kKeys - 1) / kKeys, tn = ta + (pmax - lo + kKeys) / kKeys;
    int t0, t1;
    share(tn, rank, split, t0, t1);
    if (warp == C::WARPS && lane < min(t1 - t0, C::STAGES)) {  // the first stages' rows
        const int i = t0 + lane, j0 = i < ta ? i * kKeys : lo + (i - ta) * kKeys;
        for (int d = 0; d < HD / 64; ++d) {
            prefetch_3d(&p.k, d * 64, j0, kvh);
            prefetch_3d(&p.v, d * 64, j0, kvh);
        }
    }
    pdl_wait();
    pdl_launch();
    if (warp == C::WARPS) {
        uint32_t ph = 1;
        int s = 0;
        bool ok = true;
        int i = t0;
        for (; i < t1; ++i) {
            if (!warp_wait(empty(s), ph, fail)) {
                ok = false;
                break;
            }
            const int j0 = i < ta ? i * kKeys : lo + (i - ta) * kKeys;
            const uint32_t ks = ring + s * C::STAGE, vs = ks + C::STAGE / 2;
            if (elect_one()) {
                mbar_expect_tx(full(s), C::STAGE);
#pragma unroll
                for (int d = 0; d < HD / 64; ++d)
                    tma_3d(ks + d * kKeys * 128, &p.k, d * 64, j0, kvh, full(s));
#pragma unroll
                for (int d = 0; d < HD / 64; ++d)
                    tma_3d(vs + d * kKeys * 128, &p.v, d * 64, j0, kvh, full(s));
            }
            __syncwarp();
            if (++s == C::STAGES) {
                s = 0;
                ph ^= 1;
            }
        }
        if (!ok && lane == 0)  // no copy may land after the CTA has gone
            for (int j = max(t0, i - C::STAGES); j < i; ++j) {
                const long long c0 = clock64();
                while (!mbar_try_wait(full((j - t0) % C::STAGES), ((j - t0) / C::STAGES) & 1) &&
                       clock64() - c0 < 2000000000ll) {
                }
            }
    } else {
        const int grp = warp / WK, wk = warp % WK;
        const int g = lane >> 2, t = lane & 3;
        // the lane's rows: g and g + 8
        int prow[2];
        uint32_t qf[HD / 16][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + g + 8 * h;
            const bool in = r < p.rows;
            const int tok = in ? r / a.group : 0, hh = in ? r % a.group : 0;
            prow[h] = in ? a.pos + tok : pmax;
            const uint16_t *q = a.q + tok * a.q_ts + (kvh * a.group + hh) * a.q_hs;
#pragma unroll
            for (int i = 0; i < HD / 16; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int d = i * 16 + c * 8 + 2 * t;
                    if (a.q_pairs) {
                        qf[i][h + 2 * c] =
                            in && d < a.hd ? __ldg(reinterpret_cast<const uint32_t *>(q + d)) : 0;
                    } else {
                        const uint32_t x0 = in && d < a.hd ? q[d] : 0;
                        const uint32_t x1 = in && d + 1 < a.hd ? q[d + 1] : 0;
                        qf[i][h + 2 * c] = x0 | (x1 << 16);
                    }
                }
        }
        float o[HD / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (int i = t0 + grp; i < t1; i += GR) {
            const int s = (i - t0) % C::STAGES;
            if (!warp_wait(full(s), ((i - t0) / C::STAGES) & 1, fail))
                break;
            const int j0 = (i < ta ? i * kKeys : lo + (i - ta) * kKeys) + wk * KW;
            const uint32_t ks = ring + s * C::STAGE + wk * KW * 128, vs = ks + C::STAGE / 2;
            float sc[KW / 8][4] = {};
#pragma unroll
            for (int d = 0; d < HD / 32; ++d)  // 32 elements of the heads at a time
#pragma unroll
                for (int n = 0; n < KW / 8; ++n) {
                    const int row = n * 8 + (lane & 7), ch = (d & 1) * 4 + (lane >> 3);
                    uint32_t b[4];
                    ldmatrix4(b, ks + (d >> 1) * kKeys * 128 + row * 128 + ((ch ^ (row & 7)) << 4));
                    mma_bf16(sc[n], qf[2 * d][0], qf[2 * d][1], qf[2 * d][2], qf[2 * d][3], b[0],
                             b[1]);
                    mma_bf16(sc[n], qf[2 * d + 1][0], qf[2 * d + 1][1], qf[2 * d + 1][2],
                             qf[2 * d + 1][3], b[2], b[3]);
                }
#pragma unroll
            for (int n = 0; n < KW / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sc[n][e] *= a.scale_log2;
            const bool sink = i < ta;
            if (sink ? j0 + KW > na : j0 + KW - 1 > pmin || (a.window && j0 <= pmax - a.window)) {
#pragma unroll
                for (int n = 0; n < KW / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + n * 8 + 2 * t + (e & 1), pr = prow[e >> 1];
                        const bool see = sink ? j < na
                                              : j <= pr && (!a.window || j > pr - a.window ||
                                                            j < a.sinks);
                        if (!see)
                            sc[n][e] = -INFINITY;
                    }
            }
            float corr[2], base[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float mx = m[h];
#pragma unroll
                for (int n = 0; n < KW / 8; ++n)
                    mx = fmaxf(mx, fmaxf(sc[n][2 * h], sc[n][2 * h + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                base[h] = mx == -INFINITY ? 0.f : mx;
                corr[h] = ex2(m[h] - base[h]);
                m[h] = mx;
                l[h] *= corr[h];
            }
#pragma unroll
            for (int n = 0; n < KW / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[n][e] = ex2(sc[n][e] - base[e >> 1]);
                    l[e >> 1] += sc[n][e];
                }
            if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
                for (int d = 0; d < HD / 8; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[d][e] *= corr[e >> 1];
            }
#pragma unroll
            for (int kk = 0; kk < KW / 16; ++kk) {
                const uint32_t a0 = f2_bf16(sc[2 * kk][0], sc[2 * kk][1]);
                const uint32_t a1 = f2_bf16(sc[2 * kk][2], sc[2 * kk][3]);
                const uint32_t a2 = f2_bf16(sc[2 * kk + 1][0], sc[2 * kk + 1][1]);
                const uint32_t a3 = f2_bf16(sc[2 * kk + 1][2], sc[2 * kk + 1][3]);
#pragma unroll
                for (int d = 0; d < HD / 16; ++d) {
                    const int row = kk * 16 + (lane & 15), ch = (d & 3) * 2 + (lane >> 4);
                    uint32_t b[4];
                    ldmatrix4_t(b, vs + (d >> 2) * kKeys * 128 + row * 128 +
                                       ((ch ^ (row & 7)) << 4));
                    mma_bf16(o[2 * d], a0, a1, a2, a3, b[0], b[1]);
                    mma_bf16(o[2 * d + 1], a0, a1, a2, a3, b[2], b[3]);
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty(s));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        named_bar(1, C::WARPS * 32);  // every warp has read its last stage
        float *os = reinterpret_cast<float *>(smem_raw + (ring - smem_u32(smem_raw)));
        float *ml = os + C::WARPS * C::ROWS * C::OS;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = warp * C::ROWS + g + 8 * h;
#pragma unroll
            for (int d = 0; d < HD / 8; ++d)
                *reinterpret_cast<float2 *>(os + r * C::OS + d * 8 + 2 * t) =
                    make_float2(o[d][2 * h], o[d][2 * h + 1]);
            if (t == 0) {
                ml[2 * r] = m[h];
                ml[2 * r + 1] = l[h];
            }
        }
        named_bar(1, C::WARPS * 32);
    }
    // merge: over the warps of a row, then over the cluster's CTAs
    float *os = reinterpret_cast<float *>(smem_raw + (ring - smem_u32(smem_raw)));
    float *ml = os + C::WARPS * C::ROWS * C::OS, *mc = ml + 2 * C::WARPS * C::ROWS;
    const int hd = a.hd, nt = C::WARPS * 32;
    const int quads = (hd + 3) / 4;
    if (tid < nt && !*fail)
        for (int i = tid; i < nrows * quads; i += nt) {
            const int r = i / quads, d = (i - r * quads) * 4;
            float2 w[C::WARPS];
            float M = -INFINITY, L = 0.f, O[4] = {};
#pragma unroll
            for (int k = 0; k < C::WARPS; ++k) {
                w[k] = *reinterpret_cast<const float2 *>(ml + 2 * (k * C::ROWS + r));
                M = fmaxf(M, w[k].x);
            }
#pragma unroll
            for (int k = 0; k < C::WARPS; ++k) {
                const float4 o =
                    *reinterpret_cast<const float4 *>(os + (k * C::ROWS + r) * C::OS + d);
                const float f = weigh(w[k].x, M);
                L = fmaf(w[k].y, f, L);
                O[0] = fmaf(o.x, f, O[0]);
                O[1] = fmaf(o.y, f, O[1]);
                O[2] = fmaf(o.z, f, O[2]);
                O[3] = fmaf(o.w, f, O[3]);
            }
            if (split == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (d + e < hd)
                        put(p, r0, kvh, r, d + e, O[e] / L, redo);
            } else {
                *reinterpret_cast<float4 *>(os + r * C::OS + d) =
                    make_float4(O[0], O[1], O[2], O[3]);
                if (d == 0) {
                    mc[2 * r] = M;
                    mc[2 * r + 1] = L;
                }
            }
        }
    if (split == 1) {
        __syncthreads();
    } else {
        cluster_sync_failed(fail, split);
        if (tid < nt && !*fail)
            merge_cluster<C::OS>(p, smem_u32(os), smem_u32(mc), r0, nrows, kvh, rank, tid, nt, redo);
        cluster_sync();  // no CTA leaves, or writes below, while another reads
    }
    if (warp < C::WARPS)
        redo_rows(p, redo, r0, nrows, kvh, rank, nt, warp, C::WARPS,
                  mc + 2 * C::ROWS + warp * kMaxHd);
    if (tid == 0 && *fail)
        atomicAdd(&g_timeouts, 1u);
}

// CTAs of a cluster that share a tile's keys: as many as all run at once and
// have `least` stages each (the longest tile's) to read.
int choose_split(const TileParams &p, int tile_rows, int ctas, int least)
{
    const AttnParams &a = p.a;
    const int last = a.pos + a.T - 1, first = a.pos + (p.tiles - 1) * tile_rows / a.group;
    const int lo = a.window && first - a.window + 1 > 0 ? first - a.window + 1 : 0;
    const int sinks = a.sinks < lo ? a.sinks : lo;
    const int64_t stages = (sinks + kKeys - 1) / kKeys + ((int64_t)last - lo + kKeys) / kKeys;
    const int64_t base = (int64_t)p.tiles * p.n_kv, room = (int64_t)sm_count() * ctas;
    int split = 1;
    while (split < 16 && base * split * 2 <= room && stages >= 2 * least * split)
        split *= 2;
    return split;
}

template <int HD, int WK, int GR>
cudaError_t launch_tiles(TileParams &p, cudaStream_t stream)
{
    using C = TileCfg<HD, WK, GR>;
    p.tiles = (p.rows + C::ROWS - 1) / C::ROWS;
    const int64_t base = (int64_t)p.tiles * p.n_kv;
    p.split = choose_split(p, C::ROWS, C::CTAS, 2);
    if (base * p.split > INT32_MAX)
        return cudaErrorInvalidValue;
    auto kernel = attn_tiles<HD, WK, GR>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e =
        allow_once(allowed, reinterpret_cast<const void *>(kernel), C::SMEM, true);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(base * p.split));
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
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ---- long prompts: tcgen05 --------------------------------------------------------
// Tiles of 128 rows (as above), a CTA or a cluster each, two CTAs to an SM so that one's
// products run under the other's softmax.  Both products run on tcgen05: S = Q
// K^T into one of two TMEM buffers, O += P V into a third, with P through
// shared memory in the layout the MMA reads, and V taken as it lies in the
// cache (its rows are the K of that product).  A thread of the four softmax
// warps has a row to itself: maximum and sum need no shuffles.  O is rescaled
// only when a row's maximum has grown by more than 8 (a published refinement of
// the running maximum; a factor of 256, exact in fp32 and bf16 alike); until then
// the weights are taken against the earlier maximum, which the final division by
// their sum makes good.
//
// Measured: 2048 tokens of 32 heads of 128 from position 0 on, window 1024 and 4
// sinks 59 us, without a window 58 us (594 TFLOP/s).  No pipe bounds it: tensor
// cores are busy for 27 % of the cycles, exponentials for 28 %, and a scheduler
// issues in 32 % of them.  The scores' product, the 64 keys of a thread's softmax
// and the product with V take turns within a CTA, which the other CTA of the SM
// covers in part.
template <int HD>
struct TcCfg {
    static constexpr int SUB = HD / 64;               // blocks of 64 elements of a head
    static constexpr int Q = SUB * 128 * 128, KV = SUB * kKeys * 128, P = 128 * 128;
    static constexpr int BARS = Q + 4 * KV + P;       // two stages of K and of V
    static constexpr int SMEM = BARS + 256 + 512;
    static constexpr int OS = HD + 4;                 // floats of a row of sums (padded)
    static_assert(128 * OS * 4 + 128 * 8 + 4 * kMaxHd * 4 <= Q + 4 * KV + P, "the sums reuse it all");
    static constexpr int THREADS = 256, COLS = 256;   // TMEM: two S of 64 columns, O from 128 on
};

template <int HD>
__global__ void __launch_bounds__(TcCfg<HD>::THREADS, 2)
    attn_tc(const __grid_constant__ TileParams p)
{
    using C = TcCfg<HD>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const uint32_t qs = base, ks = qs + C::Q, vs = ks + 2 * C::KV, ps = vs + 2 * C::KV;
    const uint32_t bar0 = base + C::BARS;
    const uint32_t q_full = bar0, p_full = bar0 + 8, o_done = bar0 + 16;
    auto k_full = [&](int b) { return bar0 + 24 + 8 * b; };
    auto k_empty = [&](int b) { return bar0 + 40 + 8 * b; };
    auto v_full = [&](int b) { return bar0 + 56 + 8 * b; };
    auto v_empty = [&](int b) { return bar0 + 72 + 8 * b; };
    auto s_full = [&](int b) { return bar0 + 88 + 8 * b; };
    auto s_free = [&](int b) { return bar0 + 104 + 8 * b; };
    int *flags = reinterpret_cast<int *>(smem + C::BARS + 128);  // TMEM address, failure
    volatile int *fail = flags + 1;
    int *redo = reinterpret_cast<int *>(smem + C::BARS + 256);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < 128)
        redo[tid] = 0;
    if (tid == 0) {
        flags[1] = (base & 1023) != 0;  // the swizzled layouts count from 1024-byte boundaries
        mbar_init(q_full, 4);
        mbar_init(p_full, 4);
        mbar_init(o_done, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(k_full(b), 1);
            mbar_init(k_empty(b), 1);
            mbar_init(v_full(b), 1);
            mbar_init(v_empty(b), 1);
            mbar_init(s_full(b), 1);
            mbar_init(s_free(b), 4);
        }
        mbar_init_fence();
        prefetch_map(&p.k);
        prefetch_map(&p.v);
    }
    if (warp == 2)
        tmem_alloc<C::COLS>(smem_u32(flags));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(flags);
    const AttnParams &a = p.a;
    const int split = p.split, rank = blockIdx.x % split;
    const int rest = blockIdx.x / split, kvh = rest % p.n_kv;
    const int r0 = (p.tiles - 1 - rest / p.n_kv) * 128;  // the longest rows start first
    const int nrows = min(128, p.rows - r0);
    const int pmin = a.pos + r0 / a.group, pmax = a.pos + (r0 + nrows - 1) / a.group;
    int na, lo;
    visible(a, pmin, na, lo);
    const int ta = (na + kKeys - 1) / kKeys;
    int t0, t1;
    share(ta + (pmax - lo + kKeys) / kKeys, rank, split, t0, t1);
    const int tn = *fail ? 0 : t1 - t0;  // stages of this CTA
    auto first_key = [&](int i) { return t0 + i < ta ? (t0 + i) * kKeys : lo + (t0 + i - ta) * kKeys; };
    pdl_wait();
    pdl_launch();
    if (warp == 0) {
        bool ok = true;
        int i = 0;
        for (; i < tn; ++i) {
            const int b = i & 1;
            const uint32_t ph = ((i >> 1) & 1) ^ 1;
            if (!warp_wait(k_empty(b), ph, fail)) {
                ok = false;
                break;
            }
            if (elect_one()) {
                mbar_expect_tx(k_full(b), C::KV);
#pragma unroll
                for (int d = 0; d < C::SUB; ++d)
                    tma_3d(ks + b * C::KV + d * kKeys * 128, &p.k, d * 64, first_key(i), kvh,
                           k_full(b));
            }
            __syncwarp();
            if (!warp_wait(v_empty(b), ph, fail)) {
                // K's copy of this stage is on its way
                for (int n = 0; n < (1 << 20) && !mbar_try_wait(k_full(b), ph ^ 1); ++n) {
                }
                ok = false;
                break;
            }
            if (elect_one()) {
                mbar_expect_tx(v_full(b), C::KV);
#pragma unroll
                for (int d = 0; d < C::SUB; ++d)
                    tma_3d(vs + b * C::KV + d * kKeys * 128, &p.v, d * 64, first_key(i), kvh,
                           v_full(b));
            }
            __syncwarp();
        }
        if (!ok)  // no copy may land after the CTA has gone
            for (int j = max(0, i - 2); j < i; ++j)
                for (int n = 0; n < (1 << 20) && !(mbar_try_wait(k_full(j & 1), (j >> 1) & 1) &&
                                                   mbar_try_wait(v_full(j & 1), (j >> 1) & 1));
                     ++n) {
                }
    } else if (warp == 1) {
        constexpr uint32_t is = tc_idesc(128, kKeys), io = tc_idesc(128, HD, true);
        auto pv = [&](int j) {  // O += P V of keys j
            const int b = j & 1;
            if (!warp_wait(p_full, j & 1, fail) || !warp_wait(v_full(b), (j >> 1) & 1, fail))
                return false;
            tc_fence_after();
            const uint64_t pd = tc_desc(ps), vd = tc_desc_mn(vs + b * C::KV, kKeys * 128);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)  // 16 keys: 32 bytes of P, 16 rows of V
                    tc_mma(tmem + 128, pd + 2 * k, vd + k * (16 * 128 >> 4), io, j + k ? 1u : 0u);
                tc_commit(v_empty(b));
                tc_commit(o_done);
            }
            __syncwarp();
            return true;
        };
        bool ok = tn == 0 || warp_wait(q_full, 0, fail);
        for (int i = 0; i < tn && ok; ++i) {
            const int b = i & 1;
            if (!warp_wait(k_full(b), (i >> 1) & 1, fail) ||
                !warp_wait(s_free(b), ((i >> 1) & 1) ^ 1, fail)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t qd = tc_desc(qs), kd = tc_desc(ks + b * C::KV);
            if (elect_one()) {
#pragma unroll
                for (int d = 0; d < C::SUB; ++d)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma(tmem + b * kKeys, qd + d * (128 * 128 >> 4) + 2 * k,
                               kd + d * (kKeys * 128 >> 4) + 2 * k, is, d + k ? 1u : 0u);
                tc_commit(k_empty(b));
                tc_commit(s_full(b));
            }
            __syncwarp();
            if (i > 0)
                ok = pv(i - 1);
        }
        if (ok && tn > 0)
            pv(tn - 1);
    } else if (warp >= 4) {
        const int r = tid - 128, row = r0 + r;
        const bool in = r < nrows;
        const int tok = in ? row / a.group : 0, h = kvh * a.group + (in ? row % a.group : 0);
        const int pr = in ? a.pos + tok : pmax;
        {  // the row's query, into the layout the MMA reads
            const uint16_t *q = a.q + tok * a.q_ts + h * a.q_hs;
#pragma unroll
            for (int c = 0; c < HD / 8; ++c) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (in && c * 8 + 8 <= a.hd) {
                    x = __ldg(reinterpret_cast<const uint4 *>(q) + c);
                } else if (in && c * 8 < a.hd) {
                    uint16_t e[8] = {};
                    for (int j = 0; c * 8 + j < a.hd; ++j)
                        e[j] = q[c * 8 + j];
                    memcpy(&x, e, 16);
                }
                sts128(qs + (c >> 3) * 128 * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4), x.x, x.y,
                       x.z, x.w);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full);
        }
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < tn; ++i) {
            const int b = i & 1, j0 = first_key(i);
            if (!warp_wait(s_full(b), (i >> 1) & 1, fail)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float s[kKeys];
#pragma unroll
            for (int c = 0; c < kKeys; c += 16)
                tmem_ld16(tmem + lanes + b * kKeys + c, *reinterpret_cast<float(*)[16]>(s + c));
#pragma unroll
            for (int c = 0; c < kKeys; c += 16)
                tmem_ld_wait(*reinterpret_cast<float(*)[16]>(s + c));
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(s_free(b));
            const bool sink = t0 + i < ta;
            if (sink ? j0 + kKeys > na
                     : j0 + kKeys - 1 > pmin || (a.window && j0 <= pmax - a.window)) {
                // keys j0 + e of the row: e < hi, and e >= from or e < sinks
                const int hi = sink ? na - j0 : pr - j0 + 1;
                const int from = !sink && a.window ? pr - a.window + 1 - j0 : 0;
                const int sk = sink ? 0 : a.sinks - j0;
#pragma unroll
                for (int e = 0; e < kKeys; ++e)
                    if (!(e < hi && (e >= from || e < sk)))
                        s[e] = -INFINITY;
            }
            float mx = s[0];
#pragma unroll
            for (int e = 1; e < kKeys; ++e)
                mx = fmaxf(mx, s[e]);
            mx *= a.scale_log2;  // scale > 0: the largest stays the largest
            const float mn = mx > m + 8.f || m == -INFINITY ? fmaxf(mx, m) : m;
            const float corr = mn == m ? 1.f : ex2(m - mn), ref = mn == -INFINITY ? 0.f : mn;
            m = mn;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < kKeys; ++e) {
                s[e] = ex2(fmaf(s[e], a.scale_log2, -ref));
                sum += s[e];
            }
            l = fmaf(l, corr, sum);
            if (i > 0 && !warp_wait(o_done, (i - 1) & 1, fail)) {  // O is whole, P has been read
                ok = false;
                break;
            }
            if (i > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < HD; c += 16) {
                    float o[16];
                    tmem_ld16(tmem + lanes + 128 + c, o);
                    tmem_ld_wait(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] *= corr;
                    tmem_st16(tmem + lanes + 128 + c, o);
                }
                tmem_st_wait();
            }
#pragma unroll
            for (int c = 0; c < kKeys / 8; ++c)
                sts128(ps + r * 128 + ((c ^ (r & 7)) << 4), f2_bf16(s[8 * c], s[8 * c + 1]),
                       f2_bf16(s[8 * c + 2], s[8 * c + 3]), f2_bf16(s[8 * c + 4], s[8 * c + 5]),
                       f2_bf16(s[8 * c + 6], s[8 * c + 7]));
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(p_full);
        }
        if (ok && tn > 0)
            ok = warp_wait(o_done, (tn - 1) & 1, fail);
        tc_fence_after();
        if (split > 1) {
            // this rank's sums for the cluster; every copy and product that used
            // the memory has finished (all four warps have seen the last one)
            named_bar(1, 128);
            float *os = reinterpret_cast<float *>(smem) + r * C::OS;
            float *ml = reinterpret_cast<float *>(smem) + 128 * C::OS + 2 * r;
            ml[0] = m;
            ml[1] = l;
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float o[16] = {};
                if (tn > 0) {
                    tmem_ld16(tmem + lanes + 128 + c, o);
                    tmem_ld_wait(o);
                }
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4 *>(os + c + e) =
                        make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        } else if (ok && tn > 0) {
            const float inv = 1.f / l;
            uint16_t *out = a.out + tok * a.o_ts + h * a.o_hs;
            const bool wide = ((uintptr_t)out & 15) == 0;
            bool finite = true;
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float o[16];
                tmem_ld16(tmem + lanes + 128 + c, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    o[e] *= inv;
                    finite &= c + e >= a.hd || fabsf(o[e]) < INFINITY;
                }
                if (in && wide && c + 16 <= a.hd) {
#pragma unroll
                    for (int e = 0; e < 16; e += 8)
                        *reinterpret_cast<uint4 *>(out + c + e) = make_uint4(
                            f2_bf16(o[e], o[e + 1]), f2_bf16(o[e + 2], o[e + 3]),
                            f2_bf16(o[e + 4], o[e + 5]), f2_bf16(o[e + 6], o[e + 7]));
                } else if (in) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c + e < a.hd)
                            out[c + e] = f_bf16(o[e]);
                }
            }
            // rows that are not finite again, by the warp (P has been read: its
            // memory takes the queries)
            uint32_t again = __ballot_sync(0xffffffffu, in && !finite);
            float *qrow = reinterpret_cast<float *>(smem + (ps - base)) + (warp - 4) * kMaxHd;
            while (again) {
                const int src = __ffs(again) - 1;
                again &= again - 1;
                const int t1 = __shfl_sync(0xffffffffu, tok, src);
                const int h1 = __shfl_sync(0xffffffffu, h, src);
                const uint16_t *q = a.q + t1 * a.q_ts + h1 * a.q_hs;
                __syncwarp();
                for (int d = lane; d < a.hd; d += 32)
                    qrow[d] = bf16f(q[d]) * a.scale_log2;
                __syncwarp();
                attend_row(a, t1, h1, qrow, [](int) { return true; });
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if (split > 1) {
        cluster_sync_failed(fail, split);
        const float *os = reinterpret_cast<const float *>(smem), *ml = os + 128 * C::OS;
        if (!*fail)
            merge_cluster<C::OS>(p, smem_u32(os), smem_u32(ml), r0, nrows, kvh, rank, tid,
                                 C::THREADS, redo);
        cluster_sync();  // no CTA leaves, or writes below, while another reads
        if (warp >= 4)
            redo_rows(p, redo, r0, nrows, kvh, rank, C::THREADS, warp - 4, 4,
                      reinterpret_cast<float *>(smem) + (warp - 4) * kMaxHd);
    }
    __syncthreads();
    if (tid == 0 && *fail)
        atomicAdd(&g_timeouts, 1u);
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc<C::COLS>(tmem);
    }
}

template <int HD>
cudaError_t launch_tc(TileParams &p, cudaStream_t stream)
{
    using C = TcCfg<HD>;
    p.tiles = (p.rows + 127) / 128;
    p.split = choose_split(p, 128, 2, 8);
    if ((int64_t)p.tiles * p.n_kv * p.split > INT32_MAX)
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e =
        allow_once(allowed, reinterpret_cast<const void *>(attn_tc<HD>), C::SMEM, true);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)p.tiles * p.n_kv * p.split));
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
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, attn_tc<HD>, p);
}

template <int HD>
cudaError_t launch_hd(TileParams &p, cudaStream_t stream)
{
    // Tiles of 16 rows while an SM and a half have one each: beyond that the
    // tensor cores' tiles of 128 (which want 16-byte query rows) read the cache
    // so much less often that their longer steps are made up for.  Measured: 333
    // tokens of 9 heads on 3 (189 tiles) 7.6 against 10.8 us, 128 tokens of 32
    // heads over 2128 rows (256 tiles) 29.2 against 26.4.
    const AttnParams &a = p.a;
    const int64_t small = (int64_t)((p.rows + 15) / 16) * p.n_kv;
    if (2 * small > 3 * sm_count() && aligned(a.q, 16) && a.q_ts % 8 == 0 && a.q_hs % 8 == 0)
        return launch_tc<HD>(p, stream);
    return launch_tiles<HD, 4, HD == 64 ? 2 : 1>(p, stream);
}

// Whether TMA can read the cache rows: 16-byte strides and bases.
bool fits_tiles(const amk_attention_args *a)
{
    auto rows = [&](const void *p, int64_t rs, int64_t hs) {
        return aligned(p, 16) && rs % 8 == 0 && rs >= a->head_dim &&
               (a->n_kv_heads == 1 || (hs % 8 == 0 && hs >= a->head_dim));
    };
    return a->head_dim <= 128 && (int64_t)a->n_tokens * (a->n_heads / a->n_kv_heads) < (1 << 28) &&
           rows(a->k, a->k_row_stride, a->k_head_stride) &&
           rows(a->v, a->v_row_stride, a->v_head_stride);
}

}  // namespace

cudaError_t timeouts_attention(uint32_t *n)
{
    return cudaMemcpyFromSymbol(n, g_timeouts, sizeof *n);
}

namespace {

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
    if (a->kv_rows > kMaxRows)
        return amk_set_error(AMK_ERR_UNSUPPORTED, "amk_attention: %d rows, at most %d", a->kv_rows,
                             kMaxRows);
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
    p.q_pairs = aligned(a->q, 4) && p.q_ts % 2 == 0 && p.q_hs % 2 == 0 && p.hd % 2 == 0;
    // a window or sinks beyond the last row mask nothing more, or less
    const int n = a->pos + a->n_tokens;
    p.window = a->window < n ? a->window : 0;
    p.sinks = a->sinks < n ? a->sinks : n;
    p.scale_log2 = (a->scale > 0.f ? a->scale : 1.f / sqrtf((float)a->head_dim)) * 1.4426950408889634f;
    if (!sm_count())
        return no_device("amk_attention");
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (fits_tiles(a)) {
        TileParams t;
        t.a = p;
        t.rows = a->n_tokens * p.group;
        t.n_kv = a->n_kv_heads;
        const int64_t rows = (int64_t)a->pos + a->n_tokens;  // what lies behind them reads as 0
        auto map = [&](CUtensorMap *m, const void *base, int64_t rs, int64_t hs) {
            return encode_3d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, a->head_dim, rows,
                             a->n_kv_heads, 2 * rs, 2 * (a->n_kv_heads == 1 ? rs : hs), 64, kKeys,
                             CU_TENSOR_MAP_SWIZZLE_128B);
        };
        if (!map(&t.k, a->k, a->k_row_stride, a->k_head_stride) ||
            !map(&t.v, a->v, a->v_row_stride, a->v_head_stride))
            return amk_set_error(AMK_ERR_CUDA, "amk_attention: a tensor map was refused");
        return launch_status(a->head_dim <= 64 ? launch_hd<64>(t, st) : launch_hd<128>(t, st),
                             "amk_attention");
    }
    const int64_t rows = (int64_t)a->n_tokens * a->n_heads;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((rows + 3) / 4 < (1 << 20) ? (rows + 3) / 4 : (1 << 20)));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    return launch_status(cudaLaunchKernelEx(&cfg, attn_rows, p), "amk_attention");
}
