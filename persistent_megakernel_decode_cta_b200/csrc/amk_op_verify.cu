// amk_op_verify.cu -- amk_verify_draft: drafted tokens against the target's
// distributions, and the token drawn behind them.
//
// Two launches over chunks of kChunk logits.  The first takes the statistics
// of every chunk of every row (largest logit, sum of the exponentials); the
// second merges them, decides the acceptances -- every CTA the same way, from
// the same numbers -- and weighs the chunks of the one row that is drawn from;
// its last CTA to finish finds the chunk, then the token.  Exponentials and
// sums are fp64: whether a token is taken, and between which two of up to
// vocab borders a random number falls, are decisions, and cumulative sums of
// fp32 terms would move a border past it once in some thousand calls.  The
// logits are read once (the drawn row's again, from L2).
//
// Measured (us): no draft 49152 logits 9.5, 4 drafts 9 rows of 32000 11.4, 8
// drafts without a distribution 9 rows of 128256 14.8; a caller's Python takes
// about 13 a call.  Two launches and their latencies bound it (the reads take
// under 1 us of HBM), then the fp64 exponentials.
#include <math.h>

#include "amk_ops.cuh"
#include "amk_ops.h"

namespace amk {
namespace {

constexpr int kThreadsV = 256, kWarps = kThreadsV / 32, kPer = 8;
constexpr int kChunk = kThreadsV * kPer;
constexpr int kMaxDraft = 64, kMaxRows = 2 * kMaxDraft + 1;
constexpr int kMaxVocab = 1 << 30;  // indexes and a chunk beyond them stay in 32 bits

struct RowStat {
    double sum;   // of exp((x - m) / temperature)
    float m;      // largest logit
    int32_t arg;  // its lowest index; -1: the chunk holds NaN or +inf
};

struct VerifyParams {
    const float *target, *draft, *u;
    const int32_t *tok;
    int32_t *out, *n_acc;
    RowStat *stat;     // [rows][chunks]
    double *weight;    // [chunks]: of the drawn row
    float *tok_logit;  // [rows]: the drafted token's, where it is in the vocabulary
    uint32_t *done;    // CTAs of the second launch that have finished
    int64_t ts, ds;
    int32_t d, vocab, chunks, greedy;
    double inv_t;      // 1 / temperature
};

__device__ __forceinline__ const float *row_ptr(const VerifyParams &p, int r)
{
    return r <= p.d ? p.target + r * p.ts : p.draft + (r - p.d - 1) * p.ds;
}

// exp(y) for y <= 0 by a table and a short series (Tang, Table-driven
// implementation of the exponential function in IEEE floating-point arithmetic,
// 1989): y = (n / 64) ln 2 + r with |r| <= ln 2 / 128, so that
// exp(y) = 2^(n >> 6) 2^((n & 63) / 64) exp(r), the second from a table and the
// last by its series up to r^5 (the next term is below 2^-54).  ln 2 / 64 in
// two parts keeps r exact.  Half the operations of a general exp.
struct ExpTable {
    double t[64];  // 2^(j / 64)
};
__device__ __forceinline__ void fill_table(ExpTable &e)
{
    if (threadIdx.x < 64)
        e.t[threadIdx.x] = exp2(threadIdx.x / 64.0);
}
__device__ __forceinline__ double exp_neg(const ExpTable &e, double y)
{
    if (!(y > -700.0))  // below 1e-304: 0 beside the row's largest, which is 1; NaN stays
        return y != y ? y : 0.0;
    constexpr double kHi = 0x1.62e42fefa0000p-7, kLo = 0x1.cf79abc9e3b3ap-46;  // ln 2 / 64
    const double s = fma(y, 92.332482616893656877, 6755399441055744.0);  // rounds to an integer
    const int n = __double2loint(s);
    const double f = s - 6755399441055744.0;
    const double r = fma(f, -kLo, fma(f, -kHi, y));
    double q = fma(r, 1.0 / 120, 1.0 / 24);
    q = fma(r, q, 1.0 / 6);
    q = fma(r, q, 0.5);
    q = fma(r, q, 1.0);
    const double t = e.t[n & 63];
    const double v = fma(t * r, q, t);
    return __hiloint2double(__double2hiint(v) + ((n >> 6) << 20), __double2loint(v));
}
// exp((x - m) / temperature); 0 for a chunk or row without a finite logit
__device__ __forceinline__ double weight_of(const ExpTable &e, float x, float m, double inv_t)
{
    return m == -INFINITY ? 0.0 : exp_neg(e, ((double)x - (double)m) * inv_t);
}

// Sum over the CTA in a fixed order; every thread returns it.
__device__ double block_sum(double v, double *buf)
{
#pragma unroll
    for (int off = 16; off; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    __syncthreads();  // the buffer's last readers are through
    if ((threadIdx.x & 31) == 0)
        buf[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        s += buf[w];
    return s;
}

// The thread's kPer consecutive logits of a chunk (-inf behind its end).
__device__ __forceinline__ void load_chunk(const float *row, int b, int e, float (&x)[kPer])
{
    const int i = b + (int)threadIdx.x * kPer;
    if (i + kPer <= e && ((uintptr_t)(row + i) & 15) == 0) {
#pragma unroll
        for (int j = 0; j < kPer; j += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(row + i + j));
            x[j] = f.x, x[j + 1] = f.y, x[j + 2] = f.z, x[j + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            x[j] = i + j < e ? __ldg(row + i + j) : -INFINITY;
    }
}

__global__ void __launch_bounds__(kThreadsV) verify_stats(const VerifyParams p)
{
    __shared__ float wm[kWarps];
    __shared__ int wbad[kWarps], warg[kWarps];
    __shared__ double buf[kWarps];
    __shared__ ExpTable et;
    const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
    fill_table(et);
    ops::pdl_wait();
    ops::pdl_launch();
    if (c == 0 && r == 0 && tid == 0)
        *p.done = 0;
    const int b = c * kChunk, e = min(b + kChunk, p.vocab);
    const float *row = row_ptr(p, r);
    float x[kPer];
    load_chunk(row, b, e, x);
    // the drafted token's logit in this row, for the second launch
    const int i = r <= p.d ? r : r - p.d - 1;
    const int drafted = tid == 0 && i < p.d ? __ldg(p.tok + i) : -1;
    const bool here = drafted >= b && drafted < e;
    const float its = here ? __ldg(row + drafted) : 0.f;
    float m = -INFINITY;
    int bad = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        m = fmaxf(m, x[j]);
        bad |= !(x[j] < INFINITY);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    bad = __any_sync(0xffffffffu, bad);
    if ((tid & 31) == 0) {
        wm[tid >> 5] = m;
        wbad[tid >> 5] = bad;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        m = fmaxf(m, wm[w]);
        bad |= wbad[w];
    }
    int arg = INT32_MAX;
    double s = 0;
#pragma unroll
    for (int j = kPer - 1; j >= 0; --j)
        if (x[j] == m)
            arg = b + tid * kPer + j;
    if (!p.greedy)
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            s += weight_of(et, x[j], m, p.inv_t);
    arg = __reduce_min_sync(0xffffffffu, arg);
    if ((tid & 31) == 0)
        warg[tid >> 5] = arg;
    s = block_sum(s, buf);  // also orders warg
    if (tid == 0) {
        for (int w = 0; w < kWarps; ++w)
            arg = min(arg, warg[w]);
        RowStat o;
        o.sum = s;
        o.m = m;
        o.arg = bad ? -1 : arg;
        if (here)
            p.tok_logit[r] = its;
        p.stat[(int64_t)r * p.chunks + c] = o;
    }
}

struct Shared {
    ExpTable et;
    RowStat row[kMaxRows];
    double buf[kWarps];
    int n, stop, last_cta, pick, found, fallback;
    double before;
};

// What is drawn from, once the rows' statistics are known.
struct Draw {
    const float *prow, *qrow;  // qrow null: no distribution to subtract
    float pm, qm;
    double fp, fq;  // 1 / sum of the row's exponentials
    int skip;       // a lookup draft that was rejected: all of q is on this token
};

// The weights of the thread's tokens of a chunk: max(p - q, 0), or, with
// `whole`, p itself; returns their sum.
__device__ double chunk_weights(const VerifyParams &p, const ExpTable &et, const Draw &dr, int b,
                                bool whole, double (&w)[kPer])
{
    const int e = min(b + kChunk, p.vocab);
    float x[kPer];
    load_chunk(dr.prow, b, e, x);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        w[j] = weight_of(et, x[j], dr.pm, p.inv_t);
    if (!whole) {
        if (dr.qrow) {
            load_chunk(dr.qrow, b, e, x);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                // both products rounded (no FMA), so that equal rows leave exactly 0
                w[j] = fmax(__dmul_rn(w[j], dr.fp) -
                                __dmul_rn(weight_of(et, x[j], dr.qm, p.inv_t), dr.fq),
                            0.0);
        }
        const int at = dr.skip - (b + (int)threadIdx.x * kPer);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j == at)
                w[j] = 0.0;
    }
    double s = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        s += w[j];
    return s;
}

__global__ void __launch_bounds__(kThreadsV) verify_draw(const VerifyParams p)
{
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int R = p.d + 1 + (p.draft ? p.d : 0);
    fill_table(sh.et);
    if (tid == 0)
        sh.n = p.d;
    __syncthreads();
    ops::pdl_wait();
    ops::pdl_launch();
    // the rows' statistics, merged in a fixed order: the largest logit first, so
    // that a chunk's sum takes one exponential
    const RowStat none = {0.0, -INFINITY, INT32_MAX};
    auto stat_of = [&](int r) {  // the lane's chunk of the first 32
        return r < R && lane < p.chunks ? p.stat[(int64_t)r * p.chunks + lane] : none;
    };
    RowStat next = stat_of(warp);
    for (int r = warp; r < R; r += kWarps) {
        const RowStat *st = p.stat + (int64_t)r * p.chunks, s0 = next;
        next = stat_of(r + kWarps);  // on its way while this row is merged
        float m = s0.m;
        int bad = s0.arg < 0;
        for (int c = lane + 32; c < p.chunks; c += 32) {
            m = fmaxf(m, st[c].m);
            bad |= st[c].arg < 0;
        }
#pragma unroll
        for (int off = 16; off; off >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        bad = __any_sync(0xffffffffu, bad || m == -INFINITY);  // nothing but -inf: no distribution
        double sum = s0.sum * weight_of(sh.et, s0.m, m, p.inv_t);
        int arg = s0.m == m ? s0.arg : INT32_MAX;
        for (int c = lane + 32; c < p.chunks; c += 32) {
            const RowStat s = st[c];
            sum += s.sum * weight_of(sh.et, s.m, m, p.inv_t);
            if (s.m == m)
                arg = min(arg, s.arg);
        }
        arg = __reduce_min_sync(0xffffffffu, arg);
#pragma unroll
        for (int off = 16; off; off >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) {
            RowStat s;
            s.sum = sum;
            s.m = m;
            s.arg = bad ? -1 : arg;
            sh.row[r] = s;
        }
    }
    __syncthreads();
    // the row at which the accepted run ends: the lowest one that is not
    // accepted, has no distribution, or is the last
    static_assert(kMaxDraft < kThreadsV, "a thread per row");
    bool bad = false;
    if (tid <= p.d) {
        const RowStat ps = sh.row[tid];
        bad = ps.arg < 0;
        bool ok = false;
        if (tid < p.d) {
            const int t = p.tok[tid];
            const bool in = t >= 0 && t < p.vocab;
            if (p.greedy) {
                ok = ps.arg == t;
            } else {
                double qt = 1.0;
                if (p.draft) {
                    const RowStat qs = sh.row[p.d + 1 + tid];
                    bad = bad || qs.arg < 0;
                    if (in)
                        qt = weight_of(sh.et, p.tok_logit[p.d + 1 + tid], qs.m, p.inv_t) / qs.sum;
                }
                if (in)
                    ok = (double)p.u[tid] * qt <
                         weight_of(sh.et, p.tok_logit[tid], ps.m, p.inv_t) / ps.sum;
            }
        }
        if (bad || !ok)
            atomicMin(&sh.n, tid);
    }
    __syncthreads();
    if (tid == sh.n)
        sh.stop = bad;
    __syncthreads();
    const int n = sh.n;
    auto write = [&](int token) {
        for (int i = tid; i <= p.d; i += kThreadsV)
            p.out[i] = i < n ? p.tok[i] : i == n ? token : -1;
        if (tid == 0)
            *p.n_acc = n;
    };
    if (p.greedy || sh.stop) {  // nothing to draw
        if (blockIdx.x == 0)
            write(sh.stop ? -1 : sh.row[n].arg);
        return;
    }
    Draw dr;
    const bool rejected = n < p.d;
    dr.prow = row_ptr(p, n);
    dr.pm = sh.row[n].m;
    dr.fp = 1.0;
    dr.qrow = nullptr;
    dr.qm = 0.f;
    dr.fq = 0.0;
    dr.skip = rejected && !p.draft && (uint32_t)p.tok[n] < (uint32_t)p.vocab ? p.tok[n] : -1;
    if (rejected && p.draft) {
        dr.qrow = row_ptr(p, p.d + 1 + n);
        dr.qm = sh.row[p.d + 1 + n].m;
        dr.fp = 1.0 / sh.row[n].sum;
        dr.fq = 1.0 / sh.row[p.d + 1 + n].sum;
    }
    double w[kPer];
    double own = chunk_weights(p, sh.et, dr, blockIdx.x * kChunk, false, w);  // a CTA to a chunk
    {
        const double s = block_sum(own, sh.buf);
        if (tid == 0)
            p.weight[blockIdx.x] = s;
    }
    // the last CTA to finish draws: its counter update follows its own weights
    // and precedes its loads of the others'
    if (tid == 0) {
        sh.last_cta = 1;
        if (gridDim.x > 1) {
            __threadfence();
            sh.last_cta = atomicAdd(p.done, 1u) == gridDim.x - 1;
            __threadfence();
        }
    }
    __syncthreads();
    if (!sh.last_cta)
        return;
    const double u = fmin(fmax((double)p.u[p.d], 0.0), 1.0);
    for (int whole = 0; whole < 2; ++whole) {
        // whole: max(p - q, 0) is 0 everywhere, p itself is drawn from
        if (whole) {
            for (int c = 0; c < p.chunks; ++c) {
                const double s = block_sum(chunk_weights(p, sh.et, dr, c * kChunk, true, w), sh.buf);
                if (tid == 0)
                    p.weight[c] = s;
            }
            __syncthreads();
        }
        if (warp == 0) {
            // inclusive sums of 32 chunks' weights at a time
            auto scan = [&](int c0, double &own) {
                own = c0 + lane < p.chunks ? __ldcg(p.weight + c0 + lane) : 0.0;
                double inc = own;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const double o = __shfl_up_sync(0xffffffffu, inc, off);
                    if (lane >= off)
                        inc += o;
                }
                return inc;
            };
            double own, total = 0;
            for (int c0 = 0; c0 < p.chunks; c0 += 32)
                total += __shfl_sync(0xffffffffu, scan(c0, own), 31);
            // the first chunk whose cumulative weight passes x, else (u = 1, or
            // rounding at the end) the last one with a weight
            const double x = u * total;
            double cum = 0, before = 0;
            int pick = -1;
            for (int c0 = 0; c0 < p.chunks && total > 0; c0 += 32) {
                const double inc = scan(c0, own);
                const uint32_t some = __ballot_sync(0xffffffffu, own > 0);
                const uint32_t past = __ballot_sync(0xffffffffu, own > 0 && cum + inc > x);
                const int at = past ? __ffs(past) - 1 : 31 - __clz(some);
                if (some) {
                    pick = c0 + at;
                    before = __shfl_sync(0xffffffffu, cum + (inc - own), at);
                }
                if (past)
                    break;
                cum += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) {
                sh.pick = pick;
                sh.before = x - before;  // what is left to pass within the chunk
                sh.found = INT32_MAX;
                sh.fallback = -1;
            }
        }
        __syncthreads();
        if (sh.pick < 0)
            continue;  // the same for every thread
        const double x = sh.before;
        if (whole || sh.pick != (int)blockIdx.x)  // else the weights are still here
            own = chunk_weights(p, sh.et, dr, sh.pick * kChunk, whole, w);
        double inc = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off)
                inc += o;
        }
        __syncthreads();
        if (lane == 31)
            sh.buf[warp] = inc;
        __syncthreads();
        double cum = inc - own;
        for (int k = 0; k < warp; ++k)
            cum += sh.buf[k];
        int found = INT32_MAX, last = -1;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            cum += w[j];
            if (w[j] > 0) {
                last = sh.pick * kChunk + tid * kPer + j;
                if (cum > x && found == INT32_MAX)
                    found = last;
            }
        }
        found = __reduce_min_sync(0xffffffffu, found);
        last = __reduce_max_sync(0xffffffffu, last);
        if (lane == 0) {
            atomicMin(&sh.found, found);
            atomicMax(&sh.fallback, last);
        }
        __syncthreads();
        break;
    }
    write(sh.found != INT32_MAX ? sh.found : sh.fallback);
}

int64_t workspace_bytes(int n_draft, int vocab)
{
    const int64_t chunks = ((int64_t)vocab + kChunk - 1) / kChunk;
    const int64_t rows = 2 * (int64_t)n_draft + 1;
    return rows * chunks * (int64_t)sizeof(RowStat) + chunks * (int64_t)sizeof(double) +
           rows * (int64_t)sizeof(float) + 16;
}

int check_verify(const amk_verify_args *a)
{
    auto bad = [](const char *what) {
        return amk_set_error(AMK_ERR_INVALID_ARG, "amk_verify_draft: %s", what);
    };
    if (!a)
        return bad("NULL arguments");
    if (a->n_draft < 0 || a->vocab < 1)
        return bad("n_draft < 0 or vocab < 1");
    if (a->n_draft > kMaxDraft)
        return amk_set_error(AMK_ERR_UNSUPPORTED, "amk_verify_draft: %d drafted tokens, at most %d",
                             a->n_draft, kMaxDraft);
    if (a->vocab > kMaxVocab)
        return amk_set_error(AMK_ERR_UNSUPPORTED, "amk_verify_draft: vocabulary of %d, at most %d",
                             a->vocab, kMaxVocab);
    if (!(a->temperature == 0.f || (a->temperature >= 1e-6f && a->temperature <= 1e6f)))
        return bad("temperature is not 0 or within [1e-6, 1e6]");
    if (!a->target || !a->u || !a->tokens || !a->n_accepted || (a->n_draft && !a->draft_tokens))
        return bad("a pointer is NULL");
    if (!aligned(a->target, 4) || !aligned(a->draft, 4) || !aligned(a->u, 4) ||
        !aligned(a->draft_tokens, 4) || !aligned(a->tokens, 4) || !aligned(a->n_accepted, 4))
        return bad("a pointer is not aligned to its element");
    if ((a->n_draft && a->target_stride < a->vocab) ||
        (a->n_draft > 1 && a->draft && a->draft_stride < a->vocab))
        return bad("a row stride is less than the row");
    if (!a->workspace || !aligned(a->workspace, 16) ||
        a->workspace_bytes < workspace_bytes(a->n_draft, a->vocab))
        return bad("the workspace is NULL, not 16-byte aligned or too small");
    return AMK_OK;
}

}  // namespace
}  // namespace amk

extern "C" int64_t amk_verify_workspace(int32_t n_draft, int32_t vocab)
{
    if (n_draft < 0 || n_draft > amk::kMaxDraft || vocab < 1 || vocab > amk::kMaxVocab)
        return amk_set_error(AMK_ERR_INVALID_ARG, "amk_verify_workspace: n_draft outside [0, %d] or "
                             "vocab outside [1, %d]", amk::kMaxDraft, amk::kMaxVocab);
    return amk::workspace_bytes(n_draft, vocab);
}

extern "C" int amk_verify_draft(const amk_verify_args *a, void *cuda_stream)
{
    using namespace amk;
    const int rc = check_verify(a);
    if (rc != AMK_OK)
        return rc;
    VerifyParams p{};
    p.target = a->target;
    p.draft = a->n_draft ? a->draft : nullptr;
    p.u = a->u;
    p.tok = a->draft_tokens;
    p.out = a->tokens;
    p.n_acc = a->n_accepted;
    p.ts = a->target_stride;
    p.ds = a->draft_stride;
    p.d = a->n_draft;
    p.vocab = a->vocab;
    p.chunks = (int)(((int64_t)a->vocab + kChunk - 1) / kChunk);
    p.greedy = a->temperature == 0.f;
    p.inv_t = p.greedy ? 1.0 : 1.0 / (double)a->temperature;
    const int rows = p.d + 1 + (p.draft ? p.d : 0);
    p.stat = static_cast<RowStat *>(a->workspace);
    p.weight = reinterpret_cast<double *>(p.stat + (int64_t)rows * p.chunks);
    p.tok_logit = reinterpret_cast<float *>(p.weight + p.chunks);
    p.done = reinterpret_cast<uint32_t *>(p.tok_logit + rows);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.chunks, (unsigned)rows);
    cfg.blockDim = dim3(kThreadsV);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, verify_stats, p);
    if (e == cudaSuccess) {
        cfg.gridDim = dim3((unsigned)p.chunks);
        e = cudaLaunchKernelEx(&cfg, verify_draw, p);
    }
    return launch_status(e, "amk_verify_draft");
}
