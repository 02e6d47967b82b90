// amk_ops_host.cpp -- host helpers of the multi-token step's operators: tensor
// maps and device facts.
#include <atomic>

#include "amk_ops.h"

namespace amk {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn()
{
    static std::atomic<EncodeTiled> fn{nullptr};
    EncodeTiled f = fn.load(std::memory_order_relaxed);
    if (!f) {
        void *sym = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &sym, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            f = reinterpret_cast<EncodeTiled>(sym);
            fn.store(f, std::memory_order_relaxed);
        }
        cudaGetLastError();
    }
    return f;
}

bool encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base,
            const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
            CUtensorMapSwizzle swizzle)
{
    const EncodeTiled f = encode_fn();
    const cuuint32_t one[3] = {1, 1, 1};
    return f && f(map, type, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool encode_2d(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner,
               int64_t rows, int64_t pitch, int box_inner, int box_rows, CUtensorMapSwizzle swizzle)
{
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows};
    return encode(map, type, 2, base, dims, strides, box, swizzle);
}

bool encode_3d(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner,
               int64_t rows, int64_t planes, int64_t pitch, int64_t plane_pitch, int box_inner,
               int box_rows, CUtensorMapSwizzle swizzle)
{
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)plane_pitch};
    const cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows, 1};
    return encode(map, type, 3, base, dims, strides, box, swizzle);
}

int sm_count()
{
    static std::atomic<int> sms[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    n = sms[dev].load(std::memory_order_relaxed);
    if (!n && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
        sms[dev].store(n, std::memory_order_relaxed);
    return n;
}

int no_device(const char *what)
{
    int n = 0;
    const cudaError_t err = cudaGetDeviceCount(&n);
    return launch_status(err == cudaSuccess ? cudaErrorNoDevice : err, what);
}

cudaError_t allow_once(std::atomic<uint64_t> &done, const void *kernel, int smem, bool wide_cluster)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)))
        return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && wide_cluster)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && dev < 64)
        done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

}  // namespace amk

extern "C" int amk_ops_timeouts(uint32_t *n)
{
    using namespace amk;
    if (!n)
        return amk_set_error(AMK_ERR_INVALID_ARG, "amk_ops_timeouts: NULL");
    if (!sm_count())
        return no_device("amk_ops_timeouts");
    // the copies below wait for the default stream's work alone
    const cudaError_t done = cudaDeviceSynchronize();
    if (done != cudaSuccess)
        return launch_status(done, "amk_ops_timeouts");
    uint32_t sum = 0;
    for (auto f : {timeouts_attention, linear::timeouts_bf16, linear::timeouts_int8,
                   linear::timeouts_int4}) {
        uint32_t v = 0;
        const cudaError_t e = f(&v);
        if (e != cudaSuccess)
            return launch_status(e, "amk_ops_timeouts");
        sum += v;
    }
    *n = sum;
    return AMK_OK;
}
