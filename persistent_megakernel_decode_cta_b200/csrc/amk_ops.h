// amk_ops.h -- what the operators of the multi-token step share on the host:
// the check for a device and the launch's error.
#ifndef AMK_OPS_H
#define AMK_OPS_H

#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "amk.h"
#include "amk_internal.h"

namespace amk {

inline bool aligned(const void *p, uintptr_t bytes)
{
    return ((uintptr_t)p & (bytes - 1)) == 0;
}

// AMK_OK, or why `what` cannot launch: no device, or the error that its
// launch left.
inline int launch_status(cudaError_t e, const char *what)
{
    if (e == cudaSuccess)
        return AMK_OK;
    cudaGetLastError();
    if (e == cudaErrorNoDevice || e == cudaErrorInsufficientDriver)
        return amk_set_error(AMK_ERR_NO_DEVICE, "%s: no CUDA device", what);
    return amk_set_error(AMK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Map of `rows` rows of `inner` elements, `pitch` bytes apart (and `planes` of
// them, plane_pitch bytes apart), in boxes of box_inner x box_rows; false when
// the driver refuses it.
bool encode_2d(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner,
               int64_t rows, int64_t pitch, int box_inner, int box_rows,
               CUtensorMapSwizzle swizzle);
bool encode_3d(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner,
               int64_t rows, int64_t planes, int64_t pitch, int64_t plane_pitch, int box_inner,
               int box_rows, CUtensorMapSwizzle swizzle);

int sm_count();                    // of the current device; 0: no device
int no_device(const char *what);   // the status of a call that found no device

// Limits of amk_attention: head sizes, and rows (positions and what is added to
// them stay in 32 bits).
constexpr int kAttentionMaxHd = 256;
constexpr int kAttentionMaxRows = 1 << 30;

// CTAs of the attention and linear kernels that gave up a wait on the current
// device (each source file counts its own).
cudaError_t timeouts_attention(uint32_t *n);
namespace linear {
cudaError_t timeouts_bf16(uint32_t *n);
cudaError_t timeouts_int8(uint32_t *n);
cudaError_t timeouts_int4(uint32_t *n);
}  // namespace linear

// Allows a kernel its dynamic shared memory (and clusters of 16), once per
// device; `done` is the kernel's own.
cudaError_t allow_once(std::atomic<uint64_t> &done, const void *kernel, int smem,
                       bool wide_cluster = false);

}  // namespace amk

#endif
