// amk_ops.h -- what the operators of the multi-token step share on the host:
// the check for a device and the launch's error.
#ifndef AMK_OPS_H
#define AMK_OPS_H

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

}  // namespace amk

#endif
