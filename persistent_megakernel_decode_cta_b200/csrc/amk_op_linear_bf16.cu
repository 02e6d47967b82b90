// amk_op_linear_bf16.cu -- amk_linear's kernels for bf16 weights.
#include <atomic>

#include "amk_op_linear_skinny.cuh"

namespace amk {
namespace linear {

cudaError_t launch_bf16(const Variant &v, const TcParams &p, int grid, cudaStream_t stream)
{
    return launch_variant<AMK_QUANT_BF16>(v, p, grid, stream);
}

cudaError_t skinny_bf16(const SkinnyParams &p, cudaStream_t stream)
{
    return launch_skinny_of<AMK_QUANT_BF16>(p, stream);
}

cudaError_t timeouts_bf16(uint32_t *n)
{
    return cudaMemcpyFromSymbol(n, g_timeouts, sizeof *n);
}

}  // namespace linear
}  // namespace amk
