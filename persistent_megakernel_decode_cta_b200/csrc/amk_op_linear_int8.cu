// amk_op_linear_int8.cu -- amk_linear's kernels for int8 weights.
#include <atomic>

#include "amk_op_linear_skinny.cuh"

namespace amk {
namespace linear {

cudaError_t launch_int8(const Variant &v, const TcParams &p, int grid, cudaStream_t stream)
{
    return launch_variant<AMK_QUANT_W8A16>(v, p, grid, stream);
}

cudaError_t skinny_int8(const SkinnyParams &p, cudaStream_t stream)
{
    return launch_skinny_of<AMK_QUANT_W8A16>(p, stream);
}

cudaError_t timeouts_int8(uint32_t *n)
{
    return cudaMemcpyFromSymbol(n, g_timeouts, sizeof *n);
}

}  // namespace linear
}  // namespace amk
