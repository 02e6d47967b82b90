// amk_kernel_inst_generic_gap.cu -- the generic kernel instance for steps whose
// window has moved on from the first cache rows (those of fused FFN levels too).
#include "amk_kernel_body.cuh"

namespace amk {
const void *amk_kernel_generic_gap()
{
    return reinterpret_cast<const void *>(amk_decode_kernel<0, 0, 1, 1, 1>);
}
}  // namespace amk
