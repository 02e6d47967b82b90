// amk_kernel_inst_i4_split_gap.cu -- the kernel instances of amk_kernel_inst_i4_split.cu
// for steps whose window has moved on from the first cache rows.
#include "amk_kernel_body.cuh"

namespace amk {
const void *amk_kernel_q2_f0_gap(int e)
{
    switch (e) {
    case 0: return reinterpret_cast<const void *>(amk_decode_kernel<2, 1, 0, 0, 1>);
    case 1: return reinterpret_cast<const void *>(amk_decode_kernel<2, 2, 0, 0, 1>);
    case 2: return reinterpret_cast<const void *>(amk_decode_kernel<2, 4, 0, 0, 1>);
    case 3: return reinterpret_cast<const void *>(amk_decode_kernel<2, 8, 0, 0, 1>);
    default: return reinterpret_cast<const void *>(amk_decode_kernel<2, 16, 0, 0, 1>);
    }
}
}  // namespace amk
