"""What a wait that runs out leads to in the operators' kernels (csrc/amk_ops.cuh), on the GPU in a
kernel of its own: one warp of one CTA of a cluster waits for an arrival that nothing makes, gives
up after its second, and every warp and CTA learns of it and ends."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

PROBE = r"""
#include "amk_ops.cuh"
#include <cuda_runtime.h>
using namespace amk::ops;
// out: [CTA][5]: each warp's agreed word, then the CTA's flag behind the cluster's barrier
__global__ void give_up(int *out, int cta)
{
    __shared__ __align__(8) uint64_t bars[2];
    __shared__ int fail_flag;
    volatile int *fail = &fail_flag;
    const uint32_t bar = smem_u32(bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        fail_flag = 0;
        mbar_init(bar, 1);
        mbar_init(bar + 8, 1);
        mbar_init_fence();
        mbar_arrive(bar);  // the first barrier's phase is complete, the second's never is
    }
    __syncthreads();
    bool ok = warp_wait((int)blockIdx.x == cta && warp == 1 ? bar + 8 : bar, 0, fail);
    ok = named_bar_and(1, 128, ok);
    if (lane == 0)
        out[blockIdx.x * 5 + warp] = ok;
    cluster_sync_failed(fail, gridDim.x);
    if (threadIdx.x == 0)
        out[blockIdx.x * 5 + 4] = *fail;
}
extern "C" int run(int *out, int cta, int ctas)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(128);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, give_up, out, cta);
}
"""


def test_a_warp_that_gives_up_ends_its_cluster(cuda_ok, tmp_path):
    src, so = tmp_path / "give_up.cu", tmp_path / "give_up.so"
    src.write_text(PROBE)
    csrc = os.path.join(ROOT, "persistent_megakernel_decode_cta_b200", "csrc")
    subprocess.run([os.environ.get("NVCC", "nvcc"), "-gencode", "arch=compute_100a,code=sm_100a",
                    "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", csrc, str(src),
                    "-o", str(so)], check=True)
    run = ctypes.CDLL(str(so)).run
    run.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]
    for cta, ctas in ((2, 4), (-1, 4), (0, 2)):
        out = torch.full((ctas, 5), -1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        assert run(out.data_ptr(), cta, ctas) == 0
        torch.cuda.synchronize()
        want = [[int(i != cta)] * 4 + [int(cta >= 0)] for i in range(ctas)]
        assert out.tolist() == want
