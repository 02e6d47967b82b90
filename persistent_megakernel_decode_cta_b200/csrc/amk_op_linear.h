// amk_op_linear.h -- what the kernels of amk_linear share.
#ifndef AMK_OP_LINEAR_H
#define AMK_OP_LINEAR_H

#include <cuda.h>

#include "amk_ops.h"

namespace amk {
namespace linear {

// The epilogue of an output: act(a + bias) [* (u + up_bias)] [+ residual].
struct Epilogue {
    const uint16_t *bias, *up_bias;      // bf16 [n], or null
    const uint16_t *w_scale, *up_scale;  // fp16 row scales (W8A16), or null
    const void *residual;
    void *y;
    int64_t ldr, ldy;
    int32_t m, n, act, gated, res_f32, y_f32;
};

// A launch of the tensor-core kernel.
struct TcParams {
    CUtensorMap x, w, up;
    const uint16_t *w_gs, *up_gs;  // int4 group scales [n][groups]
    int32_t groups;
    int32_t blocks;                // K blocks
    int32_t seg;                   // K blocks summed before their sum is added in fp32
    int32_t tiles_m, tiles;
    int32_t split;                 // CTAs of a cluster that share a tile's K
    Epilogue e;
};

// One variant: `nt` tokens by 128 rows of weights to a tile.
struct Variant {
    int nt;
    bool split;    // a cluster to a tile, its CTAs sharing K; else CTAs that walk the tiles
    bool promote;  // sums of `seg` K blocks are added up in fp32 registers
};

// A launch of the kernel for few tokens.
constexpr int kSkinnyTokens = 16;
constexpr int kSkinnyRows = 64;  // rows of weights of a CTA: two groups of 32
constexpr int kSkinnyKG = 4;     // warps that share a group's K
struct SkinnyParams {
    const uint16_t *x;
    const void *w, *up;
    const uint16_t *w_gs, *up_gs;  // int4 group scales [n][groups]
    int64_t ldx, row_bytes;
    int32_t k, groups;
    int32_t split;                 // CTAs of a cluster that share K
    Epilogue e;
};
cudaError_t skinny_bf16(const SkinnyParams &p, cudaStream_t stream);
cudaError_t skinny_int8(const SkinnyParams &p, cudaStream_t stream);
cudaError_t skinny_int4(const SkinnyParams &p, cudaStream_t stream);

// Launches the variant for a weight format (in its own source file each).
cudaError_t launch_bf16(const Variant &v, const TcParams &p, int grid, cudaStream_t stream);
cudaError_t launch_int8(const Variant &v, const TcParams &p, int grid, cudaStream_t stream);
cudaError_t launch_int4(const Variant &v, const TcParams &p, int grid, cudaStream_t stream);

}  // namespace linear
}  // namespace amk

#endif
