// amk_extend.h -- the multi-token step of a handle (amk_extend): what
// amk_host.cpp passes to the kernels' sequence in amk_extend.cu.
#ifndef AMK_EXTEND_H
#define AMK_EXTEND_H

#include <vector>

#include "amk_ops.h"

namespace amk {

// The caller's weights, kept by the handle (device pointers; layer arrays copied).
struct ModelWeights {
    const void *embed, *final_norm, *lm_head, *lm_head_scale;
    std::vector<const void *> norm[2];      // attention, FFN
    std::vector<const void *> mat[7];       // q k v o gate up down (W_Q ..)
    std::vector<const void *> scale[7];     // empty for bf16
};

// Activations of up to `chunk` tokens, in one block.
struct ExtendBuffers {
    int32_t chunk;
    int32_t *tokens;   // [chunk]
    float2 *rope;      // [chunk][head_dim / 2]: cosine, sine
    float *x;          // [chunk][hidden]: the residual stream
    uint16_t *xn;      // [chunk][hidden]: normed, bf16
    float *qkv;        // [chunk][qkv_rows]
    uint16_t *q;       // [chunk][n_heads * head_dim]: rotated, bf16
    uint16_t *attn;    // [chunk][n_heads * head_dim]
    uint16_t *act;     // [chunk][ffn]
};
size_t extend_bytes(const amk_config &c, int32_t chunk);
ExtendBuffers extend_buffers(const amk_config &c, int32_t chunk, void *block);

// Runs n <= chunk tokens (already in b.tokens) at positions pos .. through the
// model, appending their K and V to the cache, and the last n_logits of them
// through the head into logits [n_logits][vocab].
int extend_chunk(const amk_config &c, const ModelWeights &w, const ExtendBuffers &b, uint16_t *kv,
                 int32_t n, int32_t pos, int32_t window, int32_t sinks, int32_t n_logits,
                 float *logits, cudaStream_t stream);

}  // namespace amk

#endif
