// rope.cuh -- arguments of the rotary kernels.
#pragma once

#include "../../include/mla.h"
#include "common.cuh"

namespace mla {
namespace rp {

struct QueryParams {
    const __nv_bfloat16 *x;
    __nv_bfloat16 *y;
    int64_t ldx, x_head, ldy, y_head;  // elements
    const int32_t *positions, *seqlens;
    int tokens, heads, s_q;
};

struct AppendParams {
    const __nv_bfloat16 *x;
    int64_t ld;                  // elements between tokens
    int64_t tokens;
    int n_new;                   // tokens per sequence (cu_new null)
    const int32_t *cu_new;       // [batch + 1], or null
    const __nv_bfloat16 *weight; // [512], or null: the latent is stored as it comes
    float eps, inv_scale;
    const int32_t *positions;    // [tokens], or null: the position within the sequence
    uint8_t *kv;
    int64_t num_blocks, bt_stride;
    const int32_t *block_table, *seqlens;
    int batch;
};

}  // namespace rp
}  // namespace mla
