// shared.cuh -- what the shared-prefix decode's kernels, its partition and its host side agree on.
#pragma once

#include "common.cuh"

namespace mla {

struct SharedParams {
    const int32_t *shared_table;  // [shared_blocks]
    const int32_t *block_table;   // [batch, bt_stride]
    const int32_t *seqlens;       // [batch]
    const int32_t *tile_meta;     // [num_parts, 8]; [5]: prefix tokens that some sequence reaches
    const int32_t *num_splits;    // [units + 1] (cumulative)
    __nv_bfloat16 *out;           // [batch, s_q, h_q, 512]
    float *lse;                   // [batch, h_q, s_q]
    float *o_part;                // [prefix slots * 128 + own slots * own_rows, 512]
    float *lse_part;              // the same rows; base-2 logarithms
    int64_t num_blocks, bt_stride;
    int64_t own_base;             // first partial row of the own units
    int batch, s_q, h_q, rows;    // rows = s_q * h_q
    int total_rows;               // batch * rows
    int groups;                   // 128-row groups of one sequence
    int own_rows;                 // rows of an own unit's partial slot: min(rows, 128)
    int prefix_units, units, shared_blocks, num_parts;
    int causal, out_v8;
    float scale_log2;
};

constexpr int kSharedTileTok = 2 * kBlk;  // tokens of a tile: two cache blocks

// A sequence's length as the kernels take it (negative = 0; block and token counts stay in 32 bits).
__device__ __forceinline__ int clamp_len(int n) { return min(max(n, 0), INT32_MAX - 2 * kSharedTileTok); }

}  // namespace mla
