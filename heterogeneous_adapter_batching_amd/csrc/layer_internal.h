// Internal interface of the operators around the delta (block norm, the
// frozen layer's product): argument blocks and kernel launchers.  The public
// interface is include/lora_sgmv.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "lora_sgmv.h"

namespace lora {

// ------------------------------------------------------------ block norm ----
// One row of the residual stream per 1 (narrow rows), 4, 8 or 16 waves, held
// in registers from its loads to its stores.
struct NormArgs {
    const void *h, *o;              // o null: no block output (h' = beta h)
    const void *post_w, *post_b;    // null: ones, zeros
    const void *gate;               // null: ones; rows at ldg elements (0: one row)
    const void *pre_w, *pre_b;
    void *h_out, *u;                // null: not written
    int64_t ldh, ldo, ldg, ldho, ldu;
    int32_t T, d;
    int32_t post, pre, gate_act;    // lora_norm_kind, lora_gate_act
    float alpha, beta, eps;
    float unit;                     // added to every weight (unit_offset)
};
constexpr int kNormChunk = 8;       // consecutive elements a lane holds
constexpr int kNormMaxWidth = 16 * 64 * kNormChunk * 4;   // 16 waves of 4 chunks a lane
static_assert(kNormMaxWidth == LORA_NORM_MAX_WIDTH, "the widest row the launch takes");
hipError_t launch_block_norm(int dtype, int stream_dtype, const NormArgs &a, hipStream_t s);

}  // namespace lora
