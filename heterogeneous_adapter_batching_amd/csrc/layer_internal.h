// Internal interface of the operators around the delta (block norm, the
// frozen layer's product): argument blocks and kernel launchers.  The public
// interface is include/lora_sgmv.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "lora_sgmv.h"
#include "sgmv_internal.h"

namespace lora {

// ------------------------------------------------------------ block norm ----
// One row of the residual stream per 1 (narrow rows) to 16 waves, held in
// registers from its loads to its stores.
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

// ---------------------------------------------------------------- linear ----
// The adapters of one product call: the delta scale * B v of every token,
// added before the activation.  Columns are those before the activation
// (with a gated pair: gate's, then up's).
struct DeltaArgs {
    const int32_t *order;        // [T] token row of each plan position; null: no adapters
    const GroupRow *groups;      // adapter groups, in plan order
    const PosRow *pos;           // [T] the plan positions
    const uint8_t *v;            // the operand: [T positions][nproj][pieces][r_max],
    const float *partial;        // or (non-null) the shrink's partials it is summed from
    uint32_t partial_bytes;
    int32_t c0;                  // chunks of the partials
    const uint8_t *slab;
    int64_t coef_b[LORA_MAX_PROJ];  // B block offset = extent + r_pad * esize * coef_b[i]
    int32_t h_out[LORA_MAX_PROJ];
    int32_t y_off[LORA_MAX_PROJ];
    int32_t n_active;            // positions with an adapter (they come first)
    int32_t num_groups;          // (with the group of positions without one)
    int32_t max_rpad;            // largest padded rank of the plan
    int32_t nproj;
    int32_t r_max;
    uint32_t *dbg_word;          // debug build: where failed checks are noted
    DebugBounds dbg;
};

// The product's operand of the delta, scale * v, for every plan position of
// the adapter blocks [0, nb): of short groups' blocks summed from the
// shrink's partials, of long groups' ([0, nb_long)) read from v.
struct OperandArgs {
    const BlockDesc *blocks;
    const float *partial;
    const float *v;              // [T positions][nproj * r_max]
    const float *tok_w;          // weights by plan position (null: none)
    uint8_t *out;
    uint32_t partial_bytes;
    int32_t nb, nb_long, nproj, c0, r_max;
    uint32_t *dbg_word;          // debug build: where failed checks are noted
    DebugBounds dbg;
};
// The largest padded rank whose delta is one K-step of the matrix cores.  Up
// to it the joins (and the product of a few tokens) sum a lane's partials
// themselves, which spares a launch (q/k/v of a decode batch, rank 16: 44.7 us
// against 46.5 of kernels); beyond it every join wave would sum several steps'
// (a gated batch of ranks 8 to 64: the join 63.7 us against 43.4 with the
// operand formed once).
constexpr int one_step_rank(int dtype) { return dtype == LORA_BF16 ? 32 : 16; }
// bytes of one operand entry: three bf16 pieces, or the float32 value
constexpr int operand_bytes(int dtype) { return dtype == LORA_BF16 ? 6 : 4; }
hipError_t launch_operand(int dtype, const OperandArgs &a, hipStream_t s);

struct LinearArgs {
    const uint8_t *x, *w;        // [T][ldx], [wide][ldw]
    const uint8_t *bias;         // [wide] or null
    const uint8_t *residual;     // [T][ldr] or null
    uint8_t *y;                  // [T][ldy]
    float *partial;              // split products: [splits][T][ldp] float32
    int64_t ldx, ldw, ldr, ldy, ldp;   // elements
    int32_t T, k;
    int32_t n;                   // width of y
    int32_t wide;                // rows of w: n, or 2 n with a gated pair
    int32_t act;                 // lora_act
    int32_t tiles_t, tiles_n;    // tiles of the launch (tile kernel)
    int32_t splits, k_tiles;     // K tiles (128 bytes of a row) of one split
    int32_t units;               // workgroups with work (the grid is rounded up)
    DeltaArgs delta;
};

// How a product runs: one launch, or (joined) partial products along K and a
// launch that joins them.
enum LinearKind : int32_t { kLinearRows, kLinearTile };
struct LinearPlan {
    LinearKind kind;
    int32_t bt, bn;              // tokens and rows of w of a tile
    int32_t splits, k_tiles;     // parts along K, and K tiles of one
    bool joined;
    uint64_t ws_bytes;           // of the partial products
    uint64_t threads;            // of its largest launch
};
// Outputs of a workgroup of the join (max_rpad 0: no adapters).  A wave has 16
// columns, and 64 for bf16 adapters beyond one K-step, whose operand (6
// vectors a lane) then serves more rows of B (a gated decode batch of ranks 8
// to 64: 53.6, 42.2 and 40.7 us with 16, 32 and 64; rank 16 q/k/v 12.7 us with
// 16, 13.4 with 32).
constexpr int join_tiles(int dtype, int max_rpad) {
    return dtype == LORA_BF16 && max_rpad > one_step_rank(dtype) ? 4 : 1;
}
constexpr int join_cols(int dtype, bool glu, int max_rpad) {
    return (glu ? 32 : 64) * join_tiles(dtype, max_rpad);
}
// Whether a tile is built for products without adapters and for parts.
// float32's 128 x 128 is not: its K tile takes twice 64 x 128's, so that it is
// the better one only where the delta's K tiles, one set a token tile, weigh
// (683 x 3597 x 32 with one adapter).
constexpr bool plain_tile(int dtype, int bt, int bn) { return dtype == LORA_BF16 || bt * bn < 128 * 128; }
constexpr int kKBytes = 128;     // bytes of a row a K tile covers
constexpr int kRowsTokens = 12;  // most tokens of the rows kernel
// groups, max_rpad: adapter groups of the batch and their largest padded rank
// (0: no adapters)
LinearPlan linear_plan(int dtype, int T, int n, int k, bool glu, int groups, int max_rpad);
// the most workspace a plan of these sizes takes with at most max_groups
// adapters of padded ranks up to max_rpad
uint64_t linear_ws_bound(int dtype, int T, int n, int k, bool glu, int max_groups, int max_rpad);
// The arguments of a product call, as the entry points take them.
struct LinearCall {
    const lora_linear_desc *d;
    const void *x;
    int64_t ldx;
    const void *w;
    int64_t ldw;
    const void *bias, *residual;
    int64_t ldr;
    void *y;
    int64_t ldy;
    void *ws;
    uint64_t ws_bytes;
};
lora_status check_linear_desc(const lora_linear_desc *d);
// `need`: the workspace bytes of the call
lora_status check_linear(const LinearCall &c, const LinearPlan &pl, uint64_t need);
// Enqueues a checked call; partial sums at `partial` (of the plan's ws_bytes).
lora_status run_linear(const LinearCall &c, const LinearPlan &pl, void *partial,
                       const DeltaArgs &delta, hipStream_t s);
hipError_t launch_linear(int dtype, const LinearPlan &pl, bool glu, LinearArgs a, hipStream_t s);

}  // namespace lora
