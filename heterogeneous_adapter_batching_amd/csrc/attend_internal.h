// Internal interface of the attention around the products (rotary positions
// into a paged cache, attention over it): descriptors, argument blocks and
// kernel launchers.  The public interface is include/lora_sgmv.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "lora_sgmv.h"
#include "sgmv_internal.h"

namespace lora {

// A sequence's new tokens and the query heads of one key head make the rows of
// its products with that head's keys: row r is token r / group, head r % group.
// They are cut into tiles of rows, a tile's keys into parts (units): one
// workgroup each.
struct AttnUnit {
    int32_t seq;                 // row of the page table; -1: no work
    int32_t kv_head;
    int32_t row0, rows;          // the tile's first row, and the rows of the sequence
    int32_t tok0;                // the sequence's first token in the batch
    int32_t pos0;                // and its position: kv_len - new tokens
    int32_t key0, key1;          // the unit's keys; key0 a multiple of kAttnBlock
    int32_t slot;                // its partial sums, or -1: it has all of the tile's keys
};
static_assert(sizeof(AttnUnit) == 36, "whole dwords");
// A tile in several parts, for the launch that joins them (no parts: none).
struct AttnJoin {
    int32_t tok0, kv_head, row0, rows, slot0, slots;
};
static_assert(sizeof(AttnJoin) == 24, "whole dwords");
struct AttnToken {
    int32_t seq, pos;            // pos: of the token's key in the cache
};

constexpr int kAttnPage = 16;    // pages hold a multiple of this many tokens
constexpr int kAttnBlock = 64;   // unit boundaries are multiples of this many keys

// What the debug build checks every table entry against before it is followed
// (LORA_SGMV_DEBUG): the batch, a sequence's row of the page table, the partial
// sums.  The word notes what failed (debug_word).
struct AttnBounds {
    int32_t tokens, seqs, kv_heads, group;
    int64_t keys;                // that pages_per_seq pages hold
    int64_t slots;
    uint32_t *word;
};
// The bits of what does not hold, 0 if all does (no sum can overflow, whatever
// the plan's memory has).
constexpr uint32_t wrong_tile(const AttnBounds &b, int32_t tok0, int32_t kv_head, int32_t row0,
                              int32_t rows) {
    return kv_head >= 0 && kv_head < b.kv_heads && tok0 >= 0 && row0 >= 0 && row0 <= rows &&
                   tok0 + (int64_t(rows) + b.group - 1) / b.group <= b.tokens
               ? 0u
               : kDbgToken;
}
constexpr uint32_t wrong(const AttnBounds &b, const AttnUnit &u) {
    if (u.seq == -1) return 0u;
    return wrong_tile(b, u.tok0, u.kv_head, u.row0, u.rows) |
           (u.seq >= 0 && u.seq < b.seqs && u.key0 >= 0 && u.key0 % kAttnBlock == 0 &&
                    u.key1 <= b.keys && (u.slot == -1 || (u.slot >= 0 && u.slot < b.slots))
                ? 0u
                : kDbgRow);
}
constexpr uint32_t wrong(const AttnBounds &b, const AttnJoin &j) {
    if (j.slots == 0) return 0u;
    return wrong_tile(b, j.tok0, j.kv_head, j.row0, j.rows) |
           (j.slots > 0 && j.slot0 >= 0 && int64_t(j.slot0) + j.slots <= b.slots ? 0u : kDbgRow);
}
constexpr uint32_t wrong(const AttnBounds &b, const AttnToken &t) {
    return t.seq >= 0 && t.seq < b.seqs && t.pos < b.keys ? 0u : kDbgRow;
}

// One head's rows of the cache, in elements.
struct CacheArgs {
    uint8_t *k, *v;
    int64_t k_page, k_head, k_tok, v_page, v_head, v_tok;
    int32_t num_pages, page_size;
};

struct AttnArgs {
    CacheArgs cache;
    const uint8_t *q;            // [T][ldq]
    uint8_t *o;                  // [T][ldo]
    int64_t ldq, ldo;            // elements
    const int32_t *pages;        // [seqs][ld_pages]
    int64_t ld_pages;
    const AttnUnit *units;
    const AttnJoin *joins;
    float *partial;              // [slots][rows of a tile][padded head]
    float *lse;                  // [slots][rows of a tile], in powers of two
    int32_t num_units, num_joins;
    int32_t group, head_dim;
    int32_t causal, window;      // window 0: all keys
    float scale2;                // scale log2 e
    // prompts, whose masked scores of -inf a scale has to leave what they are:
    // of -q, so that scale2 is positive; and of zeros for every finite element of
    // q where scale2 is zero (1 is passed)
    bool negate, zero;
    AttnBounds dbg;
};

// What a head is padded to, and the most rows of a tile of the kernel for few
// rows: single tokens, and float32 chunks of any length.  bfloat16 chunks have
// a kernel of their own from 17 rows on (64 sequences of 5 to 8 tokens, 8 key
// heads of 4 query heads, 2000 keys each: 109 us, the kernel for few rows with
// tiles of 32 rows 152; of 16 tokens 117 and 231 with tiles of 64; single
// tokens, 4 rows, of the batch of 128: 163 and 151).
constexpr int attn_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
constexpr int attn_rows_most(int dtype, int head_dim) {
    return dtype == LORA_BF16 ? 16 : head_dim <= 128 ? 64 : 32;
}
// Waves of a workgroup of tiles of 16 rows: 4, or (heads of up to 128) 8.
constexpr int kManyWaves = 8;
// once: no sequence has more than one tile of rows
hipError_t launch_attn_rows(int dtype, int tile_rows, int waves, bool once, const AttnArgs &a,
                            hipStream_t s);
constexpr int kPromptRows = 128; // of a tile of prompts
hipError_t launch_attn_prompt(const AttnArgs &a, hipStream_t s);
hipError_t launch_attn_join(int dtype, int tile_rows, const AttnArgs &a, hipStream_t s);

struct RotaryArgs {
    CacheArgs cache;             // k null: nothing is appended
    const uint8_t *q, *k, *v;    // [T][ld]; q null: keys and values only
    uint8_t *q_out;
    int64_t ldq, ldqo, ldk, ldv; // elements
    const int32_t *pages;
    int64_t ld_pages;
    const AttnToken *tokens;
    const int32_t *positions;    // null: the tokens' own
    const double *freqs;         // [rotary_dim / 2] radians a position; null: no rotation
    int32_t T, heads, kv_heads, head_dim, rotary_dim;
    int32_t layout;              // lora_rotary_layout
    float magnitude;
    AttnBounds dbg;
};
hipError_t launch_rotary(int dtype, const RotaryArgs &a, hipStream_t s);

}  // namespace lora
