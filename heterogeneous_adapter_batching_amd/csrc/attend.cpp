// Host side of the attention around the products: the plan of a batch's
// sequences over a paged cache, validation and launches of rotary_append and
// paged_attention.  Nothing is enqueued unless every argument holds.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <iterator>
#include <memory>
#include <vector>

#include <hip/hip_runtime.h>

#include "attend_internal.h"
#include "lora_sgmv.h"
#include "sgmv_internal.h"

using lora::AttnJoin;
using lora::AttnToken;
using lora::AttnUnit;
using lora::set_errorf;

namespace {

int32_t esize(int32_t dtype) { return dtype == LORA_BF16 ? 2 : 4; }
bool is_dtype(int32_t d) { return d == LORA_F32 || d == LORA_BF16; }
uint64_t round_up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

constexpr int32_t kMostTokens = 1 << 23, kMostKeys = 1 << 30;
// The largest stride, in elements, and the most elements from a cache's first
// page to its last: what follows from them stays within 64 bits.
constexpr int64_t kMostStride = int64_t(1) << 36, kMostCache = int64_t(1) << 40;

// Units a launch aims for when it cuts the tiles' keys into parts, and the
// fewest keys of a part.  With heads of 128 the kernel for few rows has two
// workgroups a CU, the prompts' too: a round, or two of them (four sequences
// behind 68157 to 127138 keys, us: 512 parts 383, 768 324, 1024 299, 1536 324,
// 2048 302; 128 sequences of 19 to 7824 keys 144, 137, 141, 140, 141).  Heads of
// 64 and 256, four workgroups and one a CU, take the same numbers.
constexpr int kRowsUnits = 1024, kRowsKeys = 256;
constexpr int kPromptUnits = 512, kPromptKeys = 512;
constexpr int kCus = 256, kShortKeys = 1024;

// One kernel's share of a plan: its tiles of rows, and their keys in parts.
struct Side {
    int32_t tile_rows = 0, waves = 4;      // rows of a tile; waves of a workgroup (few rows)
    bool once = true;                      // no sequence has more than one tile (few rows)
    int64_t tiles = 0;                     // tiles of rows, over all key heads
    std::vector<AttnUnit> units;
    std::vector<AttnJoin> joins;
    int64_t cap_units = 0, cap_joins = 0, cap_slots = 0;   // places in the workspace
    uint64_t off_units = 0, off_joins = 0, off_partial = 0, off_lse = 0;

    void clear() {
        Side empty;
        empty.units.swap(units);
        empty.joins.swap(joins);
        empty.units.clear();
        empty.joins.clear();
        *this = std::move(empty);
    }
};

// What a plan holds of its batch: built as a whole, so that a rebuild that fails
// leaves the last one.
struct Batch {
    lora_attn_desc d{};
    int32_t group = 1;
    std::vector<int32_t> new_lens, kv_lens;
    std::vector<AttnToken> tokens;
    int32_t most_kv = 0;
    Side rows, prompt;
    uint64_t off_tokens = 0, image_bytes = 0, ws_bytes = 0;
};

}  // namespace

struct attn_plan : Batch {
    Batch spare;                           // where a rebuild builds; the two change places
    void *ws = nullptr;
    // pinned staging, two buffers in turn: an upload waits only for the copy
    // before last
    void *staging[2] = {nullptr, nullptr};
    uint64_t staging_bytes[2] = {0, 0};
    hipEvent_t staged[2] = {nullptr, nullptr};
    int32_t next_staging = 0;
};

namespace {

lora_status check_attn_desc(const lora_attn_desc *d) {
    if (!d) return set_errorf(LORA_EINVAL, "null attention descriptor");
    if (!is_dtype(d->dtype))
        return set_errorf(LORA_EDTYPE, "dtype %d is neither LORA_F32 nor LORA_BF16", d->dtype);
    if (d->kv_heads < 1 || d->heads < d->kv_heads || d->heads > LORA_ATTN_MAX_HEADS ||
        d->heads % d->kv_heads)
        return set_errorf(LORA_EINVAL, "%d heads over %d key heads: a multiple of them, at most %d",
                          d->heads, d->kv_heads, LORA_ATTN_MAX_HEADS);
    if (d->head_dim < 8 || d->head_dim % 8 || d->head_dim > LORA_ATTN_MAX_HEAD_DIM)
        return set_errorf(LORA_EINVAL, "head_dim %d is not a multiple of 8 in 8..%d", d->head_dim,
                          LORA_ATTN_MAX_HEAD_DIM);
    if (d->page_size < lora::kAttnPage || d->page_size % lora::kAttnPage ||
        d->page_size > LORA_ATTN_MAX_PAGE)
        return set_errorf(LORA_EINVAL, "page_size %d is not a multiple of %d in %d..%d",
                          d->page_size, lora::kAttnPage, lora::kAttnPage, LORA_ATTN_MAX_PAGE);
    if (d->causal != 0 && d->causal != 1)
        return set_errorf(LORA_EINVAL, "causal %d is neither 0 nor 1", d->causal);
    if (d->window < 0 || (d->window && !d->causal))
        return set_errorf(LORA_EINVAL, "window %d: 0 or, with causal, a number of keys", d->window);
    if (d->max_kv < 0 || d->max_kv > kMostKeys)
        return set_errorf(LORA_EINVAL, "max_kv %d not in 0..%d", d->max_kv, kMostKeys);
    return LORA_OK;
}

lora_status check_lens(const lora_attn_desc &d, const int32_t *new_lens, const int32_t *kv_lens,
                       int32_t S) {
    if (S < 0 || S > kMostTokens)
        return set_errorf(LORA_EINVAL, "num_seqs %d not in 0..%d", S, kMostTokens);
    if (S && (!new_lens || !kv_lens)) return set_errorf(LORA_EINVAL, "null table of lengths");
    int64_t tokens = 0, tiles = 0;
    for (int32_t s = 0; s < S; ++s) {
        if (new_lens[s] < 0 || new_lens[s] > kMostTokens)
            return set_errorf(LORA_EINVAL, "sequence %d: %d new tokens", s, new_lens[s]);
        if (kv_lens[s] < 0 || kv_lens[s] > kMostKeys)
            return set_errorf(LORA_EINVAL, "sequence %d: %d keys not in 0..%d", s, kv_lens[s],
                              kMostKeys);
        if (d.causal && kv_lens[s] < new_lens[s])
            return set_errorf(LORA_EINVAL, "sequence %d: %d keys are fewer than its %d new tokens",
                              s, kv_lens[s], new_lens[s]);
        if (d.max_kv && kv_lens[s] > d.max_kv)
            return set_errorf(LORA_EINVAL, "sequence %d: %d keys are more than the plan's max_kv %d",
                              s, kv_lens[s], d.max_kv);
        tokens += new_lens[s];
        tiles += (int64_t(new_lens[s]) * (d.heads / d.kv_heads) + 15) / 16 * d.kv_heads;
    }
    if (tokens > kMostTokens || tiles > kMostTokens)
        return set_errorf(LORA_EINVAL, "a batch of %lld tokens (%lld tiles of 16 rows) is too large: "
                          "at most %d", (long long)tokens, (long long)tiles, kMostTokens);
    return LORA_OK;
}

// The keys that rows row0 .. row1 - 1 see between them, from a whole block on.
void tile_keys(const Batch &p, int32_t s, int64_t row0, int64_t row1, int32_t *lo, int32_t *hi) {
    const int32_t kv = p.kv_lens[s], pos0 = kv - p.new_lens[s];
    *lo = 0;
    *hi = kv;
    if (!p.d.causal) return;
    *hi = std::min(kv, pos0 + int32_t((row1 - 1) / p.group) + 1);
    if (p.d.window) {
        const int32_t first = pos0 + int32_t(row0 / p.group) - p.d.window + 1;
        *lo = std::max(first, 0) / lora::kAttnBlock * lora::kAttnBlock;
    }
}

int64_t blocks_of(int32_t lo, int32_t hi) {
    return hi > lo ? (int64_t(hi) - lo + lora::kAttnBlock - 1) / lora::kAttnBlock : 0;
}

// Whether a sequence of so many rows is a prompt's.
bool is_prompt(const Batch &p, int64_t rows) {
    return p.d.dtype == LORA_BF16 && rows > lora::attn_rows_most(p.d.dtype, p.d.head_dim);
}

// fn(sequence, its first token, its rows) for the sequences of one side.
template <typename Fn> void each_seq(const Batch &p, bool prompt, Fn fn) {
    int32_t tok0 = 0;
    for (size_t s = 0; s < p.new_lens.size(); ++s) {
        const int64_t rows = int64_t(p.new_lens[s]) * p.group;
        if (rows && is_prompt(p, rows) == prompt) fn(int32_t(s), tok0, rows);
        tok0 += p.new_lens[s];
    }
}

// Cuts every tile's keys into parts, so that the launch has about `target`
// units, and lays them out one after another.  A tile of up to `least` keys is
// not cut; the cut is even, so that its parts may be half as long, and there are
// no more of them than tiles + target in all.
void cut(const Batch &p, Side *side, bool prompt, int64_t target, int64_t least) {
    int64_t total = 0, longest = 0;
    each_seq(p, prompt, [&](int32_t s, int32_t, int64_t rows) {
        for (int64_t r = 0; r < rows; r += side->tile_rows) {
            int32_t lo, hi;
            tile_keys(p, s, r, std::min<int64_t>(rows, r + side->tile_rows), &lo, &hi);
            total += blocks_of(lo, hi) * p.d.kv_heads;
            longest = std::max(longest, blocks_of(lo, hi));
            side->tiles += p.d.kv_heads;
        }
    });
    const int64_t low = least / lora::kAttnBlock;
    const int64_t part = std::min(std::max(low, (total + target - 1) / target), std::max(longest, low));
    int32_t slot = 0;
    each_seq(p, prompt, [&](int32_t s, int32_t tok0, int64_t rows) {
        for (int64_t r = 0; r < rows; r += side->tile_rows) {
            int32_t lo, hi;
            tile_keys(p, s, r, std::min<int64_t>(rows, r + side->tile_rows), &lo, &hi);
            const int64_t blocks = blocks_of(lo, hi);
            const int64_t parts = std::max<int64_t>(1, (blocks + part - 1) / part);
            if (parts > 1)
                for (int32_t h = 0; h < p.d.kv_heads; ++h)
                    side->joins.push_back({tok0, h, int32_t(r), int32_t(rows),
                                           slot + int32_t(h * parts), int32_t(parts)});
            // (key heads beside one another: each on an XCD of its own, whose L2
            // then keeps its keys)
            for (int64_t i = 0; i < parts; ++i) {
                const int64_t k0 = lo + blocks * i / parts * lora::kAttnBlock;
                const int64_t k1 = lo + blocks * (i + 1) / parts * lora::kAttnBlock;
                for (int32_t h = 0; h < p.d.kv_heads; ++h)
                    side->units.push_back({s, h, int32_t(r), int32_t(rows), tok0,
                                           p.kv_lens[s] - p.new_lens[s], int32_t(k0),
                                           int32_t(std::min<int64_t>(k1, hi)),
                                           parts > 1 ? slot + int32_t(h * parts + i) : -1});
            }
            if (parts > 1) slot += int32_t(parts * p.d.kv_heads);
        }
    });
    // the longest parts first, for the short ones to fill the end (sorted by
    // counting: no part has more than `part` blocks)
    std::vector<int64_t> at(size_t(part) + 2, 0);
    const auto rank = [&](const AttnUnit &u) { return size_t(part - blocks_of(u.key0, u.key1)); };
    for (const AttnUnit &u : side->units) ++at[rank(u) + 1];
    for (size_t i = 1; i < at.size(); ++i) at[i] += at[i - 1];
    std::vector<AttnUnit> sorted(side->units.size());
    for (const AttnUnit &u : side->units) sorted[size_t(at[rank(u)]++)] = u;
    side->units.swap(sorted);
    side->cap_units = int64_t(side->units.size());
    side->cap_joins = int64_t(side->joins.size());
    side->cap_slots = slot;
    if (p.d.max_kv) {
        // Room for any lengths up to max_kv, so that the launches stay the same.
        // Parts are at least total / target blocks long, so that fewer than
        // `target` tiles are cut, into at most twice as many parts.
        const int64_t most = (int64_t(p.d.max_kv) + lora::kAttnBlock - 1) / lora::kAttnBlock;
        const int64_t each = std::max<int64_t>(1, (most + low - 1) / low);
        side->cap_units = std::min(side->tiles * each, side->tiles + target);
        side->cap_joins = each > 1 ? std::min(side->tiles, target) : 0;
        side->cap_slots = each > 1 ? std::min(side->tiles * each, 2 * target) : 0;
    }
}

// (in the memory that `p` has, whatever it held)
void plan_batch(Batch *p, const lora_attn_desc &d, const int32_t *new_lens, const int32_t *kv_lens,
                int32_t S) {
    p->d = d;
    p->group = d.heads / d.kv_heads;
    p->tokens.clear();
    p->most_kv = 0;
    p->rows.clear();
    p->prompt.clear();
    p->new_lens.assign(new_lens, new_lens + S);
    p->kv_lens.assign(kv_lens, kv_lens + S);
    for (int32_t s = 0; s < S; ++s) {
        p->most_kv = std::max(p->most_kv, kv_lens[s]);
        for (int32_t i = 0; i < new_lens[s]; ++i)
            p->tokens.push_back({s, kv_lens[s] - new_lens[s] + i});
    }
    int64_t few = 0;
    each_seq(*p, false, [&](int32_t, int32_t, int64_t rows) { few = std::max(few, rows); });
    // (float32 chunks: large tiles read keys less often, small ones use more of
    // the chip)
    p->rows.tile_rows = few <= 16 ? 16 : few <= 32 ? 32 : lora::attn_rows_most(p->d.dtype, p->d.head_dim);
    auto tiles = [&](int32_t rows_a_tile) {
        int64_t n = 0;
        each_seq(*p, false, [&](int32_t, int32_t, int64_t rows) { n += (rows + rows_a_tile - 1) / rows_a_tile; });
        return n * p->d.kv_heads;
    };
    while (p->rows.tile_rows > 16 && tiles(p->rows.tile_rows) < kCus) p->rows.tile_rows /= 2;
    p->rows.once = few <= p->rows.tile_rows;
    // A few tiles over short contexts: 8 waves a workgroup and all of a tile's
    // keys, without a launch to join parts.  8 waves against 4, replayed, heads of
    // 128, us:
    //   tiles   320 keys     512          701          1000
    //       8   7.8  10.1    10.0 10.6    12.4 10.8    16.3 11.0
    //     128  10.3  12.3    13.9 13.7    17.5 17.0    22.3 18.4
    //     160  10.9  12.8    14.2 16.6    18.4 17.6    22.8 22.6
    //     192  10.9  13.7    14.3 17.2    17.8 21.7    22.4 25.1
    //     256  11.3  15.5    15.2 19.4    19.2 23.5    24.6 30.4
    // So up to 512 keys, or 1024 where 4 waves' parts would be more than a round
    // of workgroups; 1 and 2 key heads balance alike, heads of 64 a little later
    // and float32 a little earlier (at most 9% from the better of the two).
    int64_t longest = p->d.max_kv;
    if (!longest)
        each_seq(*p, false, [&](int32_t s, int32_t, int64_t rows) {
            int32_t lo, hi;
            tile_keys(*p, s, 0, rows, &lo, &hi);
            longest = std::max<int64_t>(longest, hi - lo);
        });
    const int64_t few_tiles = tiles(16);
    p->rows.waves = p->rows.tile_rows == 16 && lora::attn_dim(p->d.head_dim) <= 128 &&
                            few_tiles <= kCus && longest <= (few_tiles > 160 ? kShortKeys : kShortKeys / 2)
                        ? lora::kManyWaves
                        : 4;
    cut(*p, &p->rows, false, kRowsUnits, p->rows.waves == 4 ? kRowsKeys : kShortKeys);
    p->prompt.tile_rows = lora::kPromptRows;
    cut(*p, &p->prompt, true, kPromptUnits, kPromptKeys);

    uint64_t at = 0;
    auto place = [&](uint64_t bytes) {
        const uint64_t off = at;
        at += round_up(bytes, 256);
        return off;
    };
    p->off_tokens = place(sizeof(AttnToken) * p->tokens.size());
    for (Side *side : {&p->rows, &p->prompt}) {
        side->off_units = place(sizeof(AttnUnit) * uint64_t(side->cap_units));
        side->off_joins = place(sizeof(AttnJoin) * uint64_t(side->cap_joins));
    }
    p->image_bytes = at;
    for (Side *side : {&p->rows, &p->prompt}) {
        const uint64_t rows = uint64_t(side->cap_slots) * uint64_t(side->tile_rows);
        side->off_partial = place(rows * 4 * uint64_t(lora::attn_dim(p->d.head_dim)));
        side->off_lse = place(rows * 4);
    }
    p->ws_bytes = at;
}

bool aligned(const void *ptr, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(ptr) % uint64_t(bytes) == 0;
}

struct Rows {
    const char *name;
    const void *ptr;
    int64_t ld, width;
};
// A matrix of whole 16-byte vectors.
lora_status check_rows(const Rows &r) {
    if (!r.ptr || !aligned(r.ptr, 16))
        return set_errorf(LORA_EINVAL, "%s must be non-null and 16-byte aligned", r.name);
    if (r.ld < r.width || r.ld % 8 || r.ld > kMostStride)
        return set_errorf(LORA_EINVAL, "ld of %s (%lld) is not a multiple of 8 from its width %lld "
                          "to 2^36", r.name, (long long)r.ld, (long long)r.width);
    return LORA_OK;
}
// The bytes that T rows span, T > 0.
struct Bytes {
    uintptr_t lo, hi;
};
Bytes bytes_of(const Rows &r, int64_t T, int32_t es) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(r.ptr);
    return {lo, lo + uint64_t((T - 1) * r.ld + r.width) * es};
}
// Keys or values of a cache.
struct CacheSide {
    const char *name;
    const void *ptr;
    int64_t page, head, tok;
};
CacheSide k_side(const lora_kv_cache &c) {
    return {"k_cache", c.k, c.k_page_stride, c.k_head_stride, c.k_token_stride};
}
CacheSide v_side(const lora_kv_cache &c) {
    return {"v_cache", c.v, c.v_page_stride, c.v_head_stride, c.v_token_stride};
}
Bytes bytes_of(const Batch &p, const lora_kv_cache &c, const CacheSide &t) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(t.ptr);
    return {lo, lo + uint64_t((c.num_pages - 1) * t.page + (p.d.kv_heads - 1) * t.head +
                              (p.d.page_size - 1) * t.tok + p.d.head_dim) * esize(p.d.dtype)};
}
// Whether two matrices of T rows reach into each other: column slices of the
// same rows do not.
bool overlap(const Rows &a, const Rows &b, int64_t T, int32_t es) {
    if (!a.ptr || !b.ptr || T <= 0) return false;
    const auto [alo, ahi] = bytes_of(a, T, es);
    const auto [blo, bhi] = bytes_of(b, T, es);
    if (ahi <= blo || bhi <= alo) return false;
    if (T > 1 && a.ld == b.ld) {
        const uint64_t l = uint64_t(a.ld) * es;
        const uint64_t at = blo >= alo ? (blo - alo) % l : (l - (alo - blo) % l) % l;
        if (at >= uint64_t(a.width) * es && at + uint64_t(b.width) * es <= l) return false;
    }
    return true;
}

// Whether two different places of one side of the cache have elements in common:
// |dp page + dh head + dt tok - shift| < head_dim for distances within its pages,
// heads and tokens, not all zero.  With `same`, all zero counts too: whether
// places of a side and of another, with the same strides and `shift` elements
// on, do.  Strides of which each reaches past all that the smaller ones span
// answer it at once; else every distance along the two shorter dimensions is
// looked at, and the third solved for.
bool meet(const Batch &p, const lora_kv_cache &c, const CacheSide &t, int64_t shift, bool same) {
    struct Dim {
        int64_t stride, count;
    };
    Dim d[4] = {{t.page, c.num_pages}, {t.head, p.d.kv_heads}, {t.tok, p.d.page_size},
                {std::abs(shift), same ? 2 : 1}};
    const int64_t D = p.d.head_dim;
    std::sort(d, d + 4, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    int64_t span = D;
    bool nested = true;
    for (const Dim &x : d)
        if (x.count > 1) {
            nested &= x.stride >= span;
            span += (x.count - 1) * x.stride;
        }
    if (nested) return false;
    Dim e[3] = {{t.page, c.num_pages}, {t.head, p.d.kv_heads}, {t.tok, p.d.page_size}};
    std::sort(e, e + 3, [](const Dim &a, const Dim &b) { return a.count < b.count; });
    const Dim &x = e[0], &y = e[1], &z = e[2];
    for (int64_t i = 1 - x.count; i < x.count; ++i)
        for (int64_t j = 1 - y.count; j < y.count; ++j) {
            // the distances k along z with |k z - rest| < D
            const int64_t rest = shift - i * x.stride - j * y.stride;
            if (z.stride == 0) {
                if (std::abs(rest) < D && (same || i || j || z.count > 1)) return true;
                continue;
            }
            int64_t k = (rest - D) / z.stride - 1;
            for (k = std::max(k, 1 - z.count); k < z.count && k * z.stride < rest + D; ++k)
                if (std::abs(k * z.stride - rest) < D && (same || i || j || k)) return true;
        }
    return false;
}

// Whether no place of the keys has an element in common with one of the values:
// they lie apart as wholes, or have the same strides and do not meet, or the
// same page stride and lie apart within it.
bool sides_apart(const Batch &p, const lora_kv_cache &c) {
    const CacheSide k = k_side(c), v = v_side(c);
    const Bytes kb = bytes_of(p, c, k), vb = bytes_of(p, c, v);
    if (kb.hi <= vb.lo || vb.hi <= kb.lo) return true;
    const int64_t es = esize(p.d.dtype);
    const int64_t bytes = vb.lo >= kb.lo ? int64_t(vb.lo - kb.lo) : -int64_t(kb.lo - vb.lo);
    if (bytes % es == 0 && (c.num_pages == 1 || k.page == v.page) &&
        (p.d.kv_heads == 1 || k.head == v.head) && k.tok == v.tok)
        return !meet(p, c, k, bytes / es, true);
    if (c.num_pages == 1 || k.page != v.page) return false;
    const auto in_page = [&](const CacheSide &t) {
        return ((p.d.kv_heads - 1) * t.head + (p.d.page_size - 1) * t.tok + p.d.head_dim) * es;
    };
    const int64_t page = k.page * es, at = (bytes % page + page) % page;
    return at >= in_page(k) && at + in_page(v) <= page;
}

// The cache and its page table; and whether the tensors beside them (T rows
// each) lie apart from it.  A cache that is written has a place for each key and
// each value.
lora_status check_cache(const Batch &p, const lora_kv_cache *c, const int32_t *pages,
                        int64_t ld_pages, int32_t pages_per_seq, bool written,
                        std::initializer_list<Rows> beside) {
    if (!c) return set_errorf(LORA_EINVAL, "null cache");
    const int32_t es = esize(p.d.dtype);
    if (c->num_pages < 1) return set_errorf(LORA_EINVAL, "a cache of %d pages", c->num_pages);
    for (const CacheSide &t : {k_side(*c), v_side(*c)}) {
        if (!t.ptr || !aligned(t.ptr, 16))
            return set_errorf(LORA_EINVAL, "%s must be non-null and 16-byte aligned", t.name);
        for (int64_t st : {t.page, t.head, t.tok})
            if (st < 0 || st % 8 || st > kMostStride)
                return set_errorf(LORA_EINVAL, "a stride of %s (%lld) is no multiple of 8 in 0..2^36",
                                  t.name, (long long)st);
        if (t.page > kMostCache / c->num_pages)
            return set_errorf(LORA_EINVAL, "%s: %d pages, %lld elements apart", t.name, c->num_pages,
                              (long long)t.page);
        if (t.tok < p.d.head_dim || t.tok * es * 16 >= (int64_t(1) << 31))
            return set_errorf(LORA_EINVAL, "%s: tokens %lld elements apart, heads of %d", t.name,
                              (long long)t.tok, p.d.head_dim);
        if (written && meet(p, *c, t, 0, false))
            return set_errorf(LORA_EINVAL, "places of %s coincide: pages %lld, heads %lld, tokens %lld "
                              "elements apart", t.name, (long long)t.page, (long long)t.head,
                              (long long)t.tok);
        const Bytes all = bytes_of(p, *c, t);
        for (const Rows &r : beside) {
            const Bytes rows = bytes_of(r, int64_t(p.tokens.size()), es);
            if (r.ptr && rows.lo < all.hi && all.lo < rows.hi)
                return set_errorf(LORA_EINVAL, "%s overlaps %s", r.name, t.name);
        }
    }
    if (!pages || !aligned(pages, 4))
        return set_errorf(LORA_EINVAL, "the page table must be non-null and 4-byte aligned");
    if (written && !sides_apart(p, *c))
        return set_errorf(LORA_EINVAL, "places of k_cache and v_cache coincide");
    if (ld_pages < pages_per_seq || ld_pages > kMostStride)
        return set_errorf(LORA_EINVAL, "ld of the page table (%lld) is not from its %d pages to 2^36",
                          (long long)ld_pages, pages_per_seq);
    // (a captured call may be replayed for up to max_kv)
    const int32_t keys = std::max(p.most_kv, p.d.max_kv);
    if (int64_t(pages_per_seq) * p.d.page_size < keys)
        return set_errorf(LORA_EINVAL, "%d pages of %d a sequence do not hold %d keys",
                          pages_per_seq, p.d.page_size, keys);
    return LORA_OK;
}

// The plan's workspace holds its tables, and the call's tensors and cache (null:
// none) lie apart from it.
lora_status check_uploaded(const attn_plan *p, const lora_kv_cache *c, std::initializer_list<Rows> beside) {
    if (!p->ws) return set_errorf(LORA_ESTATE, "plan has not been uploaded");
    if (!lora::owns_workspace(p, p->ws))
        return set_errorf(LORA_ESTATE, "the plan's workspace holds another plan's tables since "
                          "(upload this plan again)");
    const int32_t es = esize(p->d.dtype);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p->ws), hi = lo + attn_plan_workspace_bytes(p);
    const auto apart = [&](const char *name, const Bytes &b) {
        return b.lo >= hi || lo >= b.hi
                   ? LORA_OK
                   : set_errorf(LORA_EINVAL, "%s overlaps the plan's workspace", name);
    };
    lora_status st = LORA_OK;
    for (const Rows &r : beside)
        if (r.ptr && (st = apart(r.name, bytes_of(r, int64_t(p->tokens.size()), es))) != LORA_OK) return st;
    if (c && ((st = apart("k_cache", bytes_of(*p, *c, k_side(*c)))) != LORA_OK ||
              (st = apart("v_cache", bytes_of(*p, *c, v_side(*c)))) != LORA_OK))
        return st;
    return LORA_OK;
}

lora::CacheArgs cache_args(const Batch &p, const lora_kv_cache &c) {
    lora::CacheArgs a{};
    a.k = static_cast<uint8_t *>(c.k);
    a.v = static_cast<uint8_t *>(c.v);
    a.k_page = c.k_page_stride;
    a.k_head = c.k_head_stride;
    a.k_tok = c.k_token_stride;
    a.v_page = c.v_page_stride;
    a.v_head = c.v_head_stride;
    a.v_tok = c.v_token_stride;
    a.num_pages = c.num_pages;
    a.page_size = p.d.page_size;
    return a;
}

// What the debug build checks a call's table entries against.
hipError_t bounds_of(const Batch &p, int32_t pages_per_seq, lora::AttnBounds *b) {
    b->tokens = int32_t(p.tokens.size());
    b->seqs = int32_t(p.new_lens.size());
    b->kv_heads = p.d.kv_heads;
    b->group = p.group;
    b->keys = int64_t(pages_per_seq) * p.d.page_size;
    return lora::debug_word(&b->word);
}

// A C entry ends with a status whatever happens below it.
template <typename Fn> lora_status guarded(Fn fn) {
    try {
        return fn();
    } catch (const std::exception &e) {
        return set_errorf(LORA_ENOSPC, "host memory: %s", e.what());
    }
}

}  // namespace

extern "C" {

lora_status attn_plan_create(attn_plan **out, const lora_attn_desc *d, const int32_t *new_lens,
                             const int32_t *kv_lens, int32_t num_seqs) {
    if (!out) return set_errorf(LORA_EINVAL, "null output pointer");
    lora_status st = check_attn_desc(d);
    if (st != LORA_OK) return st;
    if ((st = check_lens(*d, new_lens, kv_lens, num_seqs)) != LORA_OK) return st;
    return guarded([&] {
        std::unique_ptr<attn_plan> p(new attn_plan());
        plan_batch(p.get(), *d, new_lens, kv_lens, num_seqs);
        *out = p.release();
        return LORA_OK;
    });
}

lora_status attn_plan_rebuild(attn_plan *p, const int32_t *new_lens, const int32_t *kv_lens,
                              int32_t num_seqs) {
    if (!p) return set_errorf(LORA_EINVAL, "null plan");
    const lora_status st = check_lens(p->d, new_lens, kv_lens, num_seqs);
    if (st != LORA_OK) return st;
    return guarded([&] {
        plan_batch(&p->spare, p->d, new_lens, kv_lens, num_seqs);
        std::swap(static_cast<Batch &>(*p), p->spare);
        p->ws = nullptr;                   // its tables are the last batch's
        return LORA_OK;
    });
}

lora_status attn_plan_destroy(attn_plan *p) {
    if (!p) return LORA_OK;
    lora::release_workspaces(p);
    for (int i = 0; i < 2; ++i) {
        // (a copy out of the buffer may still be queued)
        if (p->staged[i]) {
            (void)hipEventSynchronize(p->staged[i]);
            (void)hipEventDestroy(p->staged[i]);
        }
        if (p->staging[i]) (void)hipHostFree(p->staging[i]);
    }
    delete p;
    return LORA_OK;
}

uint64_t attn_plan_workspace_bytes(const attn_plan *p) {
    return p ? std::max<uint64_t>(p->ws_bytes, 256) : 0;
}

lora_status attn_plan_stats(const attn_plan *p, int32_t *num_tokens, int32_t *num_units,
                            int32_t *num_joins, int32_t *max_kv) {
    if (!p) return set_errorf(LORA_EINVAL, "null plan");
    if (num_tokens) *num_tokens = int32_t(p->tokens.size());
    if (num_units) *num_units = int32_t(p->rows.units.size() + p->prompt.units.size());
    if (num_joins) *num_joins = int32_t(p->rows.joins.size() + p->prompt.joins.size());
    if (max_kv) *max_kv = p->most_kv;
    return LORA_OK;
}

lora_status attn_plan_upload(attn_plan *p, void *ws, uint64_t ws_bytes, void *stream) {
    if (!p) return set_errorf(LORA_EINVAL, "null plan");
    if (!ws || !aligned(ws, 256))
        return set_errorf(LORA_EINVAL, "workspace must be a non-null, 256-byte aligned device pointer");
    if (ws_bytes < attn_plan_workspace_bytes(p))
        return set_errorf(LORA_ESTATE, "workspace of %llu bytes < %llu needed",
                          (unsigned long long)ws_bytes,
                          (unsigned long long)attn_plan_workspace_bytes(p));
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    hipError_t e = hipStreamIsCapturing(static_cast<hipStream_t>(stream), &capture);
    if (e != hipSuccess) return set_errorf(LORA_EHIP, "plan upload: %s", hipGetErrorString(e));
    if (capture != hipStreamCaptureStatusNone)
        return set_errorf(LORA_ESTATE, "an upload cannot be captured: later ones write its staging again");
    return guarded([&] {
        const int32_t k = p->next_staging;
        e = p->staged[k] ? hipEventSynchronize(p->staged[k])
                                    : hipEventCreateWithFlags(&p->staged[k], hipEventDisableTiming);
        if (e != hipSuccess)
            return set_errorf(LORA_EHIP, "plan staging event: %s", hipGetErrorString(e));
        const uint64_t bytes = std::max<uint64_t>(p->image_bytes, 256);
        if (p->staging_bytes[k] < bytes) {
            const uint64_t want = std::max(bytes, p->staging_bytes[k] * 3 / 2);
            void *buf = nullptr;
            e = hipHostMalloc(&buf, want, hipHostMallocDefault);
            if (e != hipSuccess)
                return set_errorf(LORA_EHIP, "plan staging buffer: %s", hipGetErrorString(e));
            if (p->staging[k]) (void)hipHostFree(p->staging[k]);
            p->staging[k] = buf;
            p->staging_bytes[k] = want;
        }
        uint8_t *img = static_cast<uint8_t *>(p->staging[k]);
        auto put = [&](uint64_t off, const auto &table) {
            if (!table.empty()) std::memcpy(img + off, table.data(), sizeof(table[0]) * table.size());
        };
        put(p->off_tokens, p->tokens);
        for (const Side *side : {&p->rows, &p->prompt}) {
            put(side->off_units, side->units);
            put(side->off_joins, side->joins);
            // places without work: no sequence, no parts
            AttnUnit *u = reinterpret_cast<AttnUnit *>(img + side->off_units);
            for (int64_t i = int64_t(side->units.size()); i < side->cap_units; ++i)
                u[i] = AttnUnit{-1, 0, 0, 0, 0, 0, 0, 0, -1};
            AttnJoin *j = reinterpret_cast<AttnJoin *>(img + side->off_joins);
            for (int64_t i = int64_t(side->joins.size()); i < side->cap_joins; ++i) j[i] = AttnJoin{};
        }
        hipStream_t s = static_cast<hipStream_t>(stream);
        e = hipMemcpyAsync(ws, img, p->image_bytes, hipMemcpyHostToDevice, s);
        if (e == hipSuccess) e = hipEventRecord(p->staged[k], s);
        if (e != hipSuccess) return set_errorf(LORA_EHIP, "plan upload: %s", hipGetErrorString(e));
        p->next_staging = 1 - k;
        p->ws = ws;
        lora::claim_workspace(p, ws, attn_plan_workspace_bytes(p));
        return LORA_OK;
    });
}

lora_status paged_attention(const attn_plan *p, const void *q, int64_t ldq,
                            const lora_kv_cache *cache, const int32_t *pages, int64_t ld_pages,
                            int32_t pages_per_seq, float scale, void *o, int64_t ldo,
                            void *stream) {
    if (!p) return set_errorf(LORA_EINVAL, "null plan");
    lora_status st;
    const float scale2 = scale * 1.44269504088896340736f;
    if (!std::isfinite(scale2))
        return set_errorf(LORA_EINVAL, "scale must be finite, and its product with log2 e too");
    const int64_t T = int64_t(p->tokens.size()), width = int64_t(p->d.heads) * p->d.head_dim;
    if (T == 0) return LORA_OK;            // empty batch: no tensor is looked at
    const int32_t es = esize(p->d.dtype);
    const Rows rq{"q", q, ldq, width}, ro{"o", o, ldo, width};
    for (const Rows *r : {&rq, &ro})
        if ((st = check_rows(*r)) != LORA_OK) return st;
    if (overlap(rq, ro, T, es)) return set_errorf(LORA_EINVAL, "o overlaps q");
    if ((st = check_cache(*p, cache, pages, ld_pages, pages_per_seq, false, {ro})) != LORA_OK)
        return st;
    if ((st = check_uploaded(p, cache, {rq, ro})) != LORA_OK) return st;

    uint8_t *ws = static_cast<uint8_t *>(p->ws);
    lora::AttnArgs a{};
    a.cache = cache_args(*p, *cache);
    a.q = static_cast<const uint8_t *>(q);
    a.o = static_cast<uint8_t *>(o);
    a.ldq = ldq;
    a.ldo = ldo;
    a.pages = pages;
    a.ld_pages = ld_pages;
    a.group = p->group;
    a.head_dim = p->d.head_dim;
    a.causal = p->d.causal;
    a.window = p->d.window;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = bounds_of(*p, pages_per_seq, &a.dbg);
    for (const Side *side : {&p->rows, &p->prompt}) {
        const bool prompt = side == &p->prompt;
        a.units = reinterpret_cast<const AttnUnit *>(ws + side->off_units);
        a.joins = reinterpret_cast<const AttnJoin *>(ws + side->off_joins);
        a.partial = reinterpret_cast<float *>(ws + side->off_partial);
        a.lse = reinterpret_cast<float *>(ws + side->off_lse);
        a.num_units = int32_t(side->cap_units);
        a.num_joins = int32_t(side->cap_joins);
        a.dbg.slots = side->cap_slots;
        a.scale2 = scale2;
        if (prompt) {
            a.negate = scale2 < 0;
            a.zero = scale2 == 0;
            a.scale2 = a.zero ? 1.0f : std::fabs(scale2);
        }
        if (e == hipSuccess)
            e = prompt ? lora::launch_attn_prompt(a, s)
                       : lora::launch_attn_rows(p->d.dtype, side->tile_rows, side->waves, side->once, a, s);
        if (e == hipSuccess) e = lora::launch_attn_join(p->d.dtype, side->tile_rows, a, s);
    }
    if (e != hipSuccess)
        return set_errorf(LORA_EHIP, "attention launch: %s", hipGetErrorString(e));
    return LORA_OK;
}

lora_status rotary_frequencies(double *out, int32_t rotary_dim, double base, int32_t scaling,
                               double factor, double original_length, double low, double high) {
    if (!out) return set_errorf(LORA_EINVAL, "null output pointer");
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > LORA_ATTN_MAX_HEAD_DIM)
        return set_errorf(LORA_EINVAL, "rotary_dim %d is not even in 2..%d", rotary_dim,
                          LORA_ATTN_MAX_HEAD_DIM);
    if (!(base > 0) || !std::isfinite(base))
        return set_errorf(LORA_EINVAL, "base must be positive and finite");
    if (scaling < LORA_ROTARY_UNSCALED || scaling > LORA_ROTARY_BY_PARTS)
        return set_errorf(LORA_EINVAL, "scaling %d is not a lora_rotary_scaling", scaling);
    if (scaling != LORA_ROTARY_UNSCALED && (!(factor > 0) || !std::isfinite(factor)))
        return set_errorf(LORA_EINVAL, "factor must be positive and finite");
    if (scaling == LORA_ROTARY_BY_PARTS &&
        (!(original_length > 0) || !std::isfinite(original_length) || !std::isfinite(low) ||
         !std::isfinite(high) || !(high > low)))
        return set_errorf(LORA_EINVAL, "by parts: original_length must be positive, low less than high");
    for (int32_t i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rotary_dim);
        double keep = scaling == LORA_ROTARY_UNSCALED ? 1.0 : 0.0;
        if (scaling == LORA_ROTARY_BY_PARTS) {
            const double turns = f * original_length / 6.283185307179586477;
            keep = std::min(std::max((turns - low) / (high - low), 0.0), 1.0);
        }
        out[i] = scaling == LORA_ROTARY_UNSCALED ? f : f * keep + f / factor * (1.0 - keep);
    }
    return LORA_OK;
}

lora_status rotary_append(const attn_plan *p, const lora_rotary_desc *r, const void *q, int64_t ldq,
                          void *q_out, int64_t ldqo, const void *k, int64_t ldk, const void *v,
                          int64_t ldv, const lora_kv_cache *cache, const int32_t *pages,
                          int64_t ld_pages, int32_t pages_per_seq, const int32_t *positions,
                          const double *freqs, void *stream) {
    if (!p) return set_errorf(LORA_EINVAL, "null plan");
    lora_status st;
    if (!r) return set_errorf(LORA_EINVAL, "null rotary descriptor");
    if (r->layout != LORA_ROTARY_HALF && r->layout != LORA_ROTARY_INTERLEAVED)
        return set_errorf(LORA_EINVAL, "layout %d is not a lora_rotary_layout", r->layout);
    if (freqs && (r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > p->d.head_dim))
        return set_errorf(LORA_EINVAL, "rotary_dim %d is not even in 2..%d", r->rotary_dim,
                          p->d.head_dim);
    if (!std::isfinite(r->magnitude)) return set_errorf(LORA_EINVAL, "magnitude must be finite");
    if (!freqs && (r->rotary_dim || positions))
        return set_errorf(LORA_EINVAL, "a rotary_dim or positions without frequencies");
    if (!p->d.causal && cache)
        for (size_t s = 0; s < p->kv_lens.size(); ++s)
            if (p->kv_lens[s] < p->new_lens[s])
                return set_errorf(LORA_EINVAL, "sequence %d: %d keys are fewer than its %d new tokens",
                                  int(s), p->kv_lens[s], p->new_lens[s]);
    if (!q && !cache) return set_errorf(LORA_EINVAL, "neither queries nor a cache");
    const int64_t T = int64_t(p->tokens.size());
    if (T == 0) return LORA_OK;            // empty batch: no tensor is looked at
    const int32_t es = esize(p->d.dtype), D = p->d.head_dim;
    const int64_t wq = int64_t(p->d.heads) * D, wk = int64_t(p->d.kv_heads) * D;
    const Rows rq{"q", q, ldq, wq}, ro{"q_out", q_out, ldqo, wq}, rk{"k", k, ldk, wk},
        rv{"v", v, ldv, wk};
    if (q) {
        for (const Rows *x : {&rq, &ro})
            if ((st = check_rows(*x)) != LORA_OK) return st;
        if (overlap(rq, ro, T, es) && !(q == q_out && (ldq == ldqo || T == 1)))
            return set_errorf(LORA_EINVAL, "q_out overlaps q without being it");
    } else if (q_out) {
        return set_errorf(LORA_EINVAL, "q_out without q");
    }
    if (cache) {
        for (const Rows *x : {&rk, &rv}) {
            if ((st = check_rows(*x)) != LORA_OK) return st;
            if (q && overlap(ro, *x, T, es)) return set_errorf(LORA_EINVAL, "q_out overlaps %s", x->name);
        }
        if ((st = check_cache(*p, cache, pages, ld_pages, pages_per_seq, true, {rq, ro, rk, rv})) !=
            LORA_OK)
            return st;
    } else if (k || v) {
        return set_errorf(LORA_EINVAL, "keys or values without a cache");
    }
    if (positions && !aligned(positions, 4))
        return set_errorf(LORA_EINVAL, "positions must be 4-byte aligned");
    if (freqs && !aligned(freqs, 8)) return set_errorf(LORA_EINVAL, "freqs must be 8-byte aligned");
    if ((st = check_uploaded(p, cache, {rq, ro, rk, rv})) != LORA_OK) return st;

    lora::RotaryArgs a{};
    if (cache) a.cache = cache_args(*p, *cache);
    a.q = static_cast<const uint8_t *>(q);
    a.k = static_cast<const uint8_t *>(k);
    a.v = static_cast<const uint8_t *>(v);
    a.q_out = static_cast<uint8_t *>(q_out);
    a.ldq = ldq;
    a.ldqo = ldqo;
    a.ldk = ldk;
    a.ldv = ldv;
    a.pages = pages;
    a.ld_pages = ld_pages;
    a.tokens = reinterpret_cast<const AttnToken *>(static_cast<uint8_t *>(p->ws) + p->off_tokens);
    a.positions = positions;
    a.freqs = freqs;
    a.T = int32_t(T);
    a.heads = p->d.heads;
    a.kv_heads = p->d.kv_heads;
    a.head_dim = D;
    a.rotary_dim = freqs ? r->rotary_dim : 0;
    a.layout = r->layout;
    a.magnitude = r->magnitude;
    hipError_t e = bounds_of(*p, pages_per_seq, &a.dbg);
    if (e == hipSuccess) e = lora::launch_rotary(p->d.dtype, a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_errorf(LORA_EHIP, "rotary launch: %s", hipGetErrorString(e));
    return LORA_OK;
}

}  // extern "C"
