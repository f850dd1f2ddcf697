// Device building blocks of the attention kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "attend_internal.h"
#include "device_ops.h"

namespace lora {
namespace {

constexpr float kNone = -__builtin_inff();   // the score of a key that a row does not see

// Whether a table entry may be followed (debug build; one that may not is noted).
#ifdef LORA_SGMV_DEBUG
constexpr bool kDebug = true;
#else
constexpr bool kDebug = false;
#endif
template <typename Entry>
__device__ __forceinline__ bool held([[maybe_unused]] const AttnBounds &b, [[maybe_unused]] const Entry &e) {
    if constexpr (kDebug) {
        const uint32_t bits = wrong(b, e);
        if (bits) atomicOr(b.word, bits);
        return bits == 0;
    }
    return true;
}

// fn over both halves of the wave's rows of 16 lanes: lanes l, l ^ 16, l ^ 32
// and l ^ 48 end with the same value.
template <typename Fn> __device__ __forceinline__ float over_groups(float v, Fn fn) {
    auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fn(__uint_as_float(h[0]), __uint_as_float(h[1]));
    h = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fn(__uint_as_float(h[0]), __uint_as_float(h[1]));
}
__device__ __forceinline__ float max_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float sum_of(float a, float b) { return a + b; }

__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// A maximum to subtract: a row that has seen no key yet subtracts nothing from
// its scores, which are -inf.
__device__ __forceinline__ float finite_max(float m) { return m == kNone ? 0.f : m; }

// Whether row r of a unit sees a key at all.  Weights that sum to zero are those
// of a row that sees none, whose result is zeros, or of one whose scores are all
// -inf, whose weights exp(-inf + inf) are no numbers: this is asked of them alone.
__device__ __forceinline__ bool sees_a_key(const AttnArgs &a, const AttnUnit &u, int r) {
    const int pos = u.pos0 + r / a.group;
    const int first = a.window ? max(u.key0, pos - a.window + 1) : u.key0;
    const int last = a.causal ? min(pos, u.key1 - 1) : u.key1 - 1;
    const int32_t *table = a.pages + int64_t(u.seq) * a.ld_pages;
    if (first <= last)
        for (int p = first / a.cache.page_size; p <= last / a.cache.page_size; ++p)
            if (table[p] >= 0 && table[p] < a.cache.num_pages) return true;
    return false;
}

// The logarithm of what a part of a row's keys weighs, by which parts are
// joined: kNone for a part without keys, kLost for one whose scores are all
// -inf, which any other key's exceeds.
constexpr float kLost = -0x1.fffffep127f, kLeast = -0x1.fffffcp127f;
__device__ __forceinline__ float log_weight(float top, float total, bool lost) {
    if (total == 0.f) return lost ? kLost : kNone;
    const float w = top + log2f(total);
    return w == kLost ? kLeast : w;
}
// What a row's sums are multiplied by; split: the row has other parts.
__device__ __forceinline__ float inverse_of(float total, bool lost, bool split) {
    return total != 0.f ? 1.0f / total : lost && !split ? __builtin_nanf("") : 0.f;
}

// The parts of a word, two bf16 or a float32, that are not finite.
template <typename T> __device__ __forceinline__ uint32_t odd_mask(uint32_t w);
template <> __device__ __forceinline__ uint32_t odd_mask<uint16_t>(uint32_t w) {
    return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
           ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}
template <> __device__ __forceinline__ uint32_t odd_mask<float>(uint32_t w) {
    return (w & 0x7f800000u) == 0x7f800000u ? ~0u : 0u;
}

// A sequence's row of the page table, walked in tiles of 16 keys, each in one
// page: the tile's rows of the cache as a buffer (of no bytes for a page
// outside the cache, whose keys count as absent).
struct PageWalk {
    const int32_t *row;
    int32_t page, slot, page_size;           // of the next tile
    __device__ __forceinline__ PageWalk(const AttnArgs &a, int seq, int key)
        : row(a.pages + int64_t(seq) * a.ld_pages), page(key / a.cache.page_size),
          slot(key % a.cache.page_size), page_size(a.cache.page_size) {}
    __device__ __forceinline__ void skip(int keys) {
        slot += keys;
        while (slot >= page_size) {
            slot -= page_size;
            ++page;
        }
    }
};

// N consecutive outputs (N 4, 8 or 16) of one row.
template <int N> __device__ __forceinline__ void store_row(uint16_t *p, const float (&v)[N]) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = bf16x2_rne(v[2 * i], v[2 * i + 1]);
    if constexpr (N == 4) {
        *reinterpret_cast<u32x2 *>(p) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            reinterpret_cast<u32x4 *>(p)[i] =
                u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    }
}
template <int N> __device__ __forceinline__ void store_row(float *p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        reinterpret_cast<f32x4 *>(p)[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
}

}  // namespace
}  // namespace lora
