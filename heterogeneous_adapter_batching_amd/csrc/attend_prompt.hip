// Attention of a batch's new tokens over the pages of their sequences, many
// rows at a time: prompts and their chunks, bfloat16.
//
// The mathematics and the orientation of the products are attend.hip's; here
// the matrix cores bound them, so keys and values go through LDS, 64 of each a
// stage by direct copies, and a wave keeps QT x 32 rows' queries and sums in
// registers.  One pass runs three steps of three tiles side by side, which do
// not depend on each other: the scores of tile i + 1, the weights of tile i,
// the products of tile i - 1 with its values.  So the vector units' work (an
// exponential for every 4 head_dim operations of the matrix cores) goes on
// under the matrix instructions of one and the same wave.
//
// Weights are 2^(c s - M) with an integer M per row at least as large as the
// largest c s when it was set.  They are formed with the M of before, while
// their own tile's maximum is still being formed beside them; only where that
// exceeds M by more than kSlack (seldom, after the first tile) M is raised and
// the tile's weights are formed again.  2^kSlack of headroom costs nothing: the
// sums are float32 and the weights bfloat16, whose exponents have room.
#include <type_traits>

#include <hip/hip_runtime.h>

#include "attend_device.h"
#include "lds_copy.h"

namespace lora {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_byte;
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kPromptWaves = 4;
constexpr int kPromptThreads = kPromptWaves * kWaveSize;
constexpr int kKeys = 64;                    // keys of a stage: 16 a wave
constexpr float kSlack = 8.f;

__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// fn over lanes l and l ^ 32
template <typename Fn> __device__ __forceinline__ float over_halves(float v, Fn fn) {
    const auto h =
        __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fn(__uint_as_float(h[0]), __uint_as_float(h[1]));
}
// fn(0), ..., fn(N - 1) with constant indexes
template <int N, typename Fn, int I = 0> __device__ __forceinline__ void each(Fn fn) {
    if constexpr (I < N) {
        fn(std::integral_constant<int, I>{});
        each<N, Fn, I + 1>(fn);
    }
}

// A row of a stage is DP elements in vectors of 16 bytes, exchanged by
// (exclusive or) swizzle(row): the 16 rows that a read of K touches at one
// vector, and the 8 rows at 4 vectors of a transposing read of V, then spread
// over all banks.
template <int DP> __device__ __forceinline__ constexpr int swizzle(int row) {
    return DP == 64 ? ((row >> 1 & 3) << 1) | (row >> 3 & 1) : ((row & 7) << 1) | (row >> 3 & 1);
}

template <int DP, int QT>
__global__ __launch_bounds__(kPromptThreads, DP == 256 || QT == 2 ? 1 : 2) void
k_attend_prompt(const AttnArgs a) {
    constexpr int RB = DP * 2;                        // bytes of a row in LDS
    constexpr int KK = DP / 16, DT = DP / 32;         // steps of a score, tiles of the output
    constexpr int STAGE = kKeys * RB;                 // of K or V
    constexpr int COPIES = 16 * RB / 1024;            // of a wave's 16 rows
    __shared__ __align__(1024) uint8_t lds[4 * STAGE];   // two of K, two of V

    const AttnUnit u = load_invariant(a.units + blockIdx.x);
    if (u.seq < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
    const int n = lane & 31, h = lane >> 5;
    const int D = a.head_dim;
    const int tiles = (u.key1 - u.key0 + kKeys - 1) / kKeys;

    // the rows' queries, and the last and first key that each sees
    const int wave_row = u.row0 + w * QT * 32;
    const uint32_t flip = a.negate ? 0x80008000u : 0u;
    u32x4 q[QT][KK];
    int last[QT], first[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int r = wave_row + t * 32 + n;
        const bool row = r < u.rows;
        const int tok = r / a.group, head = u.kv_head * a.group + r % a.group;
        const uint16_t *p = reinterpret_cast<const uint16_t *>(a.q) +
                            int64_t(u.tok0 + tok) * a.ldq + int64_t(head) * D;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int e = kk * 16 + h * 8;
            q[t][kk] = u32x4{0u, 0u, 0u, 0u};
            if (row && e < D) q[t][kk] = *reinterpret_cast<const u32x4 *>(p + e) ^ flip;
        }
        last[t] = !row ? -1 : a.causal ? min(u.pos0 + tok, u.key1 - 1) : u.key1 - 1;
        first[t] = row && a.window ? u.pos0 + tok - a.window + 1 : 0;
    }
    // keys that all of the wave's rows see: from all_from to all_to
    const int tail = min(wave_row + QT * 32, u.rows) - 1;
    int all_to = a.causal ? min(u.pos0 + wave_row / a.group, u.key1 - 1) : u.key1 - 1;
    const int all_from = a.window ? u.pos0 + tail / a.group - a.window + 1 : 0;

    // pages outside the cache, whose keys are absent: none, as a rule
    const int32_t *table = a.pages + int64_t(u.seq) * a.ld_pages;
    const int ps = a.cache.page_size;
    bool bad = false;
    for (int p = u.key0 / ps + tid; p < (u.key1 + ps - 1) / ps; p += kPromptThreads)
        bad |= table[p] < 0 || table[p] >= a.cache.num_pages;
    bad = __syncthreads_or(bad);
    if (bad) all_to = -1;                             // every key is looked up

    // a lane's vector in a copy, its vector of K's rows, its parts of V's
    uint32_t k_off[COPIES], v_off[COPIES];
    const uint32_t k_row = uint32_t(a.cache.k_tok) * 2u, v_row = uint32_t(a.cache.v_tok) * 2u;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int at = i * 1024 + lane * 16, row = at / RB, vec = at % RB / 16 ^ swizzle<DP>(row);
        k_off[i] = off_or_oob(vec * 8 < D, uint32_t(row) * k_row + uint32_t(vec) * 16u);
        v_off[i] = off_or_oob(vec * 8 < D, uint32_t(row) * v_row + uint32_t(vec) * 16u);
    }
    const uint32_t base = uint32_t(reinterpret_cast<uintptr_t>((lds_byte *)lds));
    uint32_t k_at[KK], v_at[2][DT];
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
        k_at[kk] = base + uint32_t(n * RB + ((2 * kk + h) ^ swizzle<DP>(n)) * 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
            const int j = lane & 15, row = 8 * i + 4 * h + j / 4;
            const int vec = 4 * dt + 2 * (lane >> 4 & 1) + (j & 3) / 2;
            v_at[i][dt] = base + uint32_t(2 * STAGE + row * RB + (vec ^ swizzle<DP>(row)) * 16 +
                                          (j & 1) * 8);
        }

    // the copies of tile i: the wave's 16 keys of K and of V
    int page = (u.key0 + 16 * w) / ps, slot = (u.key0 + 16 * w) % ps;   // of K's next tile
    int page_v = page, slot_v = slot;
    auto resource = [&](int i, int pg, int sl, bool values) {
        const int key = u.key0 + i * kKeys + 16 * w;
        const int id = key < u.key1 ? load_invariant(table + pg) : -1;
        const bool there = id >= 0 && id < a.cache.num_pages;
        const int rows = there ? min(16, u.key1 - key) : 0;
        const uint8_t *p = values
            ? a.cache.v + (int64_t(there ? id : 0) * a.cache.v_page +
                           int64_t(u.kv_head) * a.cache.v_head + int64_t(sl) * a.cache.v_tok) * 2
            : a.cache.k + (int64_t(there ? id : 0) * a.cache.k_page +
                           int64_t(u.kv_head) * a.cache.k_head + int64_t(sl) * a.cache.k_tok) * 2;
        const uint32_t row = values ? v_row : k_row;
        return raw_rsrc(p, rows ? uint32_t(rows - 1) * row + uint32_t(D * 2) : 0u);
    };
    auto step = [&](int &pg, int &sl) {
        sl += kKeys;
        while (sl >= ps) {
            sl -= ps;
            ++pg;
        }
    };
    auto copy_k = [&](int i) {
        const u32x4 r = resource(i, page, slot, false);
        const uint32_t at = base + uint32_t((i & 1) * STAGE + w * 16 * RB);
#pragma unroll
        for (int c = 0; c < COPIES; ++c) copy_to_lds(r, k_off[c], 0, at + uint32_t(c * 1024));
        step(page, slot);
    };
    auto copy_v = [&](int i) {
        const u32x4 r = resource(i, page_v, slot_v, true);
        const uint32_t at = base + uint32_t((2 + (i & 1)) * STAGE + w * 16 * RB);
#pragma unroll
        for (int c = 0; c < COPIES; ++c) copy_to_lds(r, v_off[c], 0, at + uint32_t(c * 1024));
        step(page_v, slot_v);
    };

    auto k_frag = [&](int stage, int kt, int kk) {
        return *(lds_u32x4 *)(uintptr_t)(k_at[kk] + uint32_t(stage * STAGE + kt * 32 * RB));
    };
    auto v_frag = [&](int stage, int s, int dt) {
        const uint32_t off = uint32_t(stage * STAGE + s * 16 * RB);
        const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                      (lds_s16x4 *)(uintptr_t)(v_at[0][dt] + off)));
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                      (lds_s16x4 *)(uintptr_t)(v_at[1][dt] + off)));
        return u32x4{x[0], x[1], y[0], y[1]};
    };

    const float c2 = a.scale2;
    f32x16 o[QT][DT];
    float m[QT], l[QT];

    // the key of a lane's score r of key tile kt of tile i
    auto key_of = [&](int i, int kt, int r) {
        return u.key0 + i * kKeys + kt * 32 + 8 * (r / 4) + 4 * h + r % 4;
    };
    auto partly = [&](int i) {
        const int k0 = u.key0 + i * kKeys;
        return k0 + kKeys - 1 > all_to || k0 < all_from;
    };
    auto mask = [&](int i, f32x16 (&s)[QT][2]) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int key = key_of(i, kt, r);
                bool there = true;
                if (bad && key < u.key1) {
                    const int id = table[key / ps];
                    there = id >= 0 && id < a.cache.num_pages;
                }
#pragma unroll
                for (int t = 0; t < QT; ++t)
                    s[t][kt][r] = there && key <= last[t] && key >= first[t] ? s[t][kt][r] : kNone;
            }
    };
    // weights e, e + 1 of the lane's 32 of a row: bf16 pairs in the order of
    // the second product's right operand
    auto weigh = [&](const f32x16 (&s)[2], int e, float base_m, float &sum) {
        const float x = exp2_of(fmaf(s[e / 16][e % 16], c2, -base_m));
        const float y = exp2_of(fmaf(s[e / 16][e % 16 + 1], c2, -base_m));
        sum += x + y;
        return bf16x2_rne(x, y);
    };
    auto top_of = [&](const f32x16 (&s)[2]) {
        float v = kNone;
#pragma unroll
        for (int r = 0; r < 16; ++r) v = fmaxf(v, fmaxf(s[0][r], s[1][r]));
        return over_halves(v, max_of) * c2;
    };
    // M raised to the tile's maximum, the sums brought to it
    auto raise = [&](int t, float top) {
        const float now = fmaxf(m[t], ceilf(top));
        const float f = exp2_of(m[t] - finite_max(now));
        m[t] = now;
        l[t] *= f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[t][dt] *= f;
    };

    auto attend = [&](auto careful_tag) {
        constexpr bool CAREFUL = decltype(careful_tag)::value;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            m[t] = kNone;
            l[t] = 0.f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) o[t][dt] = f32x16{};
        }
        page = page_v = (u.key0 + 16 * w) / ps;
        slot = slot_v = (u.key0 + 16 * w) % ps;
        if (tiles <= 0) return;
        for (int i = 0; i < tiles; ++i) {
            copy_k(i);
            copy_v(i);
            wait_copies<0>();
            __syncthreads();
            f32x16 s[QT][2];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    const u32x4 f = k_frag(i & 1, kt, kk);
#pragma unroll
                    for (int t = 0; t < QT; ++t)
                        s[t][kt] = mma32(f, q[t][kk], kk ? s[t][kt] : f32x16{});
                }
            const bool part = partly(i);
            if (part) mask(i, s);
            u32x4 p[QT][4];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                const float top = top_of(s[t]);
                if (__any(top > m[t] + kSlack)) raise(t, top);
                const float b = finite_max(m[t]);
#pragma unroll
                for (int e = 0; e < 32; e += 2) p[t][e / 8][e % 8 / 2] = weigh(s[t], e, b, l[t]);
            }
#pragma unroll
            for (int st = 0; st < 4; ++st)
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    u32x4 f = v_frag(i & 1, st, dt);
                    if (CAREFUL && part) {
#pragma unroll
                        for (int d = 0; d < 4; ++d) f[d] &= ~odd_mask<uint16_t>(f[d]);
                    }
#pragma unroll
                    for (int t = 0; t < QT; ++t) o[t][dt] = mma32(f, p[t][st], o[t][dt]);
                }
            if (CAREFUL && part) {
                // the values that are not finite, key by key, for the rows that see it
                for (int at = 0; at < kKeys; ++at) {
                    const int key = u.key0 + i * kKeys + at;
                    each<4>([&](auto st) {
                        if (at / 16 != st) return;
#pragma unroll
                        for (int dt = 0; dt < DT; ++dt) {
                            u32x4 f = v_frag(i & 1, st, dt);
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
                                const int e = 16 * st + 8 * (d / 2) + 4 * h + 2 * (d % 2);
                                f[d] &= odd_mask<uint16_t>(f[d]) &
                                        (e == at ? 0xffffu : e + 1 == at ? 0xffff0000u : 0u);
                            }
#pragma unroll
                            for (int t = 0; t < QT; ++t) {
                                const bool sees = key <= last[t] && key >= first[t];
                                const f32x16 more = mma32(f, p[t][st], f32x16{});
#pragma unroll
                                for (int r = 0; r < 16; ++r) o[t][dt][r] += sees ? more[r] : 0.f;
                            }
                        }
                    });
                }
            }
            __syncthreads();
        }
    };
    attend(std::integral_constant<bool, false>{});
    // Rows that do not see all keys of a tile have a weight of zero for the
    // others, which is not enough where a value is not finite: then again, with
    // such values left to the rows that see them.
    bool odd = false;
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int r = 0; r < 16; ++r) odd |= odd_mask<float>(__float_as_uint(o[t][dt][r])) != 0;
    if (__syncthreads_or(odd)) attend(std::integral_constant<bool, true>{});

    // outputs: a lane has 4 consecutive elements, 8 apart, of its rows
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float total = over_halves(l[t], sum_of);
        const float inv = total == 0.f ? 0.f : 1.0f / total;
        const int r = wave_row + t * 32 + n;
        if (r >= u.rows) continue;
        if (u.slot >= 0) {
            const int64_t at = int64_t(u.slot) * (kPromptWaves * QT * 32) + (r - u.row0);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<f32x4 *>(a.partial + at * DP + dt * 32 + 8 * i + 4 * h) =
                        f32x4{o[t][dt][4 * i] * inv, o[t][dt][4 * i + 1] * inv,
                              o[t][dt][4 * i + 2] * inv, o[t][dt][4 * i + 3] * inv};
            if (h == 0) a.lse[at] = total == 0.f ? kNone : m[t] + log2f(total);
        } else {
            uint16_t *out = reinterpret_cast<uint16_t *>(a.o) +
                            int64_t(u.tok0 + r / a.group) * a.ldo +
                            int64_t(u.kv_head * a.group + r % a.group) * D;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = dt * 32 + 8 * i + 4 * h;
                    if (d < D)
                        *reinterpret_cast<u32x2 *>(out + d) =
                            u32x2{bf16x2_rne(o[t][dt][4 * i] * inv, o[t][dt][4 * i + 1] * inv),
                                  bf16x2_rne(o[t][dt][4 * i + 2] * inv, o[t][dt][4 * i + 3] * inv)};
                }
        }
    }
}

template <int DP> hipError_t prompt_launch(const AttnArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((k_attend_prompt<DP, kPromptRows / (32 * kPromptWaves)>), dim3(a.num_units),
                       dim3(kPromptThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs &a, hipStream_t s) {
    if (a.num_units <= 0) return hipSuccess;
    switch (attn_dim(a.head_dim)) {
        case 64: return prompt_launch<64>(a, s);
        case 128: return prompt_launch<128>(a, s);
        default: return prompt_launch<256>(a, s);
    }
}

}  // namespace lora
