// Attention of a batch's new tokens over the pages of their sequences, many
// rows at a time: prompts and their chunks, bfloat16.
//
// The mathematics and the orientation of the products are attend.hip's; here
// the matrix cores bound them, so keys and values go through LDS, 64 of each a
// stage by direct copies, two stages of each, and a wave keeps 32 rows' queries
// and sums in registers.  The scores of tile i + 1 do not depend on tile i's
// weights, so they are formed beside one another: every matrix instruction has
// a few of the vector units' behind it (an exponential, the scaling, the sum
// and half a conversion for each 4 head_dim operations of the matrix cores),
// the reads of a later one's operand, and now and then a copy for the tile after
// next.  Four waves are a workgroup and two workgroups a CU.
//
// Weights are 2^(c s - M) with an integer M per row, raised (and the row's sums
// scaled by a power of two, exactly) only where a tile's largest c s exceeds it
// by more than kSlack: seldom, after the first tile.  Up to 2^kSlack, weights
// lose nothing: the sums are float32 and the weights bfloat16, whose exponents
// have room.  (Values past 2^119 can bring a sum to infinity so; then the rows go
// again, with weights of at most 1.)  The weights are rounded to bfloat16, as
// the matrix cores take them: 2^-8 of each weight, where their sum keeps float32.
// (attend.hip, where it costs nothing, adds the remainders.)
//
// What bounds it: the matrix cores, busy half of the cycles at the 1.85 GHz that
// the chip's power leaves them.  Four prompts of 4096 tokens, 32 heads over 8
// of 128: 546 to 568 us (968 to 1006 TFLOP/s of what is seen; 16384 tokens 1130;
// the large product of linear.hip 1320 to 1350).  An eighth of it is the copies
// (the same without them: 486 us), a tenth the weights; LDS has no conflicts.
// Tried and left: two tiles of 32 rows a wave, which halve the reads of LDS, at
// one wave a SIMD (heads of 64, where they fit the registers, 868 us against
// 673); 8 waves sharing a stage (the same for prompts, chunks 156 against 123);
// the sum of a pair of weights as a dot product, which goes the matrix cores'
// way (2% slower); more or fewer reads in flight (the same).
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

constexpr int kPromptWaves = kPromptRows / 32;
constexpr int kPromptThreads = kPromptWaves * kWaveSize;
constexpr int kKeys = 64;                    // keys of a stage
constexpr int kShare = kKeys / kPromptWaves; // of them a wave copies, all in one page
constexpr float kSlack = 8.f;

__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// (a maximum with NaN is NaN: three operands to an instruction, and the row's
// result is NaN either way)
__device__ __forceinline__ float largest(float a, float b) {
    return __builtin_elementwise_maximum(a, b);
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

// Has a vector unit's result formed here, between the matrix instructions,
// where the compiler would form it where it is used.
__device__ __forceinline__ void here(float &v) { asm volatile("" : "+v"(v)); }

// A row of a stage is DP elements in vectors of 16 bytes, exchanged by
// (exclusive or) a swizzle of the row, so that the 16 rows that a part of a
// read of K touches at one vector, and the 4 rows at 4 vectors that a part of a
// transposing read of V does, spread over all banks.
template <int DP> __device__ __forceinline__ constexpr int k_swizzle(int row) {
    return DP == 64 ? row >> 1 & 7 : (row & 3) << 2 | (row >> 2 & 3);
}
template <int DP> __device__ __forceinline__ constexpr int v_swizzle(int row) {
    return DP == 64 ? (row >> 1 & 1) << 2 : (row & 3) << 2;
}

template <int DP>
__global__ __launch_bounds__(kPromptThreads, DP == 256 ? 1 : 2) void
k_attend_prompt(const AttnArgs a) {
    constexpr int RB = DP * 2;                        // bytes of a row in LDS
    constexpr int KK = DP / 16, DT = DP / 32;         // steps of a score, tiles of the output
    constexpr int STAGE = kKeys * RB;                 // of K or V
    constexpr int COPIES = kShare * RB / 1024;        // of a wave's rows
    __shared__ __align__(1024) uint8_t lds[4 * STAGE];   // two of K, two of V

    const AttnUnit u = load_invariant(a.units + blockIdx.x);
    if (!held(a.dbg, u) || u.seq < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
    const int n = lane & 31, h = lane >> 5;
    const int D = a.head_dim;
    const int tiles = (u.key1 - u.key0 + kKeys - 1) / kKeys;

    // the lane's row: its query, and the last and first key that it sees
    const int wave_row = u.row0 + w * 32, r = wave_row + n;
    const bool row = r < u.rows;
    const int tok = r / a.group, head = u.kv_head * a.group + r % a.group;
    u32x4 q[KK];
    {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(a.q) +
                            int64_t(u.tok0 + tok) * a.ldq + int64_t(head) * D;
        const uint32_t flip = a.negate ? 0x80008000u : 0u;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int e = kk * 16 + h * 8;
            q[kk] = u32x4{0u, 0u, 0u, 0u};
            if (row && e < D) q[kk] = *reinterpret_cast<const u32x4 *>(p + e) ^ flip;
            if (a.zero)
#pragma unroll
                for (int d = 0; d < 4; ++d) q[kk][d] &= odd_mask<uint16_t>(q[kk][d]);
        }
    }
    const int last = !row ? -1 : a.causal ? min(u.pos0 + tok, u.key1 - 1) : u.key1 - 1;
    const int first = row && a.window ? u.pos0 + tok - a.window + 1 : 0;
    // keys that all of the wave's rows see: from all_from to all_to
    const int tail = min(wave_row + 32, u.rows) - 1;
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

    // a lane's vector in a copy (of 1024 bytes: whole rows), its vector of K's
    // rows, its parts of V's
    constexpr int PER = 1024 / RB, V_KINDS = PER < 4 ? 4 / PER : 1;
    uint32_t k_off[COPIES], v_off[V_KINDS];
    const uint32_t k_row = uint32_t(a.cache.k_tok) * 2u, v_row = uint32_t(a.cache.v_tok) * 2u;
    const int copy_row = lane * 16 / RB, copy_vec = lane * 16 % RB / 16;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int vec = copy_vec ^ k_swizzle<DP>(w * kShare + i * PER + copy_row);
        k_off[i] = off_or_oob(vec * 8 < D, uint32_t(copy_row) * k_row + uint32_t(vec) * 16u);
        asm volatile("" : "+v"(k_off[i]));   // (kept, not formed again for every tile)
    }
#pragma unroll
    for (int i = 0; i < V_KINDS; ++i) {
        const int vec = copy_vec ^ v_swizzle<DP>(w * kShare + i * PER + copy_row);
        v_off[i] = off_or_oob(vec * 8 < D, uint32_t(copy_row) * v_row + uint32_t(vec) * 16u);
        asm volatile("" : "+v"(v_off[i]));
    }
    const uint32_t base = uint32_t(reinterpret_cast<uintptr_t>((lds_byte *)lds));
    // (256 bytes of a row, which is what swizzles reach, in registers)
    constexpr int K_AT = KK < 8 ? KK : 8, V_AT = DT < 4 ? DT : 4;
    uint32_t k_at[K_AT], v_at[V_AT];
#pragma unroll
    for (int kk = 0; kk < K_AT; ++kk)
        k_at[kk] = base + uint32_t(n * RB + ((2 * kk + h) ^ k_swizzle<DP>(n)) * 16);
#pragma unroll
    for (int dt = 0; dt < V_AT; ++dt) {
        const int j = lane & 15, row = 4 * h + j / 4;
        const int vec = 4 * dt + 2 * (lane >> 4 & 1) + (j & 3) / 2;
        v_at[dt] = base + uint32_t(2 * STAGE + row * RB + (vec ^ v_swizzle<DP>(row)) * 16 +
                                   (j & 1) * 8);
    }

    // The copies of a tile: the wave's keys of K and of V.  Where they lie is
    // looked up for 64 tiles at a time, a tile a lane.
    const uint8_t *k_head = a.cache.k + int64_t(u.kv_head) * a.cache.k_head * 2;
    const uint8_t *v_head = a.cache.v + int64_t(u.kv_head) * a.cache.v_head * 2;
    uint64_t k_place = 0, v_place = 0;                // 0: no page
    auto look_up = [&](int i) {
        const int at = i + lane, key = u.key0 + at * kKeys + w * kShare;
        k_place = v_place = 0;
        if (key < u.key1) {
            const int id = table[key / ps], slot = key % ps;
            if (id >= 0 && id < a.cache.num_pages) {
                k_place = reinterpret_cast<uint64_t>(k_head) +
                          uint64_t(id * a.cache.k_page + slot * a.cache.k_tok) * 2;
                v_place = reinterpret_cast<uint64_t>(v_head) +
                          uint64_t(id * a.cache.v_page + slot * a.cache.v_tok) * 2;
            }
        }
    };
    const uint32_t k_bytes = uint32_t(kShare - 1) * k_row + uint32_t(D * 2);
    const uint32_t v_bytes = uint32_t(kShare - 1) * v_row + uint32_t(D * 2);
    // tile i's rows of the cache as a buffer; no bytes past the unit's keys
    auto rows_of = [&](int i, uint64_t place, uint32_t row, uint32_t bytes) {
        const uint32_t lo = __builtin_amdgcn_readlane(int(uint32_t(place)), i & 63);
        const uint32_t hi = __builtin_amdgcn_readlane(int(uint32_t(place >> 32)), i & 63);
        const int over = u.key0 + i * kKeys + (w + 1) * kShare - u.key1;
        if (over > 0) bytes -= uint32_t(over) * row;
        return u32x4{lo, hi & 0xffffu, (lo | hi) != 0 && over < kShare ? bytes : 0u,
                     uint32_t(kRsrcWord3)};
    };
    auto copy_k = [&](const u32x4 &r, int stage, int c) {
        copy_to_lds(r, k_off[c], uint32_t(c * PER) * k_row,
                    base + uint32_t(stage * STAGE + w * kShare * RB + c * 1024));
    };
    auto copy_v = [&](const u32x4 &r, int stage, int c) {
        copy_to_lds(r, v_off[c % V_KINDS], uint32_t(c * PER) * v_row,
                    base + uint32_t((2 + stage) * STAGE + w * kShare * RB + c * 1024));
    };
    auto copy_all = [&](auto &&copy, const u32x4 &r, int stage) {
#pragma unroll
        for (int c = 0; c < COPIES; ++c) copy(r, stage, c);
    };
    auto k_rows = [&](int i) { return rows_of(i, k_place, k_row, k_bytes); };
    auto v_rows = [&](int i) { return rows_of(i, v_place, v_row, v_bytes); };

    auto k_frag = [&](int stage, int kt, int kk) {
        return *(lds_u32x4 *)(uintptr_t)(k_at[kk % K_AT] +
                                         uint32_t(stage * STAGE + kt * 32 * RB + kk / K_AT * 256));
    };
    auto v_frag = [&](int stage, int s, int dt) {
        const uint32_t off = v_at[dt % V_AT] + uint32_t(stage * STAGE + s * 16 * RB + dt / V_AT * 256);
        const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                      (lds_s16x4 *)(uintptr_t)off));
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                      (lds_s16x4 *)(uintptr_t)(off + 8 * RB)));
        return u32x4{x[0], x[1], y[0], y[1]};
    };

    const float c2 = a.scale2;
    f32x16 o[DT];
    float m, l;

    // the key of a lane's score i of key tile kt of tile `at`
    auto key_of = [&](int at, int kt, int i) {
        return u.key0 + at * kKeys + kt * 32 + 8 * (i / 4) + 4 * h + i % 4;
    };
    auto partly = [&](int at) {
        const int k0 = u.key0 + at * kKeys;
        return k0 + kKeys - 1 > all_to || k0 < all_from;
    };
    auto mask = [&](int at, f32x16 (&s)[2]) {
        each<4>([&](auto sub) {          // 16 keys, which lie in one page
            const int k0 = u.key0 + at * kKeys + 16 * sub;
            bool there = true;
            if (bad && k0 < u.key1) {
                const int page = load_invariant(table + k0 / ps);
                there = page >= 0 && page < a.cache.num_pages;
            }
            const int to = there ? last : -1;
#pragma unroll
            for (int i = 8 * (sub % 2); i < 8 * (sub % 2) + 8; ++i) {
                const int k = key_of(at, sub / 2, i);
                s[sub / 2][i] = k <= to && k >= first ? s[sub / 2][i] : kNone;
            }
        });
    };
    // weights 2 i, 2 i + 1 of the lane's 32, bf16 in the order of the second
    // product's right operand (the dot product that would sum the pair shares
    // the matrix cores' way: two additions cost less beside them)
    auto weigh = [&](const f32x16 (&s)[2], int i, float low, float times = 1.f) {
        const float x = exp2_of(fmaf(s[i / 8][i % 8 * 2], c2, -low)) * times;
        const float y = exp2_of(fmaf(s[i / 8][i % 8 * 2 + 1], c2, -low)) * times;
        l += x + y;
        return bf16x2_rne(x, y);
    };
    // the largest of a quarter of the lane's scores
    auto top_of = [&](const f32x16 (&s)[2], int i) {
        const f32x16 &x = s[i / 2];
        const int j = i % 2 * 8;
        float v = largest(x[j], largest(x[j + 1], x[j + 2]));
        v = largest(v, largest(x[j + 3], x[j + 4]));
        return largest(largest(v, x[j + 5]), largest(x[j + 6], x[j + 7]));
    };
    // M raised to a tile's maximum, the sums brought to it: the rows that exceed
    // it by the slack alone, so that a row's bits do not follow keys that only
    // other rows of the wave see
    auto raise = [&](float top) {
        const float now = top > m + kSlack ? ceilf(top) : m;
        const float f = exp2_of(m - finite_max(now));
        m = now;
        l *= f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] *= f;
    };

    // reads of K and V in flight (heads of 256: one more spills registers into
    // the loop, four prompts of 4096 1260 us against 1044)
    constexpr int AHEAD = DP == 256 ? 3 : 4, EARLY = DP == 256 ? 2 : 3;
    // Scores of a tile, 12 of the 16 pairs of the last one's weights beside them.
    auto scores = [&](auto stage, f32x16 (&s)[2], auto &&beside) {
        u32x4 f[AHEAD];
        each<AHEAD>([&](auto at) { f[at] = k_frag(stage, at % 2, at / 2); });
        each<2 * KK>([&](auto at) {
            constexpr int kt = at % 2, kk = at / 2, next = at + AHEAD;
            const u32x4 k = f[at % AHEAD];
            if constexpr (next < 2 * KK) f[at % AHEAD] = k_frag(stage, next % 2, next / 2);
            s[kt] = mma32(k, q[kk], kk ? s[kt] : f32x16{});
            beside(at);
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    auto begin = [&] {
        m = kNone;
        l = 0.f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] = f32x16{};
        look_up(0);
    };
    constexpr std::integral_constant<int, 0> zero{};
    constexpr std::integral_constant<int, 1> one{};

    // Tile i: its weights and their products with its values, beside the scores
    // of tile i + 1 (but for the last).
    float top = kNone;
    auto tile = [&](int i, auto stage, auto has_next, f32x16 (&s)[2], f32x16 (&next)[2]) {
        constexpr std::integral_constant<int, 1 - stage> other;
        wait_copies<0>();
        __syncthreads();                 // the copies are there, and tile i - 1 is done with
        // tile i + 2's keys go where tile i's were, tile i + 1's values where tile
        // i - 1's were: one copy at a time, between the scores
        u32x4 kr, vr;
        if constexpr (has_next) {
            vr = v_rows(i + 1);
            if ((i + 2) % 64 == 0) look_up(i + 2);
            kr = k_rows(i + 2);
        }
        top = over_halves(top, max_of) * c2;
        if (__any(top > m + kSlack)) raise(top);
        const float low = finite_max(m);
        u32x4 p[4];
        auto weights = [&](auto j) {
            p[j / 4][j % 4] = weigh(s, j, low);
            here(l);
        };
        if constexpr (has_next) {
            scores(other, next, [&](auto at) {
                each<12>([&](auto j) {
                    if constexpr (j * 2 * KK / 12 == at) weights(j);
                });
                constexpr int gap = KK / COPIES;
                if constexpr (at % gap == gap - 1) {
                    constexpr int c = at / gap;
                    if constexpr (c < COPIES) copy_v(vr, other, c);
                    else copy_k(kr, stage, c - COPIES);
                }
            });
            if (partly(i + 1)) mask(i + 1, next);
        } else {
            each<12>(weights);
        }
        constexpr int STEPS = 4 * DT;
        u32x4 f[EARLY];
        float tops[4] = {kNone, kNone, kNone, kNone};
        each<EARLY>([&](auto at) { f[at] = v_frag(stage, at / DT, at % DT); });
        each<STEPS>([&](auto at) {
            constexpr int st = at / DT, dt = at % DT, ahead = at + EARLY;
            const u32x4 v = f[at % EARLY];
            if constexpr (ahead < STEPS) f[at % EARLY] = v_frag(stage, ahead / DT, ahead % DT);
            o[dt] = mma32(v, p[st], o[dt]);
            if constexpr (at < 4) weights(std::integral_constant<int, 12 + at>{});
            if constexpr (has_next && at % DT == DT - 1) {
                tops[st] = top_of(next, st);
                here(tops[st]);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        top = largest(largest(tops[0], tops[1]), largest(tops[2], tops[3]));
    };

    begin();
    if (tiles > 0) {
        f32x16 sa[2], sb[2];
        copy_all(copy_k, k_rows(0), 0);
        copy_all(copy_v, v_rows(0), 0);
        copy_all(copy_k, k_rows(1), 1);
        wait_copies<0>();
        __syncthreads();
        scores(zero, sa, [](auto) {});
        if (partly(0)) mask(0, sa);
        top = largest(largest(top_of(sa, 0), top_of(sa, 1)), largest(top_of(sa, 2), top_of(sa, 3)));
        int i = 0;
        for (; i + 2 < tiles; i += 2) {
            tile(i, zero, std::true_type{}, sa, sb);
            tile(i + 1, one, std::true_type{}, sb, sa);
        }
        if (i + 1 < tiles) {
            tile(i, zero, std::true_type{}, sa, sb);
            tile(i + 1, one, std::false_type{}, sb, sa);
        } else {
            tile(i, zero, std::false_type{}, sa, sb);
        }
    }

    // Rows that do not see all keys of a tile have a weight of zero for the
    // others, which is not enough where a value is not finite: then all of it
    // again, step by step, with such values left to the rows that see them and
    // all weights 2^-kSlack of what they were, so that they are at most 1: the
    // same bits in the end, and finite sums where only the slack was too much.
    const float down = exp2_of(-kSlack);
    float scaled = 1.f;
    float odd = 0.f;                     // (NaN where a sum is not finite)
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) odd = fmaf(o[dt][i], 0.f, odd);
    if (__syncthreads_or(odd != 0.f)) {
        begin();
        scaled = down;
        for (int i = 0; i < tiles; ++i) {
            if (i && i % 64 == 0) look_up(i);
            copy_all(copy_k, k_rows(i), 0);
            copy_all(copy_v, v_rows(i), 0);
            wait_copies<0>();
            __syncthreads();
            f32x16 s[2];
            scores(zero, s, [](auto) {});
            const bool part = partly(i);
            if (part) mask(i, s);
            top = largest(largest(top_of(s, 0), top_of(s, 1)), largest(top_of(s, 2), top_of(s, 3)));
            top = over_halves(top, max_of) * c2;
            if (__any(top > m + kSlack)) raise(top);
            const float low = finite_max(m);
            u32x4 p[4];
            each<16>([&](auto j) { p[j / 4][j % 4] = weigh(s, j, low, down); });
            each<4 * DT>([&](auto at) {
                u32x4 v = v_frag(0, at / DT, at % DT);
                if (part) {
#pragma unroll
                    for (int d = 0; d < 4; ++d) v[d] &= ~odd_mask<uint16_t>(v[d]);
                }
                o[at % DT] = mma32(v, p[at / DT], o[at % DT]);
            });
            // the values that are not finite, key by key, for the rows that see it
            for (int at = part ? 0 : kKeys; at < kKeys; ++at) {
                const int k = u.key0 + i * kKeys + at;
                const bool sees = k <= last && k >= first;
                each<4>([&](auto st) {
                    if (at / 16 != st) return;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) {
                        u32x4 v = v_frag(0, st, dt);
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const int e = 16 * st + 8 * (d / 2) + 4 * h + 2 * (d % 2);
                            v[d] &= odd_mask<uint16_t>(v[d]) &
                                    (e == at ? 0xffffu : e + 1 == at ? 0xffff0000u : 0u);
                        }
                        const f32x16 x = mma32(v, p[st], f32x16{});
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[dt][j] += sees ? x[j] : 0.f;
                    }
                });
            }
            __syncthreads();
        }
    }

    // outputs: a lane has 4 consecutive elements, 8 apart, of its row
    const float total = over_halves(l, sum_of);
    if (!row) return;
    const bool lost = total == 0.f && sees_a_key(a, u, r);
    const float inv = inverse_of(total, lost, u.slot >= 0);
    if (u.slot >= 0) {
        const int64_t at = int64_t(u.slot) * kPromptRows + (r - u.row0);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<f32x4 *>(a.partial + at * DP + dt * 32 + 2 * i + 4 * h) =
                    f32x4{o[dt][i] * inv, o[dt][i + 1] * inv, o[dt][i + 2] * inv, o[dt][i + 3] * inv};
        if (h == 0) a.lse[at] = log_weight(m, total / scaled, lost);
    } else {
        uint16_t *out = reinterpret_cast<uint16_t *>(a.o) + int64_t(u.tok0 + tok) * a.ldo +
                        int64_t(head) * D;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const int d = dt * 32 + 2 * i + 4 * h;
                if (d < D)
                    *reinterpret_cast<u32x2 *>(out + d) =
                        u32x2{bf16x2_rne(o[dt][i] * inv, o[dt][i + 1] * inv),
                              bf16x2_rne(o[dt][i + 2] * inv, o[dt][i + 3] * inv)};
            }
    }
}

template <int DP> hipError_t prompt_launch(const AttnArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((k_attend_prompt<DP>), dim3(a.num_units), dim3(kPromptThreads), 0, s, a);
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
