// Attention of a batch's new tokens over the pages of their sequences, few
// rows at a time: single tokens, short chunks and every float32 batch.
//
//     o_r = sum_j exp(s q_r.k_j - M_r) v_j / sum_j exp(s q_r.k_j - M_r)
//
// in one pass over the keys with the running maximum M and sum of every row.
// The rows of a tile are the query heads of one key head for the new tokens of
// a sequence, so keys and values are read once for all of them.  They are few:
// the bytes of keys and values bound the kernel, and they go from HBM to
// registers.  Both products have the cache's side as the left operand of the
// matrix cores, S^T = K Q^T and O^T = V^T P^T: a lane ends the first with 4
// keys' scores of one row, which are its part of the second's right operand as
// they stand (the keys of a step are dealt to the lane groups in that order),
// and O's columns are rows again, so that a row's maximum, sum and scale are
// the lane's own.  V^T takes a lane's 8 keys of one element: it loads 8
// elements of each and exchanges halves of words among its own registers.
// bfloat16 weights enter as two values, the rounded one and the remainder
// (at most 2^-16 of the weight is lost), which costs nothing here.  128 sequences of 19
// to 7824 keys, one token each, 32 heads over 8 of 128: 730 MB in 119 to 122 us
// with the join (6.0 TB/s); four of 68157 to 127138 1.7 GB in 260 (6.5); 64 over
// 1500 states of an encoder, 16 heads of 64, 393 MB in 65 (6.0; a copy of 1 GiB
// reads and writes at 5.16).
#include <hip/hip_runtime.h>

#include "attend_device.h"

namespace lora {
namespace {

// NQ tiles of 16 rows, NW waves that take the unit's keys in turn.  ONCE: every
// tile has all of its sequence's rows, so that its keys are read once, past the
// L2 (128 sequences of 19 to 7824 keys, 730 MB: 123 us against 139; four of 68157
// to 127138, 1.7 GB: 260 against 298, 6.6 TB/s).  Float32 sequences of several
// tiles keep them there (300 tokens behind 8000 keys 672 against 706; 64 tokens
// of 32 heads over one key head, 4000 keys, 92 against 106).
template <typename T, int DP, int NQ, int NW, bool ONCE>
__global__ __launch_bounds__(NW * kWaveSize, sizeof(T) == 2 && DP <= 128 ? 2 : 1) void k_attend_rows(const AttnArgs a) {
    static_assert(NW == 4 || NQ == 1, "the join of 16 rows takes 256 threads");
    constexpr int E = Elem<T>::E;                     // elements of 16 bytes
    constexpr int KS = DP / (4 * E);                  // matrix steps of a score
    constexpr int KT = E / 4;                         // 16-key tiles of a matrix step over keys
    constexpr int BK = 16 * KT;                       // keys a wave takes at a time
    constexpr int VW = DP / 16 < E ? DP / 16 : E;     // elements of a lane's vector of V
    constexpr int VC = DP / (16 * VW);                // and its vectors of a key
    constexpr int VD = VW * int(sizeof(T)) / 4;       // words of such a vector
    constexpr int LD = DP + 4;
    constexpr int POLICY = ONCE ? kNT : 0;
    __shared__ float so[NW][16][LD];
    __shared__ float sm[NW][16], sl[NW][16];

    const AttnUnit u = load_invariant(a.units + blockIdx.x);
    if (!held(a.dbg, u) || u.seq < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
    const int n = lane & 15, g = lane >> 4;
    const int D = a.head_dim;
    constexpr int es = sizeof(T);

    // the rows' queries, and the last and first key that each sees
    u32x4 q[NQ][KS];
    int last[NQ], first[NQ];
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
        const int r = u.row0 + t * 16 + n;
        const bool row = r < u.rows;
        const int tok = r / a.group, head = u.kv_head * a.group + r % a.group;
        const T *p = reinterpret_cast<const T *>(a.q) + int64_t(u.tok0 + tok) * a.ldq +
                     int64_t(head) * D;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            const int e = (kk * 4 + g) * E;
            q[t][kk] = u32x4{0u, 0u, 0u, 0u};
            if (row && e < D) q[t][kk] = *reinterpret_cast<const u32x4 *>(p + e);
        }
        last[t] = !row ? -1 : a.causal ? min(u.pos0 + tok, u.key1 - 1) : u.key1 - 1;
        first[t] = row && a.window ? u.pos0 + tok - a.window + 1 : 0;
    }
    // keys that every row sees: from `all_from` to `all_to`
    const int tail = min(u.row0 + NQ * 16, u.rows) - 1;
    const int all_to = a.causal ? u.pos0 + u.row0 / a.group : u.key1 - 1;
    const int all_from = a.window ? u.pos0 + tail / a.group - a.window + 1 : 0;

    f32x4 o[NQ][VC][VW];
    float m[NQ], l[NQ];
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
        m[t] = kNone;
        l[t] = 0.f;
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int j = 0; j < VW; ++j) o[t][c][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // A wave takes every NW-th run of BK keys.
    struct Keys {
        u32x4 k[KT][KS];
        uint32_t v[4 * KT][VC][VD];
        bool there[KT];
    };
    PageWalk walk(a, u.seq, u.key0 + w * BK);
    const uint32_t k_row = uint32_t(a.cache.k_tok) * es, v_row = uint32_t(a.cache.v_tok) * es;
    uint32_t k_off[KS], v_off[VC];
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
        k_off[kk] = off_or_oob((kk * 4 + g) * E < D, uint32_t(n) * k_row + uint32_t(kk * 4 + g) * 16u);
#pragma unroll
    for (int c = 0; c < VC; ++c)
        v_off[c] = off_or_oob((c * 16 + n) * VW < D,
                              uint32_t(4 * g) * v_row + uint32_t((c * 16 + n) * VW * es));
    auto load16 = [](rsrc_t r, uint32_t off, uint32_t at) {
        return __builtin_amdgcn_raw_buffer_load_b128(r, int(off), int(at), POLICY);
    };
    auto load = [&](int b, Keys &x) {
#pragma unroll
        for (int tt = 0; tt < KT; ++tt) {
            const int key = b + 16 * tt;
            const int page = key < u.key1 ? load_invariant(walk.row + walk.page) : -1;
            x.there[tt] = page >= 0 && page < a.cache.num_pages;
            const int64_t at = x.there[tt] ? page : 0;
            const uint8_t *kp = a.cache.k + (at * a.cache.k_page + int64_t(u.kv_head) * a.cache.k_head +
                                             int64_t(walk.slot) * a.cache.k_tok) * es;
            const uint8_t *vp = a.cache.v + (at * a.cache.v_page + int64_t(u.kv_head) * a.cache.v_head +
                                             int64_t(walk.slot) * a.cache.v_tok) * es;
            // the tile's rows that are keys of the unit
            const int rows = x.there[tt] ? min(16, u.key1 - key) : 0;
            const rsrc_t kr = make_rsrc(kp, rows ? uint32_t(rows - 1) * k_row + uint32_t(D * es) : 0u);
            const rsrc_t vr = make_rsrc(vp, rows ? uint32_t(rows - 1) * v_row + uint32_t(D * es) : 0u);
            // (rows past the last are past the buffer's end)
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) x.k[tt][kk] = load16(kr, k_off[kk], 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VC; ++c) {
                    const uint32_t off = v_off[c], at_row = uint32_t(i) * v_row;
                    if constexpr (VD == 4) {
                        const u32x4 y = load16(vr, off, at_row);
#pragma unroll
                        for (int d = 0; d < 4; ++d) x.v[tt * 4 + i][c][d] = y[d];
                    } else {
                        const u32x2 y = __builtin_amdgcn_raw_buffer_load_b64(vr, int(off), int(at_row), POLICY);
                        x.v[tt * 4 + i][c][0] = y[0];
                        x.v[tt * 4 + i][c][1] = y[1];
                    }
                }
            walk.skip(16);
        }
        walk.skip((NW - 1) * BK);
    };
    auto attend = [&](int b, const Keys &x) {
        const auto &k = x.k;
        const auto &v = x.v;
        const auto &there = x.there;
        // V^T: element j of vector c of the lane's keys
        auto vt = [&](int c, int j) {
            u32x4 r;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if constexpr (E == 8)
                    r[d] = __builtin_amdgcn_perm(v[2 * d + 1][c][j / 2], v[2 * d][c][j / 2],
                                                 j % 2 ? 0x07060302u : 0x05040100u);
                else
                    r[d] = v[d][c][j];
            }
            return r;
        };
        // Rows that do not see all of these keys have a weight of zero for the
        // others, which is not enough where a value is not finite.
        bool careful = false;
        if (min(b + BK, u.key1) - 1 > all_to || b < all_from) {
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 4 * KT; ++i)
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int d = 0; d < VD; ++d) odd |= odd_mask<T>(v[i][c][d]) != 0;
            careful = __any(odd);
        }

#pragma unroll
        for (int t = 0; t < NQ; ++t) {
            float s[KT][4];
            float top = kNone;
#pragma unroll
            for (int tt = 0; tt < KT; ++tt) {
                f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) acc = mma<T>(k[tt][kk], q[t][kk], acc);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = b + 16 * tt + 4 * g + i;
                    s[tt][i] = there[tt] && key <= last[t] && key >= first[t] ? acc[i] * a.scale2
                                                                                  : kNone;
                    top = fmaxf(top, s[tt][i]);
                }
            }
            top = over_groups(top, max_of);
            if (__any(top > m[t])) {
                const float now = fmaxf(m[t], top);
                const float f = exp2_of(m[t] - finite_max(now));
                m[t] = now;
                l[t] *= f;
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int j = 0; j < VW; ++j) o[t][c][j] *= f;
            }
            const float base = finite_max(m[t]);
            float p[E];
#pragma unroll
            for (int tt = 0; tt < KT; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[tt * 4 + i] = exp2_of(s[tt][i] - base);
                    l[t] += p[tt * 4 + i];
                }
            VOperand<T> pp;
            pp.set(p);
            constexpr int P = E == 8 ? 2 : 1;
#pragma unroll
            for (int c = 0; c < VC; ++c)
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    u32x4 left = vt(c, j);
                    if (careful) {
#pragma unroll
                        for (int d = 0; d < 4; ++d) left[d] &= ~odd_mask<T>(left[d]);
                    }
#pragma unroll
                    for (int i = 0; i < P; ++i) o[t][c][j] = mma<T>(left, pp.piece[i], o[t][c][j]);
                }
            if (careful) {
                // the values that are not finite, key by key, for the rows that see it
                for (int at = 0; at < BK; ++at) {
                    const int key = b + at;
                    const bool sees = key <= last[t] && key >= first[t];
#pragma unroll
                    for (int c = 0; c < VC; ++c)
#pragma unroll
                        for (int j = 0; j < VW; ++j) {
                            u32x4 left = vt(c, j);
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
                                uint32_t mine;           // the key's part of word d
                                if constexpr (E == 8) {
                                    const int e = 16 * (d / 2) + 4 * g + 2 * (d % 2);
                                    mine = e == at ? 0xffffu : e + 1 == at ? 0xffff0000u : 0u;
                                } else {
                                    mine = 4 * g + d == at ? ~0u : 0u;
                                }
                                left[d] &= odd_mask<T>(left[d]) & mine;
                            }
                            const f32x4 more = mma<T>(left, pp.piece[0], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[t][c][j][i] += sees ? more[i] : 0.f;
                        }
                }
            }
        }
    };
    for (int b = u.key0 + w * BK; b < u.key1; b += NW * BK) {
        Keys x;
        load(b, x);
        attend(b, x);
    }

    // The waves' parts meet in LDS, 16 rows at a time.
    constexpr int OW = DP / 16;                       // outputs of a thread
    const int row = tid >> 4, col = (tid & 15) * OW;
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
        if (t) __syncthreads();
        const float sum = over_groups(l[t], sum_of);
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < VW; j += 4)
                    *reinterpret_cast<f32x4 *>(&so[w][n][(c * 16 + 4 * g + i) * VW + j]) =
                        f32x4{o[t][c][j][i], o[t][c][j + 1][i], o[t][c][j + 2][i], o[t][c][j + 3][i]};
        if (g == 0) {
            sm[w][n] = m[t];
            sl[w][n] = sum;
        }
        __syncthreads();
        if (NW > 4 && tid >= 256) return;
        float top = sm[0][row];
#pragma unroll
        for (int i = 1; i < NW; ++i) top = fmaxf(top, sm[i][row]);
        float total = 0.f, r[OW] = {};
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const float f = exp2_of(sm[i][row] - finite_max(top));
            total += f * sl[i][row];
#pragma unroll
            for (int e = 0; e < OW; ++e) r[e] += f * so[i][row][col + e];
        }
        const int rr = u.row0 + t * 16 + row;
        if (rr >= u.rows) continue;
        const bool lost = total == 0.f && sees_a_key(a, u, rr);
        const float inv = inverse_of(total, lost, u.slot >= 0);
#pragma unroll
        for (int e = 0; e < OW; ++e) r[e] *= inv;
        if (u.slot >= 0) {
            const int64_t at = int64_t(u.slot) * (NQ * 16) + t * 16 + row;
            store_row<OW>(a.partial + at * DP + col, r);
            if ((tid & 15) == 0) a.lse[at] = log_weight(top, total, lost);
        } else {
            T *out = reinterpret_cast<T *>(a.o) + int64_t(u.tok0 + rr / a.group) * a.ldo +
                     int64_t(u.kv_head * a.group + rr % a.group) * D;
            // (D is a multiple of 8: a thread's 4 or 8 outputs exist or do not)
            if constexpr (OW < 16) {
                if (col < D) store_row<OW>(out + col, r);
            } else {
#pragma unroll
                for (int e = 0; e < OW; e += 8) {
                    const float half[8] = {r[e], r[e + 1], r[e + 2], r[e + 3],
                                           r[e + 4], r[e + 5], r[e + 6], r[e + 7]};
                    if (col + e < D) store_row<8>(out + col + e, half);
                }
            }
        }
    }
}

// The parts of a tile's keys joined: o = sum_i 2^(lse_i - M) o_i / sum_i
// 2^(lse_i - M).  16 / WAYS rows a workgroup, a row's parts dealt to WAYS groups
// of 16 threads: a few rows in many parts (single tokens behind long contexts:
// 32 parts of 4 rows took 18 us with one way, 6 with 16) or many in a few.
template <typename T, int DP, int WAYS>
__global__ __launch_bounds__(256) void k_attend_join(const AttnArgs a, int tile_rows) {
    constexpr int OW = DP / 16, ROWS = 16 / WAYS;
    __shared__ float tops[16], totals[WAYS > 1 ? 16 : 1], sums[WAYS > 1 ? 16 : 1][DP + 4];
    const AttnJoin j = load_invariant(a.joins + blockIdx.x);
    if (!held(a.dbg, j) || j.slots <= 0 || j.row0 + int(blockIdx.y) * ROWS >= j.rows) return;
    const int group = threadIdx.x >> 4, way = group % WAYS, col = (threadIdx.x & 15) * OW;
    const int row = int(blockIdx.y) * ROWS + group / WAYS, rr = j.row0 + row;
    const bool ok = row < tile_rows && rr < j.rows;
    const float *lse = a.lse + int64_t(j.slot0) * tile_rows + row;
    const float *part = a.partial + (int64_t(j.slot0) * tile_rows + row) * DP + col;
    float top = kNone;
    if (ok)
        for (int i = way; i < j.slots; i += WAYS) top = fmaxf(top, lse[int64_t(i) * tile_rows]);
    if constexpr (WAYS > 1) {
        tops[group] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAYS; ++i) top = fmaxf(top, tops[group / WAYS * WAYS + i]);
    }
    const bool lost = top == kLost;      // no part has a score above -inf
    top = finite_max(top);
    float total = 0.f, r[OW] = {};
    if (ok && col < a.head_dim) {
#pragma unroll 4
        for (int i = way; i < j.slots; i += WAYS) {
            const float f = exp2_of(lse[int64_t(i) * tile_rows] - top);
            const float *p = part + int64_t(i) * tile_rows * DP;
            total += f;
#pragma unroll
            for (int e = 0; e < OW; e += 4) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(p + e);
#pragma unroll
                for (int d = 0; d < 4; ++d) r[e + d] += f * x[d];
            }
        }
    }
    if constexpr (WAYS > 1) {
        if (col == 0) totals[group] = total;
#pragma unroll
        for (int e = 0; e < OW; ++e) sums[group][col + e] = r[e];
        __syncthreads();
        if (way) return;
        total = 0.f;
#pragma unroll
        for (int e = 0; e < OW; ++e) r[e] = 0.f;
#pragma unroll
        for (int i = 0; i < WAYS; ++i) {
            total += totals[group + i];
#pragma unroll
            for (int e = 0; e < OW; ++e) r[e] += sums[group + i][col + e];
        }
    }
    if (!ok || col >= a.head_dim) return;
    const float inv = inverse_of(lost ? 0.f : total, lost, false);
#pragma unroll
    for (int e = 0; e < OW; ++e) r[e] *= inv;
    T *out = reinterpret_cast<T *>(a.o) + int64_t(j.tok0 + rr / a.group) * a.ldo +
             int64_t(j.kv_head * a.group + rr % a.group) * a.head_dim;
    if constexpr (OW < 16) {
        store_row<OW>(out + col, r);
    } else {
#pragma unroll
        for (int e = 0; e < OW; e += 8) {
            const float half[8] = {r[e], r[e + 1], r[e + 2], r[e + 3],
                                   r[e + 4], r[e + 5], r[e + 6], r[e + 7]};
            if (col + e < a.head_dim) store_row<8>(out + col + e, half);
        }
    }
}

template <typename T, int DP, int NQ, int NW = 4>
hipError_t rows_launch(bool once, const AttnArgs &a, hipStream_t s) {
    const dim3 grid(a.num_units), block(NW * kWaveSize);
    if (once)
        hipLaunchKernelGGL((k_attend_rows<T, DP, NQ, NW, true>), grid, block, 0, s, a);
    else if constexpr (sizeof(T) == 4)
        hipLaunchKernelGGL((k_attend_rows<T, DP, NQ, NW, false>), grid, block, 0, s, a);
    else
        return hipErrorInvalidValue;       // (a tile has all of the 16 rows there can be)
    return hipGetLastError();
}
template <typename T, int DP>
hipError_t rows_dim(int tile_rows, int waves, bool once, const AttnArgs &a, hipStream_t s) {
    if constexpr (DP <= 128) {
        if (tile_rows == 16 && waves == kManyWaves) return rows_launch<T, DP, 1, kManyWaves>(once, a, s);
    }
    if (tile_rows == 16) return rows_launch<T, DP, 1>(once, a, s);
    if constexpr (sizeof(T) == 4) {
        if (tile_rows == 32) return rows_launch<T, DP, 2>(once, a, s);
    }
    if constexpr (sizeof(T) == 4 && DP <= 128) {
        if (tile_rows == 64) return rows_launch<T, DP, 4>(once, a, s);
    }
    return hipErrorInvalidValue;
}
template <typename T>
hipError_t rows_types(int tile_rows, int waves, bool once, const AttnArgs &a, hipStream_t s) {
    switch (attn_dim(a.head_dim)) {
        case 64: return rows_dim<T, 64>(tile_rows, waves, once, a, s);
        case 128: return rows_dim<T, 128>(tile_rows, waves, once, a, s);
        default: return rows_dim<T, 256>(tile_rows, waves, once, a, s);
    }
}
template <typename T, int DP> hipError_t join_launch(int tile_rows, const AttnArgs &a, hipStream_t s) {
    const dim3 block(256);
    if (tile_rows <= 16)
        hipLaunchKernelGGL((k_attend_join<T, DP, 16>), dim3(a.num_joins, tile_rows), block, 0, s, a,
                           tile_rows);
    else
        hipLaunchKernelGGL((k_attend_join<T, DP, 1>), dim3(a.num_joins, (tile_rows + 15) / 16), block,
                           0, s, a, tile_rows);
    return hipGetLastError();
}
template <typename T> hipError_t join_types(int tile_rows, const AttnArgs &a, hipStream_t s) {
    switch (attn_dim(a.head_dim)) {
        case 64: return join_launch<T, 64>(tile_rows, a, s);
        case 128: return join_launch<T, 128>(tile_rows, a, s);
        default: return join_launch<T, 256>(tile_rows, a, s);
    }
}

}  // namespace

hipError_t launch_attn_rows(int dtype, int tile_rows, int waves, bool once, const AttnArgs &a,
                            hipStream_t s) {
    if (a.num_units <= 0) return hipSuccess;
    return dtype == LORA_F32 ? rows_types<float>(tile_rows, waves, once, a, s)
                             : rows_types<uint16_t>(tile_rows, waves, once, a, s);
}

hipError_t launch_attn_join(int dtype, int tile_rows, const AttnArgs &a, hipStream_t s) {
    if (a.num_joins <= 0) return hipSuccess;
    return dtype == LORA_F32 ? join_types<float>(tile_rows, a, s)
                             : join_types<uint16_t>(tile_rows, a, s);
}

}  // namespace lora
