// The frozen layer's product with its epilogue, and the same with the tokens'
// LoRA deltas inside it:
//
//     y = act(x W^T + b + s_i B_i (A_i x)) + residual, or with a gated pair
//     y = act(x Wg^T + bg + ...) . (x Wu^T + bu + ...) + residual
//
// A few tokens read W once and are bound by its bytes; a prompt is bound by
// the matrix cores.  So there are two kernels over W's rows (the left operand
// of every MFMA, so that a lane ends with consecutive outputs of one token):
//   k_linear_rows  up to 12 tokens: a workgroup per 16 rows of W, its waves
//                  splitting K; W goes from HBM to registers.
//   k_linear_tile  token tiles x row tiles through LDS; where the tiles are
//                  too few for the chip, K is split over workgroups into
//                  float32 partial products that k_linear_join adds.
// All work is in units of 16-byte vectors (8 bf16 or 4 float32 values along
// K), so one source serves both types.  Sums are float32; y is rounded once.
#include <type_traits>

#include <hip/hip_runtime.h>

#include "device_ops.h"
#include "layer_internal.h"

namespace lora {
namespace {

#ifdef LORA_SGMV_DEBUG
constexpr bool kDebug = true;
#else
constexpr bool kDebug = false;
#endif

// Debug build: whether a check held; one that failed is noted.
[[maybe_unused]] __device__ __forceinline__ bool dbg_held(bool ok, uint32_t *word, uint32_t bit) {
    if (!ok) atomicOr(word, bit);
    return ok;
}
// The token row of a plan position: -1 (absent) when it is outside the batch
// (debug build).
__device__ __forceinline__ int token_row(const DeltaArgs &d, int pos) {
    const int r = d.order[pos];
    if constexpr (kDebug) {
        if (!dbg_held(token_inside(d.dbg, r), d.dbg_word, kDbgToken)) return -1;
    }
    return r;
}
// The bytes of the adapter block at slab offset `off`: none when it would
// leave the slab (debug build).
__device__ __forceinline__ uint32_t block_bytes(const DeltaArgs &d, uint64_t off, uint64_t bytes) {
    if constexpr (kDebug) {
        if (!dbg_held(block_inside(d.dbg, off, bytes), d.dbg_word, kDbgSlab)) return 0u;
    }
    return uint32_t(bytes);
}

// fn(0), ..., fn(N - 1) with constant indexes, whatever the body's size.
template <int N, typename Fn, int I = 0> __device__ __forceinline__ void each(Fn fn) {
    if constexpr (I < N) {
        fn(std::integral_constant<int, I>{});
        each<N, Fn, I + 1>(fn);
    }
}

// ------------------------------------------------------------- epilogue -----
// N consecutive elements of a row at any element alignment; elements at and
// past `n` are zero (loads) or left alone (stores).
typedef uint32_t u32_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <typename T> struct Run4;
template <> struct Run4<uint16_t> {
    static __device__ __forceinline__ void load(const uint8_t *p, int64_t at, int n,
                                                float (&o)[4]) {
        const uint16_t *s = reinterpret_cast<const uint16_t *>(p) + at;
        if (n >= 4) {
            const u32x2 w = *reinterpret_cast<const u32x2_any *>(s);
            o[0] = bf16_lo(w[0]); o[1] = bf16_hi(w[0]);
            o[2] = bf16_lo(w[1]); o[3] = bf16_hi(w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = i < n ? bf16_lo(s[i]) : 0.f;
        }
    }
    static __device__ __forceinline__ void store(uint8_t *p, int64_t at, int n,
                                                 const float (&o)[4]) {
        uint16_t *s = reinterpret_cast<uint16_t *>(p) + at;
        const u32x2 w{bf16x2_rne(o[0], o[1]), bf16x2_rne(o[2], o[3])};
        if (n >= 4) {
            *reinterpret_cast<u32x2_any *>(s) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < n) s[i] = uint16_t(w[i / 2] >> (16 * (i % 2)));
        }
    }
};
template <> struct Run4<float> {
    static __device__ __forceinline__ void load(const uint8_t *p, int64_t at, int n,
                                                float (&o)[4]) {
        const float *s = reinterpret_cast<const float *>(p) + at;
        if (n >= 4) {
            const u32x4 w = *reinterpret_cast<const u32x4_any *>(s);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = i < n ? s[i] : 0.f;
        }
    }
    static __device__ __forceinline__ void store(uint8_t *p, int64_t at, int n,
                                                 const float (&o)[4]) {
        float *s = reinterpret_cast<float *>(p) + at;
        if (n >= 4) {
            *reinterpret_cast<u32x4_any *>(s) = u32x4{__float_as_uint(o[0]), __float_as_uint(o[1]),
                                                      __float_as_uint(o[2]), __float_as_uint(o[3])};
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < n) s[i] = o[i];
        }
    }
};

// v / (1 + exp(-z)).  For bf16 outputs the hardware's exponential and
// reciprocal (2^-22 relative each, and |z| 1.44 2^-24 for the exponent's
// rounding, inside half a bf16 step), of 2^-8 times the sum: the sum itself
// leaves float32 left of -88 and its reciprocal is flushed to zero left of
// -87, where silu's v e^v is still a normal number, to -91.  (v / 256 keeps 15
// bits down to the least normal v.)  float32 outputs take the full-precision
// functions, left of zero as v e / (1 + e) with e = exp(z).
template <typename T> __device__ __forceinline__ float times_logistic(float v, float z) {
    if constexpr (sizeof(T) == 2) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z, -1.4426950408889634f, -8.0f));
        return v * 0x1p-8f * __builtin_amdgcn_rcpf(0x1p-8f + e);
    }
    const float e = expf(-fabsf(z));
    return (z < 0.f ? v * e : v) / (1.0f + e);
}

template <typename T, int N> __device__ __forceinline__ void activate(float (&v)[N], int act) {
    switch (act) {                                   // uniform
    case LORA_ACT_RELU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];   // NaN stays NaN
        break;
    case LORA_ACT_SILU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = times_logistic<T>(v[i], v[i]);
        break;
    case LORA_ACT_GELU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= 0.5f * erfcf(-0.70710678118654752f * v[i]);
        break;
    case LORA_ACT_GELU_TANH:                         // (1 + tanh z) / 2 = logistic(2 z)
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = times_logistic<T>(
                v[i], 1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
        break;
    default: break;
    }
}

// N consecutive outputs of one token (N 4, or 8 for one 16-byte store of
// bf16), from column f on.
template <typename T, int N> struct RunN {
    static __device__ __forceinline__ void load(const T *p, int n, float (&o)[N]) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
            float v[4];
            Run4<T>::load(reinterpret_cast<const uint8_t *>(p), 4 * h, n - 4 * h, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[4 * h + i] = v[i];
        }
    }
    static __device__ __forceinline__ void store(T *p, int n, const float (&o)[N]) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
            const float v[4] = {o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]};
            Run4<T>::store(reinterpret_cast<uint8_t *>(p), 4 * h, n - 4 * h, v);
        }
    }
};
template <> struct RunN<uint16_t, 8> {
    static __device__ __forceinline__ void load(const uint16_t *p, int n, float (&o)[8]) {
        if (n >= 8) {
            const u32x4 w = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[2 * i] = bf16_lo(w[i]);
                o[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = i < n ? bf16_lo(p[i]) : 0.f;
        }
    }
    static __device__ __forceinline__ void store(uint16_t *p, int n, const float (&o)[8]) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = bf16x2_rne(o[2 * i], o[2 * i + 1]);
        if (n >= 8) {
            *reinterpret_cast<u32x4_any *>(p) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) p[i] = uint16_t(w[i / 2] >> (16 * (i % 2)));
        }
    }
};

// The end of one token's outputs f .. f + N - 1: bias, activation, gating,
// residual, rounding, store.  `n`: outputs from f on that exist (N or more:
// all of them, one vector each way).
template <typename T, bool GLU, int N>
__device__ __forceinline__ void finish(const LinearArgs &a, int t, int f, int n, float (&v)[N],
                                       float (&up)[N]) {
    if (t < 0 || n <= 0) return;
    if (a.bias) {
        const T *bias = reinterpret_cast<const T *>(a.bias) + f;
        float b[N];
        RunN<T, N>::load(bias, n, b);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += b[i];
        if constexpr (GLU) {
            RunN<T, N>::load(bias + a.n, n, b);
#pragma unroll
            for (int i = 0; i < N; ++i) up[i] += b[i];
        }
    }
    activate<T>(v, a.act);
    if constexpr (GLU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= up[i];
    }
    if (a.residual) {
        float r[N];
        RunN<T, N>::load(reinterpret_cast<const T *>(a.residual) + int64_t(t) * a.ldr + f, n, r);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += r[i];
    }
    RunN<T, N>::store(reinterpret_cast<T *>(a.y) + int64_t(t) * a.ldy + f, n, v);
}

// -------------------------------------------------------------- operand -----
// The delta's right operand for one (block, projection): scale * v of each
// position, as three bf16 pieces whose sum is that float32 value exactly, or
// (float32) the value.  The scale goes into v here, one float32 rounding per
// entry, so that the products below need none.
template <typename T> __global__ __launch_bounds__(256) void k_operand(const OperandArgs a) {
    constexpr int P = VOperand<T>::kPieces, E = Elem<T>::E;
    const int b = blockIdx.x / a.nproj, p = blockIdx.x % a.nproj;
    BlockDesc blk = load_invariant(a.blocks + b);
    if constexpr (kDebug) {
        blk.n_tok = dbg_held(rows_inside(a.dbg, blk.tok_off, blk.n_tok), a.dbg_word, kDbgRow)
                        ? min(blk.n_tok, kMaxBlockTokens) : 0;
    }
    const rsrc_t pr = make_rsrc(a.partial, a.partial_bytes);
    const int vecs = a.r_max / E;
    for (int i = threadIdx.x; i < blk.n_tok * vecs; i += 256) {
        const int ti = i / vecs, j = (i % vecs) * E, pos = blk.tok_off + ti;
        const float s = a.tok_w ? blk.scale * a.tok_w[pos] : blk.scale;
        float f[E];
#pragma unroll
        for (int h = 0; h < E / 4; ++h) {
            f32x4 s4{0.f, 0.f, 0.f, 0.f};
            if (j + 4 * h < blk.r_pad) {
                if (b < a.nb_long)
                    s4 = *reinterpret_cast<const f32x4 *>(
                        a.v + (int64_t(pos) * a.nproj + p) * a.r_max + j + 4 * h);
                else
                    s4 = chunk_sum(pr, partial_off(blk.rt_before, j + 4 * h, blk.slot0 + ti, p,
                                                   a.nproj, a.c0, 1),
                                   uint32_t(a.nproj * kTile * kTile), a.c0);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) f[4 * h + k] = s * s4[k];
        }
        VOperand<T> vo;
        vo.set(f);
        uint8_t *o = a.out + ((int64_t(pos) * a.nproj + p) * P * a.r_max + j) * int64_t(sizeof(T));
#pragma unroll
        for (int k = 0; k < P; ++k)
            *reinterpret_cast<u32x4 *>(o + int64_t(k) * a.r_max * int64_t(sizeof(T))) = vo.piece[k];
    }
}

// ---------------------------------------------------------------- delta -----
// The part of a lane's 4 consecutive rows that lies in a slice of ho rows, the
// first of them row o: rows outside it have no delta, and a product of zeros
// there would not do (times an infinite or NaN operand it is NaN).
__device__ __forceinline__ f32x4 in_slice(f32x4 s, int o, int ho) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = uint32_t(o + i) < uint32_t(ho) ? s[i] : 0.f;
    return s;
}

// B's vector for the second and third piece of the operand: those are what
// the first leaves of v, and zero where it holds all of it, so that an
// infinite (or NaN) B times them would be NaN where B v is infinite.  B's
// own value counts with the first piece alone, which has v's sign and is zero
// where v is.
__device__ __forceinline__ u32x4 finite_bf16(u32x4 b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((b[i] & 0x7f80u) == 0x7f80u) b[i] &= 0xffff0000u;
        if ((b[i] & 0x7f800000u) == 0x7f800000u) b[i] &= 0xffffu;
    }
    return b;
}
// Whether any lane holds a value that is not finite (uniform).
template <int N> __device__ __forceinline__ bool any_odd(const f32x4 (&s)[N]) {
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) z = __builtin_fmaf(s[j][i], 0.f, z);
    return __builtin_amdgcn_ballot_w64(z != z) != 0;
}

// The delta of 16 plan positions and 16 G outputs, added to `acc`, in order
// (row r of tile j is output f0 + 16 j + r: neighbouring rows of B are what
// its block keeps together).  Positions are in plan order, so a group's are
// neighbours: each group's B rows multiply every position's operand and are
// kept in the columns of the group's own (so one adapter's infinities stay
// with its tokens).  Of `nw` waves that share the tile, wave w takes every
// nw-th group.  What this costs is the chain of dependent loads position -> B
// rows, so the positions bring their group's extent with them and the B rows
// of NB groups are in flight together.  KS: K-steps of the plan's largest
// rank.
template <typename T, int G, int KS, bool CAREFUL>
__device__ __forceinline__ void add_groups(const DeltaArgs &d, int p0, int f0, int w, int nw,
                                          f32x4 (&acc)[G]) {
    constexpr int E = Elem<T>::E, SPAN = 4 * E, P = VOperand<T>::kPieces;
    constexpr int NB = G * KS >= 8 ? 1 : 8 / (G * KS);
    if (p0 >= d.n_active) return;                // uniform
    const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
    const int pos = p0 + n;
    PosRow pr{};
    pr.group = -1;
    if (pos < d.n_active) pr = d.pos[pos];
    const int vrow = P * d.r_max * int(sizeof(T));
    for (int p = 0; p < d.nproj; ++p) {
        const int lo = d.y_off[p], ho = d.h_out[p];
        if (f0 + 16 * G <= lo || f0 >= lo + ho) continue;
        VOperand<T> vo[KS];
        if (KS == 1 && d.partial) {              // uniform
            const rsrc_t parts = make_rsrc(d.partial, d.partial_bytes);
            const int j = q * E;
            float f[E];
#pragma unroll
            for (int h = 0; h < E / 4; ++h) {
                f32x4 s4{0.f, 0.f, 0.f, 0.f};
                if (j + 4 * h < pr.r_pad)
                    s4 = chunk_sum(parts, partial_off(pr.rt, j + 4 * h, pr.slot, p, d.nproj, d.c0, 1),
                                   uint32_t(d.nproj * kTile * kTile), d.c0);
#pragma unroll
                for (int k = 0; k < 4; ++k) f[4 * h + k] = pr.scale * s4[k];
            }
            vo[0].set(f);
        } else {
            const uint8_t *vp = d.v + (int64_t(pos) * d.nproj + p) * vrow;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    vo[ks].piece[i] = u32x4{0u, 0u, 0u, 0u};
                    const int j = ks * SPAN + q * E;
                    if (pos < d.n_active && j < d.r_max)
                        vo[ks].piece[i] = *reinterpret_cast<const u32x4 *>(
                            vp + (i * d.r_max + j) * int(sizeof(T)));
                }
        }
        // the first position of each group in the tile, one bit a lane
        const int before = __shfl_up(pr.group, 1, 16);
        uint32_t todo = uint32_t(__builtin_amdgcn_ballot_w64(
                            pr.group >= 0 && (n == 0 || pr.group != before))) & 0xffffu;
        for (int i = 0; i < w && todo; ++i) todo &= todo - 1;
        while (todo) {                           // uniform
            u32x4 bf[NB][G][KS];
            int grp[NB], rp[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const bool any = todo != 0;
                const int l = any ? __builtin_ctz(todo) : 0;
                for (int i = 0; i < nw; ++i) todo &= todo - 1;
                grp[b] = any ? __builtin_amdgcn_readlane(pr.group, l) : -2;
                rp[b] = any ? __builtin_amdgcn_readlane(pr.r_pad, l) : 0;
                const uint64_t off = extent(__builtin_amdgcn_readlane(pr.ext_lo, l),
                                            __builtin_amdgcn_readlane(pr.ext_hi, l)) +
                                     uint64_t(rp[b]) * sizeof(T) * uint64_t(d.coef_b[p]);
                const rsrc_t br = make_rsrc(
                    d.slab + off, block_bytes(d, off, uint64_t(ho) * uint64_t(rp[b]) * sizeof(T)));
                const BLayout bl = b_layout(rp[b], int(sizeof(T)));
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const int o = f0 + 16 * j + n - lo;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const int v = ks * 4 + q;
                        bf[b][j][ks] = bload16(br, off_or_oob(o >= 0 && o < ho && v < bl.nv,
                                                              b_vec_off(bl, o, v, ho)));
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const bool mine = pr.group == grp[b];
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    f32x4 s4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        if (ks * SPAN < rp[b]) {         // uniform
                            const u32x4 low = CAREFUL && P > 1 ? finite_bf16(bf[b][j][ks])
                                                               : bf[b][j][ks];
#pragma unroll
                            for (int i = P - 1; i >= 0; --i)
                                s4 = mma<T>(i ? low : bf[b][j][ks], vo[ks].piece[i], s4);
                        }
                    if constexpr (CAREFUL) s4 = in_slice(s4, f0 + 16 * j + 4 * q - lo, ho);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = mine ? acc[j][i] + s4[i] : acc[j][i];
                }
            }
        }
    }
}

// The delta into `acc`.  Only where it is not finite does it matter that rows
// outside the slice, and pieces that are zero, are left out rather than
// multiplied: then it is formed again, in that careful form.
template <typename T, int G, int KS>
__device__ __forceinline__ void delta_of(const DeltaArgs &d, int p0, int f0, int w, int nw,
                                         f32x4 (&acc)[G]) {
#pragma unroll
    for (int j = 0; j < G; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    add_groups<T, G, KS, false>(d, p0, f0, w, nw, acc);
    if (!any_odd(acc)) return;
#pragma unroll
    for (int j = 0; j < G; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    add_groups<T, G, KS, true>(d, p0, f0, w, nw, acc);
}

// ----------------------------------------------------------------- rows -----
// One workgroup per 16 outputs (rows of W; with a gated pair 16 of gate and
// the same 16 of up); wave w takes its share of K for all of them and all of
// the up to 12 tokens, in batches of F vectors a lane whose loads are in
// flight while the batch before multiplies.  The waves' sums meet in LDS.
// Bound by W's bytes: 235 MB of gate and up rows at K 4096 in 47.5 us (4.95
// TB/s; a copy of 1 GiB reads and writes 5.15).  KS: K-steps of the delta, 0
// without adapters.  The compiler is left to its own count of registers but
// for the gated bf16 pair with one K-step of delta, one register over what
// three waves a SIMD have (4 tokens, 4096 x 28672, rank 16: 71.0 us held to
// them, 72.6 without).
template <typename T, bool GLU, int KS, int NW>
__global__ __launch_bounds__(NW * kWaveSize, sizeof(T) == 2 && GLU && KS == 1 ? 3 : 1) void
k_linear_rows(const LinearArgs a) {
    constexpr int E = Elem<T>::E, SPAN = 4 * E, NR = GLU ? 2 : 1, F = 4;
    __shared__ f32x4 red[NW][NR][kWaveSize];
    const int unit = xcd_range_unit(a.units);
    if (unit >= a.units) return;                 // whole workgroup
    const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
    const int w = wave_id();
    const int f0 = unit * 16;
    const int rows = min(16, a.n - f0);
    const uint32_t wrow = uint32_t(a.ldw) * sizeof(T), xrow = uint32_t(a.ldx) * sizeof(T);
    const uint32_t kb = uint32_t(a.k) * sizeof(T);

    rsrc_t wr[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r)
        wr[r] = make_rsrc(a.w + (int64_t(r) * a.n + f0) * a.ldw * int64_t(sizeof(T)),
                          uint32_t(rows - 1) * wrow + kb);
    const rsrc_t xr = make_rsrc(a.x, uint32_t(a.T - 1) * xrow + kb);

    const int steps = (a.k + SPAN - 1) / SPAN;
    int per = (steps + NW - 1) / NW;
    per += per & 1;                              // whole 128-byte lines a wave
    const int s_lo = w * per, s_hi = min(s_lo + per, steps);

    // this lane's token row (with adapters: in plan order)
    const int tok = n < a.T ? (KS ? token_row(a.delta, n) : n) : -1;
    f32x4 acc[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};

    struct Batch {
        u32x4 w[NR][F], x[F];
    };
    auto load = [&](Batch &b, int s0) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const uint32_t kq = uint32_t(s0 + f) * (SPAN * sizeof(T)) + uint32_t(q) * 16u;
            const bool ok = s0 + f < s_hi && kq < kb;
#pragma unroll
            for (int r = 0; r < NR; ++r)
                b.w[r][f] = bload16_nt(wr[r], off_or_oob(ok && n < rows, uint32_t(n) * wrow + kq));
            b.x[f] = bload16(xr, off_or_oob(ok && tok >= 0, uint32_t(tok) * xrow + kq));
        }
    };
    auto multiply = [&](const Batch &b) {
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int r = 0; r < NR; ++r) acc[r] = mma<T>(b.w[r][f], b.x[f], acc[r]);
    };
    Batch b0, b1;
    load(b0, s_lo);
    if constexpr (KS > 0) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            f32x4 d[1];
            delta_of<T, 1, KS>(a.delta, 0, r * a.n + f0, w, NW, d);
            acc[r] = d[0];
        }
    }
    for (int s = s_lo; s < s_hi; s += 2 * F) {   // uniform
        load(b1, s + F);
        multiply(b0);
        load(b0, s + 2 * F);
        multiply(b1);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) red[w][r][lane] = acc[r];
    __syncthreads();
    if (w == 0) {
        float v[NR][4];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            f32x4 s4 = red[0][r][lane];
#pragma unroll
            for (int i = 1; i < NW; ++i) s4 += red[i][r][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[r][i] = s4[i];
        }
        finish<T, GLU>(a, tok, f0 + 4 * q, a.n - f0 - 4 * q, v[0], v[NR - 1]);
    }
}

// ----------------------------------------------------------------- tile -----
// A direct copy of 16 bytes a lane from memory to LDS at m0 + 16 * lane, past
// the registers.  Written as one instruction block: the compiler then does not
// wait for every copy before the next LDS read, and the kernel counts them
// itself.  Out-of-range lanes write zeros.  (The wait states cover a resource
// word that a vector instruction wrote just before: 5; m0 needs 1.)
// ONCE: the bytes are read by no other workgroup, and streamed past the L2.
template <bool ONCE = false>
__device__ __forceinline__ void copy_to_lds(u32x4 rsrc, uint32_t voff, uint32_t soff,
                                            uint32_t lds) {
    if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                     ::"s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     ::"s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                     : "memory");
}
template <int N> __device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ u32x4 raw_rsrc(const void *base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return u32x4{uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(p))),
                 uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(p >> 32) & 0xffffu)),
                 uint32_t(__builtin_amdgcn_readfirstlane(bytes)), uint32_t(kRsrcWord3)};
}

// One K tile of the delta as a lane copies it.
struct DeltaTile {
    BLayout bl;
    uint64_t off;                // B block in the slab
    uint32_t bytes;
    uint32_t voff;               // the lane's vector in a position's operand row
    int vrow;                    // bytes of such a row
    int first, end;              // positions of the group
    int col0, h_out;             // row of B of the tile's first output
    int vec;                     // the lane's vector of a B row
    int half;                    // 1: gate (or all), 2: up
    int head;                    // vectors of the first piece (none: at most 0)
    bool ok;                     // the lane has a vector
};

// What a stage of the delta holds: the half of W's rows (1: gate, or all; 2:
// up; 0: nothing), the group's positions, the slice's rows (the tile's first
// output is row col0 of h_out), and how many of its vectors, the first ones,
// are the operand's first piece.
struct DeltaHeld {
    int half, first, end, col0, h_out, head;
};

// The walk over a tile's delta K tiles: groups, projections, halves, then the
// 8-vector steps of pieces x vectors.  All of it is uniform.
template <typename T, int HALVES> struct DeltaTiles {
    static constexpr int P = VOperand<T>::kPieces;
    int g, g1, p, h, s, first, end, f0, feat, n;
    GroupRow gr;

    __device__ __forceinline__ int steps() const {
        return (P * (gr.r_pad * int(sizeof(T)) / 16) + 7) / 8;
    }
    __device__ __forceinline__ bool meets(const DeltaArgs &d) const {
        const int c0 = h * n + f0, lo = d.y_off[p];
        return c0 < lo + d.h_out[p] && c0 + feat > lo;
    }
    __device__ __forceinline__ void load(const DeltaArgs &d) {
        gr = load_invariant(d.groups + g);
        first = gr.first;
        end = load_invariant(&d.groups[g + 1].first);
        if constexpr (kDebug) {
            if (!dbg_held(end >= first && rows_inside(d.dbg, first, end - first), d.dbg_word, kDbgRow))
                first = end = 0;                 // no position's
            if (!dbg_held(padded_rank(gr.r_pad), d.dbg_word, kDbgSlab)) {
                gr.r_pad = 8;
                gr.ext_hi = 0x7fffffffu;         // a block that leaves the slab
            }
        }
    }
    // on to the first (projection, half) from the current one that the tile meets
    __device__ __forceinline__ void settle(const DeltaArgs &d) {
        while (g <= g1 && !meets(d)) {
            if (++h < HALVES) continue;
            h = 0;
            if (++p < d.nproj) continue;
            p = 0;
            if (++g <= g1) load(d);
        }
    }
    __device__ __forceinline__ void start(const DeltaArgs &d, int t0, int rows, int f0_, int feat_,
                                          int n_) {
        f0 = f0_;
        feat = feat_;
        n = n_;
        p = h = s = 0;
        const int last = min(t0 + rows, d.n_active) - 1;
        g = 1;
        g1 = 0;
        bool any = false;                        // a tile that meets no projection has no walk
        for (int i = 0; i < d.nproj; ++i)
            for (int k = 0; k < HALVES; ++k)
                any |= k * n + f0 < d.y_off[i] + d.h_out[i] && k * n + f0 + feat > d.y_off[i];
        if (last < t0 || !any) return;
        g = load_invariant(&d.pos[t0].group);
        g1 = load_invariant(&d.pos[last].group);
        if constexpr (kDebug) {
            // (the groups' table ends with a row of no adapter)
            if (!dbg_held(group_inside(d.num_groups - 1, g) && group_inside(d.num_groups - 1, g1),
                          d.dbg_word, kDbgRow)) {
                g = 1;
                g1 = 0;
                return;
            }
        }
        load(d);
        settle(d);
    }
    // what the current tile is; past the end one without vectors
    __device__ __forceinline__ DeltaTile tile(const DeltaArgs &d, uint32_t vec) const {
        DeltaTile e{};
        e.vrow = d.nproj * P * d.r_max * int(sizeof(T));
        if (g > g1) return e;
        e.bl = b_layout(gr.r_pad, int(sizeof(T)));
        e.off = extent(gr.ext_lo, gr.ext_hi) + uint64_t(gr.r_pad) * sizeof(T) * uint64_t(d.coef_b[p]);
        e.h_out = d.h_out[p];
        e.bytes = block_bytes(d, e.off, uint64_t(e.h_out) * uint64_t(gr.r_pad) * sizeof(T));
        const int at = s * 8 + int(vec), piece = at / e.bl.nv;
        e.vec = at - piece * e.bl.nv;
        e.ok = piece < P;
        e.voff = uint32_t(((p * P + piece) * d.r_max) * int(sizeof(T)) + e.vec * 16);
        e.first = first;
        e.end = end;
        e.col0 = h * n + f0 - d.y_off[p];
        e.half = h + 1;
        e.head = e.bl.nv - s * 8;
        return e;
    }
    __device__ __forceinline__ void next(const DeltaArgs &d) {
        if (g > g1 || ++s < steps()) return;
        s = 0;
        if (++h == HALVES) {
            h = 0;
            if (++p == d.nproj) {
                p = 0;
                if (++g <= g1) load(d);
            }
        }
        settle(d);
    }
};

// One workgroup per BT tokens x BN rows of W (with a gated pair BN / 2 of
// gate and the same BN / 2 of up), WT x WN waves, over the K tiles of its
// part.  A K tile is 128 bytes of every row, whole cache lines; S of them are
// in LDS or on their way.  A row's 8 vectors are stored exchanged by
// (row / 2) % 8 (exclusive or), so that the 16 rows a fragment read touches
// spread over all banks (no conflicts counted).
// What bounds it: prompts the matrix cores, at the clock they leave (1.7 to
// 1.9 GHz under this load: a 256 x 256 tile keeps them busy two thirds of its
// cycles; LDS reads and copies fill as many); 4096 x 4096 x 4096 bf16 107 us
// in a loop, 120 from cold caches, 4096 tokens through a gated 28672 x 4096
// pair 714 to 732 us in a loop (1.32 to 1.35 PFLOP/s).  8 waves of 128 x 64
// beat 4 of 128 x 128 (713 against 907 us), whose single wave a SIMD has
// nothing to run at a barrier, and the products spelled out between reads and
// copies beat the compiler's order (833 against 890).
// Decode batches get W at 3.2 to 3.6 TB/s in the best split of each tile (128
// x 4096 x 14336 without the join, us: 128 x 128 in 8 parts 32.4, 128 x 64 in 4
// 32.9, 64 x 128 in 4 34.6, 128 x 256 in 16 36.5), where the rows kernel gets
// 4.9 from the same matrix.  What holds them there is not found: not HBM, not
// what enters the CUs (x and W, 4.8 to 10.7 TB/s in these, 13.9 with 128 x 32
// tiles), not a stage more or less (128 x 64 with 3 instead of 4: 34.0).  K
// tiles rotated by workgroup or of 256 bytes a row measured the same, dealt in
// turn to the parts a fifth slower.  ONCE (one token tile: a row of W is one
// workgroup's) streams W past the L2, which keeps x there and leaves nothing
// behind for the next product's W to push out: in a loop over changing weights
// 36.7 us against 41.5 with the join (128 x 4096 x 14336), 124 against 131
// (the gated batch of 256 with adapters); where token tiles share W it has to
// stay.
// W's rows sit in LDS in the order that gives a lane consecutive outputs: LDS
// row 16 j + r of a wave's share is output (r / 4) 4 G + 4 j + r % 4, G tiles
// of 16 wide.
template <typename T, int BT, int BN, int WT, int WN, int S, bool GLU, bool SPLIT, bool ADAPT,
          bool ONCE = false>
__global__ __launch_bounds__(WT *WN *kWaveSize) void k_linear_tile(const LinearArgs a) {
    constexpr int NW = WT * WN, NTH = NW * kWaveSize;
    constexpr int TI = BT / WT / 16, TJ = BN / WN / 16, G = GLU ? TJ / 2 : TJ;
    constexpr int XL = BT * 8 / NTH, WL = BN * 8 / NTH;      // copies a lane per K tile
    constexpr int FEAT = GLU ? BN / 2 : BN;
    constexpr int STAGE = (BT + BN) * kKBytes;
    static_assert(XL >= 1 && WL >= 1 && XL * NTH == BT * 8 && WL * NTH == BN * 8, "whole copies");
    static_assert(!GLU || TJ % 2 == 0, "gate and up tiles in pairs");
    __shared__ __align__(1024) uint8_t lds[S * STAGE];

    const int unit = xcd_range_unit(a.units);
    if (unit >= a.units) return;
    const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, q = lane >> 4;
    const int wave = wave_id();
    const int wt = wave / WN, wn = wave % WN;
    // tiles in order: 8 token tiles beside one another, then along W, so that
    // the 32 workgroups of an XCD share 8 tiles of x and 4 of W in its L2
    const int z = unit / (a.tiles_t * a.tiles_n), in_z = unit % (a.tiles_t * a.tiles_n);
    const int group = in_z / (8 * a.tiles_n), in_g = in_z % (8 * a.tiles_n);
    const int gt = min(8, a.tiles_t - group * 8);
    const int tt = group * 8 + in_g % gt, nt = in_g / gt;
    const int t0 = tt * BT, f0 = nt * FEAT;
    const int wide = GLU ? a.n : a.wide;                     // rows of one half of W
    const uint32_t wrow = uint32_t(a.ldw) * sizeof(T), xrow = uint32_t(a.ldx) * sizeof(T);
    const uint32_t kb = uint32_t(a.k) * sizeof(T);

    const int xrows = min(BT, a.T - t0), wrows = min(FEAT, wide - f0);
    // with adapters x's rows are gathered in plan order (x spans at most 2 GiB)
    const u32x4 xr = ADAPT ? raw_rsrc(a.x, uint32_t(a.T - 1) * xrow + kb)
                           : raw_rsrc(a.x + int64_t(t0) * xrow, uint32_t(xrows - 1) * xrow + kb);
    const u32x4 wr = raw_rsrc(a.w + int64_t(f0) * wrow, uint32_t(wrows - 1) * wrow + kb);
    const u32x4 wr2 = GLU ? raw_rsrc(a.w + (int64_t(a.n) + f0) * wrow,
                                     uint32_t(wrows - 1) * wrow + kb) : wr;

    // this lane's copies: the rows, and the vector of them (the same for all:
    // its copies are a multiple of 16 rows apart)
    static_assert(NTH / 8 % 16 == 0, "one vector index a lane");
    const uint32_t vec = uint32_t((tid & 7) ^ ((tid >> 4) & 7));
    uint32_t xo[XL], wo[WL];
    int wf[WL];                                              // output of the row, from f0
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int row = (i * NTH + tid) >> 3;
        const int t = ADAPT && row < xrows ? token_row(a.delta, t0 + row) : row;
        xo[i] = row < xrows && (!kDebug || t >= 0) ? uint32_t(t) * xrow + vec * 16u : kOOB;
    }
#pragma unroll
    for (int i = 0; i < WL; ++i) {
        const int row = (i * NTH + tid) >> 3;
        const int share = row / (16 * TJ), j = row / 16 % TJ, r = row % 16;
        wf[i] = share * 16 * G + (r >> 2) * 4 * G + (j % G) * 4 + (r & 3);
        wo[i] = wf[i] < wrows ? uint32_t(wf[i]) * wrow + vec * 16u : kOOB;
    }
    const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) uint8_t *)lds));
    const int nk = (int(kb) + kKBytes - 1) / kKBytes;
    const int k_lo = SPLIT ? z * a.k_tiles : 0, k_hi = SPLIT ? min(k_lo + a.k_tiles, nk) : nk;

    auto up_rows = [&](int i) {                              // uniform
        return GLU && ((i * NTH + wave * 64) / 8 / 16) % TJ >= G;
    };
    // copy `at` of K tile kt into stage st; in a row's last tile, lanes past
    // its end, and past the last tile all lanes, are out of range
    auto fetch_one = [&](int kt, int st, auto index) {
        constexpr int at = decltype(index)::value;
        const uint32_t base = lds0 + uint32_t(st * STAGE) + uint32_t(wave) * 1024u;
        const uint32_t soff = uint32_t(kt) * kKBytes;
        const bool in = kt < k_hi && vec * 16u < kb - soff;
        if constexpr (at < XL)
            copy_to_lds(xr, in ? xo[at] : kOOB, soff, base + uint32_t(at * NTH * 16));
        else
            copy_to_lds<ONCE>(up_rows(at - XL) ? wr2 : wr, in ? wo[at - XL] : kOOB, soff,
                              base + uint32_t(BT * kKBytes + (at - XL) * NTH * 16));
    };
    auto fetch = [&](int kt, int st) {
        each<XL + WL>([&](auto at) { fetch_one(kt, st, at); });
    };
    // The delta as further K tiles: for each adapter group among the tile's
    // positions and each projection among its columns, the columns are the
    // group's operand, piece after piece (zero for other groups' positions),
    // against B's rows, repeated for each piece.  With a gated pair a tile
    // belongs to one half.
    auto fetch_delta = [&](auto &dt, int st) -> DeltaHeld {
        const uint32_t base = lds0 + uint32_t(st * STAGE) + uint32_t(wave) * 1024u;
        const DeltaArgs &d = a.delta;
        const DeltaTile e = dt.tile(d, vec);
        const u32x4 vr = raw_rsrc(d.v + int64_t(t0) * e.vrow, uint32_t(xrows) * uint32_t(e.vrow));
        const u32x4 br = raw_rsrc(d.slab + e.off, e.bytes);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int row = (i * NTH + tid) >> 3;
            const bool in = e.ok && t0 + row >= e.first && t0 + row < e.end;
            copy_to_lds(vr, in ? uint32_t(row) * uint32_t(e.vrow) + e.voff : kOOB, 0u,
                        base + uint32_t(i * NTH * 16));
        }
#pragma unroll
        for (int i = 0; i < WL; ++i) {
            const int o = e.col0 + wf[i];
            const bool in = e.ok && (!GLU || up_rows(i) == (e.half == 2)) && o >= 0 && o < e.h_out;
            copy_to_lds(br, in ? b_vec_off(e.bl, o, e.vec, e.h_out) : kOOB, 0u,
                        base + uint32_t(BT * kKBytes + i * NTH * 16));
        }
        dt.next(d);
        return DeltaHeld{e.half, e.first, e.end, e.col0, e.h_out, e.head};
    };

    f32x4 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // byte offset of this lane's fragment vector kk of a 16-row tile
    uint32_t fo[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
        fo[kk] = uint32_t(n) * kKBytes + uint32_t((kk * 4 + q) ^ ((n >> 1) & 7)) * 16u;

    auto x_frag = [&](int st, int i, int kk) {
        return *reinterpret_cast<const u32x4 *>(lds + st * STAGE + (wt * TI + i) * 16 * kKBytes +
                                                fo[kk]);
    };
    auto w_frag = [&](int st, int j, int kk) {
        return *reinterpret_cast<const u32x4 *>(lds + st * STAGE + BT * kKBytes +
                                                (wn * TJ + j) * 16 * kKBytes + fo[kk]);
    };
    struct Frags {
        u32x4 f[TJ + TI];                        // W's row tiles, then x's token tiles
    };
    auto read = [&](Frags &f, int st, int kk, auto index) {
        constexpr int r = decltype(index)::value;
        if constexpr (r < TJ) f.f[r] = w_frag(st, r, kk);
        else f.f[r] = x_frag(st, r - TJ, kk);
    };
    // One half of a K tile: the products of `use` in groups of 4, and between
    // the groups the reads of the next half's fragments into `next` (early,
    // so that they have arrived at the half's end) and `copies` of the ND
    // copies of a stage to come.  Spelled out and pinned, because a wave may
    // be alone on its SIMD: what it issues in one go, its matrix core waits for.
    constexpr int NM = TI * TJ, MG = NM >= 4 ? 4 : NM, NS = NM / MG, NR = TI + TJ, ND = XL + WL;
    constexpr int RPS = (NR + (NS + 1) / 2 - 1) / ((NS + 1) / 2), DPS = (ND + NS - 1) / NS;
    auto half = [&](const Frags &use, Frags &next, int st, int kk, auto with_copies, int kt,
                    int st_in) {
        each<NS>([&](auto step) {
            constexpr int s = decltype(step)::value;
            each<RPS>([&](auto r) {
                constexpr int at = s * RPS + decltype(r)::value;
                if constexpr (at < NR) read(next, st, kk, std::integral_constant<int, at>{});
            });
            if constexpr (decltype(with_copies)::value)
                each<DPS>([&](auto r) {
                    constexpr int at = s * DPS + decltype(r)::value;
                    if constexpr (at < ND) fetch_one(kt, st_in, std::integral_constant<int, at>{});
                });
            each<MG>([&](auto m) {
                constexpr int at = s * MG + decltype(m)::value, i = at / TJ, j = at % TJ;
                acc[i][j] = mma<T>(use.f[j], use.f[TJ + i], acc[i][j]);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // acc += a stage of one group's delta, in the columns of its positions
    // only: other positions' tiles are passed over, and in a tile that holds
    // both, a sum apart is kept or dropped by column, and at the slice's edges
    // by row (zeros in the operands would not do: an infinite or NaN adapter
    // times zero is NaN)
    auto multiply_delta = [&](int st, const DeltaHeld &e) {
        const bool upper_half = e.half == 2;
        u32x4 b[2][G];                           // B's rows, for all of the positions
        f32x4 probe[1] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                b[kk][j] = w_frag(st, (upper_half ? G : 0) + j, kk);
                if constexpr (VOperand<T>::kPieces > 1)
                    probe[0] = mma<T>(b[kk][j], u32x4{0u, 0u, 0u, 0u}, probe[0]);
            }
        if (VOperand<T>::kPieces > 1 && any_odd(probe)) {
            // pieces past the first: see finite_bf16
#pragma unroll
            for (int j = 0; j < G; ++j)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const u32x4 f = finite_bf16(b[kk][j]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[kk][j][i] = kk * 4 + q >= e.head ? f[i] : b[kk][j][i];
                }
        }
        const bool edge = e.col0 < 0 || e.col0 + FEAT > e.h_out;   // uniform
        each<TI>([&](auto index) {
            constexpr int i = decltype(index)::value;
            const int p0 = t0 + (wt * TI + i) * 16;
            if (p0 >= e.end || p0 + 16 <= e.first) return;   // uniform
            const bool mine = p0 + n >= e.first && p0 + n < e.end;
            const u32x4 x0 = x_frag(st, i, 0), x1 = x_frag(st, i, 1);
            // (both halves by selects: a branch would turn the accumulators
            // into memory)
            const bool lower = mine && !upper_half, upper = mine && upper_half;
            f32x4 s4[G];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                s4[j] = mma<T>(b[0][j], x0, f32x4{0.f, 0.f, 0.f, 0.f});
                s4[j] = mma<T>(b[1][j], x1, s4[j]);
            }
            if (edge) {
#pragma unroll
                for (int j = 0; j < G; ++j)
                    s4[j] = in_slice(s4[j], e.col0 + (wn * 16 + q * 4) * G + 4 * j, e.h_out);
            }
#pragma unroll
            for (int j = 0; j < G; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[i][j][k] = lower ? acc[i][j][k] + s4[j][k] : acc[i][j][k];
                    if constexpr (GLU)
                        acc[i][TJ - G + j][k] = upper ? acc[i][TJ - G + j][k] + s4[j][k]
                                                      : acc[i][TJ - G + j][k];
                }
        });
    };
    int st = 0;
    // Every LDS read runs under a half's products: the second half's
    // fragments are read while the first multiplies, the next stage's first
    // half while the second does; the one barrier of a K tile stands between,
    // when this wave has its second half in registers, and frees the stage
    // for the copies of K tile kt + S.
    Frags fa, fb;
    DeltaTiles<T, GLU ? 2 : 1> dt;
    DeltaHeld held[S];                           // the delta's stages to come, in order
    auto next_delta = [&](int st) {
#pragma unroll
        for (int s = 0; s < S - 1; ++s) held[s] = held[s + 1];
        held[S - 1] = fetch_delta(dt, st);
    };
    if constexpr (ADAPT) dt.start(a.delta, t0, min(BT, xrows), f0, FEAT, a.n);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (!ADAPT || k_lo + s < k_hi) fetch(k_lo + s, s);
        else next_delta(s);
    }
    wait_copies<(S - 1) * (XL + WL)>();
    __builtin_amdgcn_s_barrier();
    each<NR>([&](auto r) { read(fa, 0, 0, r); });
    auto first_half = [&] {
        half(fa, fb, st, 1, std::false_type{}, 0, 0);
        wait_copies<(S - 2) * (XL + WL)>();      // the next stage's copies, in order
        wait_lds();
        __builtin_amdgcn_s_barrier();
        const int free = st;
        st = st + 1 == S ? 0 : st + 1;
        return free;
    };
    int kt = k_lo;
    for (; kt < (ADAPT ? k_hi - S : k_hi); ++kt) {
        const int free = first_half();
        half(fb, fa, st, 0, std::true_type{}, kt + S, free);
    }
    if constexpr (ADAPT) {
        // the delta's first stages come in under the last K tiles
        for (; kt < k_hi; ++kt) {
            const int free = first_half();
            next_delta(free);
            half(fb, fa, st, 0, std::false_type{}, 0, 0);
        }
    }
    if constexpr (ADAPT) {
        // (a tile without a delta runs it once, on a stage of no positions:
        // with a way round the loop the accumulators are held twice, 75 to
        // 114 registers too many for the largest tile)
        do {
            wait_copies<(S - 1) * (XL + WL)>();
            __builtin_amdgcn_s_barrier();
            multiply_delta(st, held[0]);
            wait_lds();
            __builtin_amdgcn_s_barrier();        // the stage is free
            next_delta(st);
            st = st + 1 == S ? 0 : st + 1;
        } while (held[0].half);                  // uniform
    }
    wait_copies<0>();                            // none may land after the workgroup's end

    const int fw = f0 + wn * 16 * G;             // the wave's first output
    each<TI>([&](auto index) {                   // accumulators need constant indexes
        constexpr int i = decltype(index)::value;
        const int ti = t0 + (wt * TI + i) * 16, pos = ti + n;
        if (ti >= a.T) return;                   // uniform
        if constexpr (SPLIT) {
            if (pos < a.T) {
                float *p = a.partial + (int64_t(z) * a.T + pos) * a.ldp + fw + q * 4 * G;
#pragma unroll
                for (int j = 0; j < TJ; ++j)
                    if (fw + q * 4 * G + 4 * j < a.ldp) *reinterpret_cast<f32x4 *>(p + 4 * j) = acc[i][j];
            }
        } else {
            const int t = pos < a.T ? (ADAPT ? token_row(a.delta, pos) : pos) : -1;
            constexpr int N = G % 2 == 0 ? 8 : 4;
            each<G * 4 / N>([&](auto run) {
                constexpr int j0 = decltype(run)::value * (N / 4);
                float v[N], u[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    v[k] = acc[i][j0 + k / 4][k % 4];
                    u[k] = acc[i][TJ - G + j0 + k / 4][k % 4];
                }
                // (a tile inside W: no counts by lane)
                const int f = fw + q * 4 * G + 4 * j0;
                finish<T, GLU>(a, t, f, f0 + FEAT <= a.n ? N : a.n - f, v, u);
            });
        }
    });
}

// ----------------------------------------------------------------- join -----
// One wave per 16 tokens (with adapters: plan positions) x 16 G columns of a
// product in parts: the parts' sum and the delta.  With a gated pair gate's
// and up's columns are two waves', which meet in LDS; else waves share
// nothing.  A wave's chain of dependent loads is what it waits for, so small
// waves, many of them resident, beat fewer that share a tile through LDS (64
// columns, the parts and groups dealt to 4 or 8 waves: 12.4 and 17.7 us for
// a decode batch's q/k/v, 66 and 69 for its gated pair of mixed ranks).
template <typename T, bool GLU, int KS, int G>
__global__ __launch_bounds__(256) void k_linear_join(const LinearArgs a) {
    constexpr int NR = GLU ? 2 : 1, Z = 4, TILES = 4 / NR;   // column tiles a workgroup
    __shared__ f32x4 up[GLU ? 2 * G : 1][kWaveSize];
    const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
    const int w = wave_id(), r = GLU ? w & 1 : 0, tile = w / NR;
    const int tiles_t = (a.T + 15) / 16;
    const int p0 = blockIdx.x % tiles_t * 16;
    const int f0 = (blockIdx.x / tiles_t * TILES + tile) * 16 * G;
    const int pos = p0 + n;
    const int t = pos < a.T ? (KS ? token_row(a.delta, pos) : pos) : -1;
    const int c0 = r * a.n + f0;                 // column before the activation
    f32x4 s[G];
#pragma unroll
    for (int j = 0; j < G; ++j) s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (f0 < a.n) {                              // uniform
        if constexpr (KS > 0) delta_of<T, G, KS>(a.delta, p0, c0, 0, 1, s);
        // the parts in order, Z of them in flight
        const float *p = a.partial + int64_t(t) * a.ldp + c0 + q * 4;
        const int64_t step = int64_t(a.T) * a.ldp;
        for (int z = 0; z < a.splits; z += Z) {
            u32x4 v[Z][G];
#pragma unroll
            for (int k = 0; k < Z; ++k)
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    v[k][j] = u32x4{0u, 0u, 0u, 0u};
                    // (any alignment: the second half of a pair starts at column n)
                    if (t >= 0 && z + k < a.splits && c0 + q * 4 + 16 * j < a.wide)
                        v[k][j] = *reinterpret_cast<const u32x4_any *>(p + (z + k) * step + 16 * j);
                }
#pragma unroll
            for (int k = 0; k < Z; ++k)
#pragma unroll
                for (int j = 0; j < G; ++j) s[j] += __builtin_bit_cast(f32x4, v[k][j]);
        }
    }
    if constexpr (GLU) {
        if (r == 1) {
#pragma unroll
            for (int j = 0; j < G; ++j) up[tile * G + j][lane] = s[j];
        }
        __syncthreads();
        if (r == 1) return;
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
        const f32x4 u4 = GLU ? up[GLU ? tile * G + j : 0][lane] : f32x4{0.f, 0.f, 0.f, 0.f};
        float v[4] = {s[j][0], s[j][1], s[j][2], s[j][3]};
        float u[4] = {u4[0], u4[1], u4[2], u4[3]};
        const int f = f0 + 16 * j + 4 * q;
        finish<T, GLU>(a, t, f, a.n - f, v, u);
    }
}

// ------------------------------------------------------------- launches -----
template <typename T> constexpr int dtype_of = sizeof(T) == 2 ? LORA_BF16 : LORA_F32;

dim3 grid_of(int units) { return dim3((units + kXcds - 1) / kXcds * kXcds); }

// K-steps of the delta's largest rank, as the kernels are built for it
template <typename T> int delta_steps(const LinearArgs &a) {
    if (!a.delta.order) return 0;
    return a.delta.max_rpad <= one_step_rank(dtype_of<T>)
               ? 1 : LORA_MAX_RANK / (4 * Elem<T>::E);
}

template <typename T, bool GLU, int NW>
hipError_t rows_launch(const LinearArgs &a, hipStream_t s) {
    constexpr int KM = LORA_MAX_RANK / (4 * Elem<T>::E);
    const dim3 grid = grid_of(a.units), block(NW * 64);
    const int ks = delta_steps<T>(a);
    if (ks == 0) hipLaunchKernelGGL((k_linear_rows<T, GLU, 0, NW>), grid, block, 0, s, a);
    else if (ks == 1) hipLaunchKernelGGL((k_linear_rows<T, GLU, 1, NW>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_linear_rows<T, GLU, KM, NW>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <typename T, bool GLU> void join_launch(const LinearArgs &a, hipStream_t s) {
    constexpr int KM = LORA_MAX_RANK / (4 * Elem<T>::E);
    constexpr int GM = join_tiles(dtype_of<T>, LORA_MAX_RANK);
    const int ks = delta_steps<T>(a);
    const int cols = join_cols(dtype_of<T>, GLU, ks ? a.delta.max_rpad : 0);
    const dim3 grid((a.T + 15) / 16 * ((a.n + cols - 1) / cols)), block(256);
    if (ks == 0) hipLaunchKernelGGL((k_linear_join<T, GLU, 0, 1>), grid, block, 0, s, a);
    else if (ks == 1) hipLaunchKernelGGL((k_linear_join<T, GLU, 1, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_linear_join<T, GLU, KM, GM>), grid, block, 0, s, a);
}

template <typename T, bool GLU>
hipError_t rows_dispatch(const LinearArgs &a, hipStream_t s) {
    // waves a workgroup: with few workgroups (narrow products) more of them
    // keep the chip's loads busy: 8 against 4 take 10.6 us and 11.3 at
    // 1024 x 4096, 53.6 and 50.2 at 28672 x 4096, 30.3 and 27.2 at 4096 x 14336
    if (a.units <= 128) return rows_launch<T, GLU, 8>(a, s);
    return rows_launch<T, GLU, 4>(a, s);
}

template <typename T, int BT, int BN, int WT, int WN, int S, bool GLU>
hipError_t direct_launch(const LinearArgs &a, dim3 grid, dim3 block, hipStream_t s) {
    if (a.delta.order)
        hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, GLU, false, true>), grid, block, 0, s, a);
    else if constexpr (!plain_tile(dtype_of<T>, BT, BN))
        return hipErrorInvalidValue;
    else if (a.tiles_t == 1)
        hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, GLU, false, false, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, GLU, false, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <typename T, int BT, int BN, int WT, int WN, int S>
hipError_t tile_launch(const LinearPlan &pl, bool glu, const LinearArgs &a, hipStream_t s) {
    const dim3 grid = grid_of(a.units), block(WT * WN * 64);
    if (!pl.joined)
        return glu ? direct_launch<T, BT, BN, WT, WN, S, true>(a, grid, block, s)
                   : direct_launch<T, BT, BN, WT, WN, S, false>(a, grid, block, s);
    if constexpr (plain_tile(dtype_of<T>, BT, BN)) {
        if (a.tiles_t == 1)
            hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, false, true, false, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, false, true, false>), grid, block, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (glu) join_launch<T, true>(a, s);
        else join_launch<T, false>(a, s);
        return hipGetLastError();
    }
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t linear_dispatch(const LinearPlan &pl, bool glu, const LinearArgs &a, hipStream_t s) {
    if (pl.kind == kLinearRows)
        return glu ? rows_dispatch<T, true>(a, s) : rows_dispatch<T, false>(a, s);
    if (pl.bt == 32 && pl.bn == 64) return tile_launch<T, 32, 64, 1, 2, 4>(pl, glu, a, s);
    if (pl.bt == 64 && pl.bn == 128) return tile_launch<T, 64, 128, 1, 4, 4>(pl, glu, a, s);
    if (pl.bt == 128 && pl.bn == 128) return tile_launch<T, 128, 128, 2, 2, 4>(pl, glu, a, s);
    if constexpr (sizeof(T) == 2) {
        if (pl.bt == 128 && pl.bn == 64) return tile_launch<T, 128, 64, 2, 2, 4>(pl, glu, a, s);
        if (pl.bt == 256 && pl.bn == 128) return tile_launch<T, 256, 128, 4, 2, 3>(pl, glu, a, s);
        if (pl.bt == 256 && pl.bn == 256) return tile_launch<T, 256, 256, 2, 4, 2>(pl, glu, a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_operand(int dtype, const OperandArgs &a, hipStream_t s) {
    if (a.nb <= 0) return hipSuccess;
    const dim3 grid(a.nb * a.nproj), block(256);
    if (dtype == LORA_BF16) hipLaunchKernelGGL(k_operand<uint16_t>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_operand<float>, grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_linear(int dtype, const LinearPlan &pl, bool glu, LinearArgs a, hipStream_t s) {
    if (a.T <= 0) return hipSuccess;
    a.splits = pl.splits;
    a.k_tiles = pl.k_tiles;
    if (pl.kind == kLinearRows) {
        a.units = (a.n + 15) / 16;
    } else {
        // a joined product takes W's rows as they are, a direct one takes gate
        // and up rows in pairs
        const bool pairs = glu && !pl.joined;
        const int feat = pairs ? pl.bn / 2 : pl.bn;
        a.tiles_t = (a.T + pl.bt - 1) / pl.bt;
        a.tiles_n = ((pairs ? a.n : a.wide) + feat - 1) / feat;
        a.units = a.tiles_t * a.tiles_n * pl.splits;
    }
    return dtype == LORA_BF16 ? linear_dispatch<uint16_t>(pl, glu, a, s)
                              : linear_dispatch<float>(pl, glu, a, s);
}

}  // namespace lora
