// The frozen layer's product with its epilogue, and the same with the tokens'
// LoRA deltas inside it:
//
//     y = act(x W^T + b + s_i B_i (A_i x)) + residual, or with a gated pair
//     y = act(x Wg^T + bg + ...) . (x Wu^T + bu + ...) + residual
//
// A few tokens read W once and are bound by its bytes; a prompt is bound by
// the matrix cores.  So there are two kernels over W's rows (the left operand
// of every MFMA, so that a lane ends with consecutive outputs of one token):
//   k_linear_rows  up to 16 TT tokens: a workgroup per 16 rows of W, its waves
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

// 1 / (1 + exp(-v)).  For bf16 outputs the hardware's exponential and
// reciprocal (a few 2^-22 relative, far inside half a bf16 step); float32
// outputs take the full-precision functions.
template <typename T> __device__ __forceinline__ float logistic(float v) {
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.0f + __expf(-v));
    return 1.0f / (1.0f + expf(-v));
}

template <typename T> __device__ __forceinline__ float activate(float v, int act) {
    switch (act) {                                   // uniform
    case LORA_ACT_RELU: return v < 0.f ? 0.f : v;    // NaN stays NaN
    case LORA_ACT_SILU: return v * logistic<T>(v);
    case LORA_ACT_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    case LORA_ACT_GELU_TANH:                         // (1 + tanh z) / 2 = logistic(2 z)
        return v * logistic<T>(1.5957691216057308f * (v + 0.044715f * v * v * v));
    default: return v;
    }
}

// The end of one token's outputs f .. f + 3: bias, activation, gating,
// residual, rounding, store.
template <typename T, bool GLU>
__device__ __forceinline__ void finish(const LinearArgs &a, int t, int f, float (&v)[4],
                                       float (&up)[4]) {
    const int n = a.n - f;
    if (t >= a.T || n <= 0) return;
    if (a.bias) {
        float b[4];
        Run4<T>::load(a.bias, f, n, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += b[i];
        if constexpr (GLU) {
            Run4<T>::load(a.bias, int64_t(a.n) + f, n, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) up[i] += b[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = activate<T>(v[i], a.act);
        if constexpr (GLU) v[i] *= up[i];
    }
    if (a.residual) {
        float r[4];
        Run4<T>::load(a.residual, int64_t(t) * a.ldr + f, n, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += r[i];
    }
    Run4<T>::store(a.y, int64_t(t) * a.ldy + f, n, v);
}

// ---------------------------------------------------------------- delta -----
// Adds scale * B v to one 16-token tile's accumulators: rows of the left
// operand are outputs f(j, r) = f0 + (r / 4) 4 G + 4 j + r % 4, so a lane
// holds outputs f0 + 4 G q .. + 4 G of its token.  The tile's distinct
// adapters are taken one after another (their B rows against every token's
// v, kept only in the columns of the adapter's own tokens); of `nw` waves
// that share the tile, wave w takes every nw-th of them.  v is split into
// three bf16 pieces whose sum is v, so B v is the float32 product.
template <typename T, int G>
__device__ __forceinline__ void add_delta(const DeltaArgs &d, int T_, int t0, int f0, int w,
                                          int nw, f32x4 (&acc)[G]) {
    constexpr int E = Elem<T>::E, SPAN = 4 * E, KS = LORA_MAX_RANK / SPAN;
    const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
    const int t = t0 + n;
    TokenRow tr{0u, 0u, 0, 0.f};
    if (t < T_) tr = d.rows[t];
    const uint32_t have = uint32_t(__builtin_amdgcn_ballot_w64(tr.r_pad > 0)) & 0xffffu;
    if (!have) return;
    for (int p = 0; p < d.nproj; ++p) {
        const int lo = d.y_off[p], ho = d.h_out[p];
        if (f0 + 16 * G <= lo || f0 >= lo + ho) continue;
        VOperand<T> vo[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int j0 = ks * SPAN + q * E;
            float f[E];
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = 0.f;
            if (j0 < tr.r_pad) {
                const f32x4 *src = reinterpret_cast<const f32x4 *>(
                    d.v + int64_t(t) * d.ldv + int64_t(p) * d.r_max + j0);
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    const f32x4 s4 = src[i];
#pragma unroll
                    for (int k = 0; k < 4; ++k) f[4 * i + k] = s4[k];
                }
            }
            vo[ks].set(f);
        }
        uint32_t todo = have;
        for (int idx = 0; todo; ++idx) {
            const int l = __builtin_ctz(todo);
            const uint32_t elo = __builtin_amdgcn_readlane(tr.ext_lo, l);
            const uint32_t ehi = __builtin_amdgcn_readlane(tr.ext_hi, l);
            const int r_pad = __builtin_amdgcn_readlane(tr.r_pad, l);
            const bool mine = tr.ext_lo == elo && tr.ext_hi == ehi && tr.r_pad > 0;
            todo &= ~uint32_t(__builtin_amdgcn_ballot_w64(mine));
            if (idx % nw != w) continue;
            const uint64_t off = extent(elo, ehi) + uint64_t(r_pad) * sizeof(T) *
                                                        uint64_t(d.coef_b[p]);
            const uint64_t bytes = uint64_t(ho) * uint64_t(r_pad) * sizeof(T);
            uint32_t range = uint32_t(bytes);
            if constexpr (kDebug) {
                if (off + bytes > d.dbg.slab_bytes) {
                    atomicOr(d.dbg_word, uint32_t(kDbgSlab));
                    range = 0u;
                }
            }
            const rsrc_t br = make_rsrc(d.slab + off, range);
            const BLayout bl = b_layout(r_pad, int(sizeof(T)));
            u32x4 bf[G][KS];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int o = f0 + (n >> 2) * 4 * G + 4 * j + (n & 3) - lo;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const int v = ks * 4 + q;
                    bf[j][ks] = bload16(br, off_or_oob(o >= 0 && o < ho && v < bl.nv,
                                                       b_vec_off(bl, o, v, ho)));
                }
            }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                f32x4 s4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    if (ks * SPAN < r_pad) {             // uniform
#pragma unroll
                        for (int i = VOperand<T>::kPieces - 1; i >= 0; --i)
                            s4 = mma<T>(bf[j][ks], vo[ks].piece[i], s4);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[j][i] = mine ? acc[j][i] + tr.scale * s4[i] : acc[j][i];
            }
        }
    }
}

// The plain remap of launch order to units: each XCD takes one contiguous
// range, so that neighbouring units share an L2.
__device__ __forceinline__ int xcd_range(int units) {
    const int g = blockIdx.x;
    return (g % kXcds) * ((units + kXcds - 1) / kXcds) + g / kXcds;
}

// ----------------------------------------------------------------- rows -----
// One workgroup per 16 outputs (rows of W; with a gated pair 16 of gate and
// the same 16 of up); wave w takes its share of K for all of them and all of
// the up to 16 TT tokens, in batches of F vectors a lane whose loads are in
// flight while the batch before multiplies.  The waves' sums meet in LDS.
template <typename T, int TT, bool GLU, bool ADAPT, int NW>
__global__ __launch_bounds__(NW * kWaveSize) void k_linear_rows(const LinearArgs a) {
    constexpr int E = Elem<T>::E, SPAN = 4 * E, NR = GLU ? 2 : 1;
    constexpr int F = TT == 1 ? 4 : 2;
    __shared__ f32x4 red[NW][NR * TT][kWaveSize];
    const int unit = xcd_range(a.units);
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

    f32x4 acc[NR][TT];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) acc[r][tt] = f32x4{0.f, 0.f, 0.f, 0.f};

    struct Batch {
        u32x4 w[NR][F], x[TT][F];
    };
    auto load = [&](Batch &b, int s0) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const uint32_t kq = uint32_t(s0 + f) * (SPAN * sizeof(T)) + uint32_t(q) * 16u;
            const bool ok = s0 + f < s_hi && kq < kb;
#pragma unroll
            for (int r = 0; r < NR; ++r)
                b.w[r][f] = bload16_nt(wr[r], off_or_oob(ok && n < rows, uint32_t(n) * wrow + kq));
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
                b.x[tt][f] = bload16(xr, off_or_oob(ok && tt * 16 + n < a.T,
                                                    uint32_t(tt * 16 + n) * xrow + kq));
        }
    };
    auto multiply = [&](const Batch &b) {
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) acc[r][tt] = mma<T>(b.w[r][f], b.x[tt][f], acc[r][tt]);
    };
    Batch b0, b1;
    load(b0, s_lo);
    if constexpr (ADAPT) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                f32x4 d[1] = {acc[r][tt]};
                add_delta<T, 1>(a.delta, a.T, tt * 16, r * a.n + f0, w, NW, d);
                acc[r][tt] = d[0];
            }
    }
    for (int s = s_lo; s < s_hi; s += 2 * F) {   // uniform
        load(b1, s + F);
        multiply(b0);
        load(b0, s + 2 * F);
        multiply(b1);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) red[w][r * TT + tt][lane] = acc[r][tt];
    __syncthreads();
    if (w < TT) {
        float v[NR][4];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            f32x4 s4 = red[0][r * TT + w][lane];
#pragma unroll
            for (int i = 1; i < NW; ++i) s4 += red[i][r * TT + w][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[r][i] = s4[i];
        }
        finish<T, GLU>(a, w * 16 + n, f0 + 4 * q, v[0], v[NR - 1]);
    }
}

// ----------------------------------------------------------------- tile -----
// A direct copy of 16 bytes a lane from memory to LDS at m0 + 16 * lane, past
// the registers.  Written as one instruction block: the compiler then does not
// wait for every copy before the next LDS read, and the kernel counts them
// itself.  Out-of-range lanes write zeros.  (The wait states cover a resource
// word that a vector instruction wrote just before: 5; m0 needs 1.)
__device__ __forceinline__ void copy_to_lds(u32x4 rsrc, uint32_t voff, uint32_t soff,
                                            uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds),
                 "v"(voff), "s"(rsrc), "s"(soff)
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

// One workgroup per BT tokens x BN rows of W (with a gated pair BN / 2 of
// gate and the same BN / 2 of up), WT x WN waves, over the K tiles of its
// split.  A K tile is 128 bytes of every row; S of them are in LDS or on
// their way.  A row's 8 vectors are stored rotated by (row / 2) % 8
// (exclusive or), so that the 16 rows a fragment read touches spread over
// all banks.  W's rows sit in LDS in the order that gives a lane consecutive
// outputs: LDS row 16 j + r of a wave's share is output (r / 4) 4 G + 4 j +
// r % 4, G tiles of 16 wide.
template <typename T, int BT, int BN, int WT, int WN, int S, bool GLU, bool SPLIT, bool ADAPT>
__global__ __launch_bounds__(WT *WN *kWaveSize) void k_linear_tile(const LinearArgs a) {
    constexpr int NW = WT * WN, NTH = NW * kWaveSize;
    constexpr int TI = BT / WT / 16, TJ = BN / WN / 16, G = GLU ? TJ / 2 : TJ;
    constexpr int XL = BT * 8 / NTH, WL = BN * 8 / NTH;      // copies a lane per K tile
    constexpr int FEAT = GLU ? BN / 2 : BN;
    constexpr int STAGE = (BT + BN) * kKBytes;
    static_assert(XL >= 1 && WL >= 1 && XL * NTH == BT * 8 && WL * NTH == BN * 8, "whole copies");
    static_assert(!GLU || TJ % 2 == 0, "gate and up tiles in pairs");
    __shared__ __align__(1024) uint8_t lds[S * STAGE];

    const int unit = xcd_range(a.units);
    if (unit >= a.units) return;
    const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, q = lane >> 4;
    const int wave = wave_id();
    const int wt = wave / WN, wn = wave % WN;
    const int tt = unit % a.tiles_t, rest = unit / a.tiles_t;
    const int nt = rest % a.tiles_n, z = rest / a.tiles_n;
    const int t0 = tt * BT, f0 = nt * FEAT;
    const int wide = GLU ? a.n : a.wide;                     // rows of one half of W
    const uint32_t wrow = uint32_t(a.ldw) * sizeof(T), xrow = uint32_t(a.ldx) * sizeof(T);
    const uint32_t kb = uint32_t(a.k) * sizeof(T);

    const int xrows = min(BT, a.T - t0), wrows = min(FEAT, wide - f0);
    const u32x4 xr = raw_rsrc(a.x + int64_t(t0) * xrow, uint32_t(xrows - 1) * xrow + kb);
    const u32x4 wr = raw_rsrc(a.w + int64_t(f0) * wrow, uint32_t(wrows - 1) * wrow + kb);
    const u32x4 wr2 = GLU ? raw_rsrc(a.w + (int64_t(a.n) + f0) * wrow,
                                     uint32_t(wrows - 1) * wrow + kb) : wr;

    // this lane's copies: the row and the vector of the row each brings in
    uint32_t xo[XL], wo[WL], xc[XL], wc[WL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int row = (i * NTH + tid) >> 3;
        xc[i] = uint32_t((tid & 7) ^ ((row >> 1) & 7)) * 16u;
        xo[i] = row < xrows ? uint32_t(row) * xrow + xc[i] : kOOB;
    }
#pragma unroll
    for (int i = 0; i < WL; ++i) {
        const int row = (i * NTH + tid) >> 3;
        wc[i] = uint32_t((tid & 7) ^ ((row >> 1) & 7)) * 16u;
        const int share = row / (16 * TJ), j = row / 16 % TJ, r = row % 16;
        const int f = share * 16 * G + (r >> 2) * 4 * G + (j % G) * 4 + (r & 3);
        wo[i] = f < wrows ? uint32_t(f) * wrow + wc[i] : kOOB;
    }
    const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) uint8_t *)lds));
    const int nk = (int(kb) + kKBytes - 1) / kKBytes;
    const int k_lo = SPLIT ? z * a.k_tiles : 0, k_hi = SPLIT ? min(k_lo + a.k_tiles, nk) : nk;

    // copies of K tile kt into stage st; past the split's end, and past the
    // row's end in its last tile, lanes are out of range
    auto fetch = [&](int kt, int st) {
        const uint32_t soff = uint32_t(kt) * kKBytes;
        const uint32_t left = kt < k_hi ? kb - soff : 0u;     // bytes of the row from here
        const uint32_t base = lds0 + uint32_t(st * STAGE) + uint32_t(wave) * 1024u;
#pragma unroll
        for (int i = 0; i < XL; ++i)
            copy_to_lds(xr, xc[i] < left ? xo[i] : kOOB, soff, base + uint32_t(i * NTH * 16));
#pragma unroll
        for (int i = 0; i < WL; ++i) {
            const bool up = GLU && ((i * NTH + wave * 64) / 8 / 16) % TJ >= G;   // uniform
            copy_to_lds(up ? wr2 : wr, wc[i] < left ? wo[i] : kOOB, soff,
                        base + uint32_t(BT * kKBytes + i * NTH * 16));
        }
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

#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(k_lo + s, s);
    int st = 0, st_in = S - 1;
    for (int kt = k_lo; kt < k_hi; ++kt) {
        wait_copies<(S - 2) * (XL + WL)>();      // this stage's copies, in order
        __builtin_amdgcn_s_barrier();            // everyone's; stage st_in is free
        fetch(kt + S - 1, st_in);
        const uint8_t *xs = lds + st * STAGE + wt * (TI * 16 * kKBytes);
        const uint8_t *ws = lds + st * STAGE + BT * kKBytes + wn * (TJ * 16 * kKBytes);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            u32x4 xf[TI], wf[TJ];
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                wf[j] = *reinterpret_cast<const u32x4 *>(ws + j * 16 * kKBytes + fo[kk]);
#pragma unroll
            for (int i = 0; i < TI; ++i)
                xf[i] = *reinterpret_cast<const u32x4 *>(xs + i * 16 * kKBytes + fo[kk]);
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j) acc[i][j] = mma<T>(wf[j], xf[i], acc[i][j]);
        }
        wait_lds();                              // this wave has read the stage
        st = st + 1 == S ? 0 : st + 1;
        st_in = st_in + 1 == S ? 0 : st_in + 1;
    }
    wait_copies<0>();                            // none may land after the workgroup's end

    const int fw = f0 + wn * 16 * G;             // the wave's first output
    each<TI>([&](auto index) {                   // accumulators need constant indexes
        constexpr int i = decltype(index)::value;
        const int ti = t0 + (wt * TI + i) * 16, t = ti + n;
        if (ti >= a.T) return;                   // uniform
        if constexpr (SPLIT) {
            if (t < a.T) {
                float *p = a.partial + (int64_t(z) * a.T + t) * a.ldp + fw + q * 4 * G;
#pragma unroll
                for (int j = 0; j < TJ; ++j)
                    if (fw + q * 4 * G + 4 * j < a.ldp) *reinterpret_cast<f32x4 *>(p + 4 * j) = acc[i][j];
            }
        } else {
            f32x4 g[G], u[G];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                g[j] = acc[i][j];
                u[j] = acc[i][TJ - G + j];
            }
            if constexpr (ADAPT) {
                add_delta<T, G>(a.delta, a.T, ti, fw, 0, 1, g);
                if constexpr (GLU) add_delta<T, G>(a.delta, a.T, ti, a.n + fw, 0, 1, u);
            }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                float v[4] = {g[j][0], g[j][1], g[j][2], g[j][3]};
                float v2[4] = {u[j][0], u[j][1], u[j][2], u[j][3]};
                finish<T, GLU>(a, t, fw + q * 4 * G + 4 * j, v, v2);
            }
        }
    });
}

// ----------------------------------------------------------------- join -----
// One workgroup per 16 tokens x 64 outputs of a split product: wave w adds
// partial products w, w + 4, ... and the deltas of every fourth adapter, the
// waves' sums meet in LDS, and each wave finishes 4 tokens (a row of 64
// outputs is one contiguous store).
template <typename T, bool GLU, bool ADAPT>
__global__ __launch_bounds__(256) void k_linear_join(const LinearArgs a) {
    constexpr int NR = GLU ? 2 : 1, G = 4;
    __shared__ f32x4 red[4][NR * G][kWaveSize];
    const int unit = blockIdx.x;
    const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
    const int w = wave_id();
    const int tiles_t = (a.T + 15) / 16;
    const int t0 = unit % tiles_t * 16, f0 = unit / tiles_t * 64;
    const int t = t0 + n;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int c0 = r * a.n + f0;             // column before the activation
        f32x4 s[G];
#pragma unroll
        for (int j = 0; j < G; ++j) s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int z = w; z < a.splits; z += 4) {
            const float *p = a.partial + (int64_t(z) * a.T + t) * a.ldp + c0 + q * 16;
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (t < a.T && c0 + q * 16 + 4 * j < a.wide) {
                    // (any alignment: the second half of a pair starts at column n)
                    const u32x4 v = *reinterpret_cast<const u32x4_any *>(p + 4 * j);
                    s[j] += __builtin_bit_cast(f32x4, v);
                }
        }
        if constexpr (ADAPT) add_delta<T, G>(a.delta, a.T, t0, c0, w, 4, s);
#pragma unroll
        for (int j = 0; j < G; ++j) red[w][r * G + j][lane] = s[j];
    }
    __syncthreads();
    // outputs 4 m .. 4 m + 3 of token 4 w + lane / 16
    const int m = lane & 15, tok = 4 * w + (lane >> 4);
    float v[NR][4];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int e = (m >> 2) * 16 + tok;
        f32x4 s4 = red[0][r * G + (m & 3)][e];
#pragma unroll
        for (int i = 1; i < 4; ++i) s4 += red[i][r * G + (m & 3)][e];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[r][i] = s4[i];
    }
    finish<T, GLU>(a, t0 + tok, f0 + 4 * m, v[0], v[NR - 1]);
}

// ------------------------------------------------------------- launches -----
dim3 grid_of(int units) { return dim3((units + kXcds - 1) / kXcds * kXcds); }

template <typename T, int TT, bool GLU, int NW>
hipError_t rows_launch(const LinearArgs &a, hipStream_t s) {
    if (a.delta.rows)
        hipLaunchKernelGGL((k_linear_rows<T, TT, GLU, true, NW>), grid_of(a.units), dim3(NW * 64), 0, s, a);
    else
        hipLaunchKernelGGL((k_linear_rows<T, TT, GLU, false, NW>), grid_of(a.units), dim3(NW * 64), 0, s, a);
    return hipGetLastError();
}

template <typename T, bool GLU>
hipError_t rows_dispatch(const LinearPlan &pl, const LinearArgs &a, hipStream_t s) {
    if (pl.bt == 16) return rows_launch<T, 1, GLU, 16>(a, s);
    return rows_launch<T, 2, GLU, 8>(a, s);
}

template <typename T, int BT, int BN, int WT, int WN, int S>
hipError_t tile_launch(const LinearPlan &pl, bool glu, const LinearArgs &a, hipStream_t s) {
    const dim3 grid = grid_of(a.units), block(WT * WN * 64);
    const bool adapt = a.delta.rows != nullptr;
    if (pl.splits > 1) {
        hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, false, true, false>), grid, block, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const dim3 jgrid(((a.T + 15) / 16) * ((a.n + 63) / 64)), jblock(256);
        if (glu) {
            if (adapt) hipLaunchKernelGGL((k_linear_join<T, true, true>), jgrid, jblock, 0, s, a);
            else hipLaunchKernelGGL((k_linear_join<T, true, false>), jgrid, jblock, 0, s, a);
        } else {
            if (adapt) hipLaunchKernelGGL((k_linear_join<T, false, true>), jgrid, jblock, 0, s, a);
            else hipLaunchKernelGGL((k_linear_join<T, false, false>), jgrid, jblock, 0, s, a);
        }
    } else if (glu) {
        if (adapt) hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, true, false, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, true, false, false>), grid, block, 0, s, a);
    } else {
        if (adapt) hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, false, false, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_linear_tile<T, BT, BN, WT, WN, S, false, false, false>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t linear_dispatch(const LinearPlan &pl, bool glu, const LinearArgs &a, hipStream_t s) {
    if (pl.kind == kLinearRows)
        return glu ? rows_dispatch<T, true>(pl, a, s) : rows_dispatch<T, false>(pl, a, s);
    if (pl.bt == 64) return tile_launch<T, 64, 128, 1, 4, 4>(pl, glu, a, s);
    if (pl.bt == 128) return tile_launch<T, 128, 128, 2, 2, 2>(pl, glu, a, s);
    if constexpr (sizeof(T) == 2)
        if (pl.bt == 256) return tile_launch<T, 256, 256, 2, 4, 2>(pl, glu, a, s);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_linear(int dtype, const LinearPlan &pl, bool glu, LinearArgs a, hipStream_t s) {
    if (a.T <= 0) return hipSuccess;
    a.splits = pl.splits;
    a.k_tiles = pl.k_tiles;
    if (pl.kind == kLinearRows) {
        a.units = (a.n + 15) / 16;
    } else {
        // a split product takes W's rows as they are, a direct one takes gate
        // and up rows in pairs
        const int feat = glu && pl.splits == 1 ? pl.bn / 2 : pl.bn;
        a.tiles_t = (a.T + pl.bt - 1) / pl.bt;
        a.tiles_n = ((glu && pl.splits == 1 ? a.n : a.wide) + feat - 1) / feat;
        a.units = a.tiles_t * a.tiles_n * pl.splits;
    }
    return dtype == LORA_BF16 ? linear_dispatch<uint16_t>(pl, glu, a, s)
                              : linear_dispatch<float>(pl, glu, a, s);
}

}  // namespace lora
