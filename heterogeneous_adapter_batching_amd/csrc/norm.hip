// The norms around a block, fused with the residual stream's update:
//
//     n  = N_post(o),   h' = beta h + alpha g . n,   u = N_pre(h')
//
// with N an RMS norm (v / sqrt(mean(v^2) + eps)), a layer norm
// ((v - mean v) / sqrt(mean((v - mean v)^2) + eps)) or nothing, each with its
// weight and bias.  The work is a few operations per element read, so HBM
// bounds it: o and h are read once and h' and u written once, and a row stays
// in registers (float32) between its two reductions.  The layer norm's
// variance is the mean of the centred squares, from the registers, not a
// difference of sums, which would cancel for rows with a large mean.  u is
// formed from the unrounded h': rounding h' first would put the stored
// type's error into every element of u.
#include <algorithm>

#include <hip/hip_runtime.h>

#include "device_ops.h"
#include "layer_internal.h"

namespace lora {
namespace {

// 8 consecutive elements of a row as loaded, any element alignment (the
// hardware takes unaligned dwordx4 accesses).
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <typename T> struct Row8;
template <> struct Row8<uint16_t> {
    u32x4 r;
    __device__ __forceinline__ void zero() { r = u32x4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ void load(const uint16_t *p) {
        r = *reinterpret_cast<const u32x4_any *>(p);
    }
    __device__ __forceinline__ void load_tail(const uint16_t *p, int n) {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n) r[j / 2] |= uint32_t(p[j]) << (16 * (j % 2));
    }
    __device__ __forceinline__ float get(int j) const {
        return j % 2 ? bf16_hi(r[j / 2]) : bf16_lo(r[j / 2]);
    }
    static __device__ __forceinline__ void store(uint16_t *p, const float (&v)[8], int n) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = bf16x2_rne(v[2 * j], v[2 * j + 1]);
        if (n >= 8) {
            *reinterpret_cast<u32x4_any *>(p) = w;
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < n) p[j] = uint16_t(w[j / 2] >> (16 * (j % 2)));
        }
    }
};
template <> struct Row8<float> {
    u32x4 r[2];
    __device__ __forceinline__ void zero() { r[0] = r[1] = u32x4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ void load(const float *p) {
        r[0] = *reinterpret_cast<const u32x4_any *>(p);
        r[1] = *reinterpret_cast<const u32x4_any *>(p + 4);
    }
    __device__ __forceinline__ void load_tail(const float *p, int n) {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n) r[j / 4][j % 4] = __float_as_uint(p[j]);
    }
    __device__ __forceinline__ float get(int j) const { return __uint_as_float(r[j / 4][j % 4]); }
    static __device__ __forceinline__ void store(float *p, const float (&v)[8], int n) {
        if (n >= 8) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<u32x4_any *>(p + 4 * k) =
                    u32x4{__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]),
                          __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3])};
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < n) p[j] = v[j];
        }
    }
};

// The sum over a wave, in every lane: within rows of 16 by DPP (neighbours,
// pairs, then the mirrored halves), the four rows through scalar registers.
template <int CTRL> __device__ __forceinline__ float dpp_add(float v) {
    const int t = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true);
    return v + __builtin_bit_cast(float, t);
}
__device__ __forceinline__ float lane_value(float v, int l) {
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0xb1>(v);    // quad_perm [1, 0, 3, 2]
    v = dpp_add<0x4e>(v);    // quad_perm [2, 3, 0, 1]
    v = dpp_add<0x141>(v);   // row_half_mirror
    v = dpp_add<0x140>(v);   // row_mirror
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// The sum over the W waves of a row, in a fixed order; `red` is a slot of its
// own for every sum of the kernel, so one barrier each is enough.
template <int W> __device__ __forceinline__ float row_sum(float v, float *red, int w) {
    v = wave_sum(v);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) red[w] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < W; ++i) v += red[i];
    }
    return v;
}

// The mean (layer norm) and the factor 1 / sqrt(power + eps) of a row whose
// lane's values are v[C][8], valid for n[c] elements of chunk c.
template <int W, int C>
__device__ __forceinline__ void row_stats(const float (&v)[C][8], const int (&n)[C], int kind,
                                          int d, float eps, float (*red)[W], int w, float *mean,
                                          float *factor) {
    float m = 0.f, s = 0.f;
    if (kind == LORA_NORM_LAYER) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[c][j];   // zeros past the row's end
        m = row_sum<W>(s, red[0], w) / float(d);
    }
    s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = v[c][j] - m;
            s += j < n[c] ? t * t : 0.f;
        }
    s = row_sum<W>(s, red[1], w);
    *mean = m;
    *factor = 1.0f / sqrtf(s / float(d) + eps);
}

__device__ __forceinline__ float gate_value(float g, int act) {
    if (act == LORA_GATE_SIGMOID) return 1.0f / (1.0f + expf(-g));
    if (act == LORA_GATE_TANH) return tanhf(g);
    return g;
}

template <typename T, typename S, int W, int C>
__global__ __launch_bounds__(W < 4 ? 256 : W * 64) void k_block_norm(const NormArgs a) {
    constexpr int ROWS = W < 4 ? 4 / W : 1;      // rows of a workgroup
    static_assert(W == 1 || ROWS == 1, "a barrier is for the waves of one row");
    __shared__ float red[4][W];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int w = wave % W;
    const int row = blockIdx.x * ROWS + wave / W;
    if (row >= a.T) return;                      // W == 1 only: no barrier is skipped

    const T *o = a.o ? static_cast<const T *>(a.o) + int64_t(row) * a.ldo : nullptr;
    const S *h = static_cast<const S *>(a.h) + int64_t(row) * a.ldh;
    const T *g = a.gate ? static_cast<const T *>(a.gate) + int64_t(row) * a.ldg : nullptr;
    const T *vec[4] = {static_cast<const T *>(a.post_w), static_cast<const T *>(a.post_b),
                       static_cast<const T *>(a.pre_w), static_cast<const T *>(a.pre_b)};
    const bool tail = a.d % 8 != 0;

    int at[C], n[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        at[c] = ((c * W + w) * 64 + lane) * 8;
        n[c] = min(max(a.d - at[c], 0), 8);
    }
    // The row itself first, then (rows of few chunks) the gate and the
    // vectors, all in flight together; wider rows read the vectors, and the
    // widest h, where they are used, to stay within the register budget.
    constexpr bool EARLY = C * sizeof(T) <= 4, LATE_H = C > 2;
    Row8<T> ro[C], rg[EARLY ? C : 1], rv[4][EARLY ? C : 1];
    Row8<S> rh[LATE_H ? 1 : C];
    auto load = [&](auto &r, const auto *p, int c) {
        r.zero();
        if (p) {
            if (n[c] == 8) r.load(p + at[c]);
            if (tail && n[c] > 0 && n[c] < 8) r.load_tail(p + at[c], n[c]);
        }
    };
#pragma unroll
    for (int c = 0; c < C; ++c) {
        load(ro[c], o, c);
        if constexpr (!LATE_H) load(rh[c], h, c);
    }
    if constexpr (EARLY) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            load(rg[c], g, c);
#pragma unroll
            for (int k = 0; k < 4; ++k) load(rv[k][c], vec[k], c);
        }
    }
    // weight (w + unit, or 1) and bias of element j, from vector pair k
    auto affine = [&](float v, const Row8<T> &wt, const Row8<T> &bs, int k, int j) {
        if (vec[k]) v *= wt.get(j) + a.unit;
        if (vec[k + 1]) v += bs.get(j);
        return v;
    };

    float v[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = ro[c].get(j);
    if (a.post != LORA_NORM_NONE) {
        float m, f;
        row_stats<W, C>(v, n, a.post, a.d, a.eps, &red[0], w, &m, &f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (!EARLY) {
                load(rv[0][0], vec[0], c);
                load(rv[1][0], vec[1], c);
            }
            constexpr int E = EARLY ? 1 : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[c][j] = affine((v[c][j] - m) * f, rv[0][c * E], rv[1][c * E], 0, j);
        }
    }
    S *ho = a.h_out ? static_cast<S *>(a.h_out) + int64_t(row) * a.ldho : nullptr;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if constexpr (LATE_H) load(rh[0], h, c);
        if (g) {
            if constexpr (!EARLY) load(rg[0], g, c);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] *= gate_value(rg[EARLY ? c : 0].get(j), a.gate_act);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = rh[LATE_H ? 0 : c].get(j) * a.beta;
            // elements past the row's end stay zero (they enter the mean)
            v[c][j] = j < n[c] ? (o ? t + v[c][j] * a.alpha : t) : 0.f;
        }
        if (ho && n[c] > 0) Row8<S>::store(ho + at[c], v[c], n[c]);
    }
    if (!a.u) return;
    T *u = static_cast<T *>(a.u) + int64_t(row) * a.ldu;
    float m, f;
    row_stats<W, C>(v, n, a.pre, a.d, a.eps, &red[2], w, &m, &f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if constexpr (!EARLY) {
            load(rv[2][0], vec[2], c);
            load(rv[3][0], vec[3], c);
        }
        constexpr int E = EARLY ? 1 : 0;
        float r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[j] = affine((v[c][j] - m) * f, rv[2][c * E], rv[3][c * E], 2, j);
        if (n[c] > 0) Row8<T>::store(u + at[c], r, n[c]);
    }
}

// Row r of a matrix of E at stride ld; no matrix has none.
template <typename E, typename P> P *from_row(P *p, int64_t r, int64_t ld) {
    return p ? reinterpret_cast<P *>(reinterpret_cast<uintptr_t>(p) + uint64_t(r * ld) * sizeof(E)) : p;
}

template <typename T, typename S, int W, int C>
hipError_t norm_launch(const NormArgs &a, hipStream_t s) {
    constexpr int ROWS = W < 4 ? 4 / W : 1, THREADS = W < 4 ? 256 : W * 64;
    // (a launch holds fewer than 2^32 threads)
    constexpr int64_t MOST = (int64_t(1) << 31) / THREADS * ROWS;
    for (int64_t r = 0; r < a.T; r += MOST) {
        NormArgs b = a;
        b.T = int32_t(std::min<int64_t>(a.T - r, MOST));
        b.h = from_row<S>(a.h, r, a.ldh);
        b.o = from_row<T>(a.o, r, a.ldo);
        b.gate = from_row<T>(a.gate, r, a.ldg);
        b.h_out = from_row<S>(a.h_out, r, a.ldho);
        b.u = from_row<T>(a.u, r, a.ldu);
        const dim3 grid((b.T + ROWS - 1) / ROWS), block(THREADS);
        hipLaunchKernelGGL((k_block_norm<T, S, W, C>), grid, block, 0, s, b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Waves a row and chunks a lane, by the row's width: narrow rows one wave,
// else as many waves as leave a lane one or two chunks.  16384 rows of 4096
// (bf16 blocks, float32 stream) take 138 us with 8 waves of one chunk and 144
// with 4 of two (5.8 and 5.6 TB/s).  float32 rows of 4097 to 5120 leave a
// third of 8 waves' second chunks idle: many of them go faster with 4 waves of
// four chunks, few of them, and wider ones, with 8 of two (us, layer norms with
// biases and gate rows, 4 of four against 8 of two: 1021 x 5003 29.4 and 30.6,
// 700 x 5120 22.4 and 23.9; but 512 x 5003 19.5 and 17.9, 64 x 5003 13.0 and
// 9.1, 4096 x 7000 128 and 120, 4096 x 8192 139 and 132; 16 of one are behind
// at each: 39.1, 28.4, 21.6, 8.5, 167 and 182).
template <typename T, typename S> hipError_t norm_types(const NormArgs &a, hipStream_t s) {
    const int lanes = (a.d + kNormChunk - 1) / kNormChunk;   // chunks of the row
    if (lanes <= 64) return norm_launch<T, S, 1, 1>(a, s);
    if (lanes <= 128) return norm_launch<T, S, 1, 2>(a, s);
    if (lanes <= 256) return norm_launch<T, S, 4, 1>(a, s);
    if (lanes <= 512) return norm_launch<T, S, 8, 1>(a, s);
    if constexpr (sizeof(T) == 4) {
        if (lanes <= 640 && a.T > 512) return norm_launch<T, S, 4, 4>(a, s);
    }
    if (lanes <= 1024) return norm_launch<T, S, 8, 2>(a, s);
    if (lanes <= 2048) return norm_launch<T, S, 16, 2>(a, s);
    return norm_launch<T, S, 16, 4>(a, s);
}

}  // namespace

hipError_t launch_block_norm(int dtype, int stream_dtype, const NormArgs &a, hipStream_t s) {
    if (a.T <= 0) return hipSuccess;
    if (a.d < 1 || a.d > kNormMaxWidth) return hipErrorInvalidValue;
    if (dtype == LORA_F32) return norm_types<float, float>(a, s);
    return stream_dtype == LORA_F32 ? norm_types<uint16_t, float>(a, s)
                                    : norm_types<uint16_t, uint16_t>(a, s);
}

}  // namespace lora
