// Rotary positions on a batch's new queries and keys, and the new keys and
// values into the pages of their sequences.  With a_i = p f_i for the pair i
// of a head at position p:
//
//     x' = m (x cos a_i - y sin a_i),   y' = m (y cos a_i + x sin a_i),
//
// the pair being elements i and i + r / 2 (halves) or 2 i and 2 i + 1
// (interleaved) of a head's first r.  A position's angles are the same for all
// heads of a token, so a workgroup has a token: it forms them once, in 64 bits
// (a far position's angle has lost its fraction of a turn in 32: at 10^6 the
// first pair's by 0.06 radians) up to the fraction of a turn, whose sine and
// cosine are float32's, and every row of q, k and v is read and written once.
// HBM bounds it: 16384 tokens of 32 and 8 heads of 128, 403 MB, in 75 us (5.4
// TB/s; a copy of 1 GiB 5.16).
#include <hip/hip_runtime.h>

#include "attend_device.h"

namespace lora {
namespace {

constexpr int kThreads = 256;

// 8 consecutive elements, 16-byte aligned
template <typename T> struct Vec8;
template <> struct Vec8<uint16_t> {
    u32x4 r;
    __device__ __forceinline__ void load(const uint16_t *p) { r = *reinterpret_cast<const u32x4 *>(p); }
    __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<u32x4 *>(p) = r; }
    __device__ __forceinline__ float get(int j) const {
        return j % 2 ? bf16_hi(r[j / 2]) : bf16_lo(r[j / 2]);
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = bf16x2_rne(v[2 * j], v[2 * j + 1]);
    }
};
template <> struct Vec8<float> {
    f32x4 r[2];
    __device__ __forceinline__ void load(const float *p) {
        r[0] = reinterpret_cast<const f32x4 *>(p)[0];
        r[1] = reinterpret_cast<const f32x4 *>(p)[1];
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<f32x4 *>(p)[0] = r[0];
        reinterpret_cast<f32x4 *>(p)[1] = r[1];
    }
    __device__ __forceinline__ float get(int j) const { return r[j / 4][j % 4]; }
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j / 4][j % 4] = v[j];
    }
};
__device__ __forceinline__ float value(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ __forceinline__ float value(float v) { return v; }

enum RotaryItems : int {
    kHalves,     // pairs half the rotated part apart, whole vectors of each: 8 pairs
    kPairs,      // neighbours: a vector
    kOffset,     // halves that are not whole vectors: a vector, its elements'
                 // partners through LDS
};

// A thread reads and writes all of what it takes at a time, so that q may be
// rotated in place; kOffset has whole heads in LDS before it writes them.
// (16384 tokens of 40 heads, 90 elements of 128 rotated, us: halves 83, by 8
// unaligned pairs a thread 226, by single pairs 182; neighbours 74.)
template <typename T, int ITEMS>
__global__ __launch_bounds__(kThreads) void k_rotary(const RotaryArgs a) {
    __shared__ float2 turn[LORA_ATTN_MAX_HEAD_DIM / 2];   // (m cos, m sin) of every pair
    const int t = blockIdx.x, tid = threadIdx.x;
    const AttnToken tok = load_invariant(a.tokens + t);
    const int pairs = a.freqs ? a.rotary_dim / 2 : 0;
    if (tid < pairs) {
        const int pos = a.positions ? a.positions[t] : tok.pos;
        const double turns = double(pos) * a.freqs[tid] * 0.15915494309189533577;   // / 2 pi
        float s, c;
        sincospif(2.0f * float(turns - rint(turns)), &s, &c);
        turn[tid] = float2{a.magnitude * c, a.magnitude * s};
    }

    // the place of the token's key and value; none in a page that is none, or
    // where a replayed graph's sequence has fewer keys than new tokens now
    T *kc = nullptr, *vc = nullptr;
    if (a.cache.k && held(a.dbg, tok) && tok.pos >= 0) {
        const int p = tok.pos / a.cache.page_size, slot = tok.pos % a.cache.page_size;
        const int page = load_invariant(a.pages + int64_t(tok.seq) * a.ld_pages + p);
        if (page >= 0 && page < a.cache.num_pages) {
            kc = reinterpret_cast<T *>(a.cache.k) + int64_t(page) * a.cache.k_page +
                 int64_t(slot) * a.cache.k_tok;
            vc = reinterpret_cast<T *>(a.cache.v) + int64_t(page) * a.cache.v_page +
                 int64_t(slot) * a.cache.v_tok;
        }
    }
    const T *q = reinterpret_cast<const T *>(a.q) + int64_t(t) * a.ldq;
    const T *k = reinterpret_cast<const T *>(a.k) + int64_t(t) * a.ldk;
    const T *v = reinterpret_cast<const T *>(a.v) + int64_t(t) * a.ldv;
    T *qo = reinterpret_cast<T *>(a.q_out) + int64_t(t) * a.ldqo;

    const int vecs = a.head_dim / 8, first_k = a.q ? a.heads : 0;
    const int heads = first_k + (kc ? a.kv_heads : 0);
    const auto source = [&](int h) {
        return h < first_k ? q + int64_t(h) * a.head_dim : k + int64_t(h - first_k) * a.head_dim;
    };
    const auto target = [&](int h) {
        return h < first_k ? qo + int64_t(h) * a.head_dim
                           : kc + int64_t(h - first_k) * a.cache.k_head;
    };
    __syncthreads();
    if constexpr (ITEMS == kOffset) {
        __shared__ __align__(16) T staged[kThreads * 8];
        const int at_once = kThreads / vecs, mine = tid / vecs, e = tid % vecs * 8;
        for (int h0 = 0; h0 < heads; h0 += at_once) {
            const int h = h0 + mine;
            const bool ok = mine < at_once && h < heads;
            Vec8<T> x;
            if (ok) {
                x.load(source(h) + e);
                x.store(staged + tid * 8);
            }
            __syncthreads();
            if (ok && e < 2 * pairs) {
                const T *head = staged + tid * 8 - e;
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = e + j;
                    f[j] = x.get(j);
                    if (i >= 2 * pairs) continue;
                    const bool low = i < pairs;
                    const float2 cs = turn[low ? i : i - pairs];
                    const float z = value(head[low ? i + pairs : i - pairs]);
                    f[j] = low ? f[j] * cs.x - z * cs.y : f[j] * cs.x + z * cs.y;
                }
                x.set(f);
            }
            if (ok) x.store(target(h) + e);
            __syncthreads();
        }
    } else {
        const int turned = ITEMS == kHalves ? pairs / 8 : 0, items = vecs - turned;
        for (int i = tid; i < heads * items; i += kThreads) {
            const int h = i / items, e = i % items;
            const T *src = source(h);
            T *dst = target(h);
            Vec8<T> x;
            float f[8];
            if (ITEMS == kHalves && e < turned) {
                Vec8<T> y;
                x.load(src + e * 8);
                y.load(src + pairs + e * 8);
                float g[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 cs = turn[e * 8 + j];
                    f[j] = x.get(j) * cs.x - y.get(j) * cs.y;
                    g[j] = y.get(j) * cs.x + x.get(j) * cs.y;
                }
                x.set(f);
                y.set(g);
                x.store(dst + e * 8);
                y.store(dst + pairs + e * 8);
                continue;
            }
            const int at = (e + turned) * 8;             // (past both halves)
            x.load(src + at);
            if (ITEMS == kPairs && at < 2 * pairs) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    f[j] = x.get(j);
                    f[j + 1] = x.get(j + 1);
                    if (at + j >= 2 * pairs) continue;
                    const float2 cs = turn[at / 2 + j / 2];
                    f[j] = x.get(j) * cs.x - x.get(j + 1) * cs.y;
                    f[j + 1] = x.get(j + 1) * cs.x + x.get(j) * cs.y;
                }
                x.set(f);
            }
            x.store(dst + at);
        }
    }
    if (!vc) return;
    for (int i = tid; i < a.kv_heads * vecs; i += kThreads) {
        const int h = i / vecs, e = i % vecs;
        Vec8<T> x;
        x.load(v + int64_t(h) * a.head_dim + e * 8);
        x.store(vc + int64_t(h) * a.cache.v_head + e * 8);
    }
}

template <typename T> hipError_t rotary_types(const RotaryArgs &a, hipStream_t s) {
    const dim3 grid(a.T), block(kThreads);
    const int r = a.freqs ? a.rotary_dim : 0;
    if (a.layout == LORA_ROTARY_INTERLEAVED)
        hipLaunchKernelGGL((k_rotary<T, kPairs>), grid, block, 0, s, a);
    else if (r % 16 == 0)
        hipLaunchKernelGGL((k_rotary<T, kHalves>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_rotary<T, kOffset>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(int dtype, const RotaryArgs &a, hipStream_t s) {
    if (a.T <= 0) return hipSuccess;
    return dtype == LORA_F32 ? rotary_types<float>(a, s) : rotary_types<uint16_t>(a, s);
}

}  // namespace lora
