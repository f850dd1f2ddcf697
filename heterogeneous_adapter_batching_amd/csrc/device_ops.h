// Device building blocks shared by the gfx950 kernels: buffer resources and
// loads, bf16 conversion, the MFMA step on 16-byte fragments, the exact bf16
// split of a float32 operand.
//
// MFMA operand layout (16x16 output tile): lane l = 16 q + n holds row n of
// the left operand and column n of the right operand for the K-slice owned by
// lane group q; the 4 accumulators of lane l are output rows 4 q .. 4 q + 3 of
// column n.
#pragma once

#include <hip/hip_runtime.h>

#include "sgmv_internal.h"

namespace lora {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

template <typename T> struct Elem;
template <> struct Elem<uint16_t> { static constexpr int E = 8; };   // bf16 bit patterns
template <> struct Elem<float> { static constexpr int E = 4; };

// Buffer resources: raw (stride 0) with the byte size as the range.
constexpr uint32_t kOOB = 0x80000000u;        // offset of a masked lane: out of range
constexpr int kRsrcWord3 = 0x00020000;
// Non-temporal loads (early eviction from L2) for the shrink's A and the
// decode expand's B and y_in: each line is read whole by one instruction (the
// K-blocked A, the B block's row slices) and once; streaming B measured 2.7%
// faster per full-stack step and 5% on the multi-rank decode than the default
// policy, y_in 0.7% more on the full stack.  The shrink's partial sums keep
// the default policy (each is read by every unit of its block: 4.8% slower
// streamed).
// (While B rows were read 16 bytes a lane across 8 instructions the default
// policy was the faster one: the lines had to stay in L2 between the
// instructions.)  The prompt kernel reads B with the default policy: every
// token tile re-reads it from L2.
constexpr int kNT = 2;
// Outputs are stored at device scope (`sc1`, written through the L2): no
// dirty output lines are left for the kernel boundary to write back, which
// measured about 3% faster over the full stack than write-back stores.
constexpr int kOut = 16;

__device__ __forceinline__ rsrc_t make_rsrc(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, int(bytes),
                                             kRsrcWord3);
}
__device__ __forceinline__ uint32_t off_or_oob(bool ok, uint32_t off) { return ok ? off : kOOB; }

__device__ __forceinline__ u32x4 bload16(rsrc_t r, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, int(off), 0, 0);
}
__device__ __forceinline__ u32x4 bload16_nt(rsrc_t r, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, int(off), 0, kNT);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two floats -> packed bf16 bits (low half = a), rounded to nearest even by
// the hardware conversion (v_cvt_pk_bf16_f32); NaN stays NaN.
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <typename T> __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c);

template <> __device__ __forceinline__ f32x4 mma<uint16_t>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// float32: the four elements of a lane's fragment are four consecutive K
// indices; MFMA m takes element m of both operands, so both sides see the
// same K permutation.
template <> __device__ __forceinline__ f32x4 mma<float>(u32x4 a, u32x4 b, f32x4 c) {
    const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[0], fb[0], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[1], fb[1], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[2], fb[2], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[3], fb[3], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ int wave_id() {
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

__device__ __forceinline__ uint64_t extent(uint32_t lo, uint32_t hi) {
    return (uint64_t(hi) << 32) | lo;
}

// Reads plan memory (descriptors, token rows) through the constant address
// space, which promises that it stays unchanged for the whole dispatch: the
// plan workspace is written only by host uploads between launches, and the
// scalar cache is invalidated at each dispatch.  The dwords come in by
// scalar loads into SGPRs, so the unit's buffer resources are built in
// SGPRs (no loop around the buffer loads to make a VGPR descriptor
// uniform), and their wait counts apart from the vector loads.  3% per
// full-stack step against plain loads, which the compiler makes vector loads
// once a kernel may write memory.
template <typename D>
__device__ __forceinline__ D load_invariant(const D *p) {
    static_assert(sizeof(D) % 4 == 0, "whole dwords");
    typedef const __attribute__((address_space(4))) uint32_t *cptr;
    const cptr c = (cptr)p;
    D d;
    uint32_t *dst = reinterpret_cast<uint32_t *>(&d);
#pragma unroll
    for (int i = 0; i < int(sizeof(D) / 4); ++i) dst[i] = c[i];
    return d;
}

// Workgroup g runs on XCD g % kXcds; here each XCD takes one contiguous range
// of ceil(units / kXcds) units, in order.  For the MFMA expand, whose units
// run block by block (token slices, then projections and row chunks), the
// units that read one token tile's shrink partials then share an L2, and so
// do the blocks of one adapter, which read the same B rows: with units dealt
// round-robin, a tile's partials were fetched once per XCD its units ran on
// (the prefill q/k/v expand fetched 1.4x its bytes).  Indices past `units`
// (at most kXcds - 1 of them, on the last XCDs) are idle.
__device__ __forceinline__ int xcd_range_unit(int units) {
    const int g = blockIdx.x;
    return (g % kXcds) * ((units + kXcds - 1) / kXcds) + g / kXcds;
}

// Float offset of v entries (token slot `slot`, ranks j .. j + 3) of chunk 0
// in the shrink's partials, and the stride between chunks.  Unit u = (rank
// tile, chunk c, projection p) wrote tile u * ptt * 256: u = tile * nproj * c0
// + c * nproj + p, token slot s and rank i at s * 16 + i.
__device__ __forceinline__ uint32_t partial_off(int rt, int j, int slot, int p, int nproj, int c0,
                                                int ptt) {
    return uint32_t((rt + j / kTile) * nproj * c0 + p) * uint32_t(ptt * kTile * kTile) +
           uint32_t(slot * kTile + j % kTile);
}

// The whole chunk sum in the one order: the ways, then ((s0 + s1) + s2) + s3.
__device__ __forceinline__ f32x4 chunk_sum(rsrc_t pr, uint32_t off, uint32_t stride, int c0) {
    f32x4 w[kSumWays];
#pragma unroll
    for (int k = 0; k < kSumWays; ++k) w[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < c0; c += 8) {
        u32x4 part[8];
#pragma unroll
        for (int g = 0; g < 8; ++g)
            part[g] = bload16(pr, off_or_oob(c + g < c0, (off + uint32_t(c + g) * stride) * 4));
#pragma unroll
        for (int g = 0; g < 8; ++g)
            if (c + g < c0) w[g % kSumWays] += __builtin_bit_cast(f32x4, part[g]);
    }
    f32x4 s = w[0];
#pragma unroll
    for (int k = 1; k < kSumWays; ++k) s += w[k];
    return s;
}

// v operand of one K-step for one token: bf16 pieces (3, summing to v
// exactly) or the float32 values themselves.
template <typename T> struct VOperand;

template <> struct VOperand<uint16_t> {
    static constexpr int kPieces = 3;
    u32x4 piece[3];
    // v = h0 + h1 + h2 exactly: each residual is exact in float32 and the
    // three 8-bit significands cover float32's 24.  Inf/NaN keep no residual.
    __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = f[2 * i], b = f[2 * i + 1];
            const uint32_t w0 = bf16x2_rne(a, b);
            const float a1 = a - bf16_lo(w0), b1 = b - bf16_hi(w0);
            const uint32_t w1 = bf16x2_rne(a1, b1);
            const float a2 = a1 - bf16_lo(w1), b2 = b1 - bf16_hi(w1);
            uint32_t w2 = bf16x2_rne(a2, b2);
            uint32_t w1m = w1;
            if ((w0 & 0x7f80u) == 0x7f80u) { w1m &= 0xffff0000u; w2 &= 0xffff0000u; }
            if ((w0 & 0x7f800000u) == 0x7f800000u) { w1m &= 0xffffu; w2 &= 0xffffu; }
            piece[0][i] = w0;
            piece[1][i] = w1m;
            piece[2][i] = w2;
        }
    }
};

template <> struct VOperand<float> {
    static constexpr int kPieces = 1;
    u32x4 piece[1];
    __device__ __forceinline__ void set(const float (&f)[4]) {
        piece[0] = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]),
                         __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};

}  // namespace
}  // namespace lora
