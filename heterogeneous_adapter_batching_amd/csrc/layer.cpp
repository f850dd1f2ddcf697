// Host side of the operators around the delta: validation and launch geometry
// of block_norm and frozen_linear.  Nothing is enqueued unless every argument
// holds.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <hip/hip_runtime.h>

#include "layer_internal.h"
#include "lora_sgmv.h"
#include "sgmv_internal.h"

using lora::set_errorf;

namespace {

int32_t esize(int32_t dtype) { return dtype == LORA_BF16 ? 2 : 4; }
bool is_dtype(int32_t d) { return d == LORA_F32 || d == LORA_BF16; }

// A matrix of `rows` rows of `width` elements at stride ld in memory.
struct Span {
    const char *name;
    const void *ptr;
    int64_t ld, width, rows;
    int32_t es;
    uint64_t lo() const { return reinterpret_cast<uintptr_t>(ptr); }
    uint64_t hi() const { return lo() + (uint64_t(rows - 1) * uint64_t(ld) + uint64_t(width)) * es; }
};

lora_status check_span(const Span &s) {
    if (!s.ptr) return set_errorf(LORA_EINVAL, "%s is null", s.name);
    if (s.lo() % uint64_t(s.es))
        return set_errorf(LORA_EINVAL, "%s is not aligned to its elements", s.name);
    if (s.rows > 1 && s.ld < s.width)
        return set_errorf(LORA_EINVAL, "ld of %s (%lld) is less than its width %lld", s.name,
                          (long long)s.ld, (long long)s.width);
    if (s.ld > (int64_t(1) << 40))
        return set_errorf(LORA_EINVAL, "ld of %s (%lld) is too large", s.name, (long long)s.ld);
    return LORA_OK;
}

// Whether two matrices share an element.  Column slices of one buffer (same
// stride, disjoint columns) do not.
bool overlap(const Span &a, const Span &b) {
    if (!a.ptr || !b.ptr || a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
    const uint64_t la = uint64_t(a.ld) * a.es, lb = uint64_t(b.ld) * b.es;
    if (a.rows > 1 && b.rows > 1 && la == lb) {
        const uint64_t wa = uint64_t(a.width) * a.es, wb = uint64_t(b.width) * b.es;
        // b's first column within a's rows of la bytes
        const uint64_t at = b.lo() >= a.lo() ? (b.lo() - a.lo()) % la
                                             : (la - (a.lo() - b.lo()) % la) % la;
        if (at >= wa && at + wb <= la) return false;
    }
    return true;
}

bool same(const Span &a, const Span &b) {
    return a.ptr == b.ptr && a.es == b.es && (a.ld == b.ld || (a.rows == 1 && b.rows == 1));
}

uint64_t round_up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

// Leading dimension of the partial products: whole 64-column groups, with
// room for the vector that starts at the last column.
int64_t partial_ld(int64_t wide) { return int64_t(round_up(uint64_t(wide) + 3, 64)); }

}  // namespace

namespace lora {

// What the plan of a product chooses from, and what it goes by: the time of
// one K tile (128 bytes of every row) of one workgroup with a CU to itself,
// and the stages that fill before the first.  bf16's are measured on MI355X
// with W from HBM (1024..28672 rows of W, K 4096 and 14336, 17..4096 tokens);
// float32's are what its nominal matrix rate gives (4096^3 estimated 898 us
// takes 1148, 512 x 4096 x 4096 112 and 150).  Small tiles cost little each and
// keep every CU busy; large ones read less per product.  Estimated and measured
// (bf16, us, without the launch): 128 x 4096 x 6144 in 2 parts of 128 x 64
// 23.0 and 21.5, in 4 of 128 x 128 23.1 and 23.4; 1024 x 4096 x 4096 in 2
// parts of 256 x 128 55 and 48, unsplit 128 x 128 58 and 49; 4096 x 4096 x
// 4096 256 x 256 99 and 102, 128 x 128 231 and 216.
struct TileCost {
    int bt, bn, waves, stages;
    float us[2];                 // float32, bf16 (0: not built)
};
constexpr TileCost kTiles[] = {
    {32, 64, 2, 4, {0.35f, 0.30f}},  {64, 128, 4, 4, {0.85f, 0.55f}},  {128, 64, 4, 4, {0.f, 0.52f}},
    {128, 128, 4, 4, {1.70f, 0.85f}}, {256, 128, 8, 3, {0.f, 0.95f}}, {256, 256, 8, 2, {0.f, 1.50f}}};
constexpr int kCus = 256;
// A launch more (the join), without what its sums take and what adapters add
// to it (it measures 4 to 5 us with the sums of 128 x 4096, 15 and 41 with the
// deltas of 68 adapters of rank 16 and 64 of ranks 8 to 64), and partial sums
// written and read at about this rate (TB/s = bytes / us / 1e6).
constexpr float kJoinUs = 2.5f, kPartialBytesPerUs = 3.5e6f;
// One K tile of a delta (a dependent step of a small batch of work).
constexpr float kDeltaTileUs = 0.6f;

namespace {

int k_tiles_of(int dtype, int k) {
    return int((int64_t(k) * esize(dtype) + kKBytes - 1) / kKBytes);
}
float rounds(int64_t units) { return float((units + kCus - 1) / kCus); }

struct Choice {
    LinearPlan pl{};
    float us = 0.f;
    void offer(float t, int bt, int bn, int splits, bool joined, int k_tiles) {
        if (us != 0.f && t >= us) return;
        us = t;
        pl = LinearPlan{kLinearTile, bt, bn, splits, k_tiles, joined, 0, 0};
    }
};

// The best single launch.  With adapters it also runs, for each token tile,
// the delta's K tiles: its groups, 3 pieces (bf16) of the largest rank's
// vectors in eights, once per half of a pair.
Choice direct(int dtype, int T, int n, int k, bool glu, int groups, int max_rpad) {
    Choice c;
    const int nk = k_tiles_of(dtype, k);
    const int per = ((dtype == LORA_BF16 ? 3 : 1) * max_rpad * esize(dtype) / 16 + 7) / 8;
    for (const TileCost &t : kTiles) {
        const float us = t.us[dtype == LORA_BF16 ? 1 : 0];
        if (us == 0.f || (!groups && !plain_tile(dtype, t.bt, t.bn))) continue;
        const int64_t tt = (int64_t(T) + t.bt - 1) / t.bt;
        const int feat = glu ? t.bn / 2 : t.bn;              // gate and up rows in pairs
        float one = float(nk + t.stages) * us;
        if (groups) one += (float(groups) / float(tt) + 1.f) * float(per * (glu ? 2 : 1)) * kDeltaTileUs;
        c.offer(rounds(tt * ((int64_t(n) + feat - 1) / feat)) * one, t.bt, t.bn, 1, false, nk);
    }
    return c;
}

// The best product in parts along K (from `least` parts on) joined by a launch.
Choice joined(int dtype, int T, int64_t wide, int k, int least) {
    Choice c;
    const int nk = k_tiles_of(dtype, k);
    for (const TileCost &t : kTiles) {
        const float us = t.us[dtype == LORA_BF16 ? 1 : 0];
        if (us == 0.f || !plain_tile(dtype, t.bt, t.bn)) continue;
        const int64_t tiles = (int64_t(T) + t.bt - 1) / t.bt * ((wide + t.bn - 1) / t.bn);
        for (int want = least; want <= 16; want = want < 4 ? want + 1 : want * 2) {
            const int kt = (nk + want - 1) / want;
            if (want > 1 && kt < 4) break;                   // too short to fill the pipeline
            const int splits = (nk + kt - 1) / kt;
            c.offer(rounds(tiles * splits) * float(kt + t.stages) * us + kJoinUs +
                        8.f * float(splits) * float(T) * float(wide) / kPartialBytesPerUs,
                    t.bt, t.bn, splits, true, kt);
        }
    }
    return c;
}

// Tokens with room for a tile's positions past the last in 32 bits.
constexpr int32_t kMostTokens = INT32_MAX - 1023;

// The threads of the plan's largest launch.
uint64_t launch_threads(const LinearPlan &pl, int64_t T, int64_t n, bool glu, int cols) {
    if (pl.kind == kLinearRows) {
        const uint64_t units = uint64_t((n + 15) / 16);
        return round_up(units, kXcds) * (units <= 128 ? 512 : 256);
    }
    int waves = 0;
    for (const TileCost &t : kTiles)
        if (t.bt == pl.bt && t.bn == pl.bn) waves = t.waves;
    // (see launch_linear)
    const int64_t feat = glu && !pl.joined ? pl.bn / 2 : pl.bn, rows = glu && pl.joined ? 2 * n : n;
    const uint64_t units = uint64_t((T + pl.bt - 1) / pl.bt) * uint64_t((rows + feat - 1) / feat) *
                           uint64_t(pl.splits);
    const uint64_t tiles = round_up(units, kXcds) * uint64_t(waves) * 64;
    if (!pl.joined) return tiles;
    return std::max(tiles, uint64_t((T + 15) / 16) * uint64_t((n + cols - 1) / cols) * 256);
}

uint64_t partial_bytes(int splits, int T, int64_t wide) {
    return round_up(4ull * uint64_t(splits) * uint64_t(T) * uint64_t(partial_ld(wide)), 256);
}

}  // namespace

LinearPlan linear_plan(int dtype, int T, int n, int k, bool glu, int groups, int max_rpad) {
    // A few tokens: W straight to registers, one launch.  Around 8 to 16
    // tokens it and the tile kernel meet (4096 x 4096: 11.4 us against 13.4
    // for one token, 14.1 against 14.0 for 16).
    LinearPlan pl{kLinearRows, 16, 16, 1, k_tiles_of(dtype, k), false, 0, 0};
    if (T <= kRowsTokens) {
        pl.threads = launch_threads(pl, T, n, glu, 0);
        return pl;
    }
    const int64_t wide = glu ? 2 * int64_t(n) : n;
    const Choice d = direct(dtype, T, n, k, glu, groups, max_rpad);
    const Choice j = joined(dtype, T, wide, k, groups ? 1 : 2);
    pl = j.us != 0.f && j.us < d.us ? j.pl : d.pl;
    pl.threads = launch_threads(pl, T, n, glu, join_cols(dtype, glu, groups ? max_rpad : 0));
    if (pl.joined) pl.ws_bytes = partial_bytes(pl.splits, T, wide);
    return pl;
}

uint64_t linear_ws_bound(int dtype, int T, int n, int k, bool glu, int max_groups, int max_rpad) {
    // (the one launch's time grows with the groups and their rank, the parts'
    // does not: the most of both tells whether any batch takes parts for its
    // adapters' sake)
    const uint64_t plain = linear_plan(dtype, T, n, k, glu, 0, 0).ws_bytes;
    const int groups = std::min(T, max_groups);
    return groups < 1 ? plain
                      : std::max(plain, linear_plan(dtype, T, n, k, glu, groups, max_rpad).ws_bytes);
}

lora_status check_linear_desc(const lora_linear_desc *d) {
    if (!d) return set_errorf(LORA_EINVAL, "null product descriptor");
    if (!is_dtype(d->dtype))
        return set_errorf(LORA_EDTYPE, "dtype %d is neither LORA_F32 nor LORA_BF16", d->dtype);
    if (d->num_tokens < 0 || d->num_tokens > kMostTokens)
        return set_errorf(LORA_EINVAL, "num_tokens %d not in 0..%d", d->num_tokens, kMostTokens);
    if (d->n < 1 || d->n > (1 << 28)) return set_errorf(LORA_EINVAL, "n %d not in 1..2^28", d->n);
    if (d->k < 8 || d->k % 8 || d->k > LORA_LINEAR_MAX_K)
        return set_errorf(LORA_EINVAL, "k %d is not a multiple of 8 in 8..%d", d->k,
                          LORA_LINEAR_MAX_K);
    if (d->act < LORA_ACT_NONE || d->act > LORA_ACT_GELU_TANH)
        return set_errorf(LORA_EINVAL, "act %d is not a lora_act", d->act);
    if (d->glu != 0 && d->glu != 1) return set_errorf(LORA_EINVAL, "glu %d is neither 0 nor 1", d->glu);
    // tiles are counted in 32 bits
    if (int64_t(d->num_tokens / 64 + 1) * (int64_t(d->n) * (1 + d->glu) / 64 + 1) > (1 << 30))
        return set_errorf(LORA_EINVAL, "a product of %d x %d outputs is too large", d->num_tokens,
                          d->n);
    return LORA_OK;
}

lora_status check_linear(const LinearCall &c, const LinearPlan &pl, uint64_t need) {
    const lora_linear_desc &d = *c.d;
    if (pl.threads >= (uint64_t(1) << 32))
        return set_errorf(LORA_EINVAL, "a product of %d tokens x %d outputs is more than a launch "
                          "holds: split it", d.num_tokens, d.n);
    const int32_t es = esize(d.dtype);
    const int64_t T = d.num_tokens, n = d.n, k = d.k, wide = n * (1 + d.glu);
    const Span x{"x", c.x, c.ldx, k, T, es}, w{"w", c.w, c.ldw, k, wide, es},
        b{"bias", c.bias, wide, wide, 1, es}, r{"residual", c.residual, c.ldr, n, T, es},
        y{"y", c.y, c.ldy, n, T, es};
    lora_status st;
    for (const Span *s : {&x, &w}) {
        if ((st = check_span(*s)) != LORA_OK) return st;
        if (s->lo() % 16) return set_errorf(LORA_EINVAL, "%s must be 16-byte aligned", s->name);
        if (s->ld < k || s->ld % 8 || s->ld > LORA_LINEAR_MAX_K)
            return set_errorf(LORA_EINVAL, "ld of %s (%lld) is not a multiple of 8 in k..%d",
                              s->name, (long long)s->ld, LORA_LINEAR_MAX_K);
    }
    if ((st = check_span(y)) != LORA_OK) return st;
    if (b.ptr && (st = check_span(b)) != LORA_OK) return st;
    if (r.ptr && (st = check_span(r)) != LORA_OK) return st;
    for (const Span *in : {&x, &w, &b})
        if (overlap(y, *in)) return set_errorf(LORA_EINVAL, "y overlaps %s", in->name);
    if (overlap(y, r) && !same(y, r))
        return set_errorf(LORA_EINVAL, "y overlaps residual without being it");
    if (need) {
        if (!c.ws || (reinterpret_cast<uintptr_t>(c.ws) & 255))
            return set_errorf(LORA_EINVAL, "the workspace must be non-null and 256-byte aligned");
        if (c.ws_bytes < need)
            return set_errorf(LORA_ESTATE, "workspace of %llu bytes < %llu needed",
                              (unsigned long long)c.ws_bytes, (unsigned long long)need);
        const Span ws{"the workspace", c.ws, int64_t(need), int64_t(need), 1, 1};
        for (const Span *s : {&x, &w, &b, &r, &y})
            if (overlap(ws, *s))
                return set_errorf(LORA_EINVAL, "the workspace overlaps %s", s->name);
    }
    return LORA_OK;
}

lora_status run_linear(const LinearCall &c, const LinearPlan &pl, void *partial,
                       const DeltaArgs &delta, hipStream_t s) {
    const lora_linear_desc &d = *c.d;
    LinearArgs a{};
    a.x = static_cast<const uint8_t *>(c.x);
    a.w = static_cast<const uint8_t *>(c.w);
    a.bias = static_cast<const uint8_t *>(c.bias);
    a.residual = static_cast<const uint8_t *>(c.residual);
    a.y = static_cast<uint8_t *>(c.y);
    a.partial = static_cast<float *>(partial);
    a.ldx = c.ldx;
    a.ldw = c.ldw;
    a.ldr = c.ldr;
    a.ldy = c.ldy;
    a.T = d.num_tokens;
    a.k = d.k;
    a.n = d.n;
    a.wide = d.n * (1 + d.glu);
    a.ldp = partial_ld(a.wide);
    a.act = d.act;
    a.delta = delta;
    const hipError_t e = launch_linear(d.dtype, pl, d.glu != 0, a, s);
    if (e != hipSuccess) return set_errorf(LORA_EHIP, "product launch: %s", hipGetErrorString(e));
    return LORA_OK;
}

}  // namespace lora

extern "C" {

uint64_t frozen_linear_workspace_bytes(const lora_linear_desc *d) {
    if (lora::check_linear_desc(d) != LORA_OK || d->num_tokens == 0) return 0;
    return lora::linear_plan(d->dtype, d->num_tokens, d->n, d->k, d->glu != 0, 0, 0).ws_bytes;
}

uint64_t frozen_linear_max_workspace_bytes(const lora_linear_desc *d) {
    if (lora::check_linear_desc(d) != LORA_OK) return 0;
    uint64_t most = 0;
    for (int64_t t = 1; t <= d->num_tokens; ++t)
        most = std::max(most, lora::linear_plan(d->dtype, int(t), d->n, d->k, d->glu != 0, 0, 0).ws_bytes);
    return most;
}

lora_status frozen_linear(const lora_linear_desc *d, const void *x, int64_t ldx, const void *w,
                          int64_t ldw, const void *bias, const void *residual, int64_t ldr,
                          void *y, int64_t ldy, void *ws, uint64_t ws_bytes, void *stream) {
    lora_status st = lora::check_linear_desc(d);
    if (st != LORA_OK) return st;
    if (d->num_tokens == 0) return LORA_OK;   // empty batch: no tensor is looked at
    const lora::LinearCall c{d, x, ldx, w, ldw, bias, residual, ldr, y, ldy, ws, ws_bytes};
    const lora::LinearPlan pl = lora::linear_plan(d->dtype, d->num_tokens, d->n, d->k, d->glu != 0, 0, 0);
    st = lora::check_linear(c, pl, pl.ws_bytes);
    if (st != LORA_OK) return st;
    return lora::run_linear(c, pl, ws, lora::DeltaArgs{}, static_cast<hipStream_t>(stream));
}

lora_status block_norm(const lora_norm_desc *d, const void *h, int64_t ldh, const void *o,
                       int64_t ldo, const void *post_weight, const void *post_bias,
                       const void *gate, int64_t ldg, const void *pre_weight,
                       const void *pre_bias, void *h_out, int64_t ldho, void *u, int64_t ldu,
                       void *stream) {
    if (!d) return set_errorf(LORA_EINVAL, "null norm descriptor");
    if (!is_dtype(d->dtype) || !is_dtype(d->stream_dtype))
        return set_errorf(LORA_EDTYPE, "dtype %d or stream_dtype %d is neither LORA_F32 nor "
                          "LORA_BF16", d->dtype, d->stream_dtype);
    if (d->stream_dtype != d->dtype && d->stream_dtype != LORA_F32)
        return set_errorf(LORA_EDTYPE, "the stream's dtype is the block's or LORA_F32");
    if (d->num_tokens < 0) return set_errorf(LORA_EINVAL, "num_tokens %d < 0", d->num_tokens);
    if (d->width < 1 || d->width > LORA_NORM_MAX_WIDTH)
        return set_errorf(LORA_EINVAL, "width %d not in 1..%d", d->width, LORA_NORM_MAX_WIDTH);
    for (int32_t k : {d->post, d->pre})
        if (k < LORA_NORM_NONE || k > LORA_NORM_LAYER)
            return set_errorf(LORA_EINVAL, "norm kind %d is not a lora_norm_kind", k);
    if (d->gate_act < LORA_GATE_NONE || d->gate_act > LORA_GATE_TANH)
        return set_errorf(LORA_EINVAL, "gate_act %d is not a lora_gate_act", d->gate_act);
    if (d->unit_offset != 0 && d->unit_offset != 1)
        return set_errorf(LORA_EINVAL, "unit_offset %d is neither 0 nor 1", d->unit_offset);
    if (!std::isfinite(d->alpha) || !std::isfinite(d->beta) || !std::isfinite(d->eps) || d->eps < 0)
        return set_errorf(LORA_EINVAL, "alpha, beta and eps must be finite, eps not negative");
    if (d->num_tokens == 0) return LORA_OK;   // empty batch: no tensor is looked at
    if (!o && (d->post != LORA_NORM_NONE || post_weight || post_bias || gate))
        return set_errorf(LORA_EINVAL, "a post norm or a gate without a block output");
    if (d->post == LORA_NORM_NONE && (post_weight || post_bias))
        return set_errorf(LORA_EINVAL, "a weight or bias without a post norm");
    if (d->pre == LORA_NORM_NONE && (pre_weight || pre_bias || u))
        return set_errorf(LORA_EINVAL, "a weight, bias or output without a pre norm");
    if (d->pre != LORA_NORM_NONE && !u) return set_errorf(LORA_EINVAL, "a pre norm without u");
    if (!h_out && !u) return set_errorf(LORA_EINVAL, "neither h_out nor u is given");

    const int32_t es = esize(d->dtype), hs = esize(d->stream_dtype);
    const int64_t T = d->num_tokens, w = d->width;
    const Span sh{"h", h, ldh, w, T, hs}, so{"o", o, ldo, w, T, es},
        sg{"gate", gate, ldg, w, ldg == 0 ? 1 : T, es}, sho{"h_out", h_out, ldho, w, T, hs},
        su{"u", u, ldu, w, T, es},
        vec[4] = {{"post_weight", post_weight, w, w, 1, es}, {"post_bias", post_bias, w, w, 1, es},
                  {"pre_weight", pre_weight, w, w, 1, es}, {"pre_bias", pre_bias, w, w, 1, es}};
    lora_status st = check_span(sh);
    if (st != LORA_OK) return st;
    for (const Span *s : {&so, &sg, &sho, &su, &vec[0], &vec[1], &vec[2], &vec[3]})
        if (s->ptr && (st = check_span(*s)) != LORA_OK) return st;
    if (overlap(sho, su)) return set_errorf(LORA_EINVAL, "h_out and u overlap");
    for (const Span *out : {&sho, &su}) {
        if (out->ptr && overlap(*out, sh) && !(out == &sho && same(*out, sh)))
            return set_errorf(LORA_EINVAL, "%s overlaps h", out->name);
        for (const Span *in : {&so, &sg, &vec[0], &vec[1], &vec[2], &vec[3]})
            if (overlap(*out, *in))
                return set_errorf(LORA_EINVAL, "%s overlaps %s", out->name, in->name);
    }

    lora::NormArgs a{};
    a.h = h;
    a.o = o;
    a.post_w = post_weight;
    a.post_b = post_bias;
    a.gate = gate;
    a.pre_w = pre_weight;
    a.pre_b = pre_bias;
    a.h_out = h_out;
    a.u = u;
    a.ldh = ldh;
    a.ldo = ldo;
    a.ldg = ldg;
    a.ldho = ldho;
    a.ldu = ldu;
    a.T = d->num_tokens;
    a.d = d->width;
    a.post = d->post;
    a.pre = d->pre;
    a.gate_act = d->gate_act;
    a.alpha = d->alpha;
    a.beta = d->beta;
    a.eps = d->eps;
    a.unit = float(d->unit_offset);
    const hipError_t e = lora::launch_block_norm(d->dtype, d->stream_dtype, a,
                                                 static_cast<hipStream_t>(stream));
    if (e != hipSuccess)
        return set_errorf(LORA_EHIP, "block norm launch: %s", hipGetErrorString(e));
    return LORA_OK;
}

}  // extern "C"
