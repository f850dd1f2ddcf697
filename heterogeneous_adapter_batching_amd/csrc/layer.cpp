// Host side of the operators around the delta: validation and launch geometry
// of block_norm.  Nothing is enqueued unless every argument holds.
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

}  // namespace

extern "C" {

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
