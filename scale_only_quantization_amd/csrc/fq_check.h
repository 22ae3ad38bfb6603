// Host-side argument checks shared by the C entry points.
#pragma once

#include "fq.h"
#include "fq_internal.h"

namespace fq {

// keeps the HIP error's text for fq_last_hip_error; returns FQ_E_HIP
int hip_fail(hipError_t e);

#define FQ_TRY(expr)                                       \
    do {                                                   \
        hipError_t _e = (expr);                            \
        if (_e != hipSuccess) return hip_fail(_e);         \
    } while (0)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }

// Resolve and check a quantiser descriptor.  Returns FQ_OK or an error.
inline int check_qdesc(const fq_qdesc* d, QParams* out) {
    if (!d) return FQ_E_INVALID;
    QParams q{};
    q.kind = d->kind;
    q.gran = d->gran;
    q.group = d->group;
    q.source = d->source;
    if (q.kind < FQ_NONE || q.kind > FQ_FP8E4M3) return FQ_E_INVALID;
    if (q.kind == FQ_NONE) {
        *out = q;
        return FQ_OK;
    }
    if (q.gran < FQ_PER_TENSOR || q.gran > FQ_PER_GROUP) return FQ_E_INVALID;
    if (q.source < FQ_LEARNABLE || q.source > FQ_DYNAMIC) return FQ_E_INVALID;
    if (q.kind == FQ_NVFP4) {
        if (q.gran != FQ_PER_GROUP || q.group != 16) return FQ_E_INVALID;
        q.qmin = -6.0f;
        q.qmax = 6.0f;
    } else if (q.kind == FQ_FP8E4M3) {
        q.qmin = -448.0f;
        q.qmax = 448.0f;
        q.qdiv = 448.0f;
    } else {
        if (d->qmin >= 0 || d->qmax <= 0 || d->qmin < -128 || d->qmax > 127) return FQ_E_INVALID;
        q.qmin = (float)d->qmin;
        q.qmax = (float)d->qmax;
        q.qdiv = (float)d->qmax;
    }
    if (q.gran == FQ_PER_GROUP) {
        if (!pow2(q.group) || q.group < 8 || q.group > 512) return FQ_E_INVALID;
    }
    if (q.gran == FQ_PER_TENSOR && q.source == FQ_DYNAMIC) return FQ_E_UNSUPPORTED;
    *out = q;
    return FQ_OK;
}

// Does the quantiser own a trainable tensor (one that can receive a gradient)?
inline bool has_param(const QParams& q) {
    if (q.kind == FQ_NVFP4) return q.source != FQ_STATIC;
    return q.kind != FQ_NONE && q.source == FQ_LEARNABLE;
}
// Does it read `scale` (the per-tensor/row/group or NVFP4 block scale)?
inline bool needs_scale(const QParams& q) { return q.kind != FQ_NONE && q.source != FQ_DYNAMIC; }
inline bool four_bit(const QParams& q) {
    return q.kind == FQ_NVFP4 || (q.kind == FQ_INT && q.qmax - q.qmin < 16.0f);
}

// ------------------------------------------------------------ layer checks --
struct LayerQ {
    QParams w1, w2, a1, a2;
};

inline int check_act(const QParams& a, int64_t width) {
    if (a.kind == FQ_NONE) return FQ_OK;
    if (a.kind == FQ_NVFP4) return a.source == FQ_DYNAMIC ? FQ_OK : FQ_E_UNSUPPORTED;
    if (a.source == FQ_DYNAMIC) {
        if (a.gran == FQ_PER_GROUP && width % a.group != 0) return FQ_E_SHAPE;
        return FQ_OK;                                  // per row / per group, on the fly
    }
    return a.gran == FQ_PER_TENSOR ? FQ_OK : FQ_E_UNSUPPORTED;   // per-expert scale
}

inline int check_layer(const fq_layer_desc* L, LayerQ* q) {
    if (!L) return FQ_E_INVALID;
    if (L->E < 1 || L->E > 1024 || L->H <= 0 || L->I <= 0 || L->T < 0) return FQ_E_SHAPE;
    if (L->topk < 1 || L->topk > 64 || L->topk > L->E) return FQ_E_SHAPE;
    if (L->H % 128 || L->I % 128) return FQ_E_SHAPE;
    if (L->H > 8192 || L->I > 8192) return FQ_E_UNSUPPORTED;
    if (L->T * L->topk >= (int64_t)1 << 31) return FQ_E_SHAPE;
    int s;
    if ((s = check_qdesc(&L->w1, &q->w1)) != FQ_OK) return s;
    if ((s = check_qdesc(&L->w2, &q->w2)) != FQ_OK) return s;
    if ((s = check_qdesc(&L->a1, &q->a1)) != FQ_OK) return s;
    if ((s = check_qdesc(&L->a2, &q->a2)) != FQ_OK) return s;
    if (q->w1.gran == FQ_PER_GROUP && L->H % q->w1.group) return FQ_E_SHAPE;
    if (q->w2.gran == FQ_PER_GROUP && L->I % q->w2.group) return FQ_E_SHAPE;
    if ((s = check_act(q->a1, L->H)) != FQ_OK) return s;
    if ((s = check_act(q->a2, L->I)) != FQ_OK) return s;
    return FQ_OK;
}

}  // namespace fq
