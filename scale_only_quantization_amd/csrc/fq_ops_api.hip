// C entry points of the operators around the expert layer (declarations and
// the documented contract are in include/fq.h): argument validation, always
// before any HIP call, and the launches.
#include <cmath>

#include "fq.h"
#include "fq_check.h"
#include "fq_ops.h"

using namespace fq;

extern "C" {

// ------------------------------------------------------------------ RMS norm --
static int check_norm(int64_t rows, int64_t cols) {
    if (rows < 0 || rows >= (int64_t)1 << 31 || cols < 8 || cols % 8) return FQ_E_SHAPE;
    return cols > NORM_MAX_COLS ? FQ_E_UNSUPPORTED : FQ_OK;
}

int fq_rms_norm_fwd(const fq_qdesc* q, int64_t rows, int64_t cols, double eps, const void* x, const void* residual,
                    const void* gamma, void* sum, void* y, float* rstd, uint8_t* codes, float* scale, void* stream) {
    NormArgs a{};
    int s;
    if (q && (s = check_qdesc(q, &a.q)) != FQ_OK) return s;
    if ((s = check_norm(rows, cols)) != FQ_OK) return s;
    if (!std::isfinite(eps) || eps < 0 || (residual && !sum) || (!residual && sum)) return FQ_E_INVALID;
    if (a.q.kind != FQ_NONE) {
        if (four_bit(a.q) || (a.q.gran != FQ_PER_TENSOR && a.q.source != FQ_DYNAMIC)) return FQ_E_UNSUPPORTED;
        if (a.q.gran == FQ_PER_GROUP && cols % a.q.group) return FQ_E_SHAPE;
        if (rows > 0 && (!codes || !scale)) return FQ_E_INVALID;
    } else if (codes || scale) {
        return FQ_E_INVALID;
    }
    if (rows > 0 && (!x || !gamma || (!y && !codes && !rstd && !sum))) return FQ_E_INVALID;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(sum, 16) || !aligned(y, 16) ||
        !aligned(codes, 8) || !aligned(scale, 4) || !aligned(rstd, 4))
        return FQ_E_ALIGN;
    if (rows == 0) return FQ_OK;
    a.rows = rows;
    a.cols = (int)cols;
    a.eps = eps;
    a.x = static_cast<const uint16_t*>(x);
    a.res = static_cast<const uint16_t*>(residual);
    a.gamma = static_cast<const uint16_t*>(gamma);
    a.sum = static_cast<uint16_t*>(sum);
    a.y = static_cast<uint16_t*>(y);
    a.codes = codes;
    a.scale = scale;
    a.rstd = rstd;
    FQ_TRY(launch_norm_fwd(a, static_cast<hipStream_t>(stream)));
    return FQ_OK;
}

size_t fq_rms_norm_bwd_workspace_size(int64_t rows, int64_t cols) {
    if (check_norm(rows, cols) != FQ_OK) return 0;
    return (size_t)norm_bwd_parts(rows, cols) * (size_t)cols * sizeof(float);
}

int fq_rms_norm_bwd(int64_t rows, int64_t cols, const void* s, const void* gamma, const float* rstd, const void* dy,
                    const void* dsum, void* dx, float* dgamma, void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_norm(rows, cols);
    if (st != FQ_OK) return st;
    if (rows > 0 && (!s || !gamma || !rstd || !dy || !dx)) return FQ_E_INVALID;
    if (!aligned(s, 16) || !aligned(gamma, 16) || !aligned(rstd, 4) || !aligned(dy, 16) || !aligned(dsum, 16) ||
        !aligned(dx, 16) || !aligned(dgamma, 4) || !aligned(workspace, 16))
        return FQ_E_ALIGN;
    const size_t need = dgamma ? fq_rms_norm_bwd_workspace_size(rows, cols) : 0;
    if (workspace_bytes < need || (need && !workspace)) return FQ_E_WORKSPACE;
    NormBwdArgs a{};
    a.rows = rows;
    a.cols = (int)cols;
    a.s = static_cast<const uint16_t*>(s);
    a.gamma = static_cast<const uint16_t*>(gamma);
    a.rstd = rstd;
    a.dy = static_cast<const uint16_t*>(dy);
    a.dsum = static_cast<const uint16_t*>(dsum);
    a.dx = static_cast<uint16_t*>(dx);
    a.dgamma = dgamma;
    a.part = static_cast<float*>(workspace);
    if (rows == 0 && !dgamma) return FQ_OK;
    FQ_TRY(launch_norm_bwd(a, static_cast<hipStream_t>(stream)));
    return FQ_OK;
}

// ---------------------------------------------------- the output layer's loss --
namespace {

struct HeadLayout {
    size_t inv_n, frame, sum, step, zs, rows, stats, p, g, total;
};

HeadLayout head_layout(const fq_head_desc* d, const HeadPlan& pl, bool grad) {
    HeadLayout y{};
    const size_t T = (size_t)d->tokens;
    size_t c = 0;
    auto place = [&](size_t& at, size_t bytes) {
        at = c;
        c = round_up(c + bytes, 256);
    };
    place(y.inv_n, 4);
    place(y.frame, T * 4);
    place(y.sum, T * 4);
    place(y.step, T * 4);
    place(y.zs, T * (size_t)(d->topk + 1) * 4);
    place(y.rows, T * 4);
    place(y.stats, (size_t)(pl.vc / 64) * T * 8);
    place(y.p, grad ? T * (size_t)pl.vc * 2 : 0);
    place(y.g, grad ? (size_t)pl.splits * T * (size_t)d->hidden * 4 : 0);
    y.total = c;
    return y;
}

int check_head(const fq_head_desc* d) {
    if (!d || !std::isfinite(d->lm_weight) || !std::isfinite(d->distill_weight)) return FQ_E_INVALID;
    if (d->topk < 0 || d->topk > 64 || d->topk > d->vocab) return FQ_E_INVALID;
    if (d->tokens < 0 || d->tokens >= (int64_t)1 << 24 || d->hidden < 64 || d->hidden % 64 || d->vocab < 1 ||
        d->vocab >= (int64_t)1 << 31)
        return FQ_E_SHAPE;
    return d->hidden > 16384 ? FQ_E_UNSUPPORTED : FQ_OK;
}

}  // namespace

size_t fq_head_loss_workspace_size(const fq_head_desc* d, int32_t with_grad) {
    if (check_head(d) != FQ_OK) return 0;
    return head_layout(d, head_plan(d->tokens, d->hidden, d->vocab), with_grad != 0).total;
}

int fq_head_loss(const fq_head_desc* d, const void* h, const void* w, const float* teacher_topk_logits,
                 const int32_t* teacher_topk_ids, const int32_t* labels, float* loss, float* row_loss, void* grad,
                 void* workspace, size_t workspace_bytes, void* stream) {
    const int s = check_head(d);
    if (s != FQ_OK) return s;
    if (!loss || (d->tokens > 0 && (!h || !w))) return FQ_E_INVALID;
    if (d->tokens > 0 && d->topk == 0 && !labels) return FQ_E_INVALID;        // no loss at all
    if (d->topk > 0 ? (d->tokens > 0 && (!teacher_topk_logits || !teacher_topk_ids))
                    : (teacher_topk_logits || teacher_topk_ids))
        return FQ_E_INVALID;
    if (!aligned(h, 16) || !aligned(w, 16) || !aligned(teacher_topk_logits, 4) || !aligned(teacher_topk_ids, 4) ||
        !aligned(labels, 4) || !aligned(loss, 4) || !aligned(row_loss, 4) || !aligned(grad, 16) ||
        !aligned(workspace, 256))
        return FQ_E_ALIGN;
    if (d->tokens == 0) {                                                     // the mean of nothing: no workspace
        FQ_TRY(launch_head(HeadArgs{}, HeadPlan{}, loss, static_cast<hipStream_t>(stream)));
        return FQ_OK;
    }
    const HeadPlan pl = head_plan(d->tokens, d->hidden, d->vocab);
    const HeadLayout y = head_layout(d, pl, grad != nullptr);
    if (!workspace || workspace_bytes < y.total) return FQ_E_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    HeadArgs a{};
    a.T = d->tokens;
    a.H = (int)d->hidden;
    a.V = d->vocab;
    a.k = d->topk;
    a.lm_w = d->lm_weight;
    a.dist_w = d->distill_weight;
    a.h = static_cast<const uint16_t*>(h);
    a.w = static_cast<const uint16_t*>(w);
    a.top_v = teacher_topk_logits;
    a.top_i = teacher_topk_ids;
    a.labels = labels;
    a.row_loss = row_loss ? row_loss : reinterpret_cast<float*>(ws + y.rows);
    a.grad = static_cast<uint16_t*>(grad);
    a.inv_n = reinterpret_cast<float*>(ws + y.inv_n);
    a.frame = reinterpret_cast<float*>(ws + y.frame);
    a.sum = reinterpret_cast<float*>(ws + y.sum);
    a.step = reinterpret_cast<float*>(ws + y.step);
    a.zs = reinterpret_cast<float*>(ws + y.zs);
    a.stats = reinterpret_cast<float2*>(ws + y.stats);
    a.p = grad ? reinterpret_cast<uint16_t*>(ws + y.p) : nullptr;
    a.g = grad ? reinterpret_cast<float*>(ws + y.g) : nullptr;
    FQ_TRY(launch_head(a, pl, loss, static_cast<hipStream_t>(stream)));
    return FQ_OK;
}

// ------------------------------------------------------ packed 4-bit weights --
namespace {

// The formats and row lengths of packed weights.
int check_packed_format(const QParams& q, int64_t cols) {
    if (!four_bit(q)) return FQ_E_UNSUPPORTED;
    if (q.kind == FQ_INT && (q.qmin < -8.0f || q.qmax > 7.0f || q.gran == FQ_PER_TENSOR ||
                             (q.gran == FQ_PER_GROUP && q.group < 32)))
        return FQ_E_UNSUPPORTED;
    if (cols < 32 || cols % 32 || (q.gran == FQ_PER_GROUP && cols % q.group)) return FQ_E_SHAPE;
    return cols > 65536 ? FQ_E_UNSUPPORTED : FQ_OK;
}

// The packed form of `batch` matrices [rows, cols] under quantiser d.
int check_packed(const fq_qdesc* d, int64_t cols, const uint8_t* codes, const uint8_t* block_codes, const float* scale,
                 const float* tensor_scale, PackedW* w) {
    QParams q;
    int s = check_qdesc(d, &q);
    if (s != FQ_OK || (s = check_packed_format(q, cols)) != FQ_OK) return s;
    if (!codes) return FQ_E_INVALID;
    if (q.kind == FQ_NVFP4 ? (!block_codes || !tensor_scale || scale) : (!scale || block_codes || tensor_scale))
        return FQ_E_INVALID;
    if (!aligned(codes, 16) || !aligned(block_codes, 2) || !aligned(scale, 4) || !aligned(tensor_scale, 4))
        return FQ_E_ALIGN;
    w->codes = codes;
    w->bcodes = block_codes;
    w->scale = scale;
    w->tscale = tensor_scale;
    w->K = (int)cols;
    w->group = q.gran == FQ_PER_GROUP ? q.group : (int)(cols > 128 ? cols : 128);
    w->spr = q.gran == FQ_PER_GROUP ? (int)(cols / q.group) : 1;
    w->b8 = cols % 128 == 0 && aligned(block_codes, 8);
    w->gshift = 30;
    if (q.gran == FQ_PER_GROUP)
        for (w->gshift = 0; (q.group < 128 ? 32 : 128) << w->gshift < q.group;) ++w->gshift;
    return FQ_OK;
}

struct PackedLayout {
    size_t xhat, h, yr, order, start, count, total;
};

// an input quantiser the packed layer has: none, NVFP4 with dynamic blocks, or one scale per expert
bool packed_act(const QParams& a) {
    return a.kind == FQ_NONE || a.kind == FQ_NVFP4 || (a.gran == FQ_PER_TENSOR && a.source != FQ_DYNAMIC);
}

int check_packed_layer(const fq_layer_desc* L, LayerQ* q) {
    int s = check_layer(L, q);
    if (s != FQ_OK || (s = check_packed_format(q->w1, L->H)) != FQ_OK ||
        (s = check_packed_format(q->w2, L->I)) != FQ_OK)
        return s;
    if (!packed_act(q->a1) || !packed_act(q->a2) || L->T * L->topk > PACKED_MAX_ROWS) return FQ_E_UNSUPPORTED;
    return FQ_OK;
}

PackedLayout packed_layout(const fq_layer_desc* L, const LayerQ& q) {
    PackedLayout y{};
    const size_t R = (size_t)(L->T * L->topk);
    size_t c = 0;
    auto place = [&](size_t& at, size_t bytes) {
        at = c;
        c = round_up(c + bytes, 256);
    };
    place(y.xhat, q.a1.kind != FQ_NONE ? R * (size_t)L->H * 2 : 0);
    place(y.h, R * (size_t)L->I * 2);
    place(y.yr, R * (size_t)L->H * 4);
    place(y.order, R * 4);
    place(y.start, R * 4);
    place(y.count, R * 4);
    y.total = c;
    return y;
}

}  // namespace

int fq_packed_matvec(const fq_qdesc* d, int64_t batch, int64_t rows, int64_t cols, const uint8_t* codes,
                     const uint8_t* block_codes, const float* scale, const float* tensor_scale, int64_t m,
                     const int32_t* which, const void* x, void* y, void* stream) {
    MatvecArgs a{};
    if (batch < 1 || batch >= (int64_t)1 << 31 || rows < 1 || rows >= (int64_t)1 << 31 || m < 0) return FQ_E_SHAPE;
    const int s = check_packed(d, cols, codes, block_codes, scale, tensor_scale, &a.w);
    if (s != FQ_OK) return s;
    if (m > PACKED_MAX_ROWS) return FQ_E_UNSUPPORTED;
    if ((batch > 1 && m > 0 && !which) || (m > 0 && (!x || !y))) return FQ_E_INVALID;
    if (!aligned(x, 16) || !aligned(y, 2) || !aligned(which, 4)) return FQ_E_ALIGN;
    if (m == 0) return FQ_OK;
    if (x == y) return FQ_E_INVALID;
    a.N = rows;
    a.E = (int)batch;
    a.M = (int)m;
    a.which = which;
    a.x = static_cast<const uint16_t*>(x);
    a.y = static_cast<uint16_t*>(y);
    FQ_TRY(launch_matvec(a, static_cast<hipStream_t>(stream)));
    return FQ_OK;
}

size_t fq_packed_expert_workspace_size(const fq_layer_desc* L) {
    LayerQ q;
    if (check_packed_layer(L, &q) != FQ_OK) return 0;
    return packed_layout(L, q).total;
}

int fq_packed_expert_fwd(const fq_layer_desc* L, const fq_packed_experts* P, const void* x, const int32_t* topk_ids,
                         const float* topk_w, void* y, void* workspace, size_t workspace_bytes, void* stream) {
    LayerQ q;
    int s = check_packed_layer(L, &q);
    if (s != FQ_OK) return s;
    if (!P) return FQ_E_INVALID;
    PackedExpertArgs a{};
    if ((s = check_packed(&L->w1, L->H, P->w1_codes, P->w1_block_codes, P->s_w1, P->t_w1, &a.w1)) != FQ_OK) return s;
    if ((s = check_packed(&L->w2, L->I, P->w2_codes, P->w2_block_codes, P->s_w2, P->t_w2, &a.w2)) != FQ_OK) return s;
    if ((q.a1.kind != FQ_NONE) != (P->s_a1 != nullptr) || (q.a2.kind != FQ_NONE) != (P->s_a2 != nullptr))
        return FQ_E_INVALID;
    if (L->T > 0 && (!x || !topk_ids || !topk_w || !y)) return FQ_E_INVALID;
    if (!aligned(P->s_a1, 4) || !aligned(P->s_a2, 4) || !aligned(x, 16) || !aligned(topk_ids, 4) ||
        !aligned(topk_w, 4) || !aligned(y, 16) || !aligned(workspace, 256))
        return FQ_E_ALIGN;
    const PackedLayout lay = packed_layout(L, q);
    if (L->T > 0 && (!workspace || workspace_bytes < lay.total)) return FQ_E_WORKSPACE;
    if (L->T == 0) return FQ_OK;
    if (x == y) return FQ_E_INVALID;
    char* ws = static_cast<char*>(workspace);
    a.a1 = ActQ{q.a1, P->s_a1};
    a.a2 = ActQ{q.a2, P->s_a2};
    a.E = (int)L->E;
    a.H = (int)L->H;
    a.I = (int)L->I;
    a.k = (int)L->topk;
    a.R = (int)(L->T * L->topk);
    a.x = static_cast<const uint16_t*>(x);
    a.ids = topk_ids;
    a.tw = topk_w;
    a.y = static_cast<uint16_t*>(y);
    a.xhat = q.a1.kind != FQ_NONE ? reinterpret_cast<uint16_t*>(ws + lay.xhat) : nullptr;
    a.h = reinterpret_cast<uint16_t*>(ws + lay.h);
    a.yr = reinterpret_cast<float*>(ws + lay.yr);
    if (L->T > 1) {
        a.order = reinterpret_cast<int32_t*>(ws + lay.order);
        a.start = reinterpret_cast<int32_t*>(ws + lay.start);
        a.count = reinterpret_cast<int32_t*>(ws + lay.count);
    }
    FQ_TRY(launch_packed_expert(a, static_cast<hipStream_t>(stream)));
    return FQ_OK;
}

}  // extern "C"
