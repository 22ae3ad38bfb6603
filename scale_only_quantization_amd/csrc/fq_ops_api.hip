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

}  // extern "C"
