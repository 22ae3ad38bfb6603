// Launch interface between the C ABI (fq_ops_api.hip) and the kernels of the
// operators around the expert layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_internal.h"

namespace fq {

// --------------------------------------------------------------- RMS norm ---
struct NormArgs {
    QParams q;             // kind K_NONE: no codes
    int64_t rows;
    int cols;
    double eps;
    const uint16_t* x;
    const uint16_t* res;   // nullable
    const uint16_t* gamma;
    uint16_t* sum;         // bf16(x + res), with res
    uint16_t* y;           // nullable
    uint8_t* codes;        // with q
    float* scale;          // dynamic: written; else [1] read
    float* rstd;           // nullable
};
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st);

struct NormBwdArgs {
    int64_t rows;
    int cols;
    const uint16_t* s;
    const uint16_t* gamma;
    const float* rstd;
    const uint16_t* dy;
    const uint16_t* dsum;  // nullable
    uint16_t* dx;
    float* dgamma;         // nullable
    float* part;           // with dgamma: [norm_bwd_parts(rows, cols), cols]
};
int norm_bwd_parts(int64_t rows, int64_t cols);
hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st);
constexpr int NORM_MAX_COLS = 65536;

}  // namespace fq
