// Launch interface between the C ABI (fq_ops_api.hip) and the kernels of the
// operators around the expert layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_internal.h"

namespace fq {

// Blocks of a launch whose number the call decides: HIP takes fewer than 2^32
// threads along x, so past GRID_X blocks they go on along z, and the last row of
// the grid may hold blocks past the end, which have nothing to do.
constexpr int64_t GRID_X = 1 << 20;
inline dim3 grid_of(int64_t blocks, unsigned y = 1) {
    return dim3((unsigned)(blocks < GRID_X ? blocks : GRID_X), y, (unsigned)((blocks + GRID_X - 1) / GRID_X));
}
__device__ __forceinline__ int64_t block_id() { return (int64_t)blockIdx.z * GRID_X + blockIdx.x; }

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

// ------------------------------------------------- the output layer's loss ---
struct HeadPlan {
    int pieces, vc;        // pieces of the vocabulary, entries per piece (a multiple of 256)
    int splits, ksplit;    // splits of a piece in the gradient's product, entries per split (of 64)
};
HeadPlan head_plan(int64_t T, int64_t H, int64_t V);
struct HeadArgs {
    int64_t T;
    int H;                 // a multiple of 64
    int64_t V;
    int k;                 // the teacher's ids per token, <= 64
    float lm_w, dist_w;
    const uint16_t* h;     // [T, H]
    const uint16_t* w;     // [V, H]
    const float* top_v;    // [T, k]
    const int32_t* top_i;
    const int32_t* labels; // nullable [T]
    float* row_loss;       // [T]
    uint16_t* grad;        // nullable [T, H]
    // workspace
    float* inv_n;          // [1]
    float* frame;          // [T]
    float* sum;            // [T]
    float* step;           // [T] power of two the last piece moved the frame by
    float* zs;             // [T, k + 1] logits of the teacher's ids and the label
    float2* stats;         // [vc / 64, T] sum and frame of each strip
    uint16_t* p;           // with grad: [T, vc]
    float* g;              // with grad: [splits, T, H]
    // filled per launch
    int64_t c0;
    int vc, splits, ksplit, first;
    int bm;                // tokens per tile of the two products, <= 256
};
hipError_t launch_head(HeadArgs a, const HeadPlan& pl, float* loss, hipStream_t st);

// ------------------------------------------------- packed 4-bit weights ---
constexpr int PACKED_MAX_ROWS = 1024;
struct PackedW {           // a stack of matrices as fq_tensor's codes
    const uint8_t* codes;  // two per byte, rows of K/2
    const uint8_t* bcodes; // NVFP4: E4M3 bytes per 16 columns, else null
    const float* scale;    // INT: spr per row
    const float* tscale;   // NVFP4: per matrix
    int K;                 // a multiple of 32
    int group;             // INT: columns per scale (at least 128 where one per row)
    int spr;               // INT: scales per row
    int b8;                // NVFP4: a chunk's block codes (8 bytes) are 8-byte aligned in every row
    int gshift;            // INT: chunk >> gshift (groups from 128), 32-column segment >> gshift (below) is its scale
};
struct MatvecArgs {
    PackedW w;
    int64_t N;             // rows of a matrix
    int E, M;
    const int32_t* which;  // nullable [M]: the matrix of each row of x
    const uint16_t* x;     // [M, K]
    uint16_t* y;           // [M, N]
};
hipError_t launch_matvec(const MatvecArgs& a, hipStream_t st);

struct PackedExpertArgs {
    PackedW w1, w2;        // [E, 2I, H], [E, H, I]
    ActQ a1, a2;
    int E, H, I, k, R;     // R = tokens * k <= PACKED_MAX_ROWS
    const uint16_t* x;     // [T, H]
    const int32_t* ids;    // [R]
    const float* tw;       // [R]
    uint16_t* y;           // [T, H]
    uint16_t* xhat;        // with an input quantiser: workspace [R, H], else null
    uint16_t* h;           // workspace [R, I]
    float* yr;             // workspace [R, H]
    int32_t* order;        // workspace [R]: rows by expert; null where every row is its own group
    int32_t* start;        // [R]
    int32_t* count;        // [R]
};
hipError_t launch_packed_expert(const PackedExpertArgs& a, hipStream_t st);

}  // namespace fq
