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
// the second product alone, of a piece: g = (first ? 0 : step g) + p w
hipError_t launch_head_grad(const HeadArgs& a, hipStream_t st);

// ------------------------------------------------ log probabilities of rows ---
constexpr int LOGP_MAX_TOP = 64;
constexpr int ROWS_TPB = 256;
// keys that a chunk of a row keeps for its k best
__host__ __device__ constexpr int rows_keys(int k) { return k > 32 ? 2 * k : 64; }
struct RowsArgs {          // rows of logits in chunks of columns, then joined
    int64_t T, V;
    int m, k;              // given tokens and alternatives per row
    const void* z;         // bf16 or fp32 logits [T, ld]
    int64_t ld;
    int64_t nc;            // chunks of a row
    float4* part;          // workspace [T, nc]: maximum, sum of e^(z - max), sum of e^(z - max) (z - max)
    uint64_t* keys;        // workspace [T, nc, rows_keys(k)], with k
    const int32_t* ids;    // [T, m]
    float* logp;
    float* lse;            // nullable
    float* entropy;        // nullable
    int32_t* top_ids;      // [T, k]
    float* top_logp;
};
struct LogpBwdArgs {       // dL/dz of rows of bf16 logits
    int64_t T, V;
    int m;
    const uint16_t* z;
    int64_t ld, gld;
    const int32_t* ids;
    const float* lse;
    const float* entropy;  // with dent
    const float* dlogp;    // [T, m]
    const float* dent;     // nullable
    uint16_t* grad;        // [T, gld]; may be z
};
int64_t rows_chunk(int64_t T, int64_t V);          // columns of a chunk of bf16 logits
hipError_t launch_logprob_rows(const RowsArgs& a, hipStream_t st);
hipError_t launch_logprob_bwd(const LogpBwdArgs& a, hipStream_t st);

struct HeadLogpArgs {
    int64_t T;
    int H;                 // a multiple of 64
    int64_t V;
    int m, k;
    const uint16_t* h;     // [T, H]
    const uint16_t* w;     // [V, H]
    const int32_t* ids;    // [T, m]
    float* lse;            // forward: nullable; backward: read
    float* entropy;        // forward: nullable; backward: read with dent
    float* logp;
    int32_t* top_ids;
    float* top_logp;
    const float* dlogp;    // backward
    const float* dent;     // nullable
    uint16_t* grad;        // [T, H]
    // workspace
    float* zs;             // [T, m] the given tokens' logits
    float* thr;            // forward [T]: the k-th best logit so far
    float4* run;           // forward [T]: maximum, s and u so far (frames of z itself); few tokens: of the chunks
    uint64_t* keys;        // few tokens: of the chunks
    float* best_z;         // forward [T, k]: the best so far
    int32_t* best_i;
    float2* stats;         // forward [vc / 64, T]: maximum m and s = sum e^(z - m) of each strip
    float* ustats;         // forward [vc / 64, T], with the entropy: u = sum e^(z - m) (z - m)
    float* z;              // forward [T, vc], with k: logits of a piece's strips above thr
    float4* rowc;          // backward [T]: lse, A + b entropy, b (0 of a row of masks); the one given id's bits or -1's
    uint16_t* p;           // backward [T, vc]
    float* g;              // backward [splits, T, H]
    float* ones;           // backward [T]
    // filled per launch
    int64_t c0;
    int vc, bm, first, last;
};
constexpr int LOGP_MAX_PIECE = 131072;
constexpr int FEW_BYTES = 132 * 1024, FEW_CHUNK = 4096;     // a few tokens: hidden states in LDS, columns of a chunk
inline int64_t head_few_ld(int64_t V) { return (V + 15) / 16 * 16; }
bool head_logp_few(int64_t T, int64_t H, int64_t V, int k);
struct HeadLogpPlan {
    int first, most;       // entries of the first piece and of the longest (multiples of 256)
    int round;             // of a round of tiles over the card
    int ld;                // of the longest piece that occurs
};
HeadLogpPlan head_logp_plan(int64_t T, int64_t H, int64_t V, int k);
hipError_t launch_head_logprob_fwd(HeadLogpArgs a, const HeadLogpPlan& pl, hipStream_t st);
hipError_t launch_head_logprob_bwd(HeadLogpArgs a, const HeadPlan& pl, hipStream_t st);

// ------------------------------------------------- the norm of many gradients ---
constexpr int GRAD_CHUNK = 16384;                  // elements per block
// A launch carries its tensors in its arguments, under 4 KB of them.  `count` has
// the type in its top bit (bf16: set); blk0 is a tensor's first block of the launch.
constexpr int64_t GRAD_BF16 = INT64_MIN;
struct GradSqArgs {
    static constexpr int LIST = 192;
    const void* g[LIST];
    int64_t count[LIST];
    uint32_t blk0[LIST];
    int n;
    uint32_t blocks;
    double* part;          // [blocks]
};
struct GradClipArgs {
    static constexpr int LIST = 136;
    const void* g[LIST];
    void* out[LIST];
    int64_t count[LIST];
    uint32_t blk0[LIST];
    int n;
    uint32_t blocks;
    const float* norm;
    double max_norm;
};
static_assert(sizeof(GradSqArgs) <= 4096 && sizeof(GradClipArgs) <= 4096, "kernel arguments");
hipError_t launch_grad_sq(const GradSqArgs& a, hipStream_t st);
hipError_t launch_grad_clip(const GradClipArgs& a, hipStream_t st);
// few tensors of few elements, and few in all, in one block: the norm itself (64 of
// 128: 3.5 us, 4.3 in two launches; 32 of 1024: 3.3 and 4.3; 64 of 1024: 4.7 and 4.3)
constexpr int GRAD_SMALL = 1024, GRAD_SMALL_LIST = 64, GRAD_SMALL_ALL = 32 * 1024;
hipError_t launch_grad_norm_small(const GradSqArgs& a, float* norm, hipStream_t st);
hipError_t launch_grad_norm(const double* part, int64_t n, float* norm, hipStream_t st);

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
