// The global L2 norm of many gradients and the clipping by it: the joint
// clipping of a whole model's scales (the optim block's grad clip of the
// AngelSlim page, "Train from YAML"), whose tensors are more than one optimiser
// call takes.
//
//   norm = sqrt(sum g^2),  c = min(1, max / (norm + 1e-6)),  out = c g
//
// Each tensor is cut into chunks of GRAD_CHUNK elements, a block each; a launch
// carries the descriptors of its tensors in its arguments, so nothing is copied to
// the device first and a call can be captured.  k_grad_sq leaves a double per
// chunk, k_grad_norm adds them in a fixed order: no atomics, bitwise deterministic.
// Both passes are bound by HBM: 302 M fp32 elements are normed in 176 us (6.9 TB/s)
// and clipped in 437 (5.5 TB/s, read and write).  64 tensors of 128 take 11 us in
// the two calls, 311 of up to 60000 bf16 elements 31, six launches.
#include "fq_common.h"
#include "fq_ops.h"

namespace fq {
namespace {

constexpr int TPB = 256;

// 16 bytes at any element's address (the hardware splits what is not aligned)
typedef uint32_t words_any __attribute__((ext_vector_type(4), aligned(2)));

// The tensor of block b: the last whose first block is not past it.  One load of
// 64 entries at a time and a count (halving takes a dependent load per step).
template <typename ARGS>
__device__ __forceinline__ int find(const ARGS& a, uint32_t b) {
    const int lane = threadIdx.x & 63;
    int i = 0;
#pragma unroll
    for (int j = 0; j < ARGS::LIST; j += 64) {
        const int at = min(j + lane, ARGS::LIST - 1);
        i += __popcll(__ballot(j + lane < a.n && a.blk0[at] <= b));
    }
    return i - 1;
}
__device__ __forceinline__ int64_t length(int64_t count) { return count & ~GRAD_BF16; }

// what is read once, past the caches
__device__ __forceinline__ words_any load_once(const words_any* p) { return __builtin_nontemporal_load(p); }

template <int THREADS>
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double red[THREADS / WAVE];
#pragma unroll
    for (int m = 1; m < WAVE; m <<= 1) v += __shfl_xor(v, m);
    if ((threadIdx.x & (WAVE - 1)) == 0) red[threadIdx.x / WAVE] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / WAVE; ++w) t += red[w];
    return t;
}

__device__ __forceinline__ double sq_words(const words_any& w, bool bf) {
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (bf) {
            const double a = bf_lo(w[j]), b = bf_hi(w[j]);
            s += a * a + b * b;
        } else {
            const double a = __uint_as_float(w[j]);
            s += a * a;
        }
    }
    return s;
}

// sum of squares of elements [lo, hi) of a tensor, thread i of n
template <bool BF, int THREADS>
__device__ __forceinline__ double sq_range(const void* p, int64_t lo, int64_t hi) {
    constexpr int VEC = BF ? 8 : 4, SZ = BF ? 2 : 4;
    const char* g = static_cast<const char*>(p) + lo * SZ;
    const int n = (int)(hi - lo), nv = n / VEC;
    double acc = 0.0;
    int i = threadIdx.x % THREADS;
    for (; i + 3 * THREADS < nv; i += 4 * THREADS) {
        words_any w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = load_once(reinterpret_cast<const words_any*>(g) + i + u * THREADS);
#pragma unroll
        for (int u = 0; u < 4; ++u) acc += sq_words(w[u], BF);
    }
    for (; i < nv; i += THREADS) acc += sq_words(reinterpret_cast<const words_any*>(g)[i], BF);
    const int e = nv * VEC + threadIdx.x % THREADS;
    if (e < n) {
        const double x = BF ? bf_lo(reinterpret_cast<const uint16_t*>(g)[e]) : reinterpret_cast<const float*>(g)[e];
        acc += x * x;
    }
    return acc;
}

__global__ __launch_bounds__(TPB) void k_grad_sq(GradSqArgs a) {
    const uint32_t b = (uint32_t)block_id();
    if (b >= a.blocks) return;
    const int i = find(a, b);
    const int64_t lo = (int64_t)(b - a.blk0[i]) * GRAD_CHUNK, hi = min(lo + GRAD_CHUNK, length(a.count[i]));
    const double s = block_sum<TPB>(a.count[i] < 0 ? sq_range<true, TPB>(a.g[i], lo, hi)
                                                   : sq_range<false, TPB>(a.g[i], lo, hi));
    if (threadIdx.x == 0) a.part[b] = s;
}

// All tensors in one block, a wave per tensor in turn.
__global__ __launch_bounds__(1024) void k_grad_norm_small(GradSqArgs a, float* norm) {
    double acc = 0.0;
    for (int i = threadIdx.x / WAVE; i < a.n; i += 1024 / WAVE)
        acc += a.count[i] < 0 ? sq_range<true, WAVE>(a.g[i], 0, length(a.count[i]))
                              : sq_range<false, WAVE>(a.g[i], 0, length(a.count[i]));
    acc = block_sum<1024>(acc);
    if (threadIdx.x == 0) norm[0] = (float)sqrt(acc);
}

__global__ __launch_bounds__(1024) void k_grad_norm(const double* part, int64_t n, float* norm) {
    double acc = 0.0;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < n; i += 1024) acc += part[i];
    acc = block_sum<1024>(acc);
    if (threadIdx.x == 0) norm[0] = (float)sqrt(acc);
}

template <bool BF>
__device__ __forceinline__ void scale_range(const void* from, void* to, float c, int64_t lo, int64_t hi) {
    constexpr int VEC = BF ? 8 : 4, SZ = BF ? 2 : 4;
    const char* g = static_cast<const char*>(from) + lo * SZ;
    char* o = static_cast<char*>(to) + lo * SZ;
    const int n = (int)(hi - lo), nv = n / VEC;
    auto scaled = [&](words_any w) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = BF ? pack_bf16(bf_lo(w[j]) * c, bf_hi(w[j]) * c) : __float_as_uint(__uint_as_float(w[j]) * c);
        return w;
    };
    int i = threadIdx.x;
    for (; i + 3 * TPB < nv; i += 4 * TPB) {
        words_any w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = load_once(reinterpret_cast<const words_any*>(g) + i + u * TPB);
#pragma unroll
        for (int u = 0; u < 4; ++u) __builtin_nontemporal_store(scaled(w[u]), reinterpret_cast<words_any*>(o) + i + u * TPB);
    }
    for (; i < nv; i += TPB) reinterpret_cast<words_any*>(o)[i] = scaled(reinterpret_cast<const words_any*>(g)[i]);
    const int e = nv * VEC + threadIdx.x;
    if (e < n) {
        if (BF) {
            const float x = bf_lo(reinterpret_cast<const uint16_t*>(g)[e]) * c;
            reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)pack_bf16(x, x);
        } else {
            reinterpret_cast<float*>(o)[e] = reinterpret_cast<const float*>(g)[e] * c;
        }
    }
}

// From a tensor's last chunk to its first, as the tensors come: what the norm's
// pass read last may still be in the memory-side cache.  Loads and stores past the
// caches: 302 M elements in 437 us, 462 through them.
__global__ __launch_bounds__(TPB) void k_grad_clip(GradClipArgs a) {
    const uint32_t b = (uint32_t)block_id();
    if (b >= a.blocks) return;
    const double r = a.max_norm / ((double)a.norm[0] + 1.0e-6);
    const float c = r >= 1.0 ? 1.0f : (float)r;                // a NaN stays one
    const int i = find(a, b);
    if (c == 1.0f && a.g[i] == a.out[i]) return;
    const int64_t n = length(a.count[i]);
    const int64_t lo = ((n - 1) / GRAD_CHUNK - (b - a.blk0[i])) * GRAD_CHUNK, hi = min(lo + GRAD_CHUNK, n);
    if (a.count[i] < 0) scale_range<true>(a.g[i], a.out[i], c, lo, hi);
    else scale_range<false>(a.g[i], a.out[i], c, lo, hi);
}

}  // namespace

hipError_t launch_grad_sq(const GradSqArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(k_grad_sq, grid_of(a.blocks), dim3(TPB), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_grad_norm_small(const GradSqArgs& a, float* norm, hipStream_t st) {
    hipLaunchKernelGGL(k_grad_norm_small, dim3(1), dim3(1024), 0, st, a, norm);
    return hipGetLastError();
}

hipError_t launch_grad_norm(const double* part, int64_t n, float* norm, hipStream_t st) {
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(1024), 0, st, part, n, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const GradClipArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(k_grad_clip, grid_of(a.blocks), dim3(TPB), 0, st, a);
    return hipGetLastError();
}

}  // namespace fq
