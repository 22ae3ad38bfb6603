// The global L2 norm of many gradients and the clipping by it: the joint
// clipping of a whole model's scales (the optim block's grad clip of the
// AngelSlim page, "Train from YAML"), whose tensors are more than one optimiser
// call takes.
//
//   norm = sqrt(sum g^2),  c = min(1, max / (norm + 1e-6)),  out = c g
//
// Each tensor is cut into chunks of GRAD_CHUNK elements, a block each; a launch
// carries the descriptors of up to GRAD_LIST tensors in its arguments, so nothing
// is copied to the device first and a call can be captured.  k_grad_sq leaves a
// double per chunk, k_grad_norm adds them in a fixed order: no atomics, bitwise
// deterministic.  Both passes are bound by HBM.
#include "fq_common.h"
#include "fq_ops.h"

namespace fq {
namespace {

constexpr int TPB = 256;

// 16 bytes at any element's address (the hardware splits what is not aligned)
typedef uint32_t words_any __attribute__((ext_vector_type(4), aligned(2)));

// The tensor of block b: the last entry whose first block is not past it.
__device__ __forceinline__ int find(const GradArgs& a, int64_t b) {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.t[mid].blk0 <= b) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

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
    int i = threadIdx.x;
    for (; i + 3 * THREADS < nv; i += 4 * THREADS) {
        words_any w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = reinterpret_cast<const words_any*>(g)[i + u * THREADS];
#pragma unroll
        for (int u = 0; u < 4; ++u) acc += sq_words(w[u], BF);
    }
    for (; i < nv; i += THREADS) acc += sq_words(reinterpret_cast<const words_any*>(g)[i], BF);
    const int e = nv * VEC + threadIdx.x;
    if (e < n) {
        const double x = BF ? bf_lo(reinterpret_cast<const uint16_t*>(g)[e]) : reinterpret_cast<const float*>(g)[e];
        acc += x * x;
    }
    return acc;
}

__global__ __launch_bounds__(TPB) void k_grad_sq(GradArgs a) {
    const int64_t b = block_id();
    if (b >= a.blocks) return;
    const GradEntry& q = a.t[find(a, b)];
    const int64_t lo = (b - q.blk0) * GRAD_CHUNK, hi = min(lo + GRAD_CHUNK, q.count);
    const double s = block_sum<TPB>(q.bf ? sq_range<true, TPB>(q.g, lo, hi) : sq_range<false, TPB>(q.g, lo, hi));
    if (threadIdx.x == 0) a.part[b] = s;
}

__global__ __launch_bounds__(1024) void k_grad_norm(const double* part, int64_t n, float* norm) {
    double acc = 0.0;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < n; i += 1024) acc += part[i];
    acc = block_sum<1024>(acc);
    if (threadIdx.x == 0) norm[0] = (float)sqrt(acc);
}

template <bool BF>
__device__ __forceinline__ void scale_range(const GradEntry& q, float c, int64_t lo, int64_t hi) {
    constexpr int VEC = BF ? 8 : 4, SZ = BF ? 2 : 4;
    const char* g = static_cast<const char*>(q.g) + lo * SZ;
    char* o = static_cast<char*>(q.out) + lo * SZ;
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
        for (int u = 0; u < 4; ++u) w[u] = reinterpret_cast<const words_any*>(g)[i + u * TPB];
#pragma unroll
        for (int u = 0; u < 4; ++u) reinterpret_cast<words_any*>(o)[i + u * TPB] = scaled(w[u]);
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

__global__ __launch_bounds__(TPB) void k_grad_clip(GradArgs a) {
    const int64_t b = block_id();
    if (b >= a.blocks) return;
    const double r = a.max_norm / ((double)a.norm[0] + 1.0e-6);
    const float c = r >= 1.0 ? 1.0f : (float)r;                // a NaN stays one
    const GradEntry& q = a.t[find(a, b)];
    if (c == 1.0f && q.g == q.out) return;
    const int64_t lo = (b - q.blk0) * GRAD_CHUNK, hi = min(lo + GRAD_CHUNK, q.count);
    if (q.bf) scale_range<true>(q, c, lo, hi);
    else scale_range<false>(q, c, lo, hi);
}

}  // namespace

hipError_t launch_grad_sq(const GradArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(k_grad_sq, grid_of(a.blocks), dim3(TPB), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_grad_norm(const double* part, int64_t n, float* norm, hipStream_t st) {
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(1024), 0, st, part, n, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const GradArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(k_grad_clip, grid_of(a.blocks), dim3(TPB), 0, st, a);
    return hipGetLastError();
}

}  // namespace fq
