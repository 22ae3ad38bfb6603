// RMS norm over the rows of a bf16 matrix with the residual's addition in
// front, optionally with its output in 8 bits and scales, and its gradient.
//
//   s = bf16(x + res),  r = 1 / sqrt(mean(s^2) + eps),  y = bf16(fl32(s g r))
//   codes = the 8-bit quantiser of y (the codes fq_tensor gives on y)
//   dx = dsum + r (g dy - s r^2 mean(g dy s)),  dg = sum over rows of dy s r
//
// A row stays in registers between its statistic and its output, so each
// element is read once and written once: HBM-bound for many rows, latency for
// few.  TPR threads share a row, NV vectors of 8 elements each.  2048 columns:
// 16384 rows with the residual's sum 51 us (5.25 TB/s; a large copy 4.95), their
// gradient with dgamma 55 us, 1893 rows with sum and float8 codes 10.8 us, one
// row 3.4 us in the kernel.
//
// y is the correctly rounded fp32 value of s g r, then bf16: the squares are
// summed in fp64 (exact products), r is held as two floats rh + rl, and with
// the exact p = s g (two 8-bit significands) fl32(p r) is p rh plus the
// product's own rounding error and p rl.  A y off by one fp32 ulp would land
// on the other side of a bf16 border once in 2^16 elements, and where that
// element is its row's or group's largest it would move the scale and with it
// every code; so the codes, scales and y equal those of the definition.
#include <type_traits>

#include "fq_act.h"
#include "fq_ops.h"

namespace fq {
namespace {

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int m = 1; m < WAVE; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// Sum (or maximum) over the TPR threads of a row, in a fixed order; every
// thread gets it.  red: one slot per wave; two barriers when TPR spans waves.
template <int TPR>
__device__ __forceinline__ double row_sum64(double v, double* red) {
    v = wave_sum64(v);
    if constexpr (TPR == WAVE) return v;
    if ((threadIdx.x & (WAVE - 1)) == 0) red[threadIdx.x / WAVE] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < TPR / WAVE; ++i) t += red[i];
    __syncthreads();
    return t;
}
template <int TPR, bool MAX>
__device__ __forceinline__ float row_red(float v, float* red) {
    v = MAX ? wave_max(v) : wave_sum(v);
    if constexpr (TPR == WAVE) return v;
    if ((threadIdx.x & (WAVE - 1)) == 0) red[threadIdx.x / WAVE] = v;
    __syncthreads();
    float t = red[0];
#pragma unroll
    for (int i = 1; i < TPR / WAVE; ++i) t = MAX ? fmaxf(t, red[i]) : t + red[i];
    __syncthreads();
    return t;
}

// fl32(p r) for r = rh + rl (see above); where p rh is not finite, that.  The
// sign is the product's, also of a zero.
__device__ __forceinline__ float mul_rr(float p, float rh, float rl) {
    const float yh = p * rh;
    const float y = yh + __builtin_fmaf(p, rl, __builtin_fmaf(p, rh, -yh));
    return fabsf(yh) < INFINITY ? __builtin_copysignf(y, yh) : yh;
}

constexpr int tpb(int tpr) { return tpr < 256 ? 256 : tpr; }

template <int TPR, int NV, int KIND>
__global__ __launch_bounds__(tpb(TPR)) void k_norm_fwd(NormArgs a) {
    __shared__ double red64[TPR / WAVE];
    __shared__ float red[TPR / WAVE];
    const int tid = threadIdx.x % TPR;
    const int64_t row = block_id() * (tpb(TPR) / TPR) + threadIdx.x / TPR;
    if (row >= a.rows) return;                     // whole waves; whole blocks where a row spans waves
    const int nvec = a.cols >> 3;
    const uint4* xr = reinterpret_cast<const uint4*>(a.x + row * a.cols);
    const uint4* gr = reinterpret_cast<const uint4*>(a.gamma);
    uint4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * TPR;
        v[i] = c < nvec ? xr[c] : make_uint4(0, 0, 0, 0);
    }
    if (a.res) {
        const uint4* rr = reinterpret_cast<const uint4*>(a.res + row * a.cols);
        uint4* sr = reinterpret_cast<uint4*>(a.sum + row * a.cols);
        uint4 w[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * TPR;
            w[i] = c < nvec ? rr[c] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * TPR;
            float f[8], g[8];
            unpack8(v[i], f);
            unpack8(w[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += g[j];
            v[i] = pack8(f);
            if (c < nvec) sr[c] = v[i];
        }
    }
    double s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            s0 = __builtin_fma((double)f[j], (double)f[j], s0);
            s1 = __builtin_fma((double)f[j + 1], (double)f[j + 1], s1);
        }
    }
    const double r = 1.0 / sqrt(row_sum64<TPR>(s0 + s1, red64) / (double)a.cols + a.eps);
    const float rh = (float)r, rl = (float)(r - (double)rh);
    if (a.rstd && tid == 0) a.rstd[row] = rh;
    float amax[NV], rmax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * TPR;
        float f[8], g[8];
        unpack8(v[i], f);
        unpack8(c < nvec ? gr[c] : make_uint4(0, 0, 0, 0), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = mul_rr(f[j] * g[j], rh, rl);
        v[i] = pack8(f);
        if (a.y && c < nvec) reinterpret_cast<uint4*>(a.y + row * a.cols)[c] = v[i];
        if (KIND != K_NONE) {
            unpack8(v[i], f);
            amax[i] = amax8(f);
            rmax = fmaxf(rmax, amax[i]);
        }
    }
    if constexpr (KIND != K_NONE) {
        const int gl = a.q.gran == G_GROUP ? a.q.group >> 3 : 1;
        float rs = 0.0f;
        if (a.q.gran == G_ROW) {
            rs = row_red<TPR, true>(rmax, red) / a.q.qdiv;
            if (tid == 0) a.scale[row] = rs;
        } else if (a.q.gran == G_TENSOR) {
            rs = a.scale[0];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * TPR;
            float sc = rs;
            if (a.q.gran == G_GROUP) {             // groups are whole and within a wave's 64 vectors
                sc = group_max(amax[i], gl) / a.q.qdiv;
                if (c < nvec && (c & (gl - 1)) == 0) a.scale[row * (nvec / gl) + c / gl] = sc;
            }
            float f[8];
            unpack8(v[i], f);
            uint32_t w[2] = {0u, 0u};
            quant_group<KIND, 8>(f, sc, a.q.qmin, a.q.qmax, [&](int j, const Elem& e) {
                w[j >> 2] |= (elem_code<KIND>(e, f[j]) & 0xFFu) << (8 * (j & 3));
            });
            if (c < nvec) reinterpret_cast<uint2*>(a.codes + row * a.cols)[c] = make_uint2(w[0], w[1]);
        }
    }
}

// One row per TPR threads at a time, rows dealt out in a fixed order; with DG
// each thread keeps its columns' sums of dy s r over its rows, the block adds
// its waves' sums in order and writes one partial row.
template <int TPR, int NV, bool DG>
__global__ __launch_bounds__(tpb(TPR)) void k_norm_bwd(NormBwdArgs a) {
    constexpr int RPB = tpb(TPR) / TPR;
    __shared__ float red[TPR / WAVE];
    __shared__ float dgs[DG && RPB > 1 ? TPR * NV * 8 : 1];
    const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int nvec = a.cols >> 3;
    uint4 gv[NV];
    float acc[DG ? NV : 1][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * TPR;
        gv[i] = c < nvec ? reinterpret_cast<const uint4*>(a.gamma)[c] : make_uint4(0, 0, 0, 0);
        if (DG)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    }
    const float inv_n = 1.0f / (float)a.cols;
    for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const uint4* sr = reinterpret_cast<const uint4*>(a.s + row * a.cols);
        const uint4* dr = reinterpret_cast<const uint4*>(a.dy + row * a.cols);
        uint4 sv[NV], dv[NV], ev[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * TPR;
            sv[i] = dv[i] = ev[i] = make_uint4(0, 0, 0, 0);
            if (c < nvec) {
                sv[i] = sr[c];
                dv[i] = dr[c];
                if (a.dsum) ev[i] = reinterpret_cast<const uint4*>(a.dsum + row * a.cols)[c];
            }
        }
        const float r = a.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float s[8], d[8], g[8];
            unpack8(sv[i], s);
            unpack8(dv[i], d);
            unpack8(gv[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dot = __builtin_fmaf(d[j] * g[j], s[j], dot);
                if (DG) acc[i][j] = __builtin_fmaf(d[j], s[j] * r, acc[i][j]);
            }
        }
        const float k = row_red<TPR, false>(dot, red) * inv_n * r * r;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * TPR;
            float s[8], d[8], g[8], e[8];
            unpack8(sv[i], s);
            unpack8(dv[i], d);
            unpack8(gv[i], g);
            unpack8(ev[i], e);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = __builtin_fmaf(__builtin_fmaf(-k, s[j], d[j] * g[j]), r, e[j]);
            if (c < nvec) reinterpret_cast<uint4*>(a.dx + row * a.cols)[c] = pack8(e);
        }
    }
    if constexpr (DG) {
        if constexpr (RPB > 1) {
            for (int w = 0; w < RPB; ++w) {
                if (sub == w)
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float* p = &dgs[(i * 8 + j) * TPR + tid];
                            acc[i][j] = w == 0 ? acc[i][j] : *p + acc[i][j];
                            *p = acc[i][j];
                        }
                __syncthreads();
            }
        }
        if (sub == RPB - 1)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * TPR;
                if (c < nvec) {
                    float4* o = reinterpret_cast<float4*>(a.part + (int64_t)blockIdx.x * a.cols + c * 8);
                    o[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                    o[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
                }
            }
    }
}

// dgamma[c] = sum of the partial rows: 64 columns per block, 16 threads per
// column taking every 16th partial, their sums added in order
__global__ __launch_bounds__(1024) void k_norm_dgamma(const float* part, int parts, int cols, float* out) {
    __shared__ float red[16][64];
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
    float acc = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int p = w; p < parts; p += 16) acc += part[(int64_t)p * cols + c];
    }
    red[w][threadIdx.x & 63] = acc;
    __syncthreads();
    if (w == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 16; ++i) acc += red[i][threadIdx.x];
        out[c] = acc;
    }
}

// Threads per row and vectors per thread: one wave per row up to 2048 columns
// from WAVE_ROWS rows on, else a block of 256 per row.  2048 columns, wave
// against block: forward to bf16 1024 rows 6.2 and 5.6 us, 4096 13.4 and 14.2;
// with float8 codes 1024 rows 8.5 and 6.9, 16384 58.5 and 59.6; backward with
// dgamma 1893 rows 14.0 and 12.3, 16384 56.0 and 62.8.
constexpr int64_t WAVE_ROWS = 2048;
template <typename F>
hipError_t by_shape(int64_t rows, int cols, F&& f) {
    const int nvec = cols >> 3;
    if (nvec <= 256 && rows >= WAVE_ROWS) {
        if (nvec <= 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
        if (nvec <= 128) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
        return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    }
    if (nvec <= 256) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    if (nvec <= 512) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    if (nvec <= 1024) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    if (nvec <= 2048) return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
    if (a.rows == 0) return hipSuccess;
    return by_shape(a.rows, a.cols, [&](auto tpr_c, auto nv_c) {
        constexpr int TPR = decltype(tpr_c)::value, NV = decltype(nv_c)::value;
        constexpr int RPB = tpb(TPR) / TPR;
        const dim3 grid = grid_of((a.rows + RPB - 1) / RPB), block(tpb(TPR));
        if (a.q.kind == K_NONE) hipLaunchKernelGGL((k_norm_fwd<TPR, NV, K_NONE>), grid, block, 0, st, a);
        else if (a.q.kind == K_INT) hipLaunchKernelGGL((k_norm_fwd<TPR, NV, K_INT>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_norm_fwd<TPR, NV, K_FP8>), grid, block, 0, st, a);
        return hipGetLastError();
    });
}

// blocks of the backward: with dgamma each writes one partial row
int norm_bwd_parts(int64_t rows, int64_t cols) {
    const int64_t rpb = cols <= 2048 && rows >= WAVE_ROWS ? 4 : 1;
    const int64_t b = (rows + rpb - 1) / rpb;
    return (int)(b < 512 ? b : 512);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st) {
    if (a.rows > 0) {
        const hipError_t err = by_shape(a.rows, a.cols, [&](auto tpr_c, auto nv_c) {
            constexpr int TPR = decltype(tpr_c)::value, NV = decltype(nv_c)::value;
            constexpr int RPB = tpb(TPR) / TPR;
            const int64_t blocks = (a.rows + RPB - 1) / RPB;
            if (a.dgamma)
                hipLaunchKernelGGL((k_norm_bwd<TPR, NV, true>), dim3((unsigned)norm_bwd_parts(a.rows, a.cols)),
                                   dim3(tpb(TPR)), 0, st, a);
            else
                hipLaunchKernelGGL((k_norm_bwd<TPR, NV, false>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)),
                                   dim3(tpb(TPR)), 0, st, a);
            return hipGetLastError();
        });
        if (err != hipSuccess) return err;
    }
    if (a.dgamma) {
        const int parts = a.rows > 0 ? norm_bwd_parts(a.rows, a.cols) : 0;   // no rows: zeros
        hipLaunchKernelGGL(k_norm_dgamma, dim3((unsigned)((a.cols + 63) / 64)), dim3(1024), 0, st, a.part, parts,
                           a.cols, a.dgamma);
    }
    return hipGetLastError();
}

}  // namespace fq
