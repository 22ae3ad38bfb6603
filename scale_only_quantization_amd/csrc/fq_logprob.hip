// Log probabilities of given tokens, entropy and the most likely tokens of rows
// of logits, and their gradient: from logits, and from hidden states and the
// frozen output weight.
//
//   lse = M + log s,  s = sum e^(z - M),  u = sum e^(z - M) (z - M)
//   logp_j = z_id - lse,  entropy = log s - u / s
//   dL/dz = sum_j a_j [v = id_j] - p (A + b (log p + entropy)),  A = sum_j a_j
//
// A row is cut into chunks that a block holds in registers (each logit is read
// once); a chunk leaves its maximum, s and u and its k best entries, and k_rows_join
// combines the chunks of a row.  An entry is a key of 64 bits, the logit's order
// above the id's complement: keys are distinct, and the largest key is the
// largest logit, the lowest id among equal ones, in whatever order keys are met.
#include "fq_head_product.h"
#include "fq_ops.h"

namespace fq {
namespace {

constexpr int TPB = ROWS_TPB;
constexpr float FLOOR = -200.0f;          // e^FLOOR is 0 in fp32: keeps 0 times -inf out of sums
constexpr float FLOOR2 = -300.0f;         // and 2^FLOOR2

__device__ __forceinline__ uint64_t key_of(float z, int64_t col) {
    const uint32_t b = __float_as_uint(z + 0.0f);                  // -0 counts as 0
    const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return ((uint64_t)o << 32) | (uint32_t)~(uint32_t)col;
}
__device__ __forceinline__ int32_t key_id(uint64_t key) { return (int32_t)~(uint32_t)key; }
__device__ __forceinline__ float key_z(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// The best keys of a block, in LDS: appended in any order, cut down to the k
// best by counting for each key how many are larger.
struct Best {
    static constexpr int CAP = 768;
    uint64_t key[CAP];
    uint64_t kth;          // keys below it cannot be among the k best
    int count;
    __device__ __forceinline__ void clear() {
        if (threadIdx.x == 0) {
            count = 0;
            kth = 1;                                               // 0 is no key
        }
        __syncthreads();
    }
    __device__ __forceinline__ void push(uint64_t x) {
        const int at = atomicAdd(&count, 1);
        if (at < CAP) key[at] = x;
    }
    // room for one more key per thread?  All threads call it, between their pushes.
    __device__ __forceinline__ bool full() {
        __syncthreads();
        const bool f = count > CAP - TPB;
        __syncthreads();
        return f;
    }
    // the k best in descending order at key[0 ..]; all threads call it
    __device__ void cut(int k) {
        __syncthreads();
        const int n = min(count, CAP);
        uint64_t mine[CAP / TPB];
        int rank[CAP / TPB];
#pragma unroll
        for (int q = 0; q < CAP / TPB; ++q) {
            mine[q] = (int)threadIdx.x + q * TPB < n ? key[threadIdx.x + q * TPB] : 0;
            rank[q] = 0;
        }
        for (int j = 0; j < n; ++j) {
            const uint64_t o = key[j];
#pragma unroll
            for (int q = 0; q < CAP / TPB; ++q) rank[q] += o > mine[q] ? 1 : 0;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < CAP / TPB; ++q)
            if (mine[q] != 0 && rank[q] < k) {
                key[rank[q]] = mine[q];
                if (rank[q] == k - 1) kth = mine[q];
            }
        if (threadIdx.x == 0) count = min(n, k);
        __syncthreads();
    }
};

// v of the wave's lanes in descending order
__device__ __forceinline__ float sorted(float v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int size = 2; size <= 64; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const float o = __shfl_xor(v, d);
            const bool larger = ((lane & size) == 0) == ((lane & d) == 0);
            v = larger ? fmaxf(v, o) : fminf(v, o);
        }
    return v;
}

// 16 bytes of a row as fp32
template <typename IN>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int N = 8;
    __device__ static __forceinline__ float get(const uint4& v, int e) {
        const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
        return (e & 1) ? bf_hi(w) : bf_lo(w);
    }
    __device__ static __forceinline__ uint4 nothing() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    // elements from n on are -inf
    __device__ static __forceinline__ uint4 cut(uint4 v, int64_t n) {
        auto two = [](uint32_t w, int64_t left) {
            return left >= 2 ? w : left == 1 ? (w & 0xffffu) | 0xff800000u : 0xff80ff80u;
        };
        return make_uint4(two(v.x, n), two(v.y, n - 2), two(v.z, n - 4), two(v.w, n - 6));
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ float get(const uint4& v, int e) {
        return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
    }
    __device__ static __forceinline__ uint4 nothing() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    __device__ static __forceinline__ uint4 cut(uint4 v, int64_t n) {
        return make_uint4(n > 0 ? v.x : 0xff800000u, n > 1 ? v.y : 0xff800000u, n > 2 ? v.z : 0xff800000u,
                          n > 3 ? v.w : 0xff800000u);
    }
};

// A chunk: NL vectors per thread.
template <typename IN, int NL>
__global__ __launch_bounds__(TPB) void k_rows_chunk(RowsArgs a) {
    constexpr int VEC = Vec<IN>::N, CH = NL * VEC * TPB;
    __shared__ Best best;
    __shared__ float red[3][TPB / 64];
    const int64_t b = block_id(), t = b / a.pc, c = b - t * a.pc;
    if (t >= a.T) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const IN* row = static_cast<const IN*>(a.z) + t * a.ld;
    const int64_t lo = c * CH;
    uint4 v[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int64_t col = lo + (int64_t)(i * TPB + threadIdx.x) * VEC;
        v[i] = col < a.n ? *reinterpret_cast<const uint4*>(row + col) : Vec<IN>::nothing();
    }
    if (lo + CH > a.n) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int64_t left = a.n - (lo + (int64_t)(i * TPB + threadIdx.x) * VEC);
            if (left < VEC) v[i] = Vec<IN>::cut(v[i], left);
        }
    }
    float tm = -INFINITY;
#pragma unroll
    for (int i = 0; i < NL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) tm = fmaxf(tm, Vec<IN>::get(v[i], e));
    const float wmax = wave_max(tm);
    // The chunk's k-th best is at least what k threads reach: with a quarter of
    // k threads in each wave, the least of the waves' values there.
    const float at = a.k > 0 ? __shfl(sorted(tm), (a.k + TPB / 64 - 1) / (TPB / 64) - 1) : 0.0f;
    if (lane == 0) {
        red[0][w] = wmax;
        red[1][w] = at;
    }
    if (a.k > 0) best.clear();
    __syncthreads();
    float M = red[0][0], thr = red[1][0];
#pragma unroll
    for (int i = 1; i < TPB / 64; ++i) {
        M = fmaxf(M, red[0][i]);
        thr = fminf(thr, red[1][i]);
    }
    if (a.k > 0) {
        auto each = [&](auto&& f) {
#pragma unroll
            for (int i = 0; i < NL; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float x = Vec<IN>::get(v[i], e);
                    f(x, x >= thr && x > -INFINITY, a.c0 + lo + (int64_t)(i * TPB + threadIdx.x) * VEC + e);
                }
        };
        each([&](float x, bool in, int64_t col) {
            if (in) best.push(key_of(x, col));
        });
        __syncthreads();
        if (best.count > Best::CAP) {                              // many equal ones: again, cut down on the way
            __syncthreads();
            best.clear();
            each([&](float x, bool in, int64_t col) {
                const uint64_t key = key_of(x, col);
                if (in && key >= best.kth) best.push(key);
                if (best.full()) best.cut(a.k);
            });
        }
        best.cut(a.k);
        uint64_t* out = a.keys + (t * a.nc + a.chunk0 + c) * a.k;
        if ((int)threadIdx.x < a.k) out[threadIdx.x] = (int)threadIdx.x < best.count ? best.key[threadIdx.x] : 0;
    }
    const float f = M == -INFINITY ? 0.0f : M;
    float s = 0.0f, u = 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float d = Vec<IN>::get(v[i], e) - f;
            const float x = exp2_hw(d * LOG2E);
            s += x;
            u = __builtin_fmaf(x, fmaxf(d, FLOOR), u);
        }
    s = wave_sum(s);
    u = wave_sum(u);
    __syncthreads();
    if (lane == 0) {
        red[0][w] = s;
        red[1][w] = u;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        s = red[0][0];
        u = red[1][0];
        for (int i = 1; i < TPB / 64; ++i) {
            s += red[0][i];
            u += red[1][i];
        }
        a.part[t * a.nc + a.chunk0 + c] = make_float4(M, s, u, 0.0f);
    }
}

// The chunks of a row.
__global__ __launch_bounds__(TPB) void k_rows_join(RowsArgs a) {
    __shared__ Best best;
    __shared__ float red[4][TPB / 64];
    __shared__ uint64_t floor_key[TPB / 64];
    const int64_t t = block_id();
    if (t >= a.T) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const float4* part = a.part + t * a.nc;
    float M = -INFINITY;
    for (int64_t i = threadIdx.x; i < a.nc; i += TPB) M = fmaxf(M, part[i].x);
    M = wave_max(M);
    if (lane == 0) red[0][w] = M;
    __syncthreads();
    for (int i = 0; i < TPB / 64; ++i) M = fmaxf(M, red[0][i]);
    const float f = M == -INFINITY ? 0.0f : M;
    float s = 0.0f, u = 0.0f;
    for (int64_t i = threadIdx.x; i < a.nc; i += TPB) {
        const float4 q = part[i];
        const float d = q.x - f, x = exp2_hw(d * LOG2E);
        s = __builtin_fmaf(q.y, x, s);
        u = __builtin_fmaf(__builtin_fmaf(fmaxf(d, FLOOR), q.y, q.z), x, u);
    }
    s = wave_sum(s);
    u = wave_sum(u);
    if (lane == 0) {
        red[1][w] = s;
        red[2][w] = u;
    }
    __syncthreads();
    s = red[1][0];
    u = red[2][0];
    for (int i = 1; i < TPB / 64; ++i) {
        s += red[1][i];
        u += red[2][i];
    }
    const bool none = M == -INFINITY && s == 0.0f;                 // every logit is -inf
    const float ls = logf(s), lse = none ? -INFINITY : f + ls;
    if (threadIdx.x == 0) {
        if (a.lse) a.lse[t] = lse;
        if (a.entropy) a.entropy[t] = none ? 0.0f : ls - u / s;
    }
    auto logp = [&](float z) {
        const float x = none ? -INFINITY : z - lse;
        return x > 0.0f ? 0.0f : x;
    };
    for (int j = threadIdx.x; j < a.m; j += TPB) {
        const int id = a.ids[t * a.m + j];
        float x = 0.0f;
        if (id >= 0 && id < a.V) {
            x = a.zs ? a.zs[t * a.m + j] : bf_from_bits(static_cast<const uint16_t*>(a.z)[t * a.ld + id]);
            x = logp(x);
        }
        a.logp[t * a.m + j] = x;
    }
    if (a.k == 0) return;
    // The row's k-th best is at least what k / nc entries of every chunk reach.
    const uint64_t* keys = a.keys + t * a.nc * a.k;
    const int64_t n = a.nc * a.k, share = (a.k + a.nc - 1) / a.nc;
    uint64_t least = ~0ull;
    for (int64_t i = threadIdx.x; i < a.nc; i += TPB) {
        const uint64_t x = keys[i * a.k + share - 1];
        least = x < least ? x : least;
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t o = __shfl_xor(least, m);
        least = o < least ? o : least;
    }
    if (lane == 0) floor_key[w] = least;
    best.clear();                                                  // its barrier orders floor_key
    for (int i = 0; i < TPB / 64; ++i) least = floor_key[i] < least ? floor_key[i] : least;
    for (int64_t i0 = 0; i0 < n; i0 += TPB) {
        const uint64_t x = i0 + threadIdx.x < n ? keys[i0 + threadIdx.x] : 0;
        if (x >= least && x >= best.kth) best.push(x);
        if (best.full()) best.cut(a.k);
    }
    best.cut(a.k);
    for (int j = threadIdx.x; j < a.k; j += TPB) {
        const bool there = j < best.count;
        a.top_ids[t * a.k + j] = there ? key_id(best.key[j]) : -1;
        a.top_logp[t * a.k + j] = there ? logp(key_z(best.key[j])) : -INFINITY;
    }
}

// dL/dz: a block has NB vectors per thread of a row; the given tokens' entries
// are formed after the others, from logits read before them (grad may be z).
constexpr int NB = 4;
__global__ __launch_bounds__(TPB) void k_logp_bwd(LogpBwdArgs a) {
    constexpr int CH = NB * 8 * TPB;
    __shared__ int sid[64];
    __shared__ float sa[64], sz[64];
    const int64_t chunks = (a.V + CH - 1) / CH;
    const int64_t b = block_id(), t = b / chunks, lo = (b - t * chunks) * CH;
    if (t >= a.T) return;
    const uint16_t* row = a.z + t * a.ld;
    if ((int)threadIdx.x < a.m) {
        const int id = a.ids[t * a.m + threadIdx.x];
        const bool in = id >= 0 && id < a.V;
        sid[threadIdx.x] = in ? id : -1;
        sa[threadIdx.x] = in ? a.dlogp[t * a.m + threadIdx.x] : 0.0f;
        sz[threadIdx.x] = in && id >= lo && id - lo < CH ? bf_from_bits(row[id]) : 0.0f;
    }
    __syncthreads();
    float A = 0.0f;
    for (int j = 0; j < a.m; ++j) A += sa[j];
    const float lse = a.lse[t];
    const float bb = a.dent ? a.dent[t] : 0.0f, H = a.dent ? a.entropy[t] : 0.0f;
    const bool none = lse == -INFINITY;
    auto grad = [&](float z) {
        const float lp = none ? FLOOR : fmaxf(z - lse, FLOOR);
        const float p = exp2_hw(lp * LOG2E);
        return -p * __builtin_fmaf(bb, lp + H, A);
    };
    uint16_t* out = a.grad + t * a.gld;
    uint4 v[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t col = lo + (int64_t)(i * TPB + threadIdx.x) * 8;
        if (col < a.V) v[i] = *reinterpret_cast<const uint4*>(row + col);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t col = lo + (int64_t)(i * TPB + threadIdx.x) * 8;
        if (col >= a.V) continue;
        float x[8];
        unpack8(v[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = grad(x[e]);
        if (col + 8 <= a.V) {
            *reinterpret_cast<uint4*>(out + col) = pack8(x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e < a.V) out[col + e] = (uint16_t)pack_bf16(x[e], x[e]);
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < a.m) {
        const int id = sid[threadIdx.x];
        if (id < lo || id - lo >= CH) return;
        float g = 0.0f;
        for (int j = 0; j < a.m; ++j) {
            if (sid[j] != id) continue;
            if (j < (int)threadIdx.x) return;                      // the first of equal ids has them all
            g += sa[j];
        }
        g = none ? 0.0f : g + grad(sz[threadIdx.x]);
        out[id] = (uint16_t)pack_bf16(g, g);
    }
}

}  // namespace

// A block's columns: 16384 of bf16, or 4096 where the rows are too few for the
// card's blocks.
int64_t rows_chunk(int64_t T, int64_t V) {
    return T * ((V + 16383) / 16384) >= 512 ? 16384 : 4096;
}

static hipError_t launch_join(const RowsArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(k_rows_join, grid_of(a.T), dim3(TPB), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_logprob_rows(const RowsArgs& a, hipStream_t st) {
    if (rows_chunk(a.T, a.V) == 16384)
        hipLaunchKernelGGL((k_rows_chunk<uint16_t, 8>), grid_of(a.T * a.pc), dim3(TPB), 0, st, a);
    else
        hipLaunchKernelGGL((k_rows_chunk<uint16_t, 2>), grid_of(a.T * a.pc), dim3(TPB), 0, st, a);
    const hipError_t err = hipGetLastError();
    return err != hipSuccess ? err : launch_join(a, st);
}

hipError_t launch_logprob_bwd(const LogpBwdArgs& a, hipStream_t st) {
    const int64_t chunks = (a.V + NB * 8 * TPB - 1) / (NB * 8 * TPB);
    hipLaunchKernelGGL(k_logp_bwd, grid_of(a.T * chunks), dim3(TPB), 0, st, a);
    return hipGetLastError();
}

// ---------------------------------------------------------- from hidden states --
namespace {

// Logits of the given tokens: a wave per token and slot.
__global__ __launch_bounds__(256) void k_logp_given(HeadLogpArgs a) {
    const int64_t i = block_id() * 4 + wave_id();
    if (i >= a.T * a.m) return;
    const int lane = threadIdx.x & 63;
    const int id = __builtin_amdgcn_readfirstlane(a.ids[i]);
    float acc = 0.0f;
    if (id >= 0 && id < a.V) {
        const uint4* hr = reinterpret_cast<const uint4*>(a.h + i / a.m * a.H);
        const uint4* wr = reinterpret_cast<const uint4*>(a.w + (int64_t)id * a.H);
        for (int c = lane; c < (a.H >> 3); c += 64) {
            float x[8], y[8];
            unpack8(hr[c], x);
            unpack8(wr[c], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc = __builtin_fmaf(x[e], y[e], acc);
        }
    }
    acc = wave_sum(acc);
    if (lane == 0) a.zs[i] = acc;
}

// The tile product of the output layer's loss with another epilogue: the
// forward stores the logits, the backward P = -p (A + b (log p + entropy)) in bf16.
template <bool BWD>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) void k_head_z(HeadLogpArgs a) {
    constexpr int ROWC = BWD ? BM * 16 : 0;
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM + 2 * ROWC];
    lds_t* smem = (lds_t*)smem_raw;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int wm = wave / WVN, wn = wave % WVN;
    const int mt = (int)((a.T + a.bm - 1) / a.bm), nt = a.vc / BN;
    const int wr = (a.bm / 2 + 31) / 32 * 32;
    const int run = (mt * nt + 7) / 8, per = gridDim.x / 8;
    const int t0 = (blockIdx.x & 7) * run + (blockIdx.x >> 3), t1 = min(mt * nt, ((int)(blockIdx.x & 7) + 1) * run);
    if (t0 >= t1) return;
    auto at = [&](int i, int64_t* m0, int* tn) {
        int tm;
        tile_of(t0 + i * per, mt, nt, &tm, tn);
        *m0 = (int64_t)tm * a.bm;
        return (int)min((int64_t)a.bm, a.T - *m0);
    };
    KT la, lb;
    la.init(u32x4{}, a.H);
    lb.init(u32x4{}, a.H);
    f32x16 acc[WTM][WTN];
    auto next = [&](int i) {
        int64_t m0;
        int tn;
        const int rows = at(i, &m0, &tn);
        const int64_t v0 = a.c0 + (int64_t)tn * BN;
        const int cols = (int)min((int64_t)BN, a.V - v0);
        la.rs = make_rsrc_words(a.h + m0 * a.H, (int64_t)rows * a.H * 2);
        lb.rs = make_rsrc_words(a.w + (cols > 0 ? v0 : 0) * a.H, (int64_t)cols * a.H * 2);
        if (BWD && wave < 4) {                                     // 64 rows' constants per wave
            const uint32_t voff[1] = {(uint32_t)(wave * 64 + lane) * 16};
            stage_loads<1, 0>(make_rsrc_words(a.rowc + m0, (int64_t)rows * 16),
                              smem + SMEM + (i & 1) * ROWC + wave * 1024, voff, 0);
        }
    };
    auto nti = [&](int i) {
        int64_t m0;
        int tn;
        const int rows = at(i, &m0, &tn);
        return wm == 0 ? (min(rows, wr) + 31) / 32 : (max(rows - wr, 0) + 31) / 32;
    };
    auto epilogue = [&](int i) {
        int64_t m0;
        int tn;
        const int rows = at(i, &m0, &tn), sub = nti(i);
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int cols = (int)min((int64_t)BN, a.V - a.c0 - (int64_t)tn * BN);
#pragma unroll
        for (int ti = 0; ti < WTM; ++ti) {
            if (ti >= sub) break;
            const int row = wm * wr + ti * 32 + (lane & 31);
            if (!BWD) {
                const __amdgpu_buffer_rsrc_t zrs = make_rsrc(a.z + m0 * a.vc + (int64_t)tn * BN,
                                                             (int64_t)(rows - 1) * a.vc * 4 + BN * 4);
#pragma unroll
                for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        u32x4 c;
#pragma unroll
                        for (int j = 0; j < 4; ++j) c[j] = __float_as_uint(acc[ti][tj][4 * q + j]);
                        const int col = wn * 64 + tj * 32 + 8 * q + 4 * (lane >> 5);
                        __builtin_amdgcn_raw_buffer_store_b128(c, zrs, (uint32_t)row * (uint32_t)a.vc * 4u + col * 4, 0, 0);
                    }
            } else {
                const __amdgpu_buffer_rsrc_t prs = make_rsrc(a.p + m0 * a.vc + (int64_t)tn * BN,
                                                             (int64_t)(rows - 1) * a.vc * 2 + BN * 2);
                const __attribute__((address_space(3))) float4* rc =
                    reinterpret_cast<const __attribute__((address_space(3))) float4*>(smem + SMEM + (i & 1) * ROWC);
                const float f = rc[row].x, c = rc[row].y, b = rc[row].z * LN2;
#pragma unroll
                for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const float l = fmaxf(__builtin_fmaf(acc[ti][tj][v], LOG2E, -f), FLOOR2);   // log2 p
                        acc[ti][tj][v] = -exp2_hw(l) * __builtin_fmaf(b, l, c);
                    }
                if (cols < BN) {                                   // columns past the vocabulary
#pragma unroll
                    for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (wn * 64 + tj * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3) >= cols)
                                acc[ti][tj][v] = 0.0f;
                }
#pragma unroll
                for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        u32x4 c4;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const auto r = __builtin_amdgcn_permlane32_swap(
                                pack_bf16(acc[ti][tj][4 * q + 2 * j], acc[ti][tj][4 * q + 2 * j + 1]),
                                pack_bf16(acc[ti][tj][4 * q + 4 + 2 * j], acc[ti][tj][4 * q + 5 + 2 * j]), false, false);
                            c4[j] = r[0];
                            c4[2 + j] = r[1];
                        }
                        const int col = wn * 64 + tj * 32 + 8 * (q + (lane >> 5));
                        __builtin_amdgcn_raw_buffer_store_b128(c4, prs, (uint32_t)row * (uint32_t)a.vc * 2u + col * 2, 0, 0);
                    }
            }
        }
    };
    product(la, lb, acc, smem, (t1 - t0 + per - 1) / per, a.H / BK, wr, next, nti, epilogue);
}

// Backward: a token's constants of the epilogue above.
__global__ __launch_bounds__(256) void k_logp_rowc(HeadLogpArgs a) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= a.T) return;
    float A = 0.0f;
    for (int j = 0; j < a.m; ++j) {
        const int id = a.ids[t * a.m + j];
        A += id >= 0 && id < a.V ? a.dlogp[t * a.m + j] : 0.0f;
    }
    const float b = a.dent ? a.dent[t] : 0.0f, H = a.dent ? a.entropy[t] : 0.0f;
    a.rowc[t] = make_float4(a.lse[t] * LOG2E, __builtin_fmaf(b, H, A), b, 0.0f);
    a.ones[t] = 1.0f;
}

// The given tokens' entries of P are zero: their share is added in fp32 at the end.
__global__ __launch_bounds__(256) void k_logp_clear(HeadLogpArgs a) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= a.T * a.m) return;
    const int id = a.ids[i];
    if (id >= a.c0 && id < a.V && id - a.c0 < a.vc) a.p[i / a.m * a.vc + (id - a.c0)] = 0;
}

// dh = sum of the splits + sum_j coef_j w_id_j: a block per token
__global__ __launch_bounds__(256) void k_logp_out(HeadLogpArgs a, int splits) {
    __shared__ int sid[64];
    __shared__ float scoef[64];
    const int64_t t = block_id();
    if (t >= a.T) return;
    if ((int)threadIdx.x < a.m) {
        const int j = threadIdx.x, id = a.ids[t * a.m + j];
        const bool in = id >= 0 && id < a.V;
        bool first = in;
        for (int l = 0; l < j; ++l) first &= a.ids[t * a.m + l] != id;
        const float4 rc = a.rowc[t];
        const float l = __builtin_fmaf(a.zs[t * a.m + j], LOG2E, -rc.x);
        sid[j] = in ? id : 0;
        scoef[j] = in ? a.dlogp[t * a.m + j] - (first ? exp2_hw(l) * __builtin_fmaf(rc.z * LN2, l, rc.y) : 0.0f) : 0.0f;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < (a.H >> 3); c += 256) {
        float o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int s = 0; s < splits; ++s) {
            const float4* g = reinterpret_cast<const float4*>(a.g + ((int64_t)s * a.T + t) * a.H) + 2 * c;
            const float4 x = g[0], y = g[1];
            o[0] += x.x; o[1] += x.y; o[2] += x.z; o[3] += x.w;
            o[4] += y.x; o[5] += y.y; o[6] += y.z; o[7] += y.w;
        }
        for (int j = 0; j < a.m; ++j) {
            float x[8];
            unpack8(reinterpret_cast<const uint4*>(a.w + (int64_t)sid[j] * a.H)[c], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __builtin_fmaf(scoef[j], x[e], o[e]);
        }
        reinterpret_cast<uint4*>(a.grad + t * a.H)[c] = pack8(o);
    }
}

// rows of a tile of the product, in whole sub-tiles and equal heights
int tile_rows(int64_t T) {
    const int64_t n = (T + BM - 1) / BM;
    return (int)(((T + n - 1) / n + 31) / 32 * 32);
}

unsigned product_grid(const HeadLogpArgs& a) {
    const int64_t mt = (a.T + a.bm - 1) / a.bm, tiles = (mt * (a.vc / BN) + 7) / 8 * 8;
    return (unsigned)(a.H % (2 * BK) == 0 && tiles > CUS ? CUS : tiles);
}

}  // namespace

HeadLogpPlan head_logp_plan(int64_t T, int64_t H, int64_t V) {
    HeadLogpPlan p{};
    constexpr int64_t CH = 16384;
    int64_t most = ((int64_t)640 << 20) / (4 * (T > 0 ? T : 1));
    if (most > ((int64_t)1 << 30) / H) most = ((int64_t)1 << 30) / H;
    most = most / BN * BN;
    if (most < BN) most = BN;
    p.vc = most < V ? most : (V + BN - 1) / BN * BN;
    p.pieces = (V + p.vc - 1) / p.vc;
    p.pc = (p.vc + CH - 1) / CH;
    p.nc = p.pc * p.pieces;
    return p;
}

hipError_t launch_head_logprob_fwd(HeadLogpArgs a, const HeadLogpPlan& pl, hipStream_t st) {
    a.bm = tile_rows(a.T);
    a.vc = (int)pl.vc;
    if (a.m > 0) hipLaunchKernelGGL(k_logp_given, grid_of((a.T * a.m + 3) / 4), dim3(256), 0, st, a);
    RowsArgs r{};
    r.T = a.T;
    r.V = a.V;
    r.m = a.m;
    r.k = a.k;
    r.z = a.z;
    r.ld = pl.vc;
    r.nc = pl.nc;
    r.pc = pl.pc;
    r.part = a.part;
    r.keys = a.keys;
    r.zs = a.zs;
    r.ids = a.ids;
    r.logp = a.logp;
    r.lse = a.lse;
    r.entropy = a.entropy;
    r.top_ids = a.top_ids;
    r.top_logp = a.top_logp;
    for (int64_t i = 0; i < pl.pieces; ++i) {
        a.c0 = r.c0 = i * pl.vc;
        r.n = a.V - r.c0 < pl.vc ? a.V - r.c0 : pl.vc;
        r.chunk0 = i * pl.pc;
        hipLaunchKernelGGL(k_head_z<false>, dim3(product_grid(a)), dim3(512), 0, st, a);
        hipLaunchKernelGGL((k_rows_chunk<float, 16>), grid_of(a.T * pl.pc), dim3(TPB), 0, st, r);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return launch_join(r, st);
}

hipError_t launch_head_logprob_bwd(HeadLogpArgs a, const HeadPlan& pl, hipStream_t st) {
    a.bm = tile_rows(a.T);
    a.vc = pl.vc;
    if (a.m > 0) hipLaunchKernelGGL(k_logp_given, grid_of((a.T * a.m + 3) / 4), dim3(256), 0, st, a);
    hipLaunchKernelGGL(k_logp_rowc, dim3((unsigned)((a.T + 255) / 256)), dim3(256), 0, st, a);
    HeadArgs g{};
    g.T = a.T;
    g.H = a.H;
    g.V = a.V;
    g.w = a.w;
    g.step = a.ones;
    g.p = a.p;
    g.g = a.g;
    g.vc = pl.vc;
    g.splits = pl.splits;
    g.ksplit = pl.ksplit;
    g.bm = a.bm;
    for (int i = 0; i < pl.pieces; ++i) {
        a.c0 = g.c0 = (int64_t)i * pl.vc;
        g.first = i == 0;
        hipLaunchKernelGGL(k_head_z<true>, dim3(product_grid(a)), dim3(512), 0, st, a);
        if (a.m > 0) hipLaunchKernelGGL(k_logp_clear, grid_of((a.T * a.m + 255) / 256), dim3(256), 0, st, a);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess || (err = launch_head_grad(g, st)) != hipSuccess) return err;
    }
    hipLaunchKernelGGL(k_logp_out, grid_of(a.T), dim3(256), 0, st, a, pl.splits);
    return hipGetLastError();
}

}  // namespace fq
