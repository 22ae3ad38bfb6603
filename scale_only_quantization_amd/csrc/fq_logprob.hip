// Log probabilities of given tokens, entropy and the most likely tokens of rows
// of logits, and their gradient: from logits, and from hidden states and the
// frozen output weight.
//
//   lse = M + log s,  s = sum e^(z - M),  u = sum e^(z - M) (z - M)
//   logp_j = z_id - lse,  entropy = log s - u / s
//   dL/dz = sum_j a_j [v = id_j] - p (A + b (log p + entropy)),  A = sum_j a_j
//
// A row is cut into chunks that a block holds in registers (each logit is read
// once); a chunk leaves its maximum, s and u and the entries that can be among the
// k best, and k_rows_join combines the chunks of a row.  An entry is a key of 64
// bits, the logit's order above the id's complement: keys are distinct, and the
// largest key is the largest logit, the lowest id among equal ones, in whatever
// order keys are met.
//
// From hidden states the logits z = h W^T come from
//   k_head_rows, k_head_few   a few tokens: the weight read once, fp32 logits, then
//       the kernels above on them
//   k_head_z   more: the output layer's tile product over pieces of the vocabulary,
//       whose epilogue leaves for a token's strips of 64 columns m, s and u, and
//       stores a strip's logits only where its maximum is above the k-th best of the
//       pieces before; k_logp_merge joins a piece's strips to the tokens' running
//       sums and alternatives.  In the backward it leaves dL/dz in bf16, which the
//       loss's second product multiplies with the weight.
// 16384 tokens of hidden 2048, 151936 entries, 64 alternatives: 8.0-8.7 ms, of
// which the products 7.5-7.6 (1340 to 1355 TFLOP/s; a library product of that size
// 1357 to 1398) and the 16 merges 0.75; 2048 tokens 1.05-1.10 ms; 333 x 1024 x 32003
// 42-48 us, one tile per CU, 34 in the product, whose two stages leave each load's
// latency bare.  The gradient of 2048 tokens 1.93-2.06 ms, half in each product.
#include <algorithm>

#include "fq_head_product.h"
#include "fq_ops.h"

namespace fq {
namespace {

constexpr int TPB = ROWS_TPB;
// Blocks of rows: a row's chunks along x, rows along y and, from ROWS_Y on, z.
constexpr int ROWS_Y = 32768;
dim3 rows_grid(int64_t chunks, int64_t T) {
    return dim3((unsigned)chunks, (unsigned)std::min<int64_t>(T, ROWS_Y), (unsigned)((T + ROWS_Y - 1) / ROWS_Y));
}
constexpr float FLOOR = -200.0f;          // e^FLOOR is 0 in fp32: keeps 0 times -inf out of sums
constexpr float FLOOR2 = -300.0f;         // and 2^FLOOR2
// A chunk's frame in base 2, f = M log2 e, is rounded by d, up to half an ulp of f,
// and the largest entry enters the sum as 2^d.  A correction to first order is as
// good as fp32 while (d ln 2)^2 / 2 is below half an ulp: d <= 2^-12, |M| < 2^12.
constexpr float FAR = 0x1p12f;
// A row whose lse is below it has nothing but masks: in the gradients p = e^(z - lse),
// and an fp32 number of that size no longer holds the log of their number beside
// them (each would have p = 1).
constexpr float MASKS = -0x1p20f;

// The order of a logit as a whole number: 0 is below all of them.
__device__ __forceinline__ uint32_t order_of(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);                  // -0 counts as 0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
constexpr uint32_t ORDER_MIN = 0x007fffffu;                        // the order of -inf
__device__ __forceinline__ uint64_t key_of(float z, int64_t col) {
    return ((uint64_t)order_of(z) << 32) | (uint32_t)~(uint32_t)col;
}
__device__ __forceinline__ int32_t key_id(uint64_t key) { return (int32_t)~(uint32_t)key; }
__device__ __forceinline__ float key_z(uint64_t key) { return value_of((uint32_t)(key >> 32)); }

// of s and u; a sum of one entry may be rounded below 1
__device__ __forceinline__ float entropy_of(float s, float u) {
    const float h = logf(s) - u / s;
    return h < 0.0f ? 0.0f : h;                                    // (a NaN stays one)
}

// lanes below this one in a mask, and `from`
__device__ __forceinline__ int lanes_before(uint64_t mask, int from) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, from));
}

// Wave reductions by moves inside the vector unit (row_shr 1, 2, 4, 8, then
// row_bcast 15 and 31; the last lane has the result), about a sixth of the time of
// an exchange through LDS at each of the six steps.  In a fixed order.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t x) {            // 0 where no lane is moved in
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, ROWS == 0xf);
}
__device__ __forceinline__ uint32_t wave_top(uint32_t x) {
    x = max(x, moved<0x111, 0xf>(x));
    x = max(x, moved<0x112, 0xf>(x));
    x = max(x, moved<0x114, 0xf>(x));
    x = max(x, moved<0x118, 0xf>(x));
    x = max(x, moved<0x142, 0xa>(x));
    x = max(x, moved<0x143, 0xc>(x));
    return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ float wave_total(float x) {
    auto add = [&](uint32_t y) { x += __uint_as_float(y); };
    add(moved<0x111, 0xf>(__float_as_uint(x)));
    add(moved<0x112, 0xf>(__float_as_uint(x)));
    add(moved<0x114, 0xf>(__float_as_uint(x)));
    add(moved<0x118, 0xf>(__float_as_uint(x)));
    add(moved<0x142, 0xa>(__float_as_uint(x)));
    add(moved<0x143, 0xc>(__float_as_uint(x)));
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 63));
}

// A bound that at least `want` of the wave's 64 N numbers reach, near the largest
// such: steps down from the largest, `top`, until enough reach it, then halves
// until an eighth more than `want` do, or 2^12 is left between the bounds.  Counting is one
// comparison and a population count of its mask, without the lanes' exchange
// that a sort needs (21 steps of two moves through LDS).
template <int N>
__device__ __forceinline__ uint32_t reached_by(const uint32_t (&o)[N], int want, uint32_t top) {
    auto count = [&](uint32_t x) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) c += __popcll(__ballot(o[i] >= x));
        return c;
    };
    uint32_t lo = top, hi = top, d = 1u << 20;
    int c = count(lo);
    while (c < want) {                                             // ends at 0, which all reach
        hi = lo;
        lo = lo > d ? lo - d : 0;
        d <<= 1;
        if (d == 0) lo = 0;
        c = count(lo);
    }
    while (c > want + (want >> 3) && hi - lo > (1u << 12)) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int n = count(mid);
        if (n >= want) {
            lo = mid;
            c = n;
        } else {
            hi = mid;
        }
    }
    return lo;
}

// 64 keys, one per lane: sorted in descending order (21 exchanges), and the 64
// largest of two such lists (7).
__device__ __forceinline__ uint64_t exchanged(uint64_t x, int d, bool larger) {
    const uint64_t o = __shfl_xor((unsigned long long)x, d);
    return (x > o) == larger ? x : o;
}
__device__ __forceinline__ uint64_t sorted_keys(uint64_t x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int size = 2; size <= 64; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) x = exchanged(x, d, ((lane & size) == 0) == ((lane & d) == 0));
    return x;
}
// `reversed` is the other list's key of lane 63 - lane
__device__ __forceinline__ uint64_t merged_keys(uint64_t x, uint64_t reversed) {
    const int lane = threadIdx.x & 63;
    x = x > reversed ? x : reversed;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = exchanged(x, d, (lane & d) == 0);
    return x;
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// The best keys of a block, in LDS: appended in any order, cut down to the k
// best by counting for each key how many are larger.
template <int N>
struct Best {
    static constexpr int CAP = 2 * N + 256;
    __attribute__((aligned(16))) uint64_t key[CAP];
    uint64_t kth;          // keys below it cannot be among the k best
    int count;
    // all threads call it; a barrier has to follow before the first push
    __device__ __forceinline__ void clear() {
        if (threadIdx.x == 0) {
            count = 0;
            kth = 1;                                               // 0 is no key
        }
    }
    __device__ __forceinline__ void push(bool in, uint64_t x) {
        if (!in) return;
        const int at = atomicAdd(&count, 1);
        if (at < CAP) key[at] = x;
    }
    // room for one more key per thread?  All threads call it, between their pushes.
    __device__ __forceinline__ bool full() {
        __syncthreads();
        const bool f = count > CAP - N;
        __syncthreads();
        return f;
    }
    template <int Q>
    __device__ __forceinline__ void rank(int n, int k) {
        uint64_t mine[Q];
        int r[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            mine[q] = (int)threadIdx.x + q * N < n ? key[threadIdx.x + q * N] : 0;
            r[q] = 0;
        }
        const int to = wave_id() * WAVE < n ? n : 0;               // a wave without keys has nothing to count
        int j = 0;
        for (; j + 8 <= to; j += 8) {
            uint64_t o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = key[j + e];
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int q = 0; q < Q; ++q) r[q] += o[e] > mine[q] ? 1 : 0;
        }
        for (; j < to; ++j) {
            const uint64_t o = key[j];
#pragma unroll
            for (int q = 0; q < Q; ++q) r[q] += o > mine[q] ? 1 : 0;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (mine[q] != 0 && r[q] < k) {
                key[r[q]] = mine[q];
                if (r[q] == k - 1) kth = mine[q];
            }
    }
    // the k best in descending order at key[0 ..]; all threads call it
    __device__ void cut(int k) {
        __syncthreads();
        const int n = min(count, CAP);
        if (n <= N) rank<1>(n, k);
        else rank<(CAP + N - 1) / N>(n, k);
        if (threadIdx.x == 0) count = min(n, k);
        __syncthreads();
    }
};

// 16 bytes of a row as fp32
template <typename IN>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int N = 8;
    __device__ static __forceinline__ float one(uint16_t x) { return bf_from_bits(x); }
    __device__ static __forceinline__ float get(const uint4& v, int e) {
        const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
        return (e & 1) ? bf_hi(w) : bf_lo(w);
    }
    // elements from n on are -inf
    __device__ static __forceinline__ uint4 cut(uint4 v, int n) {
        auto two = [](uint32_t w, int left) {
            return left >= 2 ? w : left == 1 ? (w & 0xffffu) | 0xff800000u : 0xff80ff80u;
        };
        return make_uint4(two(v.x, n), two(v.y, n - 2), two(v.z, n - 4), two(v.w, n - 6));
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ float one(float x) { return x; }
    __device__ static __forceinline__ float get(const uint4& v, int e) {
        return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
    }
    __device__ static __forceinline__ uint4 cut(uint4 v, int n) {
        return make_uint4(n > 0 ? v.x : 0xff800000u, n > 1 ? v.y : 0xff800000u, n > 2 ? v.z : 0xff800000u,
                          n > 3 ? v.w : 0xff800000u);
    }
};

// A barrier that orders LDS accesses and leaves loads in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A load of what is read once: 622 MB in whole stretches of memory arrive at 7.0
// TB/s so, at 6.2 through the caches.
__device__ __forceinline__ uint4 past_caches(const uint4* p) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

// The compiler is not to keep what it formed of these before: a second set of
// registers for a chunk's unpacked elements takes a third of the instructions away
// and half of a SIMD's waves (2048 rows of 151936: 171 us so, 125 with the words).
template <int N>
__device__ __forceinline__ void opaque(uint4 (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i].x), "+v"(v[i].y), "+v"(v[i].z), "+v"(v[i].w));
}

// A chunk: NL vectors per thread.  Its alternatives are the entries that reach a
// bound which k threads' maxima reach: about 75 of 16384 for k = 64, kept
// unsorted, at most rows_keys(k) of them.  Bound by the vector unit: 8 operations
// an element, one of them an exponential: 2048 rows of 151936 with 64 alternatives
// 110-120 us and 12.5 for the join, 98 without alternatives (with 512 threads and
// 32768 columns a block 9 more).  A chunk where more than rows_keys(k) entries reach
// the bound (all equal; finite masks with fewer than k entries above them; the end
// of a row with entries for fewer than k threads) reads itself again and cuts its
// list on the way: such rows throughout take 930-990 us, masks of -inf 110-120.
template <typename IN, int NL, bool ENT>
__global__ __launch_bounds__(TPB) void k_rows_chunk(RowsArgs a) {
    constexpr int VEC = Vec<IN>::N, THREADS = TPB, CH = NL * VEC * THREADS, WAVES = THREADS / 64;
    typedef Best<THREADS> Top;
    __shared__ Top best;
    __shared__ float red[2][WAVES];
    __shared__ uint32_t maxima[THREADS], bound;
    __shared__ int found[WAVES];
    const int64_t t = (int64_t)blockIdx.z * ROWS_Y + blockIdx.y, c = blockIdx.x;
    if (t >= a.T) return;
    const int lane = threadIdx.x & 63, w = wave_id();
    const IN* row = static_cast<const IN*>(a.z) + t * a.ld;
    const int64_t lo = c * CH;
    // all loads first: past the row's end a thread reads its last vector again
    const IN* src = row + lo;
    const int left = (int)min(a.V - lo, (int64_t)CH), end = (left - 1) / VEC * VEC;
    uint4 v[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i)
        v[i] = past_caches(reinterpret_cast<const uint4*>(src + min((i * THREADS + (int)threadIdx.x) * VEC, end)));
    if (left < CH) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int n = left - (i * THREADS + (int)threadIdx.x) * VEC;
            if (n < VEC) v[i] = Vec<IN>::cut(v[i], n);
        }
    }
    float tm = -INFINITY;
#pragma unroll
    for (int i = 0; i < NL * VEC; ++i) tm = fmaxf(tm, Vec<IN>::get(v[i / VEC], i % VEC));
    maxima[threadIdx.x] = order_of(tm);
    best.clear();
    __syncthreads();
    uint32_t o[WAVES], most = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        o[i] = maxima[lane + 64 * i];
        most = max(most, o[i]);
    }
    most = wave_top(most);
    const float M = value_of(most);
    if (a.k > 0 && w == 0) {                                       // the others go on to the sums
        const uint32_t r = reached_by(o, a.k, most);
        if (lane == 0) bound = r;
    }
    // the frame is M log2 e, rounded; its rounding d is taken off at the end.  Far from
    // 0 (a chunk of finite masks) the distance to M comes first, one operation more
    const float m = M == -INFINITY ? 0.0f : M;
    const bool far = fabsf(m) >= FAR;
    const float f = m * LOG2E, d = far ? 0.0f : __builtin_fmaf(m, LOG2E, -f);
    float s = 0.0f, u = 0.0f;
    auto add = [&](float l) {
        const float x = exp2_hw(l);
        s += x;
        if (ENT) u = __builtin_fmaf(x, fmaxf(l, FLOOR2), u);
    };
    opaque(v);
    if (far) {
#pragma unroll
        for (int i = 0; i < NL * VEC; ++i) add((Vec<IN>::get(v[i / VEC], i % VEC) - m) * LOG2E);
    } else {
#pragma unroll
        for (int i = 0; i < NL * VEC; ++i) add(__builtin_fmaf(Vec<IN>::get(v[i / VEC], i % VEC), LOG2E, -f));
    }
    s = wave_total(s);
    if (ENT) u = wave_total(u);
    if (lane == 0) {
        red[0][w] = s;
        red[1][w] = u;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        s = red[0][0];
        u = red[1][0];
        for (int i = 1; i < WAVES; ++i) {
            s += red[0][i];
            u += red[1][i];
        }
        // the terms are 2^l with l = (z - M) log2 e + d: both sums by 2^-d, and d off the second's l
        const float g = __builtin_fmaf(-d, LN2, 1.0f);
        a.part[t * a.nc + c] = make_float4(M, g * s, g * LN2 * __builtin_fmaf(-d, s, u), 0.0f);
    }
    if (a.k > 0) {
        const uint32_t r = bound;
        const float thr = r > ORDER_MIN ? value_of(r) : -0x1.fffffep+127f;   // -inf is no alternative
        // A wave's own part of the list, counted in a scalar: logit and column, of
        // which the key is formed at the end.  A part that overflows writes its
        // last place again and is not used.
        constexpr int PART = Top::CAP / WAVES;
        uint64_t* part = best.key + w * PART;
        int mine = 0;
        opaque(v);
#pragma unroll
        for (int i = 0; i < NL * VEC; ++i) {
            const float z = Vec<IN>::get(v[i / VEC], i % VEC);
            const bool in = z >= thr;
            const uint64_t mask = __ballot(in);
            if (mask != 0) {
                const int at = min(lanes_before(mask, mine), PART - 1);
                if (in)
                    part[at] = ((uint64_t)__float_as_uint(z) << 32) |
                               (uint32_t)((int)threadIdx.x * VEC + i / VEC * THREADS * VEC + i % VEC);
                mine += __popcll(mask);
            }
        }
        if (lane == 0) found[w] = mine;
        __syncthreads();
        const int cap = rows_keys(a.k);
        int total = 0, base = 0, most = 0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            base += i < w ? found[i] : 0;
            total += found[i];
            most = max(most, found[i]);
        }
        uint64_t* out = a.keys + (t * a.nc + c) * cap;
        if (total <= cap && most <= PART) {
            for (int i = lane; i < mine; i += 64)
                out[base + i] = key_of(__uint_as_float((uint32_t)(part[i] >> 32)), lo + (uint32_t)part[i]);
            for (int i = total + threadIdx.x; i < cap; i += THREADS) out[i] = 0;
        } else {                                                   // many equal ones: again, cut down on the way
            __syncthreads();
            for (int col = threadIdx.x; col < CH; col += THREADS) {
                const float x = col < left ? Vec<IN>::one(src[col]) : -INFINITY;
                const uint64_t key = key_of(x, lo + col);
                best.push(x >= thr && key >= best.kth, key);
                if (total > Top::CAP && best.full()) best.cut(a.k);
            }
            best.cut(a.k);
            for (int i = threadIdx.x; i < cap; i += THREADS) out[i] = i < best.count ? best.key[i] : 0;
        }
    }
}

// The chunks of a row.  Keys come in batches of 8 a thread, of which those are
// kept that reach a bound formed as in a chunk.
template <typename IN>
__global__ __launch_bounds__(TPB) void k_rows_join(RowsArgs a) {
    constexpr int WAVES = TPB / 64, PER = 8;
    typedef Best<TPB> Top;
    __shared__ Top best;
    __shared__ float red[3][WAVES];
    __shared__ uint32_t maxima[TPB];
    const int64_t t = block_id();
    if (t >= a.T) return;
    const int lane = threadIdx.x & 63, w = wave_id();
    // the first loads of everything that does not depend on another
    const float4* part = a.part + t * a.nc;
    float4 p0 = part[min((int64_t)threadIdx.x, a.nc - 1)];
    const int cap = a.k > 0 ? rows_keys(a.k) : 0;
    const int64_t n = a.nc * cap;
    const uint64_t* keys = a.keys + t * n;
    uint64_t x[PER];
    auto load = [&](int64_t i0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = keys[min(i0 + i * TPB + threadIdx.x, n - 1)];
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = i0 + i * TPB + threadIdx.x < n ? x[i] : 0;
    };
    if (a.k > 0) load(0);
    const int id = (int)threadIdx.x < a.m ? a.ids[t * a.m + threadIdx.x] : -1;
    const bool given = id >= 0 && id < a.V;
    if ((int64_t)threadIdx.x >= a.nc) p0 = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    float zg = 0.0f;
    if (given) {
        zg = Vec<IN>::one(static_cast<const IN*>(a.z)[t * a.ld + id]);
    }
    float M = p0.x;
    for (int64_t i = threadIdx.x + TPB; i < a.nc; i += TPB) M = fmaxf(M, part[i].x);
    M = value_of(wave_top(order_of(M)));
    if (lane == 0) red[0][w] = M;
    if (a.k > 0) best.clear();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) M = fmaxf(M, red[0][i]);
    const float f = M == -INFINITY ? 0.0f : M;
    float s = 0.0f, u = 0.0f;
    auto add = [&](const float4& q) {
        const float d = q.x - f, e = exp2_hw(d * LOG2E);
        s = __builtin_fmaf(q.y, e, s);
        u = __builtin_fmaf(__builtin_fmaf(fmaxf(d, FLOOR), q.y, q.z), e, u);
    };
    add(p0);
    for (int64_t i = threadIdx.x + TPB; i < a.nc; i += TPB) add(part[i]);
    s = wave_total(s);
    u = wave_total(u);
    if (lane == 0) {
        red[1][w] = s;
        red[2][w] = u;
    }
    for (int64_t i0 = 0; i0 < n; i0 += PER * TPB) {
        if (i0 > 0) load(i0);
        uint32_t own = 0, o[WAVES], most = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) own = max(own, (uint32_t)(x[i] >> 32));
        maxima[threadIdx.x] = own;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            o[i] = maxima[lane + 64 * i];
            most = max(most, o[i]);
        }
        const uint32_t least = reached_by(o, a.k, wave_top(most));
        const uint64_t kth = best.kth;
        const int before = best.count;
        const uint64_t from = max((uint64_t)least << 32, kth);     // kth is at least 1: 0 is no key
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) best.push(x[i] >= from, x[i]);
        __syncthreads();
        if (best.count > Top::CAP) {                              // many equal ones: again, cut down on the way
            __syncthreads();
            if (threadIdx.x == 0) best.count = before;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                best.push(x[i] >= from && x[i] >= best.kth, x[i]);
                if (best.full()) best.cut(a.k);
            }
        }
        if (i0 + PER * TPB < n) {
            if (best.full()) best.cut(a.k);
        } else {
            best.cut(a.k);
        }
    }
    __syncthreads();
    s = red[1][0];
    u = red[2][0];
    for (int i = 1; i < WAVES; ++i) {
        s += red[1][i];
        u += red[2][i];
    }
    const bool none = M == -INFINITY && s == 0.0f;                 // every logit is -inf
    const float ls = logf(s), lse = none ? -INFINITY : f + ls;
    if (threadIdx.x == 0) {
        if (a.lse) a.lse[t] = lse;
        if (a.entropy) a.entropy[t] = none ? 0.0f : entropy_of(s, u);
    }
    auto logp = [&](float z) {                                     // z - f first: lse may be far from 0
        const float q = none ? -INFINITY : z - f - ls;
        return q > 0.0f ? 0.0f : q;
    };
    if ((int)threadIdx.x < a.m) a.logp[t * a.m + threadIdx.x] = given ? logp(zg) : 0.0f;
    if ((int)threadIdx.x < a.k) {
        const int j = threadIdx.x;
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
    const int64_t t = (int64_t)blockIdx.z * ROWS_Y + blockIdx.y, lo = (int64_t)blockIdx.x * CH;
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
    const bool none = lse <= MASKS;
    if (lse != lse) A = lse;                                       // a row with a NaN has no gradient but that
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
        v[i] = *reinterpret_cast<const uint4*>(row + min(col, (a.V - 1) / 8 * 8));
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

// A block's columns: 16384 of bf16, or 4096 where that leaves CUs without one
// (one row of 151936, 20 alternatives: 12 us with 4096; 32 rows 13.6 with 16384 and
// 14.8 with 4096, 128 rows and 64 alternatives 20 and 48).
int64_t rows_chunk(int64_t T, int64_t V) {
    return T * ((V + 16383) / 16384) >= CUS ? 16384 : 4096;
}

template <typename IN, int NL>
static hipError_t launch_rows(const RowsArgs& a, hipStream_t st) {
    if (a.entropy) hipLaunchKernelGGL((k_rows_chunk<IN, NL, true>), rows_grid(a.nc, a.T), dim3(TPB), 0, st, a);
    else hipLaunchKernelGGL((k_rows_chunk<IN, NL, false>), rows_grid(a.nc, a.T), dim3(TPB), 0, st, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(k_rows_join<IN>, grid_of(a.T), dim3(TPB), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_logprob_rows(const RowsArgs& a, hipStream_t st) {
    return rows_chunk(a.T, a.V) == 16384 ? launch_rows<uint16_t, 8>(a, st) : launch_rows<uint16_t, 2>(a, st);
}

hipError_t launch_logprob_bwd(const LogpBwdArgs& a, hipStream_t st) {
    const int64_t chunks = (a.V + NB * 8 * TPB - 1) / (NB * 8 * TPB);
    hipLaunchKernelGGL(k_logp_bwd, rows_grid(chunks, a.T), dim3(TPB), 0, st, a);
    return hipGetLastError();
}

// ---------------------------------------------------------- from hidden states --
namespace {

// The wave's logit of token t and id, by all its lanes.
__device__ __forceinline__ float dot_of(const HeadLogpArgs& a, int64_t t, int id) {
    const uint4* hr = reinterpret_cast<const uint4*>(a.h + t * a.H);
    const uint4* wr = reinterpret_cast<const uint4*>(a.w + (int64_t)id * a.H);
    float acc = 0.0f;
#pragma unroll 4
    for (int c = threadIdx.x & 63; c < (a.H >> 3); c += 64) {
        float x[8], y[8];
        unpack8(hr[c], x);
        unpack8(wr[c], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc = __builtin_fmaf(x[e], y[e], acc);
    }
    return wave_total(acc);
}

// Logits of up to 8 tokens, in fp32: the weight is read once, a kilobyte of a row
// per load, past the caches (a load of the matrix operand's shape, 16 rows of 64
// bytes, arrives at 5.4 TB/s, these at 6.8), and multiplied with pairs of columns
// in the vector unit: 4 operations a token for 16 bytes of a lane.  A block has a run
// of the rows, its waves 4 of them at a time; the loads of the next GO chunks of
// 512 columns are in flight while a wave multiplies, over the ends of rows too.
// (One token of 2048 by 151936: 91 us; 108 through the caches.)
constexpr int ROW_TPB = 512, ROW_N = 4;
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
template <int TT, int ROW_GO, int BYTES>
__global__ __launch_bounds__(ROW_TPB) void k_head_rows(HeadLogpArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t sh[BYTES / 2];
    const int lane = threadIdx.x & 63, H = a.H, chunks = (H + 511) / 512, Hp = chunks * 512;
    for (int i = threadIdx.x; i < TT * Hp / 8; i += ROW_TPB) {      // rows padded with zeros, tokens repeated
        const int t = i / (Hp / 8), c = i - t * (Hp / 8);
        const uint4 v = reinterpret_cast<const uint4*>(a.h + min((int64_t)t, a.T - 1) * H)[min(c, H / 8 - 1)];
        reinterpret_cast<uint4*>(sh)[i] = c < H / 8 ? v : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int64_t groups = (a.V + ROW_N - 1) / ROW_N, end = groups * (blockIdx.x + 1) / gridDim.x;
    int64_t g = groups * blockIdx.x / gridDim.x + wave_id();
    if (g >= end) return;
    int64_t lg = g;                                        // the loads' place, a step ahead
    int lc = 0;
    auto load = [&](u32x4 (&v)[ROW_GO][ROW_N]) {
        if (lg >= end) return;
#pragma unroll
        for (int j = 0; j < ROW_GO; ++j) {
            const int col = (lc + j) * 512 + lane * 8, at = col < H ? col : 0;
#pragma unroll
            for (int r = 0; r < ROW_N; ++r)
                v[j][r] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4*>(a.w + min(lg * ROW_N + r, a.V - 1) * H + at));
        }
        lc += ROW_GO;
        if (lc >= chunks) {
            lc = 0;
            lg += ROW_TPB / 64;
        }
    };
    float acc[ROW_N][TT];
#pragma unroll
    for (int r = 0; r < ROW_N; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = 0.0f;
    int c = 0;
    auto multiply = [&](const u32x4 (&v)[ROW_GO][ROW_N]) {
#pragma unroll
        for (int j = 0; j < ROW_GO; ++j) {
            if ((c + j) * 512 + lane * 8 >= H) break;              // (past the row's end are its first columns again)
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const u32x4 x = *reinterpret_cast<const u32x4*>(sh + t * Hp + (c + j) * 512 + lane * 8);
#pragma unroll
                for (int r = 0; r < ROW_N; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t p = v[j][r][e], q = x[e];
                        acc[r][t] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2v, p),
                                                                    __builtin_bit_cast(bf16x2v, q), acc[r][t], false);
                    }
            }
        }
        c += ROW_GO;
        if (c < chunks) return;
        c = 0;
        // Over the lanes: rows 2 and 3 trade halves with rows 0 and 1, row 1 (3)
        // quarters with row 0 (2), so that lanes 16 r .. 16 r + 15 have row r's
        // sums, then moves inside 16 lanes; lane 16 r + 15 has the total.
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            float x[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[r][t]), __float_as_uint(acc[r + 2][t]),
                                                                false, false);
                x[r] = __uint_as_float(h[0]) + __uint_as_float(h[1]);
            }
            const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[0]), __float_as_uint(x[1]), false, false);
            float z = __uint_as_float(q[0]) + __uint_as_float(q[1]);
            z += __uint_as_float(moved<0x111, 0xf>(__float_as_uint(z)));
            z += __uint_as_float(moved<0x112, 0xf>(__float_as_uint(z)));
            z += __uint_as_float(moved<0x114, 0xf>(__float_as_uint(z)));
            z += __uint_as_float(moved<0x118, 0xf>(__float_as_uint(z)));
            if ((lane & 15) == 15 && t < a.T) a.z[(int64_t)t * a.vc + g * ROW_N + (lane >> 4)] = z;
#pragma unroll
            for (int r = 0; r < ROW_N; ++r) acc[r][t] = 0.0f;
        }
        g += ROW_TPB / 64;
    };
    u32x4 v0[ROW_GO][ROW_N], v1[ROW_GO][ROW_N];
    load(v0);
    while (g < end) {
        load(v1);
        multiply(v0);
        if (g >= end) break;
        load(v0);
        multiply(v1);
    }
}

// Logits of more tokens: the weight is read once, 16 rows by 32 columns
// a load (64 bytes of a row in neighbouring lanes, two loads a cache line), straight
// into the matrix instruction's operand; the hidden states stand in LDS, rows 16
// bytes apart from a multiple of the banks.  A block has a run of rows, 16 at a
// time, its waves a share of the columns each, so that what the card reads at once
// are a few whole stretches of memory, past the caches (5.4 TB/s; 5.3 with whole
// rows to a wave, strided over the card).  The next rows' loads are in flight while
// a wave multiplies and the block adds its waves' sums.
constexpr int FEW_LOADS = 8, FEW_STEP = 32 * FEW_LOADS, FEW_TPB = 512, FEW_WAVES = FEW_TPB / 64;
template <int NT, int BYTES>
__global__ __launch_bounds__(FEW_TPB) void k_head_few(HeadLogpArgs a) {
    __shared__ __attribute__((aligned(16))) char sh[BYTES];
    __shared__ __attribute__((aligned(16))) float red[FEW_WAVES][256];
    const int lane = threadIdx.x & 63, tok = lane & 15, kc = lane >> 4, w = wave_id();
    const int T = (int)a.T, H = a.H, ldh = 2 * H + 16, chunks = H >> 3;
    for (int i = threadIdx.x; i < T * chunks; i += FEW_TPB) {
        const int t = i / chunks, c = i - t * chunks;
        *reinterpret_cast<uint4*>(sh + t * ldh + c * 16) = reinterpret_cast<const uint4*>(a.h)[i];
    }
    __syncthreads();
    const char* hb[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) hb[n] = sh + min(16 * n + tok, T - 1) * ldh + kc * 16;
    const int64_t tiles = (a.V + 15) / 16, end = tiles * (blockIdx.x + 1) / gridDim.x;
    int64_t tile = tiles * blockIdx.x / gridDim.x;
    const int share = (H / FEW_WAVES + 31) / 32 * 32, k0 = w * share, k1 = min(k0 + share, H);
    const int steps = (share + FEW_STEP - 1) / FEW_STEP;
    int64_t ltile = tile;                                  // the loads' place, a step ahead
    int lk = k0;
    auto load = [&](bf16x8 (&v)[FEW_LOADS]) {
        if (ltile >= end) return;
        const uint16_t* row = a.w + min(ltile * 16 + tok, a.V - 1) * H + kc * 8;
#pragma unroll
        for (int i = 0; i < FEW_LOADS; ++i) {
            const int k = lk + 32 * i;
            const bf16x8* p = reinterpret_cast<const bf16x8*>(row + (k < k1 ? k : 0));
            v[i] = NT == 1 ? __builtin_nontemporal_load(p) : *p;   // 2 to 4% each way
        }
        lk += FEW_STEP;
        if (lk >= k0 + steps * FEW_STEP) {
            lk = k0;
            ++ltile;
        }
    };
    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int k = k0;
    auto multiply = [&](const bf16x8 (&v)[FEW_LOADS]) {
#pragma unroll
        for (int i = 0; i < FEW_LOADS; ++i)
            if (k + 32 * i < k1)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        v[i], *reinterpret_cast<const bf16x8*>(hb[n] + 2 * (k + 32 * i)), acc[n], 0, 0, 0);
        k += FEW_STEP;
        if (k < k0 + steps * FEW_STEP) return;
        k = k0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            *reinterpret_cast<f32x4*>(&red[w][4 * lane]) = acc[n];
            acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            lds_barrier();
            // lane l's four sums are token l % 16, rows 4 (l / 16) and on
            const int e = threadIdx.x, t = 16 * n + ((e >> 2) & 15);
            if (e < 256 && t < T) {
                float s = red[0][e];
#pragma unroll
                for (int i = 1; i < FEW_WAVES; ++i) s += red[i][e];
                a.z[(int64_t)t * a.vc + tile * 16 + 4 * (e >> 6) + (e & 3)] = s;
            }
            lds_barrier();
        }
        ++tile;
    };
    bf16x8 v0[FEW_LOADS], v1[FEW_LOADS];
    load(v0);
    while (tile < end) {
        load(v1);
        multiply(v0);
        if (tile >= end) break;
        load(v0);
        multiply(v1);
    }
}

// log2 p of a logit, the distance first: of logits far from 0 a frame in base 2 is
// rounded by more than lse is.  At most 0, as lse may come from sums in another order.
__device__ __forceinline__ float log2_p(float z, float lse) {
    return __builtin_amdgcn_fmed3f((z - lse) * LOG2E, FLOOR2, 0.0f);
}

// The tile product of the output layer's loss with other epilogues.
//   SUMS  of each token's 64 columns of a wave: the maximum m, s = sum e^(z - m), and
//         with ENT u = sum e^(z - m) (z - m)
//   TOP   these, and the 64 logits themselves where m is above the token's bound,
//         the k-th best logit of the pieces before: of a long row that is seldom
//   GRAD  P = -p (A + b (log p + entropy)) in bf16, for the matrix units: half a bf16
//         step of each entry, of which a row of the gradient sums many, beside the
//         half step of the result.  The gradient's distance from 64 bits is 0.0016 to
//         0.0017 so and with P in fp32, the two forms 5e-4 to 7e-4 apart.  The given
//         tokens' entries stay out of it: a - p A may cancel.
enum : int { SUMS = 0, TOP = 1, GRAD = 2 };
template <int MODE, bool ENT>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) void k_head_z(HeadLogpArgs a) {
    // a token's constants of the epilogue: its bound, or its row of rowc
    constexpr int CB = MODE == GRAD ? 16 : MODE == TOP ? 4 : 0, ROWC = BM * CB;
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
        const int cols = (int)min((int64_t)BN, a.V - v0);             // may be <= 0 in the last piece's padding
        la.rs = make_rsrc_words(a.h + m0 * a.H, (int64_t)rows * a.H * 2);
        lb.rs = make_rsrc_words(a.w + (cols > 0 ? v0 : 0) * a.H, (int64_t)cols * a.H * 2);
        if (MODE != SUMS && wave < CB / 4) {                          // 1 KB per wave
            const char* c = MODE == GRAD ? reinterpret_cast<const char*>(a.rowc + m0) : reinterpret_cast<const char*>(a.thr + m0);
            const uint32_t voff[1] = {(uint32_t)(wave * 64 + lane) * 16};
            stage_loads<1, 0>(make_rsrc_words(c, (int64_t)(rows + 3) / 4 * 4 * CB),
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
        asm volatile("" : "+v"(lane));                                // what follows from it is not held through the steps
        const int cols = (int)min((int64_t)BN, a.V - a.c0 - (int64_t)tn * BN);
        const lds_t* consts = smem + SMEM + (i & 1) * ROWC;
#pragma unroll
        for (int ti = 0; ti < WTM; ++ti) {
            if (ti >= sub) break;
            const int row = wm * wr + ti * 32 + (lane & 31);
            auto past = [&](float x) {                                // the columns past the vocabulary become x
                if (cols < BN) {
#pragma unroll
                    for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (wn * 64 + tj * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3) >= cols)
                                acc[ti][tj][v] = x;
                }
            };
            if constexpr (MODE != GRAD) {
                past(-INFINITY);
                float m = acc[ti][0][0];
#pragma unroll
                for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                    for (int v = 0; v < 16; ++v) m = fmaxf(m, acc[ti][tj][v]);
                m = fmaxf(m, xor32(m));
                if constexpr (MODE == TOP) {
                    const __amdgpu_buffer_rsrc_t zrs = make_rsrc(a.z + m0 * a.vc + (int64_t)tn * BN,
                                                                 (int64_t)(rows - 1) * a.vc * 4 + BN * 4);
                    const float thr = reinterpret_cast<const __attribute__((address_space(3))) float*>(consts)[row];
                    if (a.first || m > thr) {
#pragma unroll
                        for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                u32x4 c;
#pragma unroll
                                for (int j = 0; j < 4; ++j) c[j] = __float_as_uint(acc[ti][tj][4 * q + j]);
                                const int col = wn * 64 + tj * 32 + 8 * q + 4 * (lane >> 5);
                                __builtin_amdgcn_raw_buffer_store_b128(
                                    c, zrs, (uint32_t)row * (uint32_t)a.vc * 4u + col * 4, 0, 0);
                            }
                    }
                }
                // far from 0 the distance to m comes first (always so: 16384 tokens 8140 -> 8240 us);
                // by a token's own m, so that its sums do not depend on its neighbours
                const bool far = fabsf(m) >= FAR;
                const float mf = m == -INFINITY ? 0.0f : m;                           // a strip of nothing but -inf has s = 0
                const float f = mf * LOG2E, d = far ? 0.0f : __builtin_fmaf(mf, LOG2E, -f);
                float s = 0.0f, u = 0.0f;
                auto add = [&](float x) {
                    const float e = exp2_hw(x);
                    s += e;
                    if (ENT) u = __builtin_fmaf(e, fmaxf(x, FLOOR2), u);
                };
                if (far) {
#pragma unroll
                    for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                        for (int v = 0; v < 16; ++v) add((acc[ti][tj][v] - mf) * LOG2E);
                } else {
#pragma unroll
                    for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                        for (int v = 0; v < 16; ++v) add(__builtin_fmaf(acc[ti][tj][v], LOG2E, -f));
                }
                s += xor32(s);
                if (ENT) u += xor32(u);
                const float g = __builtin_fmaf(-d, LN2, 1.0f);                        // as in a chunk of rows
                if (ENT) u = g * LN2 * __builtin_fmaf(-d, s, u);
                s *= g;
                const int64_t o = ((int64_t)tn * 4 + wn) * a.T + m0 + row;
                if (lane < 32 && row < rows) {
                    a.stats[o] = make_float2(m, s);
                    if (ENT) a.ustats[o] = u;
                }
            } else {
                const __amdgpu_buffer_rsrc_t prs = make_rsrc(a.p + m0 * a.vc + (int64_t)tn * BN,
                                                             (int64_t)(rows - 1) * a.vc * 2 + BN * 2);
                const __attribute__((address_space(3))) float4* rc =
                    reinterpret_cast<const __attribute__((address_space(3))) float4*>(consts);
                const float lse = rc[row].x, c = rc[row].y, b = rc[row].z * LN2;
#pragma unroll
                for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const float l = log2_p(acc[ti][tj][v], lse);
                        acc[ti][tj][v] = -exp2_hw(l) * __builtin_fmaf(b, l, c);
                    }
                past(0.0f);
                // the one given token's entry, if it lies in these 64 columns: its share is added in fp32 at the end
                const int own = __float_as_int(rc[row].w) - (int)(a.c0 + (int64_t)tn * BN + wn * 64);
                if (__any((unsigned)own < 64u)) {
#pragma unroll
                    for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            if (own == tj * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)) acc[ti][tj][v] = 0.0f;
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

// A piece joins its tokens' running sums and alternatives: TOK tokens per block,
// first 64 WPT threads per token over the strips of 64 columns, then WPT
// waves per token over the strips that can hold an alternative.  A wave's best are
// its lanes' keys in descending order; logits above the k-th are gathered in LDS
// and put in 64 at a time by a sort and a merge, the last few one at a time.
constexpr int MWORDS = LOGP_MAX_PIECE / 64 / 32, MLIST = 16, MPARTS = 256;
template <int WPT, int TOK>
__global__ __launch_bounds__(64 * WPT * TOK) __attribute__((amdgpu_waves_per_eu(8))) void k_logp_merge(HeadLogpArgs a) {
    constexpr int WAVES = WPT * TOK, PER = 64 * WPT, SUB = MPARTS / PER, UN = 4;
    __shared__ float red[3][WAVES][TOK];
    __shared__ float tmax[TOK][MPARTS];
    __shared__ uint32_t flag[TOK][MWORDS];
    __shared__ uint16_t list[WAVES][MLIST * 32];
    __shared__ float bound[TOK];
    __shared__ uint64_t keys[WAVES][128];
    const int tok = threadIdx.x & (TOK - 1), sl = threadIdx.x / TOK, lane = threadIdx.x & 63, w = wave_id();
    // An XCD has a run of neighbouring tokens: their strips lie in the same cache lines.
    const int group = xcd_tile(blockIdx.x, gridDim.x, (int)((a.T + TOK - 1) / TOK));
    if (group < 0) return;
    const int64_t t0 = (int64_t)group * TOK, tc = min(t0 + tok, a.T - 1);
    const int strips = (int)((min((int64_t)a.vc, a.V - a.c0) + 63) / 64), words = (strips + 31) / 32;
    const bool ent = a.entropy != nullptr, top = a.k > 0;
    if (top) {
        for (int i = sl; i < words; i += PER) flag[tok][i] = 0;
        __syncthreads();
    }
    const float thr = top && !a.first ? a.thr[tc] : -INFINITY;
    // what the later steps need of the pieces before, ahead of the strips: from
    // the barrier on wave w is part `sub` of token t
    const int tk = w / WPT, sub = w % WPT;
    const int64_t t = t0 + tk, tl = min(t, a.T - 1);
    const bool live = t < a.T;
    float4 before = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    uint64_t best = 0;                                     // the wave's best, sorted
    float kth = -INFINITY;                                 // k logits, all of lower ids, are at least this
    if (!a.first) {
        before = a.run[tl];
        if (top) {
            kth = a.thr[tl];
            if (sub == 0 && lane < a.k && a.best_i[tl * a.k + lane] >= 0)
                best = key_of(a.best_z[tl * a.k + lane], a.best_i[tl * a.k + lane]);
        }
    }
    // M, s, u of the thread's strips, maxima of SUB parts of them
    float M = -INFINITY, s = 0.0f, u = 0.0f, tm[SUB];
    auto join = [&](float m2, float s2, float u2) {        // (M, s, u) and another
        const float n = fmaxf(M, m2);
        const float d1 = fmaxf(M == n ? 0.0f : M - n, FLOOR), d2 = fmaxf(m2 == n ? 0.0f : m2 - n, FLOOR);
        const float e1 = exp2_hw(d1 * LOG2E), e2 = exp2_hw(d2 * LOG2E);
        u = __builtin_fmaf(e1, __builtin_fmaf(d1, s, u), e2 * __builtin_fmaf(d2, s2, u2));
        s = __builtin_fmaf(e1, s, e2 * s2);
        M = n;
    };
#pragma unroll
    for (int j = 0; j < SUB; ++j) tm[j] = -INFINITY;
    for (int i0 = sl; i0 < strips; i0 += PER * UN) {
        float2 v[UN];
        float vu[UN];
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            const int64_t i = min(i0 + PER * j, strips - 1) * a.T + tc;
            v[j] = a.stats[i];
            vu[j] = ent ? a.ustats[i] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            const int i = i0 + PER * j;
            if (i >= strips) break;
            const float m = v[j].x;
            tm[j % SUB] = fmaxf(tm[j % SUB], m);
            join(m, v[j].y, vu[j]);
            if (top && m > thr) atomicOr(&flag[tok][i >> 5], 1u << (i & 31));
        }
    }
    // over the token's threads: those of a wave, then the block's waves, in a fixed order
#pragma unroll
    for (int m = TOK; m < 64; m <<= 1) {
        const float m2 = __shfl_xor(M, m), s2 = __shfl_xor(s, m), u2 = __shfl_xor(u, m);
        join(m2, s2, u2);
    }
    if (lane < TOK) {
        red[0][w][tok] = M;
        red[1][w][tok] = s;
        red[2][w][tok] = u;
    }
    if (top)
#pragma unroll
        for (int j = 0; j < SUB; ++j) tmax[tok][sl * SUB + j] = tm[j];
    __syncthreads();
    M = red[0][lane % WAVES][tk];
    s = red[1][lane % WAVES][tk];
    u = red[2][lane % WAVES][tk];
#pragma unroll
    for (int m = 1; m < WAVES; m <<= 1) {
        const float m2 = __shfl_xor(M, m), s2 = __shfl_xor(s, m), u2 = __shfl_xor(u, m);
        join(m2, s2, u2);
    }
    join(before.x, before.y, before.z);
    const bool none = M == -INFINITY && s == 0.0f;         // every logit is -inf
    const float ls = logf(s), lse = none ? -INFINITY : M + ls;
    auto logp = [&](float z) {                             // z - M first: lse may be far from 0
        const float q = none ? -INFINITY : z - M - ls;
        return q > 0.0f ? 0.0f : q;
    };
    if (live && a.last && sub == 0) {
        if (lane == 0) {
            if (a.lse) a.lse[t] = lse;
            if (ent) a.entropy[t] = none ? 0.0f : entropy_of(s, u);
        }
    }
    if (live && a.last)
        for (int j = sub; j < a.m; j += WPT) {
            const int id = __builtin_amdgcn_readfirstlane(a.ids[t * a.m + j]);
            const float x = id >= 0 && id < a.V ? logp(dot_of(a, t, id)) : 0.0f;
            if (lane == 0) a.logp[t * a.m + j] = x;
        }
    // More strips above the bound than k: a bound that k parts' maxima reach keeps
    // most of them out (a first piece has no bound before: 75 strips of 1024 for k = 64).
    int marked = 0;
    float from = -INFINITY;
    if (top) {
        for (int i = lane; i < words; i += 64) marked += __popc(flag[tk][i]);
        marked = (int)wave_total((float)marked);
        if (marked > a.k) {
            uint32_t o[MPARTS / 64], most = 0;
#pragma unroll
            for (int j = 0; j < MPARTS / 64; ++j) {
                o[j] = order_of(tmax[tk][lane + 64 * j]);
                most = max(most, o[j]);
            }
            const uint32_t r = reached_by(o, a.k, wave_top(most));
            from = r > ORDER_MIN ? value_of(r) : -INFINITY;
        }
        if (lane == 0) bound[tk] = from;
    }
    // (a barrier for all: every part has read run before one writes it)
    if (__syncthreads_or(marked > a.k)) {
        for (int i = sl; i < words; i += PER) flag[tok][i] = 0;
        __syncthreads();
        const float least = bound[tok];
#pragma unroll 8
        for (int i = sl; i < strips; i += PER) {
            const float m = a.stats[(int64_t)i * a.T + tc].x;
            if (m > thr && m >= least) atomicOr(&flag[tok][i >> 5], 1u << (i & 31));
        }
        __syncthreads();
    }
    if (live && lane == 0 && sub == 0 && !a.last) a.run[t] = make_float4(M, s, u, 0.0f);
    if (!top) return;
    const float* zr = a.z + tl * a.vc;
    const int cols = (int)min((int64_t)a.vc, a.V - a.c0);
    int n = 0;
    // f(logit of this lane, the strip's first column) for the wave's part of the listed strips, N in flight
    auto strips_by = [&](int i0, auto n_c, auto&& f) {
        constexpr int N = decltype(n_c)::value;
        float z[N];
        int col[N];
#pragma unroll
        for (int q = 0; q < N; ++q) {
            col[q] = __builtin_amdgcn_readfirstlane(list[w][min(i0 + q * WPT, n - 1)]) * 64;
            z[q] = zr[min(col[q] + lane, cols - 1)];
        }
#pragma unroll
        for (int q = 0; q < N; ++q)
            if (i0 + q * WPT < n) f(col[q] + lane < cols ? z[q] : -INFINITY, col[q], q);
        return i0 + N * WPT;
    };
    auto each_strip = [&](auto&& f) {
        int i0 = sub;
        while (i0 + 4 * WPT < n) i0 = strips_by(i0, std::integral_constant<int, 16>{}, f);
        if (i0 < n) strips_by(i0, std::integral_constant<int, 4>{}, f);
    };
    int gathered = 0;
    auto put = [&](int n) {                                // the first n <= 64 gathered keys
        if (n <= 32) {
            // one at a time: the lanes it does not pass stay, the others move on
            for (int j = 0; j < n; ++j) {
                const uint64_t x = keys[w][j];
                const uint32_t lo = __builtin_amdgcn_update_dpp(-1, (int)(uint32_t)best, 0x138, 0xf, 0xf, false);
                const uint32_t hi = __builtin_amdgcn_update_dpp(-1, (int)(uint32_t)(best >> 32), 0x138, 0xf, 0xf, false);
                const uint64_t before = ((uint64_t)hi << 32) | lo;         // the lane's before (wave_shr:1)
                best = best > x ? best : before > x ? x : before;
            }
        } else {
            const uint64_t x = sorted_keys(lane < n ? keys[w][lane] : 0);
            best = merged_keys(best, __shfl((unsigned long long)x, 63 - lane));
        }
        const uint32_t o = __builtin_amdgcn_readlane((uint32_t)(best >> 32), a.k - 1);
        if (o != 0) kth = fmaxf(kth, value_of(o));
    };
    for (int w0 = 0; w0 < words; w0 += MLIST) {
        // the marked strips of MLIST words in a list, ascending
        uint32_t bits = lane < MLIST && w0 + lane < words ? flag[tk][w0 + lane] : 0;
        const int own = __popc(bits);
        int at = own;                                      // running total over the lanes
#pragma unroll
        for (int d = 1; d < MLIST; d <<= 1) {
            const int x = __shfl_up(at, d);
            at += lane >= d ? x : 0;
        }
        n = __builtin_amdgcn_readlane(at, MLIST - 1);
        at -= own;
        while (bits) {
            list[w][at++] = (uint16_t)((w0 + lane) * 32 + __ffs(bits) - 1);
            bits &= bits - 1;
        }
        each_strip([&](float z, int col, int) {
            const uint64_t mask = __ballot(z > kth && z >= from);
            if (mask == 0) return;
            if (z > kth && z >= from) keys[w][lanes_before(mask, gathered)] = key_of(z, a.c0 + col + lane);
            gathered += __popcll(mask);
            if (gathered < 64) return;
            put(64);
            gathered -= 64;
            keys[w][lane] = keys[w][64 + lane];            // a wave's own LDS accesses are in order
        });
    }
    if (gathered > 0) put(gathered);
    if (WPT > 1) {
        keys[w][lane] = best;
        __syncthreads();
        if (sub > 0) return;
#pragma unroll
        for (int i = 1; i < WPT; ++i) best = merged_keys(best, keys[w + i][63 - lane]);
        const uint32_t o = __builtin_amdgcn_readlane((uint32_t)(best >> 32), a.k - 1);
        kth = o != 0 ? value_of(o) : -INFINITY;
    }
    if (!live) return;
    if (lane < a.k) {
        const int id = best != 0 ? key_id(best) : -1;
        const float z = best != 0 ? key_z(best) : -INFINITY;
        if (a.last) {
            a.top_ids[t * a.k + lane] = id;
            a.top_logp[t * a.k + lane] = best != 0 ? logp(z) : -INFINITY;
        } else {
            a.best_z[t * a.k + lane] = z;
            a.best_i[t * a.k + lane] = id;
        }
    }
    if (lane == 0) a.thr[t] = kth;
}

// Backward: a token's constants of the epilogue above and its given tokens'
// logits, by WPT waves.
template <int WPT>
__global__ __launch_bounds__(256) void k_logp_rowc(HeadLogpArgs a) {
    const int lane = threadIdx.x & 63, w = wave_id(), sub = w % WPT;
    const int64_t t = block_id() * (4 / WPT) + w / WPT;
    if (t >= a.T) return;
    const int id = lane < a.m ? a.ids[t * a.m + lane] : -1;
    const bool in = id >= 0 && id < a.V;
    if (sub == 0) {
        const float A = wave_total(in ? a.dlogp[t * a.m + lane] : 0.0f);
        const float b = a.dent ? a.dent[t] : 0.0f, H = a.dent ? a.entropy[t] : 0.0f;
        if (lane == 0) {
            const float lse = a.lse[t];                            // (a NaN: the row's gradient is one)
            const float4 rc = lse <= MASKS ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                           : make_float4(lse, lse == lse ? __builtin_fmaf(b, H, A) : lse, b, 0.0f);
            a.rowc[t] = make_float4(rc.x, rc.y, rc.z, __int_as_float(a.m == 1 && in ? id : -1));
            a.ones[t] = 1.0f;
        }
    }
    for (int j = sub; j < a.m; j += WPT) {
        const int one = __builtin_amdgcn_readlane(in ? id : -1, j);
        const float z = one >= 0 ? dot_of(a, t, one) : 0.0f;
        if (lane == 0) a.zs[t * a.m + j] = z;
    }
}

// Several given tokens' entries of P are zero (a single one's is made so in the
// epilogue, which saves a launch): their share is added in fp32 at the end.
__global__ __launch_bounds__(256) void k_logp_clear(HeadLogpArgs a) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= a.T * a.m) return;
    const int id = a.ids[i];
    if (id >= a.c0 && id < a.V && id - a.c0 < a.vc) a.p[i / a.m * a.vc + (id - a.c0)] = 0;
}

// dh = sum of the splits + sum_j coef_j w_id_j: a block per token, VEC columns per
// thread: 4 where there are many splits, for more loads in flight (333 rows of 1024,
// 32 splits: 9.2 us and 9.6; 2048 of 2048, 4 splits: 18.7 and 16.0).
template <int VEC>
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
        const float l = log2_p(a.zs[t * a.m + j], rc.x);
        sid[j] = in ? id : 0;
        const float own = first ? exp2_hw(l) * __builtin_fmaf(rc.z * LN2, l, rc.y) : 0.0f;
        scoef[j] = in && !(a.lse[t] <= MASKS) ? a.dlogp[t * a.m + j] - own : 0.0f;
    }
    __syncthreads();
    typedef uint32_t words __attribute__((ext_vector_type(VEC / 2)));
    for (int c = threadIdx.x; c < a.H / VEC; c += 256) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = 0.0f;
#pragma unroll 16
        for (int s = 0; s < splits; ++s) {
            const float4* g = reinterpret_cast<const float4*>(a.g + ((int64_t)s * a.T + t) * a.H + VEC * c);
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float4 x = g[i];
                o[4 * i] += x.x; o[4 * i + 1] += x.y; o[4 * i + 2] += x.z; o[4 * i + 3] += x.w;
            }
        }
#pragma unroll 4
        for (int j = 0; j < a.m; ++j) {
            const float k = scoef[j];
            const words x = reinterpret_cast<const words*>(a.w + (int64_t)sid[j] * a.H)[c];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                o[2 * i] = __builtin_fmaf(k, bf_lo(x[i]), o[2 * i]);
                o[2 * i + 1] = __builtin_fmaf(k, bf_hi(x[i]), o[2 * i + 1]);
            }
        }
        words r;
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) r[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
        reinterpret_cast<words*>(a.grad + t * a.H)[c] = r;
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

// The pieces of the forward.  Without alternatives a piece is as long as its sums
// may be (640 MB).  With them a piece's logits have their place (4 bytes each, so
// at most 640 MB again), and the first piece, of which all strips are kept, is one
// round of tiles over the card, at least 4096 columns; every other is twice what
// came before it, in whole rounds: a piece keeps about k (its length / the columns
// before) strips of 64 of a token.
HeadLogpPlan head_logp_plan(int64_t T, int64_t H, int64_t V, int k) {
    HeadLogpPlan p{};
    const int64_t n = T > 0 ? T : 1, mt = (n + BM - 1) / BM;
    const int64_t bytes = k > 0 ? n * 4 : n * 12 / 64 + 1;
    int64_t most = ((int64_t)640 << 20) / bytes;
    most = std::min(most, ((int64_t)1 << 30) / H);                 // the reach of a buffer resource's offsets
    most = std::min(most, (int64_t)LOGP_MAX_PIECE);
    p.most = (int)std::max(most / BN * BN, (int64_t)BN);
    p.round = (int)std::max((CUS / mt) * BN, (int64_t)BN);
    p.first = k > 0 ? std::min(p.most, std::max(p.round, 4096)) : p.most;
    p.ld = (int)std::min((int64_t)p.most, (V + BN - 1) / BN * BN);
    return p;
}

// Tokens few enough for their hidden states to stand in LDS while the weight goes
// by, and for the logits of the whole vocabulary to stand in the workspace.
bool head_logp_few(int64_t T, int64_t H, int64_t V, int k) {
    const int64_t chunks = (V + FEW_CHUNK - 1) / FEW_CHUNK;
    return T <= 64 && T * (2 * H + 16) <= FEW_BYTES &&
           T * (head_few_ld(V) * 4 + chunks * (16 + (k > 0 ? rows_keys(k) * 8 : 0))) <= ((int64_t)640 << 20);
}

static hipError_t launch_few(HeadLogpArgs a, hipStream_t st) {
    const int64_t bytes = a.T * (2 * a.H + 16), tiles = (a.V + 15) / 16;
    a.vc = (int)head_few_ld(a.V);
    auto grid = [&](int per_cu) { return dim3((unsigned)std::min<int64_t>((int64_t)CUS * per_cu, tiles)); };
    const int64_t row = (a.H + 511) / 512 * 1024;          // bytes of a token's padded row
    // 2048 by 151936, with 20 alternatives, by rows of the weight and by the matrix
    // operand: 1 token 103 and 130 us, 8 tokens 120 and 136, 16 tokens 172 and 146; 1
    // token in the form for 8: 112, 4: 116 and not 110
    if (a.T == 1 && row <= 32768) hipLaunchKernelGGL((k_head_rows<1, 4, 32768>), grid(2), dim3(ROW_TPB), 0, st, a);
    else if (a.T <= 2 && 2 * row <= 32768) hipLaunchKernelGGL((k_head_rows<2, 4, 32768>), grid(2), dim3(ROW_TPB), 0, st, a);
    else if (a.T <= 4 && 4 * row <= 32768) hipLaunchKernelGGL((k_head_rows<4, 4, 32768>), grid(2), dim3(ROW_TPB), 0, st, a);
    else if (a.T <= 8 && 8 * row <= 65536) hipLaunchKernelGGL((k_head_rows<8, 1, 65536>), grid(2), dim3(ROW_TPB), 0, st, a);
    // two blocks a CU where LDS holds the hidden states twice (16 of 2048: 146 us and 155)
    else if (a.T <= 16 && bytes <= 67584) hipLaunchKernelGGL((k_head_few<1, 67584>), grid(2), dim3(FEW_TPB), 0, st, a);
    else if (a.T <= 16) hipLaunchKernelGGL((k_head_few<1, FEW_BYTES>), grid(1), dim3(FEW_TPB), 0, st, a);
    else if (a.T <= 32) hipLaunchKernelGGL((k_head_few<2, FEW_BYTES>), grid(1), dim3(FEW_TPB), 0, st, a);
    else hipLaunchKernelGGL((k_head_few<4, FEW_BYTES>), grid(1), dim3(FEW_TPB), 0, st, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    RowsArgs r{};
    r.T = a.T;
    r.V = a.V;
    r.m = a.m;
    r.k = a.k;
    r.z = a.z;
    r.ld = a.vc;
    r.nc = (a.V + FEW_CHUNK - 1) / FEW_CHUNK;
    r.part = a.run;
    r.keys = a.keys;
    r.ids = a.ids;
    r.logp = a.logp;
    r.lse = a.lse;
    r.entropy = a.entropy;
    r.top_ids = a.top_ids;
    r.top_logp = a.top_logp;
    return launch_rows<float, FEW_CHUNK / (4 * TPB)>(r, st);
}

hipError_t launch_head_logprob_fwd(HeadLogpArgs a, const HeadLogpPlan& pl, hipStream_t st) {
    if (head_logp_few(a.T, a.H, a.V, a.k)) return launch_few(a, st);
    a.bm = tile_rows(a.T);
    int64_t c0 = 0;
    while (c0 < a.V) {
        const int64_t left = (a.V - c0 + BN - 1) / BN * BN;
        int64_t n = c0 == 0 ? pl.first : pl.most;
        if (c0 > 0 && a.k > 0 && 2 * c0 < n) n = std::max(2 * c0 / pl.round * pl.round, (int64_t)pl.round);
        n = std::min(n, left);
        a.c0 = c0;
        a.vc = (int)n;
        a.first = c0 == 0;
        a.last = c0 + n >= a.V;
        const dim3 grid(product_grid(a));
        if (a.k > 0) {
            if (a.entropy) hipLaunchKernelGGL((k_head_z<TOP, true>), grid, dim3(512), 0, st, a);
            else hipLaunchKernelGGL((k_head_z<TOP, false>), grid, dim3(512), 0, st, a);
        } else {
            if (a.entropy) hipLaunchKernelGGL((k_head_z<SUMS, true>), grid, dim3(512), 0, st, a);
            else hipLaunchKernelGGL((k_head_z<SUMS, false>), grid, dim3(512), 0, st, a);
        }
        auto merge = [&](auto kernel, int wpt, int tok) {
            const unsigned groups = (unsigned)((a.T + tok - 1) / tok);
            hipLaunchKernelGGL(kernel, dim3((groups + 7) / 8 * 8), dim3(64 * wpt * tok), 0, st, a);
        };
        // a wave per token where tokens fill the card, else two (16384 tokens: 8070
        // us and 8290; 4096 of hidden 512: 955 and 961; 2048: 1090 and 1080; 333: 47 and 44)
        if (a.T >= 4096) merge(k_logp_merge<1, 4>, 1, 4);
        else merge(k_logp_merge<2, 4>, 2, 4);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        c0 += n;
    }
    return hipSuccess;
}

hipError_t launch_head_logprob_bwd(HeadLogpArgs a, const HeadPlan& pl, hipStream_t st) {
    a.bm = tile_rows(a.T);
    a.vc = pl.vc;
    if (a.m > 1) hipLaunchKernelGGL(k_logp_rowc<4>, grid_of(a.T), dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_logp_rowc<1>, grid_of((a.T + 3) / 4), dim3(256), 0, st, a);
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
        hipLaunchKernelGGL((k_head_z<GRAD, false>), dim3(product_grid(a)), dim3(512), 0, st, a);
        if (a.m > 1) hipLaunchKernelGGL(k_logp_clear, grid_of((a.T * a.m + 255) / 256), dim3(256), 0, st, a);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess || (err = launch_head_grad(g, st)) != hipSuccess) return err;
    }
    if (pl.splits >= 16) hipLaunchKernelGGL(k_logp_out<4>, grid_of(a.T), dim3(256), 0, st, a, pl.splits);
    else hipLaunchKernelGGL(k_logp_out<8>, grid_of(a.T), dim3(256), 0, st, a, pl.splits);
    return hipGetLastError();
}

}  // namespace fq
