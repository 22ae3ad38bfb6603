// Products of packed 4-bit weights with a few rows, and the routed SwiGLU
// expert layer on packed weights for a few tokens.
//
//   y[m, n] = sum_k x[m, k] W[n, k],  W = q s (INT4, a scale per row or group)
//                                     W = q d t (NVFP4: E2M1, E4M3 per 16, fp32 per matrix)
// A few rows against megabytes of weights: what counts is the stream of codes
// from HBM, so every byte is read once and all vector work per code is kept
// under the 2.5 operations a CU has per code at the full HBM rate.  The
// products themselves go to the matrix cores (v_mfma_f32_16x16x32_bf16, 16
// rows of x by 16 rows of W; unused rows of x cost nothing that counts): codes
// become bf16 exactly, x is bf16, sums are fp32.
//   INT4   v_and_or forms 128 + (q ^ 8) = 136 + q in bf16, two at a time, one
//          operation per code; a product of x with the constant -136, shared
//          by the wave's weight tiles, starts the sum and takes the 136 off
//          again in fp32.  The scale multiplies the sum of its group.
//   NVFP4  q d is exact in bf16 (2 + 4 significant bits): two conversions and
//          two products per pair of codes; t multiplies the end.
// A lane loads 16 bytes, 32 codes, of one weight row.  Which k a lane holds is
// free as long as x agrees: with a scale per row or per 128 and more a lane's
// four words are four products' operands as they are; with groups of 32 or 64
// the words are transposed between the four lane groups first (four lane
// swaps), so that one product covers one 32-code segment of all 16 rows.
// The waves of a block split k and add their sums in order.
#include <type_traits>

#include "fq_act.h"
#include "fq_ops.h"

namespace fq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

enum Fmt { INT_WIDE = 0, INT_NARROW = 1, NVFP4 = 2 };

constexpr int NW = 4;                     // waves of a block

__device__ __forceinline__ f32x4 mfma(u32x4 x, u32x4 w, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w), c, 0,
                                                   0, 0);
}

// 136 + q of eight INT4 codes as bf16, in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ u32x4 int_words(uint32_t w) {
    w ^= 0x88888888u;
    u32x4 o;
    o.x = (w & 0x000F000Fu) | 0x43004300u;
    o.y = ((w >> 4) & 0x000F000Fu) | 0x43004300u;
    o.z = ((w >> 8) & 0x000F000Fu) | 0x43004300u;
    o.w = ((w >> 12) & 0x000F000Fu) | 0x43004300u;
    return o;
}
// x in that order
__device__ __forceinline__ u32x4 int_order(u32x4 v) {
    u32x4 o;
    o.x = __builtin_amdgcn_perm(v.z, v.x, 0x05040100u);
    o.y = __builtin_amdgcn_perm(v.z, v.x, 0x07060302u);
    o.z = __builtin_amdgcn_perm(v.w, v.y, 0x05040100u);
    o.w = __builtin_amdgcn_perm(v.w, v.y, 0x07060302u);
    return o;
}
// q d of eight E2M1 codes as bf16 (exact)
__device__ __forceinline__ u32x4 fp4_words(uint32_t w, float d) {
    u32x4 o;
    f32x2_cvt a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    o.x = pack_bf16(a.x * d, a.y * d);
    a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    o.y = pack_bf16(a.x * d, a.y * d);
    a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    o.z = pack_bf16(a.x * d, a.y * d);
    a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    o.w = pack_bf16(a.x * d, a.y * d);
    return o;
}

// words w[i] of lane group g become words w[g] of lane group i
__device__ __forceinline__ void transpose4(u32x4& w) {
    auto a = __builtin_amdgcn_permlane32_swap(w.x, w.z, false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w.y, w.w, false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w.x = c[0];
    w.y = c[1];
    w.z = d[0];
    w.w = d[1];
}

// Sums over the 128-column chunks [c0, c1) of 16 MT rows of x with NT tiles of
// 16 weight rows: acc[mt][nt][i] is row 16 mt + 4 (lane/16) + i of x and weight
// row lane%16 of tile nt.  row: this lane's weight row of each tile (in the
// whole stack); xr: this lane's row lane%16 of each tile of x, or null
// (zeros).  U chunks' loads are in flight at once; columns past K have x = 0
// and read the row's last codes again.
template <int FMT, int MT, int NT, int U>
__device__ __forceinline__ void dot_rows(const PackedW& w, const int64_t (&row)[NT], int c0, int c1,
                                         const uint16_t* const (&xr)[MT], f32x4 (&acc)[MT][NT]) {
    const int g = (threadIdx.x & 63) >> 4;
    const int nseg = w.K >> 5;
    const u32x4 zero = {0, 0, 0, 0}, minus136 = {0xC308C308u, 0xC308C308u, 0xC308C308u, 0xC308C308u};
    for (int c = c0; c < c1; c += U) {
        u32x4 q[U][NT], x[U][MT][4];
        float s[U][NT][FMT == INT_NARROW ? 4 : 1];
        uint32_t d[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int seg = (c + u) * 4 + g, sg = min(seg, nseg - 1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                q[u][n] = *reinterpret_cast<const u32x4*>(w.codes + row[n] * (w.K >> 1) + sg * 16);
                if (FMT == NVFP4)
                    d[u][n] = *reinterpret_cast<const uint16_t*>(w.bcodes + row[n] * (w.K >> 4) + sg * 2);
                else if (FMT == INT_WIDE)
                    s[u][n][0] = w.scale[row[n] * w.spr + min((c + u) * 128, w.K - 1) / w.group];
                else
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[u][n][i] = w.scale[row[n] * w.spr + min((c + u) * 4 + i, nseg - 1) * 32 / w.group];
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = FMT == INT_NARROW ? ((c + u) * 4 + i) * 32 + 8 * g : seg * 32 + 8 * i;
                    x[u][m][i] = xr[m] && c + u < c1 && k < w.K ? *reinterpret_cast<const u32x4*>(xr[m] + k) : zero;
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f32x4 base[MT][FMT == INT_NARROW ? 4 : 1];
            if (FMT != NVFP4)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[u][m][i] = int_order(x[u][m][i]);
                        const f32x4 z = {0, 0, 0, 0};
                        if (FMT == INT_NARROW) base[m][i] = mfma(x[u][m][i], minus136, z);
                        else base[m][0] = mfma(x[u][m][i], minus136, i == 0 ? z : base[m][0]);
                    }
                }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (FMT == INT_NARROW) transpose4(q[u][n]);
                float dd[2];
                if (FMT == NVFP4) {
                    dd[0] = __builtin_amdgcn_cvt_f32_fp8((int)d[u][n], 0);
                    dd[1] = __builtin_amdgcn_cvt_f32_fp8((int)d[u][n], 1);
                }
                f32x4 part[MT];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x4 wv = FMT == NVFP4 ? fp4_words(q[u][n][i], dd[i >> 1]) : int_words(q[u][n][i]);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        if (FMT == NVFP4) {
                            acc[m][n] = mfma(x[u][m][i], wv, acc[m][n]);
                        } else if (FMT == INT_WIDE) {
                            part[m] = mfma(x[u][m][i], wv, i == 0 ? base[m][0] : part[m]);
                        } else {
                            part[m] = mfma(x[u][m][i], wv, base[m][i]);
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                acc[m][n][v] = __builtin_fmaf(part[m][v], s[u][n][i], acc[m][n][v]);
                        }
                    }
                }
                if (FMT == INT_WIDE)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            acc[m][n][v] = __builtin_fmaf(part[m][v], s[u][n][0], acc[m][n][v]);
            }
        }
    }
}

// chunks in flight: the loads' registers
constexpr int flight(int mt, int nt) { return mt * nt <= 2 ? 4 / nt : mt <= 2 ? 2 : 1; }

// The waves' sums of a block added in wave order through LDS: value (m, n, v)
// of lane l at red[wave][(m NT + n) 4 + v][l]; afterwards thread (wave v,
// lane l) calls f(m, n, row 16 m + 4 (l/16) + v of x, column l%16 of the tile, sum).
template <int MT, int NT>
struct Reduce {
    float red[NW][MT * NT * 4][64];
    __device__ __forceinline__ void put(const f32x4 (&acc)[MT][NT]) {
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int v = 0; v < 4; ++v) red[w][(m * NT + n) * 4 + v][lane] = acc[m][n][v];
        __syncthreads();
    }
    __device__ __forceinline__ float get(int m, int n) const {
        const int lane = threadIdx.x & 63, v = threadIdx.x >> 6;
        float s = red[0][(m * NT + n) * 4 + v][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += red[w][(m * NT + n) * 4 + v][lane];
        return s;
    }
};

__device__ __forceinline__ uint16_t bf16_of(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// this wave's share of the 128-column chunks
__device__ __forceinline__ void wave_chunks(int K, int w, int* c0, int* c1) {
    const int n = (K + 127) >> 7, per = (n + NW - 1) / NW;
    *c0 = w * per;
    *c1 = min(n, *c0 + per);
}

// --------------------------------------------------------------- matvec ---
// 16 NT weight rows and 16 MT rows of x per block.  With `which` a block
// belongs to row r of x: it does nothing if an earlier row names the same
// matrix, else it takes every row that does, 16 at a time.
template <int FMT, int MT, int NT>
__global__ __launch_bounds__(64 * NW) void k_matvec(MatvecArgs a) {
    __shared__ Reduce<MT, NT> red;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int n0 = blockIdx.x * 16 * NT;
    int c0, c1;
    wave_chunks(a.w.K, w, &c0, &c1);
    int64_t row[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) row[n] = min((int64_t)n0 + 16 * n + (lane & 15), a.N - 1);
    const int m0 = blockIdx.y * 16 * MT;
    const uint16_t* xr[MT];
    f32x4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = m0 + 16 * m + (lane & 15);
        xr[m] = r < a.M ? a.x + (int64_t)r * a.w.K : nullptr;
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    }
    dot_rows<FMT, MT, NT, flight(MT, NT)>(a.w, row, c0, c1, xr, acc);
    red.put(acc);
    const float t = FMT == NVFP4 ? a.w.tscale[0] : 1.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = m0 + 16 * m + 4 * (lane >> 4) + w;
            const int64_t c = (int64_t)n0 + 16 * n + (lane & 15);
            const float s = red.get(m, n);
            if (r < a.M && c < a.N) a.y[(int64_t)r * a.N + c] = bf16_of(FMT == NVFP4 ? s * t : s);
        }
}

template <int FMT>
__global__ __launch_bounds__(64 * NW) void k_matvec_which(MatvecArgs a) {
    __shared__ Reduce<1, 1> red;
    __shared__ int ids[PACKED_MAX_ROWS], list[PACKED_MAX_ROWS];
    __shared__ int count;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int n0 = blockIdx.x * 16, r0 = blockIdx.y;
    for (int i = threadIdx.x; i < a.M; i += 64 * NW) ids[i] = a.which[i];
    __syncthreads();
    const int e = ids[r0];
    const bool bad = e < 0 || e >= a.E;               // no such matrix: the row is zero
    if (w == 0) {
        int n = 0;
        for (int b = 0; b < a.M; b += 64) {
            const bool hit = b + lane < a.M && ids[b + lane] == e;
            const uint64_t mask = __ballot(hit);
            if (hit) list[n + __popcll(mask & ((1ull << lane) - 1))] = b + lane;
            n += __popcll(mask);
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    if (list[0] != r0) return;                        // an earlier row has this matrix
    int c0, c1;
    wave_chunks(a.w.K, w, &c0, &c1);
    const int64_t row[1] = {(int64_t)(bad ? 0 : e) * a.N + min((int64_t)n0 + (lane & 15), a.N - 1)};
    const float t = FMT == NVFP4 ? a.w.tscale[bad ? 0 : e] : 1.0f;
    for (int b = 0; b < count; b += 16) {
        const uint16_t* xr[1] = {
            b + (lane & 15) < count ? a.x + (int64_t)list[b + (lane & 15)] * a.w.K : nullptr};
        f32x4 acc[1][1] = {{f32x4{0, 0, 0, 0}}};
        if (!bad) dot_rows<FMT, 1, 1, flight(1, 1)>(a.w, row, c0, c1, xr, acc);
        __syncthreads();                              // the last group's sums have been read
        red.put(acc);
        const int m = b + 4 * (lane >> 4) + w;
        const int64_t c = (int64_t)n0 + (lane & 15);
        const float s = red.get(0, 0);
        if (m < count && c < a.N) a.y[(int64_t)list[m] * a.N + c] = bf16_of(FMT == NVFP4 ? s * t : s);
    }
}

// --------------------------------------------------------------- experts ---
__device__ __forceinline__ int clamp_id(int id, int E) { return id < 0 ? 0 : (id >= E ? E - 1 : id); }

// x^ of routed row r = t k + j: x[t] through expert e's input quantiser
template <int KIND>
__device__ __forceinline__ void quant_row(const PackedExpertArgs& a, int r, int e) {
    const uint4* x = reinterpret_cast<const uint4*>(a.x + (int64_t)(r / a.k) * a.H);
    uint4* o = reinterpret_cast<uint4*>(a.xhat + (int64_t)r * a.H);
    const float t = act_t<KIND>(a.a1, e);
    for (int v = threadIdx.x; v < (a.H >> 3); v += blockDim.x) {    // H % 128 == 0: lane pairs are whole
        float f[8], y[8], dfac;
        unpack8(x[v], f);
        float m = amax8(f);
        m = fmaxf(m, __shfl_xor(m, 1));
        quant8<KIND>(f, act_scale_t<KIND>(a.a1, t, m, m, 0.0f, &dfac), a.a1.q.qmin, a.a1.q.qmax, y);
        o[v] = pack8(y);
    }
}

// Block r of the first R: x^ of routed row r (with an input quantiser).  The
// last block: the routed rows sorted by expert (stable), and for each
// expert's first row where its rows start and how many they are (0: not the
// first).  R <= 1024: every row counts the rows before it, ids in LDS.
__global__ __launch_bounds__(1024) void k_packed_prep(PackedExpertArgs a) {
    const int R = a.R;
    if (a.xhat && (int)blockIdx.x < R) {
        const int r = blockIdx.x, e = clamp_id(sload(a.ids, r), a.E);
        if (a.a1.q.kind == K_NVFP4) quant_row<K_NVFP4>(a, r, e);
        else if (a.a1.q.kind == K_FP8) quant_row<K_FP8>(a, r, e);
        else quant_row<K_INT>(a, r, e);
        return;
    }
    __shared__ int ids[PACKED_MAX_ROWS];
    for (int i = threadIdx.x; i < R; i += blockDim.x) ids[i] = clamp_id(a.ids[i], a.E);
    __syncthreads();
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
        const int e = ids[r];
        int less = 0, same = 0, before = 0;
        for (int i = 0; i < R; ++i) {
            const int o = ids[i];
            less += o < e;
            same += o == e;
            before += o == e && i < r;
        }
        a.order[less + before] = r;
        a.start[r] = less;
        a.count[r] = before == 0 ? same : 0;
    }
}

// the rows of the group that routed row r opens: how many, and the i-th
struct Group {
    int count, start;
    const int32_t* order;
    int r;
    __device__ __forceinline__ Group(const PackedExpertArgs& a, int r_) : order(a.order), r(r_) {
        count = order ? sload(a.count, r_) : 1;        // without lists every row is its own group
        start = order ? sload(a.start, r_) : 0;
    }
    __device__ __forceinline__ int at(int i) const { return order ? order[start + i] : r; }
};

// fc1 and SwiGLU: 16 gate rows and their 16 up rows per block; the tile of h
// goes through the second activation quantiser on the way (a 16-block of
// NVFP4 is the tile's row)
template <int FMT>
__global__ __launch_bounds__(64 * NW) void k_packed_fc1(PackedExpertArgs a) {
    __shared__ Reduce<1, 2> red;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int r0 = blockIdx.y, i0 = blockIdx.x * 16;
    const Group gr(a, r0);
    if (gr.count == 0) return;
    const int e = clamp_id(sload(a.ids, r0), a.E);
    int c0, c1;
    wave_chunks(a.H, w, &c0, &c1);
    const int64_t base = (int64_t)e * 2 * a.I + i0 + (lane & 15);
    const int64_t row[2] = {base, base + a.I};
    const float t1 = FMT == NVFP4 ? sload(a.w1.tscale, e) : 1.0f;
    const int kind2 = a.a2.q.kind;
    const float s2 = kind2 != K_NONE ? sload(a.a2.s, e) : 0.0f;
    for (int b = 0; b < gr.count; b += 16) {
        const uint16_t* xr[1] = {nullptr};
        if (b + (lane & 15) < gr.count) {
            const int r = gr.at(b + (lane & 15));
            xr[0] = a.xhat ? a.xhat + (int64_t)r * a.H : a.x + (int64_t)(r / a.k) * a.H;
        }
        f32x4 acc[1][2] = {{f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}}};
        dot_rows<FMT, 1, 2, flight(1, 2)>(a.w1, row, c0, c1, xr, acc);
        __syncthreads();                               // the last group's sums have been read
        red.put(acc);
        const int m = b + 4 * (lane >> 4) + w;
        float gate = red.get(0, 0), up = red.get(0, 1), sig;
        if (FMT == NVFP4) {
            gate *= t1;
            up *= t1;
        }
        uint16_t hb = bf16_of(silu_sig(gate, &sig) * up);
        if (kind2 != K_NONE) {
            const float h = __uint_as_float((uint32_t)hb << 16);
            Div dv;
            float dfac;
            if (kind2 == K_NVFP4) {
                dv.set(act_scale_t<K_NVFP4>(a.a2, s2, group_max(fabsf(h), 16), 0.0f, 0.0f, &dfac));
                hb = bf16_of(quant_elem<K_NVFP4>(h, dv, -6.0f, 6.0f).q * dv.s);
            } else {
                dv.set(s2);
                const Elem q = kind2 == K_FP8 ? quant_elem<K_FP8>(h, dv, -448.0f, 448.0f)
                                              : quant_elem<K_INT>(h, dv, a.a2.q.qmin, a.a2.q.qmax);
                hb = bf16_of(q.q * s2);
            }
        }
        if (m < gr.count) a.h[(int64_t)gr.at(m) * a.I + i0 + (lane & 15)] = hb;
    }
}

// fc2 of one group of rows: y_r in fp32, one row per routed row
template <int FMT>
__global__ __launch_bounds__(64 * NW) void k_packed_fc2(PackedExpertArgs a) {
    __shared__ Reduce<1, 1> red;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int r0 = blockIdx.y, n0 = blockIdx.x * 16;
    const Group gr(a, r0);
    if (gr.count == 0) return;
    const int e = clamp_id(sload(a.ids, r0), a.E);
    int c0, c1;
    wave_chunks(a.I, w, &c0, &c1);
    const int64_t row[1] = {(int64_t)e * a.H + n0 + (lane & 15)};
    const float t2 = FMT == NVFP4 ? sload(a.w2.tscale, e) : 1.0f;
    for (int b = 0; b < gr.count; b += 16) {
        const uint16_t* xr[1] = {
            b + (lane & 15) < gr.count ? a.h + (int64_t)gr.at(b + (lane & 15)) * a.I : nullptr};
        f32x4 acc[1][1] = {{f32x4{0, 0, 0, 0}}};
        dot_rows<FMT, 1, 1, flight(1, 1)>(a.w2, row, c0, c1, xr, acc);
        __syncthreads();
        red.put(acc);
        const int m = b + 4 * (lane >> 4) + w;
        const float s = red.get(0, 0);
        if (m < gr.count) a.yr[(int64_t)gr.at(m) * a.H + n0 + (lane & 15)] = FMT == NVFP4 ? s * t2 : s;
    }
}

// y[t] = sum over the slots of w y_r, ascending
__global__ __launch_bounds__(256) void k_packed_combine(PackedExpertArgs a) {
    const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.H) return;
    float s = 0.0f;
    for (int j = 0; j < a.k; ++j) s = __builtin_fmaf(a.tw[t * a.k + j], a.yr[(int64_t)(t * a.k + j) * a.H + c], s);
    a.y[(int64_t)t * a.H + c] = bf16_of(s);
}

template <int FMT>
hipError_t run_matvec(const MatvecArgs& a, hipStream_t st) {
    const unsigned nb = (unsigned)((a.N + 15) / 16);
    if (a.which) {
        hipLaunchKernelGGL(k_matvec_which<FMT>, dim3(nb, (unsigned)a.M), dim3(64 * NW), 0, st, a);
    } else if (a.M <= 16) {
        hipLaunchKernelGGL((k_matvec<FMT, 1, 1>), dim3(nb, 1), dim3(64 * NW), 0, st, a);
    } else if (a.M <= 32) {
        hipLaunchKernelGGL((k_matvec<FMT, 2, 1>), dim3(nb, 1), dim3(64 * NW), 0, st, a);
    } else {
        hipLaunchKernelGGL((k_matvec<FMT, 4, 1>), dim3(nb, (unsigned)((a.M + 63) / 64)), dim3(64 * NW), 0, st, a);
    }
    return hipGetLastError();
}

template <int FMT>
hipError_t run_fc1(const PackedExpertArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(k_packed_fc1<FMT>, dim3((unsigned)(a.I / 16), (unsigned)a.R), dim3(64 * NW), 0, st, a);
    return hipGetLastError();
}
template <int FMT>
hipError_t run_fc2(const PackedExpertArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(k_packed_fc2<FMT>, dim3((unsigned)(a.H / 16), (unsigned)a.R), dim3(64 * NW), 0, st, a);
    return hipGetLastError();
}

int fmt_of(const PackedW& w) { return w.bcodes ? NVFP4 : w.group >= 128 ? INT_WIDE : INT_NARROW; }

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, hipStream_t st) {
    switch (fmt_of(a.w)) {
    case NVFP4: return run_matvec<NVFP4>(a, st);
    case INT_WIDE: return run_matvec<INT_WIDE>(a, st);
    default: return run_matvec<INT_NARROW>(a, st);
    }
}

hipError_t launch_packed_expert(const PackedExpertArgs& a, hipStream_t st) {
    if (a.xhat || a.order) {
        const unsigned blocks = (a.xhat ? (unsigned)a.R : 0u) + (a.order ? 1u : 0u);
        hipLaunchKernelGGL(k_packed_prep, dim3(blocks), dim3(a.order ? 1024 : 256), 0, st, a);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    const int f1 = fmt_of(a.w1), f2 = fmt_of(a.w2);
    hipError_t err = f1 == NVFP4 ? run_fc1<NVFP4>(a, st) : f1 == INT_WIDE ? run_fc1<INT_WIDE>(a, st)
                                                                          : run_fc1<INT_NARROW>(a, st);
    if (err != hipSuccess) return err;
    err = f2 == NVFP4 ? run_fc2<NVFP4>(a, st) : f2 == INT_WIDE ? run_fc2<INT_WIDE>(a, st) : run_fc2<INT_NARROW>(a, st);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(k_packed_combine, dim3((unsigned)((a.H + 255) / 256), (unsigned)(a.R / a.k)), dim3(256), 0, st,
                       a);
    return hipGetLastError();
}

}  // namespace fq
