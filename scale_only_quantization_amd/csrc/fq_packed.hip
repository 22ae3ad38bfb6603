// Products of packed 4-bit weights with a few rows, and the routed SwiGLU
// expert layer on packed weights for a few tokens.
//
//   y[m, n] = sum_k x[m, k] W[n, k],  W = q s (INT4, a scale per row or group)
//                                     W = q d t (NVFP4: E2M1, E4M3 per 16, fp32 per matrix)
// A few rows against megabytes of weights: what counts is the stream of codes
// from HBM, so one pass over them serves as many rows of x as the kernel holds
// (32; of one matrix among several 16; in the layer up to 8, fewer of long rows:
// lds_rows), and all vector work per code is kept under the 2.5 operations a CU
// has per code at the full HBM rate.  More rows take further passes, which load
// and convert the codes again.  The
// products themselves go to the matrix cores (v_mfma_f32_16x16x32_bf16, 16
// rows of x by 16 rows of W; unused rows of x cost nothing that counts): codes
// become bf16 exactly, x is bf16, sums are fp32.
//   INT4   v_and_or forms 128 + (q ^ 8) = 136 + q in bf16, two at a time, one
//          operation per code; a product of x with the constant -136, shared
//          by the wave's weight tiles, starts the sum and takes the 136 off
//          again in fp32.  The scale multiplies the sum of its group.
//   NVFP4  q d is exact in bf16 (2 + 4 significant bits): two conversions and
//          two products per pair of codes; t multiplies the end.
// A lane loads 16 bytes, 32 codes, of one weight row; the four words of the
// four lanes that hold a row's 128 columns (a chunk) are then transposed
// between them (four lane swaps), so that product i covers columns 32 i ..
// 32 i + 31 and its operand of x is 64 consecutive bytes of each row.
// KW waves of a block share a tile's columns and add their sums in order.  A
// wave holds x of a slab of four chunks in registers while NT tiles of weight
// rows pass, the next tile's codes in flight.  Reading x again for every tile
// cost more than the codes (13 rows by 12289 x 8192 in NVFP4: 37 us, of which
// 22 were x through the L2, against 15 for codes and scales alone); and the
// scales of a slab are one load, a lane group per chunk, spread by lane swaps
// (a load per chunk touches 16 cache lines for 128 bytes: 6 us of those 15).
// All loads go through buffer resources, and rows past the end read as zero
// without a branch.  In the layer a load's offset is a lane's constant plus a
// scalar; in the products the wave's index reaches the chunk as a vector value,
// and the compiler puts most loads (41 of the 61 of k_matvec<NVFP4, 1, 4, 8>, all
// in INT4) in a loop over the lanes' offsets that passes once.
// Measured: 13 rows by 12289 x 8192 in NVFP4 21 us (2.7 TB/s; a large read 6.1);
// one row by 2048 x 2048 in INT4 4.4 us in the kernel, latency; 4096 x 4096 in
// INT4 17 rows 10.8 us, 64 13.4, 256 47, 1024 183; the layer of 128 experts, 2048
// by 768, top-8: one token in INT4 16.6 us (fc1 8, fc2 6, combine 4), in NVFP4
// 21-23, 16 tokens in NVFP4 74-77 us (fc1 41, 3.8 TB/s, fc2 24), bound by the
// chains of dependent loads of blocks that pass few slabs each, and by the
// conversions (in INT4 68 us); 8 experts of 2048 by 1024, top-8, 32 tokens, five
// passes over the codes: 74 and 70 us.
#include <cmath>
#include <type_traits>

#include "fq_act.h"
#include "fq_mfma.h"
#include "fq_ops.h"

namespace fq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

enum Fmt { INT_WIDE = 0, INT_NARROW = 1, NVFP4 = 2 };

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

constexpr int FC2_KW = 2;                 // waves that split fc2's columns
constexpr int WV = 4;                     // waves of a block of the expert layer
constexpr int XC = 4;                     // chunks of a slab: one per lane group in the scales' load

// A run of weight rows as buffer resources; rows past its end read as zero.
template <int FMT>
struct Rows {
    __amdgpu_buffer_rsrc_t codes, scale;             // scale: INT scales or NVFP4 block codes
    uint32_t vc, vs;                                 // this lane's offsets: row lane%16, its quarter of a chunk
    uint32_t cb, sb;                                 // bytes per row
    __device__ __forceinline__ Rows(const PackedW& w, int64_t row0, int64_t rows) {
        const int lane = threadIdx.x & 63;
        cb = (uint32_t)w.K >> 1;
        sb = FMT == NVFP4 ? (uint32_t)w.K >> 4 : (uint32_t)w.spr * 4;
        codes = make_rsrc(w.codes + row0 * cb, rows * cb);
        scale = FMT == NVFP4 ? make_rsrc(w.bcodes + row0 * sb, rows * sb) : make_rsrc(w.scale + row0 * w.spr, rows * sb);
        vc = (lane & 15) * cb + (lane >> 4) * 16;
        vs = (lane & 15) * sb;
    }
};

// The value that each lane group (16 lanes) g holds, given to all lanes: o[g].
__device__ __forceinline__ void spread4(uint32_t v, uint32_t (&o)[4]) {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);         // groups 0 1 0 1 and 2 3 2 3
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    o[0] = a[0];
    o[1] = a[1];
    o[2] = b[0];
    o[3] = b[1];
}

// The eight block codes of a chunk: one load where they are 8-byte aligned, else
// (rows of any even number of them, or a stack that begins between) one per two.
__device__ __forceinline__ u32x2 load_factors(const PackedW& w, __amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t os) {
    if (w.b8) return __builtin_amdgcn_raw_buffer_load_b64(rs, at, os, 0);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __builtin_amdgcn_raw_buffer_load_b16(rs, at + 2 * i, os, 0);
    return u32x2{h[0] | h[1] << 16, h[2] | h[3] << 16};
}

// A slab of a tile's codes and scales, as loaded.
template <int FMT>
struct Slab {
    static constexpr int NS = FMT == NVFP4 ? 2 : FMT == INT_WIDE ? 1 : 4;        // scale words of a chunk
    u32x4 q[XC];
    uint32_t s[NS];                                  // of chunk c + lane group
    __device__ __forceinline__ void load(const PackedW& w, const Rows<FMT>& r, int row, int c) {
        const uint32_t oc = row * r.cb + c * 64, os = row * r.sb;
        const int cg = c + ((threadIdx.x & 63) >> 4);
#pragma unroll
        for (int u = 0; u < XC; ++u) q[u] = __builtin_amdgcn_raw_buffer_load_b128(r.codes, r.vc, oc + u * 64, 0);
        if (FMT == NVFP4) {
            const u32x2 v = load_factors(w, r.scale, r.vs + cg * 8, os);
            s[0] = v.x;
            s[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < NS; ++i)
                s[i] = __builtin_amdgcn_raw_buffer_load_b32(r.scale, r.vs + ((cg * NS + i) >> w.gshift) * 4, os, 0);
        }
    }
};

// acc[n][m] += 16 rows m of x times tile n's slab of chunks c .. c + 3:
// acc[n][m][v] is row 16 m + 4 (lane/16) + v of x, weight row lane%16.  x(u, o)
// fills o[m][i] with the operands of chunk u's products i (columns 32 i + 8
// (lane/16) .. + 7; INT: in int_order).  base(o, u, m): INT_WIDE, the chunk's
// sum of x times -136.
template <int FMT, int MT, int NT, typename X, typename B>
__device__ __forceinline__ void add_slab(Slab<FMT> (&k)[NT], int c, int nseg, X&& x, B&& base, f32x4 (&acc)[NT][MT]) {
    const int g = (threadIdx.x & 63) >> 4;
    const f32x4 z = {0, 0, 0, 0};
    const u32x4 minus136 = {0xC308C308u, 0xC308C308u, 0xC308C308u, 0xC308C308u};
    uint32_t sc[NT][Slab<FMT>::NS][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < Slab<FMT>::NS; ++i) spread4(k[n].s[i], sc[n][i]);
#pragma unroll
    for (int u = 0; u < XC; ++u) {
        if ((c + u) * 4 >= nseg) continue;            // past the row's end
        u32x4 xu[MT][4];
        x(u, xu);
        f32x4 b[MT];
        if (FMT == INT_WIDE)
#pragma unroll
            for (int m = 0; m < MT; ++m) b[m] = base(xu[m], u, m);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            transpose4(k[n].q[u]);
            float dd[4];
            if (FMT == NVFP4) {                       // word i is the g-th quarter of segment i: block 2 i + g/2
                const int sh = 4 * (g & 2);
                const int d0 = (int)(sc[n][0][u] >> sh), d1 = (int)(sc[n][1 % Slab<FMT>::NS][u] >> sh);
                dd[0] = __builtin_amdgcn_cvt_f32_fp8(d0, 0);
                dd[1] = __builtin_amdgcn_cvt_f32_fp8(d0, 2);
                dd[2] = __builtin_amdgcn_cvt_f32_fp8(d1, 0);
                dd[3] = __builtin_amdgcn_cvt_f32_fp8(d1, 2);
                if ((c + u) * 4 + 4 > nseg)           // another row's factors: zero, not a NaN for zero times it
#pragma unroll
                    for (int i = 1; i < 4; ++i) dd[i] = (c + u) * 4 + i < nseg ? dd[i] : 0.0f;
            }
            f32x4 part[MT];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4 wv = FMT == NVFP4 ? fp4_words(k[n].q[u][i], dd[i]) : int_words(k[n].q[u][i]);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (FMT == NVFP4) {
                        acc[n][m] = mfma(xu[m][i], wv, acc[n][m]);
                    } else if (FMT == INT_WIDE) {
                        part[m] = mfma(xu[m][i], wv, i == 0 ? b[m] : part[m]);
                    } else {
                        part[m] = mfma(xu[m][i], wv, mfma(xu[m][i], minus136, z));
                        // past the row's end: zero, as the next row's scale may be a NaN
                        const float s = (c + u) * 4 + i < nseg ? __uint_as_float(sc[n][i % Slab<FMT>::NS][u]) : 0.0f;
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[n][m][v] = __builtin_fmaf(part[m][v], s, acc[n][m][v]);
                    }
                }
            }
            if (FMT == INT_WIDE) {
                const float s = __uint_as_float(sc[n][0][u]);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[n][m][v] = __builtin_fmaf(part[m][v], s, acc[n][m][v]);
            }
        }
    }
}

// 16 MT rows of x (resource xs, this lane's row lane%16 of tile m at vx[m])
// times NT tiles of 16 weight rows that start at rows row(n) of r, over this
// wave's slabs kp, kp + KW, ... of the columns, x of a slab in registers.  The
// order of a row's sum does not depend on MT or NT.
template <int FMT, int MT, int NT, int KW, typename R>
__device__ __forceinline__ void dot_rows(const PackedW& w, const Rows<FMT>& r, R&& row, int kp,
                                         __amdgpu_buffer_rsrc_t xs, const uint32_t (&vx)[MT], f32x4 (&acc)[NT][MT]) {
    const int nseg = w.K >> 5, nch = (nseg + 3) >> 2;
    const f32x4 z = {0, 0, 0, 0};
    const u32x4 zero = {0, 0, 0, 0}, minus136 = {0xC308C308u, 0xC308C308u, 0xC308C308u, 0xC308C308u};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = z;
    Slab<FMT> sl[2][1];
    if (kp * XC < nch) sl[0][0].load(w, r, row(0), kp * XC);
    for (int c = kp * XC; c < nch; c += KW * XC) {
        u32x4 x[MT][XC][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int u = 0; u < XC; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[m][u][i] = __builtin_amdgcn_raw_buffer_load_b128(xs, vx[m], c * 256 + u * 256 + i * 64, 0);
        if ((c + XC) * 4 > nseg)                      // the row ends inside the slab
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int u = 0; u < XC; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((c + u) * 4 + i >= nseg) x[m][u][i] = zero;
        f32x4 base[MT][XC];
        if (FMT != NVFP4)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int u = 0; u < XC; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[m][u][i] = int_order(x[m][u][i]);
                        if (FMT == INT_WIDE) base[m][u] = mfma(x[m][u][i], minus136, i == 0 ? z : base[m][u]);
                    }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n + 1 < NT) sl[(n + 1) & 1][0].load(w, r, row(n + 1), c);
            else if (c + KW * XC < nch) sl[(n + 1) & 1][0].load(w, r, row(0), c + KW * XC);
            __builtin_amdgcn_sched_barrier(0);        // in flight before this tile's products
            add_slab<FMT, MT, 1>(
                sl[n & 1], c, nseg,
                [&](int u, u32x4 (&o)[MT][4]) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[m][i] = x[m][u][i];
                },
                [&](const u32x4 (&)[4], int u, int m) { return base[m][u]; },
                reinterpret_cast<f32x4 (&)[1][MT]>(acc[n]));
        }
        if (NT & 1) sl[0][0] = sl[1][0];              // the next slab's first tile
    }
}

// Rows of x in LDS, shared by a block's waves: K columns (a multiple of 128) at
// a stride of K + 8, so that 16 rows of one column fall on distinct banks;
// INT: each 8 columns in int_order.
template <int FMT>
struct XLds {
    lds_t* p;
    uint32_t stride;                                  // bytes
    __device__ __forceinline__ static uint32_t bytes_per_row(int K) { return K * 2 + 16; }
    // rows 0 .. n - 1 from src(i), by the whole block
    template <typename S>
    __device__ __forceinline__ void fill(int K, int n, S&& src) {
        for (int m = 0; m < n; ++m) {
            const uint16_t* row = src(m);             // uniform
            for (int v = threadIdx.x; v < K >> 3; v += blockDim.x) {
                u32x4 x = *reinterpret_cast<const u32x4*>(row + v * 8);
                if (FMT != NVFP4) x = int_order(x);
                *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(p + m * stride + v * 16) = x;
            }
        }
    }
};

// For rows of x in LDS: two tiles of 16 weight rows that start at rows row0 and
// row1 of a resource, up to 8 rows of x.  A load reads 128 bytes of each of 8
// weight rows, two chunks, whole cache lines (in 64-byte pieces of 16 rows fc1
// of 16 tokens took 41 us in NVFP4 and 38 in INT4, with these 39 and 35): lane
// n = lane%16 holds a quarter of chunk n%2 of row n/2 of those 8.  So that the
// chunks need no exchange between lanes, rows 0-7 of the product's x are the
// rows' even chunk and rows 8-15 their odd one: of the product, even n have
// their sum in rows 0-7 and odd n theirs in rows 8-15, the other half is of no
// meaning, and lanes 33 apart (in exclusive or) hold a weight row's two sums.
template <int FMT>
struct PairRows {
    __amdgpu_buffer_rsrc_t codes, scale;
    uint32_t vc, vs, cb, sb;
    __device__ __forceinline__ PairRows(const PackedW& w, int64_t row0, int64_t rows) {
        const int n = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
        cb = (uint32_t)w.K >> 1;
        sb = FMT == NVFP4 ? (uint32_t)w.K >> 4 : (uint32_t)w.spr * 4;
        codes = make_rsrc(w.codes + row0 * cb, rows * cb);
        scale = FMT == NVFP4 ? make_rsrc(w.bcodes + row0 * sb, rows * sb) : make_rsrc(w.scale + row0 * w.spr, rows * sb);
        vc = (n >> 1) * cb + (n & 1) * 64 + g * 16;
        vs = (8 * (g & 1) + (n >> 1)) * sb;
    }
};

// Four chunks of a tile: q[2 p + h] is of chunks c + 2 p + n%2 of rows 8 h ..
// 8 h + 7; lane group g loads the scales that go with q[g].
template <int FMT>
struct PairSlab {
    static constexpr int NS = Slab<FMT>::NS;
    u32x4 q[XC];
    uint32_t s[NS];
    __device__ __forceinline__ void load(const PackedW& w, const PairRows<FMT>& r, int row, int c) {
        const uint32_t oc = row * r.cb + c * 64, os = row * r.sb;
        const int cg = c + 2 * ((threadIdx.x & 63) >> 5) + (threadIdx.x & 1);
#pragma unroll
        for (int u = 0; u < XC; ++u)
            q[u] = __builtin_amdgcn_raw_buffer_load_b128(r.codes, r.vc, oc + (u >> 1) * 128 + (u & 1) * 8 * r.cb, 0);
        if (FMT == NVFP4) {
            const u32x2 v = load_factors(w, r.scale, r.vs + cg * 8, os);
            s[0] = v.x;
            s[NS - 1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < NS; ++i)
                s[i] = __builtin_amdgcn_raw_buffer_load_b32(r.scale, r.vs + ((cg * NS + i) >> w.gshift) * 4, os, 0);
        }
    }
};

// acc[n][h] += rows of x times tile n's rows 8 h .. 8 h + 7, chunks c .. c + 3
// of nch.  xp + xo: this lane's row of x, its quarter of a 32-column segment.
template <int FMT>
__device__ __forceinline__ void add_pairs(PairSlab<FMT> (&k)[2], int c, int nch, const lds_t* xp, uint32_t xo,
                                          f32x4 (&acc)[2][2]) {
    constexpr int NS = Slab<FMT>::NS;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const f32x4 z = {0, 0, 0, 0};
    const u32x4 zero = {0, 0, 0, 0}, minus136 = {0xC308C308u, 0xC308C308u, 0xC308C308u, 0xC308C308u};
    uint32_t sc[2][NS][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < NS; ++i) spread4(k[n].s[i], sc[n][i]);
#pragma unroll
    for (int p = 0; p < XC / 2; ++p) {
        const int cp = c + 2 * p;
        if (cp >= nch) continue;                      // past the row's end
        const bool half = cp + 1 >= nch;              // the row ends between the chunks: x and factors of the odd one zero
        const uint32_t at = xo + cp * 256 + (!half && (lane & 8) ? 256 : 0);
        u32x4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(xp + at + i * 64);
        }
        if (half) {
            asm volatile("");                         // a branch, not selects on every step
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = lane & 8 ? zero : x[i];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) sc[n][i][2 * p + h] = lane & 1 ? 0 : sc[n][i][2 * p + h];
        }
        f32x4 b = z;
        if (FMT == INT_WIDE)
#pragma unroll
            for (int i = 0; i < 4; ++i) b = mfma(x[i], minus136, b);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int u = 2 * p + h;
                transpose4(k[n].q[u]);
                float dd[4];
                if (FMT == NVFP4) {                   // word i is the g-th quarter of segment i: block 2 i + g/2
                    const int sh = 4 * (g & 2);
                    const int d0 = (int)(sc[n][0][u] >> sh), d1 = (int)(sc[n][NS - 1][u] >> sh);
                    dd[0] = __builtin_amdgcn_cvt_f32_fp8(d0, 0);
                    dd[1] = __builtin_amdgcn_cvt_f32_fp8(d0, 2);
                    dd[2] = __builtin_amdgcn_cvt_f32_fp8(d1, 0);
                    dd[3] = __builtin_amdgcn_cvt_f32_fp8(d1, 2);
                }
                f32x4 part = b;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x4 wv = FMT == NVFP4 ? fp4_words(k[n].q[u][i], dd[i]) : int_words(k[n].q[u][i]);
                    if (FMT == NVFP4) {
                        acc[n][h] = mfma(x[i], wv, acc[n][h]);
                    } else if (FMT == INT_WIDE) {
                        part = mfma(x[i], wv, part);
                    } else {
                        part = mfma(x[i], wv, mfma(x[i], minus136, z));
                        const float s = __uint_as_float(sc[n][i % NS][u]);
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[n][h][v] = __builtin_fmaf(part[v], s, acc[n][h][v]);
                    }
                }
                if (FMT == INT_WIDE) {
                    const float s = __uint_as_float(sc[n][0][u]);
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[n][h][v] = __builtin_fmaf(part[v], s, acc[n][h][v]);
                }
            }
    }
}

// Of the sums in `run`'s result, a lane has tile n's row pair_col() and rows
// 4 (lane/16 % 2) + v of x, if pair_has().
__device__ __forceinline__ int pair_col() { return 8 * (threadIdx.x & 1) + ((threadIdx.x & 15) >> 1); }
__device__ __forceinline__ bool pair_has() { return ((threadIdx.x >> 5) & 1) == (threadIdx.x & 1); }
__device__ __forceinline__ int pair_row() { return 4 * ((threadIdx.x >> 4) & 1); }

// The columns are split into VW shares (slabs s, s + VW, ... each), whose sums
// are added in order.  SHARE: this wave has the one share `s`; else it takes
// all of them in turn, with the same bits.  begin() sends the first slab's
// loads, before the rows of x are there.  One slab is in registers at a time: a
// second one (the next slab's loads during this one's products) took the
// registers that hold a fourth wave per SIMD, which was slower (fc1 of 16 tokens
// in NVFP4: 58 us against 45 then).
template <int FMT, int VW, bool SHARE>
struct DotLds {
    const PackedW& w;
    const PairRows<FMT>& r;
    int row0, row1, s;
    PairSlab<FMT> sl[2];
    __device__ __forceinline__ void load(int c) {
        sl[0].load(w, r, row0, c);
        sl[1].load(w, r, row1, c);
    }
    __device__ __forceinline__ void begin(int share) {
        s = share;
        if (s * XC * 128 < w.K) load(s * XC);
    }
    __device__ __forceinline__ void run(const lds_t* xp, uint32_t xo, f32x4 (&sum)[2]) {
        const f32x4 z = {0, 0, 0, 0};
        const int nch = w.K >> 7;
        const bool odd = threadIdx.x & 1;
        sum[0] = sum[1] = z;
        for (int v = s; v < (SHARE ? s + 1 : VW); ++v) {
            f32x4 acc[2][2] = {{z, z}, {z, z}};
            for (int c = v * XC; c < nch; c += VW * XC) {
                add_pairs<FMT>(sl, c, nch, xp, xo, acc);
                const int next = c + VW * XC < nch ? c + VW * XC : SHARE ? nch : (v + 1) * XC;
                if (next < nch) load(next);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[n][i] += (odd ? acc[n][1][i] : acc[n][0][i]) + __shfl_xor(odd ? acc[n][0][i] : acc[n][1][i], 33);
        }
    }
};

// A barrier that waits for this wave's LDS accesses but not for its loads from memory.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The KW waves' sums of a block's tiles, added in wave order through LDS.  Of
// tile n and 16 rows m of x, thread (lane, v) gets row 16 m + 4 (lane/16) + v
// and weight row lane%16.
template <int MT, int NT, int KW>
struct Reduce {
    float red[KW][MT * NT * 4][64];
    __device__ __forceinline__ void put(const f32x4 (&acc)[NT][MT]) {
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int v = 0; v < 4; ++v) red[w][(m * NT + n) * 4 + v][lane] = acc[n][m][v];
        __syncthreads();
    }
    __device__ __forceinline__ float get(int m, int n, int v) const {
        const int lane = threadIdx.x & 63;
        float s = red[0][(m * NT + n) * 4 + v][lane];
#pragma unroll
        for (int w = 1; w < KW; ++w) s += red[w][(m * NT + n) * 4 + v][lane];
        return s;
    }
};

__device__ __forceinline__ uint16_t bf16_of(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// --------------------------------------------------------------- matvec ---
// 16 NT weight rows and 16 MT rows of x per block.
template <int FMT, int MT, int NT, int KW>
__global__ __launch_bounds__(64 * KW) void k_matvec(MatvecArgs a) {
    __shared__ Reduce<MT, NT, KW> red;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n0 = block_id() * 16 * NT;
    const int m0 = blockIdx.y * 16 * MT;
    uint32_t vx[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) vx[m] = (16 * m + (lane & 15)) * (uint32_t)a.w.K * 2 + (lane >> 4) * 16;
    f32x4 acc[NT][MT];
    dot_rows<FMT, MT, NT, KW>(
        a.w, Rows<FMT>(a.w, n0, min((int64_t)16 * NT, a.N - n0)), [](int n) { return 16 * n; }, w,
        make_rsrc(a.x + (int64_t)m0 * a.w.K, (int64_t)(a.M - m0) * a.w.K * 2), vx, acc);
    red.put(acc);
    const float t = FMT == NVFP4 ? a.w.tscale[0] : 1.0f;
    for (int i = w; i < MT * NT * 4; i += KW) {
        const int m = (i >> 2) / NT, n = (i >> 2) % NT, v = i & 3;
        const int r = m0 + 16 * m + 4 * (lane >> 4) + v;
        const int64_t c = n0 + 16 * n + (lane & 15);
        const float s = red.get(m, n, v);
        if (r < a.M && c < a.N) a.y[(int64_t)r * a.N + c] = bf16_of(FMT == NVFP4 ? s * t : s);
    }
}

// With `which`: a block belongs to row r of x.  It does nothing if an earlier
// row names the same matrix, else it takes every row that does, 16 at a time.
template <int FMT, int KW>
__global__ __launch_bounds__(64 * KW) void k_matvec_which(MatvecArgs a) {
    __shared__ Reduce<1, 1, KW> red;
    __shared__ int ids[PACKED_MAX_ROWS], list[PACKED_MAX_ROWS];
    __shared__ int count;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r0 = blockIdx.y;
    const int64_t n0 = block_id() * 16;
    for (int i = threadIdx.x; i < a.M; i += 64 * KW) ids[i] = a.which[i];
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
    const float t = bad ? 0.0f : FMT == NVFP4 ? a.w.tscale[e] : 1.0f;
    const Rows<FMT> rows(a.w, (int64_t)(bad ? 0 : e) * a.N + n0, min((int64_t)16, a.N - n0));
    const __amdgpu_buffer_rsrc_t xs = make_rsrc(a.x, (int64_t)a.M * a.w.K * 2);
    for (int b = 0; b < count; b += 16) {
        const uint32_t vx[1] = {(uint32_t)list[min(b + (lane & 15), count - 1)] * (uint32_t)a.w.K * 2 + (lane >> 4) * 16};
        f32x4 acc[1][1];
        dot_rows<FMT, 1, 1, KW>(a.w, rows, [](int) { return 0; }, w, xs, vx, acc);
        red.put(acc);
        for (int v = w; v < 4; v += KW) {
            const int m = b + 4 * (lane >> 4) + v;
            const int64_t c = n0 + (lane & 15);
            const float s = bad ? 0.0f : red.get(0, 0, v);
            if (m < count && c < a.N) a.y[(int64_t)list[m] * a.N + c] = bf16_of(FMT == NVFP4 ? s * t : s);
        }
        __syncthreads();                              // read before the next rows' sums
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
    __device__ __forceinline__ int at_uniform(int i) const { return order ? sload(order, start + i) : r; }
};

// The sums of a team of KW waves for two tiles: value i = 4 tile + v of lane l
// at red[wave][i][l], added in wave order.
template <int KW>
__device__ __forceinline__ void team_put(float (*red)[8][64], const f32x4 (&sum)[2]) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        red[w][v][lane] = sum[0][v];
        red[w][4 + v][lane] = sum[1][v];
    }
    lds_barrier();
}
template <int KW>
__device__ __forceinline__ float team_get(float (*red)[8][64], int i) {
    const int lane = threadIdx.x & 63, w0 = (threadIdx.x >> 6) / KW * KW;
    float s = red[w0][i][lane];
#pragma unroll
    for (int o = 1; o < KW; ++o) s += red[w0 + o][i][lane];
    return s;
}

// fc1 and SwiGLU of one group of rows: 16 gate rows and their 16 up rows per
// block, the waves splitting the columns (SHARE), or per wave.  `cap` rows of
// x at a time are in LDS.  The tile of h goes through the second activation
// quantiser on the way (a 16-block of NVFP4 is the tile's row).
template <int FMT, bool SHARE>
__global__ __launch_bounds__(64 * WV) __attribute__((amdgpu_waves_per_eu(FMT == INT_NARROW ? 3 : 4))) void k_packed_fc1(
    PackedExpertArgs a, int cap) {
    extern __shared__ __attribute__((aligned(16))) char dyn[];
    __shared__ float red[SHARE ? WV : 1][8][64];
    const int lane = threadIdx.x & 63, w = wave_id();
    const int r0 = blockIdx.y, i0 = SHARE ? blockIdx.x * 16 : (blockIdx.x * WV + w) * 16;    // I is a multiple of 128
    const Group gr(a, r0);
    if (gr.count == 0) return;
    const int e = clamp_id(sload(a.ids, r0), a.E);
    const PairRows<FMT> rows(a.w1, (int64_t)e * 2 * a.I, 2 * a.I);
    const float t1 = FMT == NVFP4 ? sload(a.w1.tscale, e) : 1.0f;
    const int kind2 = a.a2.q.kind;
    const float s2 = kind2 != K_NONE ? sload(a.a2.s, e) : 0.0f;
    XLds<FMT> x{(lds_t*)dyn, XLds<FMT>::bytes_per_row(a.H)};
    DotLds<FMT, WV, SHARE> dot{a.w1, rows, i0, i0 + a.I};
    for (int b = 0; b < gr.count; b += cap) {
        const int n = min(cap, gr.count - b);
        dot.begin(SHARE ? w : 0);
        if (b > 0) lds_barrier();                      // the last rows and sums have been read
        x.fill(a.H, n, [&](int m) {
            const int r = gr.at_uniform(b + m);
            return a.xhat ? a.xhat + (int64_t)r * a.H : a.x + (int64_t)(r / a.k) * a.H;
        });
        lds_barrier();
        f32x4 sum[2];
        dot.run(x.p, (uint32_t)min(lane & 7, n - 1) * x.stride + (lane >> 4) * 16, sum);
        auto store = [&](int v, float gate, float up) {
            const int m = pair_row() + v;
            const bool mine = pair_has() && m < n;
            float sig;
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
                    float top = group_max(mine ? fabsf(h) : 0.0f, 16);       // the tile's row is in two half waves
                    top = fmaxf(top, __shfl_xor(top, 32));
                    dv.set(act_scale_t<K_NVFP4>(a.a2, s2, top, 0.0f, 0.0f, &dfac));
                    hb = bf16_of(quant_elem<K_NVFP4>(h, dv, -6.0f, 6.0f).q * dv.s);
                } else {
                    dv.set(s2);
                    const Elem q = kind2 == K_FP8 ? quant_elem<K_FP8>(h, dv, -448.0f, 448.0f)
                                                  : quant_elem<K_INT>(h, dv, a.a2.q.qmin, a.a2.q.qmax);
                    hb = bf16_of(q.q * s2);
                }
            }
            if (mine) a.h[(int64_t)gr.at(b + m) * a.I + i0 + pair_col()] = hb;
        };
        if constexpr (SHARE) {
            team_put<WV>(red, sum);
            store(w, team_get<WV>(red, w), team_get<WV>(red, 4 + w));
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (v < n) store(v, sum[0][v], sum[1][v]);
        }
    }
}

// fc2 of one group of rows: y_r in fp32, one row per routed row; 32 columns of
// y per pair of waves, or (not SHARE) per wave
template <int FMT, bool SHARE>
__global__ __launch_bounds__(64 * WV) __attribute__((amdgpu_waves_per_eu(FMT == INT_NARROW ? 3 : 4))) void k_packed_fc2(
    PackedExpertArgs a, int cap) {
    constexpr int KW = SHARE ? FC2_KW : 1;
    extern __shared__ __attribute__((aligned(16))) char dyn[];
    __shared__ float red[SHARE ? WV : 1][8][64];
    const int lane = threadIdx.x & 63, w = wave_id();
    const int r0 = blockIdx.y, n0 = (blockIdx.x * (WV / KW) + w / KW) * 32;      // H is a multiple of 128
    const Group gr(a, r0);
    if (gr.count == 0) return;
    const int e = clamp_id(sload(a.ids, r0), a.E);
    const PairRows<FMT> rows(a.w2, (int64_t)e * a.H, a.H);
    const float t2 = FMT == NVFP4 ? sload(a.w2.tscale, e) : 1.0f;
    XLds<FMT> x{(lds_t*)dyn, XLds<FMT>::bytes_per_row(a.I)};
    DotLds<FMT, FC2_KW, SHARE> dot{a.w2, rows, n0, n0 + 16};
    for (int b = 0; b < gr.count; b += cap) {
        const int n = min(cap, gr.count - b);
        dot.begin(SHARE ? w % KW : 0);
        if (b > 0) lds_barrier();
        x.fill(a.I, n, [&](int m) { return a.h + (int64_t)gr.at_uniform(b + m) * a.I; });
        lds_barrier();
        f32x4 sum[2];
        dot.run(x.p, (uint32_t)min(lane & 7, n - 1) * x.stride + (lane >> 4) * 16, sum);
        auto store = [&](int i, float s) {             // value 4 tile + v of this lane
            const int m = pair_row() + (i & 3);
            if (pair_has() && m < n)
                a.yr[(int64_t)gr.at(b + m) * a.H + n0 + 16 * (i >> 2) + pair_col()] = FMT == NVFP4 ? s * t2 : s;
        };
        if constexpr (SHARE) {
            team_put<KW>(red, sum);
#pragma unroll
            for (int j = 0; j < 4; ++j) store(j * KW + w % KW, team_get<KW>(red, j * KW + w % KW));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) store(i, sum[i >> 2][i & 3]);
        }
    }
}

// y[t] = sum over the slots of w y_r, ascending.  (A launch less for one token,
// with a token's slots side by side in blocks of sixteen waves, took 20.9 us
// where the two take 17.8.)
__global__ __launch_bounds__(256) void k_packed_combine(PackedExpertArgs a) {
    const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.H) return;
    float s = 0.0f;
    for (int j = 0; j < a.k; ++j) s = __builtin_fmaf(a.tw[t * a.k + j], a.yr[(int64_t)(t * a.k + j) * a.H + c], s);
    a.y[(int64_t)t * a.H + c] = bf16_of(s);
}

// Up to 2048 columns four waves split a tile's columns, above eight do (12289 x
// 8192, 13 rows, NVFP4: 22 us against 27; 49152 x 2048: 22 against 19); by the
// columns only, so that a row's bits do not depend on the other rows.  A CU
// holds one block of eight waves at a time, whose time grows with its tiles from
// a fixed part on (12289 x 8192, 13 rows: 9.3 us a round of blocks of one tile,
// 14.4 of two, 16 of three, 22 of four), so the tiles per block are those with
// the least sum over the rounds (8192 x 8192, one row, one tile 16.1 us, two
// 12.2, four 18.6).  Of four waves a CU holds three blocks of one tile (INT with
// wide groups two); with 2048 columns they share the CU's units and the same rule
// holds (12000 x 2048, 16 rows: one tile 10.0 us, two 9.6, three 8.0, four 9.1),
// but short rows are latency, and while all blocks of one tile fit at once that
// is least (one row, 8192 x 512: one tile 3.7 us and two 4.6 in INT4 and 4.8 in
// NVFP4; 10000 x 512 in NVFP4: 3.8, 4.9, three 6.1; 8192 x 1024: NVFP4 4.6 and
// 4.9; INT4 with wide groups and 16 rows 5.3 and 5.0).  Blocks past the last row
// of a grid's last line read zeros and store nothing (to return early took 0.1 us
// of every call).
template <int FMT, int KW>
hipError_t run_matvec(const MatvecArgs& a, hipStream_t st) {
    const unsigned tiles = (unsigned)((a.N + 15) / 16);
    if (a.which)
        hipLaunchKernelGGL((k_matvec_which<FMT, KW>), grid_of(tiles, (unsigned)a.M), dim3(64 * KW), 0, st, a);
    else if (a.M > 16)
        hipLaunchKernelGGL((k_matvec<FMT, 2, 2, KW>), grid_of((tiles + 1) / 2, (unsigned)((a.M + 31) / 32)),
                           dim3(64 * KW), 0, st, a);
    else {
        const bool at_once = a.w.K <= (FMT == INT_WIDE ? 512 : 1024) && tiles <= 256 * (FMT == INT_WIDE ? 2 : 3);
        unsigned best = 1, least = (tiles + 255) / 256 * 7;
        for (unsigned n = 2; n <= 4 && !at_once; ++n) {
            const unsigned cost = ((tiles + n - 1) / n + 255) / 256 * (4 + 3 * n);
            if (cost < least) best = n, least = cost;
        }
        const dim3 grid = grid_of((tiles + best - 1) / best), block(64 * KW);
        if (best == 1) hipLaunchKernelGGL((k_matvec<FMT, 1, 1, KW>), grid, block, 0, st, a);
        else if (best == 2) hipLaunchKernelGGL((k_matvec<FMT, 1, 2, KW>), grid, block, 0, st, a);
        else if (best == 3) hipLaunchKernelGGL((k_matvec<FMT, 1, 3, KW>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_matvec<FMT, 1, 4, KW>), grid, block, 0, st, a);
    }
    return hipGetLastError();
}
template <int FMT>
hipError_t run_matvec(const MatvecArgs& a, hipStream_t st) {
    return a.w.K > 2048 ? run_matvec<FMT, 8>(a, st) : run_matvec<FMT, 4>(a, st);
}

// Rows of x a block keeps in LDS at a time: as many as a group can have, up to
// 8 and to 32 KB (four blocks to a CU).
int lds_rows(int K, int T) {
    const int fit = 32768 / (K * 2 + 16), most = T < 8 ? T : 8;
    return fit < 1 ? 1 : fit < most ? fit : most;
}
// Experts that evenly routed tokens hit: as many groups of rows, and so blocks
// along the grid's other axis that have work.
double groups_hit(const PackedExpertArgs& a) {
    return a.E * (1.0 - std::pow(1.0 - (double)a.k / a.E, a.R / a.k));   // k <= E
}
// A tile per wave where that leaves blocks enough with work, else the waves share
// a tile's columns.  Shared against not, in us of the whole layer, blocks of four
// tiles with work beside them.  128 experts, 2048 by 768, top-8: NVFP4 fc1 of 24
// tokens (1210) 91.7 and 92.4, of 32 (1341) 103.0 and 102.0; INT4 fc1 of 4
// tokens (349) 31.7 and 33.0, of 8 (619) 48.2 and 46.5; fc2 in NVFP4 of 4 tokens
// (466) 35.0 and 35.4, of 8 (826) 52.4 and 52.0.  32 experts, 2048 by 1024,
// top-8, 32 tokens (512): NVFP4 fc1 77.4 and 94.3, fc2 77.4 and 83.8; INT4 fc1
// 69.5 and 76.8.  8 experts, 4096 by 4096, top-2, 64 tokens (fc1 512, fc2 256):
// NVFP4 fc1 298 and 342, fc2 298 and 350.
template <int FMT>
hipError_t run_fc1(const PackedExpertArgs& a, hipStream_t st) {
    const int cap = lds_rows(a.H, a.R / a.k);
    const size_t lds = (size_t)cap * (a.H * 2 + 16);
    if (groups_hit(a) * (a.I / 64) >= (FMT == NVFP4 ? 1280 : 576))
        hipLaunchKernelGGL((k_packed_fc1<FMT, false>), dim3((unsigned)(a.I / 64), (unsigned)a.R), dim3(64 * WV), lds, st,
                           a, cap);
    else
        hipLaunchKernelGGL((k_packed_fc1<FMT, true>), dim3((unsigned)(a.I / 16), (unsigned)a.R), dim3(64 * WV), lds, st,
                           a, cap);
    return hipGetLastError();
}
template <int FMT>
hipError_t run_fc2(const PackedExpertArgs& a, hipStream_t st) {
    const int cap = lds_rows(a.I, a.R / a.k);
    const size_t lds = (size_t)cap * (a.I * 2 + 16);
    if (groups_hit(a) * (a.H / 128) >= 704)
        hipLaunchKernelGGL((k_packed_fc2<FMT, false>), dim3((unsigned)(a.H / 128), (unsigned)a.R), dim3(64 * WV), lds, st,
                           a, cap);
    else
        hipLaunchKernelGGL((k_packed_fc2<FMT, true>), dim3((unsigned)(a.H / 64), (unsigned)a.R), dim3(64 * WV), lds, st,
                           a, cap);
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
