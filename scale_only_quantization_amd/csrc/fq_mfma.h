// Building blocks of the gfx950 matrix-core kernels: buffer resources, direct
// global->LDS stage loads, the LDS operand tiles with their swizzles and
// fragment reads (v_mfma_f32_32x32x16_bf16), and the block -> tile order.
#pragma once

#include "fq_common.h"

namespace fq {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_t;

// Buffer resource over [base, base + bytes): loads outside read as zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
    if (bytes < 0) bytes = 0;
    if (bytes > 0xFFFFFFF0ll) bytes = 0xFFFFFFF0ll;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)(uint32_t)bytes,
                                             0x00020000);
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// The same resource as four wave-uniform dwords, for stage_load below.
__device__ __forceinline__ u32x4 make_rsrc_words(const void* base, int64_t bytes) {
    if (bytes < 0) bytes = 0;
    if (bytes > 0xFFFFFFF0ll) bytes = 0xFFFFFFF0ll;
    const uint64_t a = (uint64_t)(uintptr_t)base;
    u32x4 r;
    r.x = __builtin_amdgcn_readfirstlane((uint32_t)a);
    r.y = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xFFFFu);     // stride 0
    r.z = __builtin_amdgcn_readfirstlane((uint32_t)bytes);
    r.w = 0x00020000u;
    return r;
}

// One wave's direct global->LDS loads of a stage: N loads of 16 B per lane,
// load i from resource offset voff[i] + soff into the 1 KB of LDS at
// dst + i * STEP (dst wave-uniform; lane l writes 16 B at + 16 l).  Written as
// assembly so that the compiler does not see LDS writes in flight: it would
// otherwise wait for every such load (vmcnt(0)) before the next transposing
// LDS read, i.e. put the latency of the step's loads just issued in front of
// the current step's fragment reads.  Callers order these loads against the
// LDS reads themselves, with their own vmcnt waits and barriers.  M0 carries
// each load's LDS address (one wait state between its write and the load);
// the leading s_nop 4 gives the five wait states a vector-memory read of an
// SGPR needs after a vector instruction wrote it (v_readfirstlane, or
// v_readlane restoring a spilled SGPR), which the compiler supplies for its
// own instructions but not for assembly.
template <int N, int STEP>
__device__ __forceinline__ void stage_loads(const u32x4& rs, lds_t* dst, const uint32_t (&voff)[N], uint32_t soff) {
    static_assert(N >= 1 && N <= 4, "loads per wave and stage");
    const uint32_t m = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)dst);
#define FQ_LDS_LOAD(V) "s_nop 0\n\tbuffer_load_dwordx4 " V ", %[r], %[so] offen lds\n\t"
    if constexpr (N == 1) {
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %[m]\n\t" FQ_LDS_LOAD("%[v0]")
                     :
                     : [m] "s"(m), [v0] "v"(voff[0]), [r] "s"(rs), [so] "s"(soff)
                     : "memory", "m0");
    } else if constexpr (N == 2) {
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %[m]\n\t" FQ_LDS_LOAD("%[v0]")
                     "s_add_i32 m0, %[m], %[d1]\n\t" FQ_LDS_LOAD("%[v1]")
                     :
                     : [m] "s"(m), [v0] "v"(voff[0]), [v1] "v"(voff[1]), [r] "s"(rs), [so] "s"(soff),
                       [d1] "n"(STEP)
                     : "memory", "m0");
    } else if constexpr (N == 3) {
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %[m]\n\t" FQ_LDS_LOAD("%[v0]")
                     "s_add_i32 m0, %[m], %[d1]\n\t" FQ_LDS_LOAD("%[v1]")
                     "s_add_i32 m0, %[m], %[d2]\n\t" FQ_LDS_LOAD("%[v2]")
                     :
                     : [m] "s"(m), [v0] "v"(voff[0]), [v1] "v"(voff[1]), [v2] "v"(voff[2]), [r] "s"(rs),
                       [so] "s"(soff), [d1] "n"(STEP), [d2] "n"(2 * STEP)
                     : "memory", "m0");
    } else {
        asm volatile("s_nop 4\n\ts_mov_b32 m0, %[m]\n\t" FQ_LDS_LOAD("%[v0]")
                     "s_add_i32 m0, %[m], %[d1]\n\t" FQ_LDS_LOAD("%[v1]")
                     "s_add_i32 m0, %[m], %[d2]\n\t" FQ_LDS_LOAD("%[v2]")
                     "s_add_i32 m0, %[m], %[d3]\n\t" FQ_LDS_LOAD("%[v3]")
                     :
                     : [m] "s"(m), [v0] "v"(voff[0]), [v1] "v"(voff[1]), [v2] "v"(voff[2]), [v3] "v"(voff[3]),
                       [r] "s"(rs), [so] "s"(soff), [d1] "n"(STEP), [d2] "n"(2 * STEP), [d3] "n"(3 * STEP)
                     : "memory", "m0");
    }
#undef FQ_LDS_LOAD
}

// x of lane l ^ 32: one cross-half swap (v_permlane32_swap) and a select, no
// LDS round trip.  The swap returns (lanes 0-31 of x in both halves, lanes
// 32-63 of x in both halves).
__device__ __forceinline__ float xor32(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Wait until at most n (clamped to 0..3) steps of L load instructions each
// are outstanding: vector-memory loads complete in issue order.
template <int L>
__device__ __forceinline__ void wait_steps(int n) {
    static_assert(3 * L <= 63, "vmcnt range");
    if (n <= 0) vm_wait<0>();
    else if (n == 1) vm_wait<L>();
    else if (n == 2) vm_wait<2 * L>();
    else vm_wait<3 * L>();
}

// K-contiguous operand tile [ROWS][BK]: element (row, k) at byte row*ld2 + 2k
// of the resource.  Rows of 2 BK bytes; each 1-KB wave load covers 512/BK rows.
// Swizzle: chunk ^ (row >> 2) & 3 for 64-B rows, chunk ^ (row >> 1) & 7 for
// 128-B rows, so the 16 rows one ds_read_b128 pass serves (16 lanes x 16 B,
// 64 banks) fall on distinct banks; rows 32 apart share a swizzle, so a
// wave's fragments of one k sub-step differ by constant offsets.
template <int ROWS, int BK, int NW>
struct KTile {
    static constexpr int BYTES = ROWS * BK * 2;
    static constexpr int PER_WAVE = BYTES / 1024 / NW;
    static constexpr int CPR = BK / 8;                 // 16-B chunks per row
    static constexpr int RB = 2 * BK;                  // bytes per row
    static constexpr int KS = BK / 16;                 // 16-deep sub-steps per step
    __device__ static __forceinline__ int swz(int row) {
        return BK == 32 ? ((row >> 2) & 3) : ((row >> 1) & 7);
    }
    __device__ static __forceinline__ int off(int row, int ch) {   // byte offset of 16-B chunk
        return row * RB + ((ch ^ swz(row)) << 4);
    }
    u32x4 rs;
    uint32_t voff[PER_WAVE];
    __device__ __forceinline__ void init(const u32x4& r, int64_t ld) {
        rs = r;
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) {
            const int blk = NW * i + w;                   // 1-KB block
            const int row = blk * (64 / CPR) + lane / CPR;
            const int lc = (lane % CPR) ^ swz(row);       // logical chunk stored at this position
            voff[i] = (uint32_t)(row * ld * 2 + lc * 16);
        }
    }
    __device__ __forceinline__ void issue(lds_t* tile, int k0) {
        stage_loads<PER_WAVE, NW * 1024>(rs, tile + wave_id() * 1024, voff, (uint32_t)k0 * 2);
    }
    // fragment of the 32x32x16 MFMA: row `row0 + lane%32`, k = 16 kk + 8 (lane/32) .. +7
    __device__ static __forceinline__ bf16x8 frag(const lds_t* tile, int row0, int kk) {
        const int lane = threadIdx.x & 63;
        const int row = row0 + (lane & 31);
        return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8*>(
            tile + off(row, kk * 2 + (lane >> 5)));
    }
    // A wave's fragments from per-lane offsets: one offset per sub-step kk for
    // rows row0w + 32 t + lane%32 (row0w a multiple of 32); t adds 32 RB.
    template <int WT>
    struct Frags {
        uint32_t o[KS];
        __device__ __forceinline__ void prep(int row0w) {
            const int lane = threadIdx.x & 63;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) o[kk] = (uint32_t)off(row0w + (lane & 31), kk * 2 + (lane >> 5));
        }
        __device__ __forceinline__ bf16x8 get(const lds_t* tile, int t, int kk) const {
            return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8*>(tile + o[kk] + t * 32 * RB);
        }
    };
};

// Row-contiguous operand tile [BK][ROWS] (stored as in memory): element
// (row, k) at byte k*ld2 + 2*row of the resource.  Each 1-KB wave load covers
// 1024 / (2 ROWS) k-rows.
template <int ROWS, int BK, int NW>
struct MNTile {
    static constexpr int BYTES = ROWS * BK * 2;
    static constexpr int PER_WAVE = BYTES / 1024 / NW;
    static constexpr int RB = ROWS * 2;               // bytes per k-row
    // 16-B chunk ch of k-row k is stored at chunk ch ^ 2 (k & 3) ^ 8 (bit 1 of ch)
    __device__ static __forceinline__ int phys(int k, int ch) { return ch ^ ((k & 3) << 1) ^ (((ch >> 1) & 1) << 3); }
    __device__ static __forceinline__ int off(int k, int byte) {   // swizzled byte offset
        return k * RB + (phys(k, byte >> 4) << 4) + (byte & 15);
    }
    u32x4 rs;
    uint32_t voff[PER_WAVE];
    uint32_t ld2;
    __device__ __forceinline__ void init(const u32x4& r, int64_t ld) {
        rs = r;
        ld2 = (uint32_t)(ld * 2);
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) {
            const int pos = (NW * i + w) * 1024 + lane * 16;  // byte position in the tile
            const int k = pos / RB;
            const int pc = (pos % RB) >> 4;
            const int lc = pc ^ ((k & 3) << 1) ^ ((((pc >> 1) ^ k) & 1) << 3);   // phys(k, lc) == pc
            voff[i] = (uint32_t)(k * ld * 2 + lc * 16);
        }
    }
    __device__ __forceinline__ void issue(lds_t* tile, int k0) {
        stage_loads<PER_WAVE, NW * 1024>(rs, tile + wave_id() * 1024, voff, (uint32_t)k0 * ld2);
    }
    __device__ static __forceinline__ bf16x8 frag(const lds_t* tile, int row0, int kk) {
        const int lane = threadIdx.x & 63;
        const int i = lane & 15;
        const int mb = row0 + ((lane >> 4) & 1) * 16;
        const int kb = kk * 16 + (lane >> 5) * 8 + (i >> 2);
        const int byte = (mb + 4 * (i & 3)) * 2;
        typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 v4bf;
        typedef __attribute__((address_space(3))) v4bf lds4;
        lds_t* t = const_cast<lds_t*>(tile);
        const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(t + off(kb, byte))));
        const bf16x4 hi = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(t + off(kb + 4, byte))));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // A wave's fragments from per-lane offsets: one offset per 32-row tile t
    // (rows row0w + 32 t); sub-step kk adds 16 k-rows, the second read 4.
    template <int WT>
    struct Frags {
        uint32_t o[WT];
        __device__ __forceinline__ void prep(int row0w) {
            const int lane = threadIdx.x & 63;
            const int i = lane & 15;
            const int kb = (lane >> 5) * 8 + (i >> 2);
#pragma unroll
            for (int t = 0; t < WT; ++t) {
                const int mb = row0w + 32 * t + ((lane >> 4) & 1) * 16;
                o[t] = (uint32_t)off(kb, (mb + 4 * (i & 3)) * 2);
            }
        }
        __device__ __forceinline__ bf16x8 get(const lds_t* tile, int t, int kk) const {
            typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 v4bf;
            typedef __attribute__((address_space(3))) v4bf lds4;
            lds_t* p = const_cast<lds_t*>(tile) + o[t] + kk * 16 * RB;
            const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)p));
            const bf16x4 hi = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(p + 4 * RB)));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
};

// Block -> tile with XCD locality: workgroups are dealt to the 8 XCDs (each
// with its own L2) round-robin, so XCD x = id % 8 is given the contiguous run
// of tiles [x * chunk, (x + 1) * chunk), chunk = ceil(tiles / 8); tiles that
// share operands (the N tiles of one row tile, the row tiles of one expert)
// then meet in the same L2.  Returns -1 for ids past the tile count.
__device__ __forceinline__ int xcd_tile(int id, int grid, int tiles) {
    const int chunk = (tiles + 7) / 8;
    const int t = (id % 8) * chunk + id / 8;
    return (id / 8 < chunk && t < tiles) ? t : -1;
}

}  // namespace

}  // namespace fq
