// The matrix product of the output layer's operators: a persistent tile product
// of bf16 operands with an epilogue on the fp32 accumulators, the tile order,
// and the small numbers that they share.
#pragma once

#include <type_traits>

#include "fq_mfma.h"

namespace fq {
namespace {

constexpr float LOG2E = 0x1.715476p+0f;   // log2(e) and ln(2), rounded to fp32
constexpr float LN2 = 0x1.62e430p-1f;
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float bf_from_bits(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

constexpr int BM = 256, BN = 256, BK = 64, S = 2, NW = 8, WTM = 4, WTN = 2, WVN = 4;
constexpr int KS = BK / 16;
constexpr int CUS = 256;
typedef KTile<BM, BK, NW> KT;             // a reduction-contiguous operand
typedef MNTile<BN, BK, NW> MT;            // the weight as [vocabulary, hidden], reduced over the vocabulary
constexpr int SMEM = S * (KT::BYTES + KT::BYTES);
static_assert(KT::BYTES == MT::BYTES, "both products use one LDS layout");

// acc = A B^T, nk steps of 64 for each of n tiles (nk even where n > 1), on eight
// waves in two groups of four that alternate between a memory phase (fragments
// of one step into registers, the loads of a later step) and a compute phase
// (that step's MFMAs), one phase apart: on each SIMD one wave issues MFMAs while
// the other reads.  Group 0 issues its loads of step k + 1 as its memory phase of
// step k opens, into the stage both groups finished reading in the two phases
// before.  Group 1 issues its loads of step k + 2 in its memory phase of step k,
// behind a barrier in the middle of group 0's compute phase: its other waves may
// still be reading that stage before it (without a measurable cost there; in
// group 1's own compute phase the loads cost a tenth).  Each group waits for its
// loads of step k + 1 before the barrier that opens group 0's memory phase of
// that step.  The steps run on from tile to tile: next(i) points la and lb at
// tile i before a group's first load of it, and epi(i), which uses no stage,
// opens the group's next memory phase, while the other group computes.  Wave row
// wm (the group) has the rows from wm wr on, nti(i) sub-tiles of 32 of them.
template <class AT, class BT, typename N, typename R, typename E>
__device__ __forceinline__ void product(AT& la, BT& lb, f32x16 (&acc)[WTM][WTN], lds_t* smem, int n, int nk, int wr,
                                        N&& next, R&& nti, E&& epi) {
    constexpr int LOADS = AT::PER_WAVE + BT::PER_WAVE;
    const int w = wave_id(), grp = w >> 2;
    typename AT::template Frags<WTM> fa;
    typename BT::template Frags<WTN> fb;
    fa.prep((w / WVN) * wr);
    fb.prep((w % WVN) * 32 * WTN);
    bf16x8 af[KS][WTM], bfr[KS][WTN];
    // loads of step kt of tile i, or of step kt - nk of the tile after it; false if there is none
    auto issue = [&](int i, int kt, int st) {
        if (kt >= nk) {
            if (i + 1 >= n) return false;
            if (kt == nk) next(i + 1);
            kt -= nk;
        }
        la.issue(smem + st * AT::BYTES, kt * BK);
        lb.issue(smem + S * AT::BYTES + st * BT::BYTES, kt * BK);
        return true;
    };
    auto bar = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    if (nk > 0) {
        next(0);
        issue(0, 0, 0);
    }
    vm_wait<0>();
    bar();
    if (nk > 0) issue(0, 1, 1);
    if (grp == 1) bar();
    auto phases = [&](int i, int kt, int st, auto n_c) {
        constexpr int NT = decltype(n_c)::value;
        const lds_t* sa = smem + st * AT::BYTES;
        const lds_t* sb = smem + S * AT::BYTES + st * BT::BYTES;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int t = 0; t < NT; ++t) af[kk][t] = fa.get(sa, t, kk);
            if (NT > 0)
#pragma unroll
                for (int t = 0; t < WTN; ++t) bfr[kk][t] = fb.get(sb, t, kk);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (grp == 1) {
            bar();
            const bool more = issue(i, kt + 2, st);
            if (kt > 0 || i == 0) wait_steps<LOADS>(more ? 1 : 0);
        }
        bar();
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int ti = 0; ti < NT; ++ti)
#pragma unroll
                for (int tj = 0; tj < WTN; ++tj)
                    acc[ti][tj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bfr[kk][tj], af[kk][ti], acc[ti][tj], 0, 0, 0);
            if (kk == 1 && grp == 0) bar();
        }
        if (grp == 0) vm_wait<0>();
        bar();
        if (grp == 0) issue(i, kt + 2, st);
    };
    auto steps = [&](int i, auto n_c) {
        for (int kt = 0; kt < nk; kt += S) {
#pragma unroll
            for (int u = 0; u < S; ++u)
                if (kt + u < nk) phases(i, kt + u, u, n_c);
        }
    };
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
#pragma unroll
        for (int a = 0; a < WTM; ++a)
#pragma unroll
            for (int b = 0; b < WTN; ++b)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;
        const int sub = nti(i);
        if (sub == 4) steps(i, std::integral_constant<int, 4>{});
        else if (sub == 3) steps(i, std::integral_constant<int, 3>{});
        else if (sub == 2) steps(i, std::integral_constant<int, 2>{});
        else if (sub == 1) steps(i, std::integral_constant<int, 1>{});
        else steps(i, std::integral_constant<int, 0>{});
        if (grp == 1) vm_wait<0>();                    // step 1 of the next tile, before the epilogue's stores
        epi(i);
    }
    if (grp == 0) bar();
}

// Tile t of mt x nt in the order that shares operands inside an XCD's L2:
// bands of 8 row tiles, in a band column by column; an XCD has a contiguous
// run (xcd_tile), so the 32 tiles it works on at once are about 8 x 4.
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int* m, int* n) {
    const int band = t / (8 * nt), in = t - band * 8 * nt;
    const int h = min(8, mt - band * 8);
    *n = in / h;
    *m = band * 8 + in - *n * h;
}

}  // namespace

}  // namespace fq
