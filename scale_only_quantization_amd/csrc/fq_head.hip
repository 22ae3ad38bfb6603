// The output layer's loss from hidden states, without the logits: cross
// entropy and the KL from a teacher's top logits, with the gradient on the
// hidden states (the output layer's weight stays frozen).
//
//   z = h W^T,  lse = log sum e^z,  q = e^{z - lse}
//   row = lm (lse - z_label) + dist sum_j p_j (log p_j - z_j + lse)
//   dh  = 1/n (c q W + sum_s coef_s W_s),  c = lm + dist
// The vocabulary goes by in pieces; of a piece only P = 2^{z log2 e - F}
// exists, in bf16, with a frame F per token (an integer, near the token's
// running maximum):
//   sparse  the logits of the label and of the teacher's ids, in fp32; their
//           maximum is the first frame
//   probs   one matrix product z = h W_piece^T whose epilogue turns the fp32
//           accumulators into P and sums them per token and 64 columns
//   merge   the token's running frame and sum; a strip of 64 that rose more
//           than 2^40 above the frame has a frame of its own and is brought
//           to the common one here (both are powers of two: exact), as is the
//           running gradient in the product below.  The label's and the
//           teacher's entries of P are set to zero: their share of the
//           gradient, where q - p may cancel, is added in fp32 at the end
//   grad    a second matrix product, G = f G + P W_piece in fp32 (f the step
//           of the frame, a power of two), split over the piece where tokens
//           are few
// and `out` forms each token's loss, and c/S G + sum_s coef_s W_s over the
// label and the teacher's ids, rounded to bf16 once.  So each logit is
// computed once, never stored, and rounded to bf16 only as a probability
// beside fp32 sums.  P's rounding, up to 2^-8 of each term, averages out over the
// product's sum where many entries share a token's mass; where one entry that is
// neither the label nor a teacher's id has nearly all of it, it stays beside the
// output's own rounding (relative error of such gradients 0.0019, where that
// rounding alone gives 0.0017).  The two products carry the time (16384 tokens of hidden 2048,
// 151936 entries, 64 teacher ids: 17.4-18.2 ms, of which probs 8.0 and grad 8.0,
// 1270 TFLOP/s each where a library product of that size reaches 1357; their
// matrix units are busy 65 and 77% of the time at 1.7 GHz, the clock that the
// power allows); sparse and out, 65 rows of the weight per token each, read at
// 6 to 7 TB/s.  Few tokens: 333 x 1024 x 32003 without a teacher 94 us, probs 33,
// grad 33, merge and out 10 each; with 64 teacher ids 120.  Without the gradient
// 41 us, 2048 tokens of the large vocabulary 1.07 ms, 16384 8.2 ms.
#include <algorithm>

#include "fq_mfma.h"
#include "fq_ops.h"

namespace fq {
namespace {

constexpr float LOG2E = 0x1.715476p+0f;   // log2(e) and ln(2), rounded to fp32
constexpr float LN2 = 0x1.62e430p-1f;
constexpr float FRAME_SLACK = 40.0f;      // P may reach 2^40 above its frame
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

// --------------------------------------------------------------- sparse ---
// Rows that count: those with a label in the vocabulary, or all without labels.
__device__ __forceinline__ bool counts(const HeadArgs& a, int64_t t) {
    return !a.labels || (a.labels[t] >= 0 && a.labels[t] < a.V);
}

// Logits of the label and the teacher's ids: a block per token, its waves
// take the slots in turn (slot k is the label).  Slots outside the vocabulary
// are absent (-inf).  One block more forms 1 / (rows that count, at least one).
__global__ __launch_bounds__(256) void k_head_sparse(HeadArgs a) {
    __shared__ float sz[65];
    __shared__ int red[4];
    const int64_t t = block_id();
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    if (t > a.T) return;
    if (t == a.T) {
        int n = 0;
        for (int64_t r = threadIdx.x; r < a.T; r += 256) n += counts(a, r) ? 1 : 0;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) n += __shfl_xor(n, m);
        if (lane == 0) red[w] = n;
        __syncthreads();
        if (threadIdx.x == 0) a.inv_n[0] = 1.0f / (float)max(red[0] + red[1] + red[2] + red[3], 1);
        return;
    }
    const int slots = a.k + 1, nvec = a.H >> 3;
    const uint4* hr = reinterpret_cast<const uint4*>(a.h + t * a.H);
    // four slots of a wave at a time, so that their rows are in flight together
    // (65 rows of 2048 for 16384 tokens: 622 us, 7 TB/s; one at a time 673)
    for (int j0 = w; j0 < slots; j0 += 16) {
        int id[4], some = -1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = j0 + 4 * q;
            id[q] = __builtin_amdgcn_readfirstlane(
                j < a.k ? a.top_i[t * a.k + j] : (j == a.k && a.labels ? a.labels[t] : -1));
            if (id[q] >= a.V) id[q] = -1;
            some = max(some, id[q]);
        }
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (some >= 0) {
            const uint4* wr[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)               // an absent slot reads a row that is read anyway
                wr[q] = reinterpret_cast<const uint4*>(a.w + (int64_t)(id[q] >= 0 ? id[q] : some) * a.H);
            for (int c = lane; c < nvec; c += 64) {
                float x[8], y[8];
                unpack8(hr[c], x);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    unpack8(wr[q][c], y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[q] = __builtin_fmaf(x[i], y[i], acc[q]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float z = wave_sum(acc[q]);
            if (lane == 0 && j0 + 4 * q < slots) sz[j0 + 4 * q] = id[q] >= 0 ? z : -INFINITY;
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < slots; j += 256) a.zs[t * slots + j] = sz[j];
    if (threadIdx.x < 64) {
        float m = -INFINITY;
        for (int j = lane; j < slots; j += 64) m = fmaxf(m, sz[j]);
        m = wave_max(m);
        if (lane == 0) {
            a.frame[t] = ceilf(m * LOG2E);
            a.sum[t] = 0.0f;
        }
    }
}

// ---------------------------------------------------------------- probs ---
// One block per CU (or fewer) takes tiles in turn; each XCD has a contiguous run
// of them.  P goes from the registers to memory: the four stores of a wave's 64
// columns fill whole 128-byte lines one after the other.  (A piece of 15360
// entries for 16384 tokens: 815 us, 1265 TFLOP/s; a block per tile with P through
// the stages 864; P through LDS of its own 828, past the caches then or not.)
template <bool GRAD>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) void k_head_probs(HeadArgs a) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM + 2 * BM * 4];
    lds_t* smem = (lds_t*)smem_raw;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int wm = wave / WVN, wn = wave % WVN;
    const int mt = (int)((a.T + a.bm - 1) / a.bm), nt = a.vc / BN;
    const int wr = (a.bm / 2 + 31) / 32 * 32;                 // the first wave row's rows; the second has the rest
    const int run = (mt * nt + 7) / 8, per = gridDim.x / 8;   // tiles of an XCD, its blocks
    const int t0 = (blockIdx.x & 7) * run + (blockIdx.x >> 3), t1 = min(mt * nt, ((int)(blockIdx.x & 7) + 1) * run);
    if (t0 >= t1) return;
    auto at = [&](int i, int64_t* m0, int* tn) {              // tile i's first row, its rows, its column tile
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
        const int64_t v0 = a.c0 + (int64_t)tn * BN;           // first vocabulary entry of the tile
        const int cols = (int)min((int64_t)BN, a.V - v0);     // may be <= 0 in the last piece's padding
        la.rs = make_rsrc_words(a.h + m0 * a.H, (int64_t)rows * a.H * 2);
        lb.rs = make_rsrc_words(a.w + (cols > 0 ? v0 : 0) * a.H, (int64_t)cols * a.H * 2);
        // the tile's frames, ahead of its first step, in the other buffer than
        // the tile's before
        if (wave == 0) {
            const uint32_t voff[1] = {(uint32_t)lane * 16};
            stage_loads<1, 0>(make_rsrc_words(a.frame + m0, (int64_t)(rows + 3) / 4 * 16),
                              smem + SMEM + (i & 1) * BM * 4, voff, 0);
        }
    };
    auto nti = [&](int i) {
        int64_t m0;
        int tn;
        const int rows = at(i, &m0, &tn);
        return wm == 0 ? (min(rows, wr) + 31) / 32 : (max(rows - wr, 0) + 31) / 32;
    };
    // lane holds z of token lane%32 and columns 8 (v/4) + 4 (lane/32) + v%4 of
    // each 32 x 32 sub-tile: a token's 64 columns of this wave are its own 32
    // and lane ^ 32's
    auto epilogue = [&](int i) {
        int64_t m0;
        int tn;
        const int rows = at(i, &m0, &tn), sub = nti(i);
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));                        // what follows from it is not held through the steps
        const int cols = (int)min((int64_t)BN, a.V - a.c0 - (int64_t)tn * BN);
        const __amdgpu_buffer_rsrc_t prs = make_rsrc(GRAD ? a.p + m0 * a.vc + (int64_t)tn * BN : nullptr,
                                                     (int64_t)(rows - 1) * a.vc * 2 + BN * 2);
        const __attribute__((address_space(3))) float* frames =
            reinterpret_cast<const __attribute__((address_space(3))) float*>(smem + SMEM + (i & 1) * BM * 4);
#pragma unroll
        for (int ti = 0; ti < WTM; ++ti) {
            if (ti >= sub) break;
            const int row = wm * wr + ti * 32 + (lane & 31);
            const float frame = frames[row];
            if (cols < BN) {
#pragma unroll
                for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (wn * 64 + tj * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3) >= cols)
                            acc[ti][tj][v] = -INFINITY;
            }
            float m = acc[ti][0][0];
#pragma unroll
            for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                for (int v = 0; v < 16; ++v) m = fmaxf(m, acc[ti][tj][v]);
            m = fmaxf(m, xor32(m)) * LOG2E;
            float f = m <= frame + FRAME_SLACK ? frame : ceilf(m);
            if (f == -INFINITY) f = 0.0f;                     // nothing in the strip: P = 0
            float s = 0.0f;
#pragma unroll
            for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const float e = exp2_hw(__builtin_fmaf(acc[ti][tj][v], LOG2E, -f));
                    s += e;
                    acc[ti][tj][v] = e;
                }
            s += xor32(s);
            if (lane < 32 && row < rows)
                a.stats[((int64_t)tn * 4 + wn) * a.T + m0 + row] = make_float2(s, f);
            if (GRAD)
#pragma unroll
                for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        // the halves trade, so that a lane has 8 columns in a row
                        u32x4 c;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const auto r = __builtin_amdgcn_permlane32_swap(
                                pack_bf16(acc[ti][tj][4 * q + 2 * j], acc[ti][tj][4 * q + 2 * j + 1]),
                                pack_bf16(acc[ti][tj][4 * q + 4 + 2 * j], acc[ti][tj][4 * q + 5 + 2 * j]), false, false);
                            c[j] = r[0];
                            c[2 + j] = r[1];
                        }
                        const int col = wn * 64 + tj * 32 + 8 * (q + (lane >> 5));
                        __builtin_amdgcn_raw_buffer_store_b128(c, prs, (uint32_t)row * (uint32_t)a.vc * 2u + col * 2, 0, 0);
                    }
        }
    };
    product(la, lb, acc, smem, (t1 - t0 + per - 1) / per, a.H / BK, wr, next, nti, epilogue);
}

// ---------------------------------------------------------------- merge ---
// TOK tokens per block, 1024 / TOK threads per token taking every so many-th
// strip; sums and maxima combine in a fixed tree.  One pass over the strips
// where all have the tokens' frames, as nearly always; else a second one in
// the new frames.  16 tokens (128-byte pieces of the strips' rows) where they
// fill the card, else 4 with the shorter chains of loads (333 tokens of 32003
// entries: 14 us with 4, 28 with 16; 2048 of 151936: 36 and 21; 16384, a piece
// of 15360: 41 and 20).
template <int TOK>
__global__ __launch_bounds__(1024) void k_head_merge(HeadArgs a) {
    constexpr int PER = 1024 / TOK;
    __shared__ float red_f[16][TOK], red_s[16][TOK];
    const int tok = threadIdx.x % TOK, sl = threadIdx.x / TOK, w = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * TOK + tok, tc = min(t, a.T - 1);
    const bool live = t < a.T;
    const int strips = a.vc / 64;
    const float f0 = a.frame[tc];
    auto over_token = [&](float v, bool max, float (*red)[TOK]) {
#pragma unroll
        for (int m = TOK; m < 64; m <<= 1) {
            const float o = __shfl_xor(v, m);
            v = max ? fmaxf(v, o) : v + o;
        }
        if ((threadIdx.x & 63) < TOK) red[w][tok] = v;
        __syncthreads();
        v = red[0][tok];
#pragma unroll
        for (int i = 1; i < 16; ++i) v = max ? fmaxf(v, red[i][tok]) : v + red[i][tok];
        return v;
    };
    // read ahead of the strips: what the tail needs
    const int slots = a.k + 1;
    const int64_t t0 = (int64_t)blockIdx.x * TOK;
    const int n = a.p ? (int)min((int64_t)TOK, a.T - t0) * slots : 0;
    auto id_of = [&](int i) {
        const int64_t r = t0 + i / slots;
        const int j = i % slots;
        return j < a.k ? a.top_i[r * a.k + j] : (a.labels ? a.labels[r] : -1);
    };
    const int id0 = (int)threadIdx.x < n ? id_of(threadIdx.x) : -1;
    const float before = a.sum[tc];
    float f = f0, sum = 0.0f;
    bool moved = false;
#pragma unroll 8
    for (int s = sl; s < strips; s += PER) {
        const float2 v = a.stats[(int64_t)s * a.T + tc];
        const bool other = v.y != f0 && v.x != 0.0f;
        moved |= other;
        f = other ? fmaxf(f, v.y) : f;
        sum += v.y == f0 ? v.x : 0.0f;
    }
    if (__syncthreads_or(moved && live)) {             // frames of their own: bring all to the common one
        f = over_token(f, true, red_f);
        sum = 0.0f;
        for (int s = sl; s < strips; s += PER) {
            const float2 v = a.stats[(int64_t)s * a.T + tc];
            if (v.y == f) {
                sum += v.x;
            } else if (v.x != 0.0f) {
                const float k = exp2_hw(v.y - f);
                sum += v.x * k;
                if (a.p && live) {
                    uint4* p = reinterpret_cast<uint4*>(a.p + t * a.vc + s * 64);
                    for (int i = 0; i < 8; ++i) {
                        float e[8];
                        unpack8(p[i], e);
#pragma unroll
                        for (int j = 0; j < 8; ++j) e[j] *= k;
                        p[i] = pack8(e);
                    }
                }
            }
        }
    }
    sum = over_token(sum, false, red_s);               // its barrier: the strips are in the common frame
    if (threadIdx.x < TOK && live) {
        const float step = f0 == f ? 1.0f : exp2_hw(f0 - f);
        a.sum[t] = (before == 0.0f ? 0.0f : before * step) + sum;
        a.frame[t] = f;
        a.step[t] = step;
    }
    for (int i = threadIdx.x; i < n; i += 1024) {
        const int id = i < 1024 ? id0 : id_of(i);
        if (id >= a.c0 && id < a.V && id - a.c0 < a.vc) a.p[(t0 + i / slots) * a.vc + (id - a.c0)] = 0;
    }
}

// ----------------------------------------------------------------- grad ---
// G[split][t, :] = (first piece ? 0 : step[t] G) + P W_piece over the split's
// share of the piece
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) void k_head_grad(HeadArgs a) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM];
    lds_t* smem = (lds_t*)smem_raw;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int wm = wave / WVN, wn = wave % WVN;
    const int mt = (int)((a.T + a.bm - 1) / a.bm), nt = (a.H + BN - 1) / BN;
    int tile = xcd_tile(blockIdx.x, gridDim.x, mt * nt * a.splits);
    if (tile < 0) return;
    const int split = tile / (mt * nt);
    tile -= split * mt * nt;
    int tm, tn;
    tile_of(tile, mt, nt, &tm, &tn);
    const int64_t m0 = (int64_t)tm * a.bm;
    const int rows = (int)min((int64_t)a.bm, a.T - m0);
    const int wr = (a.bm / 2 + 31) / 32 * 32;                 // the first wave row's; the second has the rest
    const int nti = wm == 0 ? (min(rows, wr) + 31) / 32 : (max(rows - wr, 0) + 31) / 32;
    const int n0 = tn * BN;
    const int k0 = split * a.ksplit, kn = min(a.ksplit, a.vc - k0);     // multiples of 64; kn may be <= 0
    const int kv = (int)min((int64_t)kn, a.V - a.c0 - k0);              // of them inside the vocabulary
    KT la;
    MT lb;
    la.init(make_rsrc_words(a.p + m0 * a.vc + k0, kn > 0 ? ((int64_t)(rows - 1) * a.vc + kn) * 2 : 0), a.vc);
    lb.init(make_rsrc_words(kv > 0 ? a.w + (a.c0 + k0) * a.H + n0 : a.w,
                            kv > 0 ? ((int64_t)(kv - 1) * a.H + (a.H - n0)) * 2 : 0),
            a.H);
    f32x16 acc[WTM][WTN];
    product(la, lb, acc, smem, 1, max(kn, 0) / BK, wr, [](int) {}, [&](int) { return nti; }, [](int) {});
    float* G = a.g + (int64_t)split * a.T * a.H;
#pragma unroll
    for (int ti = 0; ti < WTM; ++ti) {
        const int row = wm * wr + ti * 32 + (lane & 31);
        if (ti >= nti || row >= rows) continue;
        const int64_t t = m0 + row;
        const float f = a.first ? 0.0f : a.step[t];
        float* gr = G + t * a.H + n0;
#pragma unroll
        for (int tj = 0; tj < WTN; ++tj)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = wn * 64 + tj * 32 + 8 * q + 4 * (lane >> 5);
                if (n0 + col >= a.H) continue;
                float4 o = make_float4(acc[ti][tj][4 * q], acc[ti][tj][4 * q + 1], acc[ti][tj][4 * q + 2],
                                       acc[ti][tj][4 * q + 3]);
                float4* d = reinterpret_cast<float4*>(gr + col);
                if (!a.first) {
                    const float4 b = *d;
                    o.x = __builtin_fmaf(b.x, f, o.x);
                    o.y = __builtin_fmaf(b.y, f, o.y);
                    o.z = __builtin_fmaf(b.z, f, o.z);
                    o.w = __builtin_fmaf(b.w, f, o.w);
                }
                *d = o;
            }
    }
}

// ------------------------------------------------------------------ out ---
// A block per token: loss and coefficients by the first wave (lane j is slot
// j, k <= 64; the label is lane 0's second slot), then VEC columns per thread.
template <int VEC>
__global__ __launch_bounds__(256) void k_head_out(HeadArgs a) {
    __shared__ float s_coef[65];
    __shared__ int s_id[65];
    __shared__ float s_c;
    const int64_t t = blockIdx.x;
    const int slots = a.k + 1;
    if (!counts(a, t)) {                                 // uniform: padding
        if (threadIdx.x == 0) a.row_loss[t] = 0.0f;
        if (a.grad)
            for (int c = threadIdx.x; c < (a.H >> 3); c += 256)
                reinterpret_cast<uint4*>(a.grad + t * a.H)[c] = make_uint4(0, 0, 0, 0);
        return;
    }
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        const float S0 = a.sum[t], lse = __builtin_fmaf(a.frame[t], LN2, logf(S0));
        const float inv_n = a.inv_n[0];
        const int lab = a.labels ? a.labels[t] : -1;
        const float zl = a.zs[t * slots + a.k];
        // the teacher's softmax over its ids inside the vocabulary
        int id = lane < a.k ? a.top_i[t * a.k + lane] : -1;
        if (id >= a.V) id = -1;
        const float tv = id >= 0 ? a.top_v[t * a.k + lane] : -INFINITY;
        const float z = id >= 0 ? a.zs[t * slots + lane] : 0.0f;
        const float tm = wave_max(tv);
        const bool some = a.k > 0 && tm != -INFINITY;
        const float te = tv == -INFINITY ? 0.0f : expf(tv - tm);
        const float ts = wave_sum(te);
        const float pt = some ? te / ts : 0.0f;
        const float kd = wave_sum(pt == 0.0f ? 0.0f : pt * (tv - tm - logf(ts) - (z - lse)));
        const float ws = a.labels ? a.lm_w : 0.0f, wd = some ? a.dist_w : 0.0f;
        const float c = ws + wd;
        // an id's q counts once, at its first slot; the label's slot is the first of all
        bool own = id >= 0 && id != lab;
        for (int j = 0; j < a.k; ++j) {
            const int o = __builtin_amdgcn_readlane(id, j);
            if (j < lane && o == id) own = false;
        }
        if (lane < a.k) {
            s_id[lane] = id;
            s_coef[lane] = id < 0 ? 0.0f : inv_n * ((own ? c * expf(z - lse) : 0.0f) - wd * pt);
        }
        if (lane == 0) {
            s_id[a.k] = lab;
            s_coef[a.k] = lab < 0 ? 0.0f : inv_n * (c * expf(zl - lse) - ws);
            s_c = inv_n * c / S0;
            a.row_loss[t] = (a.labels ? ws * (lse - zl) : 0.0f) + (some ? wd * kd : 0.0f);
        }
    }
    if (!a.grad) return;
    __syncthreads();
    const float cs = s_c;
    typedef uint32_t words __attribute__((ext_vector_type(VEC / 2)));
    for (int c = threadIdx.x; c < a.H / VEC; c += 256) {
        float o[VEC];
        const int64_t at = t * a.H + VEC * c;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = 0.0f;
#pragma unroll 8
        for (int s = 0; s < a.splits; ++s) {
            const float4* g = reinterpret_cast<const float4*>(a.g + (int64_t)s * a.T * a.H + at);
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float4 x = g[i];
                o[4 * i] += x.x; o[4 * i + 1] += x.y; o[4 * i + 2] += x.z; o[4 * i + 3] += x.w;
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] *= cs;
#pragma unroll 4
        for (int j = 0; j < slots; ++j) {
            const float k = s_coef[j];
            const int id = max(s_id[j], 0);              // an absent slot has k = 0
            const words x = reinterpret_cast<const words*>(a.w + (int64_t)id * a.H)[c];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                o[2 * i] = __builtin_fmaf(k, __uint_as_float(x[i] << 16), o[2 * i]);
                o[2 * i + 1] = __builtin_fmaf(k, __uint_as_float(x[i] & 0xffff0000u), o[2 * i + 1]);
            }
        }
        words r;
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) r[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
        *reinterpret_cast<words*>(a.grad + at) = r;
    }
}

// loss = inv_n times the sum of the row losses, in fp64 and a fixed order
__global__ __launch_bounds__(1024) void k_head_mean(HeadArgs a, float* loss) {
    __shared__ double red[1024];
    double acc = 0.0;
    for (int64_t t = threadIdx.x; t < a.T; t += 1024) acc += a.row_loss[t];
    red[threadIdx.x] = acc;
    __syncthreads();
    for (int w = 512; w > 0; w >>= 1) {
        if ((int)threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
        __syncthreads();
    }
    if (threadIdx.x == 0) loss[0] = a.T > 0 ? (float)(red[0] * (double)a.inv_n[0]) : 0.0f;
}

}  // namespace

// The vocabulary's pieces and the second product's splits.  P of a piece takes
// at most 640 MB (and a piece of the weight 2 GB, the reach of a buffer
// resource's offsets); of the numbers of equal pieces from the least on, up to
// half as many again, the one whose first products fill the 256 CUs in the
// fewest rounds of tiles.  (16384 tokens of 151936 entries: 18.0 ms; with 1300
// MB 17.6, with 2600 17.4, half of what the logits take.)  Where the gradient's
// tiles are fewer than the CUs the piece is split until they are about as many.
HeadPlan head_plan(int64_t T, int64_t H, int64_t V) {
    HeadPlan p{};
    const int64_t mt = (T + BM - 1) / BM, nt = (H + BN - 1) / BN;
    int64_t most = ((int64_t)640 << 20) / (2 * (T > 0 ? T : 1));
    if (most > ((int64_t)1 << 30) / H) most = ((int64_t)1 << 30) / H;
    most = most / BN * BN;
    if (most < BN) most = BN;
    const int64_t least = (V + most - 1) / most;
    int64_t best = -1;
    for (int64_t n = least; n <= least + least / 2 && n <= least + 32; ++n) {
        const int64_t vc = ((V + n - 1) / n + BN - 1) / BN * BN, pieces = (V + vc - 1) / vc;
        const int64_t rounds = pieces * ((mt * (vc / BN) + 255) / 256);
        if (best >= 0 && rounds >= best) continue;
        best = rounds;
        p.vc = (int)vc;
        p.pieces = (int)pieces;
    }
    const int64_t tiles = mt * nt > 0 ? mt * nt : 1;
    int64_t sp = 256 / tiles;
    if (sp > p.vc / (8 * BK)) sp = p.vc / (8 * BK);
    if (sp < 1) sp = 1;
    p.ksplit = (int)(((p.vc + sp - 1) / sp + BK - 1) / BK * BK);
    p.splits = (p.vc + p.ksplit - 1) / p.ksplit;
    return p;
}

hipError_t launch_head(HeadArgs a, const HeadPlan& pl, float* loss, hipStream_t st) {
    if (a.T > 0) {
        // Tiles of equally many rows, in whole sub-tiles: 333 tokens are 192 and
        // 141, not 256 and 77, and a tile's time goes with its sub-tiles.
        a.bm = (int)(((a.T + (a.T + BM - 1) / BM - 1) / ((a.T + BM - 1) / BM) + 31) / 32 * 32);
        const int64_t mt = (a.T + a.bm - 1) / a.bm, nt = (a.H + BN - 1) / BN;
        a.vc = pl.vc;
        a.splits = pl.splits;
        a.ksplit = pl.ksplit;
        hipLaunchKernelGGL(k_head_sparse, grid_of(a.T + 1), dim3(256), 0, st, a);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        for (int i = 0; i < pl.pieces; ++i) {
            a.c0 = (int64_t)i * pl.vc;
            a.first = i == 0;
            const unsigned g1 = (unsigned)std::min<int64_t>((mt * (pl.vc / BN) + 7) / 8 * 8, a.H % (2 * BK) == 0 ? CUS : INT32_MAX);
            if (a.grad) hipLaunchKernelGGL(k_head_probs<true>, dim3(g1), dim3(512), 0, st, a);
            else hipLaunchKernelGGL(k_head_probs<false>, dim3(g1), dim3(512), 0, st, a);
            if (a.T >= 1024) hipLaunchKernelGGL(k_head_merge<16>, dim3((unsigned)((a.T + 15) / 16)), dim3(1024), 0, st, a);
            else hipLaunchKernelGGL(k_head_merge<4>, dim3((unsigned)((a.T + 3) / 4)), dim3(1024), 0, st, a);
            if (a.grad)
                hipLaunchKernelGGL(k_head_grad, dim3((unsigned)((mt * nt * pl.splits + 7) / 8 * 8)), dim3(512), 0, st,
                                   a);
            err = hipGetLastError();
            if (err != hipSuccess) return err;
        }
        // 4 columns a thread where the splits' sums are the most that is read,
        // for more threads; 8 where the weight's rows are (333 tokens, 32 splits
        // and no teacher: 9.6 us and 13.8; 2048, 4 splits and 65 rows: 111 and 96)
        if (pl.splits > a.k + 1) hipLaunchKernelGGL(k_head_out<4>, dim3((unsigned)a.T), dim3(256), 0, st, a);
        else hipLaunchKernelGGL(k_head_out<8>, dim3((unsigned)a.T), dim3(256), 0, st, a);
    }
    hipLaunchKernelGGL(k_head_mean, dim3(1), dim3(1024), 0, st, a, loss);
    return hipGetLastError();
}

}  // namespace fq
