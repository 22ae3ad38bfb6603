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
// beside fp32 sums (P's rounding, 2^-9 of each term, averages out over the
// product's sum).  The two products carry the time.
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
typedef KTile<BM, BK, NW> KT;             // a reduction-contiguous operand
typedef MNTile<BN, BK, NW> MT;            // the weight as [vocabulary, hidden], reduced over the vocabulary
constexpr int SMEM = S * (KT::BYTES + KT::BYTES);
static_assert(KT::BYTES == MT::BYTES, "both products use one LDS layout");
static_assert(BM * BN * 2 <= SMEM, "the output tile fits the stages");

// acc = A B^T over nk steps of 64 on eight waves in two groups of four that
// alternate between a memory phase (fragments of one step into registers, the
// loads of a later step) and a compute phase (that step's MFMAs), one phase
// apart: on each SIMD one wave issues MFMAs while the other reads.  Group 0
// issues the loads of step k + 1 in its memory phase of step k, into the stage
// both groups finished reading in the two phases before; group 1 issues those
// of step k + 2 after its own reads of step k, which group 0 made one phase
// earlier.  Each group waits for its loads of step k + 1 before the barrier
// that opens group 0's memory phase of that step.  nti: this wave's 32-row
// sub-tiles that hold rows; tail0 runs on group 0 while group 1 computes its
// last step (LDS is free then).
template <class AT, class BT, typename F>
__device__ __forceinline__ void product(AT& la, BT& lb, f32x16 (&acc)[WTM][WTN], lds_t* smem, int nk, int nti,
                                        F&& tail0) {
    constexpr int LOADS = AT::PER_WAVE + BT::PER_WAVE;
    const int w = wave_id(), grp = w >> 2;
    typename AT::template Frags<WTM> fa;
    typename BT::template Frags<WTN> fb;
    fa.prep((w / WVN) * 32 * WTM);
    fb.prep((w % WVN) * 32 * WTN);
    bf16x8 af[KS][WTM], bfr[KS][WTN];
    auto issue = [&](int kt) {
        la.issue(smem + (kt % S) * AT::BYTES, kt * BK);
        lb.issue(smem + S * AT::BYTES + (kt % S) * BT::BYTES, kt * BK);
    };
    auto bar = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int a = 0; a < WTM; ++a)
#pragma unroll
        for (int b = 0; b < WTN; ++b)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;
    const int last = grp == 0 ? S - 2 : S - 1;
#pragma unroll
    for (int p = 0; p < S; ++p)
        if (p <= last && p < nk) issue(p);
    wait_steps<LOADS>(min(last, nk - 1));
    bar();
    if (grp == 1) bar();
    auto phases = [&](int kt, int st, auto part_c) {
        constexpr bool PART = decltype(part_c)::value;
        if (grp == 0 && kt + S - 1 < nk) issue(kt + S - 1);
        const lds_t* sa = smem + st * AT::BYTES;
        const lds_t* sb = smem + S * AT::BYTES + st * BT::BYTES;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int t = 0; t < WTM; ++t)
                if (!PART || t < nti) af[kk][t] = fa.get(sa, t, kk);
            if (!PART || nti > 0)
#pragma unroll
                for (int t = 0; t < WTN; ++t) bfr[kk][t] = fb.get(sb, t, kk);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (grp == 1) {
            if (kt + S < nk) issue(kt + S);
            wait_steps<LOADS>(min(S - 1, nk - 2 - kt));
        }
        bar();
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
            for (int ti = 0; ti < WTM; ++ti)
                if (!PART || ti < nti)
#pragma unroll
                    for (int tj = 0; tj < WTN; ++tj)
                        acc[ti][tj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bfr[kk][tj], af[kk][ti], acc[ti][tj], 0,
                                                                              0, 0);
        if (grp == 0) wait_steps<LOADS>(min(S - 2, nk - 2 - kt));
        bar();
    };
    auto steps = [&](auto part_c) {
        for (int kt = 0; kt < nk; kt += S) {
#pragma unroll
            for (int u = 0; u < S; ++u)
                if (kt + u < nk) phases(kt + u, u, part_c);
        }
    };
    if (nti >= WTM) steps(std::false_type{});
    else steps(std::true_type{});
    if (grp == 0) {
        tail0();
        bar();
    }
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
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
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
    for (int j = w; j < slots; j += 4) {
        const int id = j < a.k ? a.top_i[t * a.k + j] : (a.labels ? a.labels[t] : -1);
        float z = -INFINITY;
        if (id >= 0 && id < a.V) {
            const uint4* wr = reinterpret_cast<const uint4*>(a.w + (int64_t)id * a.H);
            float acc = 0.0f;
            for (int c = lane; c < nvec; c += 64) {
                float x[8], y[8];
                unpack8(hr[c], x);
                unpack8(wr[c], y);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc = __builtin_fmaf(x[i], y[i], acc);
            }
            z = wave_sum(acc);
        }
        if (lane == 0) sz[j] = z;
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
template <bool GRAD>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) void k_head_probs(HeadArgs a) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM];
    lds_t* smem = (lds_t*)smem_raw;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / WVN, wn = wave % WVN;
    const int mt = (int)((a.T + BM - 1) / BM), nt = a.vc / BN;
    const int tile = xcd_tile(blockIdx.x, gridDim.x, mt * nt);
    if (tile < 0) return;
    int tm, tn;
    tile_of(tile, mt, nt, &tm, &tn);
    const int64_t m0 = (int64_t)tm * BM;
    const int rows = (int)min((int64_t)BM, a.T - m0);
    const int64_t v0 = a.c0 + (int64_t)tn * BN;               // first vocabulary entry of the tile
    const int cols = (int)min((int64_t)BN, a.V - v0);         // may be <= 0 in the last piece's padding
    KT la, lb;
    la.init(make_rsrc_words(a.h + m0 * a.H, (int64_t)rows * a.H * 2), a.H);
    lb.init(make_rsrc_words(a.w + (cols > 0 ? v0 : 0) * a.H, (int64_t)cols * a.H * 2), a.H);
    f32x16 acc[WTM][WTN];
    float frame[WTM];
#pragma unroll
    for (int ti = 0; ti < WTM; ++ti) {
        const int64_t t = m0 + wm * 128 + ti * 32 + (lane & 31);
        frame[ti] = t < a.T ? a.frame[t] : 0.0f;
    }
    constexpr int RB = BN * 2, CH = BN / 8;
    // lane holds z of token lane%32 and columns 8 (v/4) + 4 (lane/32) + v%4 of
    // each 32 x 32 sub-tile: a token's 64 columns of this wave are its own 32
    // and lane ^ 32's
    auto epilogue = [&]() {
#pragma unroll
        for (int ti = 0; ti < WTM; ++ti) {
            const int row = wm * 128 + ti * 32 + (lane & 31);
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
            float f = m <= frame[ti] + FRAME_SLACK ? frame[ti] : ceilf(m);
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
                    for (int q = 0; q < 4; ++q) {
                        const int col = wn * 64 + tj * 32 + 8 * q + 4 * (lane >> 5);
                        const int off = row * RB + (((col >> 3) ^ (row & 15)) << 4) + (col & 7) * 2;
                        *reinterpret_cast<__attribute__((address_space(3))) uint64_t*>(smem + off) =
                            (uint64_t)pack_bf16(acc[ti][tj][4 * q], acc[ti][tj][4 * q + 1]) |
                            ((uint64_t)pack_bf16(acc[ti][tj][4 * q + 2], acc[ti][tj][4 * q + 3]) << 32);
                    }
        }
    };
    const int nti = min(max((rows - wm * 128 + 31) / 32, 0), WTM);
    product(la, lb, acc, smem, a.H / BK, nti, epilogue);
    if (wave_id() >= 4) epilogue();
    if (!GRAD) return;
    __syncthreads();
    constexpr int RPI = 64 / CH, NIT = BM / (RPI * NW);
    u32x4 cv[NIT];
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
        const int row = (it * NW + wave) * RPI + lane / CH, c = lane % CH;
        cv[it] = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(smem + row * RB +
                                                                                   ((c ^ (row & 15)) << 4));
    }
    const __amdgpu_buffer_rsrc_t prs =
        make_rsrc(a.p + m0 * a.vc + (int64_t)tn * BN, (int64_t)(rows - 1) * a.vc * 2 + BN * 2);
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
        const int row = (it * NW + wave) * RPI + lane / CH, c = lane % CH;
        __builtin_amdgcn_raw_buffer_store_b128(cv[it], prs, (uint32_t)row * (uint32_t)a.vc * 2u + c * 16, 0, 2);
    }
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
        a.sum[t] = (a.sum[t] == 0.0f ? 0.0f : a.sum[t] * step) + sum;
        a.frame[t] = f;
        a.step[t] = step;
    }
    if (a.p) {
        const int slots = a.k + 1;
        const int64_t t0 = (int64_t)blockIdx.x * TOK;
        const int n = (int)min((int64_t)TOK, a.T - t0) * slots;
        for (int i = threadIdx.x; i < n; i += 1024) {
            const int64_t r = t0 + i / slots;
            const int j = i % slots;
            const int id = j < a.k ? a.top_i[r * a.k + j] : (a.labels ? a.labels[r] : -1);
            if (id >= a.c0 && id < a.V && id - a.c0 < a.vc) a.p[r * a.vc + (id - a.c0)] = 0;
        }
    }
}

// ----------------------------------------------------------------- grad ---
// G[split][t, :] = (first piece ? 0 : step[t] G) + P W_piece over the split's
// share of the piece
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) void k_head_grad(HeadArgs a) {
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM];
    lds_t* smem = (lds_t*)smem_raw;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / WVN, wn = wave % WVN;
    const int mt = (int)((a.T + BM - 1) / BM), nt = (a.H + BN - 1) / BN;
    int tile = xcd_tile(blockIdx.x, gridDim.x, mt * nt * a.splits);
    if (tile < 0) return;
    const int split = tile / (mt * nt);
    tile -= split * mt * nt;
    int tm, tn;
    tile_of(tile, mt, nt, &tm, &tn);
    const int64_t m0 = (int64_t)tm * BM;
    const int rows = (int)min((int64_t)BM, a.T - m0);
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
    const int nti = min(max((rows - wm * 128 + 31) / 32, 0), WTM);
    product(la, lb, acc, smem, max(kn, 0) / BK, nti, []() {});
    float* G = a.g + (int64_t)split * a.T * a.H;
#pragma unroll
    for (int ti = 0; ti < WTM; ++ti) {
        const int row = wm * 128 + ti * 32 + (lane & 31);
        if (row >= rows) continue;
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
// j, k <= 64; the label is lane 0's second slot), then 8 columns per thread.
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
            const int o = __shfl(id, j);
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
    for (int c = threadIdx.x; c < (a.H >> 3); c += 256) {
        float o[8];
        const int64_t at = t * a.H + 8 * c;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0.0f;
        for (int s = 0; s < a.splits; ++s) {
            const float4* g = reinterpret_cast<const float4*>(a.g + (int64_t)s * a.T * a.H + at);
            const float4 x = g[0], y = g[1];
            o[0] += x.x; o[1] += x.y; o[2] += x.z; o[3] += x.w;
            o[4] += y.x; o[5] += y.y; o[6] += y.z; o[7] += y.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= cs;
#pragma unroll 4
        for (int j = 0; j < slots; ++j) {
            const float k = s_coef[j];
            const int id = max(s_id[j], 0);              // an absent slot has k = 0
            float x[8];
            unpack8(reinterpret_cast<const uint4*>(a.w + (int64_t)id * a.H)[c], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __builtin_fmaf(k, x[i], o[i]);
        }
        reinterpret_cast<uint4*>(a.grad + at)[0] = pack8(o);
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
// MB 17.6, with 2600 17.4, half of what the logits take.)  Where the gradient's tiles are fewer than the CUs
// the piece is split until they are about as many.
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
        const int64_t mt = (a.T + BM - 1) / BM, nt = (a.H + BN - 1) / BN;
        a.vc = pl.vc;
        a.splits = pl.splits;
        a.ksplit = pl.ksplit;
        hipLaunchKernelGGL(k_head_sparse, dim3((unsigned)a.T + 1), dim3(256), 0, st, a);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        for (int i = 0; i < pl.pieces; ++i) {
            a.c0 = (int64_t)i * pl.vc;
            a.first = i == 0;
            const unsigned g1 = (unsigned)((mt * (pl.vc / BN) + 7) / 8 * 8);
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
        hipLaunchKernelGGL(k_head_out, dim3((unsigned)a.T), dim3(256), 0, st, a);
    }
    hipLaunchKernelGGL(k_head_mean, dim3(1), dim3(1024), 0, st, a, loss);
    return hipGetLastError();
}

}  // namespace fq
