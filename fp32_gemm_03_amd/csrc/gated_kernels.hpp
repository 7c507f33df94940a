// gated_kernels.hpp -- a gated feed-forward block's products on the matrix cores:
// gate = x G, up = x U, y = act(gate) up, and back.
//
//   * gated_tile: LDS tiles; one product of x with [G | U] (the activation in the
//     epilogue), dgate G^T + dup U^T as one sum, or x^T [dgate | dup].
//   * gated_thin: few rows; operands from memory straight to the matrix cores.
//   * gated_and_rest: 64-row tiles, the last rows as few.
//   * gated_slopes: dgate and dup from dy and what the forward kept.
//   * gated_back_few, gated_back_tiles: dx's tiles and the weights' in one launch.
//   * gated_simple: any strides.
#pragma once

#include "activations.hpp"
#include "lanes.hpp"

namespace gatedk {

using rowk::f32x4u;
using rowk::rsrc_t;
using rowk::whole_rsrc;
using sgk::f32x2;
using sgk::f32x4;
using sgk::floatx16;
typedef float floatx4 __attribute__((ext_vector_type(4)));

template <int ACT> __device__ __forceinline__ float act32(float g) { return normk::act<ACT>(g); }
__device__ __forceinline__ float act32(int kind, float g) {
    return kind == normk::kSilu ? act32<normk::kSilu>(g) : kind == normk::kGelu ? act32<normk::kGelu>(g)
                                                                                 : act32<normk::kGeluTanh>(g);
}
__device__ __forceinline__ float gated(int kind, float g, float u) { return act32(kind, g) * u; }

enum Kind { FORWARD, BACK_X, BACK_W };

// What is summed, by kind (M x N the result):
//   FORWARD  A x (M x K), B G and U (K x N)         K of both the same
//   BACK_X   A dgate and dup (M x K), B G and U (N x K)   one sum over both
//   BACK_W   A x (K x M), B dgate and dup (K x N)   a result each
struct TileArgs {
    int M, N, K, act;
    const float *A[2], *B[2];
    int64_t lda, ldb[2];
    float beta;
    float *C[2], *gate, *up;  // FORWARD: C[0] is y, gate and up may be NULL
    int64_t ldc[2], ldgate, ldup;
    int xcd_shift;
    int shares;  // BACK_X, BACK_W: of the sum, share s at C[..] + s M ldc[..]
};

// ---------------------------------------------------------------------------
// One operand's part of an LDS stage, filled by loads that write LDS directly
// (instruction p of wave w fills floats (p WAVES + w) 256 ..).
//   Along K (`Long`): rows of BK floats, the 16-byte chunks of a row permuted so
//     that loads and fragment reads both touch every bank (AKLayout).
//   Across (`Wide`): BK rows of COLS floats as they are.
// ---------------------------------------------------------------------------
template <int ROWS, int BK, int NT> struct Long {
    static constexpr int WAVES = NT / 64, P = ROWS * BK / (NT * 4), SIZE = ROWS * BK;
    static_assert(P * NT * 4 == ROWS * BK, "whole instructions");
    uint32_t off[P];
    int col[P];
    __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int f = (p * WAVES + wave) * 256 + 4 * lane, row = f / BK;
            col[p] = 4 * sgk::AKLayout<BK>::chunk_pos(row, f % BK / 4);
            off[p] = (uint32_t)((row * ld + col[p]) * 4);
        }
    }
    // r begins at the tile's first row and column; `left` columns of K are there
    __device__ __forceinline__ void load(rsrc_t r, float *lds, int wave, int p, int left) const {
        sgk::load_to_lds<4>(r, lds + (p * WAVES + wave) * 256, col[p] < left ? off[p] : rowk::kOut);
    }
    // the chunk that holds K's last column also brought what follows it in the row
    __device__ __forceinline__ void clear(float *lds, int wave, int lane, int left) const {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int n = left - col[p];
            float *q = lds + (p * WAVES + wave) * 256 + 4 * lane;
            if (n > 0 && n < 4)
#pragma unroll
                for (int j = 1; j < 4; ++j)
                    if (j >= n) q[j] = 0.0f;
        }
    }
};
template <int COLS, int BK, int NT> struct Wide {
    static constexpr int WAVES = NT / 64, P = COLS * BK / (NT * 4), SIZE = COLS * BK;
    static_assert(P * NT * 4 == COLS * BK, "whole instructions");
    uint32_t off[P];
    __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int f = (p * WAVES + wave) * 256 + 4 * lane;
            off[p] = (uint32_t)((f / COLS * ld + f % COLS) * 4);
        }
    }
    __device__ __forceinline__ void load(rsrc_t r, float *lds, int wave, int p, int) const {
        sgk::load_to_lds<4>(r, lds + (p * WAVES + wave) * 256, off[p]);
    }
};

// ---------------------------------------------------------------------------
// Tiles of BM x BN (FORWARD: BN / 2 columns of gate and the same of up), K in tiles
// of BK, two LDS stages, WM x WN per wave with v_mfma_f32_32x32x2_f32.  Within a K
// tile lane half lh takes k = lh BK / 2 + j in k-step j, of both operands.
// KG 2: two groups of waves take half of a K tile's steps each, then add up half of the sums each.
// FORWARD's wave holds gate and up of the same columns (block columns 2 j and 2 j +
// 1), so the activation's product is taken in registers.  Bound by the matrix cores, busy
// for 93% of 4096 x 4096 x 2048 on 256 x 256 tiles (964 us, 142.5 TFLOP/s; sgemm takes 948 for the
// same work), for 84% of 2000 x 2048 x 1024 on 128 x 128 (134 us): the ring's start and the stores
// at the end are a larger part of fewer K tiles.
// ---------------------------------------------------------------------------
template <int KIND, int BM, int BN, int BK, int WM, int WN, int KG = 1>
__device__ __forceinline__ void gated_tile_of(const TileArgs &a, int block, float *smem) {
    constexpr int MI = WM / 32, NI = WN / 32, WAVES_N = BN / WN, WPG = (BM / WM) * WAVES_N, NT = KG * WPG * 64;
    static_assert(KG == 1 || KG == 2, "wave groups");
    constexpr bool DUAL = KIND == FORWARD, A_WIDE = KIND == BACK_W, B_LONG = KIND == BACK_X;
    constexpr int CN = DUAL ? BN / 2 : BN;  // columns of the result
    static_assert(!DUAL || NI % 2 == 0, "gate and up in pairs of block columns");
    typedef typename std::conditional<A_WIDE, Wide<BM, BK, NT>, Long<BM, BK, NT>>::type SA;
    typedef typename std::conditional<B_LONG, Long<BN, BK, NT>, Wide<CN, BK, NT>>::type SB;
    constexpr int STAGE = (BM + BN) * BK;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 31, lh = lane >> 5;
    const int group = KG == 1 ? 0 : wave / WPG, wm = wave % WPG / WAVES_N * WM, wn = wave % WAVES_N * WN;
    const int nbm = (a.M + BM - 1) / BM, nbn = (a.N + CN - 1) / CN;
    int tm, tn, share = 0;
    const int columns = KIND == BACK_W ? 2 * nbn : nbn;
    if (KIND != FORWARD && a.shares > 1) {
        share = block / (nbm * columns);
        block -= share * (nbm * columns);
    }
    sgk::tile_of<2, 8>(block, nbm, columns, a.xcd_shift, tm, tn);
    const int which = KIND == BACK_W && tn >= nbn ? 1 : 0;  // BACK_W: dG's columns, then dU's
    const int bm = tm * BM, bn = (tn - which * nbn) * CN;

    SA sa;
    SB sb;
    sa.init(a.lda, wave, lane);
    sb.init(a.ldb[which], wave, lane);  // (FORWARD and BACK_X: of both)
    SB sb2;
    if constexpr (KIND != BACK_W) sb2.init(a.ldb[1], wave, lane);

    const int KT1 = (a.K + BK - 1) / BK, KT = KIND == BACK_X ? 2 * KT1 : KT1;
    // the K tiles of this workgroup (BACK_X: of dgate's and then dup's)
    int T0 = 0, T1 = KT;
    if (KIND != FORWARD && a.shares > 1) {  // (up to 16 shares of 2^27)
        T0 = (int)((uint32_t)KT * (uint32_t)share / (uint32_t)a.shares);
        T1 = (int)((uint32_t)KT * (uint32_t)(share + 1) / (uint32_t)a.shares);
    }
    // loads of K tile t, piece p: A's, then B's (DUAL: G's, then U's)
    constexpr int DP = SA::P + (DUAL ? 2 : 1) * SB::P;
    auto fetch = [&](float *st, int t, int p) {
        const int seg = KIND == BACK_X && t >= KT1 ? 1 : 0;
        const int64_t k0 = (int64_t)(t - seg * KT1) * BK;
        const int64_t left = t < T1 ? a.K - k0 : 0;  // (past the last tile nothing is read)
        if (p < SA::P) {
            const float *A = a.A[seg];
            const rsrc_t r = A_WIDE ? whole_rsrc(A + k0 * a.lda + bm, left > 0 ? ((left - 1) * a.lda + (a.M - bm)) * 4 : 0)
                                    : whole_rsrc(A + (int64_t)bm * a.lda + k0,
                                                 left > 0 ? ((int64_t)(a.M - bm - 1) * a.lda + left) * 4 : 0);
            sa.load(r, st, wave, p, (int)left);
            return;
        }
        p -= SA::P;
        const int src = DUAL ? (p >= SB::P ? 1 : 0) : KIND == BACK_X ? seg : which;
        const float *B = a.B[src];
        const int64_t ldb = a.ldb[src];
        const rsrc_t r = B_LONG ? whole_rsrc(B + (int64_t)bn * ldb + k0, left > 0 ? ((int64_t)(a.N - bn - 1) * ldb + left) * 4 : 0)
                                : whole_rsrc(B + k0 * ldb + bn, left > 0 ? ((left - 1) * ldb + (a.N - bn)) * 4 : 0);
        float *lds = st + SA::SIZE;
        if constexpr (DUAL) {
            if (src == 1) sb2.load(r, lds + SB::SIZE, wave, p - SB::P, (int)left);
            else sb.load(r, lds, wave, p, (int)left);
        } else if constexpr (KIND == BACK_X) {
            if (src == 1) sb2.load(r, lds, wave, p, (int)left);
            else sb.load(r, lds, wave, p, (int)left);
        } else {
            sb.load(r, lds, wave, p, (int)left);
        }
    };
    auto landed = [&](float *st, int t) {
        rowk::wait_loads<0>();
        if constexpr (KIND != BACK_W) {
            const int left = a.K - (KIND == BACK_X && t >= KT1 ? t - KT1 : t) * BK;
            if ((a.K & 3) != 0 && t < T1 && left > 0 && left < BK) {
                sa.clear(st, wave, lane, left);
                if constexpr (B_LONG) sb.clear(st + SA::SIZE, wave, lane, left);
                __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt 0
            }
        }
        rowk::meet();
    };

    // With one block a wave, odd k-steps have a sum of their own: MFMAs that add to one sum wait
    // for each other, and two shorter sums are nearer to 64 bits.
    constexpr int SUMS = MI * NI == 1 ? 2 : 1;
    floatx16 sums[SUMS][MI][NI];
#pragma unroll
    for (int c = 0; c < SUMS; ++c)
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) sums[c][i][j][r] = 0.0f;
    floatx16(&acc)[MI][NI] = sums[0];

    // A chunk is four k-steps: q of BK / 8 / KG, lane half lh and wave group their own
    constexpr int QN = BK / 8 / KG;
    static_assert(KG == 1 || QN % 2 == 0, "two sets of fragments");
    int at[QN];  // of a row's chunk (rows wm + 32 i and wn + 32 j + li: one permutation)
    if constexpr (!A_WIDE) {
#pragma unroll
        for (int q = 0; q < QN; ++q) at[q] = 4 * sgk::AKLayout<BK>::chunk_pos(li, lh * (BK / 8) + group * QN + q);
    }
    const int k_at = lh * (BK / 2) + group * 4 * QN;  // row of a stage that is across
    const int a_at = A_WIDE ? k_at * BM + wm + MI * li : (wm + li) * BK;
    const int b_at = SA::SIZE + (B_LONG ? (wn + li) * BK : k_at * CN + (DUAL ? wn / 2 + NI / 2 * li : wn + NI * li));

    float av[2][MI][4], bv[2][NI][4];
    auto read = [&](const float *__restrict__ st, int q) {
        const int d = q & 1;
        if constexpr (B_LONG) {
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(st + b_at + j * 32 * BK + at[q]);
                bv[d][j][0] = v.x;
                bv[d][j][1] = v.y;
                bv[d][j][2] = v.z;
                bv[d][j][3] = v.w;
            }
        } else {
            constexpr int W = DUAL ? NI / 2 : NI;
            typedef typename sgk::vec_t<W>::type V;
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int s = 0; s < (DUAL ? 2 : 1); ++s) {
                    const V v = *reinterpret_cast<const V *>(st + b_at + s * SB::SIZE + (4 * q + e) * CN);
#pragma unroll
                    for (int j = 0; j < W; ++j) bv[d][DUAL ? 2 * j + s : j][e] = sgk::vget(v, j);
                }
        }
        if constexpr (A_WIDE) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                typedef typename sgk::vec_t<MI>::type V;
                const V v = *reinterpret_cast<const V *>(st + a_at + (4 * q + e) * BM);
#pragma unroll
                for (int i = 0; i < MI; ++i) av[d][i][e] = sgk::vget(v, i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const float4 v = *reinterpret_cast<const float4 *>(st + a_at + i * 32 * BK + at[q]);
                av[d][i][0] = v.x;
                av[d][i][1] = v.y;
                av[d][i][2] = v.z;
                av[d][i][3] = v.w;
            }
        }
    };
    auto multiply = [&](int q, auto between) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    floatx16 &sum = sums[e % SUMS][i][j];
                    sum = __builtin_amdgcn_mfma_f32_32x32x2f32(av[q & 1][i][e], bv[q & 1][j][e], sum, 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    between((e * MI + i) * NI + j);
                }
    };
    if (T0 < T1) {
        // Fragments are read a chunk ahead, across the tiles' borders: a tile's last chunk is
        // multiplied behind the barrier that ends its reads, and the loads of tile t + 2 go
        // between its MFMAs, into the stage that was read.
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int p = 0; p < DP; ++p) fetch(smem + s * STAGE, T0 + s, p);
        landed(smem, T0);
        read(smem, 0);
        for (int t = T0; t < T1; ++t) {
            float *st = smem + (t - T0 & 1) * STAGE, *next = smem + (t - T0 + 1 & 1) * STAGE;
#pragma unroll
            for (int q = 0; q + 1 < QN; ++q) {
                read(st, q + 1);
                multiply(q, [](int) {});
            }
            landed(next, t + 1);
            read(next, 0);
            multiply(QN - 1, [&](int u) {
                constexpr int U = 4 * MI * NI;
#pragma unroll
                for (int p = 0; p < DP; ++p)
                    if (p * U / DP == u) fetch(st, t + 2, p);
                __builtin_amdgcn_sched_barrier(0);
            });
        }
        rowk::wait_loads<0>();
        if constexpr (SUMS == 2) {
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[0][0][r] += sums[1][0][0][r];
        }
    }
    if constexpr (KG == 2) {  // each group adds up and stores one half of the registers
        static_assert(2 * (BM + BN) * BK >= KG * WPG * MI * NI * 8 * 64, "the other group's half");
        rowk::meet();  // (every wave is past its last reads)
        floatx4 *part = reinterpret_cast<floatx4 *>(smem) + lane;
        auto place = [&](int of, int i, int j, int h) { return 64 * (((of * WPG + wave % WPG) * MI * NI + i * NI + j) * 2 + h); };
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int g = 0; g < 2; ++g)
                        if (g != group) {
                            const int r = 8 * g + 4 * h;
                            part[place(g, i, j, h)] = floatx4{acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
                        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const floatx4 v = part[place(group, i, j, h)];
#pragma unroll
                    for (int g = 0; g < 2; ++g)
                        if (g == group)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][j][8 * g + 4 * h + e] += v[e];
                }
    }

    // Register r of block (i, j) on lane (li, lh): block row 8 (r / 4) + 4 lh + r % 4 = b
    // of the wave's row 32 i + b (A along K) or MI b + i (across); column 32 j + li (B
    // along K), NI li + j (across), NI / 2 li + j / 2 of gate (even j) and up (odd).
    const int W = DUAL ? NI / 2 : NI;
    float *const C = a.C[which] + (int64_t)share * a.M * a.ldc[which];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (KG == 2 && r / 8 != group) continue;
            const int b = 8 * (r >> 2) + 4 * lh + (r & 3);
            const int m = bm + wm + (A_WIDE ? MI * b + i : 32 * i + b);
            if (m >= a.M) continue;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int n = bn + (B_LONG ? wn + 32 * j + li : DUAL ? wn / 2 + W * li + j : wn + W * li + j);
                if (n >= a.N) continue;
                float *c = C + (int64_t)m * a.ldc[which] + n;
                if constexpr (DUAL) {
                    const float g = acc[i][2 * j][r], u = acc[i][2 * j + 1][r];
                    *c = gated(a.act, g, u);
                    if (a.gate != nullptr) {
                        a.gate[(int64_t)m * a.ldgate + n] = g;
                        a.up[(int64_t)m * a.ldup + n] = u;
                    }
                } else {
                    *c = a.beta != 0.0f ? fmaf(a.beta, *c, acc[i][j][r]) : acc[i][j][r];
                }
            }
        }
}

template <int KIND, int BM, int BN, int BK, int WM, int WN, int KG, int WPE>
__global__ void __launch_bounds__(KG * (BM / WM) * (BN / WN) * 64) __attribute__((amdgpu_waves_per_eu(WPE)))
gated_tile(TileArgs a) {
    __shared__ __attribute__((aligned(16))) float smem[2 * (BM + BN) * BK];
    gated_tile_of<KIND, BM, BN, BK, WM, WN, KG>(a, (int)blockIdx.x, smem);
}

// ---------------------------------------------------------------------------
// Few rows: reading G and U once is the work.  16 MB rows and 16 VW columns of both a
// workgroup, its WK waves each a share of K, operands from memory straight to
// v_mfma_f32_16x16x4_f32: lane (li, lk) loads VW consecutive columns of k = 4 lk + e
// of 16 k's, and the four k's of a row of x.  Partial sums meet in LDS in order.
// 29 x 4096 x 2048, 68 MB, 18.2 us, 3.7 TB/s: every line is read once, and the matrix cores
// are busy for 42% of it (29 rows fill 32).
// ---------------------------------------------------------------------------
// Tile columns go to the XCDs in turn in runs of RUN neighbours, which share lines where a
// tile is narrower than one or rows are not aligned (one row, 4096 x 2048 on 16 columns:
// 23.8 us in runs of one, 16.3 of two or four; 29 rows, 4095 x 2047 on 32: 25.2, 23.2, 22.8);
// a column's row tiles stay on its XCD.
template <int RUN>
__device__ __forceinline__ void thin_place(int id, int nbm, int nbn, int xcd_shift, int &tm, int &tn) {
    const int span = RUN << xcd_shift, dealt = nbn / span * span;
    if (id < dealt * nbm) {
        const int x = id & ((1 << xcd_shift) - 1), i = id >> xcd_shift, c = i / nbm;
        tm = i - c * nbm;
        tn = ((c / RUN << xcd_shift) + x) * RUN + c % RUN;
        return;
    }
    const int i = id - dealt * nbm, c = i / nbm;
    tm = i - c * nbm;
    tn = dealt + c;
}

template <int MB, int VW, int WK>
__device__ __forceinline__ void gated_thin_of(const TileArgs &a, int block, float *smem) {
    constexpr int BM = 16 * MB, BN = 16 * VW;
    float(*part)[2][BM * BN] = reinterpret_cast<float(*)[2][BM * BN]>(smem);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lk = lane >> 4;
    const int nbm = (a.M + BM - 1) / BM, nbn = (a.N + BN - 1) / BN;
    int tm, tn;
    thin_place<4>(block, nbm, nbn, a.xcd_shift, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const float *A = a.A[0] + (int64_t)m0 * a.lda;
    const int64_t a_bytes = ((int64_t)(a.M - m0 - 1) * a.lda + a.K) * 4;
    uint32_t ao[MB], bo[2][4];
#pragma unroll
    for (int i = 0; i < MB; ++i) ao[i] = (uint32_t)(((16 * i + li) * a.lda + 4 * lk) * 4);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) bo[s][e] = (uint32_t)(((4 * lk + e) * a.ldb[s] + VW * li) * 4);

    floatx4 acc[2][MB][VW];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j) acc[s][i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    const int steps = (a.K + 15) / 16;
    const int u0 = (int)((int64_t)steps * w / WK), u1 = (int)((int64_t)steps * (w + 1) / WK);
    constexpr int STEP = 8 * VW + 4 * MB, D = 96 / STEP < 8 ? (96 / STEP < 2 ? 2 : 96 / STEP) : 8;
    f32x4 av[D][MB];
    float bv[D][2][4][VW];
    auto fetch = [&](int d, int u) {  // (past the wave's last step the descriptors are empty)
        const int64_t k0 = 16 * (int64_t)u;
        const bool there = u < u1;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const rsrc_t rb = whole_rsrc(a.B[s] + k0 * a.ldb[s] + n0, there ? ((a.K - k0 - 1) * a.ldb[s] + (a.N - n0)) * 4 : 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (VW == 4) {
                    const f32x4 v = sgk::raw_load_v4f32(rb, bo[s][e], 0, 0);
                    bv[d][s][e][0] = v.x;
                    bv[d][s][e][1] = v.y;
                    bv[d][s][e][2] = v.z;
                    bv[d][s][e][3] = v.w;
                } else if constexpr (VW == 2) {
                    const f32x2 v = sgk::raw_load_v2f32(rb, bo[s][e], 0, 0);
                    bv[d][s][e][0] = v.x;
                    bv[d][s][e][1] = v.y;
                } else {
                    bv[d][s][e][0] = sgk::raw_load_f32(rb, bo[s][e], 0, 0);
                }
            }
        }
        const rsrc_t ra = whole_rsrc(A + k0, there ? a_bytes - 4 * k0 : 0);
#pragma unroll
        for (int i = 0; i < MB; ++i) av[d][i] = sgk::raw_load_v4f32(ra, ao[i], 0, 0);
    };
    auto multiply = [&](int d) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < VW; ++j)
#pragma unroll
                    for (int i = 0; i < MB; ++i)
                        acc[s][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[d][i][e], bv[d][s][e][j], acc[s][i][j], 0, 0, 0);
    };
    const int whole = (int64_t)u1 * 16 > a.K ? u1 - 1 : u1;
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, u0 + d);
    for (int u = u0; u < u1; u += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (u + d == whole) {  // K's end: x's row goes on into what follows it
                const int left = a.K - 16 * whole - 4 * lk;
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) av[d][i][e] = e < left ? av[d][i][e] : 0.0f;
            }
            if (u + d < u1) multiply(d);
            if (u + D < u1) fetch(d, u + d + D);
        }
    }
    // acc[s][i][j] register r on lane (li, lk): row 16 i + 4 lk + r, column VW li + j
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < VW; ++j) part[w][s][(16 * i + 4 * lk + r) * BN + VW * li + j] = acc[s][i][j][r];
    __syncthreads();
    for (int f = tid; f < BM * BN; f += WK * 64) {
        const int m = m0 + f / BN, n = n0 + f % BN;
        if (m >= a.M || n >= a.N) continue;
        float g = part[0][0][f], u = part[0][1][f];
#pragma unroll
        for (int i = 1; i < WK; ++i) {
            g += part[i][0][f];
            u += part[i][1][f];
        }
        a.C[0][(int64_t)m * a.ldc[0] + n] = gated(a.act, g, u);
        if (a.gate != nullptr) {
            a.gate[(int64_t)m * a.ldgate + n] = g;
            a.up[(int64_t)m * a.ldup + n] = u;
        }
    }
}

template <int MB, int VW, int WK, int WPE>
__global__ void __launch_bounds__(WK * 64) __attribute__((amdgpu_waves_per_eu(WPE))) gated_thin(TileArgs a) {
    __shared__ __attribute__((aligned(16))) float smem[WK * 2 * 16 * MB * 16 * VW];
    gated_thin_of<MB, VW, WK>(a, (int)blockIdx.x, smem);
}

// Rows in whole tiles of 64 x 64 and the last ones in tiles of 16 x 32 behind them.
struct RestArgs {
    TileArgs first, rest;
    int ahead;  // workgroups of the first rows: a multiple of 8, so that the others keep their XCDs
};
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4))) gated_and_rest(RestArgs a) {
    __shared__ __attribute__((aligned(16))) float smem[2 * (64 + 128) * 32];
    static_assert(8 * 2 * 16 * 32 <= 2 * (64 + 128) * 32, "the partial sums");
    const int block = (int)blockIdx.x;
    if (block >= a.ahead) gated_thin_of<1, 2, 8>(a.rest, block - a.ahead, smem);
    else if (block < a.first.M / 64 * ((a.first.N + 63) / 64)) gated_tile_of<FORWARD, 64, 128, 32, 32, 64, 2>(a.first, block, smem);
}

// ---------------------------------------------------------------------------
// Back from few rows, both gradients in one launch: the first workgroups compute dx, which
// reads G and U once, the others dG and dU, which they write once.
//   dx: 16 MB rows and 16 VW columns a workgroup; waves 0 to 3 a share of K each of dgate
//   G^T, waves 4 to 7 of dup U^T, operands (both along K) from memory straight to
//   v_mfma_f32_16x16x4_f32; a step is 32 of K, whole lines; partial sums meet in LDS.
//   A workgroup takes in 25 to 40 GB/s with the loads that it has in flight, which bounds dx where
//   it has few tiles (K split over workgroups as well: 29 rows, 2048 x 1024, 19.5 us with the launch
//   that adds them up, 22.0 without; 1 x 4096 x 2048 36.8 against 34.7; not kept).
// ---------------------------------------------------------------------------
struct BackArgs {
    TileArgs x, w;  // of BACK_X and BACK_W
    int ahead;      // workgroups of dx (few rows: a multiple of 8, so that the others keep their XCDs)
};

template <int MB, int VW> __device__ __forceinline__ void few_rows_dx(const TileArgs &a, int block, float *part) {
    constexpr int BM = 16 * MB, BN = 16 * VW, WK = 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int seg = wave / WK, w = wave % WK;
    const int li = lane & 15, lk = lane >> 4;
    const int nbm = (a.M + BM - 1) / BM, nbn = (a.N + BN - 1) / BN;
    if (block >= nbm * nbn) return;  // (rounded up to the XCDs)
    int tm, tn;
    thin_place<1>(block, nbm, nbn, a.xcd_shift, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const float *A = a.A[seg] + (int64_t)m0 * a.lda, *B = a.B[seg] + (int64_t)n0 * a.ldb[seg];
    const int64_t a_bytes = ((int64_t)(a.M - m0 - 1) * a.lda + a.K) * 4;
    const int64_t b_bytes = ((int64_t)(a.N - n0 - 1) * a.ldb[seg] + a.K) * 4;
    uint32_t ao[MB], bo[VW];
#pragma unroll
    for (int i = 0; i < MB; ++i) ao[i] = (uint32_t)(((16 * i + li) * a.lda + 8 * lk) * 4);
#pragma unroll
    for (int j = 0; j < VW; ++j) bo[j] = (uint32_t)(((16 * j + li) * a.ldb[seg] + 8 * lk) * 4);

    floatx4 acc[MB][VW];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < VW; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    const int steps = (a.K + 31) / 32;
    const int u0 = (int)((int64_t)steps * w / WK), u1 = (int)((int64_t)steps * (w + 1) / WK);
    constexpr int STEP = 8 * (MB + VW), D = 64 / STEP < 2 ? 2 : 64 / STEP;
    f32x4 av[D][2][MB], bv[D][2][VW];
    auto fetch = [&](int d, int u) {  // (past the wave's last step the descriptors are empty)
        const int64_t k0 = 32 * (int64_t)u;
        const rsrc_t ra = whole_rsrc(A + k0, u < u1 ? a_bytes - 4 * k0 : 0);
        const rsrc_t rb = whole_rsrc(B + k0, u < u1 ? b_bytes - 4 * k0 : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < VW; ++j) bv[d][h][j] = sgk::raw_load_v4f32(rb, bo[j] + 16 * h, 0, 0);
#pragma unroll
            for (int i = 0; i < MB; ++i) av[d][h][i] = sgk::raw_load_v4f32(ra, ao[i] + 16 * h, 0, 0);
        }
    };
    auto multiply = [&](int d) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int j = 0; j < VW; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[d][h][i][e], bv[d][h][j][e], acc[i][j], 0, 0, 0);
    };
    const int whole = (int64_t)u1 * 32 > a.K ? u1 - 1 : u1;
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, u0 + d);
    for (int u = u0; u < u1; u += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (u + d == whole) {  // K's end: both rows go on into what follows them
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int left = a.K - 32 * whole - 8 * lk - 4 * h;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
#pragma unroll
                        for (int i = 0; i < MB; ++i) av[d][h][i][e] = e < left ? av[d][h][i][e] : 0.0f;
#pragma unroll
                        for (int j = 0; j < VW; ++j) bv[d][h][j][e] = e < left ? bv[d][h][j][e] : 0.0f;
                    }
                }
            }
            if (u + d < u1) multiply(d);
            if (u + D < u1) fetch(d, u + d + D);
        }
    }
    // acc[i][j] register r on lane (li, lk): row 16 i + 4 lk + r, column 16 j + li
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < VW; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) part[wave * (BM * BN) + (16 * i + 4 * lk + r) * BN + 16 * j + li] = acc[i][j][r];
    __syncthreads();
    for (int f = tid; f < BM * BN; f += 2 * WK * 64) {
        const int m = m0 + f / BN, n = n0 + f % BN;
        if (m >= a.M || n >= a.N) continue;
        float sum = part[f];
#pragma unroll
        for (int i = 1; i < 2 * WK; ++i) sum += part[i * (BM * BN) + f];
        a.C[0][(int64_t)m * a.ldc[0] + n] = sum;
    }
}

template <int MB, int VW>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4))) gated_back_few(BackArgs a) {
    constexpr int TILE = 2 * (64 + 128) * 32, PART = 8 * 16 * MB * 16 * VW;
    __shared__ __attribute__((aligned(16))) float smem[TILE > PART ? TILE : PART];
    const int block = (int)blockIdx.x;
    if (block < a.ahead) few_rows_dx<MB, VW>(a.x, block, smem);
    else gated_tile_of<BACK_W, 64, 128, 32, 32, 32>(a.w, block - a.ahead, smem);
}

// Both gradients of many rows in one launch, dx's tiles ahead: a sum of 2 N products keeps a
// CU for longer than one of T, and a CU holds three workgroups.  Where that leaves CUs without work, the
// sums are cut into shares of K tiles that `gated_sum` adds up.  2000 x 2048 x 1024: 262 us, 128
// TFLOP/s, the matrix cores busy for 85% of it.
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4))) gated_back_tiles(BackArgs a) {
    __shared__ __attribute__((aligned(16))) float smem[2 * (128 + 64) * 32];
    const int block = (int)blockIdx.x;
    if (block < a.ahead) gated_tile_of<BACK_X, 128, 64, 32, 32, 32>(a.x, block, smem);
    else gated_tile_of<BACK_W, 128, 64, 32, 32, 32>(a.w, block - a.ahead, smem);
}

// What was summed in shares: out = beta out + the shares, in order.  A thread four columns.
struct Shares {
    int rows, cols, shares;
    float beta;
    const float *part;  // rows ldp apart, shares `rows` of them
    int64_t ldp, ldo, units;
    float *out;
    int blocks;  // up to this sum's last one
};
struct SharesArgs {
    Shares of[3];
};
__global__ void __launch_bounds__(256) gated_sum(SharesArgs all) {
    const int block = (int)blockIdx.x, which = block < all.of[0].blocks ? 0 : block < all.of[1].blocks ? 1 : 2;
    const Shares &a = all.of[which];
    const int64_t unit = (int64_t)(which > 0 ? block - all.of[which - 1].blocks : block) * 256 + threadIdx.x;
    if (unit >= a.units) return;
    const int64_t per = a.ldp / 4, t = unit / per;
    const int n = 4 * (int)(unit - t * per), left = a.cols - n;  // (ldp: the columns in whole vectors)
    const float *from = a.part + t * a.ldp + n;
    f32x4u s = *reinterpret_cast<const f32x4u *>(from);
    for (int i = 1; i < a.shares; ++i) {
        const f32x4u v = *reinterpret_cast<const f32x4u *>(from + i * (a.rows * a.ldp));
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += v[e];
    }
    float *out = a.out + t * a.ldo + n;
    if (a.beta != 0.0f) {
        const f32x4u old = rowk::load4(out, left);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = fmaf(a.beta, old[e], s[e]);
    }
    rowk::store4(out, left, s);
}

// ---------------------------------------------------------------------------
// dgate = dy up act'(gate), dup = dy act(gate), rows ldz apart, the columns up to
// ldz 0 (so that what reads them along N needs no end).  HBM: 2000 x 2048, 82 MB, 17 us.
// ---------------------------------------------------------------------------
struct SlopeArgs {
    int T, N;
    const float *gate, *up, *dy;
    int64_t ldgate, ldup, lddy, ldz;
    float *dgate, *dup;
    int chunks;  // of 256 columns a wave each
    int64_t units;
};

template <int ACT> __global__ void __launch_bounds__(256) gated_slopes(SlopeArgs a) {
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (unit >= a.units) return;
    const int64_t t = unit / a.chunks;
    const int n = (int)(unit - t * a.chunks) * 256 + 4 * (threadIdx.x & 63);
    if (n >= a.ldz) return;
    const int left = a.N - n;
    const f32x4u g = rowk::load4(a.gate + t * a.ldgate + n, left), u = rowk::load4(a.up + t * a.ldup + n, left);
    const f32x4u d = rowk::load4(a.dy + t * a.lddy + n, left);
    f32x4u dg, du;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        dg[e] = d[e] * u[e] * normk::act_slope<ACT>(g[e]);
        du[e] = d[e] * act32<ACT>(g[e]);
    }
    *reinterpret_cast<f32x4u *>(a.dgate + t * a.ldz + n) = dg;
    *reinterpret_cast<f32x4u *>(a.dup + t * a.ldz + n) = du;
}

// ---------------------------------------------------------------------------
// Any strides: 32 x 32 tiles, every element checked (FORWARD and BACK_W).
// ---------------------------------------------------------------------------
template <int KIND> __global__ void __launch_bounds__(256) gated_simple(TileArgs a) {
    constexpr int T = 32;
    __shared__ float As[T][T + 1], Bs[2][T][T + 1];
    const int nbn = (a.N + T - 1) / T;
    const int cols = KIND == BACK_W ? 2 * nbn : nbn;
    const int tn = (int)(blockIdx.x % cols), which = KIND == BACK_W && tn >= nbn ? 1 : 0;
    const int64_t m0 = (int64_t)(blockIdx.x / cols) * T, n0 = (int64_t)(tn - which * nbn) * T;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    float acc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    for (int64_t k0 = 0; k0 < a.K; k0 += T) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 8 * i;
            // As[m][k], Bs[k][n]; lanes walk what is contiguous
            if (KIND == BACK_W)
                As[tx][r] = k0 + r < a.K && m0 + tx < a.M ? a.A[0][(k0 + r) * a.lda + m0 + tx] : 0.0f;
            else
                As[r][tx] = k0 + tx < a.K && m0 + r < a.M ? a.A[0][(m0 + r) * a.lda + k0 + tx] : 0.0f;
#pragma unroll
            for (int s = 0; s < (KIND == FORWARD ? 2 : 1); ++s) {
                const int src = KIND == FORWARD ? s : which;
                Bs[s][r][tx] = k0 + r < a.K && n0 + tx < a.N ? a.B[src][(k0 + r) * a.ldb[src] + n0 + tx] : 0.0f;
            }
        }
        __syncthreads();
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[0][i] = fmaf(As[ty + 8 * i][k], Bs[0][k][tx], acc[0][i]);
                if (KIND == FORWARD) acc[1][i] = fmaf(As[ty + 8 * i][k], Bs[1][k][tx], acc[1][i]);
            }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty + 8 * i, n = n0 + tx;
        if (m >= a.M || n >= a.N) continue;
        float *c = a.C[which] + m * a.ldc[which] + n;
        if (KIND == FORWARD) {
            *c = gated(a.act, acc[0][i], acc[1][i]);
            if (a.gate != nullptr) {
                a.gate[m * a.ldgate + n] = acc[0][i];
                a.up[m * a.ldup + n] = acc[1][i];
            }
        } else {
            *c = a.beta != 0.0f ? fmaf(a.beta, *c, acc[0][i]) : acc[0][i];
        }
    }
}

}  // namespace gatedk
