// i8_kernels.hpp -- the product of 8-bit rows with 8-bit channels, scaled by row and
// channel:  C[m][n] = alpha sa[m] sb[n] sum_k A[m][k] B[n][k] + beta C[m][n].
//
// Both operands run along K, so a lane's 16 bytes of a row are what the matrix
// instructions take, of A and of B alike; the order of k inside an instruction is
// the same for both and does not matter.  The sum is exact: 32-bit integers hold
// 131071 products of -128 by -128.  The rest is computed in 64 bits and rounded
// once.
//
//   * i8_tile: LDS tiles filled by loads that write LDS directly.
//   * i8_thin: few rows; operands from memory straight to the matrix cores.
//   * i8_any: rows of any alignment and any strides.
#pragma once

#include "lanes.hpp"

namespace i8k {

using rowk::meet;
using rowk::rsrc_t;
using rowk::wait_loads;
using rowk::whole_rsrc;

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx16 __attribute__((ext_vector_type(16)));

struct Args {
    int M, N, K;  // K == 0 also when alpha == 0 (A, B and the scales not read)
    float alpha, beta;
    const signed char *A, *B;
    const float *sa, *sb;  // NULL: all 1
    float *C;
    int64_t lda, ldb, ldc;
    int xcd_shift;
    bool stream;  // C's stores go past the caches (K in tiles of 256, for smaller C: always)
};

__device__ __forceinline__ double scale_at(const float *s, int64_t i) { return s == nullptr ? 1.0 : (double)s[i]; }
// (without the product, nothing of the scales: they may be NaN)
__device__ __forceinline__ float scaled(const Args &a, int sum, double s, float old) {
    const double v = a.K == 0 ? 0.0 : (double)sum * s;
    return (float)(a.beta != 0.0f ? fma((double)a.beta, (double)old, v) : v);
}

__device__ __forceinline__ intx4 load16(rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(intx4, sgk::raw_load_v4f32(r, off, 0, 0));
}
// Descriptors are checked by whole 4-byte words: a last word that K fills in part
// counts as inside (it is aligned, so no page begins in it).  They end with a matrix's
// last row: of the others a load also brings what follows K, padding or the next row.
// Only A's is cleared; what B brings is multiplied by those zeros.
__device__ __forceinline__ int words(int bytes) { return (bytes + 3) & ~3; }
// the first `left` of 16 bytes
__device__ __forceinline__ intx4 first_bytes(intx4 v, int left) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = left - 4 * i;
        v[i] = n >= 4 ? v[i] : n <= 0 ? 0 : v[i] & (int)((1u << (8 * n)) - 1u);
    }
    return v;
}

// ---------------------------------------------------------------------------
// Tiles of BM x BN, K in tiles of BK bytes, a ring of STG LDS stages; the barrier that
// ends a K tile waits for the next one only.  A row of a stage is BK / 16 chunks of 16 bytes, permuted
// (AKLayout) so that a load instruction (whole rows) and a fragment read (one chunk
// of each of 16 consecutive rows) both touch every bank.  A wave sums a WM x WN tile
// with v_mfma_i32_32x32x32_i8; lane half lh takes chunks lh BK / 32 + s.  KG 2: two
// groups of waves take half of a K tile's steps each, for small tiles, whose loads then
// come from twice as many waves; the second group's sums go through LDS.
// 4096 x 4096 x 4096: 73 us, 1.88 POPS (8192: 495, 2.2): the matrix cores are busy for 52% at a clock that
// power sets, a CU's loads of a K tile (64 KiB) take 0.95 us beside 1.04 of products, and C's
// stores 14 at the end, when every workgroup stores at once.
// ---------------------------------------------------------------------------
template <int ROWS, int BK, int NT> struct Stage {
    static constexpr int WAVES = NT / 64, CPR = BK / 16;
    static constexpr int P = ROWS * BK / (NT * 16);
    static_assert(P * NT * 16 == ROWS * BK, "whole instructions");
    uint32_t off[P];
    int col[P];

    __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int chunk = (p * WAVES + wave) * 64 + lane, row = chunk / CPR;
            col[p] = 16 * sgk::AKLayout<BK / 4>::chunk_pos(row, chunk % CPR);
            off[p] = (uint32_t)(row * ld + col[p]);
        }
    }
    __device__ __forceinline__ void load(rsrc_t r, char *lds, int wave, int p, int left) const {
        typedef __attribute__((address_space(3))) void lds_t;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_t *)(lds + (p * WAVES + wave) * 1024), 16,
                                                 col[p] < left ? off[p] : rowk::kOut, 0, 0, 0);
    }
    // the chunk that holds K's last byte also brought what follows it in the row
    __device__ __forceinline__ void clear(char *lds, int wave, int lane, int left) const {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int n = left - col[p];
            if (n > 0 && n < 16) {
                intx4 *q = reinterpret_cast<intx4 *>(lds + (p * WAVES + wave) * 1024 + 16 * lane);
                *q = first_bytes(*q, n);
            }
        }
    }
};

template <int BM, int BN, int BK, int WM, int WN, int KG, int STG, int AHEAD, int WPE>
__global__ void __launch_bounds__(KG * (BM / WM) * (BN / WN) * 64) __attribute__((amdgpu_waves_per_eu(WPE)))
i8_tile(Args a) {
    constexpr int MI = WM / 32, NI = WN / 32, WAVES_N = BN / WN, WPG = (BM / WM) * WAVES_N, NT = KG * WPG * 64;
    constexpr int STAGE = (BM + BN) * BK, STEPS = BK / 32 / KG;
    static_assert(KG == 1 || KG == 2, "wave groups");
    static_assert(KG == 1 || STG * STAGE >= BM * BN * 4, "the second group's sums");
    __shared__ __attribute__((aligned(16))) char smem[STG * STAGE];
    __shared__ __attribute__((aligned(16))) float scale[BM + BN];  // alpha's product comes later
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 31, lh = lane >> 5;
    const int group = wave / WPG, wm = wave % WPG / WAVES_N * WM, wn = wave % WAVES_N * WN;
    const int nbm = (a.M + BM - 1) / BM, nbn = (a.N + BN - 1) / BN;
    int tm, tn;
    sgk::tile_of<2, 8>((int)blockIdx.x, nbm, nbn, a.xcd_shift, tm, tn);
    const int bm = tm * BM, bn = tn * BN;

    typedef Stage<BM, BK, NT> SA;
    typedef Stage<BN, BK, NT> SB;
    SA sa;
    SB sb;
    sa.init(a.lda, wave, lane);
    sb.init(a.ldb, wave, lane);
    const signed char *A = a.A + (int64_t)bm * a.lda, *B = a.B + (int64_t)bn * a.ldb;
    const int64_t a_bytes = (int64_t)(a.M - bm - 1) * a.lda + words(a.K);
    const int64_t b_bytes = (int64_t)(a.N - bn - 1) * a.ldb + words(a.K);
    const int KT = (a.K + BK - 1) / BK;

    intx16 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

    // byte offsets of the lane's rows and of its chunk of k-step s
    const int a_row = (wm + li) * BK, b_row = BM * BK + (wn + li) * BK;
    int at[STEPS];  // (wm, wn and 32 i are multiples of 16 rows: one permutation)
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        at[s] = 16 * sgk::AKLayout<BK / 4>::chunk_pos(li, lh * (BK / 32) + group * STEPS + s);

    constexpr int DP = SA::P + SB::P;
    auto fetch = [&](char *st, int k0) {  // (past K nothing is read)
        const int left = a.K - k0;
        const rsrc_t ra = whole_rsrc(A + k0, left > 0 ? a_bytes - k0 : 0);
        const rsrc_t rb = whole_rsrc(B + k0, left > 0 ? b_bytes - k0 : 0);
#pragma unroll
        for (int p = 0; p < SA::P; ++p) sa.load(ra, st, wave, p, left);
#pragma unroll
        for (int p = 0; p < SB::P; ++p) sb.load(rb, st + BM * BK, wave, p, left);
    };
    auto landed = [&](char *st, int k0) {
        const int left = a.K - k0;
        if ((a.K & 15) != 0 && left > 0 && left < BK) {
            sa.clear(st, wave, lane, left);
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt 0
        }
        meet();
    };
    // acc[i][j] register r on lane (li, lh): row 32 i + 8 (r / 4) + 4 lh + r % 4, column
    // 32 j + li.  C through a descriptor from the tile's first element to the last one:
    // rows beyond it are cut off there, columns get an offset outside.
    const rsrc_t rc = whole_rsrc(a.C + (int64_t)bm * a.ldc + bn, ((int64_t)(a.M - bm - 1) * a.ldc + (a.N - bn)) * 4);
    const uint32_t ldc4 = (uint32_t)a.ldc * 4u;
    uint32_t col[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) {
        const int n = wn + 32 * j + li;
        col[j] = bn + n < a.N ? 4u * (uint32_t)n : rowk::kOut;
    }
    auto c_at = [&](int row, int j) { return col[j] == rowk::kOut ? rowk::kOut : (uint32_t)row * ldc4 + col[j]; };
    // With one block a wave C's old values are asked for ahead of everything else (515 x 1024 x
    // 2816, beta 1: 16.2 us with these loads at the end, 12.8 so).
    constexpr bool EARLY = MI * NI == 1;
    float early[EARLY ? 16 : 1];
    if (EARLY && a.beta != 0.0f && (KG == 1 || group == 0)) {
#pragma unroll
        for (int r = 0; r < 16; ++r) early[EARLY ? r : 0] = sgk::raw_load_f32(rc, c_at(wm + 8 * (r >> 2) + 4 * lh + (r & 3), 0), 0, 0);
    }

    constexpr int SETS = AHEAD + 1;  // of fragments: one multiplied, AHEAD being read
    static_assert(STEPS % SETS == 0, "a tile begins with the first set");
    intx4 av[SETS][MI], bv[SETS][NI];
    auto read = [&](const char *__restrict__ st, int s) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
            bv[s % SETS][j] = *reinterpret_cast<const intx4 *>(st + b_row + j * 32 * BK + at[s]);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            av[s % SETS][i] = *reinterpret_cast<const intx4 *>(st + a_row + i * 32 * BK + at[s]);
    };
    auto multiply = [&](int s) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(av[s % SETS][i], bv[s % SETS][j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (KT > 0) {
        static_assert(BM + BN <= NT, "a scale per thread");
        float mine = 1.0f;  // (asked for ahead of the tiles, so that its wait is not theirs)
        if (tid < BM + BN) {
            const float *from = tid < BM ? a.sa : a.sb;
            const int row = tid < BM ? bm + tid : bn + tid - BM, end = tid < BM ? a.M : a.N;
            if (from != nullptr && row < end) mine = from[row];
        }
        // Fragments are read AHEAD k-steps before their MFMAs, across the tiles' borders:
        // the last AHEAD steps of a tile are multiplied behind the barrier that ends its
        // reads, while the stage that it was read from is filled with tile t + STG.
#pragma unroll
        for (int s = 0; s < STG; ++s) fetch(smem + s * STAGE, s * BK);
        if (tid < BM + BN) scale[tid] = mine;
        wait_loads<(STG - 1) * DP>();
        landed(smem, 0);
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) read(smem, s);
        int cur = 0;  // stage of tile t
        for (int t = 0; t < KT; ++t) {
            char *st = smem + cur * STAGE;
            cur = cur + 1 == STG ? 0 : cur + 1;
            char *next = smem + cur * STAGE;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (s + AHEAD == STEPS) {
                    wait_loads<(STG - 2) * DP>();
                    landed(next, (t + 1) * BK);
                }
                if (s + AHEAD < STEPS) read(st, s + AHEAD);
                else read(next, s + AHEAD - STEPS);
                if (s + AHEAD == STEPS) fetch(st, (t + STG) * BK);
                multiply(s);
            }
        }
        wait_loads<0>();
        if constexpr (KG == 2) {
            meet();  // (every wave is past its last reads, every load has landed)
            intx4 *part = reinterpret_cast<intx4 *>(smem) + wave % WPG * (MI * NI * 4 * 64) + lane;
#pragma unroll
            for (int v = 0; v < MI * NI * 4; ++v) {
                intx16 &of = acc[v / 4 / NI][v / 4 % NI];
                if (group == 1) part[64 * v] = intx4{of[v % 4 * 4], of[v % 4 * 4 + 1], of[v % 4 * 4 + 2], of[v % 4 * 4 + 3]};
            }
            __syncthreads();
            if (group == 1) return;
#pragma unroll
            for (int v = 0; v < MI * NI * 4; ++v) {
                const intx4 u = part[64 * v];
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[v / 4 / NI][v / 4 % NI][v % 4 * 4 + r] += u[r];
            }
        }
    }
    if (KG == 2 && group == 1) return;

    double sb_of[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) sb_of[j] = KT > 0 ? (double)a.alpha * (double)scale[BM + wn + 32 * j + li] : 0.0;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = wm + 32 * i + 8 * q + 4 * lh;
            const float4 s = KT > 0 ? *reinterpret_cast<const float4 *>(&scale[row]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float old[4][NI];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    old[r][j] = a.beta == 0.0f ? 0.0f : EARLY ? early[EARLY ? 4 * q + r : 0] : sgk::raw_load_f32(rc, c_at(row + r, j), 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const double sr = r == 0 ? s.x : r == 1 ? s.y : r == 2 ? s.z : s.w;
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const float v = scaled(a, acc[i][j][4 * q + r], sr * sb_of[j], old[r][j]);
                    if (BK == 256 || a.stream) sgk::raw_store_f32(v, rc, c_at(row + r, j), 0, sgk::kCPolStream);
                    else sgk::raw_store_f32(v, rc, c_at(row + r, j), 0, 0);
                }
            }
        }
}

// ---------------------------------------------------------------------------
// Few rows: reading B once is the work, so 16 MB rows and 16 NB channels a
// workgroup, its WK waves each a share of K, both operands straight from memory to
// v_mfma_i32_16x16x64_i8, the partial sums added through LDS.  A step is 128 bytes
// of K: a lane takes 32 of them of its row, so that whole lines are read.  1 x 4096 x 4096, 17
// MB, 5.5 us, of which a launch alone is 2.2.
// ---------------------------------------------------------------------------
template <int MB, int NB, int WK, int WPE>
__global__ void __launch_bounds__(WK * 64) __attribute__((amdgpu_waves_per_eu(WPE))) i8_thin(Args a) {
    constexpr int BM = 16 * MB, BN = 16 * NB;
    __shared__ __attribute__((aligned(16))) int part[WK][BM * BN];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lk = lane >> 4;
    const int nbm = (a.M + BM - 1) / BM, nbn = (a.N + BN - 1) / BN;
    int tm, tn;
    sgk::tile_of<2, 8>((int)blockIdx.x, nbm, nbn, a.xcd_shift, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const signed char *A = a.A + (int64_t)m0 * a.lda, *B = a.B + (int64_t)n0 * a.ldb;
    const int64_t a_bytes = (int64_t)(a.M - m0 - 1) * a.lda + words(a.K);
    const int64_t b_bytes = (int64_t)(a.N - n0 - 1) * a.ldb + words(a.K);
    uint32_t ao[MB], bo[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) ao[i] = (uint32_t)((16 * i + li) * a.lda + 32 * lk);
#pragma unroll
    for (int j = 0; j < NB; ++j) bo[j] = (uint32_t)((16 * j + li) * a.ldb + 32 * lk);

    intx4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = intx4{0, 0, 0, 0};

    const int steps = (a.K + 127) / 128;
    const int u0 = (int)((int64_t)steps * w / WK), u1 = (int)((int64_t)steps * (w + 1) / WK);
    constexpr int STEP = 8 * (MB + NB), D = 96 / STEP < 4 ? (96 / STEP < 2 ? 2 : 96 / STEP) : 4;
    intx4 av[D][2][MB], bv[D][2][NB];
    auto fetch = [&](int d, int u) {  // (past the wave's last step the descriptors are empty)
        const int64_t k0 = 128 * (int64_t)u;
        const rsrc_t ra = whole_rsrc(A + k0, u < u1 ? a_bytes - k0 : 0), rb = whole_rsrc(B + k0, u < u1 ? b_bytes - k0 : 0);
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) bv[d][h][j] = load16(rb, bo[j] + 16 * h);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) av[d][h][i] = load16(ra, ao[i] + 16 * h);
    };
    auto multiply = [&](int d) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[d][h][i], bv[d][h][j], acc[i][j], 0, 0, 0);
    };
    const int whole = (int64_t)u1 * 128 > a.K ? u1 - 1 : u1;
    constexpr int OUT = (BM * BN + WK * 64 - 1) / (WK * 64);  // results per thread
    float sa[OUT], sb[OUT];  // (asked for ahead of the operands)
#pragma unroll
    for (int o = 0; o < OUT; ++o) {
        const int f = tid + o * WK * 64, m = m0 + f / BN, n = n0 + f % BN;
        const bool there = a.K > 0 && f < BM * BN && m < a.M && n < a.N;
        sa[o] = there && a.sa != nullptr ? a.sa[m] : 1.0f;
        sb[o] = there && a.sb != nullptr ? a.sb[n] : 1.0f;
    }
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, u0 + d);
    for (int u = u0; u < u1; u += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (u + d == whole) {  // K's end: A's row goes on into what follows it
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < MB; ++i)
                        av[d][h][i] = first_bytes(av[d][h][i], a.K - 128 * whole - 32 * lk - 16 * h);
            }
            if (u + d < u1) multiply(d);
            if (u + D < u1) fetch(d, u + d + D);
        }
    }
    // acc[i][j] register r on lane (li, lk): row 16 i + 4 lk + r, column 16 j + li
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) part[w][(16 * i + 4 * lk + r) * BN + 16 * j + li] = acc[i][j][r];
    __syncthreads();
#pragma unroll
    for (int o = 0; o < OUT; ++o) {
        const int f = tid + o * WK * 64, m = m0 + f / BN, n = n0 + f % BN;
        if (f >= BM * BN || m >= a.M || n >= a.N) continue;
        int sum = part[0][f];
#pragma unroll
        for (int i = 1; i < WK; ++i) sum += part[i][f];
        float *c = a.C + (int64_t)m * a.ldc + n;
        *c = scaled(a, sum, (double)a.alpha * (double)sa[o] * (double)sb[o], a.beta != 0.0f ? *c : 0.0f);
    }
}

// ---------------------------------------------------------------------------
// Rows of any alignment and any leading dimensions: tiles of 64 x 64, 128 bytes of K at a
// time through registers (loads of 16 bytes at any address; the bytes of a row's end one by
// one), otherwise as i8_tile.  Measured, rows K bytes apart against 16-byte aligned ones: 1000 x
// 1000 x 999 13.7 us and 7.6, 4096 x 4096 x 4095 247 and 73, 1 x 4096 x 4095 21 and 4.8.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) i8_any(Args a) {
    constexpr int BM = 64, BK = 128, STAGE = 2 * BM * BK;
    typedef sgk::AKLayout<BK / 4> Layout;
    __shared__ __attribute__((aligned(16))) char smem[2 * STAGE];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 31, lh = lane >> 5, wm = wave / 2 * 32, wn = wave % 2 * 32;
    const int nbn = (a.N + BM - 1) / BM;
    const int64_t m0 = (int64_t)(blockIdx.x / nbn) * BM, n0 = (int64_t)(blockIdx.x % nbn) * BM;
    const int KT = (a.K + BK - 1) / BK;
    // chunk p of this thread: 16 bytes of a row of A (p < 2) or of B
    intx4 held[4];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int chunk = p % 2 * 256 + tid, left = a.K - k0 - 16 * (chunk % 8);
            const int64_t row = (p < 2 ? m0 : n0) + chunk / 8;
            const signed char *from = p < 2 ? a.A + row * a.lda : a.B + row * a.ldb;
            held[p] = intx4{0, 0, 0, 0};
            if (row >= (p < 2 ? a.M : a.N) || left <= 0) continue;
            from += k0 + 16 * (chunk % 8);
            if (left >= 16) {
                __builtin_memcpy(&held[p], from, 16);
            } else {
#pragma unroll
                for (int i = 0; i < 15; ++i)
                    if (i < left) held[p][i / 4] |= (from[i] & 0xff) << (8 * (i % 4));
            }
        }
    };
    auto put = [&](char *st) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int chunk = p % 2 * 256 + tid, row = chunk / 8;
            *reinterpret_cast<intx4 *>(st + (p < 2 ? 0 : BM * BK) + row * BK + 16 * Layout::chunk_pos(row, chunk % 8)) = held[p];
        }
    };
    intx16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0;
    if (KT > 0) {
        fetch(0);
        put(smem);
        __syncthreads();
    }
    for (int t = 0; t < KT; ++t) {
        const char *st = smem + (t & 1) * STAGE;
        if (t + 1 < KT) fetch((t + 1) * BK);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int at = 16 * Layout::chunk_pos(li, 4 * lh + s);
            const intx4 av = *reinterpret_cast<const intx4 *>(st + (wm + li) * BK + at);
            const intx4 bv = *reinterpret_cast<const intx4 *>(st + BM * BK + (wn + li) * BK + at);
            acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(av, bv, acc, 0, 0, 0);
        }
        if (t + 1 < KT) put(smem + ((t + 1) & 1) * STAGE);
        __syncthreads();
    }
    const int64_t n = n0 + wn + li;
    if (n >= a.N) return;
    const double sb = a.K > 0 ? (double)a.alpha * scale_at(a.sb, n) : 0.0;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int64_t m = m0 + wm + 8 * (r >> 2) + 4 * lh + (r & 3);
        if (m >= a.M) continue;
        float *c = a.C + m * a.ldc + n;
        *c = scaled(a, acc[r], a.K > 0 ? sb * scale_at(a.sa, m) : 0.0, a.beta != 0.0f ? *c : 0.0f);
    }
}

}  // namespace i8k
