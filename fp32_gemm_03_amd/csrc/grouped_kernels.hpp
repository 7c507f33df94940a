// grouped_kernels.hpp -- products over groups of rows on the matrix cores.
//
//   * grouped_mfma: block tiles of many rows of one group, A's rows gathered
//     and C's scattered; B as K x N or N x K.
//   * grouped_tn_mfma: a group's sum of outer products, the sum running over
//     its slots.
//   * thin: groups of few rows, where reading B is all there is.
//
// All load through buffer descriptors whose byte offsets are 32-bit: an access
// past a descriptor's end reads 0.0, with no branch, and 16-byte loads need
// only 4-byte alignment.
#pragma once

#undef SGEMM_PHASES
#include "sgemm_kernels.hpp"

#include "rows_kernels.hpp"

namespace rowk {

using sgk::f32x2;
using sgk::f32x4;
using sgk::floatx16;
using sgk::rsrc_t;
typedef float floatx4 __attribute__((ext_vector_type(4)));

// A descriptor over [base, base + bytes), at most kOut bytes; an access at
// kOut is outside every one (and its 16 bytes do not wrap).
constexpr uint32_t kOut = 0xfffffff0u;
__device__ __forceinline__ rsrc_t whole_rsrc(const void *base, int64_t bytes) {
    const uint32_t n = bytes <= 0 ? 0u : (bytes >= (int64_t)kOut ? kOut : (uint32_t)bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)n, sgk::kRsrcWord3);
}

// ---------------------------------------------------------------------------
// The order of a launch's tiles.  Workgroup ids go to the XCDs in turn; each
// XCD is given one run of the sequence, and the sequence walks a group's tiles
// in bands of up to eight row tiles, a band column by column: the workgroups
// an XCD runs at once share a few rows of A and a few columns of one B.
// A wave looks at 64 groups at a time (each lane one), so every wave of a
// workgroup finds its tile by itself.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int tiles_of(const GroupedArgs &a, int g, int bm, int &lo, int &hi) {
    lo = hi = 0;
    if (g < (a.offsets != nullptr ? a.G : 1)) group_range(a, g, lo, hi);
    return hi > lo ? (hi - lo + bm - 1) / bm : 0;
}
__device__ __forceinline__ int wave_upto(int n) {  // inclusive sum over the lanes
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(n, d);
        if (lane >= d) n += o;
    }
    return n;
}

struct Tile {
    int g, p0, p1, bn;  // group, first row, the group's end, first column
};

__device__ __forceinline__ bool place_tile(const GroupedArgs &a, int bm, int bn, Tile &t) {
    const int lane = threadIdx.x & 63;
    const int nbn = (a.N + bn - 1) / bn;
    const int groups = a.offsets != nullptr ? a.G : 1;
    int lo, hi;
    long long total = 0;
    for (int base = 0; base < groups; base += 64)
        total += __builtin_amdgcn_readlane(wave_upto(tiles_of(a, base + lane, bm, lo, hi)), 63);
    total *= nbn;
    // XCD x's run of the sequence
    const int X = 1 << a.xcd_shift, x = (int)blockIdx.x & (X - 1), i = (int)(blockIdx.x >> a.xcd_shift);
    const long long q = total >> a.xcd_shift;
    const int r = (int)(total & (X - 1));
    if (i >= q + (x < r ? 1 : 0)) return false;
    long long left = x * q + (x < r ? x : r) + i;
    for (int base = 0; base < groups; base += 64) {
        const int n = tiles_of(a, base + lane, bm, lo, hi);
        const int upto = wave_upto(n);
        const unsigned long long past = __ballot((long long)upto * nbn > left);
        if (past == 0) {
            left -= (long long)__builtin_amdgcn_readlane(upto, 63) * nbn;
            continue;
        }
        const int at = __ffsll((long long)past) - 1;
        const int tiles = __builtin_amdgcn_readlane(n, at);
        const int s = (int)(left - (long long)__builtin_amdgcn_readlane(upto - n, at) * nbn);
        constexpr int BAND = 8;
        const int band = s / (BAND * nbn);
        const int in_band = s - band * BAND * nbn;
        const int rows = tiles - band * BAND < BAND ? tiles - band * BAND : BAND;
        const int col = in_band / rows;
        t.g = base + at;
        t.p0 = __builtin_amdgcn_readlane(lo, at) + (band * BAND + in_band - col * rows) * bm;
        t.p1 = __builtin_amdgcn_readlane(hi, at);
        t.bn = col * bn;
        return true;
    }
    return false;
}

// ---------------------------------------------------------------------------
// A BM x BK or BN x BK tile whose rows run along K, loaded 16 bytes per lane
// straight into LDS in AKLayout's chunk order.  Row m of the tile begins at the
// byte offset row_at(m) of the descriptor.
// ---------------------------------------------------------------------------
template <int ROWS, int BK, int NT> struct KRows {
    static constexpr int WAVES = NT / 64, P = ROWS * BK / (NT * 4);
    static_assert(ROWS * BK % (NT * 4) == 0, "whole instructions");
    uint32_t off[P];
    int col[P];
    int wave, lane;

    template <class F> __device__ __forceinline__ void init(int tid, F row_at) {
        wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        lane = tid & 63;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int f = (p * WAVES + wave) * 256 + lane * 4;
            const int m = f / BK;
            col[p] = 4 * sgk::AKLayout<BK>::chunk_pos(m, f % BK / 4);
            off[p] = row_at(m) + 4u * (uint32_t)col[p];
        }
    }
    __device__ __forceinline__ void load(rsrc_t r, float *lds, int k0, int K, int p) const {
        sgk::load_to_lds<4>(r, lds + (p * WAVES + wave) * 256, k0 + col[p] < K ? off[p] + 4u * (uint32_t)k0 : kOut);
    }
    // The chunk that holds column K - 1 also brought what follows it in memory:
    // cleared once it has landed, before the barrier that publishes the tile.
    __device__ __forceinline__ void clear_tail(float *lds, int k0, int K) const {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int valid = K - (k0 + col[p]);
            if (valid > 0 && valid < 4) {
                float *q = lds + (p * WAVES + wave) * 256 + 4 * lane;
#pragma unroll
                for (int j = 1; j < 4; ++j)
                    if (j >= valid) q[j] = 0.0f;
            }
        }
    }
};

// A BK x COLS tile as it lies in memory (rows along N), 16 bytes per lane
// straight into LDS.
template <int COLS, int BK, int NT> struct NRows {
    static constexpr int WAVES = NT / 64, P = COLS * BK / (NT * 4);
    static_assert(COLS * BK % (NT * 4) == 0, "whole instructions");
    static __device__ __forceinline__ int row(int tid, int p) { return ((p * WAVES + (tid >> 6)) * 256 + (tid & 63) * 4) / COLS; }
    static __device__ __forceinline__ int column(int tid, int p) { return ((p * WAVES + (tid >> 6)) * 256 + (tid & 63) * 4) % COLS; }
    static __device__ __forceinline__ void load(rsrc_t r, float *lds, uint32_t off, int wave, int p) {
        sgk::load_to_lds<4>(r, lds + (p * WAVES + wave) * 256, off);
    }
};

// One K tile of MFMAs where both tiles run along K: lane (li, lh) takes chunk
// lh QN + q of its row of A and of its column of B, k-step j of lane half lh
// being k = lh BK / 2 + j as in mfma_tile_kc.
template <int BK, int MI, int NI, class Hook>
__device__ __forceinline__ void mfma_tile_nt(const float *a_row, const float *b_row, const int (&off)[BK / 8],
                                             floatx16 (&acc)[MI][NI], Hook hook) {
    constexpr int QN = BK / 8;
    float4 av[2][MI], bv[2][NI];
    auto read = [&](int q) {
#pragma unroll
        for (int j = 0; j < NI; ++j) bv[q & 1][j] = *reinterpret_cast<const float4 *>(b_row + j * 32 * BK + off[q]);
#pragma unroll
        for (int i = 0; i < MI; ++i) av[q & 1][i] = *reinterpret_cast<const float4 *>(a_row + i * 32 * BK + off[q]);
    };
    read(0);
#pragma unroll
    for (int q = 0; q < QN; ++q) {
        if (q + 1 < QN) read(q + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(sgk::vget(av[q & 1][i], e), sgk::vget(bv[q & 1][j], e),
                                                                     acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    hook(4 * q + e, i * NI + j);
                    __builtin_amdgcn_sched_barrier(0);
                }
    }
}

// ---------------------------------------------------------------------------
// C rows of one group.  The K loop is that of the whole-tile K-ordered block of
// sgemm(): both tiles go straight into one of two LDS stages, the next tile's
// loads are issued over the first quarter of this one's MFMAs, one barrier per
// K tile.  What differs: A's row offsets come from the gather (kept in
// registers, so a gathered row costs what a plain one does), the tile's group
// is found from the offsets on the device, and C's rows go through an index in
// LDS.  Rows past the group's end read the tile's first row; they only reach
// rows of C that are not stored.
// ---------------------------------------------------------------------------
template <int BM, int BN, int BK, int WM, int WN, int WPE, bool TRANS_B, int RO>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * 64)
__attribute__((amdgpu_waves_per_eu(WPE))) grouped_mfma(GroupedArgs a) {
    constexpr int MI = WM / 32, NI = WN / 32, WAVES_N = BN / WN, NT = (BM / WM) * WAVES_N * 64;
    constexpr int ASZ = BM * BK, STAGE = ASZ + BK * BN;
    __shared__ __attribute__((aligned(16))) float smem[2 * STAGE];
    __shared__ int c_row[BM];
    Tile t;
    if (!place_tile(a, BM, BN, t)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = (wave / WAVES_N) * WM, wn = (wave % WAVES_N) * WN;
    const int li = lane & 31, lh = lane >> 5;
    const int K = a.rank_k ? group_rank(a, t.g, a.K) : a.K;

    for (int m = tid; m < BM; m += NT) c_row[m] = t.p0 + m < t.p1 ? (int)row_of(a, t.p0 + m, a.c_scatter) : -1;

    const float *B = a.B + (int64_t)t.g * a.stride_b;
    const int64_t a_rows = a.a_div > 1 ? (a.R + a.a_div - 1) / a.a_div : a.R;
    const int64_t a_base = a.a_div == 0 ? t.p0 : 0;
    const rsrc_t ra = whole_rsrc(a.A + a_base * a.lda, ((a_rows - a_base - 1) * a.lda + a.K) * 4);
    typedef KRows<BM, BK, NT> TA;
    typedef KRows<BN, BK, NT> TBk;
    typedef NRows<BN, BK, NT> TBn;
    constexpr int PA = TA::P, PB = TRANS_B ? TBk::P : TBn::P;
    TA ta;
    ta.init(tid, [&](int m) {
        int64_t row = row_of(a, t.p0 + m < t.p1 ? t.p0 + m : t.p0, a.a_div);
        row = row < 0 ? 0 : row - a_base;
        return (uint32_t)row * (uint32_t)a.lda * 4u;
    });
    TBk tb;
    uint32_t boff[PB];
    rsrc_t rbt;
    if constexpr (TRANS_B) {
        rbt = whole_rsrc(B + (int64_t)t.bn * a.ldb, ((int64_t)(a.N - t.bn - 1) * a.ldb + a.K) * 4);
        tb.init(tid, [&](int n) { return (uint32_t)n * (uint32_t)a.ldb * 4u; });
    } else {
#pragma unroll
        for (int p = 0; p < PB; ++p)
            boff[p] = ((uint32_t)TBn::row(tid, p) * (uint32_t)a.ldb + (uint32_t)TBn::column(tid, p)) * 4u;
    }
    const int uwave = __builtin_amdgcn_readfirstlane(wave);
    // rows k0.. of B from the tile's first column: rows from K on read 0.0
    auto b_from = [&](int k0) {
        if constexpr (TRANS_B) return rbt;
        else return whole_rsrc(B + (int64_t)k0 * a.ldb + t.bn, ((int64_t)(K - k0 - 1) * a.ldb + (a.N - t.bn)) * 4);
    };
    auto load = [&](rsrc_t rb, float *st, int k0, int piece) {
        if (piece < PA) ta.load(ra, st, k0, K, piece);
        else if constexpr (TRANS_B) tb.load(rb, st + ASZ, k0, K, piece - PA);
        else TBn::load(rb, st + ASZ, boff[piece - PA], uwave, piece - PA);
    };
    auto clear = [&](float *st, int k0) {
        if ((K & 3) != 0 && k0 < K && k0 + BK > K) {
            ta.clear_tail(st, k0, K);
            if constexpr (TRANS_B) tb.clear_tail(st + ASZ, k0, K);
        }
    };

    constexpr int CH = MI * NI == 1 && !TRANS_B ? 2 : 1;
    floatx16 acc[MI][NI], acc_odd[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = acc_odd[i][j][r] = 0.0f;

    constexpr int QN = BK / 8;
    int off[QN];
#pragma unroll
    for (int q = 0; q < QN; ++q) off[q] = 4 * sgk::AKLayout<BK>::chunk_pos(li, lh * QN + q);
    // (row wm + 32 i + li is permuted as row li: 32 rows are whole periods)
    const int a_row = (wm + li) * BK;
    const int b_at = TRANS_B ? ASZ + (wn + li) * BK : ASZ + lh * (BK / 2) * BN + wn + NI * li;
    constexpr int STEPS = BK / 2, LSTEPS = STEPS / 4 > 0 ? STEPS / 4 : 1, NU = MI * NI;
    constexpr int DP = PA + PB, DLPER = (DP + LSTEPS - 1) / LSTEPS;
    const int KT = (K + BK - 1) / BK;
    if (KT > 0) {
        const rsrc_t rb = b_from(0);
#pragma unroll
        for (int p = 0; p < DP; ++p) load(rb, smem, 0, p);
    }
    __builtin_amdgcn_s_waitcnt(0);
    if (KT > 0) clear(smem, 0);
    __syncthreads();
    sgk::KcPending<MI, NI, 1> pd;
    auto body = [&](const float *__restrict__ st, float *__restrict__ nx, int kn, bool pd_in) {
        const rsrc_t rb = b_from(kn);
        auto hook = [&](int j, int u) {
            if (j < LSTEPS) {
#pragma unroll
                for (int q = 0; q < DLPER; ++q) {
                    const int piece = j * DLPER + q;
                    if ((q * NU) / DLPER != u || piece >= DP) continue;
                    load(rb, nx, kn, piece);
                }
            }
        };
        if constexpr (TRANS_B)
            mfma_tile_nt<BK, MI, NI>(st + a_row, st + b_at, off, acc, hook);
        else
            sgk::mfma_tile_kc<BK, MI, NI, BN, 1, CH, RO, 0, BK, 1>(st + a_row, off, st + b_at, acc, acc_odd, hook, pd,
                                                                   pd_in);
    };
    for (int s = 0; s < KT; ++s) {
        // past the last tile the loads read zeros into a stage nobody reads
        body(smem + (s & 1) * STAGE, smem + ((s + 1) & 1) * STAGE, (s + 1) * BK, s > 0);
        __builtin_amdgcn_s_waitcnt(0);
        clear(smem + ((s + 1) & 1) * STAGE, (s + 1) * BK);
        __syncthreads();
    }
    if constexpr (!TRANS_B) {
        if (KT > 0) sgk::mfma_pending_kc<MI, NI, CH, 1, STEPS>(pd, acc, acc_odd);
        if (CH == 2) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[i][j] += acc_odd[i][j];
        }
    }

    // register r of block (i, j): tile row wm + 32 i + 8 (r / 4) + 4 lh + r % 4,
    // column wn + NI li + j (B as K x N) or wn + 32 j + li
    const float al = group_alpha(a, t.g);
    const int n0 = t.bn + wn + (TRANS_B ? li : NI * li);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int4 rows = *reinterpret_cast<const int4 *>(&c_row[wm + 32 * i + 8 * q + 4 * lh]);
            const int row[4] = {rows.x, rows.y, rows.z, rows.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (row[e] < 0) continue;
                float *c = a.C + (int64_t)row[e] * a.ldc + n0;
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const int at = TRANS_B ? 32 * j : j;
                    if (n0 + at >= a.N) continue;
                    const float v = al * acc[i][j][4 * q + e];
                    c[at] = a.beta != 0.0f ? fmaf(a.beta, c[at], v) : v;
                }
            }
        }
}

// ---------------------------------------------------------------------------
// A group's sum of outer products: C_g (M x N) = sum over its slots of A's row
// (as a column) times B's row.  Both tiles lie in LDS as they do in memory,
// BK slots each, so neither is transposed.  The slots' row numbers are read
// one K tile ahead of the loads that need them.
// ---------------------------------------------------------------------------
template <int BM, int BN, int BK, int WM, int WN, int WPE>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * 64)
__attribute__((amdgpu_waves_per_eu(WPE))) grouped_tn_mfma(GroupedArgs a) {
    constexpr int MI = WM / 32, NI = WN / 32, WAVES_N = BN / WN, NT = (BM / WM) * WAVES_N * 64;
    constexpr int ASZ = BM * BK, STAGE = ASZ + BK * BN;
    typedef NRows<BM, BK, NT> TA;
    typedef NRows<BN, BK, NT> TB;
    constexpr int PA = TA::P, PB = TB::P, DP = PA + PB;
    __shared__ __attribute__((aligned(16))) float smem[2 * STAGE];
    const int nbm = (a.M + BM - 1) / BM, nbn = (a.N + BN - 1) / BN;
    // an XCD's workgroups take consecutive tiles: of one group, sharing rows
    const int total = a.G * nbm * nbn;
    const int X = 1 << a.xcd_shift, x = (int)blockIdx.x & (X - 1);
    const int q0 = total >> a.xcd_shift, r0 = total & (X - 1);
    const int s = x * q0 + (x < r0 ? x : r0) + (int)(blockIdx.x >> a.xcd_shift);
    const int g = s / (nbm * nbn), rest = s - g * nbm * nbn;
    const int bm = rest % nbm * BM, bn = rest / nbm * BN;
    int p0, p1;
    group_range(a, g, p0, p1);

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int uwave = __builtin_amdgcn_readfirstlane(wave);
    const int wm = (wave / WAVES_N) * WM, wn = (wave % WAVES_N) * WN;
    const int li = lane & 31, lh = lane >> 5;
    const int64_t a_rows = a.a_div > 1 ? (a.R + a.a_div - 1) / a.a_div : a.R;
    const int64_t b_rows = a.b_div > 1 ? (a.R + a.b_div - 1) / a.b_div : a.R;
    // rows in order are taken from the group's first: their offsets stay small
    const int64_t a0 = a.a_div == 0 ? p0 : 0, b0 = a.b_div == 0 ? p0 : 0;
    const rsrc_t ra = whole_rsrc(a.A + a0 * a.lda + bm, ((a_rows - a0 - 1) * a.lda + (a.M - bm)) * 4);
    const rsrc_t rb = whole_rsrc(a.B + b0 * a.ldb + bn, ((b_rows - b0 - 1) * a.ldb + (a.N - bn)) * 4);
    const bool listed = a.a_div != 0 || a.b_div != 0;

    // the slot at this lane's row of piece p of the K tile that begins at place
    // `at` (-1: none, both its rows then read 0.0)
    auto slot = [&](int at, int piece) {
        const int p = at + (piece < PA ? TA::row(tid, piece) : TB::row(tid, piece - PA));
        if (p >= p1) return -1;
        if (!listed) return p;
        const int v = a.rows[p];
        return (unsigned)v < (unsigned)a.R ? v : -1;
    };
    auto offset = [&](int v, int at, int piece) -> uint32_t {
        const bool is_a = piece < PA;
        const int div = is_a ? a.a_div : a.b_div;
        const int p = at + (is_a ? TA::row(tid, piece) : TB::row(tid, piece - PA));
        const uint32_t row = div == 0 ? (uint32_t)(p - p0) : div == 1 ? (uint32_t)v : (uint32_t)v / (uint32_t)div;
        const uint32_t ld = (uint32_t)(is_a ? a.lda : a.ldb);
        const uint32_t col = (uint32_t)(is_a ? TA::column(tid, piece) : TB::column(tid, piece - PA));
        return v < 0 ? kOut : (row * ld + col) * 4u;
    };
    auto load = [&](float *st, uint32_t off, int piece) {
        if (piece < PA) TA::load(ra, st, off, uwave, piece);
        else TB::load(rb, st + ASZ, off, uwave, piece - PA);
    };

    constexpr int CH = MI * NI == 1 ? 2 : 1;
    floatx16 acc[MI][NI], acc_odd[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = acc_odd[i][j][r] = 0.0f;
    const int a_col = wm + MI * li;
    const int b_at = ASZ + lh * BN + wn + NI * li;
    constexpr int STEPS = BK / 2, LSTEPS = STEPS / 4 > 0 ? STEPS / 4 : 1, NU = MI * NI;
    constexpr int DLPER = (DP + LSTEPS - 1) / LSTEPS;
    const int KT = p1 > p0 ? (p1 - p0 + BK - 1) / BK : 0;

    int next[DP];  // the slots of the next K tile
    if (KT > 0) {
#pragma unroll
        for (int p = 0; p < DP; ++p) next[p] = slot(p0, p);
#pragma unroll
        for (int p = 0; p < DP; ++p) load(smem, offset(next[p], p0, p), p);
#pragma unroll
        for (int p = 0; p < DP; ++p) next[p] = slot(p0 + BK, p);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    auto body = [&](const float *__restrict__ st, float *__restrict__ nx, int at) {
        uint32_t off[DP];
#pragma unroll
        for (int p = 0; p < DP; ++p) {
            off[p] = offset(next[p], at, p);
            next[p] = slot(at + BK, p);
        }
        auto hook = [&](int j, int u) {
            if (j < LSTEPS) {
#pragma unroll
                for (int q = 0; q < DLPER; ++q) {
                    const int piece = j * DLPER + q;
                    if ((q * NU) / DLPER != u || piece >= DP) continue;
                    load(nx, off[piece], piece);
                }
            }
        };
        sgk::mfma_tile<BK, MI, NI, BM, BN, 1, false, CH>(st, a_col, lh, st + b_at, acc, acc_odd, hook);
    };
    for (int k = 0; k < KT; ++k) {
        body(smem + (k & 1) * STAGE, smem + ((k + 1) & 1) * STAGE, p0 + (k + 1) * BK);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
    }
    if (CH == 2) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] += acc_odd[i][j];
    }

    // register r of block (i, j): tile row wm + MI (8 (r / 4) + 4 lh + r % 4) + i,
    // column wn + NI li + j
    const float al = group_alpha(a, g);
    const int mr = a.rank_m ? group_rank(a, g, a.M) : a.M, nr = a.rank_n ? group_rank(a, g, a.N) : a.N;
    float *C = a.C + (int64_t)g * a.stride_c;
    const int n0 = bn + wn + NI * li;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int m = bm + wm + MI * (8 * (r >> 2) + 4 * lh + (r & 3)) + i;
            if (m >= a.M) continue;
            float *c = C + (int64_t)m * a.ldc + n0;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                if (n0 + j >= a.N) continue;
                const float v = m < mr && n0 + j < nr ? al * acc[i][j][r] : 0.0f;
                c[j] = a.beta != 0.0f ? fmaf(a.beta, c[j], v) : v;
            }
        }
}

// ---------------------------------------------------------------------------
// Few rows per group: reading B once is all there is, so B goes from memory
// straight to the matrix cores and nothing but the waves' partial sums passes
// LDS.  v_mfma_f32_16x16x4_f32 takes B's element (k l/16, column l%16) from
// lane l: a lane loads VW consecutive columns (B as K x N) or four consecutive
// k (N x K) of 16 k's at a time, and the four k's of a lane are one float4 of
// A's row l%16.  At 16 rows that is 8 MFMAs per KiB of B, 32 cycles each on one
// of four matrix cores: 20 TB/s on the chip, beyond what memory gives, so up to
// 32 rows cost the same.  WK waves split K and are summed through LDS in order.
// D steps of 16 k are in flight per wave.
// ---------------------------------------------------------------------------
template <int MB, int VW, int WK, int D, bool TRANS_B>
__global__ void __launch_bounds__(WK * 64) thin(GroupedArgs a) {
    constexpr int ROWS = 16 * MB, COLS = 16 * VW;
    __shared__ float part[WK > 1 ? WK : 1][WK > 1 ? ROWS * COLS : 1];
    const int ncol = (a.N + COLS - 1) / COLS;
    const int n0 = (int)(blockIdx.x % ncol) * COLS;
    int g, p0, p1;
    if (!find_tile(a, ROWS, (int)(blockIdx.x / ncol), g, p0, p1)) return;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lk = lane >> 4;
    const int K = a.rank_k ? group_rank(a, g, a.K) : a.K;
    const int steps = (K + 15) / 16;
    const int s0 = (int)((int64_t)steps * w / WK), s1 = (int)((int64_t)steps * (w + 1) / WK);

    const int64_t a_rows = a.a_div > 1 ? (a.R + a.a_div - 1) / a.a_div : a.R;
    const int64_t a_base = a.a_div == 0 ? p0 : 0;
    const rsrc_t ra = whole_rsrc(a.A + a_base * a.lda, ((a_rows - a_base - 1) * a.lda + a.K) * 4);
    uint32_t aoff[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int p = p0 + 16 * i + li;
        int64_t row = row_of(a, p < p1 ? p : p0, a.a_div);
        row = row < 0 ? 0 : row - a_base;
        aoff[i] = ((uint32_t)row * (uint32_t)a.lda + 4u * (uint32_t)lk) * 4u;
    }
    const float *B = a.B + (int64_t)g * a.stride_b;
    // K x N: rows from the group's first to K; N x K: from row n0 to the last
    const rsrc_t rb = TRANS_B ? whole_rsrc(B + (int64_t)n0 * a.ldb, ((int64_t)(a.N - n0 - 1) * a.ldb + a.K) * 4)
                              : whole_rsrc(B + n0, ((int64_t)(K - 1) * a.ldb + (a.N - n0)) * 4);
    const uint32_t b0 = TRANS_B ? ((uint32_t)li * (uint32_t)a.ldb + 4u * (uint32_t)lk) * 4u
                                : ((uint32_t)(4 * lk) * (uint32_t)a.ldb + (uint32_t)(VW * li)) * 4u;
    const uint32_t ldb4 = (uint32_t)a.ldb * 4u;

    floatx4 acc[MB][VW];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < VW; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    f32x4 av[D][MB];
    float bv[D][4][VW];  // [k of the lane][column]
    auto fetch = [&](int d, int s) {
        const bool in = s < s1;
#pragma unroll
        for (int i = 0; i < MB; ++i)
            av[d][i] = sgk::raw_load_v4f32(ra, in ? aoff[i] + 64u * (uint32_t)s : kOut, 0, 0);
        if constexpr (TRANS_B) {
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                const f32x4 v = sgk::raw_load_v4f32(rb, in ? b0 + 64u * (uint32_t)s + 16u * (uint32_t)j * ldb4 : kOut, 0, 0);
                bv[d][0][j] = v.x;
                bv[d][1][j] = v.y;
                bv[d][2][j] = v.z;
                bv[d][3][j] = v.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t off = in ? b0 + (16u * (uint32_t)s + (uint32_t)e) * ldb4 : kOut;
                if constexpr (VW == 4) {
                    const f32x4 v = sgk::raw_load_v4f32(rb, off, 0, 0);
                    bv[d][e][0] = v.x;
                    bv[d][e][1] = v.y;
                    bv[d][e][2] = v.z;
                    bv[d][e][3] = v.w;
                } else if constexpr (VW == 2) {
                    const f32x2 v = sgk::raw_load_v2f32(rb, off, 0, 0);
                    bv[d][e][0] = v.x;
                    bv[d][e][1] = v.y;
                } else {
                    bv[d][e][0] = sgk::raw_load_f32(rb, off, 0, 0);
                }
            }
        }
    };
    auto multiply = [&](int d, int s) {
        // k's from K on: A's row goes on into what follows it (so does B's as N x K)
        const int left = K - (16 * s + 4 * lk);
        const bool tail = 16 * s + 16 > K;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x[MB];
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                x[i] = e == 0 ? av[d][i].x : e == 1 ? av[d][i].y : e == 2 ? av[d][i].z : av[d][i].w;
                if (tail) x[i] = e < left ? x[i] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                float y = bv[d][e][j];
                if (TRANS_B && tail) y = e < left ? y : 0.0f;
#pragma unroll
                for (int i = 0; i < MB; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y, acc[i][j], 0, 0, 0);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, s0 + d);
    for (int s = s0; s < s1; s += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (s + d < s1) multiply(d, s + d);
            fetch(d, s + d + D);
        }
    }

    // acc[i][j] register r on lane (li, lk): row 16 i + 4 lk + r, column VW li + j
    // (K x N) or 16 j + li (N x K)
    const float al = group_alpha(a, g);
    auto store = [&](int row, int col, float v) {
        const int p = p0 + row, n = n0 + col;
        if (p >= p1 || n >= a.N) return;
        const int64_t c = row_of(a, p, a.c_scatter);
        if (c < 0) return;
        float *q = a.C + c * a.ldc + n;
        *q = a.beta != 0.0f ? fmaf(a.beta, *q, al * v) : al * v;
    };
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < VW; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 4 * lk + r, col = TRANS_B ? 16 * j + li : VW * li + j;
                if constexpr (WK == 1) store(row, col, acc[i][j][r]);
                else part[w][row * COLS + col] = acc[i][j][r];
            }
    if constexpr (WK > 1) {
        __syncthreads();
        for (int f = tid; f < ROWS * COLS; f += WK * 64) {
            if (p0 + f / COLS >= p1) break;
            float v = part[0][f];
#pragma unroll
            for (int i = 1; i < WK; ++i) v += part[i][f];
            store(f / COLS, f % COLS, v);
        }
    }
}

}  // namespace rowk
