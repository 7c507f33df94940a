// grouped_kernels.hpp -- products over groups of rows on the matrix cores.
//
//   * outer: a group's sum of outer products, the sum running over its slots.
//   * thin: up to 64 rows of one group at a time, A's rows gathered and C's
//     scattered; B as K x N or N x K.
//
// All load through buffer descriptors whose byte offsets are 32-bit: an access
// past a descriptor's end reads 0.0, with no branch, and 16-byte loads need
// only 4-byte alignment.
#pragma once

#include "rows_kernels.hpp"

namespace rowk {

typedef float floatx4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// The order of a launch's tiles.  Workgroup ids go to the XCDs in turn, and the
// tile columns of all groups, one group's after the other's, are dealt to the
// XCDs in turn as well: all row tiles of a column meet in one L2, and every XCD
// has its share of every group, whatever rows it holds (given runs of whole
// groups, an XCD with large ones finished last: 32 groups of 60 rows kept a CU
// busy 75% of the time).  An XCD walks a group in bands of up to eight row tiles,
// a band column by column.  A wave looks at 64 groups at a time (each lane one),
// so every wave of a workgroup finds its tile by itself.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int tiles_of(const GroupedArgs &a, int g, int bm, int &lo, int &hi) {
    lo = hi = 0;
    if (g < (a.offsets != nullptr ? a.G : 1)) group_range(a, g, lo, hi);
    return hi > lo ? (hi - lo + bm - 1) / bm : 0;
}
// inclusive sum over the lanes: inside the 16-lane rows (row_shr:n is 0x110 + n),
// then the rows' totals on to the rows behind (row_bcast:15 and :31)
__device__ __forceinline__ int wave_upto(int n) {
    n += __builtin_amdgcn_update_dpp(0, n, 0x111, 0xf, 0xf, false);
    n += __builtin_amdgcn_update_dpp(0, n, 0x112, 0xf, 0xf, false);
    n += __builtin_amdgcn_update_dpp(0, n, 0x114, 0xf, 0xf, false);
    n += __builtin_amdgcn_update_dpp(0, n, 0x118, 0xf, 0xf, false);
    n += __builtin_amdgcn_update_dpp(0, n, 0x142, 0xa, 0xf, false);
    n += __builtin_amdgcn_update_dpp(0, n, 0x143, 0xc, 0xf, false);
    return n;
}

struct Tile {
    int g, p0, p1, bn;  // group, first row, the group's end, first column
};

__device__ __forceinline__ bool place_tile(const GroupedArgs &a, int bm, int bn, int block, Tile &t) {
    const int lane = threadIdx.x & 63;
    const int nbn = (a.N + bn - 1) / bn;
    const int groups = a.offsets != nullptr ? a.G : 1;
    const int X = 1 << a.xcd_shift, x = block & (X - 1);
    int left = block >> a.xcd_shift;  // tiles of XCD x before this one
    for (int base = 0; base < groups; base += 64) {
        int lo, hi;
        const int n = tiles_of(a, base + lane, bm, lo, hi);
        // XCD x's columns of the lane's group: first, first + X, ...
        const int first = (int)(((unsigned)x - (unsigned)(base + lane) * (unsigned)nbn) & (unsigned)(X - 1));
        const int cols = first < nbn ? (nbn - first + X - 1) >> a.xcd_shift : 0;
        const int upto = wave_upto(n * cols);
        const unsigned long long past = __ballot(upto > left);
        if (past == 0) {
            left -= __builtin_amdgcn_readlane(upto, 63);
            continue;
        }
        const int at = __ffsll((long long)past) - 1;
        const int tiles = __builtin_amdgcn_readlane(n, at), mine = __builtin_amdgcn_readlane(cols, at);
        const int s = left - (__builtin_amdgcn_readlane(upto, at) - tiles * mine);
        constexpr int BAND = 8;
        const int band = s / (BAND * mine);
        const int in_band = s - band * BAND * mine;
        const int rows = tiles - band * BAND < BAND ? tiles - band * BAND : BAND;
        const int col = in_band / rows;
        t.g = base + at;
        t.p0 = __builtin_amdgcn_readlane(lo, at) + (band * BAND + in_band - col * rows) * bm;
        t.p1 = __builtin_amdgcn_readlane(hi, at);
        // An XCD's columns are taken in runs of four neighbours while they last: where
        // B's rows are not aligned, neighbours share lines (one row, 4095 x 4095: 15.8
        // us, 20.9 one by one; 64 x 64 rows, 2045 x 512: 35 against 42).  Longer runs
        // spread less over the memory (aligned, one row, 4096 x 4096: 18.1 for the
        // adapters with runs of four or one, 19.1 of eight, 21.3 of 16).
        const int turn = __builtin_amdgcn_readlane(first, at), runs = nbn >> (a.xcd_shift + 2);
        const int column = col < 4 * runs ? (((col >> 2) << a.xcd_shift) + turn) * 4 + (col & 3)
                                          : turn + (col << a.xcd_shift);
        t.bn = column * bn;
        return true;
    }
    return false;
}

// ---------------------------------------------------------------------------
// A group's sum of outer products: C_g (M x N) = sum over its slots of A's row
// (as a column) times B's row.  Both operands lie as v_mfma_f32_16x16x4_f32 takes
// B (`thin` below): lane l of a load has VM (VN) consecutive columns of the row of
// slot 4 (l / 16) + e, whole lines at a time, so neither passes LDS and what is
// loaded is used by one wave.  Each wave sums a 16 VM x 16 VN tile over its share
// of the slots, 16 slots a step, four steps in flight; the WK waves' sums are
// added through LDS in order.
// Where the slots' rows begin is worked out for 64 slots at a time, one per lane,
// and passed through a few hundred bytes of LDS of the wave's own: worked out by
// the lanes that load (each slot 16 times) it took a tenth of the time that the
// MFMAs take, on the same instruction port.
// Measured: 8 groups of 503 slots, 1024 x 2048: 174 us, 97 TFLOP/s, matrix cores
// busy 84%; one group of 8192, 4096 x 16: 31 us, 4.3 TB/s.
// ---------------------------------------------------------------------------
template <int VM, int VN, int WK, int WPE>
__global__ void __launch_bounds__(WK * 64) __attribute__((amdgpu_waves_per_eu(WPE))) outer(GroupedArgs a) {
    constexpr int BM = 16 * VM, BN = 16 * VN;
    constexpr uint32_t NONE = kOut - 4096;  // no row: outside with any column added
    __shared__ __attribute__((aligned(16))) float part[WK > 1 ? WK : 1][WK > 1 ? BM * BN : 1];
    __shared__ __attribute__((aligned(16))) uint32_t begins[WK][2][2][64];  // [wave][unit's parity][A, B][slot]
    const int nbm = (a.M + BM - 1) / BM, nbn = (a.N + BN - 1) / BN;
    // the tile columns of all groups are dealt to the XCDs in turn (as above)
    const int X = 1 << a.xcd_shift, i0 = (int)(blockIdx.x >> a.xcd_shift);
    const int column = ((int)blockIdx.x & (X - 1)) + (i0 / nbm << a.xcd_shift);
    if (column >= a.G * nbn) return;
    const int g = column / nbn;
    const int m0 = i0 % nbm * BM, n0 = (column - g * nbn) * BN;
    int p0, p1;
    group_range(a, g, p0, p1);

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lk = lane >> 4;
    const int64_t a_rows = rows_behind(a.R, a.a_div), b_rows = rows_behind(a.R, a.b_div);
    // rows in order are taken from the group's first: their offsets stay small
    const int64_t a0 = a.a_div == 0 ? p0 : 0, b0 = a.b_div == 0 ? p0 : 0;
    const rsrc_t ra = whole_rsrc(a.A + a0 * a.lda + m0, ((a_rows - a0 - 1) * a.lda + (a.M - m0)) * 4);
    const rsrc_t rb = whole_rsrc(a.B + b0 * a.ldb + n0, ((b_rows - b0 - 1) * a.ldb + (a.N - n0)) * 4);
    const bool listed = a.a_div != 0 || a.b_div != 0;
    const uint32_t lda4 = (uint32_t)a.lda * 4u, ldb4 = (uint32_t)a.ldb * 4u;
    const uint32_t acol = 4u * (uint32_t)(VM * li), bcol = 4u * (uint32_t)(VN * li);

    const int steps = p1 > p0 ? (p1 - p0 + 15) / 16 : 0;
    const int s0 = (int)((int64_t)steps * w / WK), s1 = (int)((int64_t)steps * (w + 1) / WK);
    floatx4 acc[VM][VN];
#pragma unroll
    for (int i = 0; i < VM; ++i)
#pragma unroll
        for (int j = 0; j < VN; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    constexpr int D = 4;  // steps in flight, a unit of 64 slots
    float av[D][4][VM], bv[D][4][VN];
    // this lane's slot of the unit that begins at `step` (-1: none)
    auto read_slot = [&](int step) {
        const int p = p0 + 16 * step + lane;
        if (p >= p1 || step + (lane >> 4) >= s1) return -1;
        if (!listed) return 0;
        const int v = a.rows[p];
        return (unsigned)v < (unsigned)a.R ? v : -1;
    };
    auto note = [&](int parity, int step, int slot) {
        const uint32_t at = (uint32_t)(16 * step + lane);
        const uint32_t arow = a.a_div == 0 ? at : a.a_div == 1 ? (uint32_t)slot : (uint32_t)slot / (uint32_t)a.a_div;
        const uint32_t brow = a.b_div == 0 ? at : a.b_div == 1 ? (uint32_t)slot : (uint32_t)slot / (uint32_t)a.b_div;
        begins[w][parity][0][lane] = slot < 0 ? NONE : arow * lda4;
        begins[w][parity][1][lane] = slot < 0 ? NONE : brow * ldb4;
    };
    auto read = [&](auto &v, rsrc_t r, uint32_t off) {
        constexpr int V = sizeof(v) / sizeof(float);
        if constexpr (V == 4) {
            const f32x4 x = sgk::raw_load_v4f32(r, off, 0, 0);
            v[0] = x.x;
            v[1] = x.y;
            v[2] = x.z;
            v[3] = x.w;
        } else if constexpr (V == 2) {
            const f32x2 x = sgk::raw_load_v2f32(r, off, 0, 0);
            v[0] = x.x;
            v[1] = x.y;
        } else {
            v[0] = sgk::raw_load_f32(r, off, 0, 0);
        }
    };
    auto fetch = [&](int d, int parity) {
        const uint4 ao = *reinterpret_cast<const uint4 *>(&begins[w][parity][0][16 * d + 4 * lk]);
        const uint4 bo = *reinterpret_cast<const uint4 *>(&begins[w][parity][1][16 * d + 4 * lk]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            read(av[d][e], ra, (e == 0 ? ao.x : e == 1 ? ao.y : e == 2 ? ao.z : ao.w) + acol);
            read(bv[d][e], rb, (e == 0 ? bo.x : e == 1 ? bo.y : e == 2 ? bo.z : bo.w) + bcol);
        }
    };
    auto multiply = [&](int d) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < VN; ++j)
#pragma unroll
                for (int i = 0; i < VM; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[d][e][i], bv[d][e][j], acc[i][j], 0, 0, 0);
    };
    if (s0 < s1) {
        // unit u (steps s0 + 4 u ..): its rows are noted while unit u - 2 is
        // multiplied, and its loads go while unit u - 1 is
        note(0, s0, read_slot(s0));
        note(1, s0 + D, read_slot(s0 + D));
#pragma unroll
        for (int d = 0; d < D; ++d) fetch(d, 0);
        int parity = 1;
        for (int step = s0; step < s1; step += D) {
            const int slot = read_slot(step + 2 * D);
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (step + d < s1) multiply(d);
                fetch(d, parity);
            }
            note(parity ^ 1, step + 2 * D, slot);
            parity ^= 1;
        }
    }

    // acc[i][j] register r on lane (li, lk): row VM (4 lk + r) + i, column VN li + j
    const float al = group_alpha(a, g);
    const int mr = a.rank_m ? group_rank(a, g, a.M) : a.M, nr = a.rank_n ? group_rank(a, g, a.N) : a.N;
    float *C = a.C + (int64_t)g * a.stride_c + (int64_t)m0 * a.ldc + n0;
    const int rows = a.M - m0, cols = a.N - n0;  // of C from the tile's corner
    if (VN == 4 && WK == 1 && cols >= BN && a.ldc < 1 << 22 && mr >= m0 + BM && nr >= n0 + BN) {
        // Whole rows of the tile: the lanes' offsets stay and each row's place goes
        // into a descriptor that ends at C_g's last element (64-bit addresses
        // worked out per row took as long as a tenth of the MFMAs).
        const uint32_t off = (uint32_t)(VM * 4 * lk) * (uint32_t)a.ldc * 4u + 16u * (uint32_t)li;
        const int64_t end = ((int64_t)(rows - 1) * a.ldc + cols) * 4;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < VM; ++i) {
                const int64_t row = (int64_t)(VM * r + i) * a.ldc;
                const rsrc_t rc = whole_rsrc(C + row, end - 4 * row);
                f32x4 v;
                v.x = al * acc[i][0 % VN][r];
                v.y = al * acc[i][1 % VN][r];
                v.z = al * acc[i][2 % VN][r];
                v.w = al * acc[i][3 % VN][r];
                if (a.beta != 0.0f) {
                    const f32x4 old = sgk::raw_load_v4f32(rc, off, 0, 0);
                    v.x = fmaf(a.beta, old.x, v.x);
                    v.y = fmaf(a.beta, old.y, v.y);
                    v.z = fmaf(a.beta, old.z, v.z);
                    v.w = fmaf(a.beta, old.w, v.w);
                }
                sgk::raw_store_v4f32(v, rc, off, 0, sgk::kCPolStream);
            }
        return;
    }
    auto write = [&](int m, int n, const auto &v) {
        constexpr int V = sizeof(v) / sizeof(float);
        if (m >= rows) return;
        float *c = C + (int64_t)m * a.ldc + n;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (n + j >= cols) continue;
            const float x = m0 + m < mr && n0 + n + j < nr ? al * v[j] : 0.0f;
            c[j] = a.beta != 0.0f ? fmaf(a.beta, c[j], x) : x;
        }
    };
#pragma unroll
    for (int i = 0; i < VM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v[VN];
#pragma unroll
            for (int j = 0; j < VN; ++j) v[j] = acc[i][j][r];
            const int row = VM * (4 * lk + r) + i;
            if constexpr (WK == 1) {
                write(row, VN * li, v);
            } else {
#pragma unroll
                for (int j = 0; j < VN; ++j) part[w][row * BN + VN * li + j] = v[j];
            }
        }
    if constexpr (WK > 1) {
        __syncthreads();
        for (int f = tid; f < BM * 16; f += WK * 64) {
            const int row = f / 16, col = f % 16 * VN;
            float v[VN];
#pragma unroll
            for (int j = 0; j < VN; ++j) {
                v[j] = part[0][row * BN + col + j];
#pragma unroll
                for (int i = 1; i < WK; ++i) v[j] += part[i][row * BN + col + j];
            }
            write(row, col, v);
        }
    }
}

// ---------------------------------------------------------------------------
// Few rows per group: reading B once is most of the work, so both operands go
// from memory straight to the matrix cores and nothing but the waves' partial
// sums passes LDS.  v_mfma_f32_16x16x4_f32 takes B's element (k l/16, column
// l%16) from lane l: a lane loads VW consecutive columns (B as K x N) or four
// consecutive k (N x K) of 16 k's at a time, and the four k's of a lane are one
// float4 of A's row l%16.  Per KiB of B that is 4 MFMAs of 32 cycles for every
// 16 rows, on four matrix cores 39 TB/s on the chip: beyond 100 rows the matrix
// cores, not B, set the time.  MFMAs are issued for the 16-row blocks that the
// group fills only (the K loop exists once per count of them).  WK waves split K
// and are summed through LDS in order, with no barrier inside the K loop; each
// wave has a few steps in flight.
// Measured: 64 groups of 2 or 3 rows, 1280 x 2048, N x K: 109 us, 5.2 TB/s from HBM;
// 16 groups of 512 rows, 4096 x 2048: 1030 us, 133 TFLOP/s, matrix cores busy 92%.
// ---------------------------------------------------------------------------
template <int MB, int VW, int WK, int WN, int WPE, bool TRANS_B>
__device__ __forceinline__ void thin_tile(const GroupedArgs &a, int block) {
    constexpr int ROWS = 16 * MB, COLS = 16 * VW, NT = WK * WN * 64;
    __shared__ __attribute__((aligned(16))) float part[WK > 1 ? WK : 1][WK > 1 ? WN * ROWS * COLS : 1];
    __shared__ __attribute__((aligned(16))) int c_row[ROWS];
    Tile t;
    if (!place_tile(a, ROWS, COLS * WN, block, t)) return;
    const int g = t.g, p0 = t.p0, p1 = t.p1;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6) / WN, wn = __builtin_amdgcn_readfirstlane(tid >> 6) % WN;
    const int n0 = t.bn + wn * COLS;
    const int li = lane & 15, lk = lane >> 4;
    const int live = p1 - p0 < ROWS ? (p1 - p0 + 15) / 16 : MB;  // 16-row blocks
    int my_row = -1;  // of C: thread m holds the tile's row m
    if (tid < ROWS && p0 + tid < p1) my_row = (int)c_row_of(a, p0 + tid);

    const int K = a.rank_k ? __builtin_amdgcn_readfirstlane(group_rank(a, g, a.K)) : a.K;
    const int steps = (K + 31) / 32;
    const int s0 = (int)((int64_t)steps * w / WK), s1 = (int)((int64_t)steps * (w + 1) / WK);
    const int64_t a_rows = rows_behind(a.R, a.a_div);
    const int64_t a_base = a.a_div == 0 ? p0 : 0;
    const float *a_from = a.A + a_base * a.lda;
    const int64_t a_bytes = ((a_rows - a_base - 1) * a.lda + a.K) * 4;
    uint32_t aoff[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int p = p0 + 16 * i + li;
        int64_t row = row_of(a, p < p1 ? p : p0, a.a_div);
        row = row < 0 ? 0 : row - a_base;
        aoff[i] = (uint32_t)row * (uint32_t)a.lda * 4u;
    }
    const float *B = a.B + (int64_t)g * a.stride_b;
    // K x N: rows from the group's first to K; N x K: from row n0 to the last
    const float *b_base = TRANS_B ? B + (int64_t)n0 * a.ldb : B + n0;
    const int64_t b_bytes = TRANS_B ? ((int64_t)(a.N - n0 - 1) * a.ldb + a.K) * 4 : ((int64_t)(K - 1) * a.ldb + (a.N - n0)) * 4;
    const uint32_t ldb4 = (uint32_t)a.ldb * 4u;
    constexpr int BL = TRANS_B ? VW : 4;  // loads of B per 16 k

    floatx4 acc[MB][VW];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < VW; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    auto k_loop = [&](auto blocks) __attribute__((always_inline)) {
        constexpr int L = decltype(blocks)::value;
        // A step is H halves of 16 k.  With 16 rows or fewer and B as N x K it is two,
        // so that what runs along K is read in whole 128-byte lines (1280 x 2048,
        // 64 groups of two rows: 113 us against 126); elsewhere one half at a time
        // is faster (16 groups of 512 rows, 4096 x 2048: 1019 us against 1121).  Lane
        // group lk takes k H 4 lk + 4 h + e of a step.
        constexpr int H = TRANS_B && L == 1 ? 2 : 1;
        // steps in flight: what 64 registers hold (80 for two halves).  More were
        // slower, for tall tiles too, which have the registers (8 groups of 503 rows,
        // 2048 x 1024, N x K: 172 us with two steps, 178 with three, 189 with four).
        constexpr int SHARE = H == 2 ? 80 : 64, STEP = 4 * H * (VW + L);
        constexpr int D = SHARE / STEP < 8 ? SHARE / STEP : 8;
        static_assert(D >= 2, "steps in flight");
        const int last = (K + 16 * H - 1) / (16 * H);
        const int u0 = s0 * (2 / H), u1 = s1 * (2 / H) < last ? s1 * (2 / H) : last;
        uint32_t al[L], bl[BL];
#pragma unroll
        for (int i = 0; i < L; ++i) al[i] = aoff[i] + (uint32_t)(16 * H * lk);
#pragma unroll
        for (int i = 0; i < BL; ++i)
            bl[i] = TRANS_B ? (uint32_t)(16 * i + li) * ldb4 + (uint32_t)(16 * H * lk)
                            : (uint32_t)(4 * H * lk + i) * ldb4 + 4u * (uint32_t)(VW * li);
        const uint32_t b_half = TRANS_B ? 16u : 4u * ldb4;
        f32x4 av[D][H][L];
        float bv[D][H][4][VW];  // [half][k of the lane][column]
        // A step's place goes into the descriptors (scalar instructions), so the
        // lanes' offsets never change: vector instructions would take the place
        // of MFMAs (with 0.7 of them per MFMA the matrix cores were busy 84% of
        // the time).  Past the wave's last step the descriptors are empty and nothing
        // is read, in a round of its own behind the loop (37 x 4 rows, 64 groups:
        // 112 us, 115 with the last step read again; 8192 rows, 2048 x 2048, N x K: 512
        // against 538).  Only the 64 x 128 tile reads it again (16 x 512 rows, 4096 x
        // 2048: 1034 us, 1084 with the round).
        constexpr bool AGAIN = MB > 2 && !TRANS_B;
        auto fetch = [&](int d, int u, bool there) __attribute__((always_inline)) {
            if constexpr (AGAIN) {
                u = u < u1 ? u : u1 - 1;
                there = true;
            }
            const int64_t k0 = 16 * H * (int64_t)u, b_at = TRANS_B ? k0 : k0 * a.ldb;
            const rsrc_t rb = whole_rsrc(b_base + b_at, there ? b_bytes - 4 * b_at : 0);
            const rsrc_t ra = whole_rsrc(a_from + k0, there ? a_bytes - 4 * k0 : 0);
#pragma unroll
            for (int i = 0; i < BL; ++i)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const uint32_t off = bl[i] + h * b_half;
                    if constexpr (TRANS_B) {
                        const f32x4 v = sgk::raw_load_v4f32(rb, off, 0, 0);
                        bv[d][h][0][i] = v.x;
                        bv[d][h][1][i] = v.y;
                        bv[d][h][2][i] = v.z;
                        bv[d][h][3][i] = v.w;
                    } else if constexpr (VW == 4) {
                        const f32x4 v = sgk::raw_load_v4f32(rb, off, 0, 0);
                        bv[d][h][i][0] = v.x;
                        bv[d][h][i][1] = v.y;
                        bv[d][h][i][2] = v.z;
                        bv[d][h][i][3] = v.w;
                    } else if constexpr (VW == 2) {
                        const f32x2 v = sgk::raw_load_v2f32(rb, off, 0, 0);
                        bv[d][h][i][0] = v.x;
                        bv[d][h][i][1] = v.y;
                    } else {
                        bv[d][h][i][0] = sgk::raw_load_f32(rb, off, 0, 0);
                    }
                }
#pragma unroll
            for (int i = 0; i < L; ++i)
#pragma unroll
                for (int h = 0; h < H; ++h) av[d][h][i] = sgk::raw_load_v4f32(ra, al[i] + 16u * h, 0, 0);
        };
        auto multiply = [&](int d) {
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < VW; ++j)
#pragma unroll
                        for (int i = 0; i < L; ++i) {
                            const f32x4 &v = av[d][h][i];
                            const float x = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x, bv[d][h][e][j], acc[i][j], 0, 0, 0);
                        }
        };
        if (u0 >= u1) return;
        // the last step of K, when it is not whole: A's row goes on into what
        // follows it (so does B's as N x K), which is cleared
        const int whole = (int64_t)u1 * 16 * H > K ? u1 - 1 : u1;
#pragma unroll
        for (int d = 0; d < D; ++d) fetch(d, u0 + d, u0 + d < u1);
        int u = u0;
        for (; u + (AGAIN ? D : 2 * D) <= (AGAIN ? whole : u1); u += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                multiply(d);
                fetch(d, u + d + D, true);
            }
        }
        if (!AGAIN && u + D <= whole) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                multiply(d);
                fetch(d, u + d + D, u + d + D < u1);
            }
            u += D;
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (u + d >= u1) break;
            if (u + d == whole) {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int left = K - (16 * H * whole + 4 * H * lk + 4 * h);
#pragma unroll
                    for (int i = 0; i < L; ++i) {
                        f32x4 &v = av[d][h][i];
                        v.x = 0 < left ? v.x : 0.0f;
                        v.y = 1 < left ? v.y : 0.0f;
                        v.z = 2 < left ? v.z : 0.0f;
                        v.w = 3 < left ? v.w : 0.0f;
                    }
                    if constexpr (TRANS_B) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int j = 0; j < VW; ++j) bv[d][h][e][j] = e < left ? bv[d][h][e][j] : 0.0f;
                    }
                }
            }
            multiply(d);
        }
    };
    if constexpr (MB == 1) {
        k_loop(std::integral_constant<int, 1>());
    } else if constexpr (MB == 2) {
        if (live == 1) k_loop(std::integral_constant<int, 1>());
        else k_loop(std::integral_constant<int, 2>());
    } else {
        static_assert(MB == 4, "up to four blocks of 16 rows");
        if (live == 1) k_loop(std::integral_constant<int, 1>());
        else if (live == 2) k_loop(std::integral_constant<int, 2>());
        else if (live == 3) k_loop(std::integral_constant<int, 3>());
        else k_loop(std::integral_constant<int, 4>());
    }

    // acc[i][j] register r on lane (li, lk): row 16 i + 4 lk + r, column VW li + j
    // (K x N) or 16 j + li (N x K)
    const float al = group_alpha(a, g);
    if (tid < ROWS) c_row[tid] = my_row;
    if constexpr (WK == 1) {
        static_assert(VW == 4, "whole vectors of columns");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            if (i >= live) break;
            // four rows' old values in flight
            const int4 rows = *reinterpret_cast<const int4 *>(&c_row[16 * i + 4 * lk]);
            const int row[4] = {rows.x, rows.y, rows.z, rows.w};
            f32x4u old[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                old[r] = f32x4u{0.0f, 0.0f, 0.0f, 0.0f};
                if (a.beta == 0.0f || row[r] < 0) continue;
                const float *q = a.C + (int64_t)row[r] * a.ldc + n0;
                if constexpr (TRANS_B) {
#pragma unroll
                    for (int j = 0; j < VW; ++j)
                        if (n0 + 16 * j + li < a.N) old[r][j] = q[16 * j + li];
                } else {
                    old[r] = load4(q + 4 * li, a.N - (n0 + 4 * li));
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (row[r] < 0) continue;
                float *q = a.C + (int64_t)row[r] * a.ldc + n0;
                f32x4u v;
                v.x = fmaf(a.beta, old[r].x, al * acc[i][0][r]);
                v.y = fmaf(a.beta, old[r].y, al * acc[i][1][r]);
                v.z = fmaf(a.beta, old[r].z, al * acc[i][2][r]);
                v.w = fmaf(a.beta, old[r].w, al * acc[i][3][r]);
                if constexpr (TRANS_B) {
#pragma unroll
                    for (int j = 0; j < VW; ++j)
                        if (n0 + 16 * j + li < a.N) q[16 * j + li] = v[j];
                } else {
                    store4(q + 4 * li, a.N - (n0 + 4 * li), v);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            if (i >= live) break;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float *q = &part[w][((wn * MB + i) * 16 + 4 * lk + r) * COLS];
                if constexpr (!TRANS_B && VW == 4)
                    *reinterpret_cast<float4 *>(q + 4 * li) = make_float4(acc[i][0][r], acc[i][1][r], acc[i][2][r], acc[i][3][r]);
                else
#pragma unroll
                    for (int j = 0; j < VW; ++j) q[TRANS_B ? 16 * j + li : VW * li + j] = acc[i][j][r];
            }
        }
        __syncthreads();
        // four columns per thread
        for (int f = tid; f < 16 * live * WN * (COLS / 4); f += NT) {
            const int row = f / (WN * COLS / 4), part_n = f % (WN * COLS / 4) / (COLS / 4), col = f % (COLS / 4) * 4;
            const int64_t c = c_row[row];
            const int left = a.N - (t.bn + part_n * COLS + col);
            if (c < 0 || left <= 0) continue;
            const int at = (part_n * ROWS + row) * COLS + col;
            float *q = a.C + c * a.ldc + t.bn + part_n * COLS + col;
            f32x4u old = {0.0f, 0.0f, 0.0f, 0.0f};
            if (a.beta != 0.0f) old = load4(q, left);
            float4 v = *reinterpret_cast<const float4 *>(&part[0][at]);
#pragma unroll
            for (int i = 1; i < WK; ++i) {
                const float4 o = *reinterpret_cast<const float4 *>(&part[i][at]);
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
            f32x4u out;
            out.x = fmaf(a.beta, old.x, al * v.x);
            out.y = fmaf(a.beta, old.y, al * v.y);
            out.z = fmaf(a.beta, old.z, al * v.z);
            out.w = fmaf(a.beta, old.w, al * v.w);
            store4(q, left, out);
        }
    }
}

template <int MB, int VW, int WK, int WN, int WPE, bool TRANS_B>
__global__ void __launch_bounds__(WK * WN * 64) __attribute__((amdgpu_waves_per_eu(WPE))) thin(GroupedArgs a) {
    thin_tile<MB, VW, WK, WN, WPE, TRANS_B>(a, (int)blockIdx.x);
}

// A product and, in workgroups of its own ahead of it, few rows times their
// adapters' U: neither needs the other, and together they are one launch (with
// expand_rows behind it, one row, 4096 x 4096: 18.4 us, 21.4 one after the other;
// 29 rows, 4095 x 2048: 22.7 against 25.2).
struct PairArgs {
    GroupedArgs product;
    ShrinkArgs shrink;
    int ahead;  // workgroups, a multiple of 8: the tiles keep their XCDs
};
template <int MB, int VW, int WK, int WN, int WPE>
__global__ void __launch_bounds__(WK * WN * 64) __attribute__((amdgpu_waves_per_eu(WPE))) thin_and_shrink(PairArgs a) {
    static_assert(WK * WN == 4, "shrink_row's workgroup");
    const int block = (int)blockIdx.x;
    if (block < a.ahead) shrink_row(a.shrink, block);
    else thin_tile<MB, VW, WK, WN, WPE, false>(a.product, block - a.ahead);
}

}  // namespace rowk
