// block.hip -- C ABI of a feed-forward block's operators (see include/sgemm.h):
// norm, 8-bit rows and their product, gated projections, and back.  Argument checks,
// the choice of kernel and launches on the caller's stream.  No state, no
// allocation.
#include "sgemm.h"

#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "gated_kernels.hpp"
#include "i8_kernels.hpp"
#include "norm_kernels.hpp"
#include "rows_api.hpp"

namespace {

#define NEED(position, condition) \
    if (!(condition)) return SGEMM_ERR_ARGUMENT - (position)

// a launch holds fewer than 2^32 threads
bool fits(long long grid, int threads) { return grid <= INT_MAX && grid * threads < (1LL << 32); }

template <class A>
int enqueue(void (*kernel)(A), long long grid, int threads, const A &args, hipStream_t stream) {
    if (grid <= 0) return SGEMM_OK;
    if (!fits(grid, threads)) return SGEMM_ERR_TOO_LARGE;
    (void)hipGetLastError();  // drop any stale error so the code below is this launch's
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), 0, stream, args);
    return (int)hipGetLastError();
}

// What a kernel's loop steps through in 31 bits is at most this long: no step
// beyond the end passes INT_MAX (it would go on from below 0).
constexpr int kLongest = INT_MAX - 4 * 4096;

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
size_t round_up(size_t x) { return (x + 255) / 256 * 256; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
int at_least_1(int n) { return n > 1 ? n : 1; }
bool is_act(int a) { return a == SGEMM_ACT_SILU || a == SGEMM_ACT_GELU || a == SGEMM_ACT_GELU_TANH; }

int xcd_shift() {
    int xcds = 1, shift = 0;
    (void)sgemm_device_shape(nullptr, &xcds);
    while ((2 << shift) <= xcds) ++shift;
    return shift;
}

// ---- rows in registers -------------------------------------------------------

template <class A> struct RowKernel {
    int threads, columns;
    void (*fn)(A);
};
template <class A, int N> const RowKernel<A> *row_kernel(const RowKernel<A> (&table)[N], int columns) {
    for (const RowKernel<A> &k : table)
        if (columns <= k.columns) return &k;
    return nullptr;
}
template <class A> int launch_rows(const RowKernel<A> &k, int T, const A &a, hipStream_t stream) {
    const int rows = k.threads == 64 ? 4 : 1;
    return enqueue(k.fn, ceil_div(T, rows), k.threads * rows, a, stream);
}

#define ROW(fn, NT, V, ...) {NT, 4 * NT * V, fn<NT, V, ##__VA_ARGS__>}
// Threads x vectors by columns.  Measured (us, rows x columns; threads x vectors):
//   norm to 8 bits: 4000 x 512 7.4 on 64 x 2, 8.6 on 128 x 2, 9.6 on 256 x 1; 515 x 1024 3.5
//   on 128 x 2, 3.6 on 64 x 4, 4.0 on 256 x 2; 2011 x 2048 11.2 on 256 x 2, 12.0 on 64 x 8,
//   12.3 on 512 x 1; 4095 x 4096 39.1 on 512 x 2, 39.6 on 256 x 4, 46.5 on 64 x 16, 41.7 on
//   1024 x 1; one row of 4096 3.3, 3.5, 6.0 and 3.7.
//   The gradient goes the same way (2011 x 2048 12.6 on 256 x 2, 13.3 on 128 x 4, 15.7 on 64 x 8).
const RowKernel<normk::NormArgs> kNorms[] = {
    ROW(normk::norm, 64, 1), ROW(normk::norm, 64, 2), ROW(normk::norm, 128, 2), ROW(normk::norm, 256, 2),
    ROW(normk::norm, 512, 2), ROW(normk::norm, 512, 4), ROW(normk::norm, 1024, 4)};
#define QUANTIZE(ACT)                                                                                          \
    {ROW(normk::quantize, 64, 1, ACT), ROW(normk::quantize, 64, 2, ACT), ROW(normk::quantize, 256, 1, ACT),   \
     ROW(normk::quantize, 256, 2, ACT), ROW(normk::quantize, 512, 2, ACT), ROW(normk::quantize, 512, 4, ACT), \
     ROW(normk::quantize, 1024, 4, ACT)}
const RowKernel<normk::QuantArgs> kQuants[4][7] = {QUANTIZE(0), QUANTIZE(1), QUANTIZE(2), QUANTIZE(-1)};
void (*const kLongQuants[4])(normk::QuantArgs) = {normk::quantize_long<0>, normk::quantize_long<1>,
                                                  normk::quantize_long<2>, normk::quantize_long<-1>};
const RowKernel<normk::NormGradArgs> kNormGrads[] = {
    ROW(normk::norm_grad, 64, 1), ROW(normk::norm_grad, 64, 2), ROW(normk::norm_grad, 128, 2),
    ROW(normk::norm_grad, 256, 2), ROW(normk::norm_grad, 512, 2), ROW(normk::norm_grad, 512, 4)};

// Shares that dweight is summed in, a workgroup each.  Measured (us, gradient + sum of the
// shares): 2011 x 2048 12.6 + 3.8 with 512, 14.5 + 3.3 with 256, 13.0 + 4.7 with 1024; on one
// wave a row, 4000 x 512, 9.0 + 4.6 with 1024, 12.0 + 3.7 with 512, 8.8 + 6.6 with 2048.
// Rows too long for registers have half as many, of 64 bits, where they are of more than one row.
bool long_shares(int T, int N) { return row_kernel(kNormGrads, N) == nullptr && T > 512; }
int weight_shares(int T, int N) {
    const int most = N <= 512 ? 1024 : long_shares(T, N) ? 256 : 512;
    return T < most ? T : most;
}

bool workspace_ok(const void *p, size_t have, size_t need) {
    return need == 0 || (p != nullptr && have >= need && ((uintptr_t)p & 255u) == 0);
}

size_t norm_grad_bytes(int T, int N) { return round_up((size_t)weight_shares(T, N) * N * (long_shares(T, N) ? 8 : 4)); }

// ---- 8-bit products ------------------------------------------------------------
struct I8Kernel {
    int bm, bn, threads;
    void (*fn)(i8k::Args);
};
#define I8_TILE(BM, BN, BK, WM, WN, KG, WPE) \
    {BM, BN, KG * (BM / WM) * (BN / WN) * 64, i8k::i8_tile<BM, BN, BK, WM, WN, KG, 2, 1, WPE>}
#define I8_THIN(MB, NB, WK, WPE) {16 * MB, 16 * NB, WK * 64, i8k::i8_thin<MB, NB, WK, WPE>}
const I8Kernel kI8Large = I8_TILE(256, 256, 128, 64, 64, 1, 4);  // 16 waves, one workgroup per CU
const I8Kernel kI8Mid = I8_TILE(128, 128, 128, 32, 64, 1, 4);    // 8 waves, two per CU
const I8Kernel kI8Lone = I8_TILE(128, 128, 256, 32, 64, 1, 2);   // 8 waves, one per CU
const I8Kernel kI8Small = I8_TILE(64, 64, 256, 32, 32, 2, 4);    // 8 waves in two groups, two per CU
const I8Kernel kI8Thin1 = I8_THIN(1, 1, 8, 4);
const I8Kernel kI8Thin2 = I8_THIN(2, 1, 8, 2);
const I8Kernel kI8Thin4 = I8_THIN(4, 1, 8, 2);
const I8Kernel kI8Thin42 = I8_THIN(4, 2, 8, 2);
const I8Kernel kI8Any = {64, 64, 256, i8k::i8_any};

long long tiles(const I8Kernel &k, int M, int N) { return ceil_div(M, k.bm) * ceil_div(N, k.bn); }

// Measured (us, N = K = 4096, A from memory; thin: 16, 32 and 64 rows):
//   rows           1    8   37*  64  100  200  1024  2048  4096      (* 4096 x 2048)
//   thin          5.2  5.7  6.1 12.0 18.4 33.4   145
//   64 x 64      12.5 12.5  8.0 12.6 12.7 16.3  33.3  64.5   127  (one group of 4 waves;
//     two groups, B from memory too: 100 rows 16.3 against 17.8, 515 x 1024 x 2816 12.6 against 13.4)
//   128 x 128    21.5 21.4 13.2 21.6 21.6 28.9  31.8  40.9    80
//     256 of K   18.4 18.2 11.6 18.3 18.2 22.4  25.9  53.1   104
//   256 x 256    46.3 46.2 28.6 46.3 46.6 50.6  51.7  54.0    73
// So up to 64 rows thin; then by rounds of tiles (256 CUs; 64 x 64: two on each), each
// priced by what a full one took: 64 x 64 10, 128 x 128 16 alone on its CU and 13.5
// among others, 256 x 256 48, of which 22 by how full it is (2700 x 3200 x 3328, 143 tiles of 256 x 256: 48
// us, 550 of 128 x 128: 59).  The prices are of K = 4096 and hold the start and the stores, which
// weigh more where K is short; up to 64 rows wide N was not measured.  The thin and the 64 x 64
// kernels take in about 40 GB/s per CU at these sizes, with the loads that they have in flight (256 x 256
// takes in 69), so 64 x 32 thin tiles, which take in less, win where one round of them is
// enough (100 x 4096 x 4096 14.7 against 17.4 on 64 x 64, 700 x 700 x 5000 16.1 against 23.7; 515 x
// 1024 x 2816, 288 tiles, 17.9 against 13.3).
// C's stores go past the caches, but for a large C whose rows do not begin on half a line: two
// stores fill a half there, and come to memory apart.  Measured (us; past the caches, not): 4096 x 4095
// x 4096 91, 77; 2700 x 3109 x 3298 64, 62; 4096 x 4096 x 4096 74.9, 75.0; 3000 x 6000 x 1000 43.8, 46.2;
// 1000 x 2001 x 500 (8 MB) 7.9, 8.6.
bool i8_streams(const i8k::Args &a) {
    return (a.ldc % 16 == 0 && ((uintptr_t)a.C & 63) == 0) || a.M * (int64_t)a.N < (4 << 20);
}

const I8Kernel &choose_i8(const i8k::Args &a) {
    // the fast kernels load 16 bytes at 4-byte alignment, at 32-bit offsets from a tile's
    // first row
    const bool words = ((uintptr_t)a.A & 3) == 0 && ((uintptr_t)a.B & 3) == 0 && a.lda % 4 == 0 && a.ldb % 4 == 0;
    constexpr int64_t reach = (1LL << 31) / 256 - 1024;
    if (!words || a.lda > reach || a.ldb > reach || a.ldc > reach / 4) return kI8Any;
    if (a.M <= 16) return kI8Thin1;
    if (a.M <= 32) return kI8Thin2;
    if (a.M <= 64) return kI8Thin4;
    const long long mid = tiles(kI8Mid, a.M, a.N);
    const double small = 10.0 * ceil_div(tiles(kI8Small, a.M, a.N), 512);
    const double middle = mid <= 256 ? 16.0 : 13.5 * ceil_div(mid, 256);
    const long long big = tiles(kI8Large, a.M, a.N), rounds = ceil_div(big, 256);
    const double large = 26.0 * rounds + 22.0 * big / 256;
    if (tiles(kI8Thin42, a.M, a.N) <= 256) return kI8Thin42;
    if (small <= middle && small <= large) return kI8Small;
    if (middle <= large) return mid <= 256 ? kI8Lone : kI8Mid;
    return kI8Large;
}

// ---- gated projections -----------------------------------------------------------
struct GatedKernel {
    int bm, bn, threads;  // columns of the result
    void (*fn)(gatedk::TileArgs);
};
#define FORWARD_TILE(BM, BN, BK, WM, WN, KG, WPE) \
    {BM, BN / 2, KG * (BM / WM) * (BN / WN) * 64, gatedk::gated_tile<gatedk::FORWARD, BM, BN, BK, WM, WN, KG, WPE>}
#define BACK_TILE(KIND, BM, BN, BK, WM, WN, WPE) \
    {BM, BN, (BM / WM) * (BN / WN) * 64, gatedk::gated_tile<gatedk::KIND, BM, BN, BK, WM, WN, 1, WPE>}
#define GATED_THIN(MB, VW, WK, WPE) {16 * MB, 16 * VW, WK * 64, gatedk::gated_thin<MB, VW, WK, WPE>}
const GatedKernel kForwardTile[] = {FORWARD_TILE(64, 128, 32, 32, 64, 1, 3), FORWARD_TILE(128, 128, 32, 32, 64, 1, 4),
                                    FORWARD_TILE(256, 256, 32, 64, 64, 1, 4), FORWARD_TILE(64, 128, 32, 32, 64, 2, 4)};
// rows x columns: 16 x 16, 16 x 32, 16 x 64, 32 x 32, 32 x 64
const GatedKernel kThin[] = {GATED_THIN(1, 1, 8, 4), GATED_THIN(1, 2, 8, 4), GATED_THIN(1, 4, 8, 4),
                             GATED_THIN(2, 2, 8, 2), GATED_THIN(2, 4, 8, 2)};
struct FewKernel {
    int bm, bn;  // of dx
    void (*fn)(gatedk::BackArgs);
};
#define GATED_BACK_FEW(MB, VW) {16 * MB, 16 * VW, gatedk::gated_back_few<MB, VW>}
const FewKernel kFew[] = {GATED_BACK_FEW(1, 1), GATED_BACK_FEW(2, 2)};
const GatedKernel kBackX = BACK_TILE(BACK_X, 256, 256, 32, 64, 64, 4);
const GatedKernel kBackW[] = {BACK_TILE(BACK_W, 64, 128, 32, 32, 32, 4), BACK_TILE(BACK_W, 256, 256, 32, 64, 64, 4)};
const GatedKernel kSimpleForward = {32, 32, 256, gatedk::gated_simple<gatedk::FORWARD>};
const GatedKernel kSimpleBackW = {32, 32, 256, gatedk::gated_simple<gatedk::BACK_W>};

long long tiles(const GatedKernel &k, const gatedk::TileArgs &a, int kind) {
    return ceil_div(a.M, k.bm) * ceil_div(a.N, k.bn) * (kind == gatedk::BACK_W ? 2 : 1);
}

// Up to 32 rows G and U are read once and that is the time, so the tiles are as narrow as
// gives every CU one and as wide as leaves about one round of them.  Measured (us, rows x N x
// K; by columns of a tile):
//   1 x 4096 x 2048: 16.5 (16), 18.2 (32), 26.7 (64); 1 x 6000 x 2048: 27.6, 25.3, 34.5;
//   1 x 8000 x 2048: 30.9, 26.6, 34.2; 1 x 11008 x 4096: 108, 96, 73;
//   29 rows (16-row tiles / 32-row): 1024 x 1000: 8.9, 10.9, 15.6 / 12.4, 14.9; 4096 x 2048:
//   26.2, 19.6, 27.8 / 20.7, 26.5, 42.0; 6000 x 2048: 43, 42, 35 / 42, 34, 48; 11008 x 4096:
//   162, 119, 122 / 140, 125, 91.
// More rows: the matrix cores, and how the tiles fill rounds of 256 CUs, set the time.  A
// round costs what 256 workgroups took at K = 2048 (alone; among others):
//   61 x 4096: 31.9 on 16 x 32, 28.6 on 16 x 64, 26.7 on 32 x 32, 42 on 32 x 64, 83 on 64 x 64;
//   100 x 4096: 55.7, 44.3, 50.4, 42.6, 83; 256 x 4096: 106, 84, 101, 85, 85, 136 (128 x 64);
//   400 x 4096: 165, 141, 167, 158, 142, 136; 700 x 4096: 279, 225, 265, 241, 201, 251;
//   1000 x 4096: 394, 319, 391, 340, 276, 255; 4096 x 4096: 1049 on 64 x 64, 1000 on 128 x
//   64, 965 on 256 x 128.
// A round of 64 x 64 alone on its CUs has two groups of waves (74, with one 83: 300 x 3000 x 2000 75,
// 86; 512 x 2048 x 1024 42, 48), beyond one group (1000 x 3001 x 1000 111, with two 118).
const GatedKernel &choose_forward(const gatedk::TileArgs &a, double &least) {
    if (a.M <= 16) return kThin[a.N <= 4608 ? 0 : a.N <= 9216 ? 1 : 2];
    if (a.M <= 32) return kThin[a.N <= 2304 ? 0 : a.N <= 4608 ? 1 : a.N <= 9216 ? 3 : 4];
    struct Round {
        const GatedKernel *kernel;
        double alone, among;
    };
    const Round rounds[] = {{&kThin[0], 16, 10},         {&kThin[1], 18, 13.2},        {&kThin[2], 27, 20.6},
                            {&kThin[3], 26, 25},         {&kThin[4], 42, 42},          {&kForwardTile[0], 83, 70},
                            {&kForwardTile[1], 133, 125}, {&kForwardTile[2], 482, 482}, {&kForwardTile[3], 74, 74}};
    const GatedKernel *best = nullptr;
    for (const Round &r : rounds) {
        const long long n = ceil_div(tiles(*r.kernel, a, gatedk::FORWARD), 256);
        const double cost = n <= 1 ? r.alone : r.among * (double)n;
        if (best == nullptr || cost < least) best = r.kernel, least = cost;
    }
    return *best;
}

// Rows that 64 do not divide: up to a round of tiles of 64 x 64 and the last rows in tiles of 16 x
// 32 behind them, on CUs that hold one of the others.  Priced as above (K = 2048; short K was not
// measured), and 14 for the end.  Measured (us, T x N x K; so, and one kind of tile): 455 x 2276 x
// 2069 96, 116; 456 x 2304 x 2048 87, 103.
bool rest_apart(const gatedk::TileArgs &a, double least) {
    if (a.M <= 64 || a.M % 64 == 0) return false;
    const double first = (double)(a.M / 64 * ceil_div(a.N, 64)), rest = (double)(ceil_div(a.M % 64, 16) * ceil_div(a.N, 32));
    return first <= 256 && fmax((first * 72 + rest * 13.2) / 256, 74.0) + 14 < least;
}
int launch_and_rest(gatedk::TileArgs a, hipStream_t stream) {
    a.xcd_shift = xcd_shift();
    gatedk::RestArgs r = {a, a, 0};
    const int rows = a.M / 64 * 64;
    r.first.M = rows;
    r.rest.M = a.M - rows;
    r.rest.A[0] = r.rest.A[1] = a.A[0] + rows * a.lda;
    r.rest.C[0] = r.rest.C[1] = a.C[0] + rows * a.ldc[0];
    if (a.gate != nullptr) {
        r.rest.gate = a.gate + rows * a.ldgate;
        r.rest.up = a.up + rows * a.ldup;
    }
    const long long ahead = ceil_div(rows / 64 * ceil_div(a.N, 64), 8) * 8;
    if (ahead > INT_MAX) return SGEMM_ERR_TOO_LARGE;
    r.ahead = (int)ahead;
    return enqueue(gatedk::gated_and_rest, ahead + ceil_div(r.rest.M, 16) * ceil_div(a.N, 32), 512, r, stream);
}

// 32-bit offsets from a tile's first row reach all of a tile's operands
bool reachable(const gatedk::TileArgs &a) {
    constexpr int64_t reach = (1LL << 29) / 256 - 1024;
    return a.lda <= reach && a.ldb[0] <= reach && a.ldb[1] <= reach;
}

// x^T [dgate | dup].  Measured (us, T x N x K; 64 x 128 tiles, 256 x 256, and two sums of
// outer products one after the other): 1 x 2048 x 1024 9.7, 21.5, 16.5; 500 x 2048 x 1024
// 43, 128, 46; 2000 x 2048 x 1024 140, 471, 136; 4096 x 4096 x 2048 1042, 967.
const GatedKernel &choose_back_w(const gatedk::TileArgs &a) {
    const double small = 140.0 / 2 * ceil_div(tiles(kBackW[0], a, gatedk::BACK_W), 256);
    const double large = 482.0 * ceil_div(tiles(kBackW[1], a, gatedk::BACK_W), 256);
    return kBackW[large < small ? 1 : 0];
}

int launch_gated(const GatedKernel &k, int kind, gatedk::TileArgs a, hipStream_t stream) {
    a.xcd_shift = xcd_shift();
    a.shares = 1;
    return enqueue(k.fn, tiles(k, a, kind), k.threads, a, stream);
}

// Few rows: both gradients in one launch, where dx has no more than a tile of 16 x 16, or of 32 x
// 32, for each CU.  Measured (us, T x N x K; 16 x 16, 32 x 32, and shares as below): 1 x 2048 x
// 1024 17.5, 30.8, 23.6; 29 rows 21.2, 34, 24.5; 64 rows 25, 35, 26.8; 100 rows -, 37, 31.7; 250 rows -,
// 54, 45.7; 29 x 4096 x 2048 50, 69, 61; 64 rows -, 65, 72; 128 rows -, 107, 87.
const FewKernel *choose_few(const gatedk::TileArgs &x) {
    if (!reachable(x) || x.M > 64) return nullptr;
    for (const FewKernel &k : kFew)
        if (ceil_div(x.M, k.bm) * ceil_div(x.N, k.bn) <= 256) return &k;
    return nullptr;
}

int launch_few(const FewKernel &k, gatedk::BackArgs a, hipStream_t stream) {
    a.x.xcd_shift = a.w.xcd_shift = xcd_shift();
    a.w.shares = 1;
    a.ahead = (int)(ceil_div(ceil_div(a.x.M, k.bm) * ceil_div(a.x.N, k.bn), 8) * 8);
    return enqueue(k.fn, a.ahead + tiles(kBackW[0], a.w, gatedk::BACK_W), kBackW[0].threads, a, stream);
}

// Shares that the sums of dx and of dG and dU are cut into, of their 128 x 64 tiles in one launch
// (either may have none).  Priced in K tiles of 32, about a us: a workgroup costs two beside its
// own, a CU holds three, dx's first, and goes on with what is left; a CU alone with one waits for memory
// (4 more); adding the shares up is a launch and their bytes.  Measured (us, T x N x K; dx's
// shares, the chosen one marked): 455 x 2276 x 2069 224 (1), 187 (2), 172* (3), 178 (4), 172 (8); 500 x
// 2048 x 1024 179 (1), 112 (2), 88 (3), 77* (4), 80 (8); 1000 x 2048 x 1024 207 (1), 145* (2),
// 144 (4); 2000 x 2048 x 1024 263* (1), 271 (2); 128 x 4096 x 1500 307 (1), 97 (4), 77* (6), 73 (8).
struct Cut {
    int x, w;
};
constexpr size_t kCutBytes = 32 << 20;  // of shares, at most
long long whole_vectors(int n) { return ((long long)n + 3) / 4 * 4; }
size_t cut_bytes(int T, int N, int K, const Cut &c) {
    return round_up(c.x > 1 ? (size_t)c.x * T * whole_vectors(K) * 4 : 0) +
           2 * round_up(c.w > 1 ? (size_t)c.w * K * whole_vectors(N) * 4 : 0);
}
long long tiles128x64(long long m, long long n) { return ceil_div(m, 128) * ceil_div(n, 64); }
Cut choose_cut(int T, int N, int K, bool to_x, bool to_w) {
    const double nx = to_x ? (double)tiles128x64(T, K) : 0.0, nw = to_w ? 2.0 * tiles128x64(K, N) : 0.0;
    const double lx = 2.0 * ceil_div(N, 32), lw = (double)ceil_div(T, 32);
    Cut best = {1, 1};
    double least = 0.0;
    for (int w = 1; w <= 8 && (w == 1 || (to_w && lw >= 4 * w && nw * w <= 768)); ++w)
        for (int x = 1; x <= 16 && (x == 1 || (to_x && lx >= 4 * x && nx * x <= 1024)); ++x) {
            const Cut c = {x, w};
            const double bytes = (double)cut_bytes(T, N, K, c);
            if (bytes > (double)kCutBytes) continue;
            const double bx = to_x ? lx / x + 2 : 0.0, bw = to_w ? lw / w + 2 : 0.0;
            const double held = fmin(3.0, ceil((nx * x + nw * w) / 256)), dx = fmin(held, ceil(nx * x / 256));
            const double first = fmax(dx * bx + (held - dx) * bw, fmax(bx, bw)) + (held == 1.0 ? 4 : 0);
            const double cost = fmax((nx * x * bx + nw * w * bw) / 256, first) + (bytes > 0 ? 2.5 + bytes / 12e6 : 0.0);
            if ((x == 1 && w == 1) || cost < least) best = c, least = cost;
        }
    return best;
}

// Tiles of 256 x 256 where they fill the chip: dx in one sum over both halves.
bool back_x_large(const gatedk::TileArgs &a) { return reachable(a) && tiles(kBackX, a, gatedk::BACK_X) >= 224; }

// dx alone on the kernels of sgemm_grouped(), one product after the other, up to 64 rows, for one
// round of short sums and where their tiles of 64 x 64 come in nearly whole rounds, else in shares.  Measured (us, T x N x K; products,
// shares): 1 x 2048 x 1024 13, 18; 64 rows 19, 21; 130 rows 48, 28; 500 rows 50, 46; 1000 rows (256
// tiles) 73, 80; 128 x 4096 x 2048 89, 47; 455 x 2276 x 2069 (264 tiles) 155, 108; 300 x 600 x 3000
// (235) 30, 42; 2000 x 200 x 300 16, 19.  Large ones in one sum on 256 x 256 tiles: 4096 x
// 2048 x 4096 967, 1115 as two products.
bool back_x_pair(const gatedk::TileArgs &a) {
    const long long n = ceil_div(a.M, 64) * ceil_div(a.N, 64);
    return !reachable(a) || a.M <= 64 || (a.K <= 512 && n <= 256) || ceil_div(n, 256) * 256 <= n + n / 4;
}
int gated_back_x(const gatedk::TileArgs &a, hipStream_t stream) {
    if (back_x_large(a)) return launch_gated(kBackX, gatedk::BACK_X, a, stream);
    const int ldb[2] = {(int)a.ldb[0], (int)a.ldb[1]};
    return rowk::rows_product_pair(a.M, a.N, a.K, a.A, (int)a.lda, a.B, ldb, a.C[0], (int)a.ldc[0], stream);
}

gatedk::Shares shares_of(int rows, int cols, int n, float beta, const float *part, float *out, int64_t ldo, int blocks) {
    gatedk::Shares s = {};
    s.blocks = blocks;
    if (n <= 1) return s;
    s.rows = rows;
    s.cols = cols;
    s.shares = n;
    s.beta = beta;
    s.part = part;
    s.ldp = whole_vectors(cols);
    s.out = out;
    s.ldo = ldo;
    s.units = rows * (s.ldp / 4);
    s.blocks += (int)ceil_div(s.units, 256);  // (kCutBytes / 16 / 256 at most)
    return s;
}

int launch_cut(const Cut &c, bool to_x, bool to_w, gatedk::BackArgs a, char *space, hipStream_t stream) {
    const int T = a.x.M, K = a.x.N, N = a.x.K;
    float *px = reinterpret_cast<float *>(space);
    space += c.x > 1 ? round_up((size_t)c.x * T * whole_vectors(K) * 4) : 0;
    float *pG = reinterpret_cast<float *>(space);
    space += c.w > 1 ? round_up((size_t)c.w * K * whole_vectors(N) * 4) : 0;
    float *pU = reinterpret_cast<float *>(space);
    gatedk::SharesArgs sum;
    sum.of[0] = shares_of(T, K, to_x ? c.x : 1, 0.0f, px, a.x.C[0], a.x.ldc[0], 0);
    sum.of[1] = shares_of(K, N, to_w ? c.w : 1, a.w.beta, pG, a.w.C[0], a.w.ldc[0], sum.of[0].blocks);
    sum.of[2] = shares_of(K, N, to_w ? c.w : 1, a.w.beta, pU, a.w.C[1], a.w.ldc[1], sum.of[1].blocks);
    a.x.shares = c.x;
    a.w.shares = c.w;
    a.x.xcd_shift = a.w.xcd_shift = xcd_shift();
    if (c.x > 1) {
        a.x.C[0] = a.x.C[1] = px;
        a.x.ldc[0] = a.x.ldc[1] = whole_vectors(K);
    }
    if (c.w > 1) {
        a.w.C[0] = pG;
        a.w.C[1] = pU;
        a.w.ldc[0] = a.w.ldc[1] = whole_vectors(N);
        a.w.beta = 0.0f;
    }
    const long long dx = to_x ? tiles128x64(T, K) * c.x : 0, dw = to_w ? 2 * tiles128x64(K, N) * c.w : 0;
    if (dx > INT_MAX) return SGEMM_ERR_TOO_LARGE;
    a.ahead = (int)dx;
    const int rc = enqueue(gatedk::gated_back_tiles, dx + dw, 512, a, stream);
    return rc != SGEMM_OK ? rc : enqueue(gatedk::gated_sum, sum.of[2].blocks, 256, sum, stream);
}

// Workspace of the gradient: dgate and dup, rows of N rounded up to whole vectors, and but for few
// rows the room for shares (the same for all sizes: what is enough for T rows is for fewer)
int64_t slope_ld(int N) { return ((int64_t)N + 3) / 4 * 4; }
size_t slope_bytes(int T, int N) { return 2 * round_up((size_t)T * slope_ld(N) * 4); }
size_t gated_grad_bytes(int T, int N, int K) {
    const bool few = T <= 64 && ceil_div(T, 32) * ceil_div(K, 32) <= 256;
    return slope_bytes(T, N) + (few ? 0 : kCutBytes);
}

}  // namespace

extern "C" {

int sgemm_norm(int T, int N, const float *x, int ldx, const float *residual, int ldr, const float *weight, float eps,
               float *sum, int lds, float *y, int ldy, signed char *q, int ldq, float *scales, hipStream_t stream) {
    NEED(1, T >= 0);
    NEED(2, N >= 0);
    const bool empty = T == 0 || N == 0;
    NEED(3, (empty || x != nullptr) && aligned4(x));
    NEED(4, ldx >= at_least_1(N));
    NEED(5, aligned4(residual));
    NEED(6, ldr >= at_least_1(N));
    NEED(7, aligned4(weight));
    NEED(8, eps >= 0.0f && eps <= 3.402823466e38f);
    NEED(9, aligned4(sum));
    NEED(10, lds >= at_least_1(N));
    NEED(11, aligned4(y));
    NEED(12, ldy >= at_least_1(N));
    NEED(14, ldq >= at_least_1(N));
    NEED(15, (T == 0 || q == nullptr || scales != nullptr) && aligned4(scales));
    if (T == 0 || (N == 0 && q == nullptr) || (sum == nullptr && y == nullptr && q == nullptr)) return SGEMM_OK;
    if (T > kLongest || N > kLongest) return SGEMM_ERR_TOO_LARGE;
    normk::NormArgs a;
    a.T = T;
    a.N = N;
    a.eps = (double)eps;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.ldx = ldx;
    a.ldr = ldr;
    a.sum = sum;
    a.y = y;
    a.scales = scales;
    a.lds = lds;
    a.ldy = ldy;
    a.ldq = ldq;
    a.q = q;
    const RowKernel<normk::NormArgs> *k = row_kernel(kNorms, N);
    if (k == nullptr) return enqueue(normk::norm_long, T, normk::kLongThreads, a, stream);
    return launch_rows(*k, T, a, stream);
}

size_t sgemm_norm_grad_workspace_size(int T, int N) { return T < 0 || N < 0 ? 0 : norm_grad_bytes(T, N); }

int sgemm_norm_grad(int T, int N, const float *h, int ldh, const float *weight, float eps, const float *dy, int lddy,
                    const float *dsum, int ldds, float *dh, int lddh, float beta, float *dweight, void *workspace,
                    size_t workspace_bytes, hipStream_t stream) {
    NEED(1, T >= 0);
    NEED(2, N >= 0);
    const bool empty = T == 0 || N == 0;
    NEED(3, (empty || h != nullptr) && aligned4(h));
    NEED(4, ldh >= at_least_1(N));
    NEED(5, aligned4(weight));
    NEED(6, eps >= 0.0f && eps <= 3.402823466e38f);
    NEED(7, (empty || dy != nullptr) && aligned4(dy));
    NEED(8, lddy >= at_least_1(N));
    NEED(9, aligned4(dsum));
    NEED(10, ldds >= at_least_1(N));
    NEED(11, aligned4(dh));
    NEED(12, lddh >= at_least_1(N));
    NEED(14, aligned4(dweight));
    if (N == 0 || (dh == nullptr && dweight == nullptr)) return SGEMM_OK;
    if (dweight != nullptr && !workspace_ok(workspace, workspace_bytes, norm_grad_bytes(T, N))) return SGEMM_ERR_WORKSPACE;
    const long long sums = ceil_div(N, normk::kShareColumns);
    constexpr int sum_threads = normk::kShareColumns * normk::kShareGroups;
    if (T > kLongest || N > kLongest || (dweight != nullptr && !fits(sums, sum_threads))) return SGEMM_ERR_TOO_LARGE;
    normk::NormGradArgs a;
    a.T = T;
    a.N = N;
    a.eps = (double)eps;
    a.h = h;
    a.weight = weight;
    a.dy = dy;
    a.dsum = dsum;
    a.ldh = ldh;
    a.lddy = lddy;
    a.ldds = ldds;
    a.lddh = lddh;
    a.dh = dh;
    a.part = dweight == nullptr ? nullptr : workspace;
    a.dweight = dweight;
    a.beta = beta;
    a.stream = T * (int64_t)N >= (32 << 20);  // 128 MiB, half of the last-level cache
    const bool wide = dweight != nullptr && long_shares(T, N);
    a.P = weight_shares(T, N) * (dweight == nullptr && long_shares(T, N) ? 2 : 1);  // (dh alone: 512 workgroups too)
    const RowKernel<normk::NormGradArgs> *k = row_kernel(kNormGrads, N);
    const int rc = k != nullptr ? enqueue(k->fn, a.P, k->threads, a, stream)
                                : enqueue(wide ? normk::norm_grad_long_shares : normk::norm_grad_long, a.P,
                                          normk::kLongThreads, a, stream);
    if (rc != SGEMM_OK || dweight == nullptr) return rc;
    return enqueue(wide ? normk::norm_weight_grad<double> : normk::norm_weight_grad<float>, sums, sum_threads, a, stream);
}

int sgemm_quantize(int T, int N, const float *x, int ldx, int activation, const float *gate, int ldg, signed char *q,
                   int ldq, float *scales, hipStream_t stream) {
    NEED(1, T >= 0);
    NEED(2, N >= 0);
    const bool empty = T == 0 || N == 0;
    NEED(3, (empty || x != nullptr) && aligned4(x));
    NEED(4, ldx >= at_least_1(N));
    NEED(5, is_act(activation));
    NEED(6, aligned4(gate));
    NEED(7, ldg >= at_least_1(N));
    NEED(8, empty || q != nullptr);
    NEED(9, ldq >= at_least_1(N));
    NEED(10, (T == 0 || scales != nullptr) && aligned4(scales));
    if (T == 0) return SGEMM_OK;
    if (T > kLongest || N > kLongest) return SGEMM_ERR_TOO_LARGE;
    normk::QuantArgs a;
    a.T = T;
    a.N = N;
    a.x = x;
    a.gate = gate;
    a.ldx = ldx;
    a.ldg = ldg;
    a.ldq = ldq;
    a.q = q;
    a.scales = scales;
    const int kind = gate == nullptr ? 3 : activation;
    const RowKernel<normk::QuantArgs> *k = row_kernel(kQuants[kind], N);
    if (k == nullptr) return enqueue(kLongQuants[kind], T, normk::kLongThreads, a, stream);
    return launch_rows(*k, T, a, stream);
}

int sgemm_i8(int M, int N, int K, float alpha, const signed char *A, int lda, const float *a_scales,
             const signed char *B, int ldb, const float *b_scales, float beta, float *C, int ldc, hipStream_t stream) {
    NEED(1, M >= 0);
    NEED(2, N >= 0);
    NEED(3, K >= 0);
    const bool empty = M == 0 || N == 0;
    const bool product = !empty && K > 0 && alpha != 0.0f;
    NEED(5, !product || A != nullptr);
    NEED(6, lda >= at_least_1(K));
    NEED(7, aligned4(a_scales));
    NEED(8, !product || B != nullptr);
    NEED(9, ldb >= at_least_1(K));
    NEED(10, aligned4(b_scales));
    NEED(12, (empty || C != nullptr) && aligned4(C));
    NEED(13, ldc >= at_least_1(N));
    if (empty || (!product && beta == 1.0f)) return SGEMM_OK;
    if (K > SGEMM_I8_MAX_K || M > kLongest || N > kLongest) return SGEMM_ERR_TOO_LARGE;
    i8k::Args a;
    a.M = M;
    a.N = N;
    a.K = product ? K : 0;
    a.alpha = alpha;
    a.beta = beta;
    a.A = A;
    a.B = B;
    a.sa = a_scales;
    a.sb = b_scales;
    a.C = C;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.xcd_shift = xcd_shift();
    a.stream = i8_streams(a);
    const I8Kernel &k = choose_i8(a);
    return enqueue(k.fn, tiles(k, M, N), k.threads, a, stream);
}

int sgemm_gated(int T, int N, int K, int activation, const float *x, int ldx, const float *G, int ldg, const float *U,
                int ldu, float *y, int ldy, float *gate, int ldgate, float *up, int ldup, hipStream_t stream) {
    NEED(1, T >= 0);
    NEED(2, N >= 0);
    NEED(3, K >= 0);
    NEED(4, is_act(activation));
    const bool empty = T == 0 || N == 0, product = !empty && K > 0;
    NEED(5, (!product || x != nullptr) && aligned4(x));
    NEED(6, ldx >= at_least_1(K));
    NEED(7, (!product || G != nullptr) && aligned4(G));
    NEED(8, ldg >= at_least_1(N));
    NEED(9, (!product || U != nullptr) && aligned4(U));
    NEED(10, ldu >= at_least_1(N));
    NEED(11, (empty || y != nullptr) && aligned4(y));
    NEED(12, ldy >= at_least_1(N));
    NEED(13, aligned4(gate));
    NEED(14, ldgate >= at_least_1(N));
    NEED(15, (gate == nullptr) == (up == nullptr) && aligned4(up));
    NEED(16, ldup >= at_least_1(N));
    if (empty) return SGEMM_OK;
    if (T > kLongest || N > kLongest || K > kLongest) return SGEMM_ERR_TOO_LARGE;
    gatedk::TileArgs a = {};
    a.M = T;
    a.N = N;
    a.K = K;
    a.act = activation;
    a.A[0] = a.A[1] = x;
    a.B[0] = G;
    a.B[1] = U;
    a.lda = ldx;
    a.ldb[0] = ldg;
    a.ldb[1] = ldu;
    a.C[0] = a.C[1] = y;
    a.ldc[0] = a.ldc[1] = ldy;
    a.gate = gate;
    a.up = up;
    a.ldgate = ldgate;
    a.ldup = ldup;
    if (!reachable(a)) return launch_gated(kSimpleForward, gatedk::FORWARD, a, stream);
    double cost = 0.0;
    const GatedKernel &k = choose_forward(a, cost);
    return rest_apart(a, cost) ? launch_and_rest(a, stream) : launch_gated(k, gatedk::FORWARD, a, stream);
}

size_t sgemm_gated_grad_workspace_size(int T, int N, int K) {
    return T < 0 || N < 0 || K < 0 ? 0 : gated_grad_bytes(T, N, K);
}

int sgemm_gated_grad(int T, int N, int K, int activation, const float *x, int ldx, const float *G, int ldg,
                     const float *U, int ldu, const float *gate, int ldgate, const float *up, int ldup,
                     const float *dy, int lddy, float *dx, int lddx, float beta, float *dG, int lddg, float *dU,
                     int lddu, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    NEED(1, T >= 0);
    NEED(2, N >= 0);
    NEED(3, K >= 0);
    NEED(4, is_act(activation));
    const bool to_x = dx != nullptr && T > 0 && K > 0, to_w = dG != nullptr && N > 0 && K > 0;
    const bool slopes = T > 0 && N > 0 && (to_x || to_w);  // else the sums are empty
    NEED(5, (!(slopes && to_w) || x != nullptr) && aligned4(x));
    NEED(6, ldx >= at_least_1(K));
    NEED(7, (!(slopes && to_x) || G != nullptr) && aligned4(G));
    NEED(8, ldg >= at_least_1(N));
    NEED(9, (!(slopes && to_x) || U != nullptr) && aligned4(U));
    NEED(10, ldu >= at_least_1(N));
    NEED(11, (!slopes || gate != nullptr) && aligned4(gate));
    NEED(12, ldgate >= at_least_1(N));
    NEED(13, (!slopes || up != nullptr) && aligned4(up));
    NEED(14, ldup >= at_least_1(N));
    NEED(15, (!slopes || dy != nullptr) && aligned4(dy));
    NEED(16, lddy >= at_least_1(N));
    NEED(17, aligned4(dx));
    NEED(18, lddx >= at_least_1(K));
    NEED(20, aligned4(dG));
    NEED(21, lddg >= at_least_1(N));
    NEED(22, (dG == nullptr) == (dU == nullptr) && aligned4(dU));
    NEED(23, lddu >= at_least_1(N));
    if (slopes && !workspace_ok(workspace, workspace_bytes, gated_grad_bytes(T, N, K))) return SGEMM_ERR_WORKSPACE;
    if (T > kLongest || N > kLongest || K > kLongest || (to_x && T >= rowk::kMostRows)) return SGEMM_ERR_TOO_LARGE;
    const int64_t ldz = slope_ld(at_least_1(N));  // (a leading dimension, also of no columns)
    float *dgate = static_cast<float *>(workspace);
    float *dup = reinterpret_cast<float *>(static_cast<char *>(workspace) + round_up((size_t)T * ldz * 4));
    gatedk::BackArgs a = {};
    a.x.M = T;
    a.x.N = K;
    a.x.K = N;
    a.x.A[0] = dgate;
    a.x.A[1] = dup;
    a.x.lda = ldz;
    a.x.B[0] = G;
    a.x.B[1] = U;
    a.x.ldb[0] = ldg;
    a.x.ldb[1] = ldu;
    a.x.C[0] = a.x.C[1] = dx;
    a.x.ldc[0] = a.x.ldc[1] = lddx;
    a.w.M = K;
    a.w.N = N;
    a.w.K = T;
    a.w.A[0] = a.w.A[1] = x;
    a.w.lda = ldx;
    a.w.B[0] = dgate;
    a.w.B[1] = dup;
    a.w.ldb[0] = a.w.ldb[1] = ldz;
    a.w.beta = beta;
    a.w.C[0] = dG;
    a.w.C[1] = dU;
    a.w.ldc[0] = lddg;
    a.w.ldc[1] = lddu;
    const GatedKernel &weights = reachable(a.w) ? choose_back_w(a.w) : kSimpleBackW;
    if (to_w && !fits(tiles(weights, a.w, gatedk::BACK_W), weights.threads)) return SGEMM_ERR_TOO_LARGE;  // (before any launch)
    if (slopes) {
        gatedk::SlopeArgs s;
        s.T = T;
        s.N = N;
        s.gate = gate;
        s.up = up;
        s.dy = dy;
        s.ldgate = ldgate;
        s.ldup = ldup;
        s.lddy = lddy;
        s.ldz = ldz;
        s.dgate = dgate;
        s.dup = dup;
        s.chunks = (int)ceil_div(ldz, 256);
        s.units = (int64_t)T * s.chunks;
        const int rc = enqueue(activation == SGEMM_ACT_SILU   ? gatedk::gated_slopes<normk::kSilu>
                               : activation == SGEMM_ACT_GELU ? gatedk::gated_slopes<normk::kGelu>
                                                              : gatedk::gated_slopes<normk::kGeluTanh>,
                               ceil_div(s.units, 4), 256, s, stream);
        if (rc != SGEMM_OK) return rc;
    }
    char *room = static_cast<char *>(workspace) + slope_bytes(T, N);
    const bool tiled = slopes && reachable(a.x) && reachable(a.w);
    if (tiled && to_x && to_w) {
        const FewKernel *few = choose_few(a.x);
        if (few != nullptr) return launch_few(*few, a, stream);
        if (!back_x_large(a.x) && &weights == &kBackW[0])
            return launch_cut(choose_cut(T, N, K, true, true), true, true, a, room, stream);
    }
    if (to_x) {
        const int rc = tiled && !back_x_large(a.x) && !back_x_pair(a.x)
                           ? launch_cut(choose_cut(T, N, K, true, false), true, false, a, room, stream)
                           : gated_back_x(a.x, stream);
        if (rc != SGEMM_OK) return rc;
    }
    if (to_w && !(T == 0 && beta == 1.0f)) {
        const Cut c = tiled && &weights == &kBackW[0] ? choose_cut(T, N, K, false, true) : Cut{1, 1};
        return c.w > 1 ? launch_cut(c, false, true, a, room, stream) : launch_gated(weights, gatedk::BACK_W, a.w, stream);
    }
    return SGEMM_OK;
}

}  // extern "C"
