// rows.hip -- C ABI of the calls around products whose B is picked row by row
// (see include/sgemm.h): argument checks, the choice of kernel and launches on
// the caller's stream.  No state, no allocation.
#include "sgemm.h"

#include <limits.h>
#include <stdint.h>

#include "grouped_kernels.hpp"
#include "rows_api.hpp"
#include "rows_kernels.hpp"

namespace {

using rowk::GroupedArgs;

#define NEED(position, condition) \
    if (!(condition)) return SGEMM_ERR_ARGUMENT - (position)

template <class A>
int enqueue(void (*kernel)(A), long long grid, int threads, const A &args, hipStream_t stream) {
    if (grid <= 0) return SGEMM_OK;
    // a launch holds fewer than 2^32 threads
    if (grid > INT_MAX || grid * threads >= (1LL << 32)) return SGEMM_ERR_TOO_LARGE;
    (void)hipGetLastError();  // drop any stale error so the code below is this launch's
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), 0, stream, args);
    return (int)hipGetLastError();
}

// What a kernel's loop steps through in 31 bits is at most this long: no step
// beyond the end passes INT_MAX (it would go on from below 0).
constexpr int kLongest = INT_MAX - 1024;
constexpr int kMostSlots = rowk::kMostRows;  // of sgemm_grouped, and rows of the adapters

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
size_t round_up(size_t x) { return (x + 255) / 256 * 256; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

// ---- the router ------------------------------------------------------------
typedef void (*RouteFn)(rowk::RouteArgs);
typedef void (*RouteGradFn)(rowk::RouteGradArgs);

struct RouteKernel {
    int experts, k;  // at most
    int lanes;       // per row
    RouteFn narrow, wide;
    RouteGradFn grad;
};
#define ROUTE(L, V) {(L) * (V), (L), (L), rowk::route<L, V, false>, rowk::route<L, V, true>, rowk::route_grad<L, V>}
const RouteKernel kRoutes[] = {ROUTE(16, 1), ROUTE(16, 2), ROUTE(16, 4), ROUTE(16, 8), ROUTE(16, 16),
                               ROUTE(64, 1), ROUTE(64, 4), ROUTE(64, 16)};

const RouteKernel &route_kernel(int E, int k) {
    for (const RouteKernel &r : kRoutes)
        if (E <= r.experts && k <= r.k) return r;
    return kRoutes[sizeof kRoutes / sizeof kRoutes[0] - 1];
}

// ---- products over groups of rows -------------------------------------------
// The row tiles that groups of R rows in all can need at most: one for each
// group's first row and one for every further bm rows.
long long row_tiles(const GroupedArgs &a, int bm) {
    const long long groups = a.offsets == nullptr ? 1 : (a.G < a.R ? a.G : a.R);
    return (a.R - groups) / bm + groups;
}

typedef void (*GroupedFn)(GroupedArgs);
typedef void (*PairFn)(rowk::PairArgs);
typedef void (*TwoFn)(rowk::TwoArgs);

// The fast kernels' byte offsets are 32-bit: a gathered operand is addressed
// from its first row, one in order from the tile's (tn: the group's) first.
constexpr long long kReach = 0xffffe000LL;
bool within_reach(long long rows, int div, int ld, long long tile_rows) {
    const long long reached = div == 0 ? (rows < tile_rows ? rows : tile_rows) : ceil_div(rows, div);
    return reached + 1 <= kReach / 4 / ld;
}

struct Block {
    int bm, bn, threads;
    GroupedFn fn;
    PairFn pair;  // with few rows' adapters ahead of it
    TwoFn two;    // two products into one C
};
#define THIN_NN(MB, VW, WK, WN, WPE) \
    {16 * MB, 16 * VW * WN, WK * WN * 64, rowk::thin<MB, VW, WK, WN, WPE, false>, nullptr, nullptr}
#define THIN_FEW(MB, VW, WK, WN, WPE)                                              \
    {16 * MB, 16 * VW * WN, WK * WN * 64, rowk::thin<MB, VW, WK, WN, WPE, false>, \
     rowk::thin_and_shrink<MB, VW, WK, WN, WPE>, nullptr}
#define THIN_NT(MB, VW, WK, WN, WPE)                                                        \
    {16 * MB, 16 * VW * WN, WK * WN * 64, rowk::thin<MB, VW, WK, WN, WPE, true>, nullptr, \
     rowk::thin_twice<MB, VW, WK, WN, WPE, true>}
// rows x columns of a tile; waves over K x waves over columns.  B as K x N:
const Block kTall = THIN_NN(4, 4, 2, 2, 2);      // 64 x 128, 2 x 2
const Block kLow = THIN_FEW(2, 4, 4, 1, 4);       // 32 x 64, 4 x 1
const Block kLowFlat = THIN_NN(2, 4, 1, 1, 4);   // 32 x 64, one wave
const Block kNarrow = THIN_FEW(2, 2, 4, 1, 4);    // 32 x 32, 4 x 1
const Block kLeast = THIN_FEW(1, 2, 4, 1, 4);     // 16 x 32, 4 x 1
const Block kSquare = THIN_FEW(1, 1, 4, 1, 4);    // 16 x 16, 4 x 1
// and as N x K:
const Block kTallT = THIN_NT(4, 4, 4, 1, 2);     // 64 x 64, 4 x 1
const Block kLowT = THIN_NT(2, 4, 4, 1, 4);      // 32 x 64, 4 x 1
const Block kLowFlatT = THIN_NT(2, 4, 1, 1, 4);  // 32 x 64, one wave
const Block kNarrowT = THIN_NT(2, 1, 4, 1, 4);   // 32 x 16, 4 x 1
const Block kSquareT = THIN_NT(1, 1, 4, 1, 4);   // 16 x 16, 4 x 1

// Measured (us; groups x rows in all, N x K):
//   K up to 64: one wave per tile, nothing to split (11 x 4096, 4096 x 32:
//     24 against 44 on four waves).
//   So few tiles that each has a CU to itself (256 of them): 16 rows (9 x 2000, 16 x
//     1024: 5.9 on 16 x 16 against 9.6 on 32 x 32; 4 x 3000, 32 x 2048: 10.9 on
//     16 x 32 against 15.4; with more tiles they lose: 11 x 4096, 32 x 2048: 19.1
//     against 15.8).  16 columns only where B is read for several row tiles
//     anyway: its lines are 128 bytes (16 x 2, 1024 x 2048: 9.5 against 8.8 on
//     32 columns), or no more are there (9 x 20000, 16 x 1024: 20.6 against 28).
//   Fewer than 256 tiles of 32 x 64: narrower columns, so that more CUs read B (one
//     row, 4096 x 4096: 14.4 at 32 columns and 20.6 at 64; B as N x K, where a
//     narrow tile's lines are still whole, 13.5 at 16 and 20.1 at 32).
//     The same for as few columns as an adapter's rank (1 x 8192, 32 x 4096: 26
//     against 39; N x K, 16 x 4096: 25 against 35 on 32 x 64 and 65 on 64 x 64).
//   Many rows per group: 64 rows, read fewer times (16 x 8192, 4096 x 2048: 1024
//     against 1100 on 32 rows; N x K 1110 against 1494), for K x N only where
//     64 x 128 tiles fill the chip often enough (8 x 4022, 2048 x 1024, 1100 tiles:
//     161 against 146 on 32 x 64), for N x K where every CU has a tile (1 x 8192,
//     64 x 4096, 128 tiles: 66 against 47).
//   Else 32 x 64 with four waves over K (64 x 136, 1280 x 2048: 112, 5.4 TB/s).
const Block &choose_block(const GroupedArgs &a, bool trans_b) {
    const long long groups = a.offsets == nullptr ? 1 : a.G;
    const long long squares = row_tiles(a, 16) * ceil_div(a.N, 16);
    const bool few = row_tiles(a, 32) * ceil_div(a.N, 64) < 256;
    if (trans_b) {
        if (a.K <= 64) return kLowFlatT;
        if (squares <= 256) return kSquareT;
        if (few || a.N <= 16) return kNarrowT;
        return a.R > 64 * groups && a.N > 32 && row_tiles(a, 64) * ceil_div(a.N, 64) >= 256 ? kTallT : kLowT;
    }
    if (a.K <= 64) return kLowFlat;
    if (a.N <= 16 || (squares <= 256 && a.R > 16 * groups)) return kSquare;
    if (row_tiles(a, 16) * ceil_div(a.N, 32) <= 256) return kLeast;
    if (few || a.N <= 32) return kNarrow;
    return row_tiles(a, 64) * ceil_div(a.N, 128) >= 2048 && a.R > 64 * groups ? kTall : kLow;
}

// log2 of the device's XCDs: consecutive workgroup ids go to them in turn.  With
// fewer tile columns than XCDs, 0: tiles in turn (dealt by column, an XCD would
// hold all rows of some groups and none of others).
int xcd_shift(long long columns) {
    int xcds = 1, shift = 0;
    (void)sgemm_device_shape(nullptr, &xcds);
    while ((2 << shift) <= xcds) ++shift;
    return columns < xcds ? 0 : shift;
}

// How many workgroups, and the XCDs they are dealt to.
long long grid_of(const Block &b, bool dealt, GroupedArgs &a) {
    a.xcd_shift = dealt ? xcd_shift(ceil_div(a.N, b.bn)) : 0;
    // every XCD's share of the tile columns, rounded up in every row of tiles
    const long long columns = ceil_div(ceil_div(a.N, b.bn), 1LL << a.xcd_shift) << a.xcd_shift;
    return row_tiles(a, b.bm) * columns;
}

int launch_block(const Block &b, bool dealt, GroupedArgs a, hipStream_t stream) {
    const long long grid = grid_of(b, dealt, a);
    return enqueue(b.fn, grid, b.threads, a, stream);
}

// 32-bit offsets reach all of both operands
bool reachable(const GroupedArgs &a, bool trans_b) {
    return within_reach(a.R, a.a_div, a.lda, 256) && (trans_b ? a.N : a.K) + 256LL <= kReach / 4 / a.ldb;
}

int grouped(GroupedArgs a, bool trans_b, hipStream_t stream) {
    if (a.R == 0 || a.N == 0 || a.G == 0) return SGEMM_OK;
    // the kernels count a wave's 64 groups' tiles (16 rows at least) in 31 bits, and
    // step through groups and K by up to 64 beyond their end
    if (a.R >= kMostSlots || a.G > kLongest || a.K > kLongest) return SGEMM_ERR_TOO_LARGE;
    if (a.alpha == 0.0f) a.K = 0;
    if (a.K == 0 && a.beta == 1.0f) return SGEMM_OK;
    if (reachable(a, trans_b)) return launch_block(choose_block(a, trans_b), true, a, stream);
    const Block simple = {32, 32, 256, trans_b ? rowk::grouped_simple<true> : rowk::grouped_simple<false>, nullptr, nullptr};
    return launch_block(simple, false, a, stream);
}

struct BlockTN {
    int bm, bn, threads;
    GroupedFn fn;
};
#define OUTER(VM, VN, WK, WPE) {16 * VM, 16 * VN, WK * 64, rowk::outer<VM, VN, WK, WPE>}
// rows x columns of a tile; waves over the slots
const BlockTN kOuter = OUTER(4, 4, 1, 2);           // 64 x 64, one wave
const BlockTN kOuterDeep = OUTER(4, 4, 4, 2);       // 64 x 64, 4
const BlockTN kSlim[2] = {OUTER(4, 1, 4, 4), OUTER(1, 4, 4, 4)};      // 64 x 16 and 16 x 64, 4
const BlockTN kSlimDeep[2] = {OUTER(4, 1, 8, 4), OUTER(1, 4, 8, 4)};  // the same, 8
const BlockTN kSlimLow[2] = {OUTER(2, 1, 8, 4), OUTER(1, 2, 8, 4)};   // 32 x 16 and 16 x 32, 8
const BlockTN kOuterLeast = OUTER(1, 1, 16, 4);     // 16 x 16, 16

// Each group's slots are summed by the waves of one workgroup, so the fewer tiles
// there are, the narrower they are and the more waves share the slots.  Measured
// (us; groups x slots in all, M x N):
//   1024 tiles of 64 x 64 and more: one wave each (1 x 300, 4096 x 4096: 88 against
//     128 on four); from 256 four waves (2 x 3000, 1024 x 1024: 55 against 71 on
//     64 x 16; with 144 tiles, 768 x 768, 58 against 48).
//   Then 64 x 16 along the longer side (16 x 2000, 4096 x 16: 9.7 on four waves, 14.3
//     on eight; 1 x 8192, 64 x 4096, long and 256 tiles: 57 on four, 49 on eight;
//     3 x 900, 4096 x 16, 192 tiles: 5.8 against 7.4 on 32 x 16).
//   Up to 128 of them: 32 x 16 on eight waves (1 x 16000, 8192 x 16: 110 against 131;
//     1 x 2000, 2048 x 64: 10 against 15 on four waves of 64 x 16).
//   Both sides short: 16 x 16 on 16 waves (1 x 4000, 128 x 128: 9.9 against 16, and
//     68 on 64 x 64; 256 x 256: 16 against 20).
const BlockTN &choose_tn(const GroupedArgs &a) {
    const int longer = a.M >= a.N ? a.M : a.N, shorter = a.M >= a.N ? a.N : a.M, turned = a.M >= a.N ? 0 : 1;
    const long long tiles = a.G * ceil_div(longer, 64) * ceil_div(shorter, 64);
    if (shorter > 32 && tiles >= 256) return tiles >= 1024 ? kOuter : kOuterDeep;
    const long long slim = a.G * ceil_div(longer, 64) * ceil_div(shorter, 16);
    if (slim > 128) return slim < 512 && a.R >= 512LL * a.G ? kSlimDeep[turned] : kSlim[turned];
    return shorter > 32 && slim <= 64 ? kOuterLeast : kSlimLow[turned];
}

int grouped_tn(GroupedArgs a, hipStream_t stream) {
    if (a.G == 0 || a.M == 0 || a.N == 0) return SGEMM_OK;
    if (a.alpha == 0.0f) a.R = 0;  // every group's range is then empty
    if (a.R == 0 && a.beta == 1.0f) return SGEMM_OK;
    if (a.R > kLongest) return SGEMM_ERR_TOO_LARGE;  // the slots are stepped through likewise
    const bool reach = within_reach(a.R, a.a_div, a.lda, a.R) && within_reach(a.R, a.b_div, a.ldb, a.R);
    const BlockTN simple = {32, 32, 256, rowk::grouped_tn_simple};
    const BlockTN &b = reach ? choose_tn(a) : simple;
    const long long nbm = ceil_div(a.M, b.bm), nbn = ceil_div(a.N, b.bn);
    if (nbm * nbn > INT_MAX / a.G) return SGEMM_ERR_TOO_LARGE;
    a.xcd_shift = reach ? xcd_shift(nbn) : 0;
    const long long columns = ceil_div(nbn * a.G, 1LL << a.xcd_shift) << a.xcd_shift;
    return enqueue(b.fn, nbm * columns, b.threads, a, stream);
}

// ---- slots sorted by group ---------------------------------------------------
// Slots per workgroup of the two-launch form: one turn of kGroupSlots, more beyond
// 256 workgroups (each adds up the counts of all).
int group_run(int R) { return (int)(ceil_div(R > 0 ? R : 1, 256LL * rowk::kGroupSlots) * rowk::kGroupSlots); }
int group_workgroups(int R) { return R <= rowk::kGroupSlots ? 1 : (int)ceil_div(R, group_run(R)); }

size_t group_bytes(int R, int G) {
    const int n = group_workgroups(R);
    return n == 1 ? 0 : round_up((size_t)n * G * 4);
}

template <int GMAX, int WAVES> int group_launch(rowk::GroupArgs a, int n, hipStream_t stream) {
    if (n > 1) {
        const int rc = enqueue(rowk::group_rows<GMAX, WAVES, true>, n, 64 * WAVES, a, stream);
        if (rc != SGEMM_OK) return rc;
    }
    return enqueue(rowk::group_rows<GMAX, WAVES, false>, n, 64 * WAVES, a, stream);
}

int group(int R, int G, const int *ids, int *offsets, int *rows, void *workspace, hipStream_t stream) {
    const int n = group_workgroups(R);
    rowk::GroupArgs a;
    a.R = R;
    a.G = G;
    a.run = group_run(R);
    a.ids = ids;
    a.offsets = offsets;
    a.rows = rows;
    a.counts = static_cast<int *>(workspace);
    if (R <= 64) return enqueue(rowk::group_few, 1, 64, a, stream);
    return G <= 1024 ? group_launch<1024, 16>(a, n, stream) : group_launch<SGEMM_MAX_GROUPS, 8>(a, n, stream);
}

bool workspace_ok(const void *p, size_t have, size_t need) {
    return need == 0 || (p != nullptr && have >= need && ((uintptr_t)p & 255u) == 0);
}

// ---- adapters ----------------------------------------------------------------
// Up to 64 rows, which a batch of sequences has, each with an adapter of its own: in
// one launch alpha A B + beta C and h = A[m] U_g in pieces of K, then C += alpha s h
// V_g, a wave per row and 256 columns.  More: rows sorted by adapter, H = A U_g, the
// projection, and C += H V_g.  (Summing A B and H V_g over sorted rows in one
// grouped product was slower, 4096 x 4096 x 2048 with 11 adapters 613 us against
// 559: sgemm's blocks gain more than C's extra traffic costs.)
//   Measured on both (us, few rows against sorted; K x N):
//     4096 x 4096, rank 16: 1 row 17.6 / 30.9, 29 of as many adapters 22.3 / 39.2,
//       64 of one 32.5 / 51.9, of four 43.9 / 50.9, of 64 55.6 / 52.8;
//     the same, rank 64: 64 rows of one 40.2 / 58.7, of 16 63.3 / 55.0; rank 256: 1 row
//       33.0 / 34.4, 64 rows of one 58.4 / 79.1, of four 86.0 / 63.8;
//     1024 x 2048, rank 16: 64 rows of any 12.6 / 25; rank 256: 1 row 30.0 / 17.5, 64 of
//       one 35.5 / 33.8.
//   So rows that share an adapter read it from the L2s at little cost; the few-row form
//   loses at rank 256 (a small shared product, or rows of several adapters), and at 64
//   rows of many adapters by up to 8% (rank 16) or 15% (rank 64).
constexpr int kFewRows = 64;

// Pieces of K that the few rows' h are summed in: a workgroup's loads of 128 k's
// of any rank are in flight at once.
int shrink_parts(int K) {
    const int n = K / 128;
    return n < 1 ? 1 : (n > 16 ? 16 : n);
}

// Workspace: [offsets][rows][group counts][H][dH: M x rank][sgemm's]
struct AdapterSpace {
    size_t offsets, rows, counts, h, dh, product, end;
    AdapterSpace(int M, int N, int K, int G, int rank, bool grad) {
        size_t at = 0;
        auto take = [&](size_t bytes) {
            const size_t here = at;
            at += round_up(bytes);
            return here;
        };
        offsets = take(((size_t)G + 1) * 4);
        rows = take((size_t)M * 4);
        counts = take(group_bytes(M, G));
        h = take((size_t)M * rank * 4 * (M <= kFewRows && !grad ? shrink_parts(K) : 1));
        dh = take(grad ? (size_t)M * rank * 4 : 0);
        product = take(grad || M <= 512 ? 0 : sgemm_workspace_size(M, N, K));
        end = at;
    }
};

GroupedArgs blank(int G, int R) {
    GroupedArgs a = {};
    a.G = G;
    a.R = R;
    a.alpha = 1.0f;
    return a;
}

GroupedArgs projection(int M, int N, int K, float alpha, const float *A, int lda, const float *B, int ldb, float beta,
                       float *C, int ldc) {
    GroupedArgs a = blank(1, M);
    a.N = N;
    a.K = K;
    a.alpha = alpha;
    a.beta = beta;
    a.A = A;
    a.lda = lda;
    a.B = B;
    a.ldb = ldb;
    a.C = C;
    a.ldc = ldc;
    return a;
}

// C = alpha A B + beta C: up to 512 rows on the grouped kernels, as one group (100 x
// 4096 x 4096 36 us against sgemm_ws's 42, 300 rows 94 against 98), beyond on
// sgemm's blocks (4096 x 4096 x 2048 473 against 482, 2000 x 2048 x 1024 66 against 68).
int project(int M, int N, int K, float alpha, const float *A, int lda, const float *B, int ldb, float beta, float *C,
            int ldc, void *workspace, size_t bytes, hipStream_t stream) {
    if (M > 512) return sgemm_ws(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, workspace, bytes, stream);
    return grouped(projection(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc), false, stream);
}

// H[m] = scales[g] A[m] U_g for the placed rows (trans_u: U_g rank x K)
GroupedArgs shrink(int M, int K, int G, int rank, const float *A, int lda, const float *U, int ldu,
                   long long stride_u, const float *scales, const int *offsets, const int *rows, float *H) {
    GroupedArgs a = blank(G, M);
    a.N = rank;
    a.K = K;
    a.A = A;
    a.lda = lda;
    a.a_div = 1;
    a.B = U;
    a.ldb = ldu;
    a.stride_b = stride_u;
    a.C = H;
    a.ldc = rank;
    a.c_scatter = 1;
    a.offsets = offsets;
    a.rows = rows;
    a.scales = scales;
    return a;
}

// C[m] += alpha H[m] V_g (trans_v: V_g N x rank)
GroupedArgs expand(int M, int N, int G, int rank, float alpha, const float *H, const float *V, int ldv,
                   long long stride_v, const int *ranks, const int *offsets, const int *rows, float *C, int ldc) {
    GroupedArgs a = blank(G, M);
    a.N = N;
    a.K = rank;
    a.alpha = alpha;
    a.beta = 1.0f;
    a.A = H;
    a.lda = rank;
    a.a_div = 1;
    a.B = V;
    a.ldb = ldv;
    a.stride_b = stride_v;
    a.C = C;
    a.ldc = ldc;
    a.c_scatter = 1;
    a.offsets = offsets;
    a.rows = rows;
    a.ranks = ranks;
    a.rank_k = 1;
    return a;
}

}  // namespace

int rowk::rows_product_pair(int M, int N, int K, const float *const A[2], int lda, const float *const B[2],
                            const int ldb[2], float *C, int ldc, hipStream_t stream) {
    if (M >= kMostSlots || K > kLongest) return SGEMM_ERR_TOO_LARGE;
    TwoArgs t = {projection(M, N, K, 1.0f, A[0], lda, B[0], ldb[0], 0.0f, C, ldc),
                 projection(M, N, K, 1.0f, A[1], lda, B[1], ldb[1], 1.0f, C, ldc)};
    if (M > 0 && N > 0 && K > 0 && reachable(t.first, true) && reachable(t.second, true)) {
        const Block &b = choose_block(t.first, true);
        const long long grid = grid_of(b, true, t.first);
        t.second.xcd_shift = t.first.xcd_shift;
        return enqueue(b.two, grid, b.threads, t, stream);
    }
    const int rc = grouped(t.first, true, stream);
    return rc != SGEMM_OK ? rc : grouped(t.second, true, stream);
}

extern "C" {

int sgemm_route(int T, int E, int k, int scoring, const float *logits, int ldl, const float *bias, int groups,
                int top_groups, int group_best, int renorm, float scale, int *ids, float *weights,
                hipStream_t stream) {
    NEED(1, T >= 0);
    NEED(2, E >= 1 && E <= SGEMM_ROUTE_MAX_EXPERTS);
    NEED(3, k >= 1 && k <= E && k <= SGEMM_ROUTE_MAX_K);
    NEED(4, scoring == SGEMM_SCORE_SOFTMAX || scoring == SGEMM_SCORE_SIGMOID);
    NEED(5, (T == 0 || logits != nullptr) && aligned4(logits));
    NEED(6, ldl >= E);
    NEED(7, aligned4(bias));
    NEED(8, groups >= 1 && groups <= 64 && E % groups == 0);
    NEED(9, top_groups >= 1 && top_groups <= groups);
    NEED(10, group_best == 1 || group_best == 2);
    NEED(13, (T == 0 || ids != nullptr) && aligned4(ids));
    NEED(14, (T == 0 || weights != nullptr) && aligned4(weights));
    rowk::RouteArgs a;
    a.T = T;
    a.E = E;
    a.k = k;
    a.sigmoid = scoring == SGEMM_SCORE_SIGMOID;
    a.groups = groups;
    a.top_groups = top_groups;
    a.group_best = group_best;
    a.renorm = renorm != 0;
    a.scale = scale;
    a.inv_per = 1.0f / (float)(E / groups);
    a.logits = logits;
    a.bias = bias;
    a.ldl = ldl;
    a.ids = ids;
    a.weights = weights;
    const RouteKernel &r = route_kernel(E, k);
    const bool wide = bias != nullptr || group_best == 2;  // (with one group too)
    return enqueue(wide ? r.wide : r.narrow, ceil_div(T, rowk::kRouteThreads / r.lanes), rowk::kRouteThreads, a,
                   stream);
}

int sgemm_route_grad(int T, int E, int k, int scoring, const float *logits, int ldl, int renorm, float scale,
                     const int *ids, const float *dweights, float *dlogits, int lddl, hipStream_t stream) {
    NEED(1, T >= 0);
    NEED(2, E >= 1 && E <= SGEMM_ROUTE_MAX_EXPERTS);
    NEED(3, k >= 1 && k <= E && k <= SGEMM_ROUTE_MAX_K);
    NEED(4, scoring == SGEMM_SCORE_SOFTMAX || scoring == SGEMM_SCORE_SIGMOID);
    NEED(5, (T == 0 || logits != nullptr) && aligned4(logits));
    NEED(6, ldl >= E);
    NEED(9, (T == 0 || ids != nullptr) && aligned4(ids));
    NEED(10, (T == 0 || dweights != nullptr) && aligned4(dweights));
    NEED(11, (T == 0 || dlogits != nullptr) && aligned4(dlogits));
    NEED(12, lddl >= E);
    rowk::RouteGradArgs a;
    a.T = T;
    a.E = E;
    a.k = k;
    a.sigmoid = scoring == SGEMM_SCORE_SIGMOID;
    a.renorm = renorm != 0;
    a.scale = scale;
    a.logits = logits;
    a.ldl = ldl;
    a.ids = ids;
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.lddl = lddl;
    const RouteKernel &r = route_kernel(E, k);
    return enqueue(r.grad, ceil_div(T, rowk::kRouteThreads / r.lanes), rowk::kRouteThreads, a, stream);
}

size_t sgemm_group_rows_workspace_size(int R, int G) {
    return R < 0 || G < 1 || G > SGEMM_MAX_GROUPS ? 0 : group_bytes(R, G);
}

int sgemm_group_rows(int R, int G, const int *ids, int *offsets, int *rows, void *workspace,
                     size_t workspace_bytes, hipStream_t stream) {
    NEED(1, R >= 0);
    NEED(2, G >= 1 && G <= SGEMM_MAX_GROUPS);
    NEED(3, (R == 0 || ids != nullptr) && aligned4(ids));
    NEED(4, offsets != nullptr && aligned4(offsets));
    NEED(5, (R == 0 || rows != nullptr) && aligned4(rows));
    if (!workspace_ok(workspace, workspace_bytes, group_bytes(R, G))) return SGEMM_ERR_WORKSPACE;
    return group(R, G, ids, offsets, rows, workspace, stream);
}

int sgemm_grouped(int G, int R, int N, int K, float alpha, const float *A, int lda, int a_div, const float *B,
                  int ldb, long long stride_b, int trans_b, float beta, float *C, int ldc, int c_scatter,
                  const int *offsets, const int *rows, hipStream_t stream) {
    NEED(1, G >= 0);
    NEED(2, R >= 0);
    NEED(3, N >= 0);
    NEED(4, K >= 0);
    const bool empty = G == 0 || R == 0 || N == 0;
    const bool product = !empty && K > 0 && alpha != 0.0f;
    NEED(6, (!product || A != nullptr) && aligned4(A));
    NEED(7, lda >= (K > 1 ? K : 1));
    NEED(8, a_div >= 0);
    NEED(9, (!product || B != nullptr) && aligned4(B));
    NEED(10, ldb >= (trans_b ? (K > 1 ? K : 1) : (N > 1 ? N : 1)));
    NEED(11, stride_b >= 0);
    NEED(14, (empty || C != nullptr) && aligned4(C));
    NEED(15, ldc >= (N > 1 ? N : 1));
    NEED(17, (empty || offsets != nullptr) && aligned4(offsets));
    NEED(18, (empty || rows != nullptr || (a_div == 0 && c_scatter == 0)) && aligned4(rows));
    GroupedArgs a = blank(G, R);
    a.N = N;
    a.K = K;
    a.alpha = alpha;
    a.beta = beta;
    a.A = A;
    a.lda = lda;
    a.a_div = a_div;
    a.B = B;
    a.ldb = ldb;
    a.stride_b = stride_b;
    a.C = C;
    a.ldc = ldc;
    a.c_scatter = c_scatter != 0;
    a.offsets = offsets;
    a.rows = rows;
    return grouped(a, trans_b != 0, stream);
}

int sgemm_grouped_tn(int G, int R, int M, int N, float alpha, const float *A, int lda, int a_div, const float *B,
                     int ldb, int b_div, float beta, float *C, int ldc, long long stride_c, const int *offsets,
                     const int *rows, hipStream_t stream) {
    NEED(1, G >= 0);
    NEED(2, R >= 0);
    NEED(3, M >= 0);
    NEED(4, N >= 0);
    const bool empty = G == 0 || M == 0 || N == 0;
    const bool product = !empty && R > 0 && alpha != 0.0f;
    NEED(6, (!product || A != nullptr) && aligned4(A));
    NEED(7, lda >= (M > 1 ? M : 1));
    NEED(8, a_div >= 0);
    NEED(9, (!product || B != nullptr) && aligned4(B));
    NEED(10, ldb >= (N > 1 ? N : 1));
    NEED(11, b_div >= 0);
    NEED(13, (empty || C != nullptr) && aligned4(C));
    NEED(14, ldc >= (N > 1 ? N : 1));
    NEED(15, G <= 1 || empty || stride_c >= (long long)(M - 1) * ldc + N);
    NEED(16, (!product || offsets != nullptr) && aligned4(offsets));
    NEED(17, (!product || rows != nullptr || (a_div == 0 && b_div == 0)) && aligned4(rows));
    GroupedArgs a = blank(G, R);
    a.M = M;
    a.N = N;
    a.alpha = alpha;
    a.beta = beta;
    a.A = A;
    a.lda = lda;
    a.a_div = a_div;
    a.B = B;
    a.ldb = ldb;
    a.b_div = b_div;
    a.C = C;
    a.ldc = ldc;
    a.stride_c = stride_c;
    a.offsets = offsets;
    a.rows = rows;
    if (!product) a.R = 0;  // offsets may be NULL: one empty group each
    return grouped_tn(a, stream);
}

int sgemm_combine(int T, int k, int N, int E, const int *ids, const float *weights, const float *Y, int ldy,
                  float beta, float *out, int ldo, hipStream_t stream) {
    NEED(1, T >= 0);
    NEED(2, k >= 1 && k <= SGEMM_ROUTE_MAX_K);
    NEED(3, N >= 0);
    NEED(4, E >= 0);
    const bool empty = T == 0 || N == 0;
    NEED(5, aligned4(ids));
    NEED(6, aligned4(weights));
    NEED(7, (empty || Y != nullptr) && aligned4(Y));
    NEED(8, ldy >= (N > 1 ? N : 1));
    NEED(10, (empty || out != nullptr) && aligned4(out));
    NEED(11, ldo >= (N > 1 ? N : 1));
    if (empty) return SGEMM_OK;
    rowk::CombineArgs a;
    a.T = T;
    a.k = k;
    a.N = N;
    a.E = E;
    a.ids = ids;
    a.weights = weights;
    a.Y = Y;
    a.ldy = ldy;
    a.ldo = ldo;
    a.beta = beta;
    a.out = out;
    a.chunks = (int)ceil_div(N, 256);
    a.units = (int64_t)T * a.chunks;
    return enqueue(rowk::combine, ceil_div(a.units, 4), 256, a, stream);
}

int sgemm_combine_grad(int T, int k, int N, int E, const int *ids, const float *weights, const float *dout,
                       int ldd, const float *Y, int ldy, float *dY, int lddy, float *dweights,
                       hipStream_t stream) {
    NEED(1, T >= 0);
    NEED(2, k >= 1 && k <= SGEMM_ROUTE_MAX_K);
    NEED(3, N >= 0);
    NEED(4, E >= 0);
    const bool empty = T == 0 || N == 0;
    NEED(5, aligned4(ids));
    NEED(6, aligned4(weights));
    NEED(7, (empty || dout != nullptr) && aligned4(dout));
    NEED(8, ldd >= (N > 1 ? N : 1));
    NEED(9, (empty || dweights == nullptr || Y != nullptr) && aligned4(Y));
    NEED(10, ldy >= (N > 1 ? N : 1));
    NEED(11, aligned4(dY));
    NEED(12, lddy >= (N > 1 ? N : 1));
    NEED(13, aligned4(dweights));
    if (T == 0 || (dweights == nullptr && (dY == nullptr || N == 0))) return SGEMM_OK;
    if (N > kLongest) return SGEMM_ERR_TOO_LARGE;
    rowk::CombineGradArgs a;
    a.T = T;
    a.k = k;
    a.N = N;
    a.E = E;
    a.ids = ids;
    a.weights = weights;
    a.dout = dout;
    a.ldd = ldd;
    a.Y = Y;
    a.ldy = ldy;
    a.dY = dY;
    a.lddy = lddy;
    a.dweights = dweights;
    return enqueue(rowk::combine_grad, T, 256, a, stream);
}

size_t sgemm_adapters_workspace_size(int M, int N, int K, int G, int rank) {
    if (M < 0 || N < 0 || K < 0 || G < 1 || G > SGEMM_MAX_GROUPS || rank < 1 || rank > SGEMM_MAX_RANK) return 0;
    return AdapterSpace(M, N, K, G, rank, false).end;
}

size_t sgemm_adapters_grad_workspace_size(int M, int N, int K, int G, int rank) {
    if (M < 0 || N < 0 || K < 0 || G < 1 || G > SGEMM_MAX_GROUPS || rank < 1 || rank > SGEMM_MAX_RANK) return 0;
    // (at least the forward's, so that a training step keeps one workspace)
    const size_t forward = AdapterSpace(M, N, K, G, rank, false).end, back = AdapterSpace(M, N, K, G, rank, true).end;
    return forward > back ? forward : back;
}

int sgemm_adapters(int M, int N, int K, float alpha, const float *A, int lda, const float *B, int ldb, float beta,
                   float *C, int ldc, int G, int rank, const int *ids, const int *ranks, const float *scales,
                   const float *U, int ldu, long long stride_u, const float *V, int ldv, long long stride_v,
                   void *workspace, size_t workspace_bytes, hipStream_t stream) {
    NEED(1, M >= 0);
    NEED(2, N >= 0);
    NEED(3, K >= 0);
    const bool empty = M == 0 || N == 0;
    const bool product = !empty && K > 0 && alpha != 0.0f;
    NEED(5, (!product || A != nullptr) && aligned4(A));
    NEED(6, lda >= (K > 1 ? K : 1));
    NEED(7, (!product || B != nullptr) && aligned4(B));
    NEED(8, ldb >= (N > 1 ? N : 1));
    NEED(10, (empty || C != nullptr) && aligned4(C));
    NEED(11, ldc >= (N > 1 ? N : 1));
    NEED(12, G >= 1 && G <= SGEMM_MAX_GROUPS);
    NEED(13, rank >= 1 && rank <= SGEMM_MAX_RANK);
    NEED(14, (!product || ids != nullptr) && aligned4(ids));
    NEED(15, aligned4(ranks));
    NEED(16, aligned4(scales));
    NEED(17, (!product || U != nullptr) && aligned4(U));
    NEED(18, ldu >= rank);
    NEED(19, stride_u >= 0);
    NEED(20, (!product || V != nullptr) && aligned4(V));
    NEED(21, ldv >= (N > 1 ? N : 1));
    NEED(22, stride_v >= 0);
    const AdapterSpace at(M, N, K, G, rank, false);
    if (!workspace_ok(workspace, workspace_bytes, at.end)) return SGEMM_ERR_WORKSPACE;
    if (!product) return sgemm(M, N, K, 0.0f, A, lda, B, ldb, beta, C, ldc, stream);
    if (M >= kMostSlots || K > kLongest) return SGEMM_ERR_TOO_LARGE;  // before anything is written
    char *w = static_cast<char *>(workspace);
    int *offsets = reinterpret_cast<int *>(w + at.offsets), *rows = reinterpret_cast<int *>(w + at.rows);
    float *H = reinterpret_cast<float *>(w + at.h);
    int rc;
    rowk::PairArgs p;
    p.product = projection(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc);
    // (a piece of U within 32-bit offsets, with the steps that overrun its end)
    if (M <= kFewRows && ceil_div(K, shrink_parts(K)) + 8 * 256 <= kReach / 4 / ldu && reachable(p.product, false)) {
        rowk::ShrinkArgs &h = p.shrink;
        h.M = M;
        h.K = K;
        h.G = G;
        h.rank = rank;
        h.parts = shrink_parts(K);
        h.A = A;
        h.U = U;
        h.lda = lda;
        h.ldu = ldu;
        h.stride_u = stride_u;
        h.ids = ids;
        h.ranks = ranks;
        h.H = H;
        p.ahead = (int)(ceil_div(M * h.parts, 8) * 8);
        const Block &b = K <= 64 ? kNarrow : choose_block(p.product, false);
        const long long grid = p.ahead + grid_of(b, true, p.product);
        rc = enqueue(b.pair, grid, b.threads, p, stream);
        if (rc != SGEMM_OK) return rc;
        rowk::ExpandArgs e;
        e.M = M;
        e.N = N;
        e.G = G;
        e.rank = rank;
        e.parts = h.parts;
        e.chunks = (int)ceil_div(N, 256);
        e.alpha = alpha;
        e.H = H;
        e.V = V;
        e.scales = scales;
        e.ldv = ldv;
        e.stride_v = stride_v;
        e.ldc = ldc;
        e.ids = ids;
        e.ranks = ranks;
        e.C = C;
        return enqueue(rowk::expand_rows, (long long)M * e.chunks, 64, e, stream);
    }
    rc = group(M, G, ids, offsets, rows, w + at.counts, stream);
    if (rc == SGEMM_OK)
        rc = grouped(shrink(M, K, G, rank, A, lda, U, ldu, stride_u, scales, offsets, rows, H), false, stream);
    if (rc == SGEMM_OK)
        rc = project(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, w + at.product, at.end - at.product, stream);
    if (rc == SGEMM_OK)
        rc = grouped(expand(M, N, G, rank, alpha, H, V, ldv, stride_v, ranks, offsets, rows, C, ldc), false, stream);
    return rc;
}

int sgemm_adapters_grad(int M, int N, int K, float alpha, const float *A, int lda, const float *B, int ldb,
                        const float *dC, int lddc, int G, int rank, const int *ids, const int *ranks,
                        const float *scales, const float *U, int ldu, long long stride_u, const float *V, int ldv,
                        long long stride_v, float beta, float *dA, int ldda, float *dU, int lddu,
                        long long stride_du, float *dV, int lddv, long long stride_dv, void *workspace,
                        size_t workspace_bytes, hipStream_t stream) {
    NEED(1, M >= 0);
    NEED(2, N >= 0);
    NEED(3, K >= 0);
    const bool product = M > 0 && alpha != 0.0f;
    const bool adapters = dU != nullptr || dV != nullptr;
    NEED(5, (!product || K == 0 || !adapters || A != nullptr) && aligned4(A));
    NEED(6, lda >= (K > 1 ? K : 1));
    NEED(7, (!product || K == 0 || N == 0 || dA == nullptr || B != nullptr) && aligned4(B));
    NEED(8, ldb >= (N > 1 ? N : 1));
    NEED(9, (!product || N == 0 || dC != nullptr) && aligned4(dC));
    NEED(10, lddc >= (N > 1 ? N : 1));
    NEED(11, G >= 1 && G <= SGEMM_MAX_GROUPS);
    NEED(12, rank >= 1 && rank <= SGEMM_MAX_RANK);
    NEED(13, (!product || ids != nullptr) && aligned4(ids));
    NEED(14, aligned4(ranks));
    NEED(15, aligned4(scales));
    NEED(16, (!product || K == 0 || U != nullptr) && aligned4(U));
    NEED(17, ldu >= rank);
    NEED(18, stride_u >= 0);
    NEED(19, (!product || N == 0 || V != nullptr) && aligned4(V));
    NEED(20, ldv >= (N > 1 ? N : 1));
    NEED(21, stride_v >= 0);
    NEED(23, aligned4(dA));
    NEED(24, ldda >= (K > 1 ? K : 1));
    NEED(25, (dU != nullptr || dV == nullptr) && aligned4(dU));
    NEED(26, lddu >= rank);
    NEED(27, G == 1 || K == 0 || stride_du >= (long long)(K - 1) * lddu + rank);
    NEED(28, (dV != nullptr || dU == nullptr) && aligned4(dV));
    NEED(29, lddv >= (N > 1 ? N : 1));
    NEED(30, G == 1 || N == 0 || stride_dv >= (long long)(rank - 1) * lddv + N);
    const AdapterSpace at(M, N, K, G, rank, true);
    if (!workspace_ok(workspace, workspace_bytes, sgemm_adapters_grad_workspace_size(M, N, K, G, rank)))
        return SGEMM_ERR_WORKSPACE;
    if (product && (M >= kMostSlots || N > kLongest || K > kLongest)) return SGEMM_ERR_TOO_LARGE;
    char *w = static_cast<char *>(workspace);
    int *offsets = reinterpret_cast<int *>(w + at.offsets), *rows = reinterpret_cast<int *>(w + at.rows);
    float *H = reinterpret_cast<float *>(w + at.h), *dH = reinterpret_cast<float *>(w + at.dh);
    int rc = SGEMM_OK;
    if (product) {
        rc = group(M, G, ids, offsets, rows, w + at.counts, stream);
        if (rc == SGEMM_OK)  // dH[m] = scale dC[m] V_g^T
            rc = grouped(shrink(M, N, G, rank, dC, lddc, V, ldv, stride_v, scales, offsets, rows, dH), true, stream);
    }
    if (rc == SGEMM_OK && dA != nullptr) {
        GroupedArgs a = blank(1, M);
        a.N = K;
        a.K = N;
        a.alpha = alpha;
        a.A = dC;
        a.lda = lddc;
        a.B = B;
        a.ldb = ldb;
        a.C = dA;
        a.ldc = ldda;
        rc = grouped(a, true, stream);
        if (rc == SGEMM_OK && product)
            rc = grouped(expand(M, K, G, rank, alpha, dH, U, ldu, stride_u, ranks, offsets, rows, dA, ldda), true,
                         stream);
    }
    if (rc == SGEMM_OK && adapters) {
        GroupedArgs a = blank(G, product ? M : 0);  // dU_g = alpha A^T dH
        a.M = K;
        a.N = rank;
        a.alpha = alpha;
        a.beta = beta;
        a.A = A;
        a.lda = lda;
        a.a_div = 1;
        a.B = dH;
        a.ldb = rank;
        a.b_div = 1;
        a.C = dU;
        a.ldc = lddu;
        a.stride_c = stride_du;
        a.offsets = product ? offsets : nullptr;
        a.rows = rows;
        a.ranks = ranks;
        a.rank_n = 1;
        rc = grouped_tn(a, stream);
        if (rc == SGEMM_OK && product)
            rc = grouped(shrink(M, K, G, rank, A, lda, U, ldu, stride_u, scales, offsets, rows, H), false, stream);
        if (rc == SGEMM_OK) {  // dV_g = alpha H^T dC
            GroupedArgs b = a;
            b.M = rank;
            b.N = N;
            b.A = H;
            b.lda = rank;
            b.B = dC;
            b.ldb = lddc;
            b.C = dV;
            b.ldc = lddv;
            b.stride_c = stride_dv;
            b.rank_n = 0;
            b.rank_m = 1;
            rc = grouped_tn(b, stream);
        }
    }
    return rc;
}

}  // extern "C"
