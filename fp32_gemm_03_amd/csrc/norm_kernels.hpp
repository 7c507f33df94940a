// norm_kernels.hpp -- kernels of the row operators of a feed-forward block: the
// root-mean-square norm with the residual's addition, its gradient, and rows to
// 8 bits with a scale each.
//
// All are bound by the bytes they move, so a row is read once and held in
// registers (NT threads, V vectors of four floats each), and what is summed or
// rounded is computed in 64 bits: the row's sum of squares, the factor
// (mean + eps)^-1/2, and the product that goes to the nearest whole number, where
// 32 bits would send values next to a border to the wrong one.
#pragma once

#include "activations.hpp"
#include "lanes.hpp"

namespace normk {

using rowk::f32x4u;
using rowk::reduce;
using rowk::rsrc_t;
using rowk::whole_rsrc;
using sgk::f32x4;

// ---------------------------------------------------------------------------
// Sums and maxima over the NT threads of a row.  `slot` is LDS of the kernel's
// own, one value per wave; the barriers on both sides let it be used again.
// ---------------------------------------------------------------------------
template <int NT, class T, class Op> __device__ __forceinline__ T over_row(T v, Op op, T *slot) {
    v = reduce<64>(v, op);
    if constexpr (NT > 64) {
        constexpr int W = NT / 64;
        const int w = threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) slot[w] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int i = 1; i < W; ++i) v = op(v, slot[i]);
    }
    return v;
}
struct MaxInt {
    __device__ __forceinline__ int operator()(int a, int b) const { return a > b ? a : b; }
};

// Magnitudes are compared as their bits: a NaN is above infinity, so a row's
// maximum tells whether it holds either.
__device__ __forceinline__ int magnitude(float v) { return __float_as_int(v) & 0x7fffffff; }

// 8-bit rows: scale a / 127 and q = nearest even of v (127 (1 / a)), each operation
// rounded to 64 bits (half of a is 63.5 steps give or take a rounding, so the order is
// part of the definition).  A row of zeros has scale 0; one that holds a NaN or an
// infinity scale NaN and whole numbers 0.
__device__ __forceinline__ double steps_per(int most) {
    return most > 0 && most < 0x7f800000 ? 127.0 * (1.0 / (double)__int_as_float(most)) : 0.0;
}
__device__ __forceinline__ float scale_of(int most) {
    return most < 0x7f800000 ? (float)((double)__int_as_float(most) / 127.0) : __int_as_float(0x7fc00000);
}
// |v per| <= 127 (1 + 2^-52): adding 1.5 2^52 leaves the rounded whole number in the low
// bits.  The product is rounded before: as one instruction, 63.5 steps would be taken
// for a little more or less.
__device__ __forceinline__ int whole(float v, double per, bool finite) {
#pragma clang fp contract(off)
    const double steps = (double)v * per;
    const double x = steps + 6755399441055744.0;
    return finite ? __double2loint(x) & 0xff : 0;
}
__device__ __forceinline__ void store_whole(signed char *q, int left, f32x4u v, double per, bool finite) {
    const int b0 = whole(v.x, per, finite), b1 = whole(v.y, per, finite);
    const int b2 = whole(v.z, per, finite), b3 = whole(v.w, per, finite);
    if (left >= 4) {
        const int p = b0 | b1 << 8 | b2 << 16 | b3 << 24;
        __builtin_memcpy(q, &p, 4);  // (any alignment)
    } else {
        if (left > 0) q[0] = (signed char)b0;
        if (left > 1) q[1] = (signed char)b1;
        if (left > 2) q[2] = (signed char)b2;
    }
}

__device__ __forceinline__ f32x4u row4(rsrc_t r, uint32_t i) {
    const f32x4 v = sgk::raw_load_v4f32(r, 4u * i, 0, 0);
    f32x4u u;
    u.x = v.x;
    u.y = v.y;
    u.z = v.z;
    u.w = v.w;
    return u;
}
// columns i.. of a row of N, where the row goes on so far
__device__ __forceinline__ void put4(float *row, int i, int N, f32x4u v) {
    if (i < N) rowk::store4(row + i, N - i, v);
}

// ---------------------------------------------------------------------------
// h = x + residual; y = h (mean h^2 + eps)^-1/2 weight; y to 8 bits.
// NT threads hold a row of up to 4 NT V columns; of rows of one wave a workgroup takes four.
// Bound by HBM: x, residual, sum and q of 4095 x 4096 are 218 MB in 41 us, 5.3 TB/s (a copy
// reaches 4.9; part of sum stays in the last-level cache).  One row: the launch, 3.2 us.
// ---------------------------------------------------------------------------
struct NormArgs {
    int T, N;
    double eps;
    const float *x, *residual, *weight;
    int64_t ldx, ldr;
    float *sum, *y, *scales;
    int64_t lds, ldy, ldq;
    signed char *q;
};

__device__ __forceinline__ float normed(float h, double r, float w, bool weighted) {
    const double v = (double)h * r;
    return (float)(weighted ? v * (double)w : v);
}

template <int NT, int V> __global__ void __launch_bounds__(NT == 64 ? 256 : NT) norm(NormArgs a) {
    constexpr int ROWS = NT == 64 ? 4 : 1;  // a wave each, or one of the workgroup
    __shared__ double sums[NT / 64 > 0 ? NT / 64 : 1];
    __shared__ int mosts[NT / 64 > 0 ? NT / 64 : 1];
    const int tid = threadIdx.x % NT;
    const int64_t t = __builtin_amdgcn_readfirstlane((int)blockIdx.x * ROWS + (int)threadIdx.x / NT);
    if (t >= a.T) return;  // (a whole wave, and with more than one wave a row never)
    const int64_t bytes = 4 * (int64_t)a.N;
    const rsrc_t rx = whole_rsrc(a.x + t * a.ldx, bytes);
    const rsrc_t rr = whole_rsrc(a.residual + t * a.ldr, a.residual != nullptr ? bytes : 0);
    const rsrc_t rw = whole_rsrc(a.weight, a.weight != nullptr ? bytes : 0);
    f32x4u v[V], w[V];
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] = row4(rx, 4 * (c * NT + tid));
    if (a.residual != nullptr) {
        f32x4u u[V];
#pragma unroll
        for (int c = 0; c < V; ++c) u[c] = row4(rr, 4 * (c * NT + tid));
#pragma unroll
        for (int c = 0; c < V; ++c) {
            v[c].x += u[c].x;
            v[c].y += u[c].y;
            v[c].z += u[c].z;
            v[c].w += u[c].w;
        }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) w[c] = row4(rw, 4 * (c * NT + tid));
    if (a.sum != nullptr) {
#pragma unroll
        for (int c = 0; c < V; ++c) put4(a.sum + t * a.lds, 4 * (c * NT + tid), a.N, v[c]);
    }
    if (a.y == nullptr && a.q == nullptr) return;
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        s = fma((double)v[c].x, (double)v[c].x, s);
        s = fma((double)v[c].y, (double)v[c].y, s);
        s = fma((double)v[c].z, (double)v[c].z, s);
        s = fma((double)v[c].w, (double)v[c].w, s);
    }
    s = over_row<NT>(s, rowk::Add(), sums);
    const double r = 1.0 / sqrt(s / (double)a.N + a.eps);
    const bool weighted = a.weight != nullptr;
    int most = 0;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        v[c].x = normed(v[c].x, r, w[c].x, weighted);
        v[c].y = normed(v[c].y, r, w[c].y, weighted);
        v[c].z = normed(v[c].z, r, w[c].z, weighted);
        v[c].w = normed(v[c].w, r, w[c].w, weighted);
    }
    if (a.y != nullptr) {
#pragma unroll
        for (int c = 0; c < V; ++c) put4(a.y + t * a.ldy, 4 * (c * NT + tid), a.N, v[c]);
    }
    if (a.q == nullptr) return;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int left = a.N - 4 * (c * NT + tid);  // (columns beyond the row are 0 * r, NaN where r is)
        MaxInt m;
        if (left > 0) most = m(most, magnitude(v[c].x));
        if (left > 1) most = m(most, magnitude(v[c].y));
        if (left > 2) most = m(most, magnitude(v[c].z));
        if (left > 3) most = m(most, magnitude(v[c].w));
    }
    most = over_row<NT>(most, MaxInt(), mosts);
    const double per = steps_per(most);
    const bool finite = most < 0x7f800000;
    if (tid == 0) a.scales[t] = scale_of(most);
    signed char *q = a.q + t * a.ldq;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int i = 4 * (c * NT + tid);
        if (i < a.N) store_whole(q + i, a.N - i, v[c], per, finite);
    }
}

// Rows too long for registers: the row is read again for its maximum and again for
// what is written.  After the first pass h is read from `sum` where that is given
// (it may be x's or residual's own place); a thread reads what it wrote.
constexpr int kLongThreads = 1024;

template <class Load> __device__ __forceinline__ void each(int N, Load f) {
    for (int64_t i = 4 * (int64_t)threadIdx.x; i < N; i += 4 * kLongThreads) f((int)i);
}

__global__ void __launch_bounds__(kLongThreads) norm_long(NormArgs a) {
    __shared__ double sums[kLongThreads / 64];
    __shared__ int mosts[kLongThreads / 64];
    const int64_t t = blockIdx.x;
    const float *x = a.x + t * a.ldx, *residual = a.residual == nullptr ? nullptr : a.residual + t * a.ldr;
    float *sum = a.sum == nullptr ? nullptr : a.sum + t * a.lds;
    const bool weighted = a.weight != nullptr;
    auto row = [&](int i, bool first) {
        const int left = a.N - i;
        if (!first && sum != nullptr) return rowk::load4(sum + i, left);
        f32x4u v = rowk::load4(x + i, left);
        if (residual != nullptr) {
            const f32x4u u = rowk::load4(residual + i, left);
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
        return v;
    };
    double s = 0.0;
    each(a.N, [&](int i) {
        const f32x4u v = row(i, true);
        if (sum != nullptr) rowk::store4(sum + i, a.N - i, v);
        s = fma((double)v.x, (double)v.x, s);
        s = fma((double)v.y, (double)v.y, s);
        s = fma((double)v.z, (double)v.z, s);
        s = fma((double)v.w, (double)v.w, s);
    });
    if (a.y == nullptr && a.q == nullptr) return;
    s = over_row<kLongThreads>(s, rowk::Add(), sums);
    const double r = 1.0 / sqrt(s / (double)a.N + a.eps);
    auto result = [&](int i) {
        f32x4u v = row(i, false), w = {};
        if (weighted) w = rowk::load4(a.weight + i, a.N - i);
        v.x = normed(v.x, r, w.x, weighted);
        v.y = normed(v.y, r, w.y, weighted);
        v.z = normed(v.z, r, w.z, weighted);
        v.w = normed(v.w, r, w.w, weighted);
        return v;
    };
    double per = 0.0;
    bool finite = true;
    if (a.q != nullptr) {
        int most = 0;
        each(a.N, [&](int i) {
            const f32x4u v = result(i);
            const int left = a.N - i;
            MaxInt m;
            most = m(most, magnitude(v.x));
            if (left > 1) most = m(most, magnitude(v.y));
            if (left > 2) most = m(most, magnitude(v.z));
            if (left > 3) most = m(most, magnitude(v.w));
        });
        most = over_row<kLongThreads>(most, MaxInt(), mosts);
        per = steps_per(most);
        finite = most < 0x7f800000;
        if (threadIdx.x == 0) a.scales[t] = scale_of(most);
    }
    each(a.N, [&](int i) {
        const f32x4u v = result(i);
        if (a.y != nullptr) rowk::store4(a.y + t * a.ldy + i, a.N - i, v);
        if (a.q != nullptr) store_whole(a.q + t * a.ldq + i, a.N - i, v, per, finite);
    });
}

// ---------------------------------------------------------------------------
// Rows to 8 bits, v = x or act(gate) x rounded to 32 bits.
// ---------------------------------------------------------------------------
struct QuantArgs {
    int T, N;
    const float *x, *gate;
    int64_t ldx, ldg, ldq;
    signed char *q;
    float *scales;
};

template <int ACT> __device__ __forceinline__ float gated64(float g, float x) {
    return (float)(act<ACT>((double)g) * (double)x);
}
template <int ACT> __device__ __forceinline__ f32x4u gated64(f32x4u g, f32x4u x) {
    f32x4u v;
    v.x = gated64<ACT>(g.x, x.x);
    v.y = gated64<ACT>(g.y, x.y);
    v.z = gated64<ACT>(g.z, x.z);
    v.w = gated64<ACT>(g.w, x.w);
    return v;
}

// ACT < 0: no gate.  2047 x 4096: 7.7 to 8.3 us without one (42 MB, 5 TB/s), behind SiLU and the
// tanh form 17 to 21 (75 MB, 4 TB/s; the 64-bit exponential), GELU 30 to 35 (the library's 64-bit
// erfc).  A row of 4095 3.3 us.
template <int NT, int V, int ACT> __global__ void __launch_bounds__(NT == 64 ? 256 : NT) quantize(QuantArgs a) {
    constexpr int ROWS = NT == 64 ? 4 : 1;  // a wave each, or one of the workgroup
    __shared__ int mosts[NT / 64 > 0 ? NT / 64 : 1];
    const int tid = threadIdx.x % NT;
    const int64_t t = __builtin_amdgcn_readfirstlane((int)blockIdx.x * ROWS + (int)threadIdx.x / NT);
    if (t >= a.T) return;
    const int64_t bytes = 4 * (int64_t)a.N;
    const rsrc_t rx = whole_rsrc(a.x + t * a.ldx, bytes);
    f32x4u v[V];
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] = row4(rx, 4 * (c * NT + tid));
    if constexpr (ACT >= 0) {
        const rsrc_t rg = whole_rsrc(a.gate + t * a.ldg, bytes);
        f32x4u g[V];
#pragma unroll
        for (int c = 0; c < V; ++c) g[c] = row4(rg, 4 * (c * NT + tid));
#pragma unroll
        for (int c = 0; c < V; ++c) {
            // (a wave wholly beyond the row has nothing to compute: 515 x 2816, 8 waves of two
            // vectors, 6.9 us with that and 6.0 without)
            if (c == 0 || __builtin_amdgcn_readfirstlane(4 * (c * NT + tid)) < a.N) v[c] = gated64<ACT>(g[c], v[c]);
        }
    }
    int most = 0;  // (what lies beyond the row is read as 0, and act(0) 0 is 0)
#pragma unroll
    for (int c = 0; c < V; ++c) {
        MaxInt m;
        most = m(m(m(most, magnitude(v[c].x)), m(magnitude(v[c].y), magnitude(v[c].z))), magnitude(v[c].w));
    }
    most = over_row<NT>(most, MaxInt(), mosts);
    const double per = steps_per(most);
    const bool finite = most < 0x7f800000;
    if (tid == 0) a.scales[t] = scale_of(most);
    signed char *q = a.q + t * a.ldq;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int i = 4 * (c * NT + tid);
        if (i < a.N) store_whole(q + i, a.N - i, v[c], per, finite);
    }
}

template <int ACT> __global__ void __launch_bounds__(kLongThreads) quantize_long(QuantArgs a) {
    __shared__ int mosts[kLongThreads / 64];
    const int64_t t = blockIdx.x;
    auto result = [&](int i) {
        f32x4u v = rowk::load4(a.x + t * a.ldx + i, a.N - i);
        if constexpr (ACT >= 0) v = gated64<ACT>(rowk::load4(a.gate + t * a.ldg + i, a.N - i), v);
        return v;
    };
    int most = 0;
    each(a.N, [&](int i) {
        const f32x4u v = result(i);
        MaxInt m;
        most = m(m(m(most, magnitude(v.x)), m(magnitude(v.y), magnitude(v.z))), magnitude(v.w));
    });
    most = over_row<kLongThreads>(most, MaxInt(), mosts);
    const double per = steps_per(most);
    const bool finite = most < 0x7f800000;
    if (threadIdx.x == 0) a.scales[t] = scale_of(most);
    each(a.N, [&](int i) { store_whole(a.q + t * a.ldq + i, a.N - i, result(i), per, finite); });
}

// ---------------------------------------------------------------------------
// The norm's gradient.  With g = weight dy and r = (mean h^2 + eps)^-1/2:
//   dh = r (g - h r^2 mean(g h)) + dsum,   dweight_n = sum_t dy h r.
// A workgroup takes every P-th row and sums its share of dweight in 64 bits, in registers or,
// of rows too long for them, in the workspace; the P shares are added up in order by `norm_weight_grad`.  Bound by HBM:
// 2011 x 2048 with dsum, 66 MB and 4 of shares, 12.6 us, then 3.8 for the shares.
// ---------------------------------------------------------------------------
struct NormGradArgs {
    int T, N, P;
    double eps;
    const float *h, *weight, *dy, *dsum;
    int64_t ldh, lddy, ldds, lddh;
    float *dh, *dweight;
    void *part;  // P shares of dweight: float, in norm_grad_long_shares double
    float beta;
    bool stream;  // dh is larger than the caches (norm_grad_long)
};

__device__ __forceinline__ float norm_back(float h, float dy, float w, float ds, double r, double c) {
    return (float)(fma(r, (double)dy * (double)w - (double)h * c, (double)ds));
}

template <int NT, int V> __global__ void __launch_bounds__(NT) norm_grad(NormGradArgs a) {
    __shared__ double sums[2][NT / 64];
    const int tid = threadIdx.x;
    const int64_t bytes = 4 * (int64_t)a.N;
    const rsrc_t rw = whole_rsrc(a.weight, a.weight != nullptr ? bytes : 0);
    f32x4u w[V];
    double dw[V][4];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        w[c] = row4(rw, 4 * (c * NT + tid));
        if (a.weight == nullptr) w[c] = f32x4u{1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[c][e] = 0.0;
    }
    for (int64_t t = blockIdx.x; t < a.T; t += a.P) {
        const rsrc_t rh = whole_rsrc(a.h + t * a.ldh, bytes), rd = whole_rsrc(a.dy + t * a.lddy, bytes);
        const rsrc_t rs = whole_rsrc(a.dsum + t * a.ldds, a.dsum != nullptr ? bytes : 0);
        f32x4u h[V], d[V], ds[V];
#pragma unroll
        for (int c = 0; c < V; ++c) h[c] = row4(rh, 4 * (c * NT + tid));
#pragma unroll
        for (int c = 0; c < V; ++c) d[c] = row4(rd, 4 * (c * NT + tid));
#pragma unroll
        for (int c = 0; c < V; ++c) ds[c] = row4(rs, 4 * (c * NT + tid));
        double s = 0.0, m = 0.0;
#pragma unroll
        for (int c = 0; c < V; ++c) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const double x = (double)h[c][e];
                s = fma(x, x, s);
                m = fma((double)d[c][e] * (double)w[c][e], x, m);
            }
        }
        s = over_row<NT>(s, rowk::Add(), sums[0]);
        m = over_row<NT>(m, rowk::Add(), sums[1]);
        const double r = 1.0 / sqrt(s / (double)a.N + a.eps);
        const double k = r * r * (m / (double)a.N);
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dw[c][e] = fma((double)d[c][e] * r, (double)h[c][e], dw[c][e]);
                h[c][e] = norm_back(h[c][e], d[c][e], w[c][e], ds[c][e], r, k);
            }
        if (a.dh != nullptr) {
#pragma unroll
            for (int c = 0; c < V; ++c) put4(a.dh + t * a.lddh, 4 * (c * NT + tid), a.N, h[c]);
        }
    }
    if (a.part == nullptr) return;
#pragma unroll
    for (int c = 0; c < V; ++c)
        put4(static_cast<float *>(a.part) + (int64_t)blockIdx.x * a.N, 4 * (c * NT + tid), a.N,
             f32x4u{(float)dw[c][0], (float)dw[c][1], (float)dw[c][2], (float)dw[c][3]});
}

// Rows too long for registers: a row is read twice.  For dh, and for shares of dweight that
// are one row each (P >= T).  The stores of a large dh go past the caches, which leaves them to
// the rows' second reading (dh alone, us; so, and not: 2000 x 40003 321, 341; 2048 x 65536 522, 573; 4096 x
// 16384 228, 239; of a smaller dh no difference, and what reads it next finds it there).
__global__ void __launch_bounds__(kLongThreads) norm_grad_long(NormGradArgs a) {
    __shared__ double sums[2][kLongThreads / 64];
    float *part = a.part == nullptr ? nullptr : static_cast<float *>(a.part) + (int64_t)blockIdx.x * a.N;
    for (int64_t t = blockIdx.x; t < a.T; t += a.P) {
        const float *h = a.h + t * a.ldh, *d = a.dy + t * a.lddy;
        auto weight = [&](int i) {
            return a.weight == nullptr ? f32x4u{1.0f, 1.0f, 1.0f, 1.0f} : rowk::load4(a.weight + i, a.N - i);
        };
        double s = 0.0, m = 0.0;
        each(a.N, [&](int i) {
            const f32x4u x = rowk::load4(h + i, a.N - i), y = rowk::load4(d + i, a.N - i), w = weight(i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s = fma((double)x[e], (double)x[e], s);
                m = fma((double)y[e] * (double)w[e], (double)x[e], m);
            }
        });
        s = over_row<kLongThreads>(s, rowk::Add(), sums[0]);
        m = over_row<kLongThreads>(m, rowk::Add(), sums[1]);
        const double r = 1.0 / sqrt(s / (double)a.N + a.eps);
        const double k = r * r * (m / (double)a.N);
        each(a.N, [&](int i) {
            const int left = a.N - i;
            const f32x4u x = rowk::load4(h + i, left), y = rowk::load4(d + i, left), w = weight(i);
            f32x4u ds = {0.0f, 0.0f, 0.0f, 0.0f}, p, o;
            if (a.dsum != nullptr) ds = rowk::load4(a.dsum + t * a.ldds + i, left);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[e] = (float)((double)y[e] * r * (double)x[e]);
                o[e] = norm_back(x[e], y[e], w[e], ds[e], r, k);
            }
            if (part != nullptr) rowk::store4(part + i, left, p);
            if (a.dh != nullptr) {
                float *to = a.dh + t * a.lddh + i;
                if (a.stream && left >= 4) __builtin_nontemporal_store(o, reinterpret_cast<f32x4u *>(to));
                else rowk::store4(to, left, o);
            }
        });
    }
}

// The same with several rows in a share of dweight, which is summed in its place in the
// workspace, in 64 bits: eight rows at a time, so that a share is read and written once for
// them, their factors in LDS.  Measured (us, with dh and dsum; so, one row at a time, two, four):
// 4096 x 16384 327, 413, 347, 316; 2000 x 40003 436, 639, 519, 454; 1100 x 8195 50, 61, 57, 55; 8192 x
// 12288 459, 597, 500, 437.
typedef double f64x2u __attribute__((ext_vector_type(2), aligned(8)));
__device__ __forceinline__ void get_share(const double *p, int left, double (&v)[4]) {
    if (left >= 4) {
        const f64x2u a = *reinterpret_cast<const f64x2u *>(p), b = *reinterpret_cast<const f64x2u *>(p + 2);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
        if (left > 0) v[0] = p[0];
        if (left > 1) v[1] = p[1];
        if (left > 2) v[2] = p[2];
    }
}
__device__ __forceinline__ void put_share(double *p, int left, const double (&v)[4]) {
    if (left >= 4) {
        *reinterpret_cast<f64x2u *>(p) = f64x2u{v[0], v[1]};
        *reinterpret_cast<f64x2u *>(p + 2) = f64x2u{v[2], v[3]};
    } else {
        if (left > 0) p[0] = v[0];
        if (left > 1) p[1] = v[1];
        if (left > 2) p[2] = v[2];
    }
}
__global__ void __launch_bounds__(kLongThreads) norm_grad_long_shares(NormGradArgs a) {
    constexpr int ROWS = 8;
    __shared__ double sums[2][kLongThreads / 64], factors[ROWS][2];
    double *part = static_cast<double *>(a.part) + (int64_t)blockIdx.x * a.N;
    auto weight = [&](int i) {
        return a.weight == nullptr ? f32x4u{1.0f, 1.0f, 1.0f, 1.0f} : rowk::load4(a.weight + i, a.N - i);
    };
    for (int64_t t0 = blockIdx.x; t0 < a.T; t0 += (int64_t)ROWS * a.P) {
        const int64_t there = (a.T - t0 + a.P - 1) / a.P;
        const int rows = there < ROWS ? (int)there : ROWS;
        for (int q = 0; q < rows; ++q) {
            const int64_t t = t0 + (int64_t)q * a.P;
            const float *h = a.h + t * a.ldh, *d = a.dy + t * a.lddy;
            double s = 0.0, m = 0.0;
            each(a.N, [&](int i) {
                const f32x4u x = rowk::load4(h + i, a.N - i), y = rowk::load4(d + i, a.N - i), w = weight(i);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s = fma((double)x[e], (double)x[e], s);
                    m = fma((double)y[e] * (double)w[e], (double)x[e], m);
                }
            });
            s = over_row<kLongThreads>(s, rowk::Add(), sums[0]);  // (its barriers: the last rows' factors are read)
            m = over_row<kLongThreads>(m, rowk::Add(), sums[1]);
            if (threadIdx.x == 0) {
                const double r = 1.0 / sqrt(s / (double)a.N + a.eps);
                factors[q][0] = r;
                factors[q][1] = r * r * (m / (double)a.N);
            }
        }
        __syncthreads();
        each(a.N, [&](int i) {
            const int left = a.N - i;
            const f32x4u w = weight(i);
            double p[4] = {0.0, 0.0, 0.0, 0.0};
            if (t0 != (int64_t)blockIdx.x) get_share(part + i, left, p);
#pragma unroll 2
            for (int q = 0; q < rows; ++q) {
                const int64_t t = t0 + (int64_t)q * a.P;
                const double r = factors[q][0], k = factors[q][1];
                const f32x4u x = rowk::load4(a.h + t * a.ldh + i, left), y = rowk::load4(a.dy + t * a.lddy + i, left);
                f32x4u ds = {0.0f, 0.0f, 0.0f, 0.0f}, o;
                if (a.dsum != nullptr) ds = rowk::load4(a.dsum + t * a.ldds + i, left);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = fma((double)y[e] * r, (double)x[e], p[e]);
                    o[e] = norm_back(x[e], y[e], w[e], ds[e], r, k);
                }
                if (a.dh != nullptr) rowk::store4(a.dh + t * a.lddh + i, left, o);
            }
            put_share(part + i, left, p);
        });
    }
}

// dweight = beta dweight + the sum of the P shares.  16 columns a workgroup (a line of
// each share), its 64 groups of 16 lanes take every 64th share, eight loads in flight;
// added up in order.
constexpr int kShareColumns = 16, kShareGroups = 64;
template <class Share>
__global__ void __launch_bounds__(kShareColumns * kShareGroups) norm_weight_grad(NormGradArgs a) {
    __shared__ double sums[kShareGroups][kShareColumns];
    const int col = threadIdx.x % kShareColumns, group = threadIdx.x / kShareColumns;
    const int64_t n = (int64_t)blockIdx.x * kShareColumns + col;
    double s = 0.0;
    if (n < a.N) {
        const Share *from = static_cast<const Share *>(a.part) + n;
        for (int p = group; p < a.P; p += 8 * kShareGroups) {
            Share v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = p + i * kShareGroups < a.P ? from[(int64_t)(p + i * kShareGroups) * a.N] : Share(0);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += (double)v[i];
        }
    }
    sums[group][col] = s;
    __syncthreads();
    if (group != 0 || n >= a.N) return;
#pragma unroll 8
    for (int i = 1; i < kShareGroups; ++i) s += sums[i][col];
    a.dweight[n] = (float)(a.beta != 0.0f ? fma((double)a.beta, (double)a.dweight[n], s) : s);
}

}  // namespace normk
