// lanes.hpp -- what the row and block kernels share: buffer descriptors that end at an
// operand's last element, lane exchange, four floats at any 4-byte alignment, waits for
// loads that write LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#undef SGEMM_PHASES
#include "sgemm_kernels.hpp"

namespace rowk {

using sgk::f32x2;
using sgk::f32x4;
using sgk::rsrc_t;

// A descriptor over [base, base + bytes), at most kOut bytes; an access at
// kOut is outside every one (and its 16 bytes do not wrap).
constexpr uint32_t kOut = 0xfffffff0u;
__device__ __forceinline__ uint32_t records(int64_t bytes) {
    return bytes <= 0 ? 0u : (bytes >= (int64_t)kOut ? kOut : (uint32_t)bytes);
}
__device__ __forceinline__ rsrc_t exact_rsrc(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, sgk::kRsrcWord3);
}
__device__ __forceinline__ rsrc_t whole_rsrc(const void *base, int64_t bytes) {
    return exact_rsrc(base, records(bytes));
}

// ---------------------------------------------------------------------------
// Lane exchange inside a 16-lane DPP row and across a wave's four rows.
// ---------------------------------------------------------------------------
template <int CTRL> __device__ __forceinline__ int dpp(int v) {
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true);
}
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __int_as_float(dpp<CTRL>(__float_as_int(v)));
}
template <int CTRL> __device__ __forceinline__ double dpp(double v) {
    return __hiloint2double(dpp<CTRL>(__double2hiint(v)), dpp<CTRL>(__double2loint(v)));
}
__device__ __forceinline__ int at_lane(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ float at_lane(float v, int l) { return __int_as_float(at_lane(__float_as_int(v), l)); }
__device__ __forceinline__ double at_lane(double v, int l) {
    return __hiloint2double(at_lane(__double2hiint(v), l), at_lane(__double2loint(v), l));
}

// op over the L lanes (16 or 64) that share a row; every lane gets the result,
// always combined in the same order.  row_ror:n (0x120 + n) turns a 16-lane row.
template <int L, class T, class Op> __device__ __forceinline__ T reduce(T v, Op op) {
    static_assert(L == 16 || L == 64, "a DPP row or a wave");
    v = op(v, dpp<0x128>(v));
    v = op(v, dpp<0x124>(v));
    v = op(v, dpp<0x122>(v));
    v = op(v, dpp<0x121>(v));
    if constexpr (L == 64) v = op(op(at_lane(v, 0), at_lane(v, 16)), op(at_lane(v, 32), at_lane(v, 48)));
    return v;
}
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
    __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};
struct Min {
    __device__ __forceinline__ int operator()(int a, int b) const { return a < b ? a : b; }
};
struct Add {
    template <class T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

// four floats at any 4-byte alignment (one 16-byte access on gfx950)
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ f32x4u load4(const float *p, int left) {
    f32x4u v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (left >= 4) {
        v = *reinterpret_cast<const f32x4u *>(p);
    } else {
        if (left > 0) v.x = p[0];
        if (left > 1) v.y = p[1];
        if (left > 2) v.z = p[2];
    }
    return v;
}
__device__ __forceinline__ void store4(float *p, int left, f32x4u v) {
    if (left >= 4) {
        *reinterpret_cast<f32x4u *>(p) = v;
    } else {
        if (left > 0) p[0] = v.x;
        if (left > 1) p[1] = v.y;
        if (left > 2) p[2] = v.z;
    }
}
// (element by element: no packed FP32 instructions)
template <class V> __device__ __forceinline__ V fma4(float s, V a, V c) {
    V r;
    r.x = fmaf(s, a.x, c.x);
    r.y = fmaf(s, a.y, c.y);
    r.z = fmaf(s, a.z, c.z);
    r.w = fmaf(s, a.w, c.w);
    return r;
}

// Waits until this wave's loads but the newest N have landed and its LDS accesses have
// completed (gfx9 encoding: vmcnt in bits 3:0 and 15:14, lgkmcnt 0, expcnt any).
template <int N> __device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N <= 63, "vmcnt is 6 bits");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

}  // namespace rowk
