// pairs.cuh -- vectors of a few channels per thread: loads, stores and staging through shared memory, and arithmetic on
// pairs of channels (f32x2), for the streaming kernels of the recurrence and of the conv1d's gradient.
#pragma once

#include "common.cuh"

namespace gdr {

// ---- channels in pairs -----------------------------------------------------------------------------------------------

template <int V> constexpr int kPairs = (V + 1) / 2;  // a single channel fills half of one

__device__ __forceinline__ void up2(float2 v, float &lo, float &hi) {
    lo = v.x;
    hi = v.y;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- V consecutive elements ------------------------------------------------------------------------------------

template <int N> struct Raw;
template <> struct Raw<2> { using type = unsigned short; };
template <> struct Raw<4> { using type = unsigned; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };
template <typename T, int V> using RawV = typename Raw<(int)sizeof(T) * V>::type;

template <typename T, int V> __device__ __forceinline__ void unpack(const RawV<T, V> &r, float2 (&x)[kPairs<V>]) {
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) x[i] = make_float2(to_f32(e[2 * i]), 2 * i + 1 < V ? to_f32(e[2 * i + 1 < V ? 2 * i + 1 : 0]) : 0.f);
}
template <typename T, int V> __device__ __forceinline__ void store(void *p, const float2 (&x)[kPairs<V>]) {
    RawV<T, V> r;
    T *e = reinterpret_cast<T *>(&r);
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
        float lo, hi;
        up2(x[i], lo, hi);
        e[2 * i] = from_f32<T>(lo);
        if (2 * i + 1 < V) e[2 * i + 1 < V ? 2 * i + 1 : 0] = from_f32<T>(hi);
    }
    *static_cast<RawV<T, V> *>(p) = r;
}
template <int V> __device__ __forceinline__ void load_f32(const float *p, float2 (&x)[kPairs<V>]) {
    unpack<float, V>(*reinterpret_cast<const RawV<float, V> *>(p), x);
}
template <int P> __device__ __forceinline__ void fill(float2 (&x)[P], float v) {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = both(v);
}
// a pair from the lane d below, d above
__device__ __forceinline__ float2 shfl_up2(float2 x, int d) {
    float lo, hi;
    up2(x, lo, hi);
    return make_float2(__shfl_up_sync(0xffffffffu, lo, d), __shfl_up_sync(0xffffffffu, hi, d));
}
__device__ __forceinline__ float2 shfl_down2(float2 x, int d) {
    float lo, hi;
    up2(x, lo, hi);
    return make_float2(__shfl_down_sync(0xffffffffu, lo, d), __shfl_down_sync(0xffffffffu, hi, d));
}

// ---- staging: every thread copies its own inputs to a place of its own, so that no barrier is needed to read them --

// copies one element vector to shared memory, or zeros where !on (src is then not read)
template <typename R, bool kMask> __device__ __forceinline__ void stage(R *dst, const void *src, bool on) {
    if constexpr (sizeof(R) >= 4) {
        const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
        if constexpr (!kMask) {
            if constexpr (sizeof(R) == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(sizeof(R)) : "memory");
        } else {
            const int n = on ? (int)sizeof(R) : 0;
            if constexpr (sizeof(R) == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(sizeof(R)), "r"(n)
                             : "memory");
        }
    } else {
        *dst = !kMask || on ? *static_cast<const R *>(src) : R{};
    }
}
// a thread's TS tokens of one tensor, rows `row` bytes apart, n of them valid (the others zero); src is the first
template <int TS, int kThreads, typename R>
__device__ __forceinline__ void stage_segment(R (*dst)[kThreads], const void *src, unsigned row, int n) {
    const char *p = static_cast<const char *>(src);
    if (n == TS) {
#pragma unroll
        for (int j = 0; j < TS; ++j) stage<R, false>(&dst[j][threadIdx.x], p + j * (size_t)row, true);
    } else {
#pragma unroll
        for (int j = 0; j < TS; ++j) stage<R, true>(&dst[j][threadIdx.x], j < n ? p + j * (size_t)row : p, j < n);
    }
}
// the same by warps: lx lanes lie side by side over a row's elements of R, and the 32 / lx segments of TS tokens of the warp
// follow one another, so that 16 bytes a lane cover the same lx * sizeof(R) bytes (at least 16) of one row after the
// other.  p is the warp's first token's row at the block's first channel, n its valid tokens (may be <= 0), `bytes` what
// the rows still hold there (a multiple of 16, may be <= 0).  Lanes read what others copied: __syncwarp() after the wait
// and before the next copy.
template <int TS, int kThreads, typename R>
__device__ __forceinline__ void stage_rows(R (*dst)[kThreads], const char *p, unsigned row, int lx, int n, int bytes) {
    const int lane = threadIdx.x & 31, lanes = lx * (int)sizeof(R) / 16;  // lanes of a row: a power of two
    const int sub = lane / lanes, at = (lane & (lanes - 1)) * 16, rows = 32 / lanes;
    const bool on = at < bytes;
#pragma unroll
    for (int k = 0; k < TS * (int)sizeof(R) / 16; ++k) {
        const int r = k * rows + sub;  // the warp's token
        const bool in = on && r < n;
        const unsigned d = (unsigned)__cvta_generic_to_shared(&dst[r & (TS - 1)][(threadIdx.x & ~31) + r / TS * lx]) + at;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(in ? p + r * (size_t)row + at : p),
                     "r"(in ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
// the stage committed before the last one is there
__device__ __forceinline__ void stage_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

}  // namespace gdr
