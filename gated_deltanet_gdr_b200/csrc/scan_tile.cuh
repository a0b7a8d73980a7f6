// scan_tile.cuh -- what the forward and backward kernels of the gated linear recurrence share: the cut of a sequence
// into tiles, the staging of a tile's inputs, and the composition of spans.
//
// A span of tokens maps the state at its start to the state at its end as h -> A h + B (A the product of the decays, B
// what the span writes); spans compose as (A2 A1, A2 B1 + B2).  A block of 256 threads takes a tile of LX * V channels
// and 8 * 256 / LX tokens of one (sequence, head): a thread owns V channels of kSteps consecutive tokens (a segment), LX
// lanes lie side by side over the channels, and the segments follow one another over the lanes of a warp and over the
// warps.  Every thread reduces its segment, the segments compose by shuffles within a warp and through shared memory
// between the warps, and each thread then walks its segment again, in registers, from the state it starts with: the
// inputs are read from memory once.  With few channels the blocks of a cluster take consecutive tiles and exchange
// their tiles' (A, B) through distributed shared memory.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace gdr {
namespace scan {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 8;     // tokens of a thread in a tile
constexpr int kMaxRanks = 8;  // blocks of a cluster (the portable limit)

// 1 - e^g without cancellation: the Taylor series -g (1 + g/2 (1 + g/3 (...))) near 0, where its first dropped term is
// below 2^-24 of the sum, and the difference elsewhere (e^g <= 0.78 there, so it loses under three bits)
__device__ __forceinline__ float one_minus_exp(float g, float a) {
    float p = fmaf(g, 1.f / 7.f, 1.f);
    p = fmaf(g * (1.f / 6.f), p, 1.f);
    p = fmaf(g * (1.f / 5.f), p, 1.f);
    p = fmaf(g * (1.f / 4.f), p, 1.f);
    p = fmaf(g * (1.f / 3.f), p, 1.f);
    p = fmaf(g * (1.f / 2.f), p, 1.f);
    return fabsf(g) >= 0.25f ? 1.f - a : -g * p;
}

// length of sequence b, or -1 for one outside [0, S]
__device__ __forceinline__ int seq_len(const int32_t *lengths, int b, int S) {
    const int L = lengths ? lengths[b] : S;
    return (L < 0 || L > S) ? -1 : L;
}

// ---- V consecutive elements ------------------------------------------------------------------------------------

template <int N> struct Raw;
template <> struct Raw<2> { using type = unsigned short; };
template <> struct Raw<4> { using type = unsigned; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };
template <typename T, int V> using RawV = typename Raw<(int)sizeof(T) * V>::type;

template <typename T, int V> __device__ __forceinline__ void unpack(const RawV<T, V> &r, float (&x)[V]) {
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(e[i]);
}
template <typename T, int V> __device__ __forceinline__ void store(T *p, const float (&x)[V]) {
    RawV<T, V> r;
    T *e = reinterpret_cast<T *>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_f32<T>(x[i]);
    *reinterpret_cast<RawV<T, V> *>(p) = r;
}
template <int V> __device__ __forceinline__ void load_f32(const float *p, float (&x)[V]) {
    unpack<float, V>(*reinterpret_cast<const RawV<float, V> *>(p), x);
}

// ---- staging: every thread copies its own inputs to a place of its own, so that no barrier is needed to read them --

// copies one element vector to shared memory, or zeros where !on (src is then not read)
template <typename R> __device__ __forceinline__ void stage(R *dst, const void *src, bool on) {
    if constexpr (sizeof(R) >= 4) {
        const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
        const int n = on ? (int)sizeof(R) : 0;
        if constexpr (sizeof(R) == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(sizeof(R)), "r"(n)
                         : "memory");
    } else {
        *dst = on ? *static_cast<const R *>(src) : R{};
    }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// ---- clusters -----------------------------------------------------------------------------------------------------

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// writes V floats at `p` (an address in this block's shared memory) in block `rank` of the cluster
template <int V> __device__ __forceinline__ void put_remote(float *p, int rank, const float (&x)[V]) {
    const unsigned local = (unsigned)__cvta_generic_to_shared(p);
    unsigned a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
    if constexpr (V == 4)
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3])
                     : "memory");
    else if constexpr (V == 2)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x[0]), "f"(x[1]) : "memory");
    else
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x[0]) : "memory");
}

// ---- the cut -------------------------------------------------------------------------------------------------------

struct Cut {
    int lx;     // lanes side by side over the channels, a power of two
    int slabs;  // tiles over the channels
    int ranks;  // blocks of a cluster: consecutive tiles in time
    __host__ __device__ int tile() const { return kSteps * (kThreads / lx); }  // tokens of a tile
};

// Lanes over the channels: as many as leave the fewest of them idle on this D.  Fewer where that leaves the GPU without
// two blocks for every SM, and blocks in clusters where that still does (a tile that no token reaches is never made).
inline Cut choose_cut(long long rows, int D, int V, int S, int max_lx, int sms) {
    Cut c{};
    long long best = -1;
    for (int lx = max_lx; lx >= 4; lx /= 2) {
        const long long slabs = (D + (long long)lx * V - 1) / ((long long)lx * V);
        if (best < 0 || slabs * lx < best) {
            best = slabs * lx;
            c.lx = lx;
            c.slabs = (int)slabs;
        }
    }
    const long long want = 2LL * sms;
    while (c.lx > 8 && rows * c.slabs * 2 <= want && c.tile() < S) {
        c.lx /= 2;
        c.slabs = (int)((D + (long long)c.lx * V - 1) / ((long long)c.lx * V));
    }
    c.ranks = 1;
    while (c.ranks < kMaxRanks && rows * c.slabs * c.ranks * 2 <= want && (long long)c.ranks * c.tile() < S) c.ranks *= 2;
    return c;
}

}  // namespace scan
}  // namespace gdr
