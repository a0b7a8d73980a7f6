// scan_step.cu -- the gated linear recurrence for decode (gdr_scan_step): up to 8 tokens of every sequence, from and to
// the slots of a pool of fp32 states.
//
// One thread owns V channels of one sequence and keeps their state in registers over the tokens; the state is read once
// and written once per commit, in 16-byte accesses where rows are made of whole ones.  The inputs of all tokens are
// loaded before the slot index arrives, so a call waits for two memory round trips (index, state).  64 sequences of 4096
// channels: 2.4 us one after the other in a graph, 4.9 a call through the Python binding; 256 sequences of 4 drafts, fp16 (34
// MB, 5 us at the measured copy rate): 7.9 us in a graph (8.7 with room for 8 tokens in registers), 9.7 to 10.2 a call.
#include "kernels.h"
#include "scan_tile.cuh"

namespace gdr {
namespace {
using namespace scan;

constexpr int kStepThreads = 128;

template <typename T, typename G, bool kMix, int V, int kTokens>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(const ScanStepArgs a) {
    constexpr int P = kPairs<V>;
    const unsigned per = (unsigned)a.N * a.D;  // channels of a sequence; < 2^31
    const unsigned c = (blockIdx.x * kStepThreads + threadIdx.x) * V;
    const int b = blockIdx.y;
    if (c >= per) return;
    const unsigned n = c / (unsigned)a.D, d = c - n * (unsigned)a.D;
    const size_t base = ((size_t)b * a.N + n) * a.S * a.D + d;
    const T *x = static_cast<const T *>(a.x) + base;
    const G *g = static_cast<const G *>(a.g) + base;
    T *out = static_cast<T *>(a.out) + base;
    const int32_t *idx = a.idx + (size_t)b * a.S;
    const int S = kTokens == 1 ? 1 : a.S;

    RawV<T, V> xr[kTokens];
    RawV<G, V> gr[kTokens];
    int slot[kTokens];
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
        if (t < S) {
            xr[t] = *reinterpret_cast<const RawV<T, V> *>(x + (size_t)t * a.D);
            gr[t] = *reinterpret_cast<const RawV<G, V> *>(g + (size_t)t * a.D);
            slot[t] = idx[t];
        }
    int L = a.lengths ? a.lengths[b] : S;
    unsigned bad = L < 0 || L > S ? GDR_DEVERR_LENGTH : 0u;
    int start = 0, commit = 0;
    if (!bad && L > 0) {
        if (a.per_token) {
            const int A = a.accepted ? a.accepted[b] : 1;
            if (A < 1 || A > S) bad = GDR_DEVERR_LENGTH;
            else start = A - 1;
            commit = L;
        } else {
            commit = a.accepted ? min(max(a.accepted[b], 0), L) : L;
        }
    }
    int from = 0;
    if (!bad && L > 0) {
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            if (t == start) from = slot[t];
            if (t < commit && (unsigned)slot[t] >= (unsigned)a.slots) bad = GDR_DEVERR_SLOT_INDEX;
        }
        if ((unsigned)from >= (unsigned)a.slots) bad = GDR_DEVERR_SLOT_INDEX;
    }
    if (bad) {
        if (c == 0) raise_device_error(a.err, bad);
        L = commit = 0;
    }
    float2 h[P];
    fill(h, 0.f);
    if (L > 0) load_f32<V>(a.pool + (size_t)from * per + c, h);
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
        if (t >= S) break;
        if (t < L) {
            float2 xv[P], gv[P];
            unpack<T, V>(xr[t], xv);
            unpack<G, V>(gr[t], gv);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 av, rest;
                decay<kMix>(gv[i], av, rest);
                h[i] = __ffma2_rn(av, h[i], kMix ? __fmul2_rn(xv[i], rest) : xv[i]);
            }
            if (t < commit) store<float, V>(a.pool + (size_t)slot[t] * per + c, h);
            store<T, V>(out + (size_t)t * a.D, h);
        } else {
            float2 zero[P];
            fill(zero, 0.f);
            store<T, V>(out + (size_t)t * a.D, zero);
        }
    }
}

template <typename T, typename G, bool kMix, int V> cudaError_t launch_v(const ScanStepArgs &a, cudaStream_t s) {
    const unsigned per = (unsigned)a.N * a.D;
    constexpr unsigned kPer = kStepThreads * V;
    // the sequences lie over the grid's second dimension, 65535 at a time
    for (int b0 = 0; b0 < a.B; b0 += 65535) {
        ScanStepArgs p = a;
        const int nb = a.B - b0 < 65535 ? a.B - b0 : 65535;
        const size_t tokens = (size_t)b0 * a.S;
        p.x = static_cast<const T *>(a.x) + tokens * per;
        p.g = static_cast<const G *>(a.g) + tokens * per;
        p.out = static_cast<T *>(a.out) + tokens * per;
        p.idx = a.idx + tokens;
        p.lengths = a.lengths ? a.lengths + b0 : nullptr;
        p.accepted = a.accepted ? a.accepted + b0 : nullptr;
        const dim3 grid((per + kPer - 1) / kPer, (unsigned)nb);
        if (a.S == 1) scan_step_kernel<T, G, kMix, V, 1><<<grid, kStepThreads, 0, s>>>(p);
        else if (a.S <= 4) scan_step_kernel<T, G, kMix, V, 4><<<grid, kStepThreads, 0, s>>>(p);
        else scan_step_kernel<T, G, kMix, V, kDecodeMaxTokens><<<grid, kStepThreads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

// a vector must not cross the rows of two heads
template <typename T, typename G, bool kMix> cudaError_t launch_m(const ScanStepArgs &a, cudaStream_t s) {
    if (a.D % 4 == 0) return launch_v<T, G, kMix, 4>(a, s);
    if (a.D % 2 == 0) return launch_v<T, G, kMix, 2>(a, s);
    return launch_v<T, G, kMix, 1>(a, s);
}
template <typename T, typename G> cudaError_t launch_t(const ScanStepArgs &a, cudaStream_t s) {
    return a.mode == GDR_SCAN_MIX ? launch_m<T, G, true>(a, s) : launch_m<T, G, false>(a, s);
}

}  // namespace

cudaError_t launch_scan_step(const ScanStepArgs &a, gdr_dtype dt, gdr_dtype gt, cudaStream_t s) {
    if (dt == GDR_F32) return launch_t<float, float>(a, s);
    if (dt == GDR_BF16) return gt == dt ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, s) : launch_t<__nv_bfloat16, float>(a, s);
    return gt == dt ? launch_t<__half, __half>(a, s) : launch_t<__half, float>(a, s);
}

}  // namespace gdr
