// scan.cu -- the gated linear recurrence h_t = a_t h_{t-1} + b_t per channel (a_t = exp(g_t), b_t = x_t or
// (1 - a_t) x_t): gdr_scan_fwd, gdr_scan_bwd and gdr_scan_step.
//
// One thread per channel, walking the tokens in order.
#include "common.cuh"
#include "kernels.h"

namespace gdr {
namespace {

constexpr int kThreads = 128;

// 1 - e^g without cancellation: the Taylor series -g (1 + g/2 (1 + g/3 (...))) near 0, where its first dropped term is
// below 2^-24 of the sum, and the difference elsewhere (e^g <= 0.78 there, so it loses under three bits)
__device__ __forceinline__ float one_minus_exp(float g, float a) {
    if (fabsf(g) >= 0.25f) return 1.f - a;
    float p = 1.f + g * (1.f / 7.f);
    p = fmaf(g * (1.f / 6.f), p, 1.f);
    p = fmaf(g * (1.f / 5.f), p, 1.f);
    p = fmaf(g * (1.f / 4.f), p, 1.f);
    p = fmaf(g * (1.f / 3.f), p, 1.f);
    p = fmaf(g * (1.f / 2.f), p, 1.f);
    return -g * p;
}

__device__ __forceinline__ int seq_len(const int32_t *lengths, int b, int S) {
    const int L = lengths ? lengths[b] : S;
    return (L < 0 || L > S) ? -1 : L;
}

template <typename T, typename G, bool kMix>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(const ScanStepArgs a) {
    const long long c = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long per = (long long)a.N * a.D;
    if (c >= (long long)a.B * per) return;
    const int b = (int)(c / per);
    const long long ch = c % per;
    const int n = (int)(ch / a.D), d = (int)(ch % a.D);
    const size_t base = ((size_t)b * a.N + n) * a.S * a.D + d;
    const T *x = static_cast<const T *>(a.x) + base;
    const G *g = static_cast<const G *>(a.g) + base;
    T *out = static_cast<T *>(a.out) + base;
    const int32_t *idx = a.idx + (size_t)b * a.S;
    int L = a.lengths ? a.lengths[b] : a.S;
    unsigned bad = 0;
    if (L < 0 || L > a.S) bad = GDR_DEVERR_LENGTH;
    int start = 0, commit = 0;
    if (!bad && L > 0) {
        if (a.per_token) {
            const int A = a.accepted ? a.accepted[b] : 1;
            if (A < 1 || A > a.S) bad = GDR_DEVERR_LENGTH;
            else start = A - 1;
            commit = L;
        } else {
            commit = a.accepted ? min(max(a.accepted[b], 0), L) : L;
        }
        if (!bad) {
            if ((unsigned)idx[start] >= (unsigned)a.slots) bad = GDR_DEVERR_SLOT_INDEX;
            for (int t = 0; t < commit; ++t)
                if ((unsigned)idx[t] >= (unsigned)a.slots) bad = GDR_DEVERR_SLOT_INDEX;
        }
    }
    if (bad) {
        if (ch == 0) raise_device_error(a.err, bad);
        L = 0;
    }
    float h = L > 0 ? a.pool[(size_t)idx[start] * per + ch] : 0.f;
    for (int t = 0; t < a.S; ++t) {
        const size_t at = (size_t)t * a.D;
        if (t < L) {
            const float gt = to_f32(g[at]), at_ = expf(gt), xt = to_f32(x[at]);
            h = fmaf(at_, h, kMix ? one_minus_exp(gt, at_) * xt : xt);
            if (t < commit) a.pool[(size_t)idx[t] * per + ch] = h;
        }
        out[at] = from_f32<T>(t < L ? h : 0.f);
    }
}

template <typename T, typename G, bool kMix> struct Step {
    static void go(const ScanStepArgs &a, cudaStream_t s) {
        const long long n = (long long)a.B * a.N * a.D;
        scan_step_kernel<T, G, kMix><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
    }
};

// the five pairs of input and gate types, with and without the mixing factor
template <template <typename, typename, bool> class F, typename Args>
cudaError_t dispatch(const Args &a, gdr_dtype dt, gdr_dtype gt, cudaStream_t s) {
    const bool own = gt == dt;
#define GDR_SCAN_PAIR(T, G) (a.mode == GDR_SCAN_MIX ? F<T, G, true>::go(a, s) : F<T, G, false>::go(a, s))
    if (dt == GDR_F32) GDR_SCAN_PAIR(float, float);
    else if (dt == GDR_BF16 && own) GDR_SCAN_PAIR(__nv_bfloat16, __nv_bfloat16);
    else if (dt == GDR_BF16) GDR_SCAN_PAIR(__nv_bfloat16, float);
    else if (own) GDR_SCAN_PAIR(__half, __half);
    else GDR_SCAN_PAIR(__half, float);
#undef GDR_SCAN_PAIR
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_step(const ScanStepArgs &a, gdr_dtype dt, gdr_dtype gt, cudaStream_t s) {
    return dispatch<Step>(a, dt, gt, s);
}

}  // namespace gdr
