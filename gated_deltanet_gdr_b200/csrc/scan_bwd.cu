// scan_bwd.cu -- the gradient of the gated linear recurrence (gdr_scan_bwd): with lambda_t = dout_t + mu_{t+1} and mu_t =
// a_t lambda_t, dx_t = lambda_t (or (1 - a_t) lambda_t) and dg_t = mu_t h_{t-1} (or mu_t (h_{t-1} - x_t)).
//
// One pass over x, g and dout, last tile first (scan_tile.cuh).  mu is the same recurrence run backwards, so a span of
// tokens composes forwards for h and backwards for mu with one product A.  The states come from the checkpoint before
// each chunk of 64 tokens, so only mu is handed from tile to tile (and between the blocks of a cluster).  Bound by HBM.
#include "scan_tile.cuh"

namespace gdr {
namespace {
using namespace scan;

constexpr int kSteps = 4;   // tokens of a thread in a tile: decays, states and gradients of a segment stay in registers
constexpr int kMaxLx = 16;  // so that a tile holds whole chunks

template <typename T, typename G, int V> struct Layout {
    static constexpr int kCh = kMaxLx * V;
    RawV<G, V> g[kSteps][kThreads];
    RawV<T, V> x[kSteps][kThreads], d[kSteps][kThreads];
    float wa[2][kWarps][kCh], wf[2][kWarps][kCh], wr[2][kWarps][kCh];  // A and the forward and backward B of every warp
    float ca[2][kMaxRanks][kCh], cr[2][kMaxRanks][kCh];                // A and the backward B of every block of the cluster
    uint64_t arrived[2];
};

template <typename T, typename G, bool kMix, int V>
__global__ void __launch_bounds__(kThreads, kMix ? 2 : 3) scan_bwd_kernel(const ScanBwdArgs a, const Cut cut) {
    extern __shared__ __align__(16) unsigned char smem[];
    auto &sm = *reinterpret_cast<Layout<T, G, V> *>(smem);
    constexpr int P = kPairs<V>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lx = cut.lx, cl = lane & (lx - 1);
    const int seg = tid / lx;
    const int R = cut.ranks, rank = (int)(blockIdx.x % R);
    const long long unit = blockIdx.x / R;
    const int slab = (int)(unit % cut.slabs);
    const long long bn = unit / cut.slabs;
    const int c0 = (slab * lx + cl) * V;
    const bool on = c0 < a.D;
    const int Lr = seq_len(a.lengths, (int)(bn / a.N), a.S);
    const int L = Lr < 0 ? 0 : Lr;
    if (Lr < 0 && tid == 0 && rank == 0) raise_device_error(a.err, GDR_DEVERR_LENGTH);

    const unsigned row_x = (unsigned)a.D * sizeof(T), row_g = (unsigned)a.D * sizeof(G);
    const size_t base = (size_t)bn * a.S * a.D + c0;
    const char *x = reinterpret_cast<const char *>(static_cast<const T *>(a.x) + base);
    const char *g = reinterpret_cast<const char *>(static_cast<const G *>(a.g) + base);
    const char *d = reinterpret_cast<const char *>(static_cast<const T *>(a.dout) + base);
    char *dx = reinterpret_cast<char *>(static_cast<T *>(a.dx) + base);
    char *dg = reinterpret_cast<char *>(static_cast<G *>(a.dg) + base);
    const int chunks = (a.S + kChunk - 1) / kChunk;
    const float *ck = a.checkpoints + (size_t)bn * chunks * a.D + c0;
    f2_t mu[P];  // what the tokens behind the cluster's tiles pass back, the same in every block
    fill(mu, 0.f);
    if (on && a.dfinal_state && Lr >= 0) load_f32<V>(a.dfinal_state + (size_t)bn * a.D + c0, mu);

    const int TT = kSteps * (kThreads / lx);
    const long long step = (long long)R * TT;
    const int tiles = (int)((L + step - 1) / step);
    const int chunk_warps = lx > 2 ? lx / 2 : 1;  // warps of a chunk: 64 / kSteps segments, 32 / lx of them a warp
    const unsigned exchange = (unsigned)(R * lx * V * 2 * sizeof(float));
    bool lost = false;
    if (R > 1) {
        if (tid == 0) {
            sm100::mbar_init(&sm.arrived[0], 1);
            sm100::mbar_init(&sm.arrived[1], 1);
            sm100::fence_mbar_init();
        }
        cluster_meet();
    }

    auto fetch = [&](int k) {
        const long long t0 = k * step + (long long)rank * TT + seg * kSteps;
        const int n = on ? (int)max(0LL, min((long long)kSteps, L - t0)) : 0;
        const size_t at = n > 0 ? (size_t)t0 : 0;
        stage_segment<kSteps>(sm.g, g + at * row_g, row_g, n);
        stage_segment<kSteps>(sm.x, x + at * row_x, row_x, n);
        stage_segment<kSteps>(sm.d, d + at * row_x, row_x, n);
        stage_commit();
    };
    if (tiles > 0) fetch(tiles - 1);
    for (int k = tiles - 1, n = 0; k >= 0; --k, ++n) {
        const int p = n & 1;
        const long long t0 = k * step + (long long)rank * TT + seg * kSteps;
        f2_t h[P];  // the state before the chunk
        fill(h, 0.f);
        const long long chunk = t0 / kChunk;
        if (on && chunk * kChunk < L) load_f32<V>(ck + (size_t)chunk * a.D, h);
        // a segment forwards, (A, F): h -> A h + F, and backwards, (A, B): mu -> A mu + B; behind the sequence a = 1 and
        // x = dout = 0, which changes neither
        f2_t av[kSteps][P], rest[kMix ? kSteps : 1][P], xv[kSteps][P], dv[kSteps][P], A[P], F[P], B[P];
        stage_wait();
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            f2_t gv[P];
            unpack<G, V>(sm.g[j][tid], gv);
            unpack<T, V>(sm.x[j][tid], xv[j]);
            unpack<T, V>(sm.d[j][tid], dv[j]);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                f2_t r;
                decay<kMix>(gv[i], av[j][i], r);
                if (kMix) rest[kMix ? j : 0][i] = r;
                const f2_t b = kMix ? mul2(xv[j][i], r) : xv[j][i];
                A[i] = j ? mul2(A[i], av[j][i]) : av[j][i];
                F[i] = j ? fma2(av[j][i], F[i], b) : b;
            }
        }
#pragma unroll
        for (int j = kSteps - 1; j >= 0; --j)
#pragma unroll
            for (int i = 0; i < P; ++i) B[i] = mul2(av[j][i], j < kSteps - 1 ? add2(dv[j][i], B[i]) : dv[j][i]);
        // over the segments of the warp: (EA, EF) those before this one, (LA, LB) those behind it
        f2_t EA[P], EF[P], LA[P], LB[P], TA[P], TF[P], TB[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            TA[i] = LA[i] = A[i];
            TF[i] = F[i];
            TB[i] = B[i];
        }
        for (int q = lx; q < 32; q *= 2) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const f2_t pa = shfl_up2(TA[i], q), pf = shfl_up2(TF[i], q);
                if (lane >= q) {
                    TF[i] = fma2(TA[i], pf, TF[i]);
                    TA[i] = mul2(TA[i], pa);
                }
                const f2_t na = shfl_down2(LA[i], q), nb = shfl_down2(TB[i], q);
                if (lane + q < 32) {
                    TB[i] = fma2(LA[i], nb, TB[i]);
                    LA[i] = mul2(LA[i], na);
                }
            }
        }
        if (lane >= 32 - lx) {
            store<float, V>(&sm.wa[p][warp][cl * V], TA);
            store<float, V>(&sm.wf[p][warp][cl * V], TF);
        }
        if (lane < lx) store<float, V>(&sm.wr[p][warp][cl * V], TB);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            EA[i] = shfl_up2(TA[i], lx);
            EF[i] = shfl_up2(TF[i], lx);
            LA[i] = shfl_down2(LA[i], lx);
            LB[i] = shfl_down2(TB[i], lx);
        }
        __syncthreads();
        if (k > 0) fetch(k - 1);
        if (R > 1) {  // as in the forward kernel, the block's backward map to every block of the cluster
            if (tid == 0) sm100::mbar_arrive_expect_tx(&sm.arrived[p], exchange);
            if (warp < R && lane < lx) {
                f2_t ta[P], tb[P];
                load_f32<V>(&sm.wa[p][kWarps - 1][cl * V], ta);
                load_f32<V>(&sm.wr[p][kWarps - 1][cl * V], tb);
#pragma unroll
                for (int w = kWarps - 2; w >= 0; --w) {
                    f2_t wa[P], wb[P];
                    load_f32<V>(&sm.wa[p][w][cl * V], wa);
                    load_f32<V>(&sm.wr[p][w][cl * V], wb);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        tb[i] = fma2(wa[i], tb[i], wb[i]);
                        ta[i] = mul2(ta[i], wa[i]);
                    }
                }
                put_remote<V>(&sm.ca[p][rank][cl * V], &sm.arrived[p], warp, ta);
                put_remote<V>(&sm.cr[p][rank][cl * V], &sm.arrived[p], warp, tb);
            }
            __syncwarp();
        }
        // the state before the segment: the chunk's checkpoint, the chunk's warps before this one, its segments
        for (int w = warp & ~(chunk_warps - 1); w < warp; ++w) {
            f2_t wa[P], wf[P];
            load_f32<V>(&sm.wa[p][w][cl * V], wa);
            load_f32<V>(&sm.wf[p][w][cl * V], wf);
#pragma unroll
            for (int i = 0; i < P; ++i) h[i] = fma2(wa[i], h[i], wf[i]);
        }
        if (lane >= lx) {
#pragma unroll
            for (int i = 0; i < P; ++i) h[i] = fma2(EA[i], h[i], EF[i]);
        }
        // every token's h_{t-1} (less x_t) in the place of its x
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const f2_t q = kMix ? fma2(xv[j][i], both(-1.f), h[i]) : h[i];
                h[i] = kMix ? fma2(av[j][i], h[i], mul2(xv[j][i], rest[kMix ? j : 0][i])) : fma2(av[j][i], h[i], xv[j][i]);
                xv[j][i] = q;
            }
        if (R > 1 && !lost && !wait_remote(&sm.arrived[p], (unsigned)(n >> 1) & 1u, a.wait_ns)) {
            lost = true;
            raise_device_error(a.err, GDR_DEVERR_TIMEOUT);
        }
        // what comes back to this segment: from behind the tiles, the later blocks, the later warps, the later segments
        f2_t m[P];
#pragma unroll
        for (int i = 0; i < P; ++i) m[i] = mu[i];
        for (int r = R - 1; r >= 0 && R > 1; --r) {
            f2_t ra[P], rb[P];
            load_f32<V>(&sm.ca[p][r][cl * V], ra);
            load_f32<V>(&sm.cr[p][r][cl * V], rb);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                mu[i] = fma2(ra[i], mu[i], rb[i]);
                if (r > rank) m[i] = mu[i];
            }
        }
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            if (R > 1 && w <= warp) break;
            f2_t wa[P], wb[P];
            load_f32<V>(&sm.wa[p][w][cl * V], wa);
            load_f32<V>(&sm.wr[p][w][cl * V], wb);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (R > 1) {
                    m[i] = fma2(wa[i], m[i], wb[i]);
                } else {
                    mu[i] = fma2(wa[i], mu[i], wb[i]);
                    if (w > warp) m[i] = mu[i];
                }
            }
        }
        if (lane + lx < 32) {
#pragma unroll
            for (int i = 0; i < P; ++i) m[i] = fma2(LA[i], m[i], LB[i]);
        }
        if (on && t0 < a.S) {
            const int ns = (int)min((long long)kSteps, a.S - t0), nv = (int)max(0LL, min((long long)kSteps, L - t0));
            char *ox = dx + (size_t)t0 * row_x, *og = dg + (size_t)t0 * row_g;
#pragma unroll
            for (int j = kSteps - 1; j >= 0; --j) {
                f2_t rx[P], rg[P];
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const f2_t lam = add2(dv[j][i], m[i]);
                    m[i] = mul2(av[j][i], lam);
                    rx[i] = kMix ? mul2(rest[kMix ? j : 0][i], lam) : lam;
                    rg[i] = mul2(m[i], xv[j][i]);
                    if (j >= nv) rx[i] = rg[i] = 0;
                }
                if (j < ns) {
                    store<T, V>(ox + j * (size_t)row_x, rx);
                    store<G, V>(og + j * (size_t)row_g, rg);
                }
            }
        }
    }
    if (R > 1) cluster_meet();  // a block that gave up must not leave while the others write to it
    if (!on) return;
    f2_t zero[P];
    fill(zero, 0.f);
    for (long long t = tiles * step + (long long)rank * (kThreads / lx) + seg; t < a.S; t += (long long)R * (kThreads / lx)) {
        store<T, V>(dx + (size_t)t * row_x, zero);
        store<G, V>(dg + (size_t)t * row_g, zero);
    }
    if (a.dinitial_state && seg == 0 && rank == 0) store<float, V>(a.dinitial_state + (size_t)bn * a.D + c0, mu);
}

template <typename T, typename G, bool kMix, int V> cudaError_t launch_v(const ScanBwdArgs &a, cudaStream_t s) {
    static LaunchCache cache(reinterpret_cast<const void *>(scan_bwd_kernel<T, G, kMix, V>));
    const int smem = (int)sizeof(Layout<T, G, V>);
    int grid = 0;
    cudaError_t e = cache.allow_smem(smem);
    if (e == cudaSuccess) e = cache.resident_grid(kThreads, smem, &grid);
    if (e != cudaSuccess) return e;
    const Cut cut = choose_cut((long long)a.B * a.N, a.D, V, a.S, kSteps, kMaxLx, 2, grid / (kMix ? 2 : 3));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)a.B * a.N * cut.slabs * cut.ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cut.ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cut.ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, scan_bwd_kernel<T, G, kMix, V>, a, cut);
}

template <typename T, typename G, bool kMix> cudaError_t launch_m(const ScanBwdArgs &a, cudaStream_t s) {
    if (a.D % 4 == 0) return launch_v<T, G, kMix, 4>(a, s);
    if (a.D % 2 == 0) return launch_v<T, G, kMix, 2>(a, s);
    return launch_v<T, G, kMix, 1>(a, s);
}
template <typename T, typename G> cudaError_t launch_t(const ScanBwdArgs &a, cudaStream_t s) {
    return a.mode == GDR_SCAN_MIX ? launch_m<T, G, true>(a, s) : launch_m<T, G, false>(a, s);
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanBwdArgs &a, gdr_dtype dt, gdr_dtype gt, cudaStream_t s) {
    if (dt == GDR_F32) return launch_t<float, float>(a, s);
    if (dt == GDR_BF16) return gt == dt ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, s) : launch_t<__nv_bfloat16, float>(a, s);
    return gt == dt ? launch_t<__half, __half>(a, s) : launch_t<__half, float>(a, s);
}

}  // namespace gdr
