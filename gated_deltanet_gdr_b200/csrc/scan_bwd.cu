// scan_bwd.cu -- the gradient of the gated linear recurrence (gdr_scan_bwd): with lambda_t = dout_t + mu_{t+1} and mu_t =
// a_t lambda_t, dx_t = lambda_t (or (1 - a_t) lambda_t) and dg_t = mu_t h_{t-1} (or mu_t (h_{t-1} - x_t)).
//
// One pass over x, g and dout, last tile first (scan_tile.cuh).  mu is the same recurrence run backwards, so a span of
// tokens composes forwards for h and backwards for mu with one product A.  The states come from the checkpoint before
// each chunk of 64 tokens, so only mu is handed from tile to tile (and between the blocks of a cluster).  B=4 N=32 S=4096
// D=128, bf16 with fp32 gates (941 MB): 160 us where the load makes the clocks fall, 90 % of the measured copy rate, and
// 170 to 178 at full clocks, bound by HBM either way (what the blocks ask of the memory meets otherwise then).  One sequence of
// 32769 tokens and 640 channels, fp16, mixing (210 MB): 83 us, bound by a tile's latency.
#include "scan_tile.cuh"

namespace gdr {
namespace {
using namespace scan;

// 8 tokens of 2 channels a thread: decays, states and gradients of a segment, and the mixing form's 1 - a (it cannot be
// taken from a without losing the digits it has near 0), stay in 128 registers.  Without mixing, 16-bit types take 4
// channels where a tile is a whole warp wide.  (4 channels everywhere, and 4 tokens where that is too much, spilled: fp16
// mixing, 128 rows of 128 channels and 4096 tokens, 192 us against 135.)
constexpr int kSteps = 8;
constexpr int kResident = 2;  // blocks of an SM

// kWide: all 32 lanes of a warp lie over the channels, a segment is a warp and no shuffles are needed
template <typename T, typename G, int V, bool kWide> struct Layout {
    static constexpr int kCh = (kWide ? 32 : 16) * V;
    RawV<G, V> g[kSteps][kThreads];
    RawV<T, V> x[kSteps][kThreads], d[kSteps][kThreads];
    RawV<float, V> h[kThreads];  // the state before the segment's chunk
    float wa[2][kWarps][kCh], wf[2][kWarps][kCh], wr[2][kWarps][kCh];  // A and the forward and backward B of every warp
    float ca[2][kMaxRanks][kCh], cr[2][kMaxRanks][kCh];                // A and the backward B of every block of the cluster
    uint64_t arrived[2];                                               // their bytes
    uint64_t closed;                                                   // the bytes of sent[]
    int sent[kMaxRanks];                                               // tiles that each block has sent to this one
};

template <typename T, typename G, bool kMix, int V, bool kWide, bool kRows>
__global__ void __launch_bounds__(kThreads, kResident) scan_bwd_kernel(const ScanBwdArgs a, const Cut cut) {
    extern __shared__ __align__(16) unsigned char smem[];
    auto &sm = *reinterpret_cast<Layout<T, G, V, kWide> *>(smem);
    constexpr int P = kPairs<V>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lx = kWide ? 32 : cut.lx, cl = lane & (lx - 1);
    const int seg = kWide ? warp : tid / lx;
    const int R = cut.ranks, rank = (int)(blockIdx.x % R);
    const long long unit = blockIdx.x / R;
    const int slab = (int)(unit % cut.slabs);
    const long long bn = unit / cut.slabs;
    const int c0 = (slab * lx + cl) * V;
    const bool on = c0 < a.D;
    const int Lr = seq_len(a.lengths, (int)(bn / a.N), a.S);
    const unsigned L = Lr < 0 ? 0u : (unsigned)Lr, S = (unsigned)a.S;
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
    float2 mu[P];  // what the tokens behind the cluster's tiles pass back, the same in every block
    fill(mu, 0.f);
    if (on && a.dfinal_state && Lr >= 0) load_f32<V>(a.dfinal_state + (size_t)bn * a.D + c0, mu);

    const int TT = kSteps * (kThreads / lx);
    const unsigned step = (unsigned)R * TT;  // counted without sign: tiles may end past 2^31
    const int tiles = (int)((L + step - 1) / step);
    constexpr int kSegs = kChunk / kSteps;  // segments of a chunk
    const int chunk_warps = kSegs * lx > 32 ? kSegs * lx / 32 : 1;  // warps of a chunk: no warp holds more than one
    const unsigned exchange = (unsigned)(R * lx * V * 2 * sizeof(float));
    int got = tiles;  // tiles that this warp receives: fewer when a wait runs out
    if (R > 1) {
        if (tid == 0) {
            sm100::mbar_init(&sm.arrived[0], 1);
            sm100::mbar_init(&sm.arrived[1], 1);
            sm100::mbar_init(&sm.closed, 1);
            sm100::fence_mbar_init();
            sm100::mbar_arrive_expect_tx(&sm.closed, R * (unsigned)sizeof(int));
        }
        cluster_meet();
    }

    const int left = kRows ? a.D - slab * lx * V : 0;  // channels from the slab on
    auto fetch = [&](int k) {
        const unsigned w0 = k * step + rank * TT + warp * (32 / lx) * kSteps, t0 = k * step + rank * TT + seg * kSteps;
        const int nw = w0 < L ? (int)min(L - w0, 32u * kSteps) : 0;  // valid tokens of the warp, of the thread
        const int nt = on && t0 < L ? (int)min((unsigned)kSteps, L - t0) : 0;
        // by warps where rows are made of whole 16 bytes, but for narrow tiles whose vectors are 16 bytes anyway
        auto take = [&](auto &dst, const char *src, unsigned row, int size) {
            if (kRows && (kWide || size * V < 16))
                stage_rows<kSteps>(dst, src + (nw > 0 ? (size_t)w0 * row : 0) - cl * V * size, row, lx, nw, left * size);
            else
                stage_segment<kSteps>(dst, src + (nt > 0 ? (size_t)t0 * row : 0), row, nt);
        };
        take(sm.g, g, row_g, (int)sizeof(G));
        take(sm.x, x, row_x, (int)sizeof(T));
        take(sm.d, d, row_x, (int)sizeof(T));
        const unsigned chunk = t0 / kChunk;
        const bool has = on && chunk * kChunk < L;
        stage<RawV<float, V>, true>(&sm.h[tid], ck + (has ? (size_t)chunk * a.D : 0), has);
        stage_commit();
    };
    if (tiles > 0) fetch(tiles - 1);
    for (int n = 0; n < tiles; ++n) {
        const int k = tiles - 1 - n;
        const int p = n & 1;
        const unsigned t0 = k * step + rank * TT + seg * kSteps;
        // a segment forwards, (A, F): h -> A h + F, and backwards, (A, B): mu -> A mu + B; behind the sequence a = 1 and
        // x = dout = 0, which changes neither
        float2 av[kSteps][P], rest[kMix ? kSteps : 1][P], xv[kSteps][P], A[P], F[P], B[P];
        RawV<T, V> dr[kSteps];
        stage_wait();
        if (kRows) __syncwarp();
        float2 h[P];
        unpack<float, V>(sm.h[tid], h);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            float2 gv[P];
            unpack<G, V>(sm.g[j][tid], gv);
            unpack<T, V>(sm.x[j][tid], xv[j]);
            dr[j] = sm.d[j][tid];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 r;
                decay<kMix>(gv[i], av[j][i], r);
                if (kMix) rest[kMix ? j : 0][i] = r;
                const float2 b = kMix ? __fmul2_rn(xv[j][i], r) : xv[j][i];
                A[i] = j ? __fmul2_rn(A[i], av[j][i]) : av[j][i];
                F[i] = j ? __ffma2_rn(av[j][i], F[i], b) : b;
            }
        }
#pragma unroll
        for (int j = kSteps - 1; j >= 0; --j) {
            float2 dv[P];
            unpack<T, V>(dr[j], dv);
#pragma unroll
            for (int i = 0; i < P; ++i) B[i] = __fmul2_rn(av[j][i], j < kSteps - 1 ? __fadd2_rn(dv[i], B[i]) : dv[i]);
        }
        if (kRows) __syncwarp();
        if (k > 0) fetch(k - 1);  // what this thread (this warp) copied for itself is in registers
        // over the segments of the warp: (EA, EF) those before this one, (LA, LB) those behind it
        float2 EA[P], EF[P], LA[P], LB[P];
        if constexpr (!kWide) {
            float2 TA[P];
#pragma unroll
            for (int i = 0; i < P; ++i) TA[i] = LA[i] = A[i];
            for (int q = lx; q < 32; q *= 2) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float2 pa = shfl_up2(TA[i], q), pf = shfl_up2(F[i], q);
                    if (lane >= q) {
                        F[i] = __ffma2_rn(TA[i], pf, F[i]);
                        TA[i] = __fmul2_rn(TA[i], pa);
                    }
                    const float2 na = shfl_down2(LA[i], q), nb = shfl_down2(B[i], q);
                    if (lane + q < 32) {
                        B[i] = __ffma2_rn(LA[i], nb, B[i]);
                        LA[i] = __fmul2_rn(LA[i], na);
                    }
                }
            }
            if (lane >= 32 - lx) {
                store<float, V>(&sm.wa[p][warp][cl * V], TA);
                store<float, V>(&sm.wf[p][warp][cl * V], F);
            }
            if (lane < lx) store<float, V>(&sm.wr[p][warp][cl * V], B);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                EA[i] = shfl_up2(TA[i], lx);
                EF[i] = shfl_up2(F[i], lx);
                LA[i] = shfl_down2(LA[i], lx);
                LB[i] = shfl_down2(B[i], lx);
            }
        } else {
            store<float, V>(&sm.wa[p][warp][cl * V], A);
            store<float, V>(&sm.wf[p][warp][cl * V], F);
            store<float, V>(&sm.wr[p][warp][cl * V], B);
        }
        __syncthreads();
        if (R > 1) {  // as in the forward kernel, the block's backward map to every block of the cluster
            if (tid == 0 && n <= got) sm100::mbar_arrive_expect_tx(&sm.arrived[p], exchange);
            if (warp < R && lane < lx && n <= got) {
                float2 ta[P], tb[P];
                load_f32<V>(&sm.wa[p][kWarps - 1][cl * V], ta);
                load_f32<V>(&sm.wr[p][kWarps - 1][cl * V], tb);
#pragma unroll
                for (int w = kWarps - 2; w >= 0; --w) {
                    float2 wa[P], wb[P];
                    load_f32<V>(&sm.wa[p][w][cl * V], wa);
                    load_f32<V>(&sm.wr[p][w][cl * V], wb);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        tb[i] = __ffma2_rn(wa[i], tb[i], wb[i]);
                        ta[i] = __fmul2_rn(ta[i], wa[i]);
                    }
                }
                put_remote<V>(&sm.ca[p][rank][cl * V], &sm.arrived[p], warp, ta);
                put_remote<V>(&sm.cr[p][rank][cl * V], &sm.arrived[p], warp, tb);
            }
            __syncwarp();
        }
        // the state before the segment: the chunk's checkpoint, the chunk's warps before this one, its segments
        for (int w = warp & ~(chunk_warps - 1); w < warp; ++w) {
            float2 wa[P], wf[P];
            load_f32<V>(&sm.wa[p][w][cl * V], wa);
            load_f32<V>(&sm.wf[p][w][cl * V], wf);
#pragma unroll
            for (int i = 0; i < P; ++i) h[i] = __ffma2_rn(wa[i], h[i], wf[i]);
        }
        if (!kWide && lane >= lx) {
#pragma unroll
            for (int i = 0; i < P; ++i) h[i] = __ffma2_rn(EA[i], h[i], EF[i]);
        }
        // every token's h_{t-1} (less x_t) in the place of its x
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 q = kMix ? __ffma2_rn(xv[j][i], both(-1.f), h[i]) : h[i];
                h[i] = kMix ? __ffma2_rn(av[j][i], h[i], __fmul2_rn(xv[j][i], rest[kMix ? j : 0][i])) : __ffma2_rn(av[j][i], h[i], xv[j][i]);
                xv[j][i] = q;
            }
        if (R > 1 && n <= got && !__all_sync(0xffffffffu, wait_remote(&sm.arrived[p], (unsigned)(n >> 1) & 1u, a.wait_ns))) {
            got = n;
            raise_device_error(a.err, GDR_DEVERR_TIMEOUT);
        }
        // what comes back to this segment: from behind the tiles, the later blocks, the later warps, the later segments
        float2 m[P];
        if (R > 1) {
            for (int r = R - 1; r >= 0; --r) {
                if (r == rank) {
#pragma unroll
                    for (int i = 0; i < P; ++i) m[i] = mu[i];
                }
                float2 ra[P], rb[P];
                load_f32<V>(&sm.ca[p][r][cl * V], ra);
                load_f32<V>(&sm.cr[p][r][cl * V], rb);
#pragma unroll
                for (int i = 0; i < P; ++i) mu[i] = __ffma2_rn(ra[i], mu[i], rb[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) m[i] = mu[i];
        }
#pragma unroll
        for (int w = kWarps - 1; w > 0; --w) {
            if (w <= warp) break;
            float2 wa[P], wb[P];
            load_f32<V>(&sm.wa[p][w][cl * V], wa);
            load_f32<V>(&sm.wr[p][w][cl * V], wb);
#pragma unroll
            for (int i = 0; i < P; ++i) m[i] = __ffma2_rn(wa[i], m[i], wb[i]);
        }
        if (R == 1) {  // the whole tile: on through this warp and the earlier ones
#pragma unroll
            for (int i = 0; i < P; ++i) mu[i] = m[i];
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                if (w > warp) continue;
                float2 wa[P], wb[P];
                load_f32<V>(&sm.wa[p][w][cl * V], wa);
                load_f32<V>(&sm.wr[p][w][cl * V], wb);
#pragma unroll
                for (int i = 0; i < P; ++i) mu[i] = __ffma2_rn(wa[i], mu[i], wb[i]);
            }
        }
        if (!kWide && lane + lx < 32) {
#pragma unroll
            for (int i = 0; i < P; ++i) m[i] = __ffma2_rn(LA[i], m[i], LB[i]);
        }
        char *ox = dx + (size_t)t0 * row_x, *og = dg + (size_t)t0 * row_g;
        auto back = [&](int j, float2 (&rx)[P], float2 (&rg)[P]) {
            float2 dv[P];
            unpack<T, V>(dr[j], dv);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 lam = __fadd2_rn(dv[i], m[i]);
                m[i] = __fmul2_rn(av[j][i], lam);
                rx[i] = kMix ? __fmul2_rn(rest[kMix ? j : 0][i], lam) : lam;
                rg[i] = __fmul2_rn(m[i], xv[j][i]);
            }
        };
        if (on && t0 + kSteps <= L) {
#pragma unroll
            for (int j = kSteps - 1; j >= 0; --j) {
                float2 rx[P], rg[P];
                back(j, rx, rg);
                store<T, V>(ox + j * (size_t)row_x, rx);
                store<G, V>(og + j * (size_t)row_g, rg);
            }
        } else if (on) {
#pragma unroll
            for (int j = kSteps - 1; j >= 0; --j) {
                float2 rx[P], rg[P];
                back(j, rx, rg);
                if (t0 + j >= L) {
                    fill(rx, 0.f);
                    fill(rg, 0.f);
                }
                if (t0 + j < S) {
                    store<T, V>(ox + j * (size_t)row_x, rx);
                    store<G, V>(og + j * (size_t)row_g, rg);
                }
            }
        }
    }
    if (R > 1 && warp < R && lane == 0) tell_sent(&sm.sent[rank], &sm.closed, warp, got < tiles ? got + 1 : tiles);
    if (!on) return;
    float2 zero[P];
    fill(zero, 0.f);
    for (unsigned t = tiles * step + rank * (kThreads / lx) + seg; t < S; t += R * (kThreads / lx)) {
        store<T, V>(dx + (size_t)t * row_x, zero);
        store<G, V>(dg + (size_t)t * row_g, zero);
    }
    if (a.dinitial_state && seg == 0 && rank == 0) store<float, V>(a.dinitial_state + (size_t)bn * a.D + c0, mu);
    // thread 0 is still here: a slab has one channel at least
    if (R > 1 && tid == 0 && !all_landed(sm.arrived, &sm.closed, sm.sent, R, got, tiles, exchange / R, a.wait_ns))
        raise_device_error(a.err, GDR_DEVERR_TIMEOUT);
}

template <typename T, typename G, bool kMix, int V, bool kWide, bool kRows>
cudaError_t launch_v(const ScanBwdArgs &a, const Cut &cut, cudaStream_t s) {
    static LaunchCache cache(reinterpret_cast<const void *>(scan_bwd_kernel<T, G, kMix, V, kWide, kRows>));
    const int smem = (int)sizeof(Layout<T, G, V, kWide>);
    const cudaError_t e = cache.allow_smem(smem);
    if (e != cudaSuccess) return e;
    return launch_clusters(scan_bwd_kernel<T, G, kMix, V, kWide, kRows>, (long long)a.B * a.N, cut, smem, a, s);
}

template <typename T, typename G, bool kMix> cudaError_t launch_m(const ScanBwdArgs &a, cudaStream_t s) {
    auto cut = [&](int V, int max_lx, int min_lx) {
        return choose_cut((long long)a.B * a.N, a.D, V, a.S, kSteps, max_lx, min_lx, kResident, 0.78);
    };
    if (rows_of_16<T>(a.D)) {
        const Cut c = cut(2, 32, 4);
        if constexpr (sizeof(T) == 2 && !kMix) {
            const Cut c4 = cut(4, 32, 32);
            if (c4.estimate < 2 * c.estimate) return launch_v<T, G, kMix, 4, true, true>(a, c4, s);
        }
        return c.lx == 32 ? launch_v<T, G, kMix, 2, true, true>(a, c, s) : launch_v<T, G, kMix, 2, false, true>(a, c, s);
    }
    if (a.D % 2 == 0) return launch_v<T, G, kMix, 2, false, false>(a, cut(2, 16, 4), s);
    return launch_v<T, G, kMix, 1, false, false>(a, cut(1, 16, 4), s);
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
