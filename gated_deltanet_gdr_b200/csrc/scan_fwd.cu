// scan_fwd.cu -- the gated linear recurrence over a sequence (gdr_scan_fwd): h_t = a_t h_{t-1} + b_t per channel, a_t =
// exp(g_t), b_t = x_t or (1 - a_t) x_t.
//
// One pass over x and g (scan_tile.cuh), 8 tokens of 4 channels a thread (fewer channels where rows are not made of
// whole vectors).  The next tile's inputs are on their way (cp.async) while a tile is composed and written: two blocks
// of 48 to 64 KB in flight an SM.  B=4 N=32 S=4096 D=128, bf16 with fp32 gates (537 MB): 96 us under sustained load, 85 %
// of the measured copy rate (87 us in runs too short for the clocks to fall), bound by HBM with the issue slots at 57 %.
// One sequence of 32769 tokens and 640 channels, fp16, mixing (126 MB): 55 us, bound by a tile's latency: 11 rounds of
// clusters of 6, each a load, a composition, an exchange and a store that wait for one another.
#include "scan_tile.cuh"

namespace gdr {
namespace {
using namespace scan;

constexpr int kSteps = 8;  // tokens of a thread in a tile

// kWide: all 32 lanes of a warp lie over the channels, a segment is a warp and no shuffles are needed
template <typename T, typename G, int V, bool kWide> struct Layout {
    static constexpr int kCh = (kWide ? 32 : 16) * V;  // most channels of a tile
    RawV<G, V> g[kSteps][kThreads];
    RawV<T, V> x[kSteps][kThreads];
    float wa[2][kWarps][kCh], wb[2][kWarps][kCh];        // (A, B) of every warp, for even and odd tiles
    float ca[2][kMaxRanks][kCh], cb[2][kMaxRanks][kCh];  // (A, B) of every block of the cluster
    uint64_t arrived[2];                                 // their bytes
    uint64_t closed;                                     // the bytes of sent[]
    int sent[kMaxRanks];                                 // tiles that each block has sent to this one
};

template <typename T, typename G, bool kMix, int V, bool kWide, bool kRows>
__global__ void __launch_bounds__(kThreads, 2) scan_fwd_kernel(const ScanArgs a, const Cut cut) {
    extern __shared__ __align__(16) unsigned char smem[];
    auto &sm = *reinterpret_cast<Layout<T, G, V, kWide> *>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lx = kWide ? 32 : cut.lx, cl = lane & (lx - 1);
    const int seg = kWide ? warp : tid / lx;  // lanes of a segment are adjacent
    const int R = cut.ranks, rank = (int)(blockIdx.x % R);
    const long long unit = blockIdx.x / R;
    const int slab = (int)(unit % cut.slabs);
    const long long bn = unit / cut.slabs;
    const int c0 = (slab * lx + cl) * V;
    const bool on = c0 < a.D;
    const int Lr = seq_len(a.lengths, (int)(bn / a.N), a.S);
    const unsigned L = Lr < 0 ? 0u : (unsigned)Lr, S = (unsigned)a.S;
    if (Lr < 0 && tid == 0 && rank == 0) raise_device_error(a.err, GDR_DEVERR_LENGTH);

    constexpr int P = kPairs<V>;
    const unsigned row_x = (unsigned)a.D * sizeof(T), row_g = (unsigned)a.D * sizeof(G);  // D <= 2^26
    const size_t base = (size_t)bn * a.S * a.D + c0;
    const char *x = reinterpret_cast<const char *>(static_cast<const T *>(a.x) + base);
    const char *g = reinterpret_cast<const char *>(static_cast<const G *>(a.g) + base);
    char *out = reinterpret_cast<char *>(static_cast<T *>(a.out) + base);
    float2 h[P];  // the state at the start of the cluster's next tiles, the same in every block
    fill(h, 0.f);
    if (on && a.initial_state) load_f32<V>(a.initial_state + (size_t)bn * a.D + c0, h);
    const int chunks = (a.S + kChunk - 1) / kChunk;
    float *ck = a.checkpoints ? a.checkpoints + (size_t)bn * chunks * a.D + c0 : nullptr;
    // an empty sequence makes no tile; its first checkpoint is its state
    if (L == 0 && Lr == 0 && ck && on && seg == 0 && rank == 0 && a.S > 0) store<float, V>(ck, h);

    const int TT = kSteps * (kThreads / lx);
    const unsigned step = (unsigned)R * TT;  // tokens of the cluster's tiles; counted without sign, they may end past 2^31
    const int tiles = (int)((L + step - 1) / step);
    const unsigned exchange = (unsigned)(R * lx * V * 2 * sizeof(float));  // bytes of a tile's (A, B) of all blocks
    int got = tiles;  // tiles that this warp receives: fewer when a wait runs out
    if (R > 1) {
        if (tid == 0) {
            sm100::mbar_init(&sm.arrived[0], 1);
            sm100::mbar_init(&sm.arrived[1], 1);
            sm100::mbar_init(&sm.closed, 1);
            sm100::fence_mbar_init();
            sm100::mbar_arrive_expect_tx(&sm.closed, R * (unsigned)sizeof(int));
        }
        cluster_meet();  // every block of the cluster has started, with its barriers ready
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
        stage_commit();
    };
    if (tiles > 0) fetch(0);
    for (int k = 0; k < tiles; ++k) {
        const int p = k & 1;
        const unsigned t0 = k * step + rank * TT + seg * kSteps;
        // decays and writes of the segment (tokens behind the sequence: a = 1, b = 0), and the segment as a whole
        float2 av[kSteps][P], bv[kSteps][P], A[P], B[P];
        stage_wait();
        if (kRows) __syncwarp();
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            float2 gv[P];
            unpack<G, V>(sm.g[j][tid], gv);
            unpack<T, V>(sm.x[j][tid], bv[j]);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 rest;
                decay<kMix>(gv[i], av[j][i], rest);
                if (kMix) bv[j][i] = __fmul2_rn(bv[j][i], rest);
                A[i] = j ? __fmul2_rn(A[i], av[j][i]) : av[j][i];
                B[i] = j ? __ffma2_rn(av[j][i], B[i], bv[j][i]) : bv[j][i];
            }
        }
        if (kRows) __syncwarp();
        if (k + 1 < tiles) fetch(k + 1);  // what this thread (this warp) copied for itself is in registers
        // inclusive composition over the segments of the warp; (EA, EB): the segments before this one
        float2 EA[P], EB[P];
        fill(EA, 1.f);
        fill(EB, 0.f);
        if (!kWide) {
            for (int d = lx; d < 32; d *= 2) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float2 pa = shfl_up2(A[i], d), pb = shfl_up2(B[i], d);
                    if (lane >= d) {
                        B[i] = __ffma2_rn(A[i], pb, B[i]);
                        A[i] = __fmul2_rn(A[i], pa);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 pa = shfl_up2(A[i], lx), pb = shfl_up2(B[i], lx);
                if (lane >= lx) {
                    EA[i] = pa;
                    EB[i] = pb;
                }
            }
        }
        if (lane >= 32 - lx) {  // the warp's last segment holds the whole warp
            store<float, V>(&sm.wa[p][warp][cl * V], A);
            store<float, V>(&sm.wb[p][warp][cl * V], B);
        }
        __syncthreads();
        if (R > 1) {
            // the block as a whole to every block of the cluster, one warp for each.  A block writes a place again two
            // tiles on, having received the tile between, which its owner sent after reading this one.
            if (tid == 0 && k <= got) sm100::mbar_arrive_expect_tx(&sm.arrived[p], exchange);
            if (warp < R && lane < lx && k <= got) {
                float2 ta[P], tb[P];
                load_f32<V>(&sm.wa[p][0][cl * V], ta);
                load_f32<V>(&sm.wb[p][0][cl * V], tb);
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    float2 wa[P], wb[P];
                    load_f32<V>(&sm.wa[p][w][cl * V], wa);
                    load_f32<V>(&sm.wb[p][w][cl * V], wb);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        tb[i] = __ffma2_rn(wa[i], tb[i], wb[i]);
                        ta[i] = __fmul2_rn(ta[i], wa[i]);
                    }
                }
                put_remote<V>(&sm.ca[p][rank][cl * V], &sm.arrived[p], warp, ta);
                put_remote<V>(&sm.cb[p][rank][cl * V], &sm.arrived[p], warp, tb);
            }
            __syncwarp();
            if (k <= got && !__all_sync(0xffffffffu, wait_remote(&sm.arrived[p], (unsigned)(k >> 1) & 1u, a.wait_ns))) {
                got = k;
                raise_device_error(a.err, GDR_DEVERR_TIMEOUT);
            }
        }
        // the state this thread starts from: the tile's start, the blocks and warps before it, its warp's segments
        float2 hs[P];
#pragma unroll
        for (int i = 0; i < P; ++i) hs[i] = h[i];
        for (int r = 0; r < (R > 1 ? R : 0); ++r) {
            float2 ra[P], rb[P];
            load_f32<V>(&sm.ca[p][r][cl * V], ra);
            load_f32<V>(&sm.cb[p][r][cl * V], rb);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                h[i] = __ffma2_rn(ra[i], h[i], rb[i]);
                if (r < rank) hs[i] = h[i];
            }
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (R > 1 && w >= warp) break;
            float2 wa[P], wb[P];
            load_f32<V>(&sm.wa[p][w][cl * V], wa);
            load_f32<V>(&sm.wb[p][w][cl * V], wb);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (R > 1) {
                    hs[i] = __ffma2_rn(wa[i], hs[i], wb[i]);
                } else {
                    h[i] = __ffma2_rn(wa[i], h[i], wb[i]);
                    if (w < warp) hs[i] = h[i];
                }
            }
        }
        if (!kWide) {
#pragma unroll
            for (int i = 0; i < P; ++i) hs[i] = __ffma2_rn(EA[i], hs[i], EB[i]);
        }
        if (on && t0 < S) {
            // segments are kSteps long and tiles a multiple of 64: a chunk starts where a segment does
            if (ck && (t0 & (kChunk - 1)) == 0 && t0 < L) store<float, V>(ck + (size_t)(t0 / kChunk) * a.D, hs);
            char *o = out + (size_t)t0 * row_x;
            if (t0 + kSteps <= L) {
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
#pragma unroll
                    for (int i = 0; i < P; ++i) hs[i] = __ffma2_rn(av[j][i], hs[i], bv[j][i]);
                    store<T, V>(o + j * (size_t)row_x, hs);
                }
            } else {
                const int n = (int)min((unsigned)kSteps, S - t0), nv = t0 < L ? (int)(L - t0) : 0;
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
#pragma unroll
                    for (int i = 0; i < P; ++i) hs[i] = j < nv ? __ffma2_rn(av[j][i], hs[i], bv[j][i]) : both(0.f);
                    if (j < n) store<T, V>(o + j * (size_t)row_x, hs);
                }
            }
        }
    }
    if (R > 1 && warp < R && lane == 0) tell_sent(&sm.sent[rank], &sm.closed, warp, got < tiles ? got + 1 : tiles);
    if (!on) return;
    // tokens behind the last tile
    float2 zero[P];
    fill(zero, 0.f);
    for (unsigned t = tiles * step + rank * (kThreads / lx) + seg; t < S; t += R * (kThreads / lx))
        store<T, V>(out + (size_t)t * row_x, zero);
    if (a.final_state && Lr >= 0 && seg == 0 && rank == 0) store<float, V>(a.final_state + (size_t)bn * a.D + c0, h);
    // thread 0 is still here: a slab has one channel at least
    if (R > 1 && tid == 0 && !all_landed(sm.arrived, &sm.closed, sm.sent, R, got, tiles, exchange / R, a.wait_ns))
        raise_device_error(a.err, GDR_DEVERR_TIMEOUT);
}

template <typename T, typename G, bool kMix, int V, bool kWide, bool kRows>
cudaError_t launch_v(const ScanArgs &a, const Cut &cut, cudaStream_t s) {
    static LaunchCache cache(reinterpret_cast<const void *>(scan_fwd_kernel<T, G, kMix, V, kWide, kRows>));
    const int smem = (int)sizeof(Layout<T, G, V, kWide>);
    const cudaError_t e = cache.allow_smem(smem);
    if (e != cudaSuccess) return e;
    return launch_clusters(scan_fwd_kernel<T, G, kMix, V, kWide, kRows>, (long long)a.B * a.N, cut, smem, a, s);
}

template <typename T, typename G, bool kMix> cudaError_t launch_m(const ScanArgs &a, cudaStream_t s) {
    auto cut = [&](int V, int max_lx) { return choose_cut((long long)a.B * a.N, a.D, V, a.S, kSteps, max_lx, 4, 2, 0.85); };
    if (rows_of_16<T>(a.D)) {
        const Cut c = cut(4, 32);
        return c.lx == 32 ? launch_v<T, G, kMix, 4, true, true>(a, c, s) : launch_v<T, G, kMix, 4, false, true>(a, c, s);
    }
    if (a.D % 4 == 0) return launch_v<T, G, kMix, 4, false, false>(a, cut(4, 16), s);
    if (a.D % 2 == 0) return launch_v<T, G, kMix, 2, false, false>(a, cut(2, 16), s);
    return launch_v<T, G, kMix, 1, false, false>(a, cut(1, 16), s);
}
template <typename T, typename G> cudaError_t launch_t(const ScanArgs &a, cudaStream_t s) {
    return a.mode == GDR_SCAN_MIX ? launch_m<T, G, true>(a, s) : launch_m<T, G, false>(a, s);
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs &a, gdr_dtype dt, gdr_dtype gt, cudaStream_t s) {
    if (dt == GDR_F32) return launch_t<float, float>(a, s);
    if (dt == GDR_BF16) return gt == dt ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, s) : launch_t<__nv_bfloat16, float>(a, s);
    return gt == dt ? launch_t<__half, __half>(a, s) : launch_t<__half, float>(a, s);
}

}  // namespace gdr
