// conv1d_bwd.cu -- the gradient of the depthwise causal conv1d + SiLU (gdr_conv1d_bwd).
//
// pre[u] = bias + sum_j w_j x[u - K + 1 + j];  dpre[u] = dy[u] silu'(pre[u]);
// dx[t] = sum_j w_j dpre[t + K - 1 - j];  dw_j = sum_u dpre[u] x[u - K + 1 + j];  db = sum_u dpre[u].
//
// One thread owns 4 channels and walks up to 128 tokens and the K - 1 behind them (whose dpre reaches back into its tokens),
// with a window of the last K inputs and of the last K dpre in registers.  The forward pass is computed again on the
// way, so x and dy are read and dx written once, apart from the K - 1 tokens at either end, which the neighbouring warps
// of the block read too.  Tokens come in batches of kBatch through a two-stage ring in shared memory (cp.async, every
// thread its own places: no barrier), and a batch is unrolled so that the windows move by renaming registers.  dw and db
// are summed per thread, over the four warps of a block (adjacent tokens) and, by a second kernel, over the blocks,
// always in the same order.  4 x 4096 tokens of 8192 channels: fp32 266 us, 92 % of the measured copy rate, bound by HBM;
// bf16 182 us under sustained load, 67 % (166 in short runs), bound by the latency of dependent arithmetic: the windows'
// registers leave 16 warps an SM, half of the issue slots and of the fp32 pipe stay empty.
#include "kernels.h"
#include "pairs.cuh"

namespace gdr {
namespace {

constexpr int kWarps = 4;             // warps of a block, adjacent in time
constexpr int kThreads = kWarps * 32;
// most tokens that a warp walks, which bounds the terms of a thread's sums
template <typename T> constexpr int kMaxSub = sizeof(T) == 2 ? 128 : 64;
constexpr int kBatch = 8;             // tokens of a stage
constexpr int V = 4;                  // channels of a thread
constexpr int P = V / 2;

// First element of channel group c0 of sequence b in dq, dk or dv (time 0), and that tensor's row length
template <typename T>
__device__ __forceinline__ const T *dy_base(const ConvBwdArgs &a, int b, int c0, int &row) {
    const int qk = a.Nk * a.Dk;
    const bool v = c0 >= 2 * qk;
    const void *p = v ? a.dv : c0 < qk ? a.dq : a.dk;
    const int c = v ? c0 - 2 * qk : c0 < qk ? c0 : c0 - qk;
    row = v ? a.Dv : a.Dk;
    const int head = c >> (31 - __clz(row));  // head sizes are powers of two
    return static_cast<const T *>(p) + ((size_t)b * (v ? a.Nv : a.Nk) + head) * a.S * row + (c & (row - 1));
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// silu'(p) = s (1 + p (1 - s)), s = 1 / (1 + e^{-p}): far left e^{-p} is infinite and s, and the whole, 0
__device__ __forceinline__ float2 silu_slope(float2 p) {
    float e0, e1, q0, q1;
    up2(__fmul2_rn(p, both(-1.4426950408889634f)), e0, e1);
    up2(__fadd2_rn(make_float2(ex2(e0), ex2(e1)), both(1.f)), q0, q1);
    const float2 s = make_float2(rcp(q0), rcp(q1));
    return __fmul2_rn(s, __ffma2_rn(p, __ffma2_rn(s, both(-1.f), both(1.f)), both(1.f)));
}

template <typename T> struct Stage {
    RawV<T, V> x[2][kBatch][kThreads], dy[2][kBatch][kThreads];
};

// blocks of an SM that the registers are capped for: windows, taps and sums of 4 channels take 16 K + 8 of them
template <typename T, int K> constexpr int kBlocks = K <= 4 ? 4 : 3;

template <typename T, int K>
__global__ void __launch_bounds__(kThreads, (kBlocks<T, K>)) conv1d_bwd_kernel(const ConvBwdArgs a, const int sub) {
    extern __shared__ __align__(16) unsigned char smem[];
    auto &sm = *reinterpret_cast<Stage<T> *>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = (blockIdx.x * 32 + lane) * V;
    const bool on = c0 < a.C;
    const int b = blockIdx.z;
    const int t0 = (blockIdx.y * kWarps + warp) * sub, t1 = min(t0 + sub, a.S);
    const int Lr = a.lengths ? a.lengths[b] : a.S;
    const bool bad = Lr < 0 || Lr > a.S;
    if (bad && blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) raise_device_error(a.err, GDR_DEVERR_LENGTH);
    const int L = bad ? 0 : Lr;

    float2 dw[K][P], db[P];
    fill(db, 0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) fill(dw[j], 0.f);
    const bool first = t0 == 0;  // also answers for the history before position 0
    if (on && (t0 < t1 || first)) {
        int row;
        const T *dy = dy_base<T>(a, b, c0, row);
        const T *x = static_cast<const T *>(a.x) + (size_t)b * a.S * a.C + c0;
        T *dx = static_cast<T *>(a.dx) + (size_t)b * a.S * a.C + c0;
        const size_t state = ((size_t)b * a.C + c0) * K;
        const T *ds_out = a.dstate_out && !bad ? static_cast<const T *>(a.dstate_out) + state : nullptr;
        T *ds_in = first && a.dstate_in ? static_cast<T *>(a.dstate_in) + state : nullptr;

        const int end = t1 + K - 1;  // tokens t0 .. end - 1 are walked; those from L on count as zeros
        auto fetch = [&](int u, int s) {
            const int n = max(0, min(min(kBatch, end - u), L - u));
            const size_t at = n > 0 ? (size_t)u : 0;
            stage_segment<kBatch>(sm.x[s], x + at * a.C, (unsigned)a.C * (unsigned)sizeof(T), n);
            stage_segment<kBatch>(sm.dy[s], dy + at * row, (unsigned)row * (unsigned)sizeof(T), n);
            stage_commit();
        };
        fetch(t0, 0);
        fetch(t0 + kBatch, 1);

        float2 w[K][P], bias[P], win[K - 1 + kBatch][P], dwin[K - 1 + kBatch][P];
        fill(bias, 0.f);
        if (a.bias) unpack<T, V>(*reinterpret_cast<const RawV<T, V> *>(static_cast<const T *>(a.bias) + c0), bias);
        {
            alignas(16) T taps[V * K];  // the thread's rows of the weight are adjacent
#pragma unroll
            for (int j = 0; j < K; ++j)
                reinterpret_cast<RawV<T, V> *>(taps)[j] =
                    reinterpret_cast<const RawV<T, V> *>(static_cast<const T *>(a.w) + (size_t)c0 * K)[j];
#pragma unroll
            for (int j = 0; j < K; ++j)
#pragma unroll
                for (int i = 0; i < P; ++i) w[j][i] = make_float2(to_f32(taps[2 * i * K + j]), to_f32(taps[(2 * i + 1) * K + j]));
        }
        // win[j], j < K - 1: the inputs before the batch (position u - K + 1 + j at its first token u); dwin the same
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            fill(dwin[j], 0.f);
            fill(win[j], 0.f);
            const int at = t0 - K + 1 + j;
            if (at >= 0) {
                if (at < L) unpack<T, V>(*reinterpret_cast<const RawV<T, V> *>(x + (size_t)at * a.C), win[j]);
            } else if (a.state_in && L > 0) {
                const T *s = static_cast<const T *>(a.state_in) + state;
#pragma unroll
                for (int i = 0; i < P; ++i) win[j][i] = make_float2(to_f32(s[2 * i * K + at + K]), to_f32(s[(2 * i + 1) * K + at + K]));
            }
        }
        // the oldest history entry is no input of the conv; it is passed on where the sequence is empty
        if (ds_in)
#pragma unroll
            for (int i = 0; i < V; ++i) ds_in[i * K] = from_f32<T>(ds_out && L == 0 ? to_f32(ds_out[i * K]) : 0.f);

        // token u, at place j of the windows, its inputs at place p of stage s; whole: an ordinary one of the thread's
        // tokens; halo: an ordinary one behind them.  What lies behind the sequence is told by its place, not by its zeros:
        // the windows there still hold the last inputs, whose products may overflow.
        auto step = [&](int u, int j, int s, int p, bool whole, bool halo) {
            float2 g[P];
            unpack<T, V>(sm.x[s][p][tid], win[K - 1 + j]);
            unpack<T, V>(sm.dy[s][p][tid], g);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 pre = bias[i];
#pragma unroll
                for (int q = 0; q < K; ++q) pre = __ffma2_rn(w[q][i], win[j + q][i], pre);
                const float2 d = whole || halo || u < L ? __fmul2_rn(g[i], silu_slope(pre)) : both(0.f);
                dwin[K - 1 + j][i] = d;
                if (whole || (!halo && u < t1 && u < L)) {
                    db[i] = __fadd2_rn(db[i], d);
#pragma unroll
                    for (int q = 0; q < K; ++q) dw[q][i] = __ffma2_rn(d, win[j + q][i], dw[q][i]);
                }
            }
            const int t = u - K + 1;  // its last dpre has arrived
            float2 r[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                r[i] = __fmul2_rn(w[0][i], dwin[j + K - 1][i]);
#pragma unroll
                for (int q = 1; q < K; ++q) r[i] = __ffma2_rn(w[q][i], dwin[j + K - 1 - q][i], r[i]);
            }
            if (!whole && !halo && max(t, 0) >= L) fill(r, 0.f);  // no token of the sequence takes part
            if (!whole && !halo && ds_out && t >= L - K && t < L) {
                // the new state is the history from place L on: place q of it is position L - K + q
#pragma unroll
                for (int i = 0; i < P; ++i)
                    r[i] = __fadd2_rn(r[i], make_float2(to_f32(ds_out[2 * i * K + t - L + K]), to_f32(ds_out[(2 * i + 1) * K + t - L + K])));
            }
            if ((whole && j >= K - 1) || halo || t >= t0) {
                store<T, V>(dx + (size_t)t * a.C, r);
            } else if (!whole && !halo && ds_in) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    float lo, hi;
                    up2(r[i], lo, hi);
                    ds_in[2 * i * K + t + K] = from_f32<T>(lo);
                    ds_in[(2 * i + 1) * K + t + K] = from_f32<T>(hi);
                }
            }
        };
        auto shift = [&](int by) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    win[j][i] = win[by + j][i];
                    dwin[j][i] = dwin[by + j][i];
                }
        };
        const int ordinary = ds_out ? L - 1 : L;  // tokens before it complete none that takes part in the new state
        const int reach = min(end, L + K - 1);    // tokens from here on complete padding only
        int u = t0, s = 0;
#pragma unroll 1
        for (; u < reach; u += kBatch, s ^= 1) {
            stage_wait_but_one();
            // every token of the batch is one of the thread's and of the sequence, and none that it completes lies before
            // the sequence or takes part in the new state
            if ((u > t0 || !first) && u + kBatch <= t1 && u + kBatch <= ordinary) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) step(u + j, j, s, j, true, false);
                shift(kBatch);
            } else if (u == t1 && u >= t0 + kBatch && u + K - 1 <= ordinary) {  // the last K - 1
#pragma unroll
                for (int j = 0; j < K - 1; ++j) step(u + j, j, s, j, false, true);
            } else {
#pragma unroll 1
                for (int j = 0; j < kBatch && u + j < end; ++j) {
                    step(u + j, 0, s, j, false, false);
                    shift(1);
                }
            }
            fetch(u + 2 * kBatch, s);
        }
        float2 zero[P];
        fill(zero, 0.f);
        for (int t = max(u - K + 1, t0); t < t1; ++t) store<T, V>(dx + (size_t)t * a.C, zero);
    }
    if (!a.partial) return;
    __shared__ float2 part[kWarps - 1][K + 1][P][32];
    if (warp > 0)
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
            for (int j = 0; j < K; ++j) part[warp - 1][j][i][lane] = dw[j][i];
            part[warp - 1][K][i][lane] = db[i];
        }
    __syncthreads();
    if (warp == 0 && on) {
        float *p = a.partial + ((size_t)(b * gridDim.y + blockIdx.y) * (K + 1)) * a.C + c0;
#pragma unroll
        for (int j = 0; j <= K; ++j) {
            float2 r[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                r[i] = j < K ? dw[j < K ? j : 0][i] : db[i];
#pragma unroll
                for (int q = 0; q < kWarps - 1; ++q) r[i] = __fadd2_rn(r[i], part[q][j][i][lane]);
            }
            store<float, V>(p + (size_t)j * a.C, r);
        }
    }
}

// Adds the partial sums of all blocks: 32 channels of one tap a block, 8 lanes of 4 channels beside one another and 32
// strides of the rows.  It may be launched while the kernel before it still runs, and waits for its end.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) conv1d_bwd_sum_kernel(const float *partial, int rows, int C, int K, float *dw,
                                                                     float *db) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int group = threadIdx.x & 7, stride = threadIdx.x >> 3;
    const int c = blockIdx.x * 32 + group * 4, j = blockIdx.y;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < C)  // C is a multiple of 16
        for (int r = stride; r < rows; r += 32) {
            const float4 v = *reinterpret_cast<const float4 *>(partial + ((size_t)r * (K + 1) + j) * C + c);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
    __shared__ float part[32][33];
    part[stride][group * 4] = s.x;
    part[stride][group * 4 + 1] = s.y;
    part[stride][group * 4 + 2] = s.z;
    part[stride][group * 4 + 3] = s.w;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int cw = warp * 4 + k, at = blockIdx.x * 32 + cw;
        const float t = warp_sum(part[lane][cw]);
        if (lane == 0 && at < C) {
            if (j < K) dw[(size_t)at * K + j] = t;
            else if (db) db[at] = t;
        }
    }
}

__global__ void zero_f32_kernel(float *p, size_t n) {
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) p[i] = 0.f;
}

// Tokens a warp walks: as many as pay for its beginning (4 x 4096 tokens of 8192 channels, sustained, us: bf16 182 with
// 128 tokens, 190 with 64 and 207 with 32, fp32 266 with 64 and 276 with 32).  Fewer, down to 16, where the blocks would
// not give every SM two -- the walk is the call's latency then, and the K - 1 tokens read twice cost nothing (1 x 4096
// tokens of 384 channels, bf16, in a graph: 10.5 us with 16, 10.8 with 32, 14.6 with 64) -- or where that leaves fewer
// warps without tokens.
int sub_for(int B, int S, int C, int most) {
    const long long groups = (long long)B * ((C + 32 * V - 1) / (32 * V));
    auto blocks = [&](int sub) { return (S + (long long)kWarps * sub - 1) / (kWarps * sub); };
    int sub = most;
    while (sub > 16 && (groups * blocks(sub) < 2 * sm_count() || blocks(sub / 2) * 9 <= blocks(sub) * 16)) sub /= 2;
    return sub;
}
// blocks along the tokens: at most 65535, of at least 64 tokens each, since S <= 65535 * 64
int tiles(int S, int sub) { return (int)((S + (long long)kWarps * sub - 1) / (kWarps * sub)); }

template <typename T, int K>
cudaError_t launch_tk(const ConvBwdArgs &a, cudaStream_t s) {
    static LaunchCache cache(reinterpret_cast<const void *>(conv1d_bwd_kernel<T, K>));
    const int smem = (int)sizeof(Stage<T>);
    cudaError_t e = cache.allow_smem(smem);
    if (e != cudaSuccess) return e;
    const unsigned gx = (unsigned)((a.C + 32 * V - 1) / (32 * V));
    const int sub = sub_for(a.B, a.S, a.C, kMaxSub<T>);
    const unsigned gy = (unsigned)(a.S > 0 ? tiles(a.S, sub) : 1);  // without tokens, the state's gradient alone
    conv1d_bwd_kernel<T, K><<<dim3(gx, gy, a.B), kThreads, smem, s>>>(a, sub);
    e = cudaGetLastError();
    if (e != cudaSuccess || !a.partial) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.C + 31) / 32), K + 1);
    cfg.blockDim = dim3(kSumThreads);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, conv1d_bwd_sum_kernel, static_cast<const float *>(a.partial), (int)(a.B * gy), a.C, K, a.dw,
                              a.db);
}

template <typename T>
cudaError_t launch_t(const ConvBwdArgs &a, int K, cudaStream_t s) {
    switch (K) {
        case 1: return launch_tk<T, 1>(a, s);
        case 2: return launch_tk<T, 2>(a, s);
        case 3: return launch_tk<T, 3>(a, s);
        case 4: return launch_tk<T, 4>(a, s);
        case 5: return launch_tk<T, 5>(a, s);
        case 6: return launch_tk<T, 6>(a, s);
        case 7: return launch_tk<T, 7>(a, s);
        case 8: return launch_tk<T, 8>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

size_t conv1d_bwd_workspace(int B, int S, int C, int K) {
    return (size_t)B * tiles(S, sub_for(B, S, C, kMaxSub<float>)) * (K + 1) * C * sizeof(float);  // the most of any type
}

cudaError_t launch_conv1d_bwd(const ConvBwdArgs &a, int K, gdr_dtype dt, cudaStream_t s) {
    if ((long long)a.B * a.S == 0) {  // nothing to sum
        const size_t n = (size_t)a.C * K;
        zero_f32_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a.dw, n);
        if (a.db) zero_f32_kernel<<<(unsigned)((a.C + 255) / 256), 256, 0, s>>>(a.db, (size_t)a.C);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || a.B == 0 || !a.dstate_in) return e;
    }
    if (dt == GDR_BF16) return launch_t<__nv_bfloat16>(a, K, s);
    if (dt == GDR_F16) return launch_t<__half>(a, K, s);
    return launch_t<float>(a, K, s);
}

}  // namespace gdr
