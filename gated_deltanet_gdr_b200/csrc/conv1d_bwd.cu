// conv1d_bwd.cu -- the gradient of the depthwise causal conv1d + SiLU (gdr_conv1d_bwd).
//
// pre[u] = bias + sum_j w_j x[u - K + 1 + j];  dpre[u] = dy[u] silu'(pre[u]);
// dx[t] = sum_j w_j dpre[t + K - 1 - j];  dw_j = sum_u dpre[u] x[u - K + 1 + j];  db = sum_u dpre[u].
//
// One thread owns 4 channels and walks kSub tokens and the K - 1 behind them (whose dpre reaches back into its tokens),
// with a window of the last K inputs and of the last K dpre.  The forward pass is computed again on the way, so x, dy
// are read and dx written once, apart from the K - 1 tokens at either end.  dw and db are summed per thread, over the
// four warps of a block (adjacent tokens) and, by a second kernel, over the blocks, always in the same order.
#include "common.cuh"
#include "kernels.h"

namespace gdr {
namespace {

constexpr int kWarps = 4;            // warps of a block, adjacent in time
constexpr int kSub = 64;             // tokens a warp walks
constexpr int kTile = kWarps * kSub; // tokens of a block
constexpr int V = 4;                 // channels of a thread

template <typename T> __device__ __forceinline__ void load4(const T *p, float (&x)[V]);
template <> __device__ __forceinline__ void load4<float>(const float *p, float (&x)[V]) {
    const float4 f = *reinterpret_cast<const float4 *>(p);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
}
template <> __device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[V]) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
    const float2 a = __bfloat1622float2(h[0]), b = __bfloat1622float2(h[1]);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
template <> __device__ __forceinline__ void load4<__half>(const __half *p, float (&x)[V]) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const __half2 *h = reinterpret_cast<const __half2 *>(&u);
    const float2 a = __half22float2(h[0]), b = __half22float2(h[1]);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
template <typename T> __device__ __forceinline__ void store4(T *p, const float (&x)[V]);
template <> __device__ __forceinline__ void store4<float>(float *p, const float (&x)[V]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, const float (&x)[V]) {
    __nv_bfloat162 h[2] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(h);
}
template <> __device__ __forceinline__ void store4<__half>(__half *p, const float (&x)[V]) {
    __half2 h[2] = {__floats2half2_rn(x[0], x[1]), __floats2half2_rn(x[2], x[3])};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(h);
}

// First element of channel group c0 of sequence b in dq, dk or dv (time 0), and that tensor's row length
template <typename T>
__device__ __forceinline__ const T *dy_base(const ConvBwdArgs &a, int b, int c0, int &row) {
    const int qk = a.Nk * a.Dk;
    if (c0 < 2 * qk) {
        const void *p = c0 < qk ? a.dq : a.dk;
        const int c = c0 < qk ? c0 : c0 - qk;
        row = a.Dk;
        return static_cast<const T *>(p) + ((size_t)b * a.Nk + c / a.Dk) * a.S * a.Dk + c % a.Dk;
    }
    const int c = c0 - 2 * qk;
    row = a.Dv;
    return static_cast<const T *>(a.dv) + ((size_t)b * a.Nv + c / a.Dv) * a.S * a.Dv + c % a.Dv;
}

// value of the history (state followed by x) at index i of sequence b, channel c: i < K from the state
template <typename T, int K>
__device__ __forceinline__ float hist_at(const ConvBwdArgs &a, int b, int c, int i) {
    if (i < K) return a.state_in ? to_f32(static_cast<const T *>(a.state_in)[((size_t)b * a.C + c) * K + i]) : 0.f;
    return to_f32(static_cast<const T *>(a.x)[((size_t)b * a.S + (i - K)) * a.C + c]);
}

template <typename T, int K>
__global__ void __launch_bounds__(kWarps * 32) conv1d_bwd_kernel(const ConvBwdArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = (blockIdx.x * 32 + lane) * V;
    const bool on = c0 < a.C;
    const int b = blockIdx.z;
    const int t0 = blockIdx.y * kTile + warp * kSub, t1 = min(t0 + kSub, a.S);
    const int Lr = a.lengths ? a.lengths[b] : a.S;
    const bool bad = Lr < 0 || Lr > a.S;
    if (bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) raise_device_error(a.err, GDR_DEVERR_LENGTH);
    const int L = bad ? 0 : Lr;

    float dw[K][V] = {}, db[V] = {};
    const bool first = t0 == 0;  // also answers for the history before position 0
    if (on && (t0 < t1 || first)) {
        int row;
        const T *dy = dy_base<T>(a, b, c0, row);
        const T *x = static_cast<const T *>(a.x) + (size_t)b * a.S * a.C + c0;
        T *dx = static_cast<T *>(a.dx) + (size_t)b * a.S * a.C + c0;
        const T *ds_out = a.dstate_out && !bad ? static_cast<const T *>(a.dstate_out) + ((size_t)b * a.C + c0) * K : nullptr;
        T *ds_in = first && a.dstate_in ? static_cast<T *>(a.dstate_in) + ((size_t)b * a.C + c0) * K : nullptr;
        float w[K][V], win[K][V], dwin[K][V], bias[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = a.bias ? to_f32(static_cast<const T *>(a.bias)[c0 + i]) : 0.f;
#pragma unroll
            for (int j = 0; j < K; ++j) {
                w[j][i] = to_f32(static_cast<const T *>(a.w)[(size_t)(c0 + i) * K + j]);
                dwin[j][i] = 0.f;
                // win[j] holds position u - K + 1 + j at step u: one short of it before the first step
                win[j][i] = t0 < L && j > 0 ? hist_at<T, K>(a, b, c0 + i, t0 + j) : 0.f;
            }
        }
        // the oldest history entry is no input of the conv; it is passed on where the sequence is empty
        if (ds_in)
#pragma unroll
            for (int i = 0; i < V; ++i) ds_in[i * K] = from_f32<T>(ds_out && L == 0 ? to_f32(ds_out[i * K]) : 0.f);
        for (int u = t0; u < t1 + K - 1; ++u) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    win[j][i] = win[j + 1][i];
                    dwin[j][i] = dwin[j + 1][i];
                }
#pragma unroll
            for (int i = 0; i < V; ++i) dwin[K - 1][i] = 0.f;
            if (u < L) {
                float g[V];
                load4(x + (size_t)u * a.C, win[K - 1]);
                load4(dy + (size_t)u * row, g);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float p = bias[i];
#pragma unroll
                    for (int j = 0; j < K; ++j) p = fmaf(w[j][i], win[j][i], p);
                    const float s = 1.f / (1.f + expf(-p));
                    const float d = g[i] * (s * fmaf(p, 1.f - s, 1.f));
                    dwin[K - 1][i] = d;
                    if (u < t1) {
                        db[i] += d;
#pragma unroll
                        for (int j = 0; j < K; ++j) dw[j][i] = fmaf(d, win[j][i], dw[j][i]);
                    }
                }
            }
            const int t = u - K + 1;  // its last dpre has arrived
            float r[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                r[i] = 0.f;
#pragma unroll
                for (int j = 0; j < K; ++j) r[i] = fmaf(w[j][i], dwin[K - 1 - j][i], r[i]);
                // the new state is the history from place L on: place j of it is position L - K + j
                if (ds_out && t >= L - K && t < L) r[i] += to_f32(ds_out[i * K + t - L + K]);
            }
            if (t >= t0) {
                if (t >= L)
#pragma unroll
                    for (int i = 0; i < V; ++i) r[i] = 0.f;
                store4(dx + (size_t)t * a.C, r);
            } else if (ds_in) {
#pragma unroll
                for (int i = 0; i < V; ++i) ds_in[i * K + t + K] = from_f32<T>(r[i]);
            }
        }
    }
    if (!a.partial) return;
    __shared__ float part[kWarps - 1][K + 1][V][32];
    if (warp > 0)
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < K; ++j) part[warp - 1][j][i][lane] = dw[j][i];
            part[warp - 1][K][i][lane] = db[i];
        }
    __syncthreads();
    if (warp == 0 && on) {
        float *p = a.partial + ((size_t)(b * gridDim.y + blockIdx.y) * (K + 1)) * a.C + c0;
#pragma unroll
        for (int j = 0; j <= K; ++j) {
            float r[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                r[i] = j < K ? dw[j < K ? j : 0][i] : db[i];
#pragma unroll
                for (int q = 0; q < kWarps - 1; ++q) r[i] += part[q][j][i][lane];
            }
            store4(p + (size_t)j * a.C, r);
        }
    }
}

// adds the partial sums of all blocks: 32 channels of one tap a block, its 32 warps each a stride of the rows
__global__ void __launch_bounds__(1024) conv1d_bwd_sum_kernel(const float *partial, int rows, int C, int K, float *dw,
                                                              float *db) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
    float s = 0.f;
    if (c < C)
        for (int r = warp; r < rows; r += 32) s += partial[((size_t)r * (K + 1) + j) * C + c];
    __shared__ float part[32][33];
    part[warp][lane] = s;
    __syncthreads();
    s = warp_sum(part[lane][warp]);  // this warp: channel blockIdx.x * 32 + warp
    const int cw = blockIdx.x * 32 + warp;
    if (lane == 0 && cw < C) {
        if (j < K) dw[(size_t)cw * K + j] = s;
        else if (db) db[cw] = s;
    }
}

__global__ void zero_f32_kernel(float *p, size_t n) {
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) p[i] = 0.f;
}

int tiles(int S) { return (S + kTile - 1) / kTile; }

template <typename T, int K>
cudaError_t launch_tk(const ConvBwdArgs &a, cudaStream_t s) {
    const unsigned gx = (unsigned)((a.C + 32 * V - 1) / (32 * V));
    const unsigned gy = (unsigned)(a.S > 0 ? tiles(a.S) : 1);  // without tokens, the state's gradient alone
    conv1d_bwd_kernel<T, K><<<dim3(gx, gy, a.B), kWarps * 32, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.partial) return e;
    conv1d_bwd_sum_kernel<<<dim3((unsigned)((a.C + 31) / 32), K + 1), 1024, 0, s>>>(a.partial, (int)(a.B * gy), a.C, K,
                                                                                 a.dw, a.db);
    return cudaGetLastError();
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
    return (size_t)B * tiles(S) * (K + 1) * C * sizeof(float);
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
