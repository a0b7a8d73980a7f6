// api.cu -- the C ABI of libgdr.so: argument checks, dispatch, device error word.
//
// Every entry point validates its arguments on the host before touching the GPU; on a
// non-zero status nothing has been launched.  The library allocates no device memory.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <unordered_map>
#include <unordered_set>
#include <vector>

#include "../../include/gdr.h"
#include "kernels.h"

namespace gdr {

// The device error word (GDR_DEVERR_* bits) of this library, one per device.
__device__ unsigned int g_device_error = 0;
// Snapshots of the error word taken by gdr_get_error, one slot per concurrent call (a call takes the next slot
// round-robin, so calls on different streams or host threads do not share one).
constexpr int kErrSlots = 64;
__device__ unsigned int g_error_snapshot[kErrSlots];

// Reads and clears the error word in one atomic step, so no bit raised meanwhile by another stream's kernel is lost.
__global__ void take_error_kernel(unsigned int *err, unsigned int *slot) { *slot = atomicExch(err, 0u); }

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_dev_checked[kMaxDevices];        // 0 unknown, 1 sm_100, -1 unusable
unsigned int *g_err_ptr[kMaxDevices];  // device address of g_device_error per device
unsigned int *g_snap_ptr[kMaxDevices]; // device address of g_error_snapshot per device
unsigned int g_snap_next = 0;          // next snapshot slot (under g_mu)

int g_sm_count[kMaxDevices];           // multiprocessors per device (0 until first asked)
int g_chunk_schedule = 0;              // tensor-core prefill schedule: 0 by shape, 1 one kernel, 2 two kernels

}  // namespace

// Multiprocessors of the current device; 148 (a full B200) when no device can be asked, so that the workspace
// query answers the same on a machine without a GPU.
int sm_count() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return 148;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_sm_count[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            return 148;
        }
        g_sm_count[dev] = n;
    }
    return g_sm_count[dev];
}

namespace {

bool supported_head(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// The tensor-core prefill's two-kernel schedule (a WY pass over every chunk on every SM, then the chains) pays
// off when the (b, value head) chains occupy at most a third of the SMs: the one-kernel schedule would leave the
// rest idle while each chain solves its chunks' WY systems in turn.  With more chains the one-kernel schedule,
// which needs no workspace, is faster.
bool two_kernel_schedule(int B, int Nv) {
    if (g_chunk_schedule == 1) return false;
    if (g_chunk_schedule == 2) return true;
    return (long long)B * Nv * 3 <= sm_count();
}
bool aligned16(const void *p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks the current device once (sm_100 family) and fetches the address of the error
// word on it.  Returns GDR_OK, GDR_ERR_DEVICE or GDR_ERR_LAUNCH.
int device_setup(unsigned int **err) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return GDR_ERR_DEVICE;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_dev_checked[dev] == 0) {
        int major = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) {
            cudaGetLastError();
            return GDR_ERR_DEVICE;
        }
        if (major != 10) {
            g_dev_checked[dev] = -1;
            return GDR_ERR_DEVICE;
        }
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) {
            cudaGetLastError();
            return GDR_ERR_LAUNCH;
        }
        g_err_ptr[dev] = static_cast<unsigned int *>(p);
        if (cudaGetSymbolAddress(&p, g_error_snapshot) != cudaSuccess) {
            cudaGetLastError();
            return GDR_ERR_LAUNCH;
        }
        g_snap_ptr[dev] = static_cast<unsigned int *>(p);
        g_dev_checked[dev] = 1;
    }
    if (g_dev_checked[dev] < 0) return GDR_ERR_DEVICE;
    *err = g_err_ptr[dev];
    return GDR_OK;
}

int check_common(int B, int Nk, int Nv, int S, int Dk, int Dv, int dtype) {
    if (dtype != GDR_F32 && dtype != GDR_BF16 && dtype != GDR_F16) return GDR_ERR_DTYPE;
    if (B < 0 || S < 0 || Nk < 1 || Nv < 1 || Dk < 1 || Dv < 1) return GDR_ERR_SHAPE;
    if (Nv % Nk != 0) return GDR_ERR_SHAPE;
    if (!supported_head(Dk) || !supported_head(Dv)) return GDR_ERR_UNSUPPORTED;
    // grids are one-dimensional: B * Nv * (column slabs) blocks
    if ((long long)B * Nv * 8 >= (1LL << 31)) return GDR_ERR_SHAPE;
    return GDR_OK;
}

int check_prologue(const gdr_prologue *p, const float *g) {
    if (!p) return GDR_OK;
    if (p->A_log && (!p->dt_bias || !g)) return GDR_ERR_NULL;
    if (p->l2norm_qk && !(p->eps >= 0.f)) return GDR_ERR_SHAPE;
    return GDR_OK;
}

// ---- checked mode (environment variable GDR_CHECKS=1): host-side validation of the index and length arrays ----
// The kernels never trap on bad lengths or slots (they skip the sequence and flag the error word), and two
// sequences that share a slot race silently.  In checked mode the library copies the arrays to the host before
// launching (a synchronisation on the caller's stream, so for debugging only) and rejects such calls with
// GDR_ERR_SHAPE.
bool checks_enabled() {
    const char *v = std::getenv("GDR_CHECKS");
    return v && v[0] && std::strcmp(v, "0") != 0;
}

bool copy_i32(std::vector<int32_t> &h, const int32_t *d, size_t n, cudaStream_t s) {
    h.assign(n, 0);
    if (n == 0 || !d) return true;
    if (cudaMemcpyAsync(h.data(), d, n * sizeof(int32_t), cudaMemcpyDeviceToHost, s) != cudaSuccess) return false;
    return cudaStreamSynchronize(s) == cudaSuccess;
}

// lengths within [0, S]
int check_lengths_host(const int32_t *lengths, int B, int S, cudaStream_t s) try {
    if (!lengths) return GDR_OK;
    std::vector<int32_t> L;
    if (!copy_i32(L, lengths, (size_t)B, s)) return GDR_ERR_LAUNCH;
    for (int b = 0; b < B; ++b)
        if (L[b] < 0 || L[b] > S) return GDR_ERR_SHAPE;
    return GDR_OK;
} catch (...) {  // no memory for the copies: no exception leaves a C entry
    return GDR_ERR_LAUNCH;
}

// Decode: lengths in [0, S], accepted counts in range, every slot a sequence reads or writes in [0, slots), and
// no slot touched by two sequences.  per_token selects the speculative-decoding reading (the chain starts at token
// A - 1's slot and every processed token's state goes to its own slot); otherwise the chain starts at token 0's
// slot and the first min(A, L) states are committed.
int check_decode_lists(const int32_t *idx, const std::vector<int32_t> &L, const int32_t *accepted, int B, int S,
                       int slots, int per_token, cudaStream_t s) try {
    std::vector<int32_t> I, A;
    if (!copy_i32(I, idx, (size_t)B * S, s) || !copy_i32(A, accepted, accepted ? (size_t)B : 0, s))
        return GDR_ERR_LAUNCH;
    std::unordered_map<int32_t, int> owner;
    for (int b = 0; b < B; ++b) {
        const int Lb = L[b];
        if (Lb < 0 || Lb > S) return GDR_ERR_SHAPE;
        if (Lb == 0) continue;
        int Ab = accepted ? A[b] : (per_token ? 1 : Lb);
        std::vector<int32_t> touched;
        if (per_token) {
            if (Ab < 1 || Ab > S) return GDR_ERR_SHAPE;
            touched.push_back(I[(size_t)b * S + Ab - 1]);
            for (int t = 0; t < Lb; ++t) touched.push_back(I[(size_t)b * S + t]);
        } else {
            if (Ab < 0) return GDR_ERR_SHAPE;
            touched.push_back(I[(size_t)b * S]);
            for (int t = 0; t < (Ab < Lb ? Ab : Lb); ++t) touched.push_back(I[(size_t)b * S + t]);
        }
        for (int32_t x : touched) {
            if (x < 0 || x >= slots) return GDR_ERR_SHAPE;
            auto it = owner.find(x);
            if (it != owner.end() && it->second != b) return GDR_ERR_SHAPE;
            owner[x] = b;
        }
    }
    return GDR_OK;
} catch (...) {
    return GDR_ERR_LAUNCH;
}

int check_decode_host(const int32_t *idx, const int32_t *lengths, const int32_t *accepted, int B, int S, int slots,
                      int per_token, cudaStream_t s) try {
    std::vector<int32_t> L;
    if (!lengths) L.assign((size_t)B, S);  // every sequence has S tokens
    else if (!copy_i32(L, lengths, (size_t)B, s)) return GDR_ERR_LAUNCH;
    return check_decode_lists(idx, L, accepted, B, S, slots, per_token, s);
} catch (...) {
    return GDR_ERR_LAUNCH;
}

// Slot calls: what the kernels would skip and flag (an index out of range, a copy's target that is another copy's source or
// target), and for a fork also a slot that two rows share.
int check_copy_host(const int32_t *src, const int32_t *dst, int n, int slots, cudaStream_t s) try {
    std::vector<int32_t> S, D;
    if (!copy_i32(S, src, (size_t)n, s) || !copy_i32(D, dst, (size_t)n, s)) return GDR_ERR_LAUNCH;
    auto moves = [&](int i) { return S[i] != -1 && D[i] != -1 && S[i] != D[i]; };
    std::unordered_set<int32_t> targets;
    for (int i = 0; i < n; ++i) {
        if (!moves(i)) continue;
        if (S[i] < 0 || S[i] >= slots || D[i] < 0 || D[i] >= slots) return GDR_ERR_SHAPE;
        if (!targets.insert(D[i]).second) return GDR_ERR_SHAPE;
    }
    for (int i = 0; i < n; ++i)
        if (moves(i) && targets.count(S[i])) return GDR_ERR_SHAPE;
    return GDR_OK;
} catch (...) {
    return GDR_ERR_LAUNCH;
}

int check_fork_host(const int32_t *table, const int32_t *parents, int n, int slots, cudaStream_t s) try {
    std::vector<int32_t> T, P;
    if (!copy_i32(T, table, (size_t)n, s) || !copy_i32(P, parents, (size_t)n, s)) return GDR_ERR_LAUNCH;
    auto in_range = [&](int32_t x) { return x >= 0 && x < slots; };
    std::unordered_set<int32_t> seen;
    std::vector<char> continued((size_t)n, 0);
    std::vector<int> extra, dead;  // rows that take another row's slot, rows nobody continues from: as many
    for (int i = 0; i < n; ++i) {
        if (P[i] < -1 || P[i] >= n) return GDR_ERR_SHAPE;
        if (in_range(T[i]) && !seen.insert(T[i]).second) return GDR_ERR_SHAPE;
        if (P[i] >= 0 && !continued[P[i]]) continued[P[i]] = 1;
        else extra.push_back(i);
    }
    for (int i = 0; i < n; ++i)
        if (!continued[i]) dead.push_back(i);
    for (size_t k = 0; k < extra.size(); ++k) {
        const int32_t r = P[extra[k]];
        if (r >= 0 && (!in_range(T[r]) || !in_range(T[dead[k]]))) return GDR_ERR_SHAPE;
    }
    return GDR_OK;
} catch (...) {
    return GDR_ERR_LAUNCH;
}

int check_free_host(const int32_t *idx, int n, int slots, cudaStream_t s) try {
    std::vector<int32_t> I;
    if (!copy_i32(I, idx, (size_t)n, s)) return GDR_ERR_LAUNCH;
    for (int32_t x : I)
        if (x < -1 || x >= slots) return GDR_ERR_SHAPE;
    return GDR_OK;
} catch (...) {
    return GDR_ERR_LAUNCH;
}

// Whether no output shares bytes with an input or another output (spans without a pointer or without bytes share none)
struct Span {
    const void *p;
    unsigned long long n;
};
bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x && y && a.n && b.n && x < y + b.n && y < x + a.n;
}
template <int NO, int NI> bool disjoint(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlap(outs[i], ins[j])) return false;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return false;
    }
    return true;
}
unsigned long long elt(int dtype) { return dtype == GDR_F32 ? 4 : 2; }

int check_epilogue(const gdr_epilogue *e) {
    if (!e) return GDR_OK;
    if (!e->z || !e->norm_w) return GDR_ERR_NULL;
    if (!(e->eps >= 0.f)) return GDR_ERR_SHAPE;
    if (!aligned16(e->z) || !aligned16(e->norm_w)) return GDR_ERR_ALIGN;
    return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" size_t gdr_chunk_fwd_workspace(int B, int Nk, int Nv, int S, int Dk, int Dv, gdr_dtype dtype) {
    if (check_common(B, Nk, Nv, S, Dk, Dv, dtype) != GDR_OK) return 0;
    if ((long long)B * S == 0 || !chunk_tc_supported(Dk, Dv, dtype, S)) return 0;
    return two_kernel_schedule(B, Nv) ? chunk_wy_workspace(B, Nv, S) : 0;
}

extern "C" int gdr_chunk_fwd(const void *q, const void *k, const void *v, const void *beta, const float *g,
                             const void *initial_state, const int32_t *actual_seq_lengths, float scale, int B,
                             int Nk, int Nv, int S, int Dk, int Dv, gdr_dtype dtype, const gdr_prologue *prologue,
                             const gdr_epilogue *epilogue, void *out, void *final_state, void *workspace,
                             size_t ws_bytes, gdr_stream_t stream) {
    int st = check_common(B, Nk, Nv, S, Dk, Dv, dtype);
    if (st) return st;
    if ((st = check_prologue(prologue, g))) return st;
    if ((st = check_epilogue(epilogue))) return st;
    if ((long long)B * S > 0 && (!q || !k || !v || !beta || !out)) return GDR_ERR_NULL;
    const void *ptrs[] = {q, k, v, beta, g, initial_state, actual_seq_lengths, out, final_state, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGN;
    // a workspace of at least the queried size selects the two-kernel schedule where the query asks for one; no
    // workspace runs the one-kernel schedule, which needs none
    const size_t need = gdr_chunk_fwd_workspace(B, Nk, Nv, S, Dk, Dv, dtype);
    if (workspace && ws_bytes < need) return GDR_ERR_WORKSPACE;
    if (B == 0 || (S == 0 && !final_state)) return GDR_OK;
    unsigned int *err = nullptr;
    if ((st = device_setup(&err))) return st;

    ChunkArgs a{};
    a.q = q; a.k = k; a.v = v; a.beta = beta; a.g = g;
    a.initial_state = initial_state;
    a.lengths = actual_seq_lengths;
    a.scale = scale;
    a.B = B; a.Nk = Nk; a.Nv = Nv; a.S = S;
    a.out = out; a.final_state = final_state;
    a.l2norm = prologue ? prologue->l2norm_qk : 0;
    a.eps = prologue ? prologue->eps : 0.f;
    a.beta_logits = prologue ? prologue->beta_logits : 0;
    a.A_log = prologue ? prologue->A_log : nullptr;
    a.dt_bias = prologue ? prologue->dt_bias : nullptr;
    a.err = err;
    a.workspace = workspace;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() && (st = check_lengths_host(actual_seq_lengths, B, S, cs))) return st;
    cudaError_t e;
    if (chunk_tc_supported(Dk, Dv, dtype, S)) {
        if (epilogue) {  // fused into the tensor-core kernel's out epilogue
            a.epi_z = epilogue->z;
            a.epi_w = epilogue->norm_w;
            a.epi_eps = epilogue->eps;
        }
        e = (need > 0 && workspace) ? launch_chunk_wy(a, dtype, cs) : launch_chunk_tc(a, dtype, cs);
    } else {
        e = launch_chunk_simt(a, Dk, Dv, dtype, cs);
        if (e == cudaSuccess && epilogue && S > 0)
            e = launch_gated_rmsnorm(out, epilogue->z, epilogue->norm_w, epilogue->eps, actual_seq_lengths, B, Nv,
                                     S, Dv, dtype, cs);
    }
    return e == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

namespace {
int recurrent_step(const void *q, const void *k, const void *v, const void *beta, const float *g, const float *gk,
                   void *state_pool, int slots, const int32_t *ssm_state_indices, const int32_t *actual_seq_lengths,
                   const int32_t *num_accepted_tokens, float scale, int B, int Nk, int Nv, int S, int Dk, int Dv,
                   gdr_dtype dtype, gdr_dtype state_dtype, const gdr_prologue *prologue, const gdr_epilogue *epilogue,
                   void *out, gdr_stream_t stream, int per_token) {
    int st = check_common(B, Nk, Nv, S, Dk, Dv, dtype);
    if (st) return st;
    if (state_dtype != GDR_F32 && state_dtype != GDR_BF16 && state_dtype != GDR_F16) return GDR_ERR_DTYPE;
    // fp16 inputs take an fp16 or fp32 state; an fp16 state takes fp16 inputs
    if ((dtype == GDR_F16 && state_dtype == GDR_BF16) || (state_dtype == GDR_F16 && dtype != GDR_F16))
        return GDR_ERR_DTYPE;
    if (S < 1 || S > kDecodeMaxTokens || slots < 1) return GDR_ERR_SHAPE;
    // the kernels address the pool by (slot, head) tile in 32-bit arithmetic
    if ((long long)slots * Nv >= (1LL << 31)) return GDR_ERR_SHAPE;
    if ((st = check_prologue(prologue, g))) return st;
    if ((st = check_epilogue(epilogue))) return st;
    if (B > 0 && (!q || !k || !v || !beta || !out || !state_pool || !ssm_state_indices || !actual_seq_lengths))
        return GDR_ERR_NULL;
    const void *ptrs[] = {q, k, v, beta, g, gk, state_pool, ssm_state_indices, actual_seq_lengths,
                          num_accepted_tokens, out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGN;
    if (B == 0) return GDR_OK;
    unsigned int *err = nullptr;
    if ((st = device_setup(&err))) return st;

    DecodeArgs a{};
    a.q = q; a.k = k; a.v = v; a.beta = beta; a.g = g; a.gk = gk;
    a.pool = state_pool; a.slots = slots;
    a.idx = ssm_state_indices; a.lengths = actual_seq_lengths; a.accepted = num_accepted_tokens;
    a.scale = scale;
    a.B = B; a.Nk = Nk; a.Nv = Nv; a.S = S;
    a.out = out;
    a.l2norm = prologue ? prologue->l2norm_qk : 0;
    a.eps = prologue ? prologue->eps : 0.f;
    a.beta_logits = prologue ? prologue->beta_logits : 0;
    a.A_log = prologue ? prologue->A_log : nullptr;
    a.dt_bias = prologue ? prologue->dt_bias : nullptr;
    a.err = err;
    a.per_token = per_token;
    a.wait_ns = chunk_wait_ns();
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() &&
        (st = check_decode_host(ssm_state_indices, actual_seq_lengths, num_accepted_tokens, B, S, slots, per_token,
                                cs)))
        return st;
    cudaError_t e = launch_decode(a, Dk, Dv, dtype, state_dtype, cs);
    if (e == cudaSuccess && epilogue)
        e = launch_gated_rmsnorm(out, epilogue->z, epilogue->norm_w, epilogue->eps, actual_seq_lengths, B, Nv, S, Dv,
                                 dtype, cs);
    return e == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}
}  // namespace

extern "C" int gdr_recurrent_step(const void *q, const void *k, const void *v, const void *beta, const float *g,
                                  const float *gk, void *state_pool, int slots, const int32_t *ssm_state_indices,
                                  const int32_t *actual_seq_lengths, const int32_t *num_accepted_tokens,
                                  float scale, int B, int Nk, int Nv, int S, int Dk, int Dv, gdr_dtype dtype,
                                  gdr_dtype state_dtype, const gdr_prologue *prologue,
                                  const gdr_epilogue *epilogue, void *out, gdr_stream_t stream) {
    return recurrent_step(q, k, v, beta, g, gk, state_pool, slots, ssm_state_indices, actual_seq_lengths,
                          num_accepted_tokens, scale, B, Nk, Nv, S, Dk, Dv, dtype, state_dtype, prologue, epilogue,
                          out, stream, 0);
}

extern "C" int gdr_recurrent_step_spec(const void *q, const void *k, const void *v, const void *beta,
                                       const float *g, const float *gk, void *state_pool, int slots,
                                       const int32_t *ssm_state_indices, const int32_t *actual_seq_lengths,
                                       const int32_t *num_accepted_tokens, float scale, int B, int Nk, int Nv, int S,
                                       int Dk, int Dv, gdr_dtype dtype, gdr_dtype state_dtype,
                                       const gdr_prologue *prologue, const gdr_epilogue *epilogue, void *out,
                                       gdr_stream_t stream) {
    return recurrent_step(q, k, v, beta, g, gk, state_pool, slots, ssm_state_indices, actual_seq_lengths,
                          num_accepted_tokens, scale, B, Nk, Nv, S, Dk, Dv, dtype, state_dtype, prologue, epilogue,
                          out, stream, 1);
}

extern "C" int gdr_conv1d(const void *x, const void *weight, const void *bias, const void *conv_state_in,
                          const int32_t *actual_seq_lengths, int B, int S, int Nk, int Nv, int Dk, int Dv, int K,
                          gdr_dtype dtype, void *q, void *k, void *v, void *conv_state_out, gdr_stream_t stream) {
    int st = check_common(B, Nk, Nv, S, Dk, Dv, dtype);
    if (st) return st;
    if (K < 1 || K > 8) return GDR_ERR_SHAPE;
    // grid: (channel groups, 64-step time tiles, B)
    if (B > 65535 || (long long)S > 65535LL * 64) return GDR_ERR_SHAPE;
    if ((long long)B * S > 0 && (!x || !weight || !q || !k || !v)) return GDR_ERR_NULL;
    if (B > 0 && conv_state_out && !weight) return GDR_ERR_NULL;
    const void *ptrs[] = {x, weight, bias, conv_state_in, actual_seq_lengths, q, k, v, conv_state_out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGN;
    if (B == 0 || (S == 0 && !conv_state_out)) return GDR_OK;
    unsigned int *err = nullptr;
    if ((st = device_setup(&err))) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() && (st = check_lengths_host(actual_seq_lengths, B, S, cs))) return st;
    cudaError_t e = launch_conv1d(x, weight, bias, conv_state_in, actual_seq_lengths, B, S, Nk, Nv, Dk, Dv, K, dtype,
                                  q, k, v, conv_state_out, err, cs);
    return e == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

extern "C" size_t gdr_conv1d_bwd_workspace(int B, int S, int Nk, int Nv, int Dk, int Dv, int K) {
    if (check_common(B, Nk, Nv, S, Dk, Dv, GDR_F32) != GDR_OK || K < 1 || K > 8) return 0;
    return conv1d_bwd_workspace(B, S, 2 * Nk * Dk + Nv * Dv, K);
}

extern "C" int gdr_conv1d_bwd(const void *x, const void *weight, const void *bias, const void *conv_state_in,
                              const int32_t *actual_seq_lengths, const void *dq, const void *dk, const void *dv,
                              const void *dconv_state_out, int B, int S, int Nk, int Nv, int Dk, int Dv, int K,
                              gdr_dtype dtype, void *dx, float *dweight, float *dbias, void *dconv_state_in,
                              void *workspace, size_t ws_bytes, gdr_stream_t stream) {
    int st = check_common(B, Nk, Nv, S, Dk, Dv, dtype);
    if (st) return st;
    if (K < 1 || K > 8) return GDR_ERR_SHAPE;
    if (B > 65535 || (long long)S > 65535LL * 64) return GDR_ERR_SHAPE;  // as gdr_conv1d
    // a row's bytes are kept in 32 bits
    if (2LL * Nk * Dk + 1LL * Nv * Dv > 1LL << 26) return GDR_ERR_SHAPE;
    if (!dweight) return GDR_ERR_NULL;
    if ((long long)B * S > 0 && (!x || !weight || !dq || !dk || !dv || !dx)) return GDR_ERR_NULL;
    if (B > 0 && dconv_state_in && !weight) return GDR_ERR_NULL;
    const void *ptrs[] = {x, weight, bias, conv_state_in, actual_seq_lengths, dq, dk, dv, dconv_state_out, dx, dweight,
                          dbias, dconv_state_in, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGN;
    const size_t need = gdr_conv1d_bwd_workspace(B, S, Nk, Nv, Dk, Dv, K);
    if (need > 0 && !workspace) return GDR_ERR_NULL;
    if (ws_bytes < need) return GDR_ERR_WORKSPACE;
    const unsigned long long C = 2ull * Nk * Dk + 1ull * Nv * Dv, e = elt(dtype), qk = e * B * Nk * S * Dk;
    const Span ins[] = {{x, e * B * S * C}, {weight, e * C * K}, {bias, e * C}, {conv_state_in, e * B * C * K},
                        {actual_seq_lengths, 4ull * B}, {dq, qk}, {dk, qk}, {dv, e * B * Nv * S * Dv},
                        {dconv_state_out, e * B * C * K}};
    const Span outs[] = {{dx, e * B * S * C}, {dweight, 4 * C * K}, {dbias, 4 * C}, {dconv_state_in, e * B * C * K},
                         {workspace, need}};
    if (!disjoint(outs, ins)) return GDR_ERR_SHAPE;
    unsigned int *err = nullptr;
    if ((st = device_setup(&err))) return st;
    ConvBwdArgs a{};
    a.x = x; a.w = weight; a.bias = bias; a.state_in = conv_state_in; a.lengths = actual_seq_lengths;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dstate_out = dconv_state_out;
    a.dx = dx; a.dw = dweight; a.db = dbias; a.dstate_in = dconv_state_in;
    a.partial = need > 0 ? static_cast<float *>(workspace) : nullptr;
    a.B = B; a.S = S; a.C = 2 * Nk * Dk + Nv * Dv; a.Nk = Nk; a.Nv = Nv; a.Dk = Dk; a.Dv = Dv;
    a.err = err;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() && (st = check_lengths_host(actual_seq_lengths, B, S, cs))) return st;
    return launch_conv1d_bwd(a, K, dtype, cs) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

namespace {
int check_scan(int B, int N, int S, int D, int dtype, int gate_dtype, int mode) {
    if (dtype != GDR_F32 && dtype != GDR_BF16 && dtype != GDR_F16) return GDR_ERR_DTYPE;
    if (gate_dtype != GDR_F32 && gate_dtype != dtype) return GDR_ERR_DTYPE;
    if (mode != GDR_SCAN_ADD && mode != GDR_SCAN_MIX) return GDR_ERR_SHAPE;
    if (B < 0 || S < 0 || N < 1 || D < 1) return GDR_ERR_SHAPE;
    if (D > 1 << 26) return GDR_ERR_SHAPE;  // the kernels keep a row's bytes in 32 bits
    // channels are counted in 31 bits (grids, channel indices); offsets into the tensors are 64-bit
    if ((long long)B * N >= (1LL << 31) || (long long)B * N * D >= (1LL << 31)) return GDR_ERR_SHAPE;
    if ((long long)N * D >= (1LL << 31) || (double)B * N * D * S >= 0x1p60) return GDR_ERR_SHAPE;
    return GDR_OK;
}
}  // namespace

extern "C" int gdr_scan_fwd(const void *x, const void *g, const float *initial_state,
                            const int32_t *actual_seq_lengths, int B, int N, int S, int D, gdr_dtype dtype,
                            gdr_dtype gate_dtype, int mode, void *out, float *final_state, float *checkpoints,
                            gdr_stream_t stream) {
    int st = check_scan(B, N, S, D, dtype, gate_dtype, mode);
    if (st) return st;
    if ((long long)B * S > 0 && (!x || !g || !out)) return GDR_ERR_NULL;
    const void *ptrs[] = {x, g, initial_state, actual_seq_lengths, out, final_state, checkpoints};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGN;
    const unsigned long long rows = (unsigned long long)B * N, all = rows * S * D, state = rows * D * 4;
    const Span ins[] = {{x, all * elt(dtype)}, {g, all * elt(gate_dtype)},
                        {initial_state == final_state ? nullptr : initial_state, state},
                        {actual_seq_lengths, 4ull * B}};
    const Span outs[] = {{out, all * elt(dtype)}, {final_state, state},
                         {checkpoints, state * ((S + kChunk - 1ull) / kChunk)}};
    if (!disjoint(outs, ins)) return GDR_ERR_SHAPE;
    if (B == 0 || (S == 0 && !final_state)) return GDR_OK;
    unsigned int *err = nullptr;
    if ((st = device_setup(&err))) return st;
    ScanArgs a{};
    a.x = x; a.g = g; a.initial_state = initial_state; a.lengths = actual_seq_lengths;
    a.B = B; a.N = N; a.S = S; a.D = D; a.mode = mode;
    a.out = out; a.final_state = final_state; a.checkpoints = checkpoints; a.err = err; a.wait_ns = chunk_wait_ns();
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() && (st = check_lengths_host(actual_seq_lengths, B, S, cs))) return st;
    return launch_scan_fwd(a, dtype, gate_dtype, cs) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

extern "C" int gdr_scan_bwd(const void *x, const void *g, const float *checkpoints, const void *dout,
                            const float *dfinal_state, const int32_t *actual_seq_lengths, int B, int N, int S, int D,
                            gdr_dtype dtype, gdr_dtype gate_dtype, int mode, void *dx, void *dg,
                            float *dinitial_state, gdr_stream_t stream) {
    int st = check_scan(B, N, S, D, dtype, gate_dtype, mode);
    if (st) return st;
    if ((long long)B * S > 0 && (!x || !g || !checkpoints || !dout || !dx || !dg)) return GDR_ERR_NULL;
    const void *ptrs[] = {x, g, checkpoints, dout, dfinal_state, actual_seq_lengths, dx, dg, dinitial_state};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGN;
    const unsigned long long rows = (unsigned long long)B * N, all = rows * S * D, state = rows * D * 4;
    const Span ins[] = {{x, all * elt(dtype)}, {g, all * elt(gate_dtype)},
                        {checkpoints, state * ((S + kChunk - 1ull) / kChunk)}, {dout, all * elt(dtype)},
                        {dfinal_state == dinitial_state ? nullptr : dfinal_state, state},
                        {actual_seq_lengths, 4ull * B}};
    const Span outs[] = {{dx, all * elt(dtype)}, {dg, all * elt(gate_dtype)}, {dinitial_state, state}};
    if (!disjoint(outs, ins)) return GDR_ERR_SHAPE;
    if (B == 0 || (S == 0 && !dinitial_state)) return GDR_OK;
    unsigned int *err = nullptr;
    if ((st = device_setup(&err))) return st;
    ScanBwdArgs a{};
    a.x = x; a.g = g; a.checkpoints = checkpoints; a.dout = dout; a.dfinal_state = dfinal_state;
    a.lengths = actual_seq_lengths;
    a.B = B; a.N = N; a.S = S; a.D = D; a.mode = mode;
    a.dx = dx; a.dg = dg; a.dinitial_state = dinitial_state; a.err = err; a.wait_ns = chunk_wait_ns();
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() && (st = check_lengths_host(actual_seq_lengths, B, S, cs))) return st;
    return launch_scan_bwd(a, dtype, gate_dtype, cs) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

extern "C" int gdr_scan_step(const void *x, const void *g, float *state_pool, int slots,
                             const int32_t *ssm_state_indices, const int32_t *actual_seq_lengths,
                             const int32_t *num_accepted_tokens, int B, int N, int S, int D, gdr_dtype dtype,
                             gdr_dtype gate_dtype, int mode, int per_token, void *out, gdr_stream_t stream) {
    int st = check_scan(B, N, S, D, dtype, gate_dtype, mode);
    if (st) return st;
    if (S < 1 || S > kDecodeMaxTokens || slots < 1 || (double)slots * N * D >= 0x1p60) return GDR_ERR_SHAPE;
    if (B > 0 && (!x || !g || !state_pool || !ssm_state_indices || !out)) return GDR_ERR_NULL;
    const void *ptrs[] = {x, g, state_pool, ssm_state_indices, actual_seq_lengths, num_accepted_tokens, out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGN;
    const unsigned long long all = (unsigned long long)B * N * S * D;
    const Span ins[] = {{x, all * elt(dtype)}, {g, all * elt(gate_dtype)}, {ssm_state_indices, 4ull * B * S},
                        {actual_seq_lengths, 4ull * B}, {num_accepted_tokens, 4ull * B}};
    const Span outs[] = {{out, all * elt(dtype)}, {state_pool, 4ull * slots * N * D}};
    if (!disjoint(outs, ins)) return GDR_ERR_SHAPE;
    if (B == 0) return GDR_OK;
    unsigned int *err = nullptr;
    if ((st = device_setup(&err))) return st;
    ScanStepArgs a{};
    a.x = x; a.g = g; a.pool = state_pool; a.slots = slots;
    a.idx = ssm_state_indices; a.lengths = actual_seq_lengths; a.accepted = num_accepted_tokens;
    a.B = B; a.N = N; a.S = S; a.D = D; a.mode = mode; a.per_token = per_token != 0;
    a.out = out; a.err = err;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() && (st = check_decode_host(ssm_state_indices, actual_seq_lengths, num_accepted_tokens, B, S,
                                                    slots, a.per_token, cs)))
        return st;
    return launch_scan_step(a, dtype, gate_dtype, cs) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

namespace {
// the pools of a slot call, checked and copied into the kernels' argument block
int take_pools(const gdr_pool *pools, int n_pools, int slots, long long max_slots, SlotPools *out) {
    if (n_pools < 1 || n_pools > GDR_MAX_POOLS || slots < 1 || slots > max_slots) return GDR_ERR_SHAPE;
    if (!pools) return GDR_ERR_NULL;
    *out = SlotPools{};
    for (int i = 0; i < n_pools; ++i) {
        if (!pools[i].data) return GDR_ERR_NULL;
        if (!aligned16(pools[i].data)) return GDR_ERR_ALIGN;
        // (the kernels count the units of 4 KB of a slot of all pools in 32 bits)
        if (pools[i].slot_bytes < 1 || pools[i].slot_bytes > (1ull << 37)) return GDR_ERR_SHAPE;
        out->data[i] = static_cast<char *>(pools[i].data);
        out->bytes[i] = pools[i].slot_bytes;
    }
    // pools that share bytes would be moved twice, in no order
    for (int i = 0; i < n_pools; ++i)
        for (int j = 0; j < i; ++j) {
            const char *a = out->data[i], *b = out->data[j];
            if (a < b + out->bytes[j] * (unsigned long long)slots && b < a + out->bytes[i] * (unsigned long long)slots)
                return GDR_ERR_SHAPE;
        }
    out->n = n_pools;
    out->slots = slots;
    return GDR_OK;
}

constexpr long long kMaxSlots = (1LL << 24) - 1;

// whether an array of n words lies in a pool, where a move could change it while it is read
bool in_pools(const SlotPools &p, const void *a, long long n) {
    for (int i = 0; i < p.n; ++i)
        if (overlap({p.data[i], p.bytes[i] * (unsigned long long)p.slots}, {a, 4ull * n})) return true;
    return false;
}
}  // namespace

extern "C" int gdr_slot_copy(const gdr_pool *pools, int n_pools, int slots, const int32_t *src, const int32_t *dst,
                             int n, gdr_stream_t stream) {
    SlotPools p;
    int st = take_pools(pools, n_pools, slots, kMaxSlots, &p);
    if (st) return st;
    if (n < 0 || n > kMaxSlotMoves) return GDR_ERR_SHAPE;
    if (n > 0 && (!src || !dst)) return GDR_ERR_NULL;
    if (!aligned16(src) || !aligned16(dst)) return GDR_ERR_ALIGN;
    if (in_pools(p, src, n) || in_pools(p, dst, n)) return GDR_ERR_SHAPE;
    if (n == 0) return GDR_OK;
    if ((st = device_setup(&p.err))) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() && (st = check_copy_host(src, dst, n, slots, cs))) return st;
    return launch_slot_copy(p, src, dst, n, cs) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

extern "C" int gdr_slot_fork(const gdr_pool *pools, int n_pools, int slots, const int32_t *slot_table,
                             const int32_t *parents, int n, int32_t *new_slot_table, gdr_stream_t stream) {
    SlotPools p;
    int st = take_pools(pools, n_pools, slots, kMaxSlots, &p);
    if (st) return st;
    if (n < 0 || n > kMaxForkRows) return GDR_ERR_SHAPE;
    if (n > 0 && (!slot_table || !parents || !new_slot_table)) return GDR_ERR_NULL;
    if (!aligned16(slot_table) || !aligned16(parents) || !aligned16(new_slot_table)) return GDR_ERR_ALIGN;
    // every block reads both inputs while one writes the result
    if (n > 0 && (new_slot_table < slot_table + n && slot_table < new_slot_table + n)) return GDR_ERR_SHAPE;
    if (n > 0 && (new_slot_table < parents + n && parents < new_slot_table + n)) return GDR_ERR_SHAPE;
    if (in_pools(p, slot_table, n) || in_pools(p, parents, n) || in_pools(p, new_slot_table, n)) return GDR_ERR_SHAPE;
    if (n == 0) return GDR_OK;
    if ((st = device_setup(&p.err))) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() && (st = check_fork_host(slot_table, parents, n, slots, cs))) return st;
    return launch_slot_fork(p, slot_table, parents, n, new_slot_table, cs) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

extern "C" int gdr_slot_compact(const gdr_pool *pools, int n_pools, int slots, const int32_t *live, int32_t *new_slot,
                                int32_t *n_live, gdr_stream_t stream) {
    SlotPools p;
    int st = take_pools(pools, n_pools, slots, kMaxCompactSlots, &p);
    if (st) return st;
    if (!live || !new_slot || !n_live) return GDR_ERR_NULL;
    if (!aligned16(live) || !aligned16(new_slot) || !aligned16(n_live)) return GDR_ERR_ALIGN;
    if (new_slot < live + slots && live < new_slot + slots) return GDR_ERR_SHAPE;
    if (n_live >= live && n_live < live + slots) return GDR_ERR_SHAPE;
    if (n_live >= new_slot && n_live < new_slot + slots) return GDR_ERR_SHAPE;
    if (in_pools(p, live, slots) || in_pools(p, new_slot, slots) || in_pools(p, n_live, 1)) return GDR_ERR_SHAPE;
    if ((st = device_setup(&p.err))) return st;
    return launch_slot_compact(p, live, new_slot, n_live, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDR_OK : GDR_ERR_LAUNCH;
}

extern "C" int gdr_slot_free(const gdr_pool *pools, int n_pools, int slots, const int32_t *idx, int n, int32_t *live,
                             gdr_stream_t stream) {
    SlotPools p;
    int st = take_pools(pools, n_pools, slots, kMaxSlots, &p);
    if (st) return st;
    if (n < 0 || n > kMaxSlotMoves) return GDR_ERR_SHAPE;
    if (n > 0 && !idx) return GDR_ERR_NULL;
    if (!aligned16(idx) || !aligned16(live)) return GDR_ERR_ALIGN;
    if (n > 0 && live && idx < live + slots && live < idx + n) return GDR_ERR_SHAPE;
    if (in_pools(p, idx, n) || (live && in_pools(p, live, slots))) return GDR_ERR_SHAPE;
    if (n == 0) return GDR_OK;
    if ((st = device_setup(&p.err))) return st;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (checks_enabled() && (st = check_free_host(idx, n, slots, cs))) return st;
    return launch_slot_free(p, idx, n, live, cs) == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

extern "C" int gdr_prologue_apply(const void *q, const void *k, const void *b, const float *a, const float *A_log,
                                  const float *dt_bias, float eps, int B, int Nk, int Nv, int S, int Dk,
                                  gdr_dtype dtype, void *q_hat, void *k_hat, void *beta, float *g,
                                  gdr_stream_t stream) {
    if (dtype != GDR_F32 && dtype != GDR_BF16 && dtype != GDR_F16) return GDR_ERR_DTYPE;
    if (B < 0 || S < 0 || Nk < 1 || Nv < 1 || Dk < 1) return GDR_ERR_SHAPE;
    if (!(eps >= 0.f)) return GDR_ERR_SHAPE;
    if ((q && !q_hat) || (k && !k_hat) || (b && !beta) || (a && (!g || !A_log || !dt_bias))) return GDR_ERR_NULL;
    const void *ptrs[] = {q, k, b, a, A_log, dt_bias, q_hat, k_hat, beta, g};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGN;
    if ((long long)B * S == 0 || (!q && !k && !b && !a)) return GDR_OK;
    unsigned int *err = nullptr;
    int st = device_setup(&err);
    if (st) return st;
    cudaError_t e = launch_prologue(q, k, b, a, A_log, dt_bias, eps, B, Nk, Nv, S, Dk, dtype, q_hat, k_hat, beta, g,
                                    reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDR_OK : GDR_ERR_LAUNCH;
}

extern "C" int gdr_get_error(gdr_stream_t stream, int *device_error) {
    if (!device_error) return GDR_ERR_NULL;
    *device_error = 0;
    unsigned int *err = nullptr;
    int st = device_setup(&err);
    if (st) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    unsigned int *slot = nullptr;
    {
        int dev = 0;
        cudaGetDevice(&dev);
        std::lock_guard<std::mutex> lk(g_mu);
        slot = g_snap_ptr[dev] + (g_snap_next++ % kErrSlots);
    }
    unsigned int host = 0;
    take_error_kernel<<<1, 1, 0, s>>>(err, slot);
    if (cudaGetLastError() != cudaSuccess) return GDR_ERR_LAUNCH;
    if (cudaMemcpyAsync(&host, slot, sizeof(host), cudaMemcpyDeviceToHost, s) != cudaSuccess) return GDR_ERR_LAUNCH;
    if (cudaStreamSynchronize(s) != cudaSuccess) return GDR_ERR_LAUNCH;
    *device_error = (int)host;
    return GDR_OK;
}

extern "C" const char *gdr_status_string(int status) {
    switch (status) {
        case GDR_OK: return "ok";
        case GDR_ERR_SHAPE: return "invalid shape or size argument";
        case GDR_ERR_DTYPE: return "unsupported dtype";
        case GDR_ERR_NULL: return "a required pointer is NULL";
        case GDR_ERR_ALIGN: return "a pointer is not 16-byte aligned";
        case GDR_ERR_UNSUPPORTED: return "head size not built (Dk and Dv must be 16, 32, 64 or 128)";
        case GDR_ERR_DEVICE: return "no usable sm_100 CUDA device";
        case GDR_ERR_LAUNCH: return "a CUDA call or kernel launch failed";
        case GDR_ERR_WORKSPACE: return "workspace smaller than the call's workspace query returns";
        default: return "unknown status";
    }
}

extern "C" int gdr_version(void) { return 200; }

extern "C" int gdr_debug_set_wait_limit(unsigned long long ns) {
    chunk_tc_set_wait_ns(ns);
    return GDR_OK;
}

extern "C" int gdr_debug_timeout_site(unsigned int *site) {
    if (!site) return GDR_ERR_NULL;
    *site = 0;
    unsigned int *err = nullptr;
    int st = device_setup(&err);
    if (st) return st;
    unsigned int one = 0, two = 0;
    if (chunk_tc_take_timeout_site(&one) != cudaSuccess || chunk_wy_take_timeout_site(&two) != cudaSuccess)
        return GDR_ERR_LAUNCH;
    *site = one ? one : two;
    return GDR_OK;
}

extern "C" int gdr_debug_set_chunk_schedule(int schedule) {
    if (schedule < 0 || schedule > 2) return GDR_ERR_SHAPE;
    g_chunk_schedule = schedule;
    return GDR_OK;
}
