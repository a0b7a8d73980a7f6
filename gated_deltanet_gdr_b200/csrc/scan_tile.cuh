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

#include "kernels.h"
#include "pairs.cuh"
#include "sm100.cuh"

namespace gdr {
namespace scan {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRanks = 8;  // most blocks of a cluster (the portable limit)

// a = e^g, and (kRest) rest = 1 - e^g, of a pair.  Near 0 the Taylor series, whose first dropped term is below a tenth
// of a rounding (2^-24) of a for |g| < 1/8, or below one rounding of the rest for |g| < 1/4: the rest keeps its digits, and
// a decay close to 1 is good to a rounding -- it is applied hundreds of times, and what ex2.approx loses (up to 2^-22)
// would add up.  Elsewhere ex2(g log2 e), whose argument is rounded once more (|g| 2^-24): there a state fades soon.
template <bool kRest> __device__ __forceinline__ void decay(float g, float &a, float &rest) {
    const float far = ex2(g * 1.4426950408889634f);
    if (kRest) {  // -g (1 + g/2 + ... + g^5/720)
        float p = fmaf(g, -1.f / 720.f, -1.f / 120.f);
        p = fmaf(p, g, -1.f / 24.f);
        p = fmaf(p, g, -1.f / 6.f);
        p = fmaf(p, g, -0.5f);
        p = fmaf(p, g, -1.f);
        const float near = p * g;
        const bool s = fabsf(g) < 0.25f;
        rest = s ? near : 1.f - far;
        a = s ? 1.f - near : far;
    } else {  // 1 + g + ... + g^5/120
        float p = fmaf(g, 1.f / 120.f, 1.f / 24.f);
        p = fmaf(p, g, 1.f / 6.f);
        p = fmaf(p, g, 0.5f);
        p = fmaf(p, g, 1.f);
        p = fmaf(p, g, 1.f);
        a = fabsf(g) < 0.125f ? p : far;
    }
}
template <bool kRest> __device__ __forceinline__ void decay(float2 g, float2 &a, float2 &rest) {
    float g0, g1, a0, a1, r0 = 0.f, r1 = 0.f;
    up2(g, g0, g1);
    decay<kRest>(g0, a0, r0);
    decay<kRest>(g1, a1, r1);
    a = make_float2(a0, a1);
    rest = make_float2(r0, r1);
}

// length of sequence b, or -1 for one outside [0, S]
__device__ __forceinline__ int seq_len(const int32_t *lengths, int b, int S) {
    const int L = lengths ? lengths[b] : S;
    return (L < 0 || L > S) ? -1 : L;
}

// ---- clusters -----------------------------------------------------------------------------------------------------

// every thread of every block of the cluster passes together; orders no memory but mbarrier initialisations fenced before
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();  // the barrier is for whole warps, whose lanes may have left a wait apart
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// writes V floats at `p` and their bytes to the count of `bar` (both given as this block's addresses) in block `rank`
template <int V> __device__ __forceinline__ void put_remote(const float *p, const uint64_t *bar, int rank, const float2 (&v)[kPairs<V>]) {
    float x[2 * kPairs<V>];
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) up2(v[i], x[2 * i], x[2 * i + 1]);
    unsigned a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(sm100::smem_u32(p)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(sm100::smem_u32(bar)), "r"(rank));
    if constexpr (V == 4)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
                     "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "r"(b)
                     : "memory");
    else if constexpr (V == 2)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(a), "f"(x[0]),
                     "f"(x[1]), "r"(b)
                     : "memory");
    else
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(a), "f"(x[0]), "r"(b)
                     : "memory");
}
// waits, for at most limit_ns, until the phase of `bar` with this parity has completed: the bytes of every block of the
// cluster are there to be read.  A limit shorter than the global timer's steps is over at the first test that fails.
__device__ __forceinline__ bool wait_remote(uint64_t *bar, unsigned parity, uint64_t limit_ns) {
    constexpr uint64_t kTimerStep = 1024;
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(sm100::smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (limit_ns < kTimerStep) return false;
    const uint64_t t0 = sm100::global_ns();
    for (;;) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.b32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(sm100::smem_u32(bar)), "r"(parity), "r"(limit_ns < 0x10000ull ? (unsigned)limit_ns : 0x10000u)
            : "memory");
        if (ok) return true;
        if (sm100::global_ns() - t0 >= limit_ns) return false;
    }
}

// ---- leaving a cluster ---------------------------------------------------------------------------------------------
//
// Warp w of a block sends its tiles' (A, B) to block w, and thread 0 counts what the block receives.  A warp whose wait for
// a tile runs out waits for no later tile, sends none and (the first warp) counts none, but walks on through its tokens: so
// the phase of an mbarrier is only ever begun with the phase before it complete.  A block leaves when every byte that the
// others send to its shared memory has landed: at its end each warp tells its block how many tiles it has sent there, and
// thread 0 waits for what is still on its way.

constexpr uint64_t kDrainNs = 1000000000ull;  // more than a tile's limit that these waits are given: the others end theirs first

// tells block `rank` that `tiles` tiles have been sent there (sent and closed given as this block's addresses)
__device__ __forceinline__ void tell_sent(const int *sent, const uint64_t *closed, int rank, int tiles) {
    unsigned a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(sm100::smem_u32(sent)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(sm100::smem_u32(closed)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(a), "r"(tiles), "r"(b)
                 : "memory");
}
// Where a wait ran out: thread 0, having counted `mine` tiles, waits (bounded) until what every block r has sent to this
// one, its tiles before sent[r], is there.  All tiles before mine - 1 have been received here.  The phase of tile mine - 1
// expects the bytes of all blocks and gets those of the ones that sent it.  A warp sends tile t having received tile t - 1 of
// all blocks; this block's warps send tile mine at most, since mine - 1 is the last one counted, so nobody sends more
// than tile mine + 1: the phases of tiles mine and mine + 1 have only the bytes of the blocks ahead.  bytes: of one
// block's (A, B) of a tile.
static __device__ __noinline__ bool drain(uint64_t *arrived, const int *sent, int R, int mine, unsigned bytes, uint64_t limit_ns) {
    for (int t = mine > 0 ? mine - 1 : 0; t < mine + 2; ++t) {
        unsigned n = 0;  // blocks that sent tile t
        for (int r = 0; r < R; ++r) n += sent[r] > t;
        uint64_t *bar = &arrived[t & 1];
        if (t >= mine) {
            if (n == 0) break;
            sm100::mbar_arrive_expect_tx(bar, n * bytes);
        } else if (n < (unsigned)R) {
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(sm100::smem_u32(bar)),
                         "r"((R - n) * bytes)
                         : "memory");
        }
        if (!wait_remote(bar, (unsigned)(t >> 1) & 1u, limit_ns)) return false;
    }
    return true;
}
// Thread 0 at a block's end: waits (bounded) until every byte sent to this block is there; false if a wait ran out.  got:
// tiles that its warp has received
__device__ __forceinline__ bool all_landed(uint64_t *arrived, uint64_t *closed, const int *sent, int R, int got, int tiles,
                                           unsigned bytes, uint64_t limit_ns) {
    limit_ns = limit_ns < ~0ull - kDrainNs ? limit_ns + kDrainNs : limit_ns;
    if (!wait_remote(closed, 0u, limit_ns)) return false;
    bool all = got == tiles;
    for (int r = 0; r < R; ++r) all = all && sent[r] == tiles;
    return all || drain(arrived, sent, R, got + 1 < tiles ? got + 1 : tiles, bytes, limit_ns);
}

// ---- the cut -------------------------------------------------------------------------------------------------------

// whether rows are made of whole 16 bytes: tiles are then staged by warps
template <typename T> bool rows_of_16(int D) { return D * (long long)sizeof(T) % 16 == 0; }

struct Cut {
    int lx;     // lanes side by side over the channels, a power of two from 4 to 32
    int slabs;  // tiles over the channels
    int ranks;  // blocks of a cluster: consecutive tiles in time
    double estimate;
};

// The cut of the least estimated time.  A block spends about the same time on every tile, whatever its shape (a little
// more with fewer lanes, for the shuffles; `wide` with 32, which need none), so a cut costs the tiles that a block
// walks through, times what the blocks of the fullest SM cost together: 1 for one, 0.8 more for each of the up to
// `resident` that share it at a time.  A cluster lies within one of the GPU's groups of SMs, which are not multiples of
// it: kFit, as the occupancy query reports it. Measured, forward, sustained, us: 640 channels and 32769 tokens, 4 lanes (40
// clusters, at most two on an SM): 55 with clusters of 6 (22 fit side by side), 61 of 5, 76 of 7 and 81 of 8 (15 fit); 8
// lanes (20 clusters): 57 of 6, 66 of 5, 71 of 8, 78 of 7; 128 rows of 128 channels and 4096 tokens: 96 with 32 lanes and 2
// blocks, 103 with 16 and 1, 106 with 32 and 1, 110 with 8 and 1; 64 channels and 65536 tokens: 47 with 4 lanes and 8
// blocks, 84 with 8 lanes.
inline Cut choose_cut(long long rows, int D, int V, int S, int TS, int max_lx, int min_lx, int resident, double wide) {
    // clusters of 1 .. 8 blocks that a B200 of 148 SMs holds with one block on an SM
    constexpr int kFit[kMaxRanks] = {148, 74, 45, 33, 26, 22, 15, 15};
    const int sms = sm_count();
    auto together = [&](long long n) {
        auto share = [](long long m) { return m ? 1.0 + 0.8 * (double)(m - 1) : 0.0; };
        return (double)(n / resident) * share(resident) + share(n % resident);
    };
    Cut best{};
    for (int lx = max_lx; lx >= min_lx; lx /= 2) {
        const long long slabs = (D + (long long)lx * V - 1) / ((long long)lx * V), clusters = rows * slabs;
        const long long tile = (long long)TS * (kThreads / lx);
        const double shuffles = lx == 32 ? wide : lx == 16 ? 0.93 : lx == 8 ? 1.0 : 1.11;
        for (int r = 1; r <= kMaxRanks && (r == 1 || (r - 1) * tile < S); ++r) {
            const long long fit = kFit[r - 1] * sms >= 148 ? kFit[r - 1] * sms / 148 : 1;
            const double t = shuffles * (1.0 + 0.02 * r) * (double)((S + r * tile - 1) / (r * tile)) *
                             together((clusters + fit - 1) / fit);
            if (!best.lx || t < best.estimate) {
                best.lx = lx;
                best.slabs = (int)slabs;
                best.ranks = r;
                best.estimate = t;
            }
        }
    }
    return best;
}

template <typename Args>
cudaError_t launch_clusters(void (*kernel)(Args, Cut), long long rows, const Cut &cut, int smem, const Args &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * cut.slabs * cut.ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cut.ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cut.ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, cut);
}

}  // namespace scan
}  // namespace gdr
