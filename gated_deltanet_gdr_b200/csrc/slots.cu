// slots.cu -- copying, forking, compacting and freeing slots of the state pools (gdr_slot_copy, gdr_slot_fork,
// gdr_slot_compact, gdr_slot_free).
//
// All four are moves of whole slots (or zero fills).  A slot is counted in units of kUnit bytes, and the units of all
// moves are dealt out evenly, in runs, to the resident blocks.  Which slots move is worked out on the device: every
// block derives the same plan from the index arrays in its own shared memory, so one launch does everything and the
// host never waits for a count.  Bound by HBM: 128 slots of 1.1 MB copied (285 MB moved) in 54 us a call, one call
// after another, 5.3 TB/s, 80 % of the measured copy rate.
#include "common.cuh"
#include "kernels.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kUnit = kThreads * 16;  // bytes of a unit: one 16-byte access of every thread
constexpr int kBatch = 8;                  // units whose loads are all issued before the first store

// units of all pools of one slot, counted up: unit q belongs to the pool p with first[p] <= q < first[p + 1]
struct Units {
    unsigned first[GDR_MAX_POOLS + 1];
};

__device__ __forceinline__ void count_units(const SlotPools &p, Units &us) {
    if (threadIdx.x == 0) {
        unsigned at = 0;
        for (int i = 0; i < p.n; ++i) {
            us.first[i] = at;
            at += (unsigned)((p.bytes[i] + kUnit - 1) / kUnit);
        }
        us.first[p.n] = at;
    }
    __syncthreads();
}

// up to kBatch units in elements of U; src NULL: zeros.  What is written leaves the L2 cache first, so that sources which
// several moves share stay (96 copies of 1.1 MB from random sources, in a graph: 35.9 us, 36.2 with plain stores; 64 beams
// with random parents: 13.2 with either).
template <typename U>
__device__ __forceinline__ void move_elements(const char *src, char *dst, unsigned bytes) {
    const unsigned n = bytes / sizeof(U);
    const U *s = reinterpret_cast<const U *>(src);
    U *d = reinterpret_cast<U *>(dst);
    for (unsigned i = threadIdx.x; i < n; i += kThreads * kBatch) {
        U v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            v[k] = U{};
            if (src && i + k * kThreads < n) v[k] = s[i + k * kThreads];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (i + k * kThreads < n) __stcs(d + i + k * kThreads, v[k]);
    }
}

// moves units q .. of slot src (negative: zeros) to slot dst, at most `most` and kBatch of them, all of one pool; returns
// how many
__device__ __forceinline__ unsigned move_units(const SlotPools &p, const Units &us, unsigned q, unsigned long long most, int src,
                                               int dst) {
    int i = 0;
    while (q >= us.first[i + 1]) ++i;
    unsigned run = us.first[i + 1] - q;
    if (run > (unsigned)kBatch) run = kBatch;
    if (run > most) run = (unsigned)most;
    const unsigned long long sb = p.bytes[i], off = (unsigned long long)(q - us.first[i]) * kUnit;
    const unsigned n = (unsigned)(sb - off < run * kUnit ? sb - off : run * kUnit);
    const char *s = src < 0 ? nullptr : p.data[i] + (unsigned long long)src * sb + off;
    char *d = p.data[i] + (unsigned long long)dst * sb + off;
    // slots begin on the largest power of two up to 16 that divides their size
    if ((sb & 15) == 0) move_elements<uint4>(s, d, n);
    else if ((sb & 7) == 0) move_elements<uint2>(s, d, n);
    else if ((sb & 3) == 0) move_elements<unsigned>(s, d, n);
    else if ((sb & 1) == 0) move_elements<unsigned short>(s, d, n);
    else move_elements<unsigned char>(s, d, n);
    return run;
}

// Index lists of up to this many entries are read into shared memory once, so that what a block looks up between its moves
// does not wait for memory (64 beams of 1.1 MB, in a graph: 13.5 us without this, 13.2 with it).
constexpr int kCached = 4096;

// both lists, from shared memory where they fit; the whole block takes part (and passes a barrier afterwards)
__device__ __forceinline__ void cache_lists(int *buf, int n, const int32_t *&a, const int32_t *&b) {
    if (n > kCached) return;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        buf[i] = a[i];
        buf[n + i] = b[i];
    }
    a = buf;
    b = buf + n;
}
constexpr int cached_bytes(int n) { return n <= kCached ? 2 * n * (int)sizeof(int) : 0; }

// this block's share [lo, hi) of n units
__device__ __forceinline__ void share(unsigned long long n, unsigned long long &lo, unsigned long long &hi) {
    lo = n * blockIdx.x / gridDim.x;
    hi = n * (blockIdx.x + 1) / gridDim.x;
}

__global__ void __launch_bounds__(kThreads) slot_copy_kernel(const SlotPools p, const int32_t *src, const int32_t *dst,
                                                             int n) {
    extern __shared__ unsigned smem[];
    __shared__ Units us;
    cache_lists(reinterpret_cast<int *>(smem), n, src, dst);
    count_units(p, us);
    const unsigned per = us.first[p.n];
    unsigned long long lo, hi;
    share((unsigned long long)n * per, lo, hi);
    int now = -1, s = -1, d = -1;
    bool go = false;
    for (unsigned long long it = lo; it < hi;) {
        const int i = (int)(it / per);
        const unsigned q = (unsigned)(it - (unsigned long long)i * per);
        if (i != now) {  // the same for the whole block
            now = i;
            s = src[i];
            d = dst[i];
            go = s != -1 && d != -1 && s != d;
            if (go) {
                bool clash = (unsigned)s >= (unsigned)p.slots || (unsigned)d >= (unsigned)p.slots;
                if (!clash) {
                    for (int j = threadIdx.x; j < n; j += kThreads) {
                        const int sj = src[j], dj = dst[j];
                        if (j == i || sj == dj || (unsigned)sj >= (unsigned)p.slots || (unsigned)dj >= (unsigned)p.slots)
                            continue;
                        clash |= sj == d || (dj == d && j < i);
                    }
                }
                clash = __syncthreads_or(clash);
                if (clash) {
                    if (threadIdx.x == 0) raise_device_error(p.err, GDR_DEVERR_SLOT_INDEX);
                    go = false;
                }
            }
        }
        it += go ? move_units(p, us, q, hi - it, s, d) : per - q;
    }
}

__global__ void __launch_bounds__(kThreads) slot_free_kernel(const SlotPools p, const int32_t *idx, int n,
                                                             int32_t *live) {
    __shared__ Units us;
    count_units(p, us);
    const unsigned per = us.first[p.n];
    unsigned long long lo, hi;
    share((unsigned long long)n * per, lo, hi);
    for (unsigned long long it = lo; it < hi;) {
        const int i = (int)(it / per);
        const unsigned q = (unsigned)(it - (unsigned long long)i * per);
        const int d = idx[i];
        if ((unsigned)d >= (unsigned)p.slots) {
            if (d != -1 && q == 0 && threadIdx.x == 0) raise_device_error(p.err, GDR_DEVERR_SLOT_INDEX);
            it += per - q;
            continue;
        }
        if (live && q == 0 && threadIdx.x == 0) live[d] = 0;
        it += move_units(p, us, q, hi - it, -1, d);
    }
}

// ---- sets as bitmaps with the number of members before each word: rank and selection without lists ------------

struct Bits {
    unsigned *word, *before;  // before[w]: members in the words before w; before[words]: all
    int words;
};

// members of the set below i
__device__ __forceinline__ int rank_of(const Bits &b, int i) {
    return (int)(b.before[i >> 5] + __popc(b.word[i >> 5] & ((1u << (i & 31)) - 1u)));
}

// the k-th member (k < before[words])
__device__ __forceinline__ int member(const Bits &b, unsigned k) {
    int lo = 0, hi = b.words;  // before[lo] <= k < before[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (b.before[m] <= k) lo = m;
        else hi = m;
    }
    unsigned w = b.word[lo];
    for (unsigned r = k - b.before[lo]; r > 0; --r) w &= w - 1;
    return lo * 32 + __ffs(w) - 1;
}

// fills before[] from word[]; the whole block takes part
__device__ __forceinline__ void count_words(const Bits &b) {
    __shared__ unsigned warp_sum_[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (b.words + kThreads - 1) / kThreads, w0 = min((int)threadIdx.x * per, b.words),
              w1 = min(w0 + per, b.words);
    unsigned mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(b.word[w]);
    unsigned inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) warp_sum_[warp] = inc;
    __syncthreads();
    unsigned at = inc - mine;
    for (int i = 0; i < warp; ++i) at += warp_sum_[i];
    for (int w = w0; w < w1; ++w) {
        b.before[w] = at;
        at += __popc(b.word[w]);
    }
    if (threadIdx.x == kThreads - 1) b.before[b.words] = at;  // at: all members, whatever this thread's own share
    __syncthreads();
}

__host__ __device__ constexpr int words_of(int n) { return (n + 31) / 32; }

__global__ void __launch_bounds__(kThreads) slot_fork_kernel(const SlotPools p, const int32_t *table,
                                                             const int32_t *parents, int n, int32_t *new_table) {
    extern __shared__ unsigned smem[];
    __shared__ Units us;
    const int W = words_of(n);
    int *first = reinterpret_cast<int *>(smem);  // the lowest row that continues from row r, n if none
    Bits extra{smem + n, smem + n + W, W};       // rows that take another row's slot
    Bits dead{smem + n + 2 * W + 1, smem + n + 3 * W + 1, W};  // rows nobody continues from
    cache_lists(first + n + 4 * W + 2, n, table, parents);
    for (int i = threadIdx.x; i < n; i += kThreads) first[i] = n;
    count_units(p, us);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int r = parents[i];
        if ((unsigned)r < (unsigned)n) atomicMin(&first[r], i);
        else if (r != -1 && blockIdx.x == 0) raise_device_error(p.err, GDR_DEVERR_SLOT_INDEX);
    }
    __syncthreads();
    for (int i0 = 0; i0 < W * 32; i0 += kThreads) {  // whole warps: kThreads is a multiple of 32
        const int i = i0 + threadIdx.x;
        const int r = i < n ? parents[i] : 0;
        const unsigned e = __ballot_sync(0xffffffffu, i < n && !((unsigned)r < (unsigned)n && first[r] == i));
        const unsigned d = __ballot_sync(0xffffffffu, i < n && first[i < n ? i : 0] == n);
        if ((threadIdx.x & 31) == 0 && (i >> 5) < W) {
            extra.word[i >> 5] = e;
            dead.word[i >> 5] = d;
        }
    }
    __syncthreads();
    count_words(extra);
    count_words(dead);
    // as many rows take another slot as slots are left: n less the rows that are continued
    const unsigned moves = extra.before[W], per = us.first[p.n];
    if (blockIdx.x == gridDim.x - 1)
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int r = parents[i];
            const bool keeps = (unsigned)r < (unsigned)n && first[r] == i;
            new_table[i] = table[keeps ? r : member(dead, rank_of(extra, i))];
        }
    unsigned long long lo, hi;
    share((unsigned long long)moves * per, lo, hi);
    long long now = -1;
    int s = -1, d = -1;
    bool go = false;
    for (unsigned long long it = lo; it < hi;) {
        const unsigned k = (unsigned)(it / per), q = (unsigned)(it - (unsigned long long)k * per);
        if (k != now) {
            now = k;
            const int row = member(dead, k), r = parents[member(extra, k)];
            go = (unsigned)r < (unsigned)n;
            if (go) {
                s = table[r];
                d = table[row];
                bool clash = (unsigned)s >= (unsigned)p.slots || (unsigned)d >= (unsigned)p.slots;
                if (!clash)
                    for (int j = threadIdx.x; j < n; j += kThreads) clash |= j != row && table[j] == d;
                clash = __syncthreads_or(clash);
                if (clash) {
                    if (threadIdx.x == 0) raise_device_error(p.err, GDR_DEVERR_SLOT_INDEX);
                    go = false;
                }
            }
        }
        it += go ? move_units(p, us, q, hi - it, s, d) : per - q;
    }
}

__global__ void __launch_bounds__(kThreads) slot_compact_kernel(const SlotPools p, const int32_t *live,
                                                                int32_t *new_slot, int32_t *n_live) {
    extern __shared__ unsigned smem[];
    __shared__ Units us;
    count_units(p, us);
    const int n = p.slots, W = words_of(n);
    Bits used{smem, smem + W, W}, hole{smem + 2 * W + 1, smem + 3 * W + 1, W};
    for (int i0 = 0; i0 < W * 32; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        const unsigned u = __ballot_sync(0xffffffffu, i < n && live[i < n ? i : 0] != 0);
        if ((threadIdx.x & 31) == 0 && (i >> 5) < W) {
            used.word[i >> 5] = u;
            hole.word[i >> 5] = ~u & (n - (i & ~31) >= 32 ? 0xffffffffu : (1u << (n - (i & ~31))) - 1u);
        }
    }
    __syncthreads();
    count_words(used);
    count_words(hole);
    const int all = (int)used.before[W];
    const int stay = all < n ? rank_of(used, all) : all;  // live slots that are in place already
    const unsigned moves = (unsigned)(all - stay), per = us.first[p.n];
    if (blockIdx.x == 0 && threadIdx.x == 0) *n_live = all;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) {
        const bool u = used.word[i >> 5] >> (i & 31) & 1;
        new_slot[i] = !u ? -1 : i < all ? i : member(hole, rank_of(used, i) - stay);
    }
    unsigned long long lo, hi;
    share((unsigned long long)moves * per, lo, hi);
    long long now = -1;
    int s = 0, d = 0;
    for (unsigned long long it = lo; it < hi;) {
        const unsigned k = (unsigned)(it / per), q = (unsigned)(it - (unsigned long long)k * per);
        if (k != now) {
            now = k;
            s = member(used, stay + k);
            d = member(hole, k);
        }
        it += move_units(p, us, q, hi - it, s, d);
    }
}

LaunchCache copy_cache(reinterpret_cast<const void *>(slot_copy_kernel));
LaunchCache free_cache(reinterpret_cast<const void *>(slot_free_kernel));
LaunchCache fork_cache(reinterpret_cast<const void *>(slot_fork_kernel));
LaunchCache compact_cache(reinterpret_cast<const void *>(slot_compact_kernel));

// blocks: all that are resident at once, but no more than there can be units
cudaError_t grid_for(LaunchCache &c, const SlotPools &p, long long slots, int smem, int *grid) {
    cudaError_t e = c.allow_smem(smem);
    if (e != cudaSuccess) return e;
    e = c.resident_grid(kThreads, smem, grid);
    if (e != cudaSuccess) return e;
    unsigned long long per = 0;
    for (int i = 0; i < p.n; ++i) per += (p.bytes[i] + kUnit - 1) / kUnit;
    const unsigned long long units = per * (unsigned long long)slots;
    if (units < (unsigned long long)*grid) *grid = units > 0 ? (int)units : 1;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_slot_copy(const SlotPools &p, const int32_t *src, const int32_t *dst, int n, cudaStream_t s) {
    int grid = 0;
    const int smem = cached_bytes(n);
    cudaError_t e = grid_for(copy_cache, p, n, smem, &grid);
    if (e != cudaSuccess) return e;
    slot_copy_kernel<<<grid, kThreads, smem, s>>>(p, src, dst, n);
    return cudaGetLastError();
}

cudaError_t launch_slot_free(const SlotPools &p, const int32_t *idx, int n, int32_t *live, cudaStream_t s) {
    int grid = 0;
    cudaError_t e = grid_for(free_cache, p, n, 0, &grid);
    if (e != cudaSuccess) return e;
    slot_free_kernel<<<grid, kThreads, 0, s>>>(p, idx, n, live);
    return cudaGetLastError();
}

cudaError_t launch_slot_fork(const SlotPools &p, const int32_t *table, const int32_t *parents, int n,
                             int32_t *new_table, cudaStream_t s) {
    int grid = 0;
    const int smem = (n + 4 * words_of(n) + 2) * (int)sizeof(unsigned) + cached_bytes(n);
    cudaError_t e = grid_for(fork_cache, p, n, smem, &grid);
    if (e != cudaSuccess) return e;
    slot_fork_kernel<<<grid, kThreads, smem, s>>>(p, table, parents, n, new_table);
    return cudaGetLastError();
}

cudaError_t launch_slot_compact(const SlotPools &p, const int32_t *live, int32_t *new_slot, int32_t *n_live,
                                cudaStream_t s) {
    int grid = 0;
    const int smem = (4 * words_of(p.slots) + 2) * (int)sizeof(unsigned);
    cudaError_t e = grid_for(compact_cache, p, p.slots, smem, &grid);
    if (e != cudaSuccess) return e;
    slot_compact_kernel<<<grid, kThreads, smem, s>>>(p, live, new_slot, n_live);
    return cudaGetLastError();
}

}  // namespace gdr
