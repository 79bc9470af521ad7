// Page operations of paged caches: reserving blocks for the tokens to come (with the
// window's blocks given back and shared blocks copied before they are written), forking and
// releasing requests, and compacting the pool.
//
// "vLLM, from the inside out", PagedAttention: a shared pool of fixed-size blocks and a
// block table per request.  ref[block] counts the table entries (and the caller's own
// holds) that name a block; 0 is free.  The state lives on the device, so a serving loop
// reserves, appends and attends without a copy to the host.
//
// Everything is decided by prefix sums over (request, block index) and over block ids, never
// by the order in which atomics land: the k-th block wanted gets the k-th free id.  The
// decisions are integers over a few hundred KB, bound by the latency of a handful of
// dependent steps, so each call's bookkeeping is one launch of one cluster of 8 blocks whose
// barriers separate the steps (a grid-wide barrier in hardware; a launch per step took
// 2-3 us each); pages are moved by a second launch, at the rate of the memory, unless they are
// few.
#include <algorithm>

#include "common.cuh"

namespace sk {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kAllWarps = kCluster * kWarps;
constexpr int kMaxBatch = kThreads;   // a thread per request in the scans
constexpr int kMaxLayers = 128;

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Inclusive sum over the block's threads; `total` the sum of all.  s: kWarps ints of shared memory.
__device__ __forceinline__ int block_scan(int x, int* s, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s[warp] = x;
    __syncthreads();
    int sum = s[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += y;
    }
    *total = __shfl_sync(kFull, sum, 31);
    const int before = __shfl_sync(kFull, sum, warp > 0 ? warp - 1 : 0);
    __syncthreads();
    return x + (warp > 0 ? before : 0);
}

// The block ids that a warp of the cluster looks through: [lo, hi), in the order of the warps.
struct IdRange {
    int64_t lo, hi;
    __device__ __forceinline__ IdRange(int64_t n, int warp_of_all) {
        const int64_t per = (n + 32 * kAllWarps - 1) / (32 * kAllWarps) * 32;
        lo = min(n, per * warp_of_all);
        hi = min(n, lo + per);
    }
};

// What comes before this warp in an array of one count per warp of the cluster (global
// memory, written before a cluster barrier; x: thread i's is count i), and the sum of all.
// Every thread of the block must call this.  s: kAllWarps + kWarps ints of shared memory.
__device__ __forceinline__ int count_of(const int32_t* counts) {  // this thread's count, for before_warp
    return threadIdx.x < kAllWarps ? __ldcg(counts + threadIdx.x) : 0;
}

__device__ __forceinline__ int before_warp(int x, int warp_of_all, int* s, int* total) {
    const int inc = block_scan(x, s + kAllWarps, total);
    if (threadIdx.x < kAllWarps) s[threadIdx.x] = inc - x;
    __syncthreads();
    const int r = s[warp_of_all];
    __syncthreads();
    return r;
}

// ---------------------------------------------------------------------------
// Moving pages
// ---------------------------------------------------------------------------

struct MoveParams {
    void* pool[2 * kMaxLayers];
    int32_t bytes[2 * kMaxLayers];  // of a page of the pool
    int n_pools;
    int pieces;          // of kPiece bytes in the largest page
    const int32_t* src;  // move i: block src[i * stride] to dst[i * stride]
    const int32_t* dst;
    const int32_t* n;    // moves, on the device
    int stride;
    // compact: the tables to rewrite, or null
    const int32_t* map;
    int32_t* table;
    int64_t entries, NB;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;
constexpr int kPiece = 32 * 16 * kMoveUnroll;  // bytes a warp moves at a time

// Warp `warp` of `warps` takes every warps-th piece of 4 KB of the n moves in all pools, 8 loads
// of 16 bytes a lane in flight; the ids of its next piece are on their way meanwhile.  (Pools one
// after the other, each with its ids to wait for, took 0.4 us a pool.)  Pieces are counted as if
// every page were the largest.  The moves' blocks are all different: sources are in use,
// destinations were free.
__device__ __forceinline__ void move_pieces(const MoveParams& p, uint32_t n, uint32_t warp, uint32_t warps, int lane) {
    const uint32_t pieces = uint32_t(p.pieces), pools = uint32_t(p.n_pools);
    if (n == 0 || pools == 0) return;
    const uint32_t step_m = warps / pieces, step_pc = warps % pieces;
    uint32_t m = warp / pieces, pc = warp % pieces, l = m / n;
    m %= n;
    if (l >= pools) return;
    int32_t from = __ldcg(p.src + int64_t(m) * p.stride), to = __ldcg(p.dst + int64_t(m) * p.stride);
    for (;;) {
        const int bytes = p.bytes[l];
        const int64_t at = int64_t(pc) * kPiece + lane * 16;
        uint8_t* const pool = static_cast<uint8_t*>(p.pool[l]);
        const uint8_t* a = pool + int64_t(from) * bytes + at;
        uint8_t* b = pool + int64_t(to) * bytes + at;
        uint4 v[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (at + u * 512 < bytes) v[u] = __ldcs(reinterpret_cast<const uint4*>(a + u * 512));
        pc += step_pc;
        m += step_m;
        if (pc >= pieces) {
            pc -= pieces;
            ++m;
        }
        if (m >= n) {
            l += m / n;
            m %= n;
        }
        const bool more = l < pools;
        if (more) {
            from = __ldcg(p.src + int64_t(m) * p.stride);
            to = __ldcg(p.dst + int64_t(m) * p.stride);
        }
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (at + u * 512 < bytes) __stcs(reinterpret_cast<uint4*>(b + u * 512), v[u]);
        if (!more) return;
    }
}

__global__ void __launch_bounds__(kMoveThreads) move_pages_kernel(const __grid_constant__ MoveParams p) {
    pdl_trigger();
    pdl_wait();
    if (p.map != nullptr) {
        for (int64_t i = int64_t(blockIdx.x) * kMoveThreads + threadIdx.x; i < p.entries;
             i += int64_t(gridDim.x) * kMoveThreads) {
            const int32_t e = p.table[i];
            if (e >= 0 && e < p.NB) {
                const int32_t to = p.map[e];
                if (to != e) p.table[i] = to;
            }
        }
    }
    move_pieces(p, uint32_t(*p.n), blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5),
                gridDim.x * (kMoveThreads / 32), threadIdx.x & 31);
}

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------

struct ReserveParams {
    int32_t* table;        // [B][MB]
    int32_t* ref;          // [NB]
    const int64_t* lens;   // [B]
    const int32_t* n_new;  // [B] or null: 1 each
    int32_t* granted;      // [B]
    uint32_t* err;
    int64_t NB;
    int B, MB, bs_log2, S, W, sink_len;
    // workspace
    int32_t* free_ids;     // [NB] the free ids in ascending order, as many as are wanted
    int32_t* old_ids;      // [NB] the shared block that free_ids[i] takes the place of, or -1
    int32_t* need;         // [B] blocks wanted; kRefused, kNothing
    int32_t* shared_of;    // [B] the shared block in which the request's next token falls, or -1
    int32_t* copies;       // [n_copies][2] a block to copy and its copy
    int32_t* n_copies;
    int32_t* counts;       // [kAllWarps]
};

constexpr int kMostBlocks = 1 << 20;  // for one request in one call: the scans are 32-bit sums of kMaxBatch of them
constexpr int kRefused = -1;  // the request cannot be served whatever the pool holds
constexpr int kNothing = -2;  // nothing asked for

// Table entries a lane looks at together.  More overlap more loads, but a call runs most of its
// code once and waits for the instructions (measured: 8 take 2.3 us longer than 2).
constexpr int kAhead = 2;

// The request's part of a block table row that its new tokens fall into.
struct Wanted {
    int64_t len;
    int64_t n;          // new tokens
    int first, last;    // table entries [first, last]
    bool partial;       // entry `first` holds tokens already
    bool fits;
    __device__ __forceinline__ Wanted(const ReserveParams& p, int64_t length, int new_tokens) {
        len = length;
        n = new_tokens;
        fits = len >= 0 && len + n <= (int64_t(p.MB) << p.bs_log2);
        first = fits ? int(len >> p.bs_log2) : 0;
        last = fits && n > 0 ? int((len + n - 1) >> p.bs_log2) : -1;
        partial = fits && n > 0 && (len & ((int64_t(1) << p.bs_log2) - 1)) != 0;
    }
};

// Table entries j, j + 32, .. up to `last`: the block, or -1 for one outside the pool (or past
// `last`), and whether it is shared.
__device__ __forceinline__ void load_entries(const ReserveParams& p, const int32_t* row, int64_t j, int last,
                                             int32_t* e, bool* shared) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) e[u] = j + 32 * u <= last ? row[j + 32 * u] : -1;
    int32_t r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        if (e[u] < 0 || e[u] >= p.NB) e[u] = -1;
        r[u] = e[u] >= 0 ? __ldcg(p.ref + e[u]) : 0;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) shared[u] = r[u] > 1;
}

// `moves`: the copies to make here, where they are few bytes at most; n_pools = 0 leaves them
// to move_pages_kernel.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    reserve_kernel(ReserveParams p, const __grid_constant__ MoveParams moves) {
    __shared__ int s_scan[kAllWarps + kWarps];
    __shared__ int s_shared[kMaxBatch];            // shared_of, in every block
    __shared__ int s_base[kMaxBatch];              // rank of a request's first new block, or -1: not granted
    __shared__ unsigned char s_keeps[kMaxBatch];   // the request writes its shared block where it is
    __shared__ int64_t s_len[kMaxBatch];
    __shared__ int s_new[kMaxBatch];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wa = int(blockIdx.x) * kWarps + warp;
    const int64_t bs = int64_t(1) << p.bs_log2;
    pdl_trigger();
    pdl_wait();

    if (blockIdx.x == 0 && threadIdx.x == 0) *p.n_copies = 0;
    if (threadIdx.x < p.B) {
        s_len[threadIdx.x] = p.lens[threadIdx.x];
        s_new[threadIdx.x] = p.n_new != nullptr ? p.n_new[threadIdx.x] : 1;
    }
    __syncthreads();

    // ---- give back the blocks that the window has left ----
    if (p.W > 0) {
        for (int b = wa; b < p.B; b += kAllWarps) {
            const int64_t len = s_len[b], n = s_new[b];
            // a key at logical position sink_len + i is seen by the next query (or, with no new
            // token, by the last one) while i >= keep
            const int64_t keep = len + max(int64_t(0), min(n, int64_t(1))) - p.W;
            const int64_t j0 = (max(0, p.S - p.sink_len) + bs - 1) >> p.bs_log2;
            const int64_t j1 = keep > 0 ? min(keep >> p.bs_log2, int64_t(p.MB)) : 0;
            int32_t* row = p.table + int64_t(b) * p.MB;
            for (int64_t j = j0 + lane; j < j1; j += 32 * kAhead) {
                int32_t e[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) e[u] = j + 32 * u < j1 ? row[j + 32 * u] : -1;
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (e[u] >= 0 && e[u] < p.NB) {
                        row[j + 32 * u] = -1;
                        atomicSub(p.ref + e[u], 1);
                    }
            }
        }
        cluster_sync();
    }

    // ---- what each request wants, and how many blocks are free ----
    int n_shared = 0;  // shared blocks that the warp's requests want to write
    for (int b = wa; b < p.B; b += kAllWarps) {
        const Wanted w(p, s_len[b], s_new[b]);
        int need = 0, shared = -1;
        bool ok = w.fits;
        if (w.n <= 0) {
            need = kNothing;
        } else if (ok) {
            const int32_t* row = p.table + int64_t(b) * p.MB;
            for (int64_t j0 = w.first; j0 <= w.last; j0 += 32 * kAhead) {
                int32_t e[kAhead];
                bool sh[kAhead];
                load_entries(p, row, j0 + lane, w.last, e, sh);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int64_t j = j0 + lane + 32 * u;
                    need += __popc(__ballot_sync(kFull, j <= w.last && (e[u] < 0 || sh[u])));
                    n_shared += __popc(__ballot_sync(kFull, j <= w.last && sh[u]));
                    if (j == w.first && w.partial) {
                        if (e[u] < 0) ok = false;
                        else if (sh[u]) shared = e[u];
                    }
                }
            }
            ok = __all_sync(kFull, ok);
            shared = __shfl_sync(kFull, shared, 0);  // entry `first` was lane 0's
            if (!ok && lane == 0) set_error(p.err, SK_DEVERR_BLOCK_TABLE);
            if (need > kMostBlocks) {
                ok = false;
                if (lane == 0) set_error(p.err, SK_DEVERR_CAPACITY);
            }
        } else if (lane == 0) {
            set_error(p.err, w.len < 0 ? SK_DEVERR_STATE : SK_DEVERR_CAPACITY);
        }
        if (lane == 0) {
            p.need[b] = w.n <= 0 ? kNothing : (ok ? need : kRefused);
            p.shared_of[b] = ok ? shared : -1;
        }
    }
    const IdRange ids(p.NB, wa);
    int zeros = 0;
#pragma unroll 4
    for (int64_t i = ids.lo; i < ids.hi; i += 32)
        zeros += __popc(__ballot_sync(kFull, i + lane < ids.hi && __ldcg(p.ref + i + lane) == 0));
    if (lane == 0) {
        p.counts[wa] = zeros;
        p.counts[kAllWarps + wa] = n_shared;
    }
    cluster_sync();

    // ---- who is served, from which rank on (every block works this out for itself) ----
    int n_free, unused;
    const int b = threadIdx.x;
    const int my_zeros = count_of(p.counts), my_shared = count_of(p.counts + kAllWarps);
    int need = b < p.B ? __ldcg(p.need + b) : kNothing;
    const int shared = b < p.B ? __ldcg(p.shared_of + b) : -1;
    s_shared[b] = shared;
    const int free_before = before_warp(my_zeros, wa, s_scan, &n_free);
    const bool any_shared = __syncthreads_or(my_shared > 0);  // the same in every block
    bool keeps = false;
    if (any_shared) {
        // where all that hold a shared block are about to write it, the last of them keeps it
        if (shared >= 0) {
            int writers = 0, latest = b;
            for (int o = 0; o < p.B; ++o)
                if (s_shared[o] == shared) {
                    ++writers;
                    latest = o;
                }
            keeps = latest == b && writers == __ldcg(p.ref + shared);
        }
    }
    if (keeps) --need;
    const int upto = block_scan(max(need, 0), s_scan, &unused);
    const bool grant = need != kRefused && (need == kNothing || upto <= n_free);
    int wanted;  // blocks handed out: those of the granted requests, which come first
    {
        int x = grant ? max(need, 0) : 0;
        block_scan(x, s_scan, &wanted);
    }
    s_base[b] = grant && need >= 0 ? upto - need : -1;
    s_keeps[b] = keeps;
    if (blockIdx.x == 0 && b < p.B) {
        p.granted[b] = grant ? 1 : 0;
        if (!grant && need != kRefused) set_error(p.err, SK_DEVERR_CAPACITY);
    }

    // ---- the free ids in order ----
    int rank = free_before;
    for (int64_t i = ids.lo; i < ids.hi && rank < wanted; i += 32) {
        const bool is_free = i + lane < ids.hi && __ldcg(p.ref + i + lane) == 0;
        const uint32_t m = __ballot_sync(kFull, is_free);
        const int r = rank + __popc(m & ((1u << lane) - 1));
        if (is_free && r < wanted) p.free_ids[r] = int32_t(i + lane);
        rank += __popc(m);
    }
    cluster_sync();  // also: this block's s_base and s_keeps

    // ---- tables, counts and the copies to make ----
    for (int b2 = wa; b2 < p.B; b2 += kAllWarps) {
        int base = s_base[b2];
        int src = -1, dst = -1;
        if (base >= 0) {
            const Wanted w(p, s_len[b2], s_new[b2]);
            int32_t* row = p.table + int64_t(b2) * p.MB;
            const bool keep = s_keeps[b2];
            for (int64_t j0 = w.first; j0 <= w.last; j0 += 32 * kAhead) {
                int32_t e[kAhead];
                bool sh[kAhead];  // the counts of shared blocks change below
                load_entries(p, row, j0 + lane, w.last, e, sh);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int64_t j = j0 + lane + 32 * u;
                    const bool alloc = j <= w.last && (e[u] < 0 || sh[u]) && !(keep && j == w.first);
                    const uint32_t m = __ballot_sync(kFull, alloc);
                    if (alloc) {
                        const int r = base + __popc(m & ((1u << lane) - 1));
                        const int32_t id = __ldcg(p.free_ids + r);
                        row[j] = id;
                        p.ref[id] = 1;
                        p.old_ids[r] = sh[u] ? e[u] : -1;
                        if (sh[u] && j == w.first && w.partial) {
                            src = e[u];
                            dst = id;
                        }
                    }
                    base += __popc(m);
                }
            }
        }
        src = __shfl_sync(kFull, src, 0);
        dst = __shfl_sync(kFull, dst, 0);
        if (lane == 0 && src >= 0) {  // their order decides only which warp copies which
            const int i = atomicAdd(p.n_copies, 1);
            p.copies[2 * i] = src;
            p.copies[2 * i + 1] = dst;
        }
    }
    if (!any_shared) return;
    cluster_sync();
    for (int r = int(blockIdx.x) * kThreads + threadIdx.x; r < wanted; r += kCluster * kThreads) {
        const int32_t e = __ldcg(p.old_ids + r);
        if (e >= 0) atomicSub(p.ref + e, 1);
    }
    if (moves.n_pools > 0) move_pieces(moves, uint32_t(__ldcg(moves.n)), wa, kAllWarps, lane);
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------

struct ForkParams {
    int32_t* table;
    int32_t* ref;
    const int32_t* parents;
    uint32_t* err;
    int64_t NB;
    int B, MB, table_blocks, n_lens;
    int64_t* lens[kMaxLayers];
};

constexpr int kForkCols = 8;     // table columns of a block: one 32-byte sector of each row
constexpr int kForkThreads = 256;

// Row b becomes row parents[b] as it was (-1: an empty row).  Columns are independent: a block
// holds its columns of every row in shared memory before it writes any, so no copy of the
// table is needed.  The blocks behind the last column do the same for the lengths.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const __grid_constant__ ForkParams p) {
    extern __shared__ __align__(16) int32_t s_rows[];  // [B][kForkCols], or int64 [B]
    pdl_trigger();
    pdl_wait();
    const int blk = blockIdx.x;
    if (blk >= p.table_blocks) {
        int64_t* lens = p.lens[blk - p.table_blocks];
        int64_t* s_lens = reinterpret_cast<int64_t*>(s_rows);
        for (int b = threadIdx.x; b < p.B; b += kForkThreads) s_lens[b] = lens[b];
        __syncthreads();
        for (int b = threadIdx.x; b < p.B; b += kForkThreads) {
            const int from = p.parents[b];
            if (from == b) continue;
            if (from < -1 || from >= p.B) {
                set_error(p.err, SK_DEVERR_STATE);
                continue;
            }
            lens[b] = from < 0 ? 0 : s_lens[from];
        }
        return;
    }
    const int j0 = blk * kForkCols, cols = min(kForkCols, p.MB - j0);
    for (int i = threadIdx.x; i < p.B * kForkCols; i += kForkThreads) {
        const int b = i / kForkCols, j = i % kForkCols;
        s_rows[i] = j < cols ? p.table[int64_t(b) * p.MB + j0 + j] : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.B * kForkCols; i += kForkThreads) {
        const int b = i / kForkCols, j = i % kForkCols;
        const int from = p.parents[b];
        if (j >= cols || from == b || from < -1 || from >= p.B) continue;
        const int32_t was = s_rows[i], now = from < 0 ? -1 : s_rows[from * kForkCols + j];
        if (was == now) continue;
        p.table[int64_t(b) * p.MB + j0 + j] = now;
        if (was >= 0 && was < p.NB) atomicSub(p.ref + was, 1);
        if (now >= 0 && now < p.NB) atomicAdd(p.ref + now, 1);
    }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------

struct CompactParams {
    int32_t* ref;
    int32_t* map;            // [NB] new id of each block in use, -1 for the others
    int32_t* used;           // one past the highest id in use afterwards
    const int32_t* sink_blocks;
    int64_t NB;
    int n_sinks;
    // workspace
    int32_t* src;            // [NB]
    int32_t* dst;            // [NB]
    int32_t* n_moves;
    int32_t* top_fixed;      // one past the highest static sink block in use
    int32_t* counts;         // [4][kAllWarps]
};

// Blocks in use move to the lowest ids: with the static sink blocks left where they are, the n
// others end in the first n places that are not theirs; of the blocks behind those places the
// k-th goes to the k-th free place among them.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1) compact_kernel(CompactParams p) {
    __shared__ int s_scan[kAllWarps + kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wa = int(blockIdx.x) * kWarps + warp;
    const int tid = int(blockIdx.x) * kThreads + threadIdx.x;
    const IdRange ids(p.NB, wa);
    pdl_trigger();
    pdl_wait();
    if (tid == 0) *p.top_fixed = 0;
    if (p.n_sinks > 0) {  // map = -2 marks a static sink block
        for (int64_t i = tid; i < p.NB; i += kCluster * kThreads) p.map[i] = -1;
        cluster_sync();
        for (int i = tid; i < p.n_sinks; i += kCluster * kThreads) {
            const int32_t e = p.sink_blocks[i];
            if (e >= 0 && e < p.NB) {
                p.map[e] = -2;
                if (__ldcg(p.ref + e) > 0) atomicMax(p.top_fixed, e + 1);
            }
        }
        cluster_sync();
    }
    auto is_fixed = [&](int64_t i) { return p.n_sinks > 0 && __ldcg(p.map + i) == -2; };

    // ---- blocks in use, and places, of each warp's ids ----
    int live = 0, places = 0;
#pragma unroll 4
    for (int64_t i0 = ids.lo; i0 < ids.hi; i0 += 32) {
        const int64_t i = i0 + lane;
        const bool place = i < ids.hi && !is_fixed(i);
        live += __popc(__ballot_sync(kFull, place && __ldcg(p.ref + i) > 0));
        places += __popc(__ballot_sync(kFull, place));
    }
    if (lane == 0) {
        p.counts[wa] = live;
        p.counts[kAllWarps + wa] = places;
    }
    cluster_sync();
    int n_live, unused;
    before_warp(count_of(p.counts), wa, s_scan, &n_live);
    const int places_before = before_warp(count_of(p.counts + kAllWarps), wa, s_scan, &unused);

    // ---- free places in front, blocks in use behind ----
    // f(i, in use, in front) for each id of the warp's range that is not fixed
    auto each = [&](auto f) {
        int place = places_before;
        for (int64_t i0 = ids.lo; i0 < ids.hi; i0 += 32) {
            const int64_t i = i0 + lane;
            const bool inside = i < ids.hi;
            const bool fixed = inside && is_fixed(i);
            const uint32_t m = __ballot_sync(kFull, inside && !fixed);
            const bool front = place + __popc(m & ((1u << lane) - 1)) < n_live;
            f(i, inside && !fixed, inside && __ldcg(p.ref + i) > 0, front, inside && fixed);
            place += __popc(m);
        }
    };
    int holes = 0, movers = 0;
    each([&](int64_t, bool place, bool in_use, bool front, bool) {
        holes += __popc(__ballot_sync(kFull, place && front && !in_use));
        movers += __popc(__ballot_sync(kFull, place && !front && in_use));
    });
    if (lane == 0) {
        p.counts[2 * kAllWarps + wa] = holes;
        p.counts[3 * kAllWarps + wa] = movers;
    }
    cluster_sync();
    int n_moves;
    int hole = before_warp(count_of(p.counts + 2 * kAllWarps), wa, s_scan, &unused);
    int mover = before_warp(count_of(p.counts + 3 * kAllWarps), wa, s_scan, &n_moves);
    int top = 0;  // one past the last place in front
    each([&](int64_t i, bool place, bool in_use, bool front, bool fixed) {
        const uint32_t mh = __ballot_sync(kFull, place && front && !in_use);
        const uint32_t mm = __ballot_sync(kFull, place && !front && in_use);
        const uint32_t before = (1u << lane) - 1;
        if (place && front && !in_use) p.dst[hole + __popc(mh & before)] = int32_t(i);
        if (place && !front && in_use) p.src[mover + __popc(mm & before)] = int32_t(i);
        if (place && front) top = int(i) + 1;
        if (place && !(!front && in_use)) p.map[i] = in_use ? int32_t(i) : -1;
        if (fixed) p.map[i] = in_use ? int32_t(i) : -1;
        hole += __popc(mh);
        mover += __popc(mm);
    });
    top = __reduce_max_sync(kFull, top);
    if (lane == 0 && top > 0) atomicMax(p.top_fixed, top);
    if (tid == 0) *p.n_moves = n_moves;
    cluster_sync();
    for (int k = tid; k < n_moves; k += kCluster * kThreads) {
        const int32_t from = __ldcg(p.src + k), to = __ldcg(p.dst + k);
        p.map[from] = to;
        p.ref[to] = p.ref[from];
        p.ref[from] = 0;
    }
    if (tid == 0) *p.used = __ldcg(p.top_fixed);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

size_t page_bytes(const sk_paged_layer& L, bool v) {
    const size_t rows = size_t(L.n_kv_heads) * L.block_size;
    if (L.k_dtype == SK_I4) return v ? 0 : rows * SK_KV4_ROW_BYTES(L.head_dim);
    return rows * L.head_dim * (L.k_dtype == SK_F32 ? 4 : 2);
}

// Layers of one table: every layer's check, and the fields they must share.
sk_status check_pages(const sk_paged_layer* layers, int32_t n_layers, const int32_t* ref) {
    SK_RET_IF(layers == nullptr || ref == nullptr || n_layers < 1 || n_layers > kMaxLayers, SK_ERR_ARG);
    const sk_paged_layer& A = layers[0];
    for (int i = 0; i < n_layers; ++i) {
        const sk_paged_layer& L = layers[i];
        SK_RET_IF(paged_layer_check(L) != SK_OK, SK_ERR_ARG);
        SK_RET_IF(L.block_table != A.block_table || L.batch != A.batch || L.max_blocks != A.max_blocks ||
                      L.block_size != A.block_size || L.n_blocks != A.n_blocks || L.sinks != A.sinks ||
                      L.window != A.window || L.n_sink_blocks != A.n_sink_blocks ||
                      L.sink_block_ids != A.sink_block_ids,
                  SK_ERR_ARG);
        SK_RET_IF(page_bytes(L, false) > (size_t(1) << 30), SK_ERR_UNSUPPORTED);
    }
    SK_RET_IF(A.batch > kMaxBatch, SK_ERR_UNSUPPORTED);
    SK_RET_IF(A.n_blocks > 0x7fffffff - 32, SK_ERR_UNSUPPORTED);  // block ids are int32
    return SK_OK;
}

// Workspace in int32: [0, 4 kAllWarps) counts, 4 scalars, 4 B per-request words, 2 NB ids.
constexpr int64_t kWsScalars = 4 * kAllWarps, kWsRequests = kWsScalars + 4;
int64_t ws_ids(const sk_paged_layer& L) { return kWsRequests + 4 * int64_t(L.batch); }
size_t pages_ws(const sk_paged_layer& L) { return size_t(ws_ids(L) + 2 * L.n_blocks) * 4; }

sk_status check_ws(const sk_paged_layer& L, const void* ws, size_t bytes) {
    SK_RET_IF(ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 15u) || bytes < pages_ws(L), SK_ERR_ARG);
    return SK_OK;
}

void move_pools(const sk_paged_layer* layers, int n_layers, MoveParams* m) {
    for (int i = 0; i < n_layers; ++i)
        for (int v = 0; v < 2; ++v)
            if (const size_t bytes = page_bytes(layers[i], v != 0)) {
                m->pool[m->n_pools] = v ? layers[i].v_pool : layers[i].k_pool;
                m->bytes[m->n_pools++] = int32_t(bytes);
                m->pieces = std::max(m->pieces, int((bytes + kPiece - 1) / kPiece));
            }
}

// Where all requests together could copy at most this many bytes, the reserving cluster makes the
// copies itself, at the rate of its 8 SMs.  Most calls of a serving loop copy nothing, and a second
// launch costs those 0.5-1 us on the device and 1-1.5 us of the host's time at any size.  When
// every request copies, the cluster takes (against two launches, on the device) 7.6 us (8.2) for
// 20 KB, 8.7 (8.4) for 80 KB, 10.9 (9.9) for 320 KB, 13.7 (10.3) for 2 MB and 17.3 (9.3) for 4 MB.
constexpr int64_t kCopyHere = 2 << 20;

// One block per piece of the most that can move, at most 8 per SM.
unsigned move_grid(const MoveParams& m, int64_t pages) {
    const int64_t pieces = pages * m.pieces * m.n_pools;
    return unsigned(std::max<int64_t>(1, std::min<int64_t>((pieces + kMoveThreads / 32 - 1) / (kMoveThreads / 32),
                                                           int64_t(device_sm_count()) * 8)));
}

}  // namespace
}  // namespace sk

using namespace sk;

extern "C" size_t sk_paged_pages_workspace_bytes(const sk_paged_layer* layer) {
    if (layer == nullptr || paged_layer_check(*layer) != SK_OK || layer->batch > kMaxBatch ||
        layer->n_blocks > 0x7fffffff - 32)
        return 0;
    return pages_ws(*layer);
}

extern "C" sk_status sk_paged_reserve(const sk_paged_layer* layers, int32_t n_layers, int32_t* ref,
                                      const int32_t* n_new, int32_t* granted, void* workspace, size_t ws_bytes,
                                      void* stream) {
    const sk_status s = check_pages(layers, n_layers, ref);
    if (s != SK_OK) return s;
    const sk_paged_layer& L = layers[0];
    SK_RET_IF(granted == nullptr, SK_ERR_ARG);
    SK_RET_IF(check_ws(L, workspace, ws_bytes) != SK_OK, SK_ERR_ARG);
    int32_t* ws = static_cast<int32_t*>(workspace);
    ReserveParams p{};
    p.table = const_cast<int32_t*>(L.block_table);
    p.ref = ref;
    p.lens = L.seq_lens;
    p.n_new = n_new;
    p.granted = granted;
    p.err = L.err;
    p.NB = L.n_blocks;
    p.B = L.batch;
    p.MB = L.max_blocks;
    p.bs_log2 = __builtin_ctz(unsigned(L.block_size));
    p.S = L.sinks;
    p.W = L.window;
    p.sink_len = L.n_sink_blocks * L.block_size;
    p.counts = ws;
    p.n_copies = ws + kWsScalars + 2;
    p.need = ws + kWsRequests;
    p.shared_of = p.need + L.batch;
    p.copies = p.shared_of + L.batch;
    p.free_ids = ws + ws_ids(L);
    p.old_ids = p.free_ids + L.n_blocks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    MoveParams m{};
    move_pools(layers, n_layers, &m);
    m.src = p.copies;
    m.dst = p.copies + 1;
    m.stride = 2;
    m.n = p.n_copies;
    int64_t most = 0;  // bytes, if every request copies a block
    for (int i = 0; i < m.n_pools; ++i) most += int64_t(L.batch) * m.bytes[i];
    MoveParams here{};
    if (most <= kCopyHere) here = m;
    SK_CUDA_RET(launch_pdl(reserve_kernel, dim3(kCluster), dim3(kThreads), 0, st, p, here));
    if (most <= kCopyHere) return SK_OK;
    SK_CUDA_RET(launch_pdl(move_pages_kernel, dim3(move_grid(m, L.batch)), dim3(kMoveThreads), 0, st, m));
    return SK_OK;
}

extern "C" sk_status sk_paged_fork(const sk_paged_layer* layers, int32_t n_layers, int32_t* ref,
                                   const int32_t* parents, void* stream) {
    const sk_status s = check_pages(layers, n_layers, ref);
    if (s != SK_OK) return s;
    SK_RET_IF(parents == nullptr, SK_ERR_ARG);
    const sk_paged_layer& L = layers[0];
    ForkParams p{};
    p.table = const_cast<int32_t*>(L.block_table);
    p.ref = ref;
    p.parents = parents;
    p.err = L.err;
    p.NB = L.n_blocks;
    p.B = L.batch;
    p.MB = L.max_blocks;
    p.table_blocks = (L.max_blocks + kForkCols - 1) / kForkCols;
    for (int i = 0; i < n_layers; ++i) {  // lengths that layers share move once
        bool seen = false;
        for (int j = 0; j < p.n_lens; ++j) seen = seen || p.lens[j] == layers[i].seq_lens;
        if (!seen) p.lens[p.n_lens++] = layers[i].seq_lens;
    }
    const size_t smem = size_t(L.batch) * kForkCols * 4;
    SK_CUDA_RET(launch_pdl(fork_kernel, dim3(unsigned(p.table_blocks + p.n_lens)), dim3(kForkThreads), smem,
                           static_cast<cudaStream_t>(stream), p));
    return SK_OK;
}

extern "C" sk_status sk_paged_compact(const sk_paged_layer* layers, int32_t n_layers, int32_t* ref,
                                      int32_t* block_map, int32_t* used, void* workspace, size_t ws_bytes,
                                      void* stream) {
    const sk_status s = check_pages(layers, n_layers, ref);
    if (s != SK_OK) return s;
    const sk_paged_layer& L = layers[0];
    SK_RET_IF(block_map == nullptr || used == nullptr, SK_ERR_ARG);
    SK_RET_IF(check_ws(L, workspace, ws_bytes) != SK_OK, SK_ERR_ARG);
    int32_t* ws = static_cast<int32_t*>(workspace);
    CompactParams p{};
    p.ref = ref;
    p.map = block_map;
    p.used = used;
    p.sink_blocks = L.sink_block_ids;
    p.n_sinks = L.n_sink_blocks;
    p.NB = L.n_blocks;
    p.counts = ws;
    p.n_moves = ws + kWsScalars;
    p.top_fixed = ws + kWsScalars + 1;
    p.src = ws + ws_ids(L);
    p.dst = p.src + L.n_blocks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    SK_CUDA_RET(launch_pdl(compact_kernel, dim3(kCluster), dim3(kThreads), 0, st, p));
    MoveParams m{};
    move_pools(layers, n_layers, &m);
    m.src = p.src;
    m.dst = p.dst;
    m.stride = 1;
    m.n = p.n_moves;
    m.map = block_map;
    m.table = const_cast<int32_t*>(L.block_table);
    m.entries = int64_t(L.batch) * L.max_blocks;
    m.NB = L.n_blocks;
    SK_CUDA_RET(launch_pdl(move_pages_kernel, dim3(move_grid(m, L.n_blocks)), dim3(kMoveThreads), 0, st, m));
    return SK_OK;
}
