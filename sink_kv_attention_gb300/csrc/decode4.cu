// Split-K decode attention over 4-bit cache rows (kv4.cuh) of ring, global and paged
// layers.
//
// A visible row costs 5 d_h / 4 bytes where a bf16 cache streams 4 d_h: at 32 x 4096 rows
// of 8 kv heads the HBM floor falls to a third, and one multiply-add per value on the
// CUDA cores, as the bf16 kernel does them, would then take longer than the stream.  So
// both products run on the tensor cores, with no arithmetic on the codes:
//
//   q.k^ = sum_grp s_grp (sum_i q_i c_i) + m_grp (sum_i q_i)         (per key, group)
//   out  = sum_grp sum_key (p s_grp) c + sum_key p m_grp
//
// mma.sync m16n8k16 (fp16 in, fp32 accumulate): the M side holds the codes (16 keys of
// K, or 16 dims of V), the N side the up to 8 q heads of a kv head.  The shapes are those
// of one query per sequence: N = 8 is what a kv head has to offer, and tcgen05 would want
// 128 rows of codes written out to shared memory as fp16 first.  A 4-bit code masked in
// place is the fp16 subnormal code * 2^-24 (bits 0-3) or code * 2^-20 (bits 4-7), which
// the tensor cores take exactly: a word of 8 codes becomes 4 operand registers with 4
// ANDs and a shift, and the factors 2^24 / 2^20 are undone on q (even / odd nibbles) and
// on the finished output.  q is scaled by a power of two per head to sit at the top of
// fp16's range (bf16 q: exact; fp32 q: in two fp16 parts, 24 bits).  The per-group scale
// and minimum are applied in fp32 to the products of K; for V the scale goes into the
// probabilities, and the minimum is summed in fp32.
//
// The tensor core adds a step's products and the accumulator after cutting each, towards 0,
// to the precision of the largest as its exponents tell, which for subnormal operands is up
// to 2^10 too large: sums are good to about 2^-18 of the largest product (measured: rms
// 2^-22, 2^-26 with normal operands).  That is far below a bf16 output.  fp32 calls turn the
// codes into normal fp16 integers around 0 (code - 8, and m + 8 s for m: an OR and a
// subtraction more), make the upper parts of q and of P' multiples of one unit, so that their
// products add exactly, and add lower parts, upper parts and a tile's sums to the running
// ones in fp32 (six fp32 keys against 64 bits: 3e-6 before, 3e-7 so).
//
// P' = p s_grp is rounded to fp16 (11 bits; fp32 io: two parts).  Its range is kept by
// the reference of the online softmax: weights are 2^(score - mref) with
// mref = (running max of the head) + (exponent of the largest V scale seen) - kHead, so
// that P' < 2^(kHead + kSlack + 1) < 65504.  The running max is only moved when a score
// passes it by kSlack (bf16: a factor 2^8 of room), which in practice is once per unit: the
// vote costs less than a reduction per tile.  Row sums are of the unrounded fp32 weights.
//
// Work split: the visible rows of all units (a sequence and one or two kv heads) are laid
// end to end and each block takes an equal share.  In a block each warp takes 32-row tiles
// (16 rows of two kv heads) in turn and owns a ring of SLOTS tiles in shared memory that it
// fills with bulk copies itself (one copy per tile and kv head, or per page): no producer,
// and no barrier between warps until a unit ends and its warps' states are merged, each
// through the ring slot that its warp has just emptied.
//
// One kernel: a block that holds all of a unit writes its output; a unit cut between blocks
// is finished by whichever of them finds every partial written when it has written its own
// (softmax states in the workspace, added in the blocks' order, so the result does not depend
// on who that is, and two that find it so write the same bits).  A partial is marked by a word
// that holds a number of this launch's own, so the workspace needs no initialisation; who
// finishes a unit takes its marks back (a graph replays its launch with the same number).
// Nothing waits for another block, and there is no counter for the blocks to queue at (a
// compare-and-swap counter took 0.35 us for each block of a unit).
//
// Rows are visited in an order that spreads a quarter warp's 16-byte loads over all
// banks: matrix row r of a 16-row tile is key kappa(r), chosen so that (0,1), (2,3), ..
// are 16 words apart mod 32 (K fragments) and so are (0,2,4,6) and (1,3,5,7) 8 apart (V).
//
// The code around the tile loop runs once or twice in a launch and is fetched once, so its
// loops are not unrolled (a kernel of 126 KB became one of 77 KB: calls of 5 to 25 us 1-5%
// faster, code warm).
#include "decode4.cuh"

#include <atomic>
#include <chrono>
#include <type_traits>

#include <cuda_fp16.h>
#include <unistd.h>

#include "decode_kernels.cuh"
#include "kv4.cuh"

namespace sk {
namespace {

constexpr float kRefNone = -1e30f;  // reference of a head that has seen no key
// log2 of the weight at the reference, V scale 1, and how far a score may pass the reference.
// fp32 calls leave no slack: their weights' upper parts are multiples of a fixed unit.
template <bool F32> constexpr int kHead = F32 ? 13 : 6;
template <bool F32> constexpr float kSlack = F32 ? 0.0f : 8.0f;
constexpr int kExpFloor = -60;      // V scales below 2^-60 are taken as 2^-60 in the reference
constexpr uint32_t kLowNibbles = 0x000F000Fu, kHighNibbles = 0x00F000F0u;

// A unit of a block that other blocks share.
struct Cut4 {
    int64_t unit, first;  // the unit and the workspace slot of its first partial
    int n, own;           // its partials, and which of them is this block's
};

// KVH kv heads share a block's unit: their q heads are columns 4 kv .. 4 kv + NREP - 1 of
// the N side (KVH = 2, NREP <= 4) or 0 .. NREP - 1 (KVH = 1).
template <typename T, int D, int NREP, int KVH> struct Cfg4 {
    static constexpr int NG = D / 32;                      // groups
    static constexpr int ROWB = kv4_row_bytes(D);
    static constexpr int HEADS = NREP * KVH;               // q heads of a unit
    static constexpr int TR = 32 / KVH;                    // rows of a tile (of each kv head)
    // 12 warps where their registers allow (measured: 8 warps 4-10% slower on bf16 calls)
    static constexpr int NWARPS = (HEADS == 8 && KVH == 1) || sizeof(T) == 4 ? 8 : 12;
    static constexpr int HEAD_BYTES = TR * ROWB;           // a kv head's rows in a slot
    static constexpr int SLOT_BYTES = KVH * HEAD_BYTES;
    static constexpr int SLOTS = NWARPS == 8 ? 4 : 3;
    // a partial: the sums [HEADS][D], the references [HEADS], the sums of weights [HEADS]
    static constexpr int PARTIAL_FLOATS = (HEADS * (D + 2) + 3) / 4 * 4;
    static constexpr int Q_BYTES = HEADS * D * int(sizeof(T));   // a unit's q rows
    static constexpr size_t OFF_Q = size_t(NWARPS) * SLOTS * SLOT_BYTES;
    static constexpr size_t OFF_BAR = OFF_Q + 2 * Q_BYTES;       // slot barriers, then two of the q rows
    static constexpr size_t OFF_ROWS = OFF_BAR + (NWARPS * SLOTS + 2) * 8;   // Rows4
    static constexpr size_t OFF_M = (OFF_ROWS + (3 * kMaxBatch + 1) * 8 + 15) / 16 * 16;  // the warps' (m, l) per head
    static constexpr size_t OFF_FLAGS = OFF_M + 2 * HEADS * NWARPS * 4;      // slot of each warp's sums
    static constexpr size_t SMEM = OFF_FLAGS + NWARPS * 4 + 2 * sizeof(Cut4);
    static constexpr int THREADS = NWARPS * 32;
    static_assert(HEADS * D * 4 <= SLOT_BYTES, "a slot holds a warp's sums");
    // workspace: a mark per partial, then the partials (a slot for each unit and block)
    __host__ __device__ static constexpr int64_t marks_floats(int64_t slots) { return (slots + 1) / 2 * 4; }
    static_assert(KVH == 1 || (KVH == 2 && NREP <= 4), "columns");
    static_assert(OFF_Q % 16 == 0 && OFF_BAR % 16 == 0 && OFF_M % 16 == 0 && NWARPS % 4 == 0, "alignment");
    static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ int kappa(int r) { return (0x57463120 >> (4 * r)) & 7; }

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a zero C.
__device__ __forceinline__ void mma16816_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// An 8 x 8 matrix of 16-bit values, one row per 4 lanes, transposed within the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 half2_floats(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ uint32_t half2_times(uint32_t w, __half2 f) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&w), f);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A masked word as the M side takes it: as it stands (subnormals), or as fp16 integers
// code - 8 (HIGH: 16 (code - 8)).
template <bool F32, bool HIGH> __device__ __forceinline__ uint32_t codes_of(uint32_t masked) {
    if constexpr (!F32) return masked;
    const uint32_t w = masked | 0x64006400u;  // 1024 + code (or + 16 code)
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(HIGH ? 1152.0f : 1032.0f));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// (s, m) of a parameter word, m the value of the code that counts as 0.
template <bool F32> __device__ __forceinline__ float2 scale_and_zero(uint32_t par) {
    const float s = __uint_as_float(par & 0xFFFF0000u), m = __uint_as_float(par << 16);
    return make_float2(s, F32 ? fmaf(8.0f, s, m) : m);
}

// x to the nearest multiple of 2^e (|x| < 2^(e + 22)).
template <int e> __device__ __forceinline__ float to_multiple(float x) {
    constexpr float magic = 12582912.0f * float(1 << e);  // 1.5 * 2^23 units
    return __fadd_rn(__fadd_rn(x, magic), -magic);
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }  // normal range

template <int NG> __device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
    if constexpr (NG == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x; w[1] = u.y;
    }
}

__device__ __forceinline__ int64_t div_rows(int64_t a, int64_t b) {  // a, b >= 0
    return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// The rows of the batch in shared memory.  The split counts `extra` rows more for each unit,
// in front of its own: taking up a unit and merging its warps costs a block about as much as
// those rows would, and a share of short units would otherwise take several times as long as
// one of long ones (ragged 16-token pages: measured 51.7 us without).
struct Rows4 {
    int64_t* start;  // [B + 1] counted rows before sequence b: Hu units of len + extra each
    int64_t* len;    // [B] visible rows of a unit of sequence b
    int64_t* shift;  // [B] paged: rows behind the sinks hold key row + shift (0: every row its key)
    int extra;
};

// The units of a share of counted rows, in order, as far as they have rows of their own in
// it.  A share has fewer than 2^31 rows (its rows are bytes of HBM), so offsets into it are 32
// bits.
struct Units4 {
    int b, g;     // sequence, unit of the sequence
    int rows;     // the unit's rows in the share
    int rest;     // counted rows of the share behind them
    int64_t r0;   // the unit's first row in the share
    __device__ __forceinline__ void take(const Rows4& rw, int64_t from) {  // from: counted rows of it before the share
        const int64_t counted = rw.len[b] + rw.extra;
        const int64_t to = min(counted, from + rest);
        rest -= int(to - from);
        r0 = max(int64_t(0), from - rw.extra);
        rows = int(max(int64_t(0), to - rw.extra - r0));
    }
    // the next unit of the share; false: there is none
    __device__ __forceinline__ bool next(const Rows4& rw, int Hu) {
        if (rest == 0) return false;
        if (++g == Hu) {
            g = 0;
            do { ++b; } while (rw.len[b] == 0);  // rows are left, so a sequence with rows is
        }
        take(rw, 0);
        return rows > 0;
    }
    __device__ __forceinline__ void begin(const Rows4& rw, int B, int Hu, int64_t lo, int64_t hi) {
        int l = 0, h = B;  // largest b with start[b] <= lo < start[b + 1]
        while (h - l > 1) {
            const int m = (l + h) >> 1;
            if (rw.start[m] <= lo) l = m; else h = m;
        }
        b = l;
        const int64_t counted = rw.len[b] + rw.extra, off = lo - rw.start[b];
        g = int(div_rows(off, counted));
        rest = int(hi - lo);
        take(rw, off - g * counted);
        if (rows == 0) next(rw, Hu);  // the share has a row: it is longer than `extra`
    }
};

// The tiles of a block's share that fall to one warp, in order: tile i of the share
// (counted over all its units) goes to warp i % NWARPS.  Tiles of a paged unit end where the
// key is a multiple of TR, so that they lie in as few pages as possible; the first may be
// shorter.
template <int NWARPS, int TR, bool PAGED>
struct TileWalk {
    Units4 u;
    int warp0;             // the warp that takes the unit's first tile
    int at, left;          // this warp's tile: its first row - r0 (negative for a short first tile: the
                           // tile starts at 0), and the part's end - at
    __device__ __forceinline__ int lead(const Rows4& rows) const {  // rows that the first tile lacks
        return PAGED ? int(u.r0 + rows.shift[u.b]) & (TR - 1) : 0;
    }
    __device__ __forceinline__ void unit(const Rows4& rows, int warp) {
        at = (warp >= warp0 ? warp - warp0 : warp + NWARPS - warp0) * TR - lead(rows);
        left = u.rows - at;
    }
    __device__ __forceinline__ void begin(const Rows4& rows, int B, int Hu, int64_t lo, int64_t hi, int warp) {
        u.begin(rows, B, Hu, lo, hi);
        warp0 = 0;
        unit(rows, warp);
    }
    __device__ __forceinline__ void step() {
        at += NWARPS * TR;
        left -= NWARPS * TR;
    }
    __device__ __forceinline__ bool next_unit(const Rows4& rows, int Hu, int warp) {
        const int tiles = (u.rows + lead(rows) + TR - 1) / TR;
        if (!u.next(rows, Hu)) return false;
        warp0 = (warp0 + tiles) % NWARPS;
        unit(rows, warp);
        return true;
    }
    __device__ __forceinline__ int first() const { return PAGED ? max(at, 0) : at; }
    __device__ __forceinline__ int count() const { return PAGED ? min(left, TR) + min(at, 0) : min(left, TR); }
};

// The loading side of a warp's walk: the current tile's source.
template <typename C, int KVH, bool PAGED>
struct Loader {
    TileWalk<C::NWARPS, C::TR, PAGED> t;
    const uint8_t* src;   // contiguous: the tile's rows of the unit's first kv head
    // paged, of row lane % TR of the tile: its key, and the pool block that the table names,
    // looked up when the tile before is loaded (its latency is then hidden)
    int64_t key;
    int32_t block;
    bool more;
    __device__ __forceinline__ void source(const DecodeParams& p) {
        if constexpr (!PAGED)
            src = static_cast<const uint8_t*>(p.kc) +
                  ((int64_t(t.u.b) * p.Hkv + t.u.g) * KVH * p.cap + t.u.r0 + t.at) * C::ROWB;
    }
    // moves on to a unit with a tile for this warp
    __device__ __forceinline__ void settle(const DecodeParams& p, const Rows4& rows, int warp, int lane) {
        bool moved = false;
        while (t.left <= 0) {
            if (!t.next_unit(rows, p.Hkv, warp)) {
                more = false;
                return;
            }
            moved = true;
        }
        if (moved) source(p);
        if constexpr (PAGED) {
            const int i = lane % C::TR;
            const int64_t row = t.u.r0 + t.first() + i;
            key = row < p.S ? row : row + rows.shift[t.u.b];
            block = -1;
            if (i < t.count()) {
                if (key < p.sink_len) {
                    block = p.sink_blocks[key >> p.bs_log2];
                } else {
                    const int64_t j = (key - p.sink_len) >> p.bs_log2;
                    if (j < p.max_blocks) block = p.block_table[int64_t(t.u.b) * p.max_blocks + j];
                }
            }
        }
    }
    __device__ __forceinline__ void begin(const DecodeParams& p, const Rows4& rows, int warp, int lane) {
        more = true;
        source(p);
        settle(p, rows, warp, lane);
    }
    __device__ __forceinline__ void step(const DecodeParams& p, const Rows4& rows, int warp, int lane) {
        t.step();
        if constexpr (!PAGED) src += C::NWARPS * C::HEAD_BYTES;
        settle(p, rows, warp, lane);
    }
    // Fills `slot` with the tile (the whole warp): the rows of each kv head of the unit, one
    // after the other.  Contiguous: one copy per kv head.  Paged: lane kv TR + i has row i of
    // kv head kv; the first row of each run of consecutive pool rows copies the run (both kv
    // heads at once where the tile is a whole page).
    __device__ __forceinline__ void load(const DecodeParams& p, uint8_t* slot, uint64_t* bar, uint64_t policy,
                                         int lane, bool* bad) const {
        const int n = t.count();
        if constexpr (!PAGED) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, uint32_t(KVH * n) * C::ROWB);
#pragma unroll
                for (int kv = 0; kv < KVH; ++kv)
                    bulk_copy_g2s(slot + kv * C::HEAD_BYTES, src + kv * p.cap * C::ROWB, uint32_t(n) * C::ROWB, bar,
                                  policy);
            }
        } else {
            const int i = lane % C::TR, kv = lane / C::TR;
            const bool active = i < n;
            int64_t blk = block;
            if (active && (blk < 0 || blk >= p.pool_blocks)) {
                *bad = true;
                blk = 0;  // stay inside the pool; the error word reports it
            }
            const int in = int(key) & (p.bs - 1);
            const bool jump = t.u.r0 + t.first() + i == p.S;  // the window's first row
            const bool whole = KVH > 1 && p.bs == C::TR && n == C::TR &&
                               __all_sync(kFull, in == i && !(jump && i > 0));
            const bool first = active && (i == 0 || in == 0 || jump);
            const uint32_t firsts = __ballot_sync(kFull, first);
            if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(KVH * n) * C::ROWB);
            __syncwarp();
            if (first && !(whole && kv > 0)) {
                // rows up to the next run of this kv head, or to the tile's end
                const uint32_t later = (lane == 31 ? 0u : firsts >> (lane + 1)) & ((1u << (C::TR - 1 - i)) - 1u);
                const int len = whole ? KVH * C::TR : (later != 0 ? __ffs(int(later)) : n - i);
                const int64_t head = blk * (p.Hkv * KVH) + t.u.g * KVH + kv;
                bulk_copy_g2s(slot + kv * C::HEAD_BYTES + i * C::ROWB,
                              static_cast<const uint8_t*>(p.kc) + (head * p.bs + in) * C::ROWB,
                              uint32_t(len) * C::ROWB, bar, policy);
            }
        }
    }
};

// The online softmax state of one warp over a unit, for the lane's columns 2t, 2t + 1.
template <int NG> struct State4 {
    float o[NG][2][4];    // group, dim pair i of the lane's 4 dims (4 g + 2 i + {0, 1}): (dim, head) products
    float2 om[NG];        // sum of weight * m
    float2 l;             // sum of weights (this lane's rows)
    float2 ref;           // reference score of each head (the same in all lanes of a t)
    float2 limit;         // raw score that outgrows it
    int vexp;             // exponent of the V scale in the reference (the same in all lanes)
};

// Output of 4 dims of a unit's head h: weighted sums a and the sum of weights l at reference
// M (both in 2^(score - M)), and the learned sink, one more logit of the denominator.
template <typename T, int D, int HEADS>
__device__ __forceinline__ void finish(const DecodeParams& p, int64_t unit, int h, int dim, float M, float l,
                                       const float4& a) {
    const int Hq = p.Hkv * HEADS;
    float f = 1.0f;
    if (p.sink_logits != nullptr) {
        const float z = fminf(fmaxf(p.sink_logits[int(unit % p.Hkv) * HEADS + h], kSinkLogitMin), kSinkLogitMax) *
                        kLog2e;
        const float top = fmaxf(M, z);
        f = fast_exp2_approx(M - top);
        l = l * f + fast_exp2_approx(z - top);
    }
    const float inv = l > 0.0f ? f / l : (l == l ? 0.0f : l);  // NaN stays
    T* o = static_cast<T*>(p.out) + (unit / p.Hkv * Hq + unit % p.Hkv * HEADS + h) * D + dim;
    const float v[4] = {a.x * inv, a.y * inv, a.z * inv, a.w * inv};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, float>::value) o[i] = v[i];
        else o[i] = __float2bfloat16_rn(v[i]);
    }
}

// The output of a unit from its n partials, `first` on, added in their order (the block).
// w: room for 2 (n + 1) HEADS floats of shared memory.
template <typename T, int D, int HEADS, int PF, int THREADS>
__device__ __noinline__ void combine_unit(const DecodeParams& p, int64_t unit, const float* first, int n,
                                             float* w) {
    constexpr int U = 16;  // partials in flight; the first are asked for before the weights are known
    constexpr int VALS = HEADS * D / 4;
    static_assert(VALS <= THREADS, "a thread per 4 values");
    const int idx = min(int(threadIdx.x), VALS - 1), h = idx / (D / 4);
    const float* part = first + idx * 4;
    float4 v[U];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u < n) v[u] = __ldcg(reinterpret_cast<const float4*>(part + int64_t(i0 + u) * PF));
    };
    fetch(0);
    float* ls = w + n * HEADS;        // [n][HEADS] sums of weights
    float* top = ls + n * HEADS;      // [HEADS] reference, then the sum of weights
    const int lane = threadIdx.x & 31;
    // a warp per head, a lane per partial (a thread per head took 0.3 us longer at 4 partials)
    for (int k = threadIdx.x >> 5; k < HEADS; k += THREADS / 32) {
        float M = -INFINITY, l = 0.0f;
#pragma unroll 2
        for (int i = lane; i < n; i += 32) {
            const float* ml = first + int64_t(i) * PF + HEADS * D + k;
            const float m = __ldcg(ml);
            w[i * HEADS + k] = m;
            ls[i * HEADS + k] = __ldcg(ml + HEADS);
            M = fmaxf(M, m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
#pragma unroll 1
        for (int i = lane; i < n; i += 32) {
            const float f = fast_exp2_approx(w[i * HEADS + k] - M);
            w[i * HEADS + k] = f;
            l = fmaf(ls[i * HEADS + k], f, l);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
        if (lane == 0) {
            top[k] = M;
            top[HEADS + k] = l;
        }
    }
    __syncthreads();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = 0;;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= n) break;
            const float f = w[(i0 + u) * HEADS + h];
            a.x = fmaf(v[u].x, f, a.x);
            a.y = fmaf(v[u].y, f, a.y);
            a.z = fmaf(v[u].z, f, a.z);
            a.w = fmaf(v[u].w, f, a.w);
        }
        i0 += U;
        if (i0 >= n) break;
        fetch(i0);
    }
    if (threadIdx.x < VALS) finish<T, D, HEADS>(p, unit, h, idx % (D / 4) * 4, top[h], top[HEADS + h], a);
    __syncthreads();
}

// Marks a unit's partial `own` as written (the warp; its block's threads have all passed a
// fence and a barrier since they wrote it) and tells whether all n are.  Of the blocks that
// mark theirs, the last in the order of the fences sees all.
__device__ __forceinline__ bool mark_partial(uint64_t* marks, int own, int n, uint64_t tag, int lane) {
    volatile uint64_t* m = marks;
    if (lane == 0) m[own] = tag;
    __syncwarp();
    __threadfence();
    bool all = true;
#pragma unroll 1
    for (int i = lane; i < n; i += 32) all = all && m[i] == tag;
    return __all_sync(kFull, all);
}

template <typename T, int D, int NREP, int KVH, bool PAGED>
__global__ void __launch_bounds__(Cfg4<T, D, NREP, KVH>::THREADS, 1) decode4_kernel(DecodeParams p, uint64_t tag) {
    using C = Cfg4<T, D, NREP, KVH>;
    constexpr int NG = C::NG, NWARPS = C::NWARPS, SLOTS = C::SLOTS, TR = C::TR, HEADS = C::HEADS;
    constexpr bool F32 = std::is_same<T, float>::value;
    static_assert(!F32 || KVH == 1, "fp32 calls: registers for one kv head's q");
    constexpr int NQ = F32 ? 2 : 1;          // fp16 parts of q and of P'
    constexpr int NM = KVH == 1 ? 2 : 1;     // 16-row matrix tiles of scores
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g8 = lane >> 2, t4 = lane & 3;
    uint64_t* all_bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* bars = all_bars + warp * SLOTS;
    uint64_t* q_bars = all_bars + NWARPS * SLOTS;
    uint8_t* ring = smem + size_t(warp) * SLOTS * C::SLOT_BYTES;
    Rows4 rows{reinterpret_cast<int64_t*>(smem + C::OFF_ROWS),
                     reinterpret_cast<int64_t*>(smem + C::OFF_ROWS) + kMaxBatch + 1,
                     reinterpret_cast<int64_t*>(smem + C::OFF_ROWS) + 2 * kMaxBatch + 1, 0};
    float* warp_m = reinterpret_cast<float*>(smem + C::OFF_M);  // [HEADS][NWARPS] references
    float* warp_l = warp_m + HEADS * NWARPS;                    // [HEADS][NWARPS] sums, at the block's reference
    int* warp_slot = reinterpret_cast<int*>(smem + C::OFF_FLAGS);  // [NWARPS] where a warp's sums are; -1: none
    Cut4* cuts = reinterpret_cast<Cut4*>(warp_slot + NWARPS);      // [2]
    pdl_trigger();
    if (lane == 0) {
        for (int s = 0; s < SLOTS; ++s) mbar_init(&bars[s], 1);
        if (warp == 0) {
            mbar_init(&q_bars[0], 1);
            mbar_init(&q_bars[1], 1);
        }
        fence_barrier_init();
    }
    // The split of the batch is worked out twice at most: from the state as it reads before
    // the wait, while the kernel ahead (an append, another layer) still runs, and again after
    // it where a length has changed by then (a full ring's does not).
    const uint64_t policy = l2_policy_evict_first();
    const int64_t units = int64_t(p.B) * p.Hkv;
    const int c = blockIdx.x;
    bool timed_out = false, bad = false;
    int64_t R = 0;
    int P = 0;
    TileWalk<NWARPS, TR, PAGED> w;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        if (pass == 1) pdl_wait();  // the append has written the state, q and the new rows
        bool changed = false;
#pragma unroll 1
        for (int b = threadIdx.x; b < p.B; b += C::THREADS) {
            int64_t n, shift = 0;
            if constexpr (PAGED) {
                const int64_t most = int64_t(p.max_blocks) << p.bs_log2;
                int64_t L = p.pos[b];
                if (L > most) {  // more tokens than its table names blocks for
                    if (pass == 1) bad = true;
                    L = most;
                }
                if (L > 0) L += p.sink_len;
                n = max(int64_t(0), L);
                if (p.W > 0 && n > int64_t(p.S) + p.W) {
                    n = int64_t(p.S) + p.W;
                    shift = L - n;
                }
            } else {
                n = max(int64_t(0), min(visible_rows(p, b), p.cap));
            }
            if (pass == 0 || rows.len[b] != n || (PAGED && rows.shift[b] != shift)) {
                rows.len[b] = n;
                if (PAGED) rows.shift[b] = shift;
                changed = true;
            }
        }
        if (!__syncthreads_or(changed)) break;
        if (warp == 0) {  // rows before each sequence, uncounted extras left out for now
            int64_t carry = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int b = b0 + lane;
                int64_t x = b < p.B ? p.Hkv * rows.len[b] : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(kFull, x, o);
                    if (lane >= o) x += y;
                }
                if (b < p.B) rows.start[b + 1] = carry + x;
                carry += __shfl_sync(kFull, x, 31);
            }
            if (lane == 0) rows.start[0] = 0;
        }
        __syncthreads();
        // Blocks that take part: enough for one tile a warp, or one unit each if that is more.
        R = rows.start[p.B];
        P = int(min(int64_t(gridDim.x), max(min(units, R), R / (NWARPS * TR))));
        // Units of one length: the same number of blocks for each, so that no block has parts of
        // two, unless that leaves more than a quarter (one block each) or an eighth of the GPU's
        // blocks idle.  Measured: 128 units of 4096 rows over 152 SMs 41.4 -> 36.7 us (the stream
        // alone the same), 4 of 4096 17.1 -> 12.8, 16 of 4096 17.1 -> 14.3.
        bool even = false;
        if (R > 0 && units <= gridDim.x && R == units * rows.len[0]) {
            const int n = int(units), grid = int(gridDim.x);
            const int up = (P + n - 1) / n * n, down = P / n * n;
            if (n * 4 >= grid * 3) P = n;
            else if (up <= grid) P = up;
            else if ((grid - down) * 8 <= grid) P = down;
            even = P % n == 0;
        }
        // at most half a share, so that every share has rows of its own
        rows.extra = P > 0 && !even ? int(min(int64_t(2 * NWARPS * TR), div_rows(R, P) / 2)) : 0;
        __syncthreads();  // every thread has R
        if (warp == 0) {
            int before = 0;  // sequences with rows
#pragma unroll 1
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int b = b0 + lane;
                const uint32_t m = __ballot_sync(kFull, b < p.B && rows.len[b] > 0);
                if (b < p.B)
                    rows.start[b + 1] += int64_t(p.Hkv) * rows.extra *
                                         (before + __popc(m & (0xffffffffu >> (31 - lane))));
                before += __popc(m);
            }
        }
        __syncthreads();
        R = rows.start[p.B];  // counted rows from here on
        if (c < P)
            w.begin(rows, p.B, p.Hkv, div_rows(int64_t(c) * R + P - 1, P), div_rows(int64_t(c + 1) * R + P - 1, P),
                    warp);
    }

    // sequences with nothing visible: zeros, each from one block
#pragma unroll 1
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
        if (rows.len[b] == 0)
#pragma unroll 1
            for (int i = threadIdx.x; i < p.Hkv * HEADS * D; i += C::THREADS)
                static_cast<T*>(p.out)[int64_t(b) * p.Hkv * HEADS * D + i] = T(0.0f);
    if (c >= P) return;  // R = 0 too
    // q rows of the share's units, two units ahead, into two slots (one thread)
    Units4 qu = w.u;
    bool q_more = true;
    auto load_q = [&](int qs) {
        mbar_arrive_expect_tx(&q_bars[qs], C::Q_BYTES);
        bulk_copy_g2s_nohint(smem + C::OFF_Q + qs * C::Q_BYTES,
                             static_cast<const T*>(p.q) + (int64_t(qu.b) * p.Hkv + qu.g) * (HEADS * D), C::Q_BYTES,
                             &q_bars[qs]);
        q_more = qu.next(rows, p.Hkv);
    };
    if (threadIdx.x == 0) {
        load_q(0);
        if (q_more) load_q(1);
    }
    int q_at = 0;
    uint32_t q_phase = 0;
    uint64_t* marks = reinterpret_cast<uint64_t*>(p.ws);
    float* partials = p.ws + C::marks_floats(units + gridDim.x);
    int n_cuts = 0;
    Loader<C, KVH, PAGED> ld;
    ld.t = w;
    ld.begin(p, rows, warp, lane);
    int slot = 0;
    uint32_t phase = 0;
    for (int s = 0; s < SLOTS && ld.more; ++s) {
        ld.load(p, ring + s * C::SLOT_BYTES, &bars[s], policy, lane, &bad);
        ld.step(p, rows, warp, lane);
    }

    auto low = [](uint32_t w) { return codes_of<F32, false>(w & kLowNibbles); };
    auto high = [](uint32_t w) { return codes_of<F32, true>(w & kHighNibbles); };
    const uint32_t half_sel = (g8 & 1) ? 0x7632u : 0x5410u;  // which 4 codes of a word of 8 are this lane's
    const int my_kv = KVH == 1 ? 0 : t4 >> 1;                // kv head of the lane's columns
    // this lane's places in a slot: K words of row kappa(g8), parameters of that row (of the
    // columns' kv head), V words of rows kappa(2 t4) and kappa(2 t4 + 1)
    const int k_at = kappa(g8) * C::ROWB + kv4_word_offset(D, t4, 0);
    const int par_at = kappa(g8) * C::ROWB + my_kv * C::HEAD_BYTES + kv4_param_offset(D, 0);
    const int v_at0 = kappa(2 * t4) * C::ROWB + kv4_half_bytes(D) + kv4_word_offset(D, g8 >> 1, 0);
    const int v_at1 = kappa(2 * t4 + 1) * C::ROWB + kv4_half_bytes(D) + kv4_word_offset(D, g8 >> 1, 0);
    // the N side column g8 belongs to kv head g8 / 4 (KVH = 2): a product with one kv head's
    // codes takes zeros in the other's columns (P' is multiplied by 1 or 0)
    const __half2 keep[2] = {__float2half2_rn(KVH == 1 || g8 < 4 ? 1.0f : 0.0f),
                             __float2half2_rn(g8 < 4 ? 0.0f : 1.0f)};
    do {
        const int64_t unit = int64_t(w.u.b) * p.Hkv + w.u.g;
        // ---- q as the N-side operand: column g8, dims 32 grp + 8 t4 .. + 7 ----
        uint32_t qb[KVH][NQ][NG][4];
        float fac;  // score units (log2) per accumulator unit, of column g8
        {
            const int qh = KVH == 1 ? g8 : (g8 >> 2) * NREP + (g8 & 3);
            const bool real = KVH == 1 ? g8 < NREP : (g8 & 3) < NREP;
            float qf[NG][8];
            float amax = 0.0f;
            const T* qrow = reinterpret_cast<const T*>(smem + C::OFF_Q + q_at * C::Q_BYTES) + qh * D;
            if (!mbar_wait_bounded(&q_bars[q_at], q_phase)) timed_out = true;
#pragma unroll
            for (int r = 0; r < NG; ++r) {
                constexpr int V = ElemIO<T>::kPerVec;
#pragma unroll
                for (int i = 0; i < 8 / V; ++i) {
                    const uint4 raw = real ? reinterpret_cast<const uint4*>(qrow + 32 * r + 8 * t4)[i]
                                           : make_uint4(0, 0, 0, 0);
                    ElemIO<T>::unpack(raw, qf[r] + V * i);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(qf[r][i]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
            // 2^e puts the largest |q| into [2^14, 2^15)
            const int e = amax > 0.0f ? max(-102, min(14 - (int(__float_as_uint(amax) >> 23) - 127), 100)) : 0;
            fac = p.qscale * pow2f((F32 ? 0 : 24) - e);
            const float f0 = pow2f(e), f1 = pow2f(e - 4);  // even / odd nibbles
#pragma unroll
            for (int r = 0; r < NG; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = qf[r][i] * ((i & 1) ? f1 : f0), y = qf[r][i + 4] * ((i & 1) ? f1 : f0);
#pragma unroll
                    for (int h = 0; h < NQ; ++h) {
                        // fp32, the upper part: a multiple of 2^4 (even; 2^0 odd) below 2^15 (2^11)
                        const bool upper = F32 && h == 0;
                        const uint32_t bits =
                            !upper ? half2_bits(x, y)
                                   : ((i & 1) ? half2_bits(to_multiple<0>(x), to_multiple<0>(y))
                                              : half2_bits(to_multiple<4>(x), to_multiple<4>(y)));
                        const float2 part = half2_floats(bits);
                        x -= part.x;
                        y -= part.y;
#pragma unroll
                        for (int kv = 0; kv < KVH; ++kv) qb[kv][h][r][i] = KVH == 1 || (g8 >> 2) == kv ? bits : 0u;
                    }
                }
        }
        const float2 fac2 = make_float2(__shfl_sync(kFull, fac, 8 * t4), __shfl_sync(kFull, fac, 8 * t4 + 4));
        // sum of q over each group, in accumulator units: the product with codes of 1
        float2 qsum[NG];
#pragma unroll
        for (int r = 0; r < NG; ++r) {
            const uint32_t one = F32 ? 0x3C003C00u : 0x00010001u, sixteen = F32 ? 0x4C004C00u : 0x00100010u;
            float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kv = 0; kv < KVH; ++kv)
#pragma unroll
                for (int h = NQ - 1; h >= 0; --h) {
                    float part[4];
                    mma16816_first(part, one, one, sixteen, sixteen, qb[kv][h][r][0], qb[kv][h][r][1]);
                    mma16816(part, one, one, sixteen, sixteen, qb[kv][h][r][2], qb[kv][h][r][3]);
                    a[0] += part[0];
                    a[1] += part[1];
                }
            qsum[r] = make_float2(a[0], a[1]);
        }

        State4<NG> st;
#pragma unroll
        for (int r = 0; r < NG; ++r) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.o[r][i][e] = 0.0f;
            st.om[r] = make_float2(0.f, 0.f);
        }
        st.l = make_float2(0.f, 0.f);
        st.ref = make_float2(kRefNone, kRefNone);
        st.limit = make_float2(-INFINITY, -INFINITY);
        st.vexp = kExpFloor;

        int last = -1;  // the slot of the warp's last tile of the unit
        for (; w.left > 0; w.step()) {
            const int n = w.count();
            uint8_t* tile = ring + slot * C::SLOT_BYTES;
            if (!mbar_wait_bounded(&bars[slot], phase)) timed_out = true;
            if (n < TR) {  // rows past the tile's last one: zeros (whatever the slot held)
#pragma unroll
                for (int kv = 0; kv < KVH; ++kv)
#pragma unroll 1
                    for (int i = n * C::ROWB + lane * 16; i < C::HEAD_BYTES; i += 512)
                        *reinterpret_cast<uint4*>(tile + kv * C::HEAD_BYTES + i) = make_uint4(0, 0, 0, 0);
                __syncwarp();
            }

            // ---- scores: row m of matrix tile j is tile row 16 j + 8 (m / 8) + kappa(m % 8) ----
            float2 sc[2 * NM];         // [2 j + row half]: the lane's two columns, accumulator units
            uint32_t vpar[2 * NM][NG]; // V (m, s) of the same rows
#pragma unroll
            for (int j = 0; j < NM; ++j) {
                const uint8_t* base = tile + 16 * j * C::ROWB;
                float a[NG][4];
#pragma unroll
                for (int kv = 0; kv < KVH; ++kv) {
                    uint32_t kw[2][NG];
                    load_words<NG>(base + kv * C::HEAD_BYTES + k_at, kw[0]);
                    load_words<NG>(base + kv * C::HEAD_BYTES + k_at + 8 * C::ROWB, kw[1]);
#pragma unroll
                    for (int r = 0; r < NG; ++r) {
                        const uint32_t x = kw[0][r] >> 8, y = kw[1][r] >> 8;
                        const uint32_t k0[4] = {low(kw[0][r]), low(kw[1][r]), high(kw[0][r]), high(kw[1][r])};
                        const uint32_t k1[4] = {low(x), low(y), high(x), high(y)};
                        if (kv == 0)
                            mma16816_first(a[r], k0[0], k0[1], k0[2], k0[3], qb[kv][0][r][0], qb[kv][0][r][1]);
                        else
                            mma16816(a[r], k0[0], k0[1], k0[2], k0[3], qb[kv][0][r][0], qb[kv][0][r][1]);
                        mma16816(a[r], k1[0], k1[1], k1[2], k1[3], qb[kv][0][r][2], qb[kv][0][r][3]);
                        if constexpr (F32) {
                            float lower[4];
                            mma16816_first(lower, k0[0], k0[1], k0[2], k0[3], qb[kv][1][r][0], qb[kv][1][r][1]);
                            mma16816(lower, k1[0], k1[1], k1[2], k1[3], qb[kv][1][r][2], qb[kv][1][r][3]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) a[r][e] += lower[e];
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t* row = base + par_at + 8 * h * C::ROWB;
                    uint32_t kp[NG];
                    load_words<NG>(row, kp);
                    load_words<NG>(row + kv4_half_bytes(D), vpar[2 * j + h]);
                    float2 s0 = make_float2(0.f, 0.f);
#pragma unroll
                    for (int r = 0; r < NG; ++r) {
                        const float2 sm = scale_and_zero<F32>(kp[r]);
                        s0 = __ffma2_rn(make_float2(sm.x, sm.x), make_float2(a[r][2 * h], a[r][2 * h + 1]), s0);
                        s0 = __ffma2_rn(make_float2(sm.y, sm.y), qsum[r], s0);
                    }
                    sc[2 * j + h] = s0;
                }
            }
            if (n < TR) {
#pragma unroll
                for (int i = 0; i < 2 * NM; ++i)
                    if (8 * i + kappa(g8) >= n) sc[i] = make_float2(-INFINITY, -INFINITY);
            }

            // ---- reference: moved when a score or a V scale outgrows it ----
            float2 top = sc[0];
            uint32_t vtop = 0;
#pragma unroll
            for (int i = 0; i < 2 * NM; ++i) {
                top = make_float2(fmaxf(top.x, sc[i].x), fmaxf(top.y, sc[i].y));
#pragma unroll
                for (int r = 0; r < NG; ++r) vtop = max(vtop, vpar[i][r]);
            }
            const bool outgrown = top.x > st.limit.x || top.y > st.limit.y || int(vtop >> 23) - 127 > st.vexp;
            if (__any_sync(kFull, outgrown)) {
                const float2 old = st.ref;
                const int old_exp = st.vexp;
                top = __fmul2_rn(top, fac2);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    top.x = fmaxf(top.x, __shfl_xor_sync(kFull, top.x, o));
                    top.y = fmaxf(top.y, __shfl_xor_sync(kFull, top.y, o));
                }
                // a non-finite scale spoils its own group and is kept out of the reference
                vtop = 0;
#pragma unroll
                for (int i = 0; i < 2 * NM; ++i)
#pragma unroll
                    for (int r = 0; r < NG; ++r) vtop = max(vtop, vpar[i][r] < 0x7F800000u ? vpar[i][r] : 0u);
                vtop = __reduce_max_sync(kFull, vtop);
                st.ref.x = fmaxf(st.ref.x, top.x);
                st.ref.y = fmaxf(st.ref.y, top.y);
                st.limit = make_float2((st.ref.x + kSlack<F32>) / fac2.x, (st.ref.y + kSlack<F32>) / fac2.y);
                st.vexp = max(st.vexp, int(vtop >> 23) - 127);
                const float de = float(old_exp - st.vexp);
                const float2 al = make_float2(fast_exp2_approx(old.x - st.ref.x + de),
                                              fast_exp2_approx(old.y - st.ref.y + de));
                st.l = __fmul2_rn(st.l, al);
#pragma unroll
                for (int r = 0; r < NG; ++r) {
                    st.om[r] = __fmul2_rn(st.om[r], al);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        st.o[r][i][0] *= al.x;
                        st.o[r][i][1] *= al.y;
                        st.o[r][i][2] *= al.x;
                        st.o[r][i][3] *= al.y;
                    }
                }
            }

            // ---- weights, and their products with V ----
            // fp32 calls take the power of two after the exponential: the argument is then near
            // 0 for the largest weights, and its rounding with it
            const float shift = F32 ? 0.0f : float(kHead<F32> - st.vexp);
            const float2 off = make_float2(shift - st.ref.x, shift - st.ref.y);
            const float after = pow2f(min(kHead<F32> - st.vexp, 127));
#pragma unroll
            for (int j = 0; j < NM; ++j) {
                float2 pr[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 x = __ffma2_rn(sc[2 * j + h], fac2, off);
                    pr[h] = make_float2(fast_exp2_approx(x.x), fast_exp2_approx(x.y));
                    if constexpr (F32) pr[h] = __fmul2_rn(pr[h], make_float2(after, after));
                    st.l = __fadd2_rn(st.l, pr[h]);
                }
                // this lane's keys as the K side of the second product: 2t, 2t + 1 and + 8
                uint32_t vw[KVH][4][NG];
#pragma unroll
                for (int kv = 0; kv < KVH; ++kv) {
                    const uint8_t* base = tile + kv * C::HEAD_BYTES + 16 * j * C::ROWB;
                    load_words<NG>(base + v_at0, vw[kv][0]);
                    load_words<NG>(base + v_at1, vw[kv][1]);
                    load_words<NG>(base + v_at0 + 8 * C::ROWB, vw[kv][2]);
                    load_words<NG>(base + v_at1 + 8 * C::ROWB, vw[kv][3]);
                }
#pragma unroll
                for (int r = 0; r < NG; ++r) {
                    uint32_t pb[NQ][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 sm = scale_and_zero<F32>(vpar[2 * j + h][r]);
                        float2 ps = __fmul2_rn(pr[h], make_float2(sm.x, sm.x));
                        st.om[r] = __ffma2_rn(pr[h], make_float2(sm.y, sm.y), st.om[r]);
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            // fp32, the upper part: a multiple of 2^3 below 2^14
                            const uint32_t hp = F32 && q == 0 ? half2_bits(to_multiple<3>(ps.x), to_multiple<3>(ps.y))
                                                              : half2_bits(ps.x, ps.y);
                            pb[q][h] = transpose8x8(hp);
                            const float2 part = half2_floats(hp);
                            ps = make_float2(ps.x - part.x, ps.y - part.y);
                        }
                    }
#pragma unroll
                    for (int kv = 0; kv < KVH; ++kv) {
                        const uint32_t x = __byte_perm(vw[kv][0][r], vw[kv][1][r], half_sel);
                        const uint32_t y = __byte_perm(vw[kv][2][r], vw[kv][3][r], half_sel);
                        const uint32_t xs = x >> 8, ys = y >> 8;
                        const uint32_t v0[4] = {low(x), high(x), low(y), high(y)};
                        const uint32_t v1[4] = {low(xs), high(xs), low(ys), high(ys)};
                        if constexpr (F32) {
                            float o[2][2][4];  // upper and lower part of P'
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                mma16816_first(o[q][0], v0[0], v0[1], v0[2], v0[3], pb[q][0], pb[q][1]);
                                mma16816_first(o[q][1], v1[0], v1[1], v1[2], v1[3], pb[q][0], pb[q][1]);
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) st.o[r][i][e] += o[0][i][e] + o[1][i][e];
                        } else {
                            const uint32_t b0 = KVH == 1 ? pb[0][0] : half2_times(pb[0][0], keep[kv]);
                            const uint32_t b1 = KVH == 1 ? pb[0][1] : half2_times(pb[0][1], keep[kv]);
                            mma16816(st.o[r][0], v0[0], v0[1], v0[2], v0[3], b0, b1);
                            mma16816(st.o[r][1], v1[0], v1[1], v1[2], v1[3], b0, b1);
                        }
                    }
                }
            }
            // the slot has been read; zeros written to it come before the next copy.  The slot
            // of the warp's last tile of the unit is refilled after the merge, which uses it.
            if (n < TR) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (ld.more && w.left > NWARPS * TR) {
                ld.load(p, tile, &bars[slot], policy, lane, &bad);
                ld.step(p, rows, warp, lane);
            }
            last = slot;
            if (++slot == SLOTS) { slot = 0; phase ^= 1; }
        }

        // ---- merge the warps' states ----
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            st.l.x += __shfl_xor_sync(kFull, st.l.x, o);
            st.l.y += __shfl_xor_sync(kFull, st.l.y, o);
#pragma unroll
            for (int r = 0; r < NG; ++r) {
                st.om[r].x += __shfl_xor_sync(kFull, st.om[r].x, o);
                st.om[r].y += __shfl_xor_sync(kFull, st.om[r].y, o);
            }
        }
        // column 2 t4 + e is head h_of(e) of the unit, if it is one
        auto h_of = [&](int e) { return KVH == 1 ? 2 * t4 + e : (t4 >> 1) * NREP + ((2 * t4 + e) & 3); };
        auto is_head = [&](int e) { return KVH == 1 ? 2 * t4 + e < NREP : ((2 * t4 + e) & 3) < NREP; };
        const float mshift = float(st.vexp - kHead<F32>);
        const float m_own[2] = {last < 0 ? -INFINITY : st.ref.x + mshift, last < 0 ? -INFINITY : st.ref.y + mshift};
        if (g8 == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (is_head(e)) warp_m[h_of(e) * NWARPS + warp] = m_own[e];
        }
        if (lane == 0) warp_slot[warp] = last;
        __syncthreads();
        {
            float* sums = reinterpret_cast<float*>(ring + max(last, 0) * C::SLOT_BYTES);  // [HEADS][D]
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!is_head(e)) continue;
                const int h = h_of(e);
                const float4* ms = reinterpret_cast<const float4*>(warp_m + h * NWARPS);
                float M = -INFINITY;
#pragma unroll
                for (int i = 0; i < NWARPS / 4; ++i)
                    M = fmaxf(fmaxf(M, fmaxf(ms[i].x, ms[i].y)), fmaxf(ms[i].z, ms[i].w));
                const float f = last < 0 ? 0.0f : fast_exp2_approx(m_own[e] - M);  // M >= m_own > -inf
                const float f24 = f * (F32 ? 1.0f : 16777216.0f), f20 = f24 * 0.0625f;  // even / odd nibbles
                if (g8 == 0) warp_l[h * NWARPS + warp] = last < 0 ? 0.0f : (e ? st.l.y : st.l.x) * f;
                if (last < 0) continue;  // the slots hold tiles of the next unit
#pragma unroll
                for (int r = 0; r < NG; ++r) {
                    const float m = (e ? st.om[r].y : st.om[r].x) * f;
                    *reinterpret_cast<float4*>(sums + h * D + 32 * r + 4 * g8) =
                        make_float4(fmaf(st.o[r][0][e], f24, m), fmaf(st.o[r][0][2 + e], f20, m),
                                    fmaf(st.o[r][1][e], f24, m), fmaf(st.o[r][1][2 + e], f20, m));
                }
            }
        }
        __syncthreads();
        const bool whole = w.u.rows == rows.len[w.u.b];
        float* part = partials + (unit + c) * C::PARTIAL_FLOATS;
#pragma unroll 1
        for (int idx = threadIdx.x; idx < HEADS * D / 4; idx += C::THREADS) {
            const int h = idx / (D / 4);
            const float4* ms = reinterpret_cast<const float4*>(warp_m + h * NWARPS);
            const float4* ls = reinterpret_cast<const float4*>(warp_l + h * NWARPS);
            float M = -INFINITY, l = 0.0f;
            float4 v[NWARPS];
#pragma unroll
            for (int ww = 0; ww < NWARPS; ++ww) {
                const int at = warp_slot[ww];
                v[ww] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (at >= 0)
                    v[ww] = reinterpret_cast<const float4*>(smem + (ww * SLOTS + at) * C::SLOT_BYTES)[idx];
            }
            float4 a = v[0];
#pragma unroll
            for (int ww = 1; ww < NWARPS; ++ww)
                a = make_float4(a.x + v[ww].x, a.y + v[ww].y, a.z + v[ww].z, a.w + v[ww].w);
#pragma unroll
            for (int i = 0; i < NWARPS / 4; ++i) {
                M = fmaxf(fmaxf(M, fmaxf(ms[i].x, ms[i].y)), fmaxf(ms[i].z, ms[i].w));
                l += (ls[i].x + ls[i].y) + (ls[i].z + ls[i].w);
            }
            if (whole) {
                finish<T, D, HEADS>(p, unit, h, idx % (D / 4) * 4, M, l, a);
            } else {
                reinterpret_cast<float4*>(part)[idx] = a;
                if (idx % (D / 4) == 0) {
                    part[HEADS * D + h] = M;
                    part[HEADS * (D + 1) + h] = l;
                }
            }
        }
        if (!whole) {  // a share has two cut units at most: its first and its last
            if (threadIdx.x == 0) {
                const int64_t counted = rows.len[w.u.b] + rows.extra;
                const int64_t start = rows.start[w.u.b] + w.u.g * counted;
                const int64_t from = div_rows((start + rows.extra) * P, R);  // the unit's blocks: from, from + 1, ..
                cuts[n_cuts].unit = unit;
                cuts[n_cuts].first = unit + from;
                cuts[n_cuts].own = int(c - from);
                cuts[n_cuts].n = int(div_rows((start + counted - 1) * P, R) - from) + 1;
            }
            ++n_cuts;
        }
        // sums were written to the slots the ordinary way; bulk copies come next
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        if (last >= 0 && ld.more) {
            ld.load(p, ring + last * C::SLOT_BYTES, &bars[last], policy, lane, &bad);
            ld.step(p, rows, warp, lane);
        }
        if (threadIdx.x == 0 && q_more) load_q(q_at);
        if (++q_at == 2) { q_at = 0; q_phase ^= 1; }
    } while (w.next_unit(rows, p.Hkv, warp));

    // ---- the cut units: mark this block's partials, and finish the units that are now whole ----
    if (n_cuts > 0) {
        __threadfence();  // the partials are visible before their marks
        __syncthreads();
        if (warp < n_cuts) {
            const Cut4 cut = cuts[warp];
            const bool all = mark_partial(marks + cut.first, cut.own, cut.n, tag, lane);
            if (lane == 0) warp_slot[warp] = all;
        }
        __syncthreads();
        __threadfence();
        // the ring is empty: its first bytes hold the weights of the partials
#pragma unroll 1
        for (int i = 0; i < n_cuts; ++i) {
            const Cut4 cut = cuts[i];
            if (!warp_slot[i]) continue;
            combine_unit<T, D, HEADS, C::PARTIAL_FLOATS, C::THREADS>(
                p, cut.unit, partials + cut.first * C::PARTIAL_FLOATS, cut.n, reinterpret_cast<float*>(smem));
#pragma unroll 1
            for (int j = threadIdx.x; j < cut.n; j += C::THREADS) marks[cut.first + j] = 0;
        }
    }
    if (timed_out) set_error(p.err, SK_DEVERR_TIMEOUT);
    if (bad) set_error(p.err, SK_DEVERR_BLOCK_TABLE);
}

// A number that no other launch of this process has, never 0, from a start of its own.
uint64_t launch_tag() {
    static std::atomic<uint64_t> next{[] {
        uint64_t x = uint64_t(std::chrono::system_clock::now().time_since_epoch().count()) ^ (uint64_t(getpid()) << 40);
        x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
        return x ^ (x >> 27);
    }()};
    const uint64_t tag = next.fetch_add(1, std::memory_order_relaxed);
    return tag != 0 ? tag : next.fetch_add(1, std::memory_order_relaxed);
}

template <typename T, int D, int NREP, int KVH, bool PAGED>
cudaError_t run4(DecodeParams p, int64_t rows_most, cudaStream_t st) {
    using C = Cfg4<T, D, NREP, KVH>;
    static PerDevice<cudaError_t> attr;
    const cudaError_t a = set_smem_limit_once(attr, decode4_kernel<T, D, NREP, KVH, PAGED>, int(C::SMEM));
    if (a != cudaSuccess) return a;
    p.Hkv /= KVH;  // units of KVH kv heads
    // no more blocks than rows the cache can hold
    p.n_blocks = int(std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), rows_most / KVH)));
    return launch_pdl(decode4_kernel<T, D, NREP, KVH, PAGED>, dim3(p.n_blocks), dim3(C::THREADS), C::SMEM, st, p,
                      launch_tag());
}

template <typename T, int D>
bool dispatch4(int nrep, const DecodeParams& p, int64_t rows_most, cudaStream_t st, cudaError_t* e) {
    const bool paged = p.kind == kKindPaged;
    constexpr bool f32 = std::is_same<T, float>::value;
    // Two kv heads to a unit where they fill the 8 columns better: the work per score and per
    // weight (scales, exponentials, rounding, transposing) is then done once for both.
    const bool pair = !f32 && p.Hkv % 2 == 0;
    switch (nrep) {
#define SK_CASE(N)                                                                              \
    case N:                                                                                     \
        if (pair && N <= 4)                                                                     \
            *e = paged ? run4<T, D, N, (N <= 4 && !f32) ? 2 : 1, true>(p, rows_most, st)        \
                       : run4<T, D, N, (N <= 4 && !f32) ? 2 : 1, false>(p, rows_most, st);      \
        else                                                                                    \
            *e = paged ? run4<T, D, N, 1, true>(p, rows_most, st)                               \
                       : run4<T, D, N, 1, false>(p, rows_most, st);                             \
        return true;
        SK_CASE(1)
        SK_CASE(2)
        SK_CASE(4)
        SK_CASE(8)
#undef SK_CASE
        default:
            return false;
    }
}

}  // namespace

size_t kv4_decode_workspace(int batch, int n_kv_heads, int head_dim, int nrep) {
    if ((head_dim != 64 && head_dim != 128) || (nrep != 1 && nrep != 2 && nrep != 4 && nrep != 8)) return 0;
    // a mark and a partial for each block and unit; a unit has the q heads of one kv head (fp32
    // calls always), or of two: room for either
    size_t most = 0;
    for (int pair = 1; pair <= (nrep <= 4 && n_kv_heads % 2 == 0 ? 2 : 1); ++pair) {
        const int64_t slots = device_sm_count() + int64_t(batch) * n_kv_heads / pair;
        const int64_t heads = int64_t(nrep) * pair;
        most = std::max(most, size_t((slots + 1) / 2 * 4 + slots * ((heads * (head_dim + 2) + 3) / 4 * 4)));
    }
    return most * sizeof(float);
}

bool kv4_decode_run(const Kv4DecodeArgs& a, cudaStream_t st, cudaError_t* e) {
    DecodeParams p{};
    p.q = a.q;
    p.sink_logits = a.sink_logits;
    p.out = a.out;
    p.ws = static_cast<float*>(a.ws);
    int D;
    int64_t unit_rows;  // most rows of a unit
    if (a.paged != nullptr) {
        const sk_paged_layer& L = *a.paged;
        p.kc = L.k_pool;
        p.pos = L.seq_lens;
        p.err = L.err;
        p.B = L.batch;
        p.Hkv = L.n_kv_heads;
        p.S = L.sinks;
        p.kind = kKindPaged;
        p.block_table = L.block_table;
        p.sink_blocks = L.sink_block_ids;
        p.pool_blocks = L.n_blocks;
        p.bs = L.block_size;
        p.bs_log2 = __builtin_ctz(unsigned(L.block_size));
        p.max_blocks = L.max_blocks;
        p.sink_len = L.n_sink_blocks * L.block_size;
        p.W = L.window;
        D = L.head_dim;
        int64_t keys = int64_t(L.max_blocks) * L.block_size + p.sink_len;
        if (L.window > 0) keys = std::min<int64_t>(keys, int64_t(L.sinks) + L.window);
        unit_rows = keys;
    } else {
        const sk_kv_layer& L = *a.layer;
        p.kc = L.k;
        p.count = L.count;
        p.pos = L.pos;
        p.err = L.err;
        p.cap = L.capacity;
        p.B = L.batch;
        p.Hkv = L.n_kv_heads;
        p.S = L.sinks;
        p.kind = L.kind;
        D = L.head_dim;
        unit_rows = L.capacity;
    }
    // a block's share is counted in 32 bits
    if (double(p.B) * p.Hkv * double(unit_rows) / device_sm_count() > 1e9) return false;
    const int64_t rows_most = int64_t(p.B) * p.Hkv * unit_rows;
    p.qscale = kLog2e / sqrtf(float(D));
    if (a.io_dtype == SK_BF16) {
        if (D == 128) return dispatch4<__nv_bfloat16, 128>(a.nrep, p, rows_most, st, e);
        if (D == 64) return dispatch4<__nv_bfloat16, 64>(a.nrep, p, rows_most, st, e);
    } else if (a.io_dtype == SK_F32) {
        if (D == 128) return dispatch4<float, 128>(a.nrep, p, rows_most, st, e);
        if (D == 64) return dispatch4<float, 64>(a.nrep, p, rows_most, st, e);
    }
    return false;
}

}  // namespace sk
