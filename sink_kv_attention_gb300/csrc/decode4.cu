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
// fp16's range (bf16 q: exact; fp32 q: in two fp16 parts, 22 bits).  The per-group scale
// and minimum are applied in fp32 to the products of K; for V the scale goes into the
// probabilities, and the minimum is summed in fp32.
//
// P' = p s_grp is rounded to fp16 (11 bits; fp32 io: two parts).  Its range is kept by
// the reference of the online softmax: weights are 2^(score - mref) with
// mref = (running max of the head) + (exponent of the largest V scale seen) - kHead, so
// that P' <= 2^(kHead + kSlack + 1) < 65504.  The running max is only moved when a score
// passes it by kSlack (a factor 2^8 of room), which in practice is once per unit: the
// vote costs less than a reduction per tile.  Row sums are of the unrounded fp32 weights.
//
// Work split: as decode_kernels.cuh (the visible rows of all units end to end, an equal
// share per block, partials combined by its combine kernels).  In a block each warp takes
// 32-row tiles in turn and owns a ring of SLOTS tiles in shared memory that it fills with
// bulk copies itself (one copy per tile, or per page): no producer, and no barrier
// between warps until a unit ends and its warps' states are merged.
//
// Rows are visited in an order that spreads a quarter warp's 16-byte loads over all
// banks: matrix row r of a 16-row tile is key kappa(r), chosen so that (0,1), (2,3), ..
// are 16 words apart mod 32 (K fragments) and so are (0,2,4,6) and (1,3,5,7) 8 apart (V).
#include "decode4.cuh"

#include <type_traits>

#include <cuda_fp16.h>

#include "decode_kernels.cuh"
#include "kv4.cuh"

namespace sk {
namespace {

constexpr int kTileRows = 32;
constexpr float kRefNone = -1e30f;  // reference of a head that has seen no key
constexpr int kHead = 6;            // log2 of the weight at the reference, V scale 1
constexpr float kSlack = 8.0f;      // a score may pass the reference by this much
constexpr int kExpFloor = -60;      // V scales below 2^-60 are taken as 2^-60 in the reference
constexpr uint32_t kLowNibbles = 0x000F000Fu, kHighNibbles = 0x00F000F0u;

template <int D, int NREP> struct Cfg4 {
    static constexpr int NG = D / 32;                      // groups
    static constexpr int ROWB = kv4_row_bytes(D);
    static constexpr int NWARPS = NREP == 8 ? 8 : 12;
    static constexpr int SLOTS = NREP == 8 ? 4 : 3;
    static constexpr int SLOT_BYTES = kTileRows * ROWB;
    static constexpr int MERGE_FLOATS = NREP * (D + 2);    // per warp
    static constexpr size_t OFF_ZERO = size_t(NWARPS) * SLOTS * SLOT_BYTES;  // a row of zeros
    static constexpr size_t OFF_MERGE = OFF_ZERO + (ROWB + 15) / 16 * 16;
    static constexpr size_t OFF_PRE = OFF_MERGE + size_t(NWARPS) * MERGE_FLOATS * 4;
    static constexpr size_t OFF_BAR = OFF_PRE + (kMaxBatch + 1) * 8;
    static constexpr size_t SMEM = OFF_BAR + NWARPS * SLOTS * 8;
    static constexpr int THREADS = NWARPS * 32;
    static constexpr int PARTIAL_FLOATS = NREP * (D + 2);
    static_assert(OFF_PRE % 8 == 0 && SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ int kappa(int r) { return (0x57463120 >> (4 * r)) & 7; }

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// The tiles of a block's share that fall to one warp, in order: tile i of the share
// (counted over all its units) goes to warp i % NWARPS.
template <int NWARPS>
struct TileWalk {
    UnitWalk w;
    int64_t lo, hi, cap;   // the share; rows a unit may hold
    int64_t r0, r1;        // the unit's rows in the share
    int gt0, nt, k;        // share index of the unit's first tile, its tiles, this warp's next one
    __device__ __forceinline__ void unit(int warp) {
        const int64_t st = w.start();
        r0 = max(lo, st) - st;
        r1 = min(min(hi, st + w.len()) - st, cap);
        nt = r1 > r0 ? int((r1 - r0 + kTileRows - 1) / kTileRows) : 0;
        k = (warp + NWARPS - gt0 % NWARPS) % NWARPS;
    }
    __device__ __forceinline__ void begin(const int64_t* pre, int B, int Hkv, int64_t lo_, int64_t hi_, int64_t cap_,
                                          int warp) {
        w = UnitWalk{pre, B, Hkv, 0, 0};
        w.seek(lo_);
        lo = lo_;
        hi = hi_;
        cap = cap_;
        gt0 = 0;
        unit(warp);
    }
    // the next unit of the share; false: there is none
    __device__ __forceinline__ bool next_unit(int warp) {
        if (!w.next() || w.start() >= hi) return false;
        gt0 += nt;
        unit(warp);
        return true;
    }
    // moves to a unit that still has a tile for this warp; false: the share is done
    __device__ __forceinline__ bool settle(int warp) {
        while (k >= nt)
            if (!next_unit(warp)) return false;
        return true;
    }
    __device__ __forceinline__ int64_t row() const { return r0 + int64_t(k) * kTileRows; }
    __device__ __forceinline__ int rows() const { return int(min(int64_t(kTileRows), r1 - row())); }
};

// Fills `slot` with the walk's tile (the whole warp).  Contiguous: one copy.  Paged: lane
// i finds the pool row of the tile's row i; the first row of each run of consecutive pool
// rows copies the run.
template <typename C, bool PAGED, typename Walk>
__device__ __forceinline__ void load_tile(const DecodeParams& p, const Walk& t, uint8_t* slot, uint64_t* bar,
                                          uint64_t policy, int lane, bool* bad) {
    const int n = t.rows();
    const int b = t.w.b, g = t.w.g;
    const uint8_t* rows = static_cast<const uint8_t*>(p.kc);
    if constexpr (!PAGED) {
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, uint32_t(n) * C::ROWB);
            bulk_copy_g2s(slot, rows + ((int64_t(b) * p.Hkv + g) * p.cap + t.row()) * C::ROWB,
                          uint32_t(n) * C::ROWB, bar, policy);
        }
    } else {
        const int64_t n_req = p.pos[b];
        const int64_t Lk = n_req > 0 ? n_req + p.sink_len : 0;
        const bool split = p.W > 0 && Lk > int64_t(p.S) + p.W;  // sinks, then the last W keys
        const int64_t row = t.row() + lane;
        const int64_t key = split && row >= p.S ? Lk - p.W + (row - p.S) : row;
        const bool active = lane < n;
        int64_t blk = 0;
        if (active) {
            if (key < p.sink_len) {
                blk = p.sink_blocks[key >> p.bs_log2];
            } else {
                const int64_t j = (key - p.sink_len) >> p.bs_log2;
                blk = j < p.max_blocks ? p.block_table[int64_t(b) * p.max_blocks + j] : -1;
            }
            if (blk < 0 || blk >= p.pool_blocks) {
                *bad = true;
                blk = 0;  // stay inside the pool; the error word reports it
            }
        }
        const int64_t in = key & (p.bs - 1);
        const bool first = active && (lane == 0 || in == 0 || (split && row == p.S));
        const uint32_t firsts = __ballot_sync(kFull, first);
        if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(n) * C::ROWB);
        __syncwarp();
        if (first) {
            const uint32_t later = lane == 31 ? 0u : firsts >> (lane + 1);
            const int len = later != 0 ? __ffs(int(later)) : n - lane;
            bulk_copy_g2s(slot + lane * C::ROWB, rows + ((blk * p.Hkv + g) * p.bs + in) * C::ROWB,
                          uint32_t(len) * C::ROWB, bar, policy);
        }
    }
}

// The online softmax state of one warp over a unit, for the lane's heads 2t, 2t + 1.
template <int NG> struct State4 {
    float o[NG][2][4];    // group, dim pair i of the lane's 4 dims (4 g + 2 i + {0, 1}): (dim, head) products
    float2 om[NG];        // sum of weight * m
    float2 l;             // sum of weights (this lane's rows)
    float2 ref;           // reference score of each head (the same in all lanes of a t)
    int vexp;             // exponent of the V scale in the reference (the same in all lanes)
};

template <typename T, int D, int NREP, bool PAGED>
__global__ void __launch_bounds__(Cfg4<D, NREP>::THREADS, 1) decode4_split_kernel(DecodeParams p) {
    using C = Cfg4<D, NREP>;
    constexpr int NG = C::NG, NWARPS = C::NWARPS, SLOTS = C::SLOTS;
    constexpr bool F32 = std::is_same<T, float>::value;
    constexpr int NQ = F32 ? 2 : 1;  // fp16 parts of q and of P'
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* zero_row = smem + C::OFF_ZERO;
    float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
    int64_t* pre = reinterpret_cast<int64_t*>(smem + C::OFF_PRE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g8 = lane >> 2, t4 = lane & 3;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * SLOTS;
    uint8_t* ring = smem + size_t(warp) * SLOTS * C::SLOT_BYTES;
    pdl_trigger();
    if (lane == 0) {
        for (int s = 0; s < SLOTS; ++s) mbar_init(&bars[s], 1);
        fence_barrier_init();
    }
    for (int i = threadIdx.x; i < C::ROWB / 4; i += C::THREADS) reinterpret_cast<uint32_t*>(zero_row)[i] = 0;
    pdl_wait();  // the append before this kernel has written the state, q and the new rows
    if (warp == 0) unit_prefix(p, pre, lane);
    __syncthreads();

    const int P = gridDim.x, c = blockIdx.x;
    const int64_t R = pre[p.B];
    const int64_t lo = (int64_t(c) * R + P - 1) / P;
    const int64_t hi = (int64_t(c + 1) * R + P - 1) / P;
    if (R == 0 || lo >= hi) return;
    const int64_t cap = PAGED ? (int64_t(1) << 62) : p.cap;
    const uint64_t policy = l2_policy_evict_first();
    bool timed_out = false, bad = false;

    TileWalk<NWARPS> ld, w;
    w.begin(pre, p.B, p.Hkv, lo, hi, cap, warp);
    ld = w;
    bool more = ld.settle(warp);
    int slot = 0;
    uint32_t phase = 0;
    for (int s = 0; s < SLOTS && more; ++s) {
        load_tile<C, PAGED>(p, ld, ring + s * C::SLOT_BYTES, &bars[s], policy, lane, &bad);
        ld.k += NWARPS;
        more = ld.settle(warp);
    }

    const uint32_t half_sel = (g8 & 1) ? 0x7632u : 0x5410u;  // which 4 codes of a word of 8 are this lane's
    do {
        const int b = w.w.b, g = w.w.g;
        const int64_t unit = int64_t(b) * p.Hkv + g;
        // ---- q as the N-side operand: head g8, dims 32 grp + 8 t4 .. + 7 ----
        uint32_t qb[NQ][NG][4];
        float fac;  // score units (log2) per accumulator unit, of head g8
        {
            float qf[NG][8];
            float amax = 0.0f;
            const T* qrow = static_cast<const T*>(p.q) + (unit * NREP + g8) * D;
#pragma unroll
            for (int r = 0; r < NG; ++r) {
                constexpr int V = ElemIO<T>::kPerVec;
#pragma unroll
                for (int i = 0; i < 8 / V; ++i) {
                    const uint4 raw = g8 < NREP ? reinterpret_cast<const uint4*>(qrow + 32 * r + 8 * t4)[i]
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
            fac = p.qscale * pow2f(24 - e);
            const float f0 = pow2f(e), f1 = pow2f(e - 4);  // even / odd nibbles
#pragma unroll
            for (int r = 0; r < NG; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = qf[r][i] * ((i & 1) ? f1 : f0), y = qf[r][i + 4] * ((i & 1) ? f1 : f0);
#pragma unroll
                    for (int h = 0; h < NQ; ++h) {
                        qb[h][r][i] = half2_bits(x, y);
                        const float2 part = half2_floats(qb[h][r][i]);
                        x -= part.x;
                        y -= part.y;
                    }
                }
        }
        const float2 fac2 = make_float2(__shfl_sync(kFull, fac, 8 * t4), __shfl_sync(kFull, fac, 8 * t4 + 4));
        // sum of q over each group, in accumulator units: the product with codes of 1
        float2 qsum[NG];
#pragma unroll
        for (int r = 0; r < NG; ++r) {
            float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < NQ; ++h)
#pragma unroll
                for (int i = 0; i < 4; i += 2)
                    mma16816(a, 0x00010001u, 0x00010001u, 0x00100010u, 0x00100010u, qb[h][r][i], qb[h][r][i + 1]);
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
        st.vexp = kExpFloor;

        for (; w.k < w.nt; w.k += NWARPS) {
            const int n = w.rows();
            const uint8_t* tile = ring + slot * C::SLOT_BYTES;
            if (!mbar_wait_bounded(&bars[slot], phase)) timed_out = true;

            // ---- scores: row m of matrix tile mt is tile row 16 mt + 8 (m / 8) + kappa(m % 8) ----
            const int kr = kappa(g8);
            float2 sc[4];         // [2 mt + row half]: the lane's two heads
            uint32_t vpar[4][NG]; // V (m, s) of the same rows
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t kw[2][NG], kp[2][NG];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 16 * mt + 8 * h + kr;
                    const uint8_t* row = r < n ? tile + r * C::ROWB : zero_row;
                    load_words<NG>(row + kv4_word_offset(D, t4, 0), kw[h]);
                    load_words<NG>(row + kv4_param_offset(D, 0), kp[h]);
                    load_words<NG>(row + kv4_half_bytes(D) + kv4_param_offset(D, 0), vpar[2 * mt + h]);
                }
                float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
                for (int r = 0; r < NG; ++r) {
                    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int h = 0; h < NQ; ++h) {
                        mma16816(a, kw[0][r] & kLowNibbles, kw[1][r] & kLowNibbles, kw[0][r] & kHighNibbles,
                                 kw[1][r] & kHighNibbles, qb[h][r][0], qb[h][r][1]);
                        const uint32_t x = kw[0][r] >> 8, y = kw[1][r] >> 8;
                        mma16816(a, x & kLowNibbles, y & kLowNibbles, x & kHighNibbles, y & kHighNibbles,
                                 qb[h][r][2], qb[h][r][3]);
                    }
                    const float ka = __uint_as_float(kp[0][r] & 0xFFFF0000u), ma = __uint_as_float(kp[0][r] << 16);
                    const float kb = __uint_as_float(kp[1][r] & 0xFFFF0000u), mb = __uint_as_float(kp[1][r] << 16);
                    s0 = __ffma2_rn(make_float2(ka, ka), make_float2(a[0], a[1]), s0);
                    s1 = __ffma2_rn(make_float2(kb, kb), make_float2(a[2], a[3]), s1);
                    s0 = __ffma2_rn(make_float2(ma, ma), qsum[r], s0);
                    s1 = __ffma2_rn(make_float2(mb, mb), qsum[r], s1);
                }
                sc[2 * mt] = __fmul2_rn(s0, fac2);
                sc[2 * mt + 1] = __fmul2_rn(s1, fac2);
            }
            if (n < kTileRows) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (16 * (i >> 1) + 8 * (i & 1) + kr >= n) sc[i] = make_float2(-INFINITY, -INFINITY);
            }

            // ---- reference: moved when a score or a V scale outgrows it ----
            float2 top = make_float2(fmaxf(fmaxf(sc[0].x, sc[1].x), fmaxf(sc[2].x, sc[3].x)),
                                     fmaxf(fmaxf(sc[0].y, sc[1].y), fmaxf(sc[2].y, sc[3].y)));
            uint32_t vtop = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < NG; ++r) vtop = max(vtop, vpar[i][r]);
            const bool outgrown = top.x > st.ref.x + kSlack || top.y > st.ref.y + kSlack ||
                                  int(vtop >> 23) - 127 > st.vexp;
            if (__any_sync(kFull, outgrown)) {
                const float2 old = st.ref;
                const int old_exp = st.vexp;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    top.x = fmaxf(top.x, __shfl_xor_sync(kFull, top.x, o));
                    top.y = fmaxf(top.y, __shfl_xor_sync(kFull, top.y, o));
                }
                // a non-finite scale spoils its own group and is kept out of the reference
                vtop = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < NG; ++r) vtop = max(vtop, vpar[i][r] < 0x7F800000u ? vpar[i][r] : 0u);
                vtop = __reduce_max_sync(kFull, vtop);
                st.ref.x = fmaxf(st.ref.x, top.x);
                st.ref.y = fmaxf(st.ref.y, top.y);
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
            const float shift = float(kHead - st.vexp);
            const float2 off = make_float2(shift - st.ref.x, shift - st.ref.y);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                float2 pr[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 x = __fadd2_rn(sc[2 * mt + h], off);
                    pr[h] = make_float2(fast_exp2_approx(x.x), fast_exp2_approx(x.y));
                    st.l = __fadd2_rn(st.l, pr[h]);
                }
                // this lane's keys as the K side of the second product: 2t, 2t + 1 and + 8
                uint32_t vw[4][NG];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 16 * mt + 8 * (i >> 1) + kappa(2 * t4 + (i & 1));
                    const uint8_t* row = r < n ? tile + r * C::ROWB : zero_row;
                    load_words<NG>(row + kv4_half_bytes(D) + kv4_word_offset(D, g8 >> 1, 0), vw[i]);
                }
#pragma unroll
                for (int r = 0; r < NG; ++r) {
                    uint32_t pb[NQ][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float s = __uint_as_float(vpar[2 * mt + h][r] & 0xFFFF0000u);
                        const float m = __uint_as_float(vpar[2 * mt + h][r] << 16);
                        float2 ps = __fmul2_rn(pr[h], make_float2(s, s));
                        st.om[r] = __ffma2_rn(pr[h], make_float2(m, m), st.om[r]);
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            const uint32_t hp = half2_bits(ps.x, ps.y);
                            pb[q][h] = transpose8x8(hp);
                            const float2 part = half2_floats(hp);
                            ps = make_float2(ps.x - part.x, ps.y - part.y);
                        }
                    }
                    const uint32_t x = __byte_perm(vw[0][r], vw[1][r], half_sel);
                    const uint32_t y = __byte_perm(vw[2][r], vw[3][r], half_sel);
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        mma16816(st.o[r][0], x & kLowNibbles, x & kHighNibbles, y & kLowNibbles, y & kHighNibbles,
                                 pb[q][0], pb[q][1]);
                        mma16816(st.o[r][1], (x >> 8) & kLowNibbles, (x >> 8) & kHighNibbles, (y >> 8) & kLowNibbles,
                                 (y >> 8) & kHighNibbles, pb[q][0], pb[q][1]);
                    }
                }
            }
            __syncwarp();  // the slot has been read
            if (more) {
                load_tile<C, PAGED>(p, ld, ring + slot * C::SLOT_BYTES, &bars[slot], policy, lane, &bad);
                ld.k += NWARPS;
                more = ld.settle(warp);
            }
            if (++slot == SLOTS) { slot = 0; phase ^= 1; }
        }

        // ---- merge the warps' states and write this block's partial of the unit ----
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
        float* mw = merge + warp * C::MERGE_FLOATS;
        const float mshift = float(st.vexp - kHead);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = 2 * t4 + e;
            if (h < NREP) {
                if (g8 == 0) {
                    const float ref = e ? st.ref.y : st.ref.x;
                    mw[h] = ref == kRefNone ? -INFINITY : ref + mshift;
                    mw[NREP + h] = e ? st.l.y : st.l.x;
                }
#pragma unroll
                for (int r = 0; r < NG; ++r) {
                    const float m = e ? st.om[r].y : st.om[r].x;
                    float4 v;
                    v.x = fmaf(st.o[r][0][e], 16777216.0f, m);        // 2^24: even nibbles
                    v.y = fmaf(st.o[r][0][2 + e], 1048576.0f, m);     // 2^20: odd nibbles
                    v.z = fmaf(st.o[r][1][e], 16777216.0f, m);
                    v.w = fmaf(st.o[r][1][2 + e], 1048576.0f, m);
                    float* d = mw + 2 * NREP + h * D + 32 * r + 4 * g8;
                    reinterpret_cast<float2*>(d)[0] = make_float2(v.x, v.y);
                    reinterpret_cast<float2*>(d)[1] = make_float2(v.z, v.w);
                }
            }
        }
        __syncthreads();
        float* outp = p.ws + (unit + c) * C::PARTIAL_FLOATS;
        for (int idx = threadIdx.x; idx < NREP * D; idx += C::THREADS) {
            const int h = idx / D;
            float M = -INFINITY;
#pragma unroll
            for (int ww = 0; ww < NWARPS; ++ww) M = fmaxf(M, merge[ww * C::MERGE_FLOATS + h]);
            const float Mu = M == -INFINITY ? 0.0f : M;
            float a = 0.0f, lsum = 0.0f;
#pragma unroll
            for (int ww = 0; ww < NWARPS; ++ww) {
                const float* mm = merge + ww * C::MERGE_FLOATS;
                const float f = fast_exp2_approx(mm[h] - Mu);
                a = fmaf(f, mm[2 * NREP + idx], a);
                lsum = fmaf(f, mm[NREP + h], lsum);
            }
            outp[2 * NREP + idx] = a;
            if (idx % D == 0) {
                outp[h] = M;
                outp[NREP + h] = lsum;
            }
        }
        __syncthreads();
    } while (w.next_unit(warp));
    if (timed_out) set_error(p.err, SK_DEVERR_TIMEOUT);
    if (bad) set_error(p.err, SK_DEVERR_BLOCK_TABLE);
}

template <typename T, int D, int NREP, bool PAGED>
cudaError_t run4(DecodeParams p, int64_t rows_most, cudaStream_t st) {
    using C = Cfg4<D, NREP>;
    static PerDevice<cudaError_t> attr;
    const cudaError_t a = set_smem_limit_once(attr, decode4_split_kernel<T, D, NREP, PAGED>, int(C::SMEM));
    if (a != cudaSuccess) return a;
    const int64_t units = int64_t(p.B) * p.Hkv;
    // no more blocks than rows the cache can hold: they would only add partials to skip
    p.n_blocks = int(std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), rows_most)));
    cudaError_t e = launch_pdl(decode4_split_kernel<T, D, NREP, PAGED>, dim3(p.n_blocks), dim3(C::THREADS), C::SMEM,
                               st, p);
    if (e != cudaSuccess) return e;
    p.combine_wpu = combine_wpu(p.n_blocks, units);
    const int64_t warps = units * NREP * p.combine_wpu;
    return p.combine_wpu == 1
               ? launch_pdl(decode_combine_kernel<T, D, NREP>, dim3(unsigned((warps + 7) / 8)), dim3(256), 0, st, p)
               : launch_pdl(decode_combine_group_kernel<T, D, NREP>, dim3(unsigned((warps + 7) / 8)), dim3(256), 0,
                            st, p);
}

template <typename T, int D>
bool dispatch4(int nrep, const DecodeParams& p, int64_t rows_most, cudaStream_t st, cudaError_t* e) {
    const bool paged = p.kind == kKindPaged;
    switch (nrep) {
#define SK_CASE(N)                                                        \
    case N:                                                               \
        *e = paged ? run4<T, D, N, true>(p, rows_most, st)                \
                   : run4<T, D, N, false>(p, rows_most, st);              \
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
    return size_t(device_sm_count() + int64_t(batch) * n_kv_heads) * nrep * (head_dim + 2) * sizeof(float);
}

bool kv4_decode_run(const Kv4DecodeArgs& a, cudaStream_t st, cudaError_t* e) {
    DecodeParams p{};
    p.q = a.q;
    p.sink_logits = a.sink_logits;
    p.out = a.out;
    p.ws = static_cast<float*>(a.ws);
    int D;
    int64_t rows_most;
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
        rows_most = int64_t(L.batch) * L.n_kv_heads * keys;
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
        rows_most = int64_t(L.batch) * L.n_kv_heads * L.capacity;
    }
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
