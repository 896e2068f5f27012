// Attention of a grid's tokens to states of another length, and its backward
// pass. Token i and state j of an entry, head h of q and h / G of k and v
// (G = NH / NKV):
//   s_ij = q_i . k_j where doc_i = kv_doc_j >= 0, else masked,
//   out_i = sum_j p_ij v_j, p the softmax, lse_i = log sum_j e^s_ij;
// backward, dp = dout_i . v_j, delta_i = sum_j p dp, ds = p (dp - delta_i):
//   dq_i = sum_j ds k_j, dk_j = sum_i ds q_i, dv_j = sum_i p dout_i.
//
// All kernels work on tiles of 128 rows (tokens with the G heads that share a
// head of k, or states) against a stream of column tiles. Documents are taken
// one at a time: a pass over a row tile streams the column tiles that hold
// document d, masks whole columns of other documents and is written to the
// rows of d alone. So a mask is one bit a column, the same for every row, and
// what other documents' rows and columns hold stays out of it: their columns are
// zeroed in shared memory where they would meet a product as 0 times a value.
#include <atomic>
#include <climits>

#include "na3d_cross.cuh"
#include "na3d_host.cuh"
#include "sm103_ptx.cuh"

namespace na3d {

__device__ unsigned int g_cross_timeout_flag = 0;

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 500000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kSumLimit = 4294967296.0f;   // 2^32: of a row's probabilities in one tile

// About a millisecond a tick.
__device__ __forceinline__ uint32_t beat_clock() { return uint32_t(globaltimer_ns() >> 20); }
constexpr uint32_t kWaitTicks = uint32_t(kWaitLimitNs >> 20);

struct Sync {
    uint32_t bar0;
    // behind it the beat: when the producer, which tells nothing meanwhile, was last looking for a document
    volatile uint32_t* abort_flag;
    __device__ __forceinline__ uint32_t bar(int i) const { return bar0 + 8u * i; }
    __device__ __forceinline__ void still_going(int lane) const {
        if (lane == 0) abort_flag[1] = beat_clock();
    }
    // Wait for a barrier phase; false once this block has given up, kWaitLimitNs after this wait began and after
    // the last beat.
    __device__ __forceinline__ bool wait(uint32_t b, uint32_t parity) const {
        if (mbar_try_wait(b, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            if (mbar_try_wait(b, parity)) return true;
            if ((it & 1023u) == 0u) {
                if (*abort_flag) return false;
                // (a beat may be given between the two reads)
                if (globaltimer_ns() - t0 > kWaitLimitNs && int32_t(beat_clock() - abort_flag[1]) > int32_t(kWaitTicks)) {
                    *abort_flag = 1u;
                    atomicOr(&g_cross_timeout_flag, 1u);
                    return false;
                }
            }
        }
    }
    // The same with an outcome that the whole warp shares.
    __device__ __forceinline__ bool wait_warp(uint32_t b, uint32_t parity) const { return __all_sync(kAll, wait(b, parity)); }
};

__device__ __forceinline__ void drained(uint32_t bar, uint32_t parity) {
    if (!mbar_wait_bounded(bar, parity, kDrainLimitNs)) atomicOr(&g_cross_timeout_flag, 1u);
}

// One column of this thread's lane (32x32b shape).
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
    float v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(v) : "r"(taddr) : "memory");
    tmem_wait_ld();
    asm volatile("" : "+f"(v));
    return v;
}

// The values of a tensor-memory load stay behind the wait for it.
__device__ __forceinline__ void behind_wait(float* v) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                     "+f"(v[i + 6]), "+f"(v[i + 7]));
}

// A kernel lets the next one of its stream start, and waits for the one before
// it to be through (nothing to wait for where it was launched plainly).
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The products are issued by a warp that walks its loop as one, with the one
// lane that issues as a predicate of the instruction: so descriptors stay in
// uniform registers. Issued inside a branch of one lane, a product took 83
// cycles to issue, more than the 64 that it computes.
__device__ __forceinline__ uint32_t elect() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes;
}
// D (+)= A B^T, A and B in shared memory (ss) or A in tensor memory (ts).
template <uint32_t ACC>
__device__ __forceinline__ void mma_ss(uint32_t yes, uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .b64 da, db;\n\t.reg .pred p, q;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi),
        "r"(idesc), "n"(ACC), "r"(yes)
        : "memory");
}
template <uint32_t ACC>
__device__ __forceinline__ void mma_ts(uint32_t yes, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .b64 db;\n\t.reg .pred p, q;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc),
        "n"(ACC), "r"(yes)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t yes, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(yes)
        : "memory");
}

// head * HD + column, heads, tokens, entries: a box of tokens with `heads` heads.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int col, int head, int token, int entry) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(token),
        "r"(entry), "r"(bar)
        : "memory");
}

// ------------------------------------------------------------------ steps

// What the producer tells the other roles of a step: a column tile of one pass.
struct alignas(16) Step {
    uint32_t flags;
    int32_t doc;
    int32_t t0;         // the unit's first token ...
    int32_t pad;
    uint32_t mask[4];   // columns of the document
    int64_t row;        // ... its row of out
    int64_t token;      // ... and of doc
};
enum : uint32_t {
    kFirst = 1,       // of its pass
    kLast = 2,
    kUnitFirst = 4,   // of its row tiles
    kUnitLast = 8,
    kTile0 = 16,      // which row tiles the step is for
    kTile1 = 512,
    kMasked = 32,     // some columns are masked ...
    kForeign = 64,    // ... for their document
    kNone = 128,      // the rows see no column at all
    kEnd = 256,       // no more rows
    // of forward passes, where the two row tiles may be one, which takes the steps in turns
    kTileFirst = 1024,   // the first of the unit for its row tiles
    kTileLast = 2048,
    kPassLast = 4096,    // of the pass, for both row tiles (kLast: for the step's)
    kJoin = 8192         // ... which both have taken steps of
};
constexpr int kSteps = 8;   // steps that the producer may be ahead in telling

// The documents of one side: of token or state i of entry b, 0 for all where
// there are none.
struct Docs {
    const int32_t* at;
    int n;
    __device__ __forceinline__ int of(int64_t b, int i) const { return at ? __ldg(at + b * n + i) : 0; }
};

// A warp's view of the column tiles of an entry, 32 at a time, one to a lane: the
// smallest document >= 0 and the largest, and whether there is but one. Where a row
// tile has several documents, each is looked for among the same tiles: the warp
// then keeps the smallest and the largest document of 32 runs of them as well, and
// looks at those that may hold the document. So documents whose states lie
// together cost about their own tiles, documents that are scattered all of them
// each. (A look at 4096 states takes 3.7 us. 5120 tokens of 256 documents, 4 heads
// of 64 over 262144 states: sorted 118 -> 5.0 ms, in runs that come in any order
// 118 -> 60; scattered over 16384 states 39 -> 41.) N: loads to a tile, 32 documents
// each.
template <int N>
struct Tiles {
    Docs docs;
    int per;             // tokens to a tile, up to 32 N
    Sync sync;
    int64_t b = -1, run_b = -1;
    int first = -1, run_first = -1, run_tiles = 32;   // of the runs: the first tile, the tiles of each
    int lo, hi, run_lo, run_hi;
    bool pure, runs = false;
    __device__ __forceinline__ void look(int64_t entry, int tile) {
        if (entry == b && (tile & ~31) == first) return;
        b = entry;
        first = tile & ~31;
        const int lane = threadIdx.x & 31;
        sync.still_going(lane);
        lo = INT_MAX;
        hi = INT_MIN;
        pure = false;
        if (!docs.at) {
            if (int64_t(first + lane) * per < docs.n) {
                lo = hi = 0;
                pure = true;
            }
            return;
        }
        constexpr int TILES = 8 / N;   // whose loads are in flight at once
        const int32_t* at = docs.at + entry * docs.n + int64_t(first) * per + lane;
#pragma unroll 1
        for (int t0 = 0; t0 < 32; t0 += TILES, at += TILES * per) {
            const int64_t left = docs.n - int64_t(first + t0) * per;   // documents from here on
            if (left <= 0) break;
            int d[TILES][N];
            uint32_t negative = 0;   // tiles that hold negative ones
            if (per == 32 * N && left >= TILES * 32 * N) {
#pragma unroll
                for (int t = 0; t < TILES; ++t)
#pragma unroll
                    for (int j = 0; j < N; ++j) d[t][j] = __ldg(at + 32 * (t * N + j));
#pragma unroll
                for (int t = 0; t < TILES; ++t)
#pragma unroll
                    for (int j = 0; j < N; ++j) negative |= uint32_t(d[t][j] >> 31) & 1u << t;
            } else {
#pragma unroll
                for (int t = 0; t < TILES; ++t)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const int i = 32 * j + lane;
                        const bool in = i < per && t * per + i < left;
                        d[t][j] = in ? __ldg(at + t * per + 32 * j) : INT_MIN;
                        if (in && d[t][j] < 0) negative |= 1u << t;
                    }
            }
            negative = __reduce_or_sync(kAll, negative);
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                uint32_t least = uint32_t(d[t][0]);   // negative ones are above all others
                int most = d[t][0];
#pragma unroll
                for (int j = 1; j < N; ++j) {
                    least = min(least, uint32_t(d[t][j]));
                    most = max(most, d[t][j]);
                }
                least = __reduce_min_sync(kAll, least);
                most = __reduce_max_sync(kAll, most);
                if (lane == t0 + t) {
                    lo = int(min(least, uint32_t(INT_MAX)));
                    hi = most;
                    pure = !(negative >> t & 1u) && lo == hi;
                }
            }
        }
    }
    // Before the tiles from k0 to k1 are looked through, for several documents or one.
    __device__ __forceinline__ void begin(int64_t entry, int k0, int k1, bool several) {
        runs = entry == run_b && k0 == run_first;
        if (runs || !several || k1 - k0 <= 32) return;
        runs = true;
        run_b = entry;
        run_first = k0;
        run_tiles = (k1 - (k0 & ~31) + 1023) / 1024 * 32;
        run_lo = INT_MAX;
        run_hi = INT_MIN;
        for (int t = k0 & ~31; t < k1; t += 32) {
            look(entry, t);
            const int least = __reduce_min_sync(kAll, lo), most = __reduce_max_sync(kAll, hi);
            if (int(threadIdx.x & 31) == (t - (k0 & ~31)) / run_tiles) {
                run_lo = min(run_lo, least);
                run_hi = max(run_hi, most);
            }
        }
    }
    // The first tile from `tile` on, before `end`, that may hold document d; `end` where none does.
    __device__ __forceinline__ int find(int64_t entry, int tile, int end, int d, bool* whole) {
        while (tile < end) {
            if (runs) {
                const int start = run_first & ~31, run = (tile - start) / run_tiles;
                const uint32_t can = __ballot_sync(kAll, run_lo <= d && d <= run_hi) & (kAll << run);
                if (!can) return end;
                tile = max(tile, start + (__ffs(can) - 1) * run_tiles);
                if (tile >= end) return end;
            }
            look(entry, tile);
            const uint32_t can = __ballot_sync(kAll, lo <= d && d <= hi) & (kAll << (tile & 31));
            if (can) {
                const int at = __ffs(can) - 1;
                *whole = __shfl_sync(kAll, int(pure), at) != 0;
                return min(first + at, end);
            }
            tile = first + 32;
        }
        return end;
    }
};

// The smallest document > d of this warp's lanes' values (v[i] < 0: none); INT_MAX where there is none.
template <int N>
__device__ __forceinline__ int next_doc(const int (&v)[N], int d) {
    int least = INT_MAX;
    bool any = false;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (v[i] > d) {
            least = min(least, v[i]);
            any = true;
        }
    if (!__any_sync(kAll, any)) return -1;
    return __reduce_min_sync(kAll, least);
}

// Geometry that the roles share, for head size HD.
template <int HD>
struct Geom {
    static constexpr int HDB = HD < 64 ? HD : 64;      // columns of a shared-memory row
    static constexpr int NREG = HD / HDB;
    static constexpr int ROWB = HDB * 2;
    static constexpr uint32_t SWZ = HDB == 64 ? kSwizzle128B : HDB == 32 ? kSwizzle64B : kSwizzle32B;
    static constexpr int SBO = 8 * ROWB;
    static constexpr int kPer = HDB / 16;              // 16-column steps of a row
};

// D (+)= A B^T over HD columns, both operands row by row in shared memory.
template <int HD, int REG_A, int REG_B>
__device__ __forceinline__ void scores(uint32_t yes, uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
    using G = Geom<HD>;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t ao = ((kk / G::kPer) * REG_A + (kk % G::kPer) * 32) >> 4;
        const uint32_t bo = ((kk / G::kPer) * REG_B + (kk % G::kPer) * 32) >> 4;
        if (kk == 0) mma_ss<0>(yes, d, a_lo + ao, a_hi, b_lo + bo, b_hi, idesc);
        else mma_ss<1>(yes, d, a_lo + ao, a_hi, b_lo + bo, b_hi, idesc);
    }
}

// D (+)= P Y: P (bf16, 128 x N) in tensor memory, Y's N rows in shared memory, its columns outermost.
template <int HD, int N>
__device__ __forceinline__ void product(uint32_t yes, uint32_t d, uint32_t p, uint32_t y_lo, uint32_t y_hi, uint32_t idesc, bool fresh) {
    if (fresh) mma_ts<0>(yes, d, p, y_lo, y_hi, idesc);
    else mma_ts<1>(yes, d, p, y_lo, y_hi, idesc);
#pragma unroll
    for (int kk = 1; kk < N / 16; ++kk) mma_ts<1>(yes, d, p + kk * 8, y_lo + ((kk * 16 * Geom<HD>::ROWB) >> 4), y_hi, idesc);
}

// Zeros over row r of a tile of rows of HD values (regions of REG bytes).
template <int HD, int REG>
__device__ __forceinline__ void zero_row(uint32_t tile, int r) {
    using G = Geom<HD>;
#pragma unroll
    for (int c = 0; c < HD / 8; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + (c / (G::HDB / 8)) * REG + r * G::ROWB + (c % (G::HDB / 8)) * 16),
                     "r"(0) : "memory");
}

// ------------------------------------------------------------------ forward

struct FwdParams {
    int32_t L, S, NH, NKV, G, rpt;        // rpt: tokens of a row tile
    int32_t pairs, units, tiles, splits, per_split;   // pairs of row tiles of an entry; column tiles
    int32_t out_v8;
    int32_t lone;                         // the grid has one row tile: both are that one
    const int32_t *doc, *kv_doc;
    uint16_t* out;
    float* lse;
    float* part;       // splits > 1: fp32 out of each split, (split, row, HD)
    float* part_lse;   // ... and its log2-sum-exp2 (split, row)
    int64_t rows;      // B * L * NH
    int32_t B;
};

struct Unit {
    int pair, kh, split;
    int64_t b;
    __device__ __forceinline__ Unit(const FwdParams& p, int u) {
        pair = u % p.pairs;
        u /= p.pairs;
        kh = u % p.NKV;
        u /= p.NKV;
        b = u % p.B;
        split = u / p.B;
    }
};

template <int HD>
struct FwdShape : Geom<HD> {
    using G = Geom<HD>;
    static constexpr int REG = 128 * G::ROWB, TILE = G::NREG * REG;
    static constexpr int SLOTS = HD == 128 ? 5 : 8;    // of k and v in turn
    static constexpr int OFF_KV = 2 * TILE, OFF_STEP = OFF_KV + SLOTS * TILE, OFF_BAR = OFF_STEP + kSteps * 48;
    // Steps until k's (and v's) slots come round. A slot's k and v have barriers of their own: who waits for
    // the k's alone would take the phase of a v between them, still on its way, for one that is over.
    static constexpr uint32_t CYCLE = SLOTS % 2 ? SLOTS : SLOTS / 2;
    static constexpr int B_KFULL = 0, B_VFULL = SLOTS, B_EMPTY = 2 * SLOTS, B_QFULL = 3 * SLOTS, B_QEMPTY = B_QFULL + 2, B_SFULL = B_QEMPTY + 2,
                         B_PFULL = B_SFULL + 4, B_OFULL = B_PFULL + 4, B_OREAD = B_OFULL + 2, B_STAT = B_OREAD + 2, B_DONE = B_STAT + 2, B_TOLD = B_DONE + 4, B_HEARD = B_TOLD + kSteps,
                         B_DRAIN = B_HEARD + kSteps, NBAR = B_DRAIN + 3;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // tensor memory, abort flag, beat, the slots' flags
    // The columns of the last 8 steps that have some: before a step is told, k and v of the one before it
    // have their slots, and so the v of four (SLOTS 5; 8: of five) steps before it has been used.
    static constexpr int OFF_MASK = (OFF_MISC + 12 + 4 * SLOTS + 15) & ~15, MASKS = 8;
    static constexpr int OFF_STAT = OFF_MASK + 16 * MASKS;   // sum and reference of each row
    // one block on an SM, which tensor memory is shared out for
    static constexpr int NEED = OFF_STAT + 2 * 128 * 8, SMEM = NEED > 120 * 1024 ? NEED : 120 * 1024;
    static constexpr uint32_t TM_S = 0, TM_O = 256, OW = HD < 32 ? 32 : HD;   // scores of either row tile; their sums
    static_assert(SMEM <= 232448, "shared memory");
};

constexpr int kFwdThreads = 512;
enum { kPlain, kDocuments, kFew };   // kernels of calls without documents, with them, of few rows
// registers: what the softmax, the way out and the rest take of 512 x 128. The producer needs few where it
// does not search (24576 tokens over 6144 states 782 -> 748 us with more for the softmax), a hundred where it
// does: 8 tokens over 131072 states, head size 64, 42.7 us by kDocuments' split, 41 by kFew's; 49152 tokens
// over 128 states of each of 4 documents, 16 heads of 128, 119 us by kFew's split, 108 by kDocuments'.
template <int KIND>
struct FwdRegs {
    static constexpr uint32_t kSoftmax = KIND == kPlain ? 160 : KIND == kDocuments ? 144 : 152;
    static constexpr uint32_t kOut = KIND == kFew ? 104 : 112, kLow = KIND == kPlain ? 80 : KIND == kDocuments ? 112 : 104;
    static_assert(2 * kSoftmax + kOut + kLow <= 4 * 128, "register split");
};

template <int HD, int KIND>
__device__ __forceinline__ void fwd_producer(const FwdParams& p, const Sync& sy, uint32_t base, uint8_t* base_ptr, Step* steps, volatile uint32_t* said,
                                             const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv) {
    using F = FwdShape<HD>;
    const bool lone = KIND == kFew && p.lone;
    const int lane = threadIdx.x & 31;
    Tiles<4> tiles{{p.kv_doc, p.S}, 128, sy};
    const Docs rows{p.doc, p.L};
    const bool plain = KIND == kPlain || (!p.doc && !p.kv_doc);   // every column is of every row's document
    uint32_t told = 0, slot_n = 0, q_n[2] = {0, 0};

    // One operand tile into the next slot, with its step's flags.
    auto load = [&](const CUtensorMap* map, int fulls, const Unit& U, int tile, uint32_t flags) -> bool {
        const uint32_t st = slot_n % F::SLOTS;
        if (!sy.wait_warp(sy.bar(F::B_EMPTY + st), ((slot_n / F::SLOTS) & 1u) ^ 1u)) return false;
        ++slot_n;
        if (lane == 0) {
            const uint32_t full = sy.bar(fulls + st);
            said[st] = flags;
            if (flags & kEnd) {
                mbar_arrive(full);
                return true;
            }
            mbar_arrive_expect_tx(full, F::TILE);
            for (int r = 0; r < F::NREG; ++r)
                load_box(base + F::OFF_KV + st * F::TILE + r * F::REG, map, full, r * F::HDB, U.kh, tile * 128, int(U.b));
        }
        return true;
    };
    uint4* const masks = reinterpret_cast<uint4*>(base_ptr + F::OFF_MASK);
    auto tell = [&](const Step& s) -> bool {
        const uint32_t e = told % kSteps;
        if (!sy.wait_warp(sy.bar(F::B_HEARD + e), ((told / kSteps) & 1u) ^ 1u)) return false;
        ++told;
        if (lane == 0) {
            steps[e] = s;
            masks[slot_n / 2 % F::MASKS] = *reinterpret_cast<const uint4*>(s.mask);
            mbar_arrive(sy.bar(F::B_TOLD + e));
        }
        return true;
    };
    // A step is told once the one behind it is known, which says where passes and units end.
    struct Found { int tile, doc; bool whole; };
    auto run = [&]() {
        for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
            const Unit U(p, u);
            const int t0 = U.pair * 2 * p.rpt, n_tok = min(2 * p.rpt, p.L - t0);
            const bool two = n_tok > p.rpt;
            int doc[8] = {};
            if (!plain)
#pragma unroll
                for (int i = 0; i < 8; ++i) doc[i] = lane + 32 * i < n_tok ? rows.of(U.b, t0 + lane + 32 * i) : -1;
            const int k0 = U.split * p.per_split, k1 = min(k0 + p.per_split, p.tiles);
            int d = plain ? 0 : next_doc(doc, -1);
            if (!plain) tiles.begin(U.b, k0, k1, next_doc(doc, d) >= 0);
            auto next = [&](Found* f) {   // from f->tile on, of document d or those behind it
                if (plain) {
                    f->doc = 0;
                    f->whole = true;
                    return f->tile < k1;
                }
                for (; d >= 0; d = next_doc(doc, d), f->tile = k0) {
                    f->tile = tiles.find(U.b, f->tile, k1, d, &f->whole);
                    while (f->tile < k1) {
                        f->doc = d;
                        if (f->whole) return true;
                        // in range is not in it: look whether any of its columns is of the document
                        bool any = false;
                        for (int i = 0; i < 4; ++i) {
                            const int j = f->tile * 128 + 32 * i + lane;
                            any |= j < p.S && tiles.docs.of(U.b, j) == d;
                        }
                        if (__any_sync(kAll, any)) return true;
                        f->tile = tiles.find(U.b, f->tile + 1, k1, d, &f->whole);
                    }
                }
                return false;
            };
            const int64_t token0 = U.b * p.L + t0, row0 = token0 * p.NH + U.kh * p.G + (p.splits > 1 ? U.split * p.rows : 0);
            auto behind = [&](const Found& f) {
                Found g = f;
                ++g.tile;
                if (f.doc < 0 || !next(&g)) g.doc = -1;
                return g;
            };
            // this step's tile, the next one's and the one's after that; document < 0: none
            Found f{k0, -1, false};
            if (!next(&f)) {
                if (!tell({kNone | kUnitLast, -1, t0, 0, {}, row0, token0})) return false;
                continue;
            }
            Found f1 = behind(f), f2 = behind(f1);
            int was[2] = {-1, -1};   // documents of the last steps but one, and but none, of either row tile's
            for (int n = 0; f.doc >= 0; ++n) {
                const uint32_t tiles_of = !lone ? (two ? kTile0 | kTile1 : uint32_t(kTile0)) : n & 1 ? uint32_t(kTile1) : uint32_t(kTile0);
                const int before = lone ? was[0] : was[1], after = lone ? f2.doc : f1.doc;   // of the same row tiles
                const bool first = n < (lone ? 2 : 1);
                Step s{tiles_of, f.doc, t0, 0, {}, row0, token0};
                if (f.doc != before) s.flags |= kFirst;
                if (f.doc != after) s.flags |= kLast;
                if (f.doc != f1.doc) s.flags |= f.doc == was[1] ? kPassLast | kJoin : uint32_t(kPassLast);
                if (n == 0) s.flags |= kUnitFirst;
                if (f1.doc < 0) s.flags |= kUnitLast;
                if (first) s.flags |= kTileFirst;
                if (after < 0) s.flags |= kTileLast;
                was[0] = was[1];
                was[1] = f.doc;
                if (plain && f.tile * 128 + 128 <= p.S) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s.mask[i] = kAll;
                } else {
                    bool gaps = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = f.tile * 128 + 32 * i + lane;
                        const bool in = j < p.S, mine = in && (f.whole || tiles.docs.of(U.b, j) == f.doc);
                        s.mask[i] = __ballot_sync(kAll, mine);
                        if (s.mask[i] != kAll) s.flags |= kMasked;
                        gaps |= in && !mine;
                    }
                    if (__any_sync(kAll, gaps)) s.flags |= kForeign;
                }
                if (!tell(s) || !load(tk, F::B_KFULL, U, f.tile, s.flags)) return false;
                if (first) {
                    for (int a = 0; a < 2; ++a) {
                        if (!(tiles_of & (a ? kTile1 : kTile0))) continue;
                        if (!sy.wait_warp(sy.bar(F::B_QEMPTY + a), (q_n[a] & 1u) ^ 1u)) return false;
                        ++q_n[a];
                        if (lane == 0) {
                            const uint32_t full = sy.bar(F::B_QFULL + a);
                            mbar_arrive_expect_tx(full, p.rpt * p.G * HD * 2);
                            for (int r = 0; r < F::NREG; ++r)
                                load_box(base + a * F::TILE + r * F::REG, tq, full, r * F::HDB, U.kh * p.G, t0 + (lone ? 0 : a * p.rpt), int(U.b));
                        }
                    }
                }
                if (!load(tv, F::B_VFULL, U, f.tile, s.flags)) return false;
                f = f1;
                f1 = f2;
                f2 = behind(f1);
            }
        }
        const Unit none(p, 0);
        return tell({kEnd, -1}) && load(tk, F::B_KFULL, none, 0, kEnd) && load(tv, F::B_VFULL, none, 0, kEnd);
    };
    run();
    // every issued load lands before the block may exit
    if (lane == 0) {
        for (uint32_t n = slot_n < F::SLOTS ? 0u : slot_n - F::SLOTS; n < slot_n; ++n)   // k's are even
            drained(sy.bar((n & 1u ? F::B_VFULL : F::B_KFULL) + n % F::SLOTS), (n / 2u / F::CYCLE) & 1u);
        for (int a = 0; a < 2; ++a)
            if (q_n[a]) drained(sy.bar(F::B_QFULL + a), (q_n[a] - 1u) & 1u);
    }
}

// The slots of k (from 0) or v (from 1) of one step after another, and the parity of their barriers.
template <int SLOTS>
struct Slot {
    const uint32_t first;
    uint32_t st, par = 0;
    __device__ __forceinline__ explicit Slot(uint32_t at) : first(at), st(at) {}
    __device__ __forceinline__ void next() {
        st = st + 2 < SLOTS ? st + 2 : st + 2 - SLOTS;
        par ^= st == first ? 1u : 0u;
    }
};

// Three warps issue, the scores of either row tile and the products of both. The
// scores of a step are two tiles of 64 columns in buffers of their own, which the
// probabilities take over: a half's next scores follow when its product is through,
// while the softmax works on the other half. (Each barrier that is waited for or
// committed to costs an issuing warp some 100 cycles in which it issues nothing: one
// warp for scores and products took 3600 cycles a step of HD 128, whose products are
// 2048.)
template <int HD>
__device__ __forceinline__ void fwd_scores(const Sync& sy, uint32_t base, uint32_t tmem, const volatile uint32_t* said, int a) {
    using F = FwdShape<HD>;
    constexpr uint32_t id_s = make_idesc_bf16(128, 64, 0, 0);
    constexpr uint32_t half_rows = (64 * F::ROWB) >> 4;   // to the second 64 rows of a tile
    const uint64_t qd = make_smem_desc(base + a * F::TILE, 16, F::SBO, F::SWZ), kd = make_smem_desc(base + F::OFF_KV, 16, F::SBO, F::SWZ);
    const uint32_t q_lo = uint32_t(qd), q_hi = uint32_t(qd >> 32), k_lo = uint32_t(kd), k_hi = uint32_t(kd >> 32);
    const uint32_t t_s = tmem + F::TM_S + 128 * a;
    const uint32_t yes = elect();
    uint32_t q_n = 0, n = 0;
    Slot<F::SLOTS> k(0);
    auto run = [&]() {
        for (;; k.next()) {
            if (!sy.wait_warp(sy.bar(F::B_KFULL + k.st), k.par)) return;
            const uint32_t flags = __reduce_or_sync(kAll, said[k.st]);
            if (flags & kEnd) return;
            const bool mine = flags & (a ? kTile1 : kTile0);
            if (mine && (flags & kTileFirst)) {
                if (!sy.wait_warp(sy.bar(F::B_QFULL + a), q_n++ & 1u)) return;
            }
            if (!mine) {
                if (yes) mbar_arrive(sy.bar(F::B_EMPTY + k.st));
                continue;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!sy.wait_warp(sy.bar(F::B_DONE + 2 * a + h), (n & 1u) ^ 1u)) return;
                tc_fence_after();
                scores<HD, F::REG, F::REG>(yes, t_s + 64 * h, q_lo, q_hi, k_lo + ((k.st * F::TILE) >> 4) + half_rows * h, k_hi, id_s);
                commit(yes, sy.bar(F::B_SFULL + 2 * a + h));
            }
            ++n;
            if (flags & kTileLast) commit(yes, sy.bar(F::B_QEMPTY + a));
            commit(yes, sy.bar(F::B_EMPTY + k.st));
        }
    };
    run();
    commit(yes, sy.bar(F::B_DRAIN + a));
    if (yes) drained(sy.bar(F::B_DRAIN + a), 0);
}

template <int HD, int KIND>
__device__ __forceinline__ void fwd_products(const Sync& sy, uint32_t base, const uint8_t* base_ptr, uint32_t tmem, const volatile uint32_t* said) {
    using F = FwdShape<HD>;
    constexpr uint32_t id_o = make_idesc_bf16(128, HD, 0, 1);
    constexpr uint32_t half_rows = (64 * F::ROWB) >> 4;
    const uint64_t vd = make_smem_desc(base + F::OFF_KV, F::REG, F::SBO, F::SWZ);
    const uint32_t v_lo = uint32_t(vd), v_hi = uint32_t(vd >> 32);
    const uint32_t yes = elect();
    uint32_t n[2] = {0, 0}, o_n[2] = {0, 0}, v_n = 0;
    Slot<F::SLOTS> v(1);
    auto run = [&]() {
        for (;; v.next(), ++v_n) {
            if (!sy.wait_warp(sy.bar(F::B_VFULL + v.st), v.par)) return;
            const uint32_t flags = __reduce_or_sync(kAll, said[v.st]);
            if (flags & kEnd) return;
            if (KIND != kPlain && (flags & kForeign)) {
                // Columns of other documents, whose probabilities are 0: 0 times their values must be 0. By
                // this warp, since it waits for every v; who did so for some alone could take the phase of an
                // earlier one, still on its way, for its own.
                const uint32_t* const mask = reinterpret_cast<const uint32_t*>(base_ptr + F::OFF_MASK) + 4 * (v_n % F::MASKS);
#pragma unroll 1
                for (int i = 0; i < 4; ++i)
                    if (!(mask[i] >> (threadIdx.x & 31) & 1u))
                        zero_row<HD, F::REG>(base + F::OFF_KV + v.st * F::TILE, 32 * i + int(threadIdx.x & 31));
                fence_proxy_async_smem();
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int h = i >> 1, a = i & 1;
                if (!(flags & (a ? kTile1 : kTile0))) continue;
                if (h == 0 && (flags & kFirst) && !sy.wait_warp(sy.bar(F::B_OREAD + a), (o_n[a]++ & 1u) ^ 1u)) return;
                if (!sy.wait_warp(sy.bar(F::B_PFULL + 2 * a + h), n[a] & 1u)) return;
                tc_fence_after();
                product<HD, 64>(yes, tmem + F::TM_O + F::OW * a, tmem + F::TM_S + 128 * a + 64 * h,
                                v_lo + ((v.st * F::TILE) >> 4) + half_rows * h, v_hi, id_o, h == 0 && (flags & kFirst) != 0);
                commit(yes, sy.bar(F::B_DONE + 2 * a + h));
                if (h == 1) {
                    ++n[a];
                    if (flags & kLast) commit(yes, sy.bar(F::B_OFULL + a));
                }
            }
            if (yes) mbar_arrive(sy.bar(F::B_EMPTY + v.st));   // k's slots are given back by two
            commit(yes, sy.bar(F::B_EMPTY + v.st));
        }
    };
    run();
    commit(yes, sy.bar(F::B_DRAIN + 2));
    if (yes) drained(sy.bar(F::B_DRAIN + 2), 0);
}

// One row of scores to a thread, which keeps the reference of its powers and their
// sum, and leaves them for the way out.
template <int HD>
__device__ __forceinline__ void fwd_softmax(const Sync& sy, uint8_t* base_ptr, uint32_t tmem, const Step* steps) {
    using F = FwdShape<HD>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, a = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + F::TM_S + 128 * a, t_o = t_lane + F::TM_O + F::OW * a;
    float2* const stat = reinterpret_cast<float2*>(base_ptr + F::OFF_STAT) + a * 128 + r;
    uint32_t heard = 0, s_n = 0, passes = 0;
    float ref = 0.f, l = 0.f;
    for (;;) {
        const uint32_t e = heard % kSteps;
        if (!sy.wait_warp(sy.bar(F::B_TOLD + e), (heard / kSteps) & 1u)) return;
        ++heard;
        const uint32_t flags = steps[e].flags;
        const uint4 columns = *reinterpret_cast<const uint4*>(steps[e].mask);
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.bar(F::B_HEARD + e));
        if (flags & kEnd) return;
        if (flags & (a ? kTile1 : kTile0)) {
            if (flags & kFirst) l = 0.f;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (!sy.wait_warp(sy.bar(F::B_SFULL + 2 * a + h), s_n & 1u)) return;
                tc_fence_after();
                const uint32_t t_h = t_s + 64 * h;
                float s[64];
                tmem_ld32(t_h, s);
                tmem_ld32(t_h + 32, s + 32);
                tmem_wait_ld();
                behind_wait(s);
                behind_wait(s + 32);
                if (flags & kMasked) {
                    const uint32_t m0 = h ? columns.z : columns.x, m1 = h ? columns.w : columns.y;
#pragma unroll
                    for (int j = 0; j < 64; ++j) s[j] = ((j < 32 ? m0 : m1) >> (j & 31)) & 1u ? s[j] : -INFINITY;
                }
                // By the reference of the tiles before, which the probabilities, their sums and O hold at
                // any scale: only where a row's sum leaves 2^32, or is 0 so far, does its maximum become it.
                // (One copy of this code for all of that: more of it did not stay in the instruction cache.)
                float sum = 0.f;
                bool anew = l == 0.f;
#pragma unroll 1
                for (bool again = false;; again = true) {
                    if (__any_sync(kAll, anew)) {
                        float t0 = fmaxf(s[0], s[1]), t1 = fmaxf(s[2], s[3]);
#pragma unroll
                        for (int j = 4; j < 64; j += 4) {
                            t0 = max3f(t0, s[j], s[j + 1]);
                            t1 = max3f(t1, s[j + 2], s[j + 3]);
                        }
                        const float top = fmaxf(t0, t1) * kLog2e, old = ref;
                        if (l == 0.f) ref = top == -INFINITY ? 0.f : top;
                        else if (anew) ref = fmaxf(ref, top);
                        const float by = l == 0.f ? 1.f : ex2_approx(old - ref);
                        if (__any_sync(kAll, by != 1.f)) {
                            // O of the halves before this one
                            if (!sy.wait_warp(sy.bar(F::B_DONE + 2 * a + (h ^ 1)), (s_n + h + 1) & 1u)) {
                                tmem_wait_st();
                                return;
                            }
                            tc_fence_after();
                            l *= by;
#pragma unroll 1
                            for (int q = 0; q < (HD + 31) / 32; ++q) {
                                float o[32];
                                tmem_ld32(t_o + 32 * q, o);
                                tmem_wait_ld();
                                behind_wait(o);
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] *= by;
                                tmem_st32(t_o + 32 * q, o);
                            }
                        }
                    }
                    const uint64_t l2e2 = f2_pack(kLog2e, kLog2e), neg2 = f2_pack(-ref, -ref);
                    uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float e0, e1;
                            f2_unpack(f2_fma(f2_pack(s[32 * q + 2 * j], s[32 * q + 2 * j + 1]), l2e2, neg2), e0, e1);
                            e0 = ex2_approx(e0);
                            e1 = ex2_approx(e1);
                            pk[j] = pack_bf16x2(e0, e1);
                            if (j & 1) acc1 = f2_add(acc1, f2_pack(e0, e1));
                            else acc0 = f2_add(acc0, f2_pack(e0, e1));
                        }
                        tmem_st16(t_h + 16 * q, pk);
                    }
                    float x0, x1;
                    f2_unpack(f2_add(acc0, acc1), x0, x1);
                    sum = x0 + x1;
                    anew = !(sum <= kSumLimit);
                    if (again || !__any_sync(kAll, anew)) break;
                }
                l += sum;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sy.bar(F::B_PFULL + 2 * a + h));
            }
            ++s_n;
            if (flags & kLast) {
                // the pass before has left (else its values and a barrier's phase would be overtaken)
                if (!sy.wait_warp(sy.bar(F::B_OREAD + a), (passes++ & 1u) ^ 1u)) return;
                *stat = make_float2(l, ref);
                __syncwarp();
                if (lane == 0) mbar_arrive(sy.bar(F::B_STAT + a));
            }
        }
    }
}

// The sums of a pass on their way out, by warps of their own: the softmax goes on
// with the next rows meanwhile. (With its own threads' stores in its way a unit of
// four steps took 11.3 us, 7.8 of them its steps.)
template <int HD, int KIND>
__device__ __forceinline__ void fwd_out(const FwdParams& p, const Sync& sy, uint8_t* base_ptr, uint32_t tmem, const Step* steps) {
    using F = FwdShape<HD>;
    const bool lone = KIND == kFew && p.lone, split = KIND == kFew && p.splits > 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16) + F::TM_O;
    const float2* const stat = reinterpret_cast<const float2*>(base_ptr + F::OFF_STAT) + r;
    const int tok = r / p.G, g = r - tok * p.G;
    uint32_t heard = 0, passes[2] = {0, 0};
    int64_t row[2] = {-1, -1};   // of out; < 0: none
    int doc[2] = {-1, -1};
    bool written[2] = {false, false};
    // One row tile that both have taken steps of: their sums joined, by references of their own.
    auto out_joined = [&](uint32_t flags, bool mine, int64_t to_row) -> bool {
        const bool has[2] = {(flags & (kTile0 | kJoin)) != 0, (flags & (kTile1 | kJoin)) != 0};
        float2 st[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            if (!has[a]) continue;
            const uint32_t n = passes[a]++;
            if (!sy.wait_warp(sy.bar(F::B_STAT + a), n & 1u)) return false;
            st[a] = stat[a * 128];
            if (!sy.wait_warp(sy.bar(F::B_OFULL + a), n & 1u)) return false;
        }
        tc_fence_after();
        const bool r0 = st[0].x != 0.f, r1 = st[1].x != 0.f;
        const float ref = r0 && r1 ? fmaxf(st[0].y, st[1].y) : r0 ? st[0].y : st[1].y;
        const float w0 = r0 ? exp2f(st[0].y - ref) : 0.f, w1 = r1 ? exp2f(st[1].y - ref) : 0.f;
        const float l = st[0].x * w0 + st[1].x * w1, inv = r0 || r1 ? 1.f / l : 0.f, by0 = w0 * inv, by1 = w1 * inv;
#pragma unroll 1
        for (int q = 0; q < (HD + 31) / 32; ++q) {
            __syncwarp();
            float o[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0.f;
            if (has[0]) {
                tmem_ld32(t_lane + 32 * q, o);
                tmem_wait_ld();
                behind_wait(o);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= by0;
            if (has[1]) {
                float x[32];
                tmem_ld32(t_lane + F::OW + 32 * q, x);
                tmem_wait_ld();
                behind_wait(x);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = fmaf(x[j], by1, o[j]);
            }
            if (!mine) continue;
            constexpr int W = HD < 32 ? HD : 32;
            if (split) {
                float4* const to = reinterpret_cast<float4*>(p.part + to_row * HD + 32 * q);
#pragma unroll
                for (int j = 0; j < W / 4; ++j) to[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            } else {
                uint4* const to = reinterpret_cast<uint4*>(p.out + to_row * HD + 32 * q);
#pragma unroll
                for (int j = 0; j < W / 8; ++j)
                    to[j] = make_uint4(pack_bf16x2(o[8 * j], o[8 * j + 1]), pack_bf16x2(o[8 * j + 2], o[8 * j + 3]),
                                       pack_bf16x2(o[8 * j + 4], o[8 * j + 5]), pack_bf16x2(o[8 * j + 6], o[8 * j + 7]));
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
            for (int a = 0; a < 2; ++a)
                if (has[a]) mbar_arrive(sy.bar(F::B_OREAD + a));
        if (!mine) return false;
        const float lse2 = r0 || r1 ? ref + log2f(l) : -INFINITY;
        if (split) p.part_lse[to_row] = lse2;
        else if (p.lse) p.lse[to_row] = lse2 * kLn2;
        return true;
    };
    for (;;) {
        const uint32_t e = heard % kSteps;
        if (!sy.wait_warp(sy.bar(F::B_TOLD + e), (heard / kSteps) & 1u)) return;
        ++heard;
        const uint32_t flags = steps[e].flags;
        const int d = steps[e].doc;
        if (flags & (kUnitFirst | kNone)) {
            const int t0 = steps[e].t0;
            const int64_t row0 = steps[e].row, token0 = steps[e].token;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const int i = a * p.rpt + tok;
                row[a] = tok < p.rpt && t0 + i < p.L && !(a && lone) ? row0 + int64_t(i) * p.NH + g : -1;
                doc[a] = KIND != kPlain && row[a] >= 0 && p.doc ? __ldg(p.doc + token0 + i) : 0;
                written[a] = false;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.bar(F::B_HEARD + e));
        if (flags & kEnd) return;
        if (lone) {
            if (flags & kPassLast) written[0] |= out_joined(flags, row[0] >= 0 && doc[0] == d, row[0]);
        } else if (flags & kLast) {
#pragma unroll 1
            for (int a = 0; a < ((flags & kTile1) ? 2 : 1); ++a) {
                const int64_t to_row = a ? row[1] : row[0];
                const bool mine = to_row >= 0 && (a ? doc[1] : doc[0]) == d;
                const uint32_t n = a ? passes[1]++ : passes[0]++;
                if (!sy.wait_warp(sy.bar(F::B_STAT + a), n & 1u)) return;
                const float2 st = stat[a * 128];
                const bool real = st.x > 0.f || st.x != st.x;
                const float inv = real ? 1.f / st.x : 0.f;
                if (!sy.wait_warp(sy.bar(F::B_OFULL + a), n & 1u)) return;
                tc_fence_after();
                if (split) {   // in 32 bits
#pragma unroll 1
                    for (int q = 0; q < (HD + 31) / 32; ++q) {
                        __syncwarp();
                        float o[32];
                        tmem_ld32(t_lane + F::OW * a + 32 * q, o);
                        tmem_wait_ld();
                        behind_wait(o);
                        if (!mine) continue;
                        float4* const to = reinterpret_cast<float4*>(p.part + to_row * HD + 32 * q);
#pragma unroll
                        for (int j = 0; j < (HD < 32 ? HD : 32) / 4; ++j)
                            to[j] = make_float4(o[4 * j] * inv, o[4 * j + 1] * inv, o[4 * j + 2] * inv, o[4 * j + 3] * inv);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sy.bar(F::B_OREAD + a));
                } else {
                    // 32 columns, or 64, to a round: the registers of a whole row are too many
                    constexpr int Q = (HD + 31) / 32, N = Q < 2 ? Q : 2, COLS = HD < 64 ? HD : 64;
#pragma unroll 1
                    for (int c = 0; c < Q / N; ++c) {
                        __syncwarp();
                        uint32_t kept[16 * N];
#pragma unroll
                        for (int q = 0; q < N; ++q) {
                            float o[32];
                            tmem_ld32(t_lane + F::OW * a + 32 * (N * c + q), o);
                            tmem_wait_ld();
                            behind_wait(o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) kept[16 * q + j] = pack_bf16x2(o[2 * j] * inv, o[2 * j + 1] * inv);
                        }
                        if (c == Q / N - 1) {   // the next pass's products may come
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(sy.bar(F::B_OREAD + a));
                        }
                        if (!mine) continue;
                        uint16_t* const to = p.out + to_row * HD + 32 * N * c;
                        if (p.out_v8) {
#pragma unroll
                            for (int j = 0; j < COLS / 16; ++j) st_global_v8(to + 16 * j, kept + 8 * j);
                        } else {
#pragma unroll
                            for (int j = 0; j < COLS / 8; ++j)
                                reinterpret_cast<uint4*>(to)[j] = make_uint4(kept[4 * j], kept[4 * j + 1], kept[4 * j + 2], kept[4 * j + 3]);
                        }
                    }
                }
                if (mine) {
                    const float lse2 = real ? st.y + log2f(st.x) : -INFINITY;
                    if (split) p.part_lse[to_row] = lse2;
                    else if (p.lse) p.lse[to_row] = lse2 * kLn2;
                    if (a) written[1] = true;
                    else written[0] = true;
                }
            }
        }
        if (flags & kUnitLast) {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                if (row[a] < 0 || written[a]) continue;   // else a row that sees nothing
                if (split) {
                    p.part_lse[row[a]] = -INFINITY;
                } else {
                    uint4* const to = reinterpret_cast<uint4*>(p.out + row[a] * HD);
#pragma unroll 1
                    for (int j = 0; j < HD / 8; ++j) to[j] = make_uint4(0, 0, 0, 0);
                    if (p.lse) p.lse[row[a]] = -INFINITY;
                }
            }
        }
    }
}

// out and lse of the softmax over a stream of column tiles: s = q k^T into tensor
// memory, p = 2^(s log2e - ref) back into its place in bf16, O += p v. A row keeps
// its reference while its sums stay in range, so O is scaled anew only where they
// do not. Where the grid has one row tile, the block's two are the same rows and
// take the column tiles in turns: one chain of scores, softmax and products leaves
// the block waiting (one token, 16 heads of 128 over 65536 states of 4 heads: 40 us
// by one, 33 by two). Few rows share their states out over blocks as well.
//
// Bound by the chain of its warps where the states are few: each half of a step
// passes from the scores to the softmax to the products and back, and every hand-over
// costs some 170 to 230 cycles. 49152 tokens, 16 heads of 128 over 512 states: 168 us,
// 1.23 PFLOP/s, tensor cores 68 % busy; 24576 over 6144: 748 us, 1.65 PFLOP/s, 87 %
// (1.93 is a large product alone). Few rows at head size 128 are near the memory's
// bound: 8 tokens over 131072 states of 4 heads 5.7 TB/s; below it the chain's (64:
// 3.3 TB/s).
//
// Two row tiles to a block, one block to an SM, persistent. Its warps of five kinds
// share little room for instructions, so what a call does not need is left out:
// KIND kFew has row tiles so few that the states are split, or one alone; kDocuments
// the search for documents' tiles, which kPlain does without (24576 tokens over 6144
// states 862 -> 782 us, 49152 over 512 183 -> 170 by that alone). The same source laid
// out otherwise by the compiler is up to 5 % faster or slower.
//
//   warps 0..3, 4..7  the softmax of either row tile;
//   warps 8..11       results on their way out;
//   warp 12           finds the column tiles that the rows see, TMA;
//   warps 13, 14      issue the scores of either row tile; 13 owns the tensor memory;
//   warp 15           issues the products.
template <int HD, int KIND>
__global__ void __launch_bounds__(kFwdThreads, 1)
cross_fwd_tiles(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                const __grid_constant__ FwdParams p) {
    using F = FwdShape<HD>;
    extern __shared__ __align__(1024) uint8_t base_ptr[];   // no room to align it here
    const uint32_t base = smem_u32(base_ptr);
    if (base & 1023u) {
        if (threadIdx.x == 0) atomicOr(&g_cross_timeout_flag, 1u);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile uint32_t* const misc = reinterpret_cast<volatile uint32_t*>(base_ptr + F::OFF_MISC);
    Step* const steps = reinterpret_cast<Step*>(base_ptr + F::OFF_STEP);
    const Sync sy{base + F::OFF_BAR, misc + 1};
    // rows of q's tiles that no load writes (G does not divide 128) hold zeros
    if (p.rpt * p.G != 128)
        for (int i = threadIdx.x; i < 2 * F::TILE / 16; i += kFwdThreads) reinterpret_cast<uint4*>(base_ptr)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (threadIdx.x == 0) {
        for (int i = 0; i < F::NBAR; ++i) {
            const bool by_warps = (i >= F::B_PFULL && i < F::B_PFULL + 4) || (i >= F::B_OREAD && i < F::B_OREAD + 2) ||
                                  (i >= F::B_STAT && i < F::B_STAT + 2);
            mbar_init(sy.bar(i), i >= F::B_EMPTY && i < F::B_EMPTY + F::SLOTS ? 2u : by_warps ? 4u
                                 : i >= F::B_HEARD && i < F::B_HEARD + kSteps ? 12u : 1u);
        }
        misc[1] = 0u;
        misc[2] = beat_clock() - kWaitTicks - 1u;   // long ago
        fence_mbar_init();
    }
    if (warp == 12 && lane == 0) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    if (warp == 13) {
        tmem_alloc(base + F::OFF_MISC, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    dependents_may_start();
    if (warp < 8) {
        regs_increase<FwdRegs<KIND>::kSoftmax>();
        fwd_softmax<HD>(sy, base_ptr, tmem, steps);
    } else if (warp < 12) {
        regs_decrease<FwdRegs<KIND>::kOut>();
        fwd_out<HD, KIND>(p, sy, base_ptr, tmem, steps);
    } else {
        regs_decrease<FwdRegs<KIND>::kLow>();
        if (warp == 12) fwd_producer<HD, KIND>(p, sy, base, base_ptr, steps, misc + 3, &tq, &tk, &tv);
        if (warp == 13 || warp == 14) fwd_scores<HD>(sy, base, __reduce_or_sync(kAll, tmem), misc + 3, warp - 13);
        if (warp == 15) fwd_products<HD, KIND>(sy, base, base_ptr, __reduce_or_sync(kAll, tmem), misc + 3);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The splits of a row joined: out = sum_s 2^(lse_s - top) out_s / sum_s 2^(lse_s - top),
// by `parts` groups of HD / 4 threads, each of every so many-th split and by a
// reference of its own. Bound by the latency of its loads: all of a group's are in
// flight at once.
template <int HD>
__global__ void __launch_bounds__(256) cross_join(const FwdParams p, int parts) {
    constexpr int PER = HD / 4;
    __shared__ float4 sums[256];
    __shared__ float2 weights[256];
    const int rows = 256 / (PER * parts);   // of a block
    const int group = threadIdx.x / PER, part = group % parts, c = threadIdx.x % PER * 4;
    const int64_t row = int64_t(blockIdx.x) * rows + group / parts;
    wait_for_primary();
    const bool in = row < p.rows;
    float top = -INFINITY, sum = 0.f, o[4] = {};
    if (in) {
        for (int s0 = part; s0 < p.splits; s0 += 8 * parts) {
            float x[8];
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = s0 + i * parts;
                x[i] = s < p.splits ? p.part_lse[s * p.rows + row] : -INFINITY;
                if (s < p.splits) v[i] = *reinterpret_cast<const float4*>(p.part + (s * p.rows + row) * HD + c);
            }
            float most = top;
#pragma unroll
            for (int i = 0; i < 8; ++i) most = fmaxf(most, x[i]);
            const float by = top == -INFINITY ? 0.f : exp2f(top - most);
            sum *= by;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] *= by;
            top = most;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (x[i] == -INFINITY) continue;   // nothing written there
                const float w = exp2f(x[i] - top);
                sum += w;
                o[0] = fmaf(w, v[i].x, o[0]);
                o[1] = fmaf(w, v[i].y, o[1]);
                o[2] = fmaf(w, v[i].z, o[2]);
                o[3] = fmaf(w, v[i].w, o[3]);
            }
        }
    }
    sums[threadIdx.x] = make_float4(o[0], o[1], o[2], o[3]);
    weights[threadIdx.x] = make_float2(top, sum);
    __syncthreads();
    if (!in || part) return;
    float ref = top;
    for (int i = 1; i < parts; ++i) ref = fmaxf(ref, weights[threadIdx.x + i * PER].x);
    if (ref == -INFINITY) ref = 0.f;
    const float by = exp2f(top - ref);
    sum *= by;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] *= by;
    for (int i = 1; i < parts; ++i) {
        const float4 v = sums[threadIdx.x + i * PER];
        const float2 x = weights[threadIdx.x + i * PER];
        const float w = exp2f(x.x - ref);
        sum = fmaf(w, x.y, sum);
        o[0] = fmaf(w, v.x, o[0]);
        o[1] = fmaf(w, v.y, o[1]);
        o[2] = fmaf(w, v.z, o[2]);
        o[3] = fmaf(w, v.w, o[3]);
    }
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    *reinterpret_cast<uint2*>(p.out + row * HD + c) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    if (p.lse && c == 0) p.lse[row] = sum > 0.f || sum != sum ? (ref + log2f(sum)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------------ backward

// Two passes of one kernel, each with fixed rows and streamed columns, so that
// every sum has a place and an order of its own:
//   DQ:  rows q, dout; columns k, v:   dq += ds k;
//   DKV: rows k, v; columns q, dout:   dv += p^T dout, dk += ds^T q,
// with s = rows0 columns0^T and dp = rows1 columns1^T, 128 x 64 a step, in two
// buffers of tensor memory that two warpgroups take in turns; p and ds take the
// place of s and dp and are multiplied from there.
struct BwdParams {
    int32_t nr, nc, rpt, cpt;            // tokens of an entry and of a tile, rows' and columns'
    int32_t Gr, Gc, heads, NH, NKV, G;   // heads of a row's and a column's token in a tile; heads of a row's token
    int32_t tiles_r, tiles_c, splits, per_split, units, B;
    const int32_t *doc_r, *doc_c;
    const uint16_t *out, *dout;          // for the statistics
    const float* lse;
    float2* stat;                        // (row of q): -lse log2e, -delta: out . dout
    float2* stat_kv;                     // ... as DQ leaves it for DKV: where it has the sum itself, that
    uint16_t* grad[2];                   // DQ: dq; DKV: dv, dk
    int64_t ts[2];
    float* part;                         // splits > 1: (split, gradient, row, HD) in 32 bits
    int64_t rows;                        // B * nr * heads
};

constexpr int kBwdSteps = 4;

template <int HD>
struct BwdShape : Geom<HD> {
    using G = Geom<HD>;
    static constexpr int XREG = 128 * G::ROWB, XTILE = G::NREG * XREG, YREG = 64 * G::ROWB, YTILE = G::NREG * YREG;
    static constexpr int STAGES = 5;
    static constexpr int OFF_Y = 2 * XTILE, OFF_STAT = OFF_Y + STAGES * 2 * YTILE, OFF_STEP = OFF_STAT + STAGES * 512;
    static constexpr int OFF_BAR = OFF_STEP + kBwdSteps * 48;
    static constexpr int B_FULL = 0, B_EMPTY = STAGES, B_XFULL = 2 * STAGES, B_XEMPTY = B_XFULL + 1, B_SFULL = B_XEMPTY + 1,
                         B_PFULL = B_SFULL + 2, B_AFULL = B_PFULL + 2, B_AREAD = B_AFULL + 2, B_TOLD = B_AREAD + 2,
                         B_HEARD = B_TOLD + kBwdSteps, B_DRAIN = B_HEARD + kBwdSteps, NBAR = B_DRAIN + 2;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // tensor memory, abort flag, beat, the stages' flags
    static constexpr int NEED = OFF_MISC + 12 + 4 * STAGES, SMEM = NEED > 120 * 1024 ? NEED : 120 * 1024;
    // sums: dv and dk, or dq of one pass and of the next; s and dp of either buffer
    static constexpr uint32_t AW = HD < 32 ? 32 : HD, TM_S = 256;
    static_assert(SMEM <= 232448, "shared memory");
};

constexpr int kBwdThreads = 512;
constexpr uint32_t kBwdSoftmax = 144, kBwdOut = 112, kBwdLow = 112;   // of 512 x 128
static_assert(2 * kBwdSoftmax + kBwdOut + kBwdLow <= 4 * 128, "register split");

// -lse log2e and -delta of every row of q, HD / 8 lanes to a row. Bound by the
// read of out and dout (24576 tokens, 16 heads of 128: 33 us, 6.2 TB/s). A row that
// sees nothing gets -infinity: its powers are 0.
constexpr int kStatLoads = 4;   // of either tensor to a thread, in flight at once

template <int HD>
__global__ void __launch_bounds__(256) cross_stat(const BwdParams p, int64_t rows) {
    constexpr int PER = HD / 8;
    const int64_t first = int64_t(blockIdx.x) * (256 * kStatLoads) + threadIdx.x;
    dependents_may_start();
    uint4 x[kStatLoads], y[kStatLoads];
    float lse[kStatLoads];
#pragma unroll
    for (int k = 0; k < kStatLoads; ++k) {
        const int64_t i = first + 256 * k, row = i / PER;
        x[k] = y[k] = make_uint4(0, 0, 0, 0);
        lse[k] = 0.f;
        if (row >= rows) continue;
        x[k] = __ldcs(reinterpret_cast<const uint4*>(p.out + i * 8));
        y[k] = *reinterpret_cast<const uint4*>(p.dout + i * 8);
        if (i % PER == 0) lse[k] = p.lse[row];
    }
#pragma unroll
    for (int k = 0; k < kStatLoads; ++k) {
        const int64_t i = first + 256 * k, row = i / PER;
        const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, v[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum = fmaf(__uint_as_float(u[j] << 16), __uint_as_float(v[j] << 16), sum);
            sum = fmaf(__uint_as_float(u[j] & 0xffff0000u), __uint_as_float(v[j] & 0xffff0000u), sum);
        }
#pragma unroll
        for (int o = PER / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (row < rows && i % PER == 0) {
            const float2 st = make_float2(lse[k] == -INFINITY ? -INFINITY : -lse[k] * kLog2e, -sum);
            p.stat[row] = st;
            p.stat_kv[row] = st;
        }
    }
}

template <int HD, bool DKV>
__device__ __forceinline__ void bwd_producer(const BwdParams& p, const Sync& sy, uint32_t base, uint8_t* base_ptr, Step* steps, volatile uint32_t* said,
                                             const CUtensorMap* tx0, const CUtensorMap* tx1, const CUtensorMap* ty0, const CUtensorMap* ty1) {
    using F = BwdShape<HD>;
    const int lane = threadIdx.x & 31;
    Tiles<2> tiles{{p.doc_c, p.nc}, p.cpt, sy};
    const Docs rows{p.doc_r, p.nr};
    const bool plain = !p.doc_r && !p.doc_c;   // every column is of every row's document
    uint32_t told = 0, it = 0, x_n = 0;
    // this lane's columns of a tile: token and head
    const int ctok[2] = {lane / p.Gc, (lane + 32) / p.Gc}, chead[2] = {lane % p.Gc, (lane + 32) % p.Gc};

    auto tell = [&](const Step& s) -> bool {
        const uint32_t e = told % kBwdSteps;
        if (!sy.wait_warp(sy.bar(F::B_HEARD + e), ((told / kBwdSteps) & 1u) ^ 1u)) return false;
        ++told;
        if (lane == 0) {
            steps[e] = s;
            mbar_arrive(sy.bar(F::B_TOLD + e));
        }
        return true;
    };
    struct Found { int tile, doc; bool whole; };
    auto run = [&]() {
        for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
            int rest = u;
            const int tile_r = rest % p.tiles_r;
            rest /= p.tiles_r;
            const int kh = rest % p.NKV;
            rest /= p.NKV;
            const int64_t b = rest % p.B;
            const int split = rest / p.B;
            const int t0 = tile_r * p.rpt, n_tok = min(p.rpt, p.nr - t0);
            const int64_t token0 = b * p.nr + t0, row0 = token0 * p.heads + kh * p.Gr + split * (DKV ? 2 : 1) * p.rows;
            int doc[4] = {};
            if (!plain)
#pragma unroll
                for (int i = 0; i < 4; ++i) doc[i] = lane + 32 * i < n_tok ? rows.of(b, t0 + lane + 32 * i) : -1;
            const int k0 = split * p.per_split, k1 = min(k0 + p.per_split, p.tiles_c);
            int d = plain ? 0 : next_doc(doc, -1);
            if (!plain) tiles.begin(b, k0, k1, next_doc(doc, d) >= 0);
            // of document d from the tile on, or of those behind it; the columns of this lane that are
            auto mine = [&](int tile, int dd, int i) {
                const int t = tile * p.cpt + ctok[i];
                return ctok[i] < p.cpt && t < p.nc && tiles.docs.of(b, t) == dd;
            };
            auto next = [&](Found* f) {
                if (plain) {
                    f->doc = 0;
                    f->whole = true;
                    return f->tile < k1;
                }
                for (; d >= 0; d = next_doc(doc, d), f->tile = k0) {
                    f->tile = tiles.find(b, f->tile, k1, d, &f->whole);
                    while (f->tile < k1) {
                        f->doc = d;
                        if (f->whole || __any_sync(kAll, mine(f->tile, d, 0) || mine(f->tile, d, 1))) return true;
                        f->tile = tiles.find(b, f->tile + 1, k1, d, &f->whole);
                    }
                }
                return false;
            };
            Found f{k0, -1, false};
            bool have = next(&f);
            if (!have) {
                if (!tell({kNone | kUnitLast, -1, t0, kh, {}, row0, token0})) return false;
                continue;
            }
            // DKV: a step's statistics are read a step ahead
            float2 st[2], ahead[2];
            auto read = [&](const Found& x) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = x.tile * p.cpt + ctok[i];
                    const bool of = ctok[i] < p.cpt && t < p.nc && (x.whole || tiles.docs.of(b, t) == x.doc);
                    ahead[i] = of ? p.stat_kv[(b * p.nc + t) * p.NH + kh * p.G + chead[i]] : make_float2(0.f, 0.f);
                }
            };
            if (DKV) read(f);
            int was = -1;
            for (bool first = true; have; first = false) {
                Found g = f;
                ++g.tile;
                const bool more = next(&g);
                st[0] = ahead[0];
                st[1] = ahead[1];
                if (DKV && more) read(g);
                Step s{0, f.doc, t0, kh, {}, row0, token0};
                if (f.doc != was) s.flags |= kFirst;
                if (!more || g.doc != f.doc) s.flags |= kLast;
                if (first) s.flags |= kUnitFirst;
                if (!more) s.flags |= kUnitLast;
                was = f.doc;
                if (plain && p.cpt * p.Gc == 64 && (f.tile + 1) * p.cpt <= p.nc) {
                    s.mask[0] = s.mask[1] = kAll;
                } else {
                    bool gaps = false;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = f.tile * p.cpt + ctok[i];
                        const bool in = ctok[i] < p.cpt && t < p.nc, of = in && (f.whole || tiles.docs.of(b, t) == f.doc);
                        s.mask[i] = __ballot_sync(kAll, of);
                        if (s.mask[i] != kAll) s.flags |= kMasked;
                        gaps |= in && !of;
                    }
                    if (__any_sync(kAll, gaps)) s.flags |= kForeign;
                }
                if (!tell(s)) return false;
                const uint32_t sl = it % F::STAGES;
                if (!sy.wait_warp(sy.bar(F::B_EMPTY + sl), ((it / F::STAGES) & 1u) ^ 1u)) return false;
                ++it;
                if (DKV) {
                    float* const to = reinterpret_cast<float*>(base_ptr + F::OFF_STAT + sl * 512);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        to[lane + 32 * i] = st[i].x;
                        to[64 + lane + 32 * i] = st[i].y;
                    }
                    __syncwarp();
                }
                if (lane == 0) {
                    const uint32_t full = sy.bar(F::B_FULL + sl), to = base + F::OFF_Y + sl * 2 * F::YTILE;
                    said[sl] = s.flags;
                    mbar_arrive_expect_tx(full, 2 * p.cpt * p.Gc * HD * 2);
                    for (int r = 0; r < F::NREG; ++r) {
                        load_box(to + r * F::YREG, ty0, full, r * F::HDB, kh * p.Gc, f.tile * p.cpt, int(b));
                        load_box(to + F::YTILE + r * F::YREG, ty1, full, r * F::HDB, kh * p.Gc, f.tile * p.cpt, int(b));
                    }
                }
                if (first) {
                    if (!sy.wait_warp(sy.bar(F::B_XEMPTY), (x_n & 1u) ^ 1u)) return false;
                    ++x_n;
                    if (lane == 0) {
                        const uint32_t full = sy.bar(F::B_XFULL);
                        mbar_arrive_expect_tx(full, 2 * p.rpt * p.Gr * HD * 2);
                        for (int r = 0; r < F::NREG; ++r) {
                            load_box(base + r * F::XREG, tx0, full, r * F::HDB, kh * p.Gr, t0, int(b));
                            load_box(base + F::XTILE + r * F::XREG, tx1, full, r * F::HDB, kh * p.Gr, t0, int(b));
                        }
                    }
                }
                have = more;
                f = g;
            }
        }
        if (!tell({kEnd, -1})) return false;
        const uint32_t sl = it % F::STAGES;
        if (!sy.wait_warp(sy.bar(F::B_EMPTY + sl), ((it / F::STAGES) & 1u) ^ 1u)) return false;
        ++it;
        if (lane == 0) {
            said[sl] = kEnd;
            mbar_arrive(sy.bar(F::B_FULL + sl));
        }
        return true;
    };
    run();
    // every issued load lands before the block may exit
    if (lane == 0) {
        for (uint32_t s = 0; s < F::STAGES; ++s) {
            const uint32_t n = it / F::STAGES + (s < it % F::STAGES ? 1u : 0u);
            if (n) drained(sy.bar(F::B_FULL + s), (n - 1u) & 1u);
        }
        if (x_n) drained(sy.bar(F::B_XFULL), (x_n - 1u) & 1u);
    }
}

// Two warps issue: one the scores of a step, once the products of the last but one
// are through with their place, one those products. (One warp for both took 2800
// cycles a step of HD 128, its waits and commits between 24 products of 50.)
template <int HD>
__device__ __forceinline__ void bwd_scores(const Sync& sy, uint32_t base, uint32_t tmem, const volatile uint32_t* said) {
    using F = BwdShape<HD>;
    constexpr uint32_t id_s = make_idesc_bf16(128, 64, 0, 0);
    const uint64_t xd = make_smem_desc(base, 16, F::SBO, F::SWZ), yd = make_smem_desc(base + F::OFF_Y, 16, F::SBO, F::SWZ);
    const uint32_t x_lo = uint32_t(xd), x_hi = uint32_t(xd >> 32), y_lo = uint32_t(yd), y_hi = uint32_t(yd >> 32);
    const uint32_t yes = elect();
    uint32_t x_n = 0;
    uint32_t sl = 0, par = 0, was = F::STAGES - 2, was_par = 1;   // this step's stage and that of the last but one
    for (uint32_t i = 0;; ++i) {
        if (!sy.wait_warp(sy.bar(F::B_FULL + sl), par)) break;
        const uint32_t flags = __reduce_or_sync(kAll, said[sl]);
        if (flags & kEnd) break;
        if ((flags & kUnitFirst) && !sy.wait_warp(sy.bar(F::B_XFULL), x_n++ & 1u)) break;
        if (i >= 2 && !sy.wait_warp(sy.bar(F::B_EMPTY + was), was_par)) break;
        tc_fence_after();
        const uint32_t t_s = tmem + F::TM_S + 128 * (i & 1u), y = y_lo + ((sl * 2 * F::YTILE) >> 4);
        scores<HD, F::XREG, F::YREG>(yes, t_s, x_lo, x_hi, y, y_hi, id_s);
        scores<HD, F::XREG, F::YREG>(yes, t_s + 64, x_lo + (F::XTILE >> 4), x_hi, y + (F::YTILE >> 4), y_hi, id_s);
        commit(yes, sy.bar(F::B_SFULL + (i & 1u)));
        if (flags & kUnitLast) commit(yes, sy.bar(F::B_XEMPTY));
        if (++sl == F::STAGES) { sl = 0; par ^= 1u; }
        if (++was == F::STAGES) { was = 0; was_par ^= 1u; }
    }
    commit(yes, sy.bar(F::B_DRAIN));
    if (yes) drained(sy.bar(F::B_DRAIN), 0);
}

template <int HD, bool DKV>
__device__ __forceinline__ void bwd_products(const Sync& sy, uint32_t base, uint32_t tmem, const volatile uint32_t* said) {
    using F = BwdShape<HD>;
    constexpr uint32_t id_a = make_idesc_bf16(128, HD, 0, 1);
    const uint64_t zd = make_smem_desc(base + F::OFF_Y, F::YREG, F::SBO, F::SWZ);   // Y's columns outermost
    const uint32_t z_lo = uint32_t(zd), z_hi = uint32_t(zd >> 32);
    const uint32_t yes = elect();
    uint32_t passes = 0, sl = 0, par = 0;
    for (uint32_t i = 0;; ++i) {
        if (!sy.wait_warp(sy.bar(F::B_FULL + sl), par)) break;
        const uint32_t flags = __reduce_or_sync(kAll, said[sl]);
        if (flags & kEnd) break;
        const uint32_t buf = DKV ? 0u : passes & 1u;
        if ((flags & kFirst) && !sy.wait_warp(sy.bar(F::B_AREAD + buf), ((DKV ? passes : passes >> 1) & 1u) ^ 1u)) break;
        if (!sy.wait_warp(sy.bar(F::B_PFULL + (i & 1u)), (i >> 1) & 1u)) break;
        tc_fence_after();
        const uint32_t t_s = tmem + F::TM_S + 128 * (i & 1u), z = z_lo + ((sl * 2 * F::YTILE) >> 4);
        const bool fresh = (flags & kFirst) != 0;
        if (DKV) product<HD, 64>(yes, tmem, t_s, z + (F::YTILE >> 4), z_hi, id_a, fresh);
        product<HD, 64>(yes, tmem + F::AW * (DKV ? 1u : buf), t_s + 64, z, z_hi, id_a, fresh);
        if (!DKV) product<HD, 64>(yes, tmem + F::AW * buf, t_s, z, z_hi, id_a, false);
        commit(yes, sy.bar(F::B_EMPTY + sl));
        if (flags & kLast) {
            commit(yes, sy.bar(F::B_AFULL + buf));
            ++passes;
        }
        if (++sl == F::STAGES) { sl = 0; par ^= 1u; }
    }
    commit(yes, sy.bar(F::B_DRAIN + 1));
    if (yes) drained(sy.bar(F::B_DRAIN + 1), 0);
}

// Probabilities and their gradients of every second step, a row to a thread.
template <int HD, bool DKV>
__device__ __forceinline__ void bwd_softmax(const BwdParams& p, const Sync& sy, uint32_t base, uint8_t* base_ptr, uint32_t tmem, const Step* steps) {
    using F = BwdShape<HD>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, a = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16), t_s = t_lane + F::TM_S + 128 * a;
    const int tok = r / p.Gr, g = r - tok * p.Gr;
    uint32_t heard = 0, n = 0;   // n: steps with columns
    bool in = false;
    int doc = -1;
    int64_t row = 0;   // DQ: of the statistics
    float2 st = make_float2(0.f, 0.f);
    for (;;) {
        const uint32_t e = heard % kBwdSteps;
        if (!sy.wait_warp(sy.bar(F::B_TOLD + e), (heard / kBwdSteps) & 1u)) return;
        ++heard;
        const uint32_t flags = steps[e].flags;
        const int d = steps[e].doc;
        const uint2 columns = *reinterpret_cast<const uint2*>(steps[e].mask);
        if (!DKV && (flags & kUnitFirst)) {
            in = tok < p.rpt && steps[e].t0 + tok < p.nr;
            const int64_t token = steps[e].token + tok;
            doc = in && p.doc_r ? __ldg(p.doc_r + token) : 0;
            row = token * p.NH + steps[e].pad * p.G + g;
            if (in) st = p.stat[row];   // written by an earlier kernel
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.bar(F::B_HEARD + e));
        if (flags & kEnd) return;
        if (!(flags & kNone) && (n & 1u) == uint32_t(a)) {
            if (!sy.wait_warp(sy.bar(F::B_SFULL + a), (n >> 1) & 1u)) return;
            tc_fence_after();
            const uint32_t sl = n % F::STAGES;
            const float4* const cs = reinterpret_cast<const float4*>(base_ptr + F::OFF_STAT + sl * 512);
            const uint64_t l2e2 = f2_pack(kLog2e, kLog2e);
            auto load = [&](int q, float (&s)[32], float (&dp)[32]) {
                tmem_ld32(t_s + 32 * q, s);
                tmem_ld32(t_s + 64 + 32 * q, dp);
                tmem_wait_ld();
                behind_wait(s);
                behind_wait(dp);
                if (flags & kMasked) {
                    const uint32_t m = q ? columns.y : columns.x;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        s[j] = (m >> j) & 1u ? s[j] : -INFINITY;
                        dp[j] = (m >> j) & 1u ? dp[j] : 0.f;
                    }
                }
            };
            if (!DKV && (flags & (kFirst | kLast)) == (kFirst | kLast)) {
                // A row that sees one tile alone: delta from its products, without the rounding that out has,
                // as a mean of dp by its distances from the first seen column's, so that it is that dp, and ds
                // 0, where there is one state, or all have the same dp, whatever the rounding of p.
                const float at = tmem_ld1(t_s + 64 + (columns.x ? __ffs(columns.x) - 1 : (__ffs(columns.y) + 31) & 63));
                float total = 0.f, lean = 0.f;
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {
                    float s[32], dp[32];
                    load(q, s, dp);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float p0 = ex2_approx(fmaf(s[j], kLog2e, st.x));
                        total += p0;
                        lean = fmaf(p0, dp[j] - at, lean);
                    }
                }
                // Of a split the tile is all that the row sees where its probabilities are 1 in all: less may
                // be missing than their own error or what out's rounding would do. (Other splits' blocks
                // keep what p.stat has, whenever they read it: equal inputs, equal bits.)
                if (in && doc == d && (p.splits == 1 || total >= 1.f - 0x1p-12f - fminf(fabsf(st.x) * 0x1p-20f, 0x1p-4f))) {
                    st.y = -(at + (total == 0.f ? 0.f : lean / total));   // 0: scores of -infinity alone, ds 0 as well
                    p.stat_kv[row] = st;
                }
            }
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                float s[32], dp[32];
                load(q, s, dp);
                uint32_t pk[16], dk[16];   // p or, DQ, what the rounding of ds leaves; ds
                uint64_t nl = f2_pack(st.x, st.x), nd = f2_pack(st.y, st.y);
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float4 l4, d4;
                    if (DKV) {
                        l4 = cs[(32 * q + j) / 4];
                        d4 = cs[16 + (32 * q + j) / 4];
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (DKV) {
                            nl = i ? f2_pack(l4.z, l4.w) : f2_pack(l4.x, l4.y);
                            nd = i ? f2_pack(d4.z, d4.w) : f2_pack(d4.x, d4.y);
                        }
                        const int c = j + 2 * i;
                        float p0, p1, d0, d1;
                        f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), l2e2, nl), p0, p1);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        if (DKV) pk[c / 2] = pack_bf16x2(p0, p1);
                        f2_unpack(f2_mul(f2_pack(p0, p1), f2_add(f2_pack(dp[c], dp[c + 1]), nd)), d0, d1);
                        const uint32_t high = dk[c / 2] = pack_bf16x2(d0, d1);
                        // dq's ds in two parts: delta brings the rounding of out into it as well
                        if (!DKV) pk[c / 2] = pack_bf16x2(d0 - __uint_as_float(high << 16), d1 - __uint_as_float(high & 0xffff0000u));
                    }
                }
                tmem_st16(t_s + 16 * q, pk);
                tmem_st16(t_s + 64 + 16 * q, dk);
            }
            if (flags & kForeign) {
                // columns of other documents, whose probabilities are 0: 0 times their values must be 0
                const int c = r & 63;
                if (!((c < 32 ? columns.x : columns.y) >> (c & 31) & 1u))
                    zero_row<HD, F::YREG>(base + F::OFF_Y + sl * 2 * F::YTILE + (r < 64 ? 0 : F::YTILE), c);
                fence_proxy_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sy.bar(F::B_PFULL + a));
        }
        if (!(flags & kNone)) ++n;
    }
}

// The gradients of a pass on their way out.
template <int HD, bool DKV>
__device__ __forceinline__ void bwd_out(const BwdParams& p, const Sync& sy, uint32_t tmem, const Step* steps) {
    using F = BwdShape<HD>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16);
    const int tok = r / p.Gr, g = r - tok * p.Gr;
    constexpr int GRADS = DKV ? 2 : 1, W = HD < 32 ? HD : 32;
    uint32_t heard = 0, passes = 0;
    bool in = false, written = false;
    int doc = -1, kh = 0;
    int64_t row = 0, token = 0;   // of the workspace's rows and of the gradient's tokens
    for (;;) {
        const uint32_t e = heard % kBwdSteps;
        if (!sy.wait_warp(sy.bar(F::B_TOLD + e), (heard / kBwdSteps) & 1u)) return;
        ++heard;
        const uint32_t flags = steps[e].flags;
        const int d = steps[e].doc;
        if (flags & (kUnitFirst | kNone)) {
            in = tok < p.rpt && steps[e].t0 + tok < p.nr;
            kh = steps[e].pad;
            token = steps[e].token + tok;
            row = steps[e].row + int64_t(tok) * p.heads + g;
            doc = in && p.doc_r ? __ldg(p.doc_r + token) : 0;
            written = false;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.bar(F::B_HEARD + e));
        if (flags & kEnd) return;
        const bool last = (flags & kLast) != 0, end = (flags & kUnitLast) != 0;
        if (!last && !end) continue;
        const uint32_t buf = DKV ? 0u : passes & 1u;
        if (last && !sy.wait_warp(sy.bar(F::B_AFULL + buf), (DKV ? passes : passes >> 1) & 1u)) return;
        if (last) tc_fence_after();
        // a row of another document, or one that is written, is left; one that sees nothing gets zeros
        const bool mine = last && in && doc == d, none = end && in && !written && !mine;
#pragma unroll 1
        for (int i = 0; i < GRADS * ((HD + 31) / 32); ++i) {
            const int n = DKV ? i / ((HD + 31) / 32) : 0, q = DKV ? i % ((HD + 31) / 32) : i;
            __syncwarp();
            float o[32];
            if (last) {
                tmem_ld32(t_lane + F::AW * (DKV ? n : buf) + 32 * q, o);
                tmem_wait_ld();
                behind_wait(o);
            }
            if (!mine) {
                if (!none) continue;
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = 0.f;
            }
            if (p.splits > 1) {
                float4* const to = reinterpret_cast<float4*>(p.part + (row + n * p.rows) * HD + 32 * q);
#pragma unroll
                for (int j = 0; j < W / 4; ++j) to[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            } else {
                uint4* const to = reinterpret_cast<uint4*>(p.grad[n] + token * p.ts[n] + int64_t(kh * p.Gr + g) * HD + 32 * q);
#pragma unroll
                for (int j = 0; j < W / 8; ++j)
                    to[j] = make_uint4(pack_bf16x2(o[8 * j], o[8 * j + 1]), pack_bf16x2(o[8 * j + 2], o[8 * j + 3]),
                                       pack_bf16x2(o[8 * j + 4], o[8 * j + 5]), pack_bf16x2(o[8 * j + 6], o[8 * j + 7]));
            }
        }
        if (mine) written = true;
        if (last) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sy.bar(F::B_AREAD + buf));
            ++passes;
        }
    }
}

// Eight products in the two passes, where one pass would make five: s and dp are
// made anew, so that each sum stays in one block's tensor memory, no gradient needs
// an atomic, and equal inputs give equal bits; and dq takes ds in two bf16 parts,
// the second what the rounding of the first leaves. (Its error over that of a result
// rounded once falls from 1.5 to 1.1 at head size 16, from 1.44 to 1.15 at 128, for
// 15 us of the next figure.) Bound as the forward pass over few states is: 24576
// tokens, 16 heads of 128 over 512 states, dq 176 us, dk and dv 179 us (1.15 PFLOP/s,
// tensor cores 66 % busy).
//
// One row tile to a block, one block to an SM, persistent:
//   warps 0..3, 4..7  every second step's probabilities each;
//   warps 8..11       results on their way out;
//   warp 12           finds the column tiles that the rows see, TMA;
//   warps 13, 14      issue the scores and the products; 13 owns the tensor memory.
template <int HD, bool DKV>
__global__ void __launch_bounds__(kBwdThreads, 1)
cross_bwd_tiles(const __grid_constant__ CUtensorMap tx0, const __grid_constant__ CUtensorMap tx1, const __grid_constant__ CUtensorMap ty0,
                const __grid_constant__ CUtensorMap ty1, const __grid_constant__ BwdParams p) {
    using F = BwdShape<HD>;
    extern __shared__ __align__(1024) uint8_t base_ptr[];   // no room to align it here
    const uint32_t base = smem_u32(base_ptr);
    if (base & 1023u) {
        if (threadIdx.x == 0) atomicOr(&g_cross_timeout_flag, 1u);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile uint32_t* const misc = reinterpret_cast<volatile uint32_t*>(base_ptr + F::OFF_MISC);
    Step* const steps = reinterpret_cast<Step*>(base_ptr + F::OFF_STEP);
    const Sync sy{base + F::OFF_BAR, misc + 1};
    // rows that no load writes (G does not divide a tile's) hold zeros
    if (p.rpt * p.Gr != 128 || p.cpt * p.Gc != 64)
        for (int i = threadIdx.x; i < F::OFF_STAT / 16; i += kBwdThreads) reinterpret_cast<uint4*>(base_ptr)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (threadIdx.x == 0) {
        for (int i = 0; i < F::NBAR; ++i)
            mbar_init(sy.bar(i), (i >= F::B_PFULL && i < F::B_PFULL + 2) || (i >= F::B_AREAD && i < F::B_AREAD + 2) ? 4u
                                 : i >= F::B_HEARD && i < F::B_HEARD + kBwdSteps ? 12u : 1u);
        misc[1] = 0u;
        misc[2] = beat_clock() - kWaitTicks - 1u;   // long ago
        fence_mbar_init();
    }
    if (warp == 12 && lane == 0) {
        tma_prefetch_desc(&tx0);
        tma_prefetch_desc(&tx1);
        tma_prefetch_desc(&ty0);
        tma_prefetch_desc(&ty1);
    }
    if (warp == 13) {
        tmem_alloc(base + F::OFF_MISC, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    dependents_may_start();
    wait_for_primary();   // the statistics
    if (warp < 8) {
        regs_increase<kBwdSoftmax>();
        bwd_softmax<HD, DKV>(p, sy, base, base_ptr, tmem, steps);
    } else if (warp < 12) {
        regs_decrease<kBwdOut>();
        bwd_out<HD, DKV>(p, sy, tmem, steps);
    } else {
        regs_decrease<kBwdLow>();
        if (warp == 12) bwd_producer<HD, DKV>(p, sy, base, base_ptr, steps, misc + 3, &tx0, &tx1, &ty0, &ty1);
        if (warp == 13) bwd_scores<HD>(sy, base, __reduce_or_sync(kAll, tmem), misc + 3);
        if (warp == 14) bwd_products<HD, DKV>(sy, base, __reduce_or_sync(kAll, tmem), misc + 3);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The splits of a gradient summed in order, bound by their read (7 splits of dk and
// dv of 512 states, 16 heads of 128: 59 MB in 14 us). grads: 1 (dq) or 2 (dv, dk).
template <int HD>
__global__ void __launch_bounds__(256) cross_sum(const BwdParams p, int grads) {
    constexpr int PER = HD / 4;
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x, row = i / PER;
    const int c = int(i % PER) * 4, n = blockIdx.y;
    dependents_may_start();
    wait_for_primary();
    if (row >= p.rows) return;
    float o[4] = {};
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        const float4 v = *reinterpret_cast<const float4*>(p.part + ((int64_t(s) * grads + n) * p.rows + row) * HD + c);
        o[0] += v.x;
        o[1] += v.y;
        o[2] += v.z;
        o[3] += v.w;
    }
    const int64_t token = row / p.heads;
    uint16_t* const to = p.grad[n] + token * p.ts[n] + (row - token * p.heads) * HD + c;
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
}

// ------------------------------------------------------------------ host side

// A tensor of heads (B, n, heads, HD), ts elements from token to token: boxes of
// `tokens` tokens with `box_heads` heads, HDB columns.
bool encode_heads(CUtensorMap* m, const void* ptr, int HD, int64_t B, int64_t n, int64_t heads, int64_t ts, int box_heads, int tokens) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int hdb = HD < 64 ? HD : 64;
    const cuuint64_t dims[4] = {cuuint64_t(HD), cuuint64_t(heads), cuuint64_t(n), cuuint64_t(B)};
    const cuuint64_t strides[3] = {cuuint64_t(HD) * 2, cuuint64_t(ts) * 2, cuuint64_t(ts) * 2 * n};
    const cuuint32_t box[4] = {cuuint32_t(hdb), cuuint32_t(box_heads), cuuint32_t(tokens), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle swz = hdb == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                   : hdb == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                               : CU_TENSOR_MAP_SWIZZLE_32B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSms = 152;   // what the work is shared out for: equal on every device

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Each of the two copies of the statistics of the backward pass; the splits' sums lie behind them.
int64_t stat_bytes(int64_t B, int64_t L, int64_t NH) { return (B * L * NH * 8 + 127) / 128 * 128; }

struct FwdPlan {
    int64_t rpt, pairs, tiles, splits, per_split;
    FwdPlan(int64_t B, int64_t L, int64_t S, int64_t NH, int64_t NKV) {
        rpt = 128 / (NH / NKV);
        pairs = ceil_div(L, 2 * rpt);
        tiles = ceil_div(S, 128);
        // few rows: the states shared out too, four column tiles to a split at least
        const int64_t units = B * NKV * pairs;
        splits = units * 2 > kSms ? 1 : kSms / units;
        if (splits > tiles / 4) splits = tiles / 4;
        if (splits < 1) splits = 1;
        per_split = ceil_div(tiles, splits);
        splits = ceil_div(tiles, per_split);
    }
};

template <typename... Args>
cudaError_t launch_after(void (*kernel)(Args...), int64_t grid, int threads, int smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = dim3(unsigned(grid));
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

template <int HD>
cudaError_t fwd(const CrossParams& c, int sms, cudaStream_t stream) {
    const FwdPlan pl(c.B, c.L, c.S, c.NH, c.NKV);
    const int64_t units = int64_t(c.B) * c.NKV * pl.pairs * pl.splits;
    if (units >= (int64_t(1) << 31) - sms) return cudaErrorInvalidValue;
    FwdParams p{};
    p.B = c.B; p.L = c.L; p.S = c.S; p.NH = c.NH; p.NKV = c.NKV;
    p.G = c.NH / c.NKV;
    p.rpt = int(pl.rpt);
    p.pairs = int(pl.pairs);
    p.units = int(units);
    p.tiles = int(pl.tiles);
    p.splits = int(pl.splits);
    p.per_split = int(pl.per_split);
    p.lone = c.L <= pl.rpt && pl.per_split > 1;
    p.rows = int64_t(c.B) * c.L * c.NH;
    p.out_v8 = reinterpret_cast<uintptr_t>(c.out) % 32 == 0;
    p.doc = c.doc;
    p.kv_doc = c.kv_doc;
    p.out = c.out;
    p.lse = c.lse;
    p.part = static_cast<float*>(c.work);
    p.part_lse = p.part + pl.splits * p.rows * HD;
    CUtensorMap tq, tk, tv;
    if (!encode_heads(&tq, c.q, HD, c.B, c.L, c.NH, c.q_ts, p.G, p.rpt - c.withhold) || !encode_heads(&tk, c.k, HD, c.B, c.S, c.NKV, c.k_ts, 1, 128) ||
        !encode_heads(&tv, c.v, HD, c.B, c.S, c.NKV, c.v_ts, 1, 128))
        return cudaErrorInvalidValue;
    const auto kernel = p.lone || p.splits > 1 ? cross_fwd_tiles<HD, kFew> : p.doc || p.kv_doc ? cross_fwd_tiles<HD, kDocuments> : cross_fwd_tiles<HD, kPlain>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FwdShape<HD>::SMEM);
    if (e != cudaSuccess) return e;
    kernel<<<unsigned(units < sms ? units : sms), kFwdThreads, FwdShape<HD>::SMEM, stream>>>(tq, tk, tv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    int parts = 1;   // four splits to a group of threads, as far as a block's go
    while (parts < 256 / (HD / 4) && parts * 4 < p.splits) parts *= 2;
    return launch_after(cross_join<HD>, ceil_div(p.rows * (HD / 4) * parts, 256), 256, 0, stream, p, parts);
}

// How a backward pass is shared out: `units` row tiles over `tiles` column tiles each, in so
// many splits that the blocks' rounds hold the least of column tiles.
struct BwdPlan {
    int64_t rpt, cpt, tiles_r, tiles_c, splits, per_split, rows, grads;
    BwdPlan(bool dkv, int64_t B, int64_t L, int64_t S, int64_t NH, int64_t NKV) {
        const int64_t G = NH / NKV;
        rpt = dkv ? 128 : 128 / G;
        cpt = dkv ? 64 / G : 64;
        tiles_r = ceil_div(dkv ? S : L, rpt);
        tiles_c = ceil_div(dkv ? L : S, cpt);
        rows = dkv ? B * S * NKV : B * L * NH;
        grads = dkv ? 2 : 1;
        const int64_t units = B * NKV * tiles_r;
        splits = 1;
        // a unit's beginning and end cost some four column tiles, a split's sums their memory
        int64_t best = ceil_div(units, kSms) * (tiles_c + 4);
        for (int64_t s = 2; s <= 64 && units < 4 * kSms && tiles_c / s >= 4; ++s) {
            const int64_t cost = ceil_div(units * s, kSms) * (ceil_div(tiles_c, s) + 6);
            if (cost < best - best / 16) {
                best = cost;
                splits = s;
            }
        }
        per_split = ceil_div(tiles_c, splits);
        splits = ceil_div(tiles_c, per_split);
    }
    int64_t part_bytes(int64_t HD) const { return splits > 1 ? splits * grads * rows * HD * 4 : 0; }
};

template <int HD, bool DKV>
cudaError_t bwd_pass(const CrossParams& c, int sms, cudaStream_t stream) {
    const BwdPlan pl(DKV, c.B, c.L, c.S, c.NH, c.NKV);
    const int64_t units = int64_t(c.B) * c.NKV * pl.tiles_r * pl.splits;
    if (units >= (int64_t(1) << 31) - sms) return cudaErrorInvalidValue;
    BwdParams p{};
    p.B = c.B; p.NH = c.NH; p.NKV = c.NKV; p.G = c.NH / c.NKV;
    p.nr = DKV ? c.S : c.L;
    p.nc = DKV ? c.L : c.S;
    p.rpt = int(pl.rpt);
    p.cpt = int(pl.cpt);
    p.Gr = DKV ? 1 : p.G;
    p.Gc = DKV ? p.G : 1;
    p.heads = DKV ? c.NKV : c.NH;
    p.tiles_r = int(pl.tiles_r);
    p.tiles_c = int(pl.tiles_c);
    p.splits = int(pl.splits);
    p.per_split = int(pl.per_split);
    p.units = int(units);
    p.doc_r = DKV ? c.kv_doc : c.doc;
    p.doc_c = DKV ? c.doc : c.kv_doc;
    p.out = c.out;
    p.dout = c.dout;
    p.lse = c.lse;
    uint8_t* const work = static_cast<uint8_t*>(c.work);
    p.stat = reinterpret_cast<float2*>(work);
    p.stat_kv = reinterpret_cast<float2*>(work + stat_bytes(c.B, c.L, c.NH));
    p.rows = pl.rows;
    p.part = reinterpret_cast<float*>(work + 2 * stat_bytes(c.B, c.L, c.NH));
    p.grad[0] = DKV ? c.dv : c.dq;
    p.grad[1] = c.dk;
    p.ts[0] = DKV ? c.dv_ts : c.dq_ts;
    p.ts[1] = c.dk_ts;
    if (!DKV) {   // the first of the two passes: the statistics before it
        const int64_t rows = int64_t(c.B) * c.L * c.NH, blocks = ceil_div(rows * (HD / 8), 256 * kStatLoads);
        if (blocks >= int64_t(1) << 31) return cudaErrorInvalidValue;
        cross_stat<HD><<<unsigned(blocks), 256, 0, stream>>>(p, rows);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const int64_t row = int64_t(c.NH) * HD;
    CUtensorMap q, d, k, v;
    const int qt = DKV ? p.cpt : p.rpt - c.withhold, kt = DKV ? p.rpt - c.withhold : p.cpt;
    if (!encode_heads(&q, c.q, HD, c.B, c.L, c.NH, c.q_ts, p.G, qt) || !encode_heads(&d, c.dout, HD, c.B, c.L, c.NH, row, p.G, qt) ||
        !encode_heads(&k, c.k, HD, c.B, c.S, c.NKV, c.k_ts, 1, kt) || !encode_heads(&v, c.v, HD, c.B, c.S, c.NKV, c.v_ts, 1, kt))
        return cudaErrorInvalidValue;
    constexpr int smem = BwdShape<HD>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(cross_bwd_tiles<HD, DKV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = units < sms ? units : sms;
    e = DKV ? launch_after(cross_bwd_tiles<HD, DKV>, grid, kBwdThreads, smem, stream, k, v, q, d, p)
            : launch_after(cross_bwd_tiles<HD, DKV>, grid, kBwdThreads, smem, stream, q, d, k, v, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(unsigned(ceil_div(pl.rows * (HD / 4), 256)), unsigned(pl.grads));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cross_sum<HD>, p, int(pl.grads));
}

template <int HD>
cudaError_t bwd(const CrossParams& c, int sms, cudaStream_t stream) {
    const cudaError_t e = bwd_pass<HD, false>(c, sms, stream);
    return e != cudaSuccess ? e : bwd_pass<HD, true>(c, sms, stream);
}

}  // namespace

static std::atomic<bool> g_launched{false};

int64_t cross_workspace(int64_t B, int64_t L, int64_t S, int64_t NH, int64_t NKV, int64_t HD, bool backward) {
    const int64_t rows = B * L * NH;
    if (backward) {
        const int64_t a = BwdPlan(false, B, L, S, NH, NKV).part_bytes(HD), b = BwdPlan(true, B, L, S, NH, NKV).part_bytes(HD);
        return 2 * stat_bytes(B, L, NH) + (a > b ? a : b);
    }
    const FwdPlan pl(B, L, S, NH, NKV);
    return pl.splits > 1 ? pl.splits * rows * (HD + 1) * 4 : 0;
}

cudaError_t launch_cross_fwd(int hd, const CrossParams& p, int sms, cudaStream_t stream) {
    g_launched = true;
    switch (hd) {
        case 16: return fwd<16>(p, sms, stream);
        case 32: return fwd<32>(p, sms, stream);
        case 64: return fwd<64>(p, sms, stream);
        case 128: return fwd<128>(p, sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_cross_bwd(int hd, const CrossParams& p, int sms, cudaStream_t stream) {
    g_launched = true;
    switch (hd) {
        case 16: return bwd<16>(p, sms, stream);
        case 32: return bwd<32>(p, sms, stream);
        case 64: return bwd<64>(p, sms, stream);
        case 128: return bwd<128>(p, sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

// The flag is taken as for the attention kernel: one atomic exchange per
// status request, its old value left in a slot of that request's own. A process
// that has launched none of these kernels has nothing to ask for.
constexpr unsigned int kStatusSlots = 256;
__device__ unsigned int g_cross_status_slots[kStatusSlots];

__global__ void take_cross_flag(unsigned int slot) { g_cross_status_slots[slot] = atomicExch(&g_cross_timeout_flag, 0u); }

cudaError_t take_cross_error(cudaStream_t stream, unsigned int* flag) {
    *flag = 0;
    if (!g_launched) return cudaSuccess;
    static std::atomic<unsigned int> next{0};
    const unsigned int slot = next.fetch_add(1u) % kStatusSlots;
    take_cross_flag<<<1, 1, 0, stream>>>(slot);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbolAsync(flag, g_cross_status_slots, sizeof(unsigned int), slot * sizeof(unsigned int),
                                  cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(stream);
}

}  // namespace na3d
