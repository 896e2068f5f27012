// How the score-shaped attention cuts a problem: rows, bricks, chunks and their
// walk. Host and device read the same functions; nothing here needs a GPU.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "na3d_kernel.cuh"
#include "na3d_scored.cuh"

namespace na3d {
namespace scored {

__host__ __device__ __forceinline__ int win_start(int i, int K, int N) {
    const int s = i - K / 2 < N - K ? i - K / 2 : N - K;
    return s > 0 ? s : 0;
}

// The queries whose windows hold position j of an axis: [first, last].
__host__ __device__ __forceinline__ int inv_first(int j, int K) { return j < K ? 0 : j - K / 2; }
__host__ __device__ __forceinline__ int inv_last(int j, int K, int N) { return j >= N - K ? N - 1 : j + K / 2; }

enum { kFwd, kDq, kDkv };

// Blocks an SM holds, and the most warps of a block: as many rows in flight as
// the registers of an instance allow (accumulators, fixed fragments and about
// 60 more a thread).
__host__ __device__ constexpr int blocks_per_sm(int hd, int mode) { return hd <= 32 && mode == kFwd ? 2 : 1; }
__host__ __device__ constexpr int max_warps(int hd, int mode) {
    return blocks_per_sm(hd, mode) == 2 || hd > 32 ? 8 : 12;
}
// Buffers of the fixed tensors: two where a step reads them again (their
// fragments and the accumulators together exceed the registers).
__host__ __device__ constexpr int fixed_buffers(int hd, int mode) { return hd > 64 && mode == kDkv ? 2 : 1; }

constexpr int kMaxStages = 6, kMaxRing = kMaxStages + 2;   // ring places: stages and fixed buffers
constexpr int kControl = 8 + 8 * kMaxRing;                     // bytes of the control words

// The positions that row i of an axis of length N meets: keys of its window
// (FWD, DQ), or the queries whose windows hold it (DKV). Both ends grow with i.
__host__ __device__ __forceinline__ int range_lo(bool dkv, int i, int K, int N) {
    return dkv ? inv_first(i, K) : win_start(i, K, N);
}
__host__ __device__ __forceinline__ int range_hi(bool dkv, int i, int K, int N) {   // exclusive
    return dkv ? inv_last(i, K, N) + 1 : win_start(i, K, N) + K;
}

// From so many keys on capped scores take the plain steps, with a table. Forward these have no running
// maximum: a row of one key has out off by the rounding of its probability, which would be 1. Their
// cap, the backward passes' too, is exact to 2^-21 of the cap, and so is lse, which is near the scores:
// at unit scores and a cap of 50 lse is 2.7e-6 of its norm off over one key, 1.2e-6 over three and
// 7e-7 over five. (1,16,64,64,8,64) with windows of (1,1,1), (1,1,3) and (3,1,1) takes 75, 85 and 133 us
// so and 87, 108 and 168 in the general steps, its gradients 216, 241 and 380 and 235, 280 and 437.
constexpr int kManyKeys = 5;

// Geometry of one launch. A block's brick is st x (nw * sh) x sw rows, warp w
// the sh grid rows from w * sh; its columns stream in chunks of one frame,
// cr grid rows and cc columns. sw <= 8, so that rows r and r + 8 of a warp, a
// thread's two, lie in one column of the grid.
struct TileGeom {
    int32_t st, sh, sw, nw, bh;   // st, sh and sw: powers of two
    int32_t sw_log2;
    int32_t nbt, nbh, nbw;
    int32_t cr, cc;
    int32_t nt, nhc, nwc;      // chunks of a unit: frames, and parts along H and W
    int32_t stages;
    int32_t lut;               // 1: a frame's biases and (h, w) windows come from a table of each warp,
                               // 0: its windows from mask words
    int32_t lut_pitch;         // floats of a table row (one for each (h, w) of the warp's rows)
    int32_t frame_steps;       // steps of 16 columns that a warp's box takes in a frame, at most,
    int32_t chunk_steps;       // and in a chunk
    int32_t units, bricks;     // (head, brick) pairs, brick fastest
    // shared memory, bytes from a 1024-byte boundary
    int32_t x_bytes;           // one streamed tensor of a stage (regions of 64 columns)
    int32_t off_x, off_stat, off_doc, off_lut, off_hw, off_bar, smem;
    FastDiv div_bricks, div_nbw, div_nbh, div_nbt;
};

__host__ __device__ __forceinline__ int fast_div(const FastDiv& d, int n) {
    return int((uint64_t(uint32_t(n)) * d.mul) >> d.shift);
}

struct Brick {
    int b, t0, h0, w0;   // first row
};

// Bricks run along T first: neighbours there share their rows' places in the
// grid's (h, w) plane, and most of their frames.
__host__ __device__ __forceinline__ Brick brick_of(const TileGeom& g, int n) {
    Brick o;
    int q = fast_div(g.div_nbt, n);
    o.t0 = (n - q * g.nbt) * g.st; n = q;
    q = fast_div(g.div_nbw, n);
    o.w0 = (n - q * g.nbw) * g.sw; n = q;
    o.b = fast_div(g.div_nbh, n);
    o.h0 = (n - o.b * g.nbh) * g.bh;
    return o;
}

// Union of the ranges of n rows from i (rows past the axis end count as the last).
__host__ __device__ __forceinline__ int2 box_of(bool dkv, int i, int n, int K, int N) {
    const int first = i < N ? i : N - 1, last = i + n <= N ? i + n - 1 : N - 1;
    return make_int2(range_lo(dkv, first, K, N), range_hi(dkv, last, K, N));
}

// The (head, brick) of a unit and the box that its chunks cover.
struct Unit {
    Brick o;
    int head;
    int2 bt, bh, bw;
};

template <bool DKV>
__host__ __device__ __forceinline__ Unit unit_of(const ScoredParams& p, const TileGeom& g, int u) {
    Unit x;
    x.head = fast_div(g.div_bricks, u);
    x.o = brick_of(g, u - x.head * g.bricks);
    x.bt = box_of(DKV, x.o.t0, g.st, p.KT, p.T);
    x.bh = box_of(DKV, x.o.h0, g.bh, p.KH, p.H);
    x.bw = box_of(DKV, x.o.w0, g.sw, p.KW, p.W);
    return x;
}

// The unit after x.
template <bool DKV>
__host__ __device__ __forceinline__ void next_unit(const ScoredParams& p, const TileGeom& g, Unit& x) {
    x.o.t0 += g.st;
    if (x.o.t0 >= p.T) {
        x.o.t0 = 0;
        x.o.w0 += g.sw;
        if (x.o.w0 >= p.W) {
            x.o.w0 = 0;
            x.o.h0 += g.bh;
            if (x.o.h0 >= p.H) {
                x.o.h0 = 0;
                if (++x.o.b == p.B) {
                    x.o.b = 0;
                    ++x.head;
                }
            }
            x.bh = box_of(DKV, x.o.h0, g.bh, p.KH, p.H);
        }
        x.bw = box_of(DKV, x.o.w0, g.sw, p.KW, p.W);
    }
    x.bt = box_of(DKV, x.o.t0, g.st, p.KT, p.T);
}

// The grid rows that warp `warp` of a unit's block meets; none where its own lie past the grid.
template <bool DKV>
__host__ __device__ __forceinline__ int2 warp_rows(const ScoredParams& p, const TileGeom& g, const Unit& x, int warp) {
    const int h = x.o.h0 + warp * g.sh;
    return h < p.H ? box_of(DKV, h, g.sh, p.KH, p.H) : make_int2(0, 0);
}

// A warp's part of a chunk: n columns (none where n <= 0) from (hf, w) in rows of g.cc.
struct Part {
    int hf, w, n;
};

// ... of chunk (ih, iw) of a frame, for a warp that meets the grid rows `mine`.
__host__ __device__ __forceinline__ Part part_of(const TileGeom& g, const Unit& x, int2 mine, int ih, int iw) {
    const int h = x.bh.x + ih * g.cr;
    Part o;
    o.w = x.bw.x + iw * g.cc;
    o.hf = mine.x > h ? mine.x : h;
    o.n = o.w < x.bw.y ? ((mine.y < h + g.cr ? mine.y : h + g.cr) - o.hf) * g.cc : 0;
    return o;
}

// Does a unit's frame t have columns? Every unit walks g.nt frames, and the box of one at the end
// of the axis is shorter: the frames behind it bring nothing and may lie past the grid.
__host__ __device__ __forceinline__ bool has_frame(const Unit& x, int t) { return t < x.bt.y; }

// Largest union of the ranges of `step` consecutive rows that start at a
// multiple of step: inside an axis K + step - 1; a key near a border is held
// by up to K + K/2 queries' windows, most in the rows around K and N - K.
inline int widest(bool dkv, int step, int K, int N) {
    const int inner = K <= N - step ? K + step - 1 : N;
    if (!dkv) return inner;
    int best = inner;
    const int at[2] = {(K - 1) / step * step, (N - K) / step * step};
    for (const int i : at) {
        const int last = i < N - step ? i + step - 1 : N - 1;
        const int e = range_hi(true, last, K, N) - range_lo(true, i, K, N);
        if (e > best) best = e;
    }
    return best;
}

inline int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

constexpr int kSmemMax = 227 * 1024;

// Shared memory of a geometry with `stages` stages and chunks of cr x cc; false where it is more
// than `room`. The sizes are summed in 64 bits: a large window's masks alone pass 2^31 bytes.
inline bool lay_out(TileGeom* g, int hd, int mode, bool docs, int64_t frame_steps, int room) {
    const bool dkv = mode == kDkv;
    const int64_t nf = (mode == kFwd ? 1 : 2) * fixed_buffers(hd, mode), nw = g->nw, columns = int64_t(g->cr) * g->cc + 16;
    const int64_t chunk = nw * g->chunk_steps * 16;
    const int64_t hdb = hd > 64 ? 64 : hd, reg = hd > 64 ? hd / 64 : 1;
    const int64_t f_region = align_up(int64_t(g->st) * g->bh * g->sw * hdb * 2, 1024);
    const int64_t x_bytes = align_up(columns * hdb * 2, 1024) * reg;
    const int64_t off_x = f_region * reg * nf;
    const int64_t off_stat = off_x + 2 * g->stages * x_bytes;
    const int64_t off_doc = off_stat + (dkv ? chunk * 8 : 0);
    const int64_t off_lut = off_doc + (docs ? chunk * 4 : 0);
    const int64_t pitch = frame_steps * 16 + 8;
    const int64_t off_hw = align_up(off_lut + nw * (g->lut ? g->sh * g->sw * pitch * 4 : frame_steps * 32), 16);
    const int64_t off_bar = align_up(off_hw + columns * 8, 16);
    const int64_t smem = off_bar + kControl + 8 * kMaxRing + 1024;
    if (smem > room) return false;
    g->frame_steps = int32_t(frame_steps);
    g->lut_pitch = int32_t(pitch);
    g->x_bytes = int32_t(x_bytes);
    g->off_x = int32_t(off_x);
    g->off_stat = int32_t(off_stat);
    g->off_doc = int32_t(off_doc);
    g->off_lut = int32_t(off_lut);
    g->off_hw = int32_t(off_hw);
    g->off_bar = int32_t(off_bar);
    g->smem = int32_t(smem);
    return true;
}

// Chooses rows, brick and chunks for the least modelled time; false where none holds the problem:
// the masks of a frame's window, 2 bytes a key, want room for one warp's at least.
inline bool plan_tiles(TileGeom* best, const ScoredParams& p, int hd, int mode, int sms) {
    const bool dkv = mode == kDkv, docs = p.doc != nullptr;
    const int blocks = blocks_per_sm(hd, mode), room = kSmemMax / blocks - 1024;
    // positions and bricks past an axis' end are still numbers, frames' distances exact in fp32
    constexpr int most = INT32_MAX - 4096;
    if (p.T > most || p.H > most || p.W > most || p.KT > (1 << 23) || int64_t(p.KH) * p.KW * 2 > kSmemMax) return false;
    const bool few = p.softcap > 0.f && int64_t(p.KT) * p.KH * p.KW < kManyKeys;
    double best_cost = 0;
    bool found = false;
    for (int st = 1; st <= 16; st *= 2)
        for (int sh = 1; st * sh <= 16; sh *= 2) {
            const int sw = 16 / (st * sh);
            if (sw > 8) continue;
            const int et = widest(dkv, st, p.KT, p.T), ew = widest(dkv, sw, p.KW, p.W);
            const int eh_w = widest(dkv, sh, p.KH, p.H);
            for (int nw = 1; nw <= max_warps(hd, mode); ++nw) {
                if ((nw - 1) * sh >= p.H) break;
                TileGeom g{};
                g.st = st; g.sh = sh; g.sw = sw; g.nw = nw;
                g.sw_log2 = sw == 8 ? 3 : sw == 4 ? 2 : sw == 2 ? 1 : 0; g.bh = nw * sh;
                if (g.bh > 256) continue;
                g.nbt = (p.T + st - 1) / st;
                g.nbh = (p.H + g.bh - 1) / g.bh;
                g.nbw = (p.W + sw - 1) / sw;
                // (at most 2^34 rows, a unit for each at worst)
                const int64_t units = int64_t(p.B) * g.nbt * g.nbh * g.nbw * p.NH;
                if (units >= (int64_t(1) << 31)) continue;
                g.units = int32_t(units);
                g.bricks = g.units / p.NH;
                const int eh = widest(dkv, g.bh, p.KH, p.H);
                // chunks: whole rows of the box, as many as leave room for two
                // stages; narrower ones where a single row does not
                g.nwc = (ew + 255) / 256;
                if (int64_t(eh_w) * ew * 2 > room) continue;
                for (int parts = (eh + 255) / 256;; ++parts) {
                    if (parts > eh) break;
                    g.cc = (ew + g.nwc - 1) / g.nwc;
                    g.cr = (eh + parts - 1) / parts;
                    const int nhc = (eh + g.cr - 1) / g.cr;
                    g.nt = et;
                    g.nhc = nhc;
                    // steps of a warp: its box in each chunk that it meets, rounded up to 16
                    const int met = (eh_w + g.cr - 2) / g.cr + 1 < nhc ? (eh_w + g.cr - 2) / g.cr + 1 : nhc;
                    const int64_t frame = int64_t(g.nwc) * ((int64_t(eh_w) * g.cc + 15) / 16 + met - 1);
                    // the table of a frame (its pitch puts the rows of four lanes in different
                    // banks), or mask words where it does not fit
                    const int64_t chunks = int64_t(et) * nhc * g.nwc;
                    g.chunk_steps = ((eh_w < g.cr ? eh_w : g.cr) * g.cc + 15) / 16;
                    g.stages = chunks < 2 ? 1 : 2;
                    g.lut = few ? 0 : 1;
                    if (few || !lay_out(&g, hd, mode, docs, frame, room)) {
                        g.lut = 0;
                        if (!lay_out(&g, hd, mode, docs, frame, room)) {
                            if (g.cr > 1) {   // on to the next smaller cr
                                parts = (eh + g.cr - 2) / (g.cr - 1) - 1;
                                continue;
                            }
                            if (found || g.cc == 1) break;
                            g.nwc *= 2;
                            parts = (eh + 255) / 256 - 1;
                            continue;
                        }
                    }
                    while (g.stages < kMaxStages && g.stages < chunks) {
                        TileGeom more = g;
                        ++more.stages;
                        if (!lay_out(&more, hd, mode, docs, frame, room)) break;
                        g = more;
                    }
                    // cycles: a step issues about 140 instructions (more without the table) on
                    // four schedulers that find one ready in two cycles of three; a frame's
                    // load takes its latency and 60 bytes a cycle, and hides behind the
                    // computation, all of it where two frames fit
                    const double instr = (mode == kFwd ? 140.0 : 190.0) * (hd + 64) / 128 * (g.lut ? 1.0 : 1.4);
                    const double work = double(frame) * nw * blocks * instr / 2.6;
                    const double lat = double(frame) * instr * 2.5;
                    const double comp = work > lat ? work : lat;
                    const double load = 1000.0 + double(g.nwc) * nhc * g.cr * g.cc * hd * 4 * blocks / 60.0;
                    const bool deep = g.stages >= 2 * g.nwc * nhc;
                    const double more = comp > load ? comp : load, less = comp + load - more;
                    const double frame_t = more + (deep ? 0.0 : 0.3 * less);
                    const double unit = et * (frame_t + 0.1 * (comp + load)) + 3000.0;
                    const double slots = double(sms) * blocks;
                    const double waves = g.units <= slots ? 1.0 : double(g.units) / slots;
                    const double cost = waves * unit;
                    if (!found || cost < best_cost) {
                        found = true;
                        best_cost = cost;
                        *best = g;
                    }
                    if (g.cr == 1 || parts >= 12) break;
                }
            }
        }
    if (found) {
        best->div_bricks = make_fastdiv(best->bricks);
        best->div_nbw = make_fastdiv(best->nbw);
        best->div_nbh = make_fastdiv(best->nbh);
        best->div_nbt = make_fastdiv(best->nbt);
    }
    return found;
}

}  // namespace scored
}  // namespace na3d
