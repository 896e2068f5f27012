// Neighbourhood attention with shaped scores, forward and backward.
//
// For query i and key j of its window (the window rule of na3d_fwd):
//   a = q_i . k_j                                  (q arrives scaled)
//   b = c tanh(a / c) for a cap c > 0, else a
//   s = b - sum_axis slope[head][axis] |i_axis - j_axis|
// j is masked where doc_i != doc_j or doc_i < 0, and, with a prefix length
// P of the batch entry, where t_j > t_i and t_j >= P.
//   lse_i = log sum_j e^s,  p = e^(s - lse),  out_i = sum_j p v_j;
// a row that sees no key has out 0 and lse -inf.
// Backward, with dp = dout_i . v_j and delta_i = dout_i . out_i:
//   ds = p (dp - delta_i),  da = ds (1 - tanh(a / c)^2)
//   dq_i = sum_j da k_j,  dk_j = sum_i da q_i,  dv_j = sum_i p dout_i.
//
// The tile kernel (scored_tiles) computes all three passes. One warp holds 16
// rows, a small box of the grid, and streams the union of their windows in
// steps of 16 keys through mma.sync. Warps of 16 rows were taken for the few
// scores that no row wants: 320 keys a row against 784 of a 128-row tcgen05
// tile of 2 x 8 x 8, for a (3,7,7) window of 147. A capped score costs three
// special-function operations, so that 784 of them would be bound by those
// near 250 us at (1,16,64,64,8,64), where this takes 260. For scores without a
// cap the count is no reason: na3d_fwd's 128-row tiles take 65 us for each
// (8,64,33,8,64) entry with a (3,7,33) window, where this takes 222 with a bias
// and documents. What bounds this kernel is latency (see scored_tiles).
//
// The row functions compute one row of one head by one warp, its lanes
// splitting the head dim, and skip masked keys, so what those hold never
// reaches the row. They serve the rows of the tile kernel that met a value
// that is not finite: 0 times infinity is not 0 in a tile's products.
#include <atomic>
#include <cstring>
#include <type_traits>
#include <cuda_bf16.h>

#include "na3d_host.cuh"
#include "na3d_kernel.cuh"
#include "na3d_scored.cuh"
#include "na3d_scored_plan.cuh"
#include "sm103_ptx.cuh"

namespace na3d {

__device__ unsigned int g_scored_timeout_flag = 0;

namespace {

using namespace scored;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// HD values of one head spread over a warp: E per lane (lanes past HD hold 0).
template <int HD>
struct Row {
    static constexpr int E = HD >= 32 ? HD / 32 : 1;
    float x[E];
    __device__ __forceinline__ void load(const uint16_t* p, int lane) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = lane * E + e;
            x[e] = c < HD ? __uint_as_float(uint32_t(p[c]) << 16) : 0.f;
        }
    }
    __device__ __forceinline__ void store(uint16_t* p, int lane) const {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = lane * E + e;
            if (c < HD) p[c] = __bfloat16_as_ushort(__float2bfloat16_rn(x[e]));
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
    }
    __device__ __forceinline__ float dot(const Row& o) const {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(x[e], o.x[e], s);
        return warp_sum(s);
    }
    __device__ __forceinline__ void axpy(float a, const Row& o) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = fmaf(a, o.x[e], x[e]);
    }
};

struct Pos {
    int b, t, h, w, head;
    int64_t token;
};

__device__ __forceinline__ int64_t token_of(const ScoredParams& p, int b, int t, int h, int w) {
    return ((int64_t(b) * p.T + t) * p.H + h) * p.W + w;
}

// Place of a token's statistics: one head's are together, along the grid.
__device__ __forceinline__ int64_t stat_at(const ScoredParams& p, int b, int64_t token, int head) {
    return token + (int64_t(b) * (p.NH - 1) + head) * (int64_t(p.T) * p.H * p.W);
}

// May the query in document `qdoc` at frame qt see the key at frame kt?
__device__ __forceinline__ bool visible(const ScoredParams& p, int qdoc, int kdoc, int qt, int kt, int prefix) {
    if (p.doc && (qdoc != kdoc || qdoc < 0)) return false;
    return !p.prefix || kt <= qt || kt < prefix;
}

// The shaped score of a, and d score / d a.
__device__ __forceinline__ float shape_score(const ScoredParams& p, float a, const float* slope, int dt,
                                             int dh, int dw, float* slope_a) {
    *slope_a = 1.f;
    if (p.softcap > 0.f) {
        const float th = tanhf(a / p.softcap);
        a = p.softcap * th;
        *slope_a = 1.f - th * th;
    }
    if (p.slopes) a -= slope[0] * float(abs(dt)) + slope[1] * float(abs(dh)) + slope[2] * float(abs(dw));
    return a;
}

__device__ __forceinline__ void load_slopes(const ScoredParams& p, int head, float* s) {
#pragma unroll
    for (int a = 0; a < 3; ++a) s[a] = p.slopes ? p.slopes[head * 3 + a] : 0.f;
}

// About a millisecond a tick.
__device__ __forceinline__ uint32_t beat_clock() { return uint32_t(globaltimer_ns() >> 20); }

// A warp on a row by itself keeps the others of its block from their next
// stages, for longer than their waits allow where the window is large: once a
// line of the window it leaves the time, the block's beat, and they wait on.
__device__ __forceinline__ void still_going(volatile uint32_t* beat, int lane) {
    if (lane == 0) *beat = beat_clock();
}

// Forward row: a running maximum m, the sum l of e^(s - m) and the weighted
// sum of v, rescaled when m grows.
template <int HD>
__device__ void row_fwd(const ScoredParams& p, const Pos& o, int lane, volatile uint32_t* beat) {
    Row<HD> q, acc, x;
    q.load(p.q + o.token * p.q_ts + int64_t(o.head) * HD, lane);
    acc.zero();
    float slope[3], m = -INFINITY, l = 0.f, unused;
    load_slopes(p, o.head, slope);
    const int qdoc = p.doc ? p.doc[o.token] : 0, prefix = p.prefix ? p.prefix[o.b] : 0;
    const int t0 = win_start(o.t, p.KT, p.T), h0 = win_start(o.h, p.KH, p.H), w0 = win_start(o.w, p.KW, p.W);
    for (int t = t0; t < t0 + p.KT; ++t)
        for (int h = h0; h < h0 + p.KH; ++h) {
            still_going(beat, lane);
            for (int w = w0; w < w0 + p.KW; ++w) {
                const int64_t tok = token_of(p, o.b, t, h, w);
                if (!visible(p, qdoc, p.doc ? p.doc[tok] : 0, o.t, t, prefix)) continue;
                x.load(p.k + tok * p.k_ts + int64_t(o.head) * HD, lane);
                const float s = shape_score(p, q.dot(x), slope, o.t - t, o.h - h, o.w - w, &unused);
                if (s == -INFINITY) continue;
                const float mn = fmaxf(m, s);
                const float r = m == -INFINITY ? 0.f : expf(m - mn), e = expf(s - mn);
                x.load(p.v + tok * p.v_ts + int64_t(o.head) * HD, lane);
#pragma unroll
                for (int i = 0; i < Row<HD>::E; ++i) acc.x[i] = fmaf(e, x.x[i], acc.x[i] * r);
                l = fmaf(l, r, e);
                m = mn;
            }
        }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < Row<HD>::E; ++i) acc.x[i] *= inv;
    const int64_t row = o.token * p.NH + o.head;
    acc.store(p.out + row * HD, lane);
    if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

// Gradient of one query.
template <int HD>
__device__ void row_dq(const ScoredParams& p, const Pos& o, int lane, volatile uint32_t* beat) {
    Row<HD> q, g, acc, x, y;
    const int64_t row = o.token * p.NH + o.head;
    q.load(p.q + o.token * p.q_ts + int64_t(o.head) * HD, lane);
    g.load(p.dout + row * HD, lane);
    y.load(p.out + row * HD, lane);
    const float lse = p.lse[row];
    // a row that sees nothing has no part in any gradient, whatever dout holds
    const float delta = lse == -INFINITY ? 0.f : g.dot(y);
    acc.zero();
    float slope[3], ds, inner = 0.f;
    load_slopes(p, o.head, slope);
    const int qdoc = p.doc ? p.doc[o.token] : 0, prefix = p.prefix ? p.prefix[o.b] : 0;
    const int t0 = win_start(o.t, p.KT, p.T), h0 = win_start(o.h, p.KH, p.H), w0 = win_start(o.w, p.KW, p.W);
    if (lse != -INFINITY)
        for (int t = t0; t < t0 + p.KT; ++t)
            for (int h = h0; h < h0 + p.KH; ++h) {
                still_going(beat, lane);
                for (int w = w0; w < w0 + p.KW; ++w) {
                    const int64_t tok = token_of(p, o.b, t, h, w);
                    if (!visible(p, qdoc, p.doc ? p.doc[tok] : 0, o.t, t, prefix)) continue;
                    x.load(p.k + tok * p.k_ts + int64_t(o.head) * HD, lane);
                    const float s = shape_score(p, q.dot(x), slope, o.t - t, o.h - h, o.w - w, &ds);
                    y.load(p.v + tok * p.v_ts + int64_t(o.head) * HD, lane);
                    const float e = expf(s - lse), dp = g.dot(y);
                    inner = fmaf(e, dp, inner);
                    acc.axpy(e * (dp - delta) * ds, x);
                }
            }
    if (lane == 0) p.stat[stat_at(p, o.b, o.token, o.head)].y = inner;
    acc.store(p.dq + o.token * p.dq_ts + int64_t(o.head) * HD, lane);
}

// Gradients of one key and value, over the queries whose windows hold it.
template <int HD>
__device__ void row_dkv(const ScoredParams& p, const Pos& o, int lane, volatile uint32_t* beat) {
    Row<HD> k, v, dk, dv, x, g;
    k.load(p.k + o.token * p.k_ts + int64_t(o.head) * HD, lane);
    v.load(p.v + o.token * p.v_ts + int64_t(o.head) * HD, lane);
    dk.zero();
    dv.zero();
    float slope[3], ds;
    load_slopes(p, o.head, slope);
    const int kdoc = p.doc ? p.doc[o.token] : 0, prefix = p.prefix ? p.prefix[o.b] : 0;
    const int t1 = inv_last(o.t, p.KT, p.T), h1 = inv_last(o.h, p.KH, p.H), w1 = inv_last(o.w, p.KW, p.W);
    for (int t = inv_first(o.t, p.KT); t <= t1; ++t)
        for (int h = inv_first(o.h, p.KH); h <= h1; ++h) {
            still_going(beat, lane);
            for (int w = inv_first(o.w, p.KW); w <= w1; ++w) {
                const int64_t tok = token_of(p, o.b, t, h, w), row = tok * p.NH + o.head;
                if (!visible(p, p.doc ? p.doc[tok] : 0, kdoc, t, o.t, prefix)) continue;
                const float lse = p.lse[row];
                if (lse == -INFINITY) continue;
                x.load(p.q + tok * p.q_ts + int64_t(o.head) * HD, lane);
                const float s = shape_score(p, x.dot(k), slope, o.t - t, o.h - h, o.w - w, &ds);
                g.load(p.dout + row * HD, lane);
                const float e = expf(s - lse);
                dv.axpy(e, g);
                dk.axpy(e * (g.dot(v) - p.stat[stat_at(p, o.b, tok, o.head)].y) * ds, x);
            }
        }
    dk.store(p.dk + o.token * p.dk_ts + int64_t(o.head) * HD, lane);
    dv.store(p.dv + o.token * p.dv_ts + int64_t(o.head) * HD, lane);
}

// ------------------------------------------------------------------ tiles

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;      // log2 growth of the scores past the kept maximum before a rescale
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 500000000ull;

// What the rounding of x and y to the pair p leaves of them, rounded itself. dQ
// takes da in two such parts: of the three gradients it alone has the rounding
// of out in it, through delta, and one rounding more would count.
__device__ __forceinline__ uint32_t left_over(float x, float y, uint32_t p) {
    return pack_bf16x2(x - __uint_as_float(p << 16), y - __uint_as_float(p & 0xffff0000u));
}

// Has the block given up? It does kWaitLimitNs after this wait began (t0) and after the last beat.
// (One given between the reads of clock and beat is ahead: the difference is signed.)
__device__ __noinline__ bool gave_up(volatile uint32_t* abort_flag, uint64_t t0) {
    if (abort_flag[0]) return true;
    if (globaltimer_ns() - t0 <= kWaitLimitNs || int32_t(beat_clock() - abort_flag[1]) <= int32_t(kWaitLimitNs >> 20)) return false;
    abort_flag[0] = 1u;
    atomicOr(&g_scored_timeout_flag, 1u);
    return true;
}

struct Sync {
    uint32_t bar0;
    volatile uint32_t* abort_flag;   // behind it the beat
    __device__ __forceinline__ uint32_t bar(int i) const { return bar0 + 8u * i; }
    // Wait for a barrier phase; false once this block has given up.
    __device__ __forceinline__ bool wait(uint32_t b, uint32_t parity) const {
        if (mbar_try_wait(b, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            if (mbar_try_wait(b, parity)) return true;
            if ((it & 255u) == 0u && gave_up(abort_flag, t0)) return false;
        }
    }
};

// A kernel lets the next one of its stream start, and waits for the one before
// it to be through.
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of the 16-byte chunk c of row r in a box of HD-column rows as
// TMA writes it: rows of up to 128 bytes, their chunks permuted over the
// banks; HD 128 takes two such regions.
template <int HD>
__device__ __forceinline__ uint32_t swizzled(int r, int c, uint32_t region) {
    if (HD == 16) return uint32_t(r) * 32 + ((c ^ ((r >> 2) & 1)) << 4);
    if (HD == 32) return uint32_t(r) * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return (c >> 3) * region + uint32_t(r) * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint64_t f2_dup(float x) { return f2_pack(x, x); }

// tanh z = z + z^3 P(z^2) for |z| <= 1/2.
__device__ constexpr float kTanh[4] = {-0.333331435918808f, 0.13325878977775574f, -0.05304548144340515f,
                                       0.0172414667904377f};

// tanh to about 2^-22 of its value. Up to 1/2 (a score of half the cap) an odd
// polynomial, fitted for the least largest relative error (1.5e-8), keeps the
// special-function unit free; larger values take 1 - 2 / (1 + e^2|z|), once
// any of the warp's needs it.
__device__ __forceinline__ uint64_t tanh_poly(uint64_t z) {
    const uint64_t y = f2_mul(z, z);
    uint64_t p = f2_fma(y, f2_dup(kTanh[3]), f2_dup(kTanh[2]));
    p = f2_fma(y, p, f2_dup(kTanh[1]));
    p = f2_fma(y, p, f2_dup(kTanh[0]));
    return f2_fma(f2_mul(z, y), p, z);
}
__device__ __forceinline__ float tanh_exp(float z) {
    const float e = ex2_approx(fabsf(z) * (2.f * kLog2e));
    return copysignf(fmaf(-2.f, rcp_approx(e + 1.f), 1.f), z);
}

// Largest of a, |b| and |c|, NaN where one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return d;
}

// z[0..3], pairs, to their tanh.
__device__ __forceinline__ void tanh_all(uint64_t* z) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(z[i], x[2 * i], x[2 * i + 1]);
    const float big = fmaxf(max3f(fabsf(x[0]), fabsf(x[1]), fabsf(x[2])),
                            fmaxf(max3f(fabsf(x[3]), fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7]))));
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = tanh_poly(z[i]);
    if (__any_sync(0xffffffffu, big > 0.5f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, up;
            f2_unpack(z[i], lo, up);
            z[i] = f2_pack(fabsf(x[2 * i]) > 0.5f ? tanh_exp(x[2 * i]) : lo,
                           fabsf(x[2 * i + 1]) > 0.5f ? tanh_exp(x[2 * i + 1]) : up);
        }
    }
}

// The reference of row i of a thread's two moves up by the returned amount, for
// scores (minus the old one) up to `top`: what the row has summed is scaled. A
// row that has met a key moves up only; the first keys set the reference.
template <int N>
__device__ __forceinline__ float move_reference(float top, float& grow, float& ref, float& l, float (&acc)[N][4], int i) {
    float x = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
    const bool begun = grow == kGrow;
    if (begun || x == -INFINITY) x = fmaxf(x, 0.f);
    else grow = kGrow;
    const float r = begun ? ex2_approx(-x) : 0.f;
    ref += x;
    l *= r;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        acc[j][2 * i] *= r;
        acc[j][2 * i + 1] *= r;
    }
    return x;
}

// One persistent block; nw warps, 16 rows each.
//   FWD: fixed rows Q; streamed K, V. DQ: fixed Q, dO; streamed K, V.
//   DKV: fixed K, V; streamed Q, dO and each query's (lse, delta).
// A block takes a contiguous run of units, consecutive bricks of one head, so
// that most find the table of their predecessor: it depends on the head and on
// where the rows' windows lie about them, the same for all rows away from the
// borders. The warps run freely over a ring of stages; the warp that is last
// to be done with a stage starts the load of the chunk that is next to use it,
// so no warp waits for an empty stage and none is kept for loading (a
// thirteenth would cost the other twelve a fifth of their registers).
//
// What bounds it: latency. At (1,16,64,64,8,64) with a (3,7,7) window, cap and
// bias (forward, 260 us) the schedulers issue in 36 % of the cycles with two
// warps each, mma.sync takes 26 % of its pipe, memory 24 % of its rate; without
// its loads the kernel takes 230 of 257 us, without its products 220, without
// cap, bias and exponential 227, and without any step the units' and frames'
// own work takes 95. More warps need registers that a step does not have to
// spare: 12 warps of 168 registers 274 us, 16 of 128 spill, 446. Steps that
// take the next one's scores early, or two or three steps at once, are 4 to 9 %
// slower. Whole-row (3,7,33) windows with packed, padded clips at
// (1,8,64,33,8,64): 222 us; HD 128, causal, at (1,8,48,64,16,128): 375 us. A
// training step at (1,16,32,48,8,64), (3,7,7): 112 us forward, 144 dQ, 243 dK
// and dV (four products a step, and 11 columns of a row where the others have
// 10: near a border more windows hold a key).
template <int HD, int MODE>
__global__ void __launch_bounds__(max_warps(HD, MODE) * 32, blocks_per_sm(HD, MODE))
scored_tiles(const __grid_constant__ CUtensorMap tm_f0, const __grid_constant__ CUtensorMap tm_f1,
             const __grid_constant__ CUtensorMap tm_x0, const __grid_constant__ CUtensorMap tm_x1,
             const __grid_constant__ ScoredParams p, const __grid_constant__ TileGeom g) {
    constexpr bool DKV = MODE == kDkv;
    constexpr int NF = MODE == kFwd ? 1 : 2;           // fixed tensors
    constexpr int FB = fixed_buffers(HD, MODE);
    constexpr int NFR = FB == 2 ? 1 : NF;              // fixed tensors whose fragments stay in registers
    constexpr int KB = HD / 16;                        // 16-column blocks of the head dim
    constexpr int REG = HD > 64 ? HD / 64 : 1;         // 64-column regions
    constexpr int HDB = HD > 64 ? 64 : HD;             // columns of a box
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nw = g.nw, S = g.stages;
    const int f_rows = g.st * g.bh * g.sw;
    const uint32_t f_region = (uint32_t(f_rows) * HDB * 2 + 1023u) & ~1023u, f_bytes = f_region * REG;
    const uint32_t x_bytes = g.x_bytes, x_region = REG > 1 ? x_bytes / REG : 0;
    const bool docs = p.doc != nullptr;

    if (MODE == kDq) dependents_may_start();

    // control words: abort flag, beat, then done and issued counts of each ring
    // (the stages, then the fixed buffers); barriers: one a ring place
    uint32_t* misc = reinterpret_cast<uint32_t*>(base_ptr + g.off_bar);
    const Sync sy{base + g.off_bar + kControl, misc};
    uint32_t *done = misc + 2, *issued = misc + 2 + kMaxRing;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S + FB; ++i) {
            mbar_init(sy.bar(i), 1);
            done[i] = 0;
            issued[i] = 0;
        }
        misc[0] = 0u;
        misc[1] = beat_clock() - uint32_t(kWaitLimitNs >> 20) - 1u;   // long ago
        fence_mbar_init();
    }
    // The stages start as zeros: a step reads up to 15 rows past a chunk's box,
    // whose probabilities are 0, and those rows must hold numbers.
    for (int i = threadIdx.x * 16; i < g.off_lut - g.off_x; i += blockDim.x * 16)
        *reinterpret_cast<uint4*>(base_ptr + g.off_x + i) = make_uint4(0, 0, 0, 0);
    // (row, column) of the chunk's index, as floats
    float2* const hw = reinterpret_cast<float2*>(base_ptr + g.off_hw);
    for (int i = threadIdx.x; i < g.cr * g.cc + 16; i += blockDim.x) hw[i] = make_float2(float(i / g.cc), float(i % g.cc));
    fence_proxy_async_smem();
    // the kernel before brings the statistics (the forward pass has none that lets it start early)
    if (MODE != kFwd) wait_for_primary();
    __syncthreads();

    const int u0 = int(int64_t(g.units) * blockIdx.x / gridDim.x);
    const int u1 = int(int64_t(g.units) * (blockIdx.x + 1) / gridDim.x);

    // Start the load of chunk (it, ih, iw) of a unit into stage s. A chunk
    // past the brick's own box (the boxes at the borders are smaller) brings nothing.
    auto load_chunk = [&](const Unit& x, int it, int ih, int iw, int s) {   // one thread
        const int t = x.bt.x + it, h = x.bh.x + ih * g.cr, w = x.bw.x + iw * g.cc;
        const bool inside = t < x.bt.y && h < x.bh.y && w < x.bw.y;
        const uint32_t full = sy.bar(s), x0 = base + g.off_x + 2 * s * x_bytes;
        ++issued[s];
        if (!inside) {
            mbar_arrive(full);
            return;
        }
        mbar_arrive_expect_tx(full, 2 * REG * g.cr * g.cc * HDB * 2);
        for (int r = 0; r < REG; ++r) {
            tma_load_5d(x0 + r * x_region, &tm_x0, full, x.head * HD + r * 64, w, h, t, x.o.b);
            tma_load_5d(x0 + x_bytes + r * x_region, &tm_x1, full, x.head * HD + r * 64, w, h, t, x.o.b);
        }
    };
    auto load_fixed = [&](const Unit& x, int f) {   // one thread
        const uint32_t full = sy.bar(S + f), to = base + f * NF * f_bytes;
        ++issued[S + f];
        mbar_arrive_expect_tx(full, NF * REG * f_rows * HDB * 2);
        for (int r = 0; r < REG; ++r) {
            tma_load_5d(to + r * f_region, &tm_f0, full, x.head * HD + r * 64, x.o.w0, x.o.h0, x.o.t0, x.o.b);
            if (NF == 2)
                tma_load_5d(to + f_bytes + r * f_region, &tm_f1, full, x.head * HD + r * 64, x.o.w0, x.o.h0, x.o.t0, x.o.b);
        }
    };
    // This warp is done with a ring place; true, in lane 0, where it is the last to be.
    auto last_done = [&](int i) {
        __syncwarp();
        if (lane != 0) return false;
        uint32_t n;
        asm volatile("atom.acq_rel.cta.shared::cta.inc.u32 %0, [%1], %2;"
                     : "=r"(n) : "r"(smem_u32(done + i)), "r"(uint32_t(nw - 1)) : "memory");
        return n == uint32_t(nw - 1);
    };
    Unit cur = unit_of<DKV>(p, g, min(u0, g.units - 1));
    // the chunk that is S after the current one: its place in its unit, and whether
    // that is the next (there are at most per_unit stages)
    int nt_i = 0, nh_i = 0, nw_i = 0;
    bool in_next = false;
    auto advance = [&] {
        if (++nw_i < g.nwc) return;
        nw_i = 0;
        if (++nh_i < g.nhc) return;
        nh_i = 0;
        if (++nt_i < g.nt) return;
        nt_i = 0;
        in_next = true;
    };
    for (int s = 0; s < S; ++s) {
        if (threadIdx.x == 0 && u0 < u1) load_chunk(cur, nt_i, nh_i, nw_i, s);
        advance();
    }
    if (warp == 0 && lane == 0 && u0 < u1) {
        load_fixed(cur, 0);
        if (FB == 2 && u0 + 1 < u1) load_fixed(unit_of<DKV>(p, g, u0 + 1), 1);
    }

    const int r0 = lane >> 2, c2 = lane & 3;    // this thread's rows r0, r0 + 8 and column pair of a fragment
    const int hi = lane >> 4;
    const int n_hw = g.sh * g.sw;               // (h, w) places of a warp's rows
    const bool same_hw = n_hw <= 8, use_lut = g.lut != 0;
    float* const lut = reinterpret_cast<float*>(base_ptr + g.off_lut) + warp * n_hw * g.lut_pitch;
    uint32_t* const mask = reinterpret_cast<uint32_t*>(base_ptr + g.off_lut) + warp * g.frame_steps * 8;
    const float* const lut_row = lut + (r0 % n_hw) * g.lut_pitch + 2 * c2;
    const int row_t0 = r0 / n_hw, row_t1 = (r0 + 8) / n_hw;
    const int row_h0 = r0 / g.sw % g.sh, row_h1 = (r0 + 8) / g.sw % g.sh, row_w = r0 % g.sw;
    const int frag_row = (((lane & 15) / n_hw) * g.bh + warp * g.sh + (lane & 15) / g.sw % g.sh) * g.sw + (lane & 15) % g.sw;
    const bool one_chunk = g.nhc * g.nwc == 1;
    const float inv_cap = p.softcap > 0.f ? 1.f / p.softcap : 0.f;
    const bool capped = p.softcap > 0.f, biased = p.slopes != nullptr;
    const float to_log2 = capped ? p.softcap * kLog2e : kLog2e;
    const float exp_scale = 2.f * kLog2e * inv_cap;
    // Columns' documents and (lse, delta): a warp keeps those of its current chunk in a
    // buffer of its own and the next chunk's first ones in registers meanwhile.
    constexpr int PF = 3;
    int* const col_doc = reinterpret_cast<int*>(base_ptr + g.off_doc) + warp * g.chunk_steps * 16;
    float2* const col_stat = reinterpret_cast<float2*>(base_ptr + g.off_stat) + warp * g.chunk_steps * 16;
    int pre_doc[PF] = {};
    float2 pre_stat[DKV ? PF : 1];
    int lut_head = -1, lut_h = -2, lut_w = -2, lut_chunk = -1;   // what the table holds
    float sl[3] = {0.f, 0.f, 0.f};
    int s = 0;             // stage of the current chunk, and the parity of its turn
    uint32_t turn = 0, ft = 0;
    bool ok = true;

    for (int u = u0; u < u1; ++u, ++ft) {
        in_next = S == g.nt * g.nhc * g.nwc;
        const Brick o = cur.o;
        const int head = cur.head, wh0 = o.h0 + warp * g.sh;
        // this warp's part of the streamed rows; none where its rows lie past the grid
        const int2 mine = warp_rows<DKV>(p, g, cur, warp);

        // rows r0 and r0 + 8, in one column of the grid
        const int rw = o.w0 + row_w;
        const int rt[2] = {o.t0 + row_t0, o.t0 + row_t1}, rh[2] = {wh0 + row_h0, wh0 + row_h1};
        const bool row_in[2] = {rw < p.W && rh[0] < p.H && rt[0] < p.T, rw < p.W && rh[1] < p.H && rt[1] < p.T};
        float ref[2] = {0.f, 0.f}, delta[2] = {0.f, 0.f};   // log2 reference that scores are taken from
        int row_doc[2] = {-1, -1};
        // the frames that a row sees (FWD, DQ) or that see it: its window's, less those that
        // come too late; none for a row past the grid or in no document
        const int prefix = p.prefix ? p.prefix[o.b] : 0;
        int t_lo[2], t_n[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int lo = range_lo(DKV, rt[i], p.KT, p.T), end = range_hi(DKV, rt[i], p.KT, p.T);
            if (p.prefix) {
                if (!DKV) end = min(end, max(rt[i] + 1, prefix));
                else if (rt[i] >= prefix) lo = max(lo, rt[i]);
            }
            if (MODE == kDq || docs) {
                const int64_t token = row_in[i] ? token_of(p, o.b, rt[i], rh[i], rw) : 0;
                if (MODE == kDq) {
                    const float2 x = p.stat[stat_at(p, o.b, token, head)];
                    ref[i] = x.x;
                    delta[i] = x.y;
                }
                if (docs) row_doc[i] = p.doc[token];
            }
            t_lo[i] = lo;
            t_n[i] = row_in[i] && !(docs && row_doc[i] < 0) ? end - lo : 0;
        }
        if (biased && head != lut_head) {
            load_slopes(p, head, sl);
#pragma unroll
            for (int a = 0; a < 3; ++a) sl[a] *= -kLog2e;
        }

        const int d0 = docs ? __shfl_sync(0xffffffffu, row_doc[0], 0) : 0;
        const int64_t stat0 = DKV ? stat_at(p, o.b, 0, head) : 0;
        // column i of a chunk's part; past the part and the grid there is nothing, and no row sees it
        auto fetch = [&](int i, const Part& at, int t, int& doc, float2& stat) {
            doc = d0;
            stat = make_float2(0.f, 0.f);
            if (i >= at.n) return;
            const float2 off = hw[i];
            const int x = at.w + int(off.y);
            if (x >= p.W) return;
            const int64_t token = token_of(p, o.b, t, at.hf + int(off.x), x);
            if (docs) doc = p.doc[token];
            if (DKV) stat = p.stat[stat0 + token];
        };
        auto prefetch = [&](int it, int ih, int iw) {
            const int t = cur.bt.x + it;
            if (!has_frame(cur, t)) return;
            const Part at = part_of(g, cur, mine, ih, iw);
#pragma unroll
            for (int j = 0; j < PF; ++j) fetch(lane + 32 * j, at, t, pre_doc[j], pre_stat[DKV ? j : 0]);
        };
        if (DKV || docs) prefetch(0, 0, 0);

        // Scores under a cap whose bias falls with the distance need no running maximum: a
        // row's largest lies within the cap of 0 (its own position has no bias), so that
        // the powers stay in the range of fp32 and bf16 with 0 as the reference. (Windows of one
        // to three keys have no table and take the general steps: see kManyKeys.)
        const bool bounded = MODE == kFwd && capped && to_log2 <= 96.f && fmaxf(fmaxf(sl[0], sl[1]), sl[2]) <= 0.f;
        // The table: for each (h, w) of the rows, the bias of a frame's columns, -inf
        // outside the window (or the mask words: word r of a step holds row r in its low
        // and row r + 8 in its high half). It is kept while the head (where it matters) and
        // the rows' place stay; rows away from the borders all have the same.
        const int place_h = wh0 >= p.KH && wh0 + g.sh - 1 < p.H - p.KH ? -1 : wh0;
        const int place_w = o.w0 >= p.KW && o.w0 + g.sw - 1 < p.W - p.KW ? -1 : o.w0;
        const int in_chunk = g.nhc > 1 ? mine.x - cur.bh.x : 0;
        if ((biased && head != lut_head) || place_h != lut_h || place_w != lut_w || in_chunk != lut_chunk) {
            __syncwarp();
            // a lane takes one row's place and, with others of the same, the columns in turn
            const int places = use_lut ? n_hw : 16, r = lane & (places - 1), at_once = 32 / places;
            const int lh = wh0 + ((r >> g.sw_log2) & (g.sh - 1)), lw = o.w0 + (r & (g.sw - 1));
            const int h_lo = range_lo(DKV, lh, p.KH, p.H), w_lo = range_lo(DKV, lw, p.KW, p.W);
            const int h_n = lh < p.H && lw < p.W ? range_hi(DKV, lh, p.KH, p.H) - h_lo : 0;
            const int w_n = range_hi(DKV, lw, p.KW, p.W) - w_lo;
            int at_step = 0;
            for (int ih = 0; ih < g.nhc; ++ih)
                for (int iw = 0; iw < g.nwc; ++iw) {
                    const Part part = part_of(g, cur, mine, ih, iw);
                    const int hf = part.hf, w = part.w, n = part.n, steps = n > 0 ? (n + 15) >> 4 : 0;
                    if (use_lut) {
                        float* const to = lut + r * g.lut_pitch + at_step * 16;
#pragma unroll 4
                        for (int i = lane / places; i < steps * 16; i += at_once) {
                            const float2 at = hw[i];
                            const int y = hf + int(at.x), x = w + int(at.y);
                            const bool in = i < n && uint32_t(y - h_lo) < uint32_t(h_n) && uint32_t(x - w_lo) < uint32_t(w_n);
                            to[i] = in ? fmaf(sl[1], float(abs(y - lh)), sl[2] * float(abs(x - lw))) : -INFINITY;
                        }
                    } else {
                        for (int k = 0; k < steps; ++k) {   // eight columns a lane, then both halves' together
                            uint32_t bits = 0;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int i = 16 * k + 8 * hi + j;
                                const float2 at = hw[i];
                                const int y = hf + int(at.x), x = w + int(at.y);
                                const bool in = i < n && uint32_t(y - h_lo) < uint32_t(h_n) && uint32_t(x - w_lo) < uint32_t(w_n);
                                bits |= uint32_t(in) << (8 * hi + j);
                            }
                            bits |= __shfl_xor_sync(0xffffffffu, bits, 16);
                            if (hi == 0)
                                reinterpret_cast<uint16_t*>(mask)[(at_step + k) * 16 + 2 * (r & 7) + (r >> 3)] = uint16_t(bits);
                        }
                    }
                    at_step += steps;
                }
            __syncwarp();
            lut_head = head;
            lut_h = place_h;
            lut_w = place_w;
            lut_chunk = in_chunk;
        }

        // fixed fragments
        uint32_t fa[NFR][KB][4];
        const int fb = ft % FB;
        if (!(ok = sy.wait(sy.bar(S + fb), (ft / FB) & 1u))) break;
        const uint32_t f_at = base + fb * NF * f_bytes;
#pragma unroll
        for (int n = 0; n < NFR; ++n)
#pragma unroll
            for (int kk = 0; kk < KB; ++kk)
                ldsm4(f_at + n * f_bytes + swizzled<HD>(frag_row, 2 * kk + hi, f_region), fa[n][kk]);
        if (NFR == NF && last_done(S + fb) && u + 1 < u1) {
            Unit next = cur;
            next_unit<DKV>(p, g, next);
            load_fixed(next, fb);
        }

        float acc0[2 * KB][4], acc1[MODE == kDkv ? 2 * KB : 1][4];   // O, dQ or dK; dV
#pragma unroll
        for (int j = 0; j < 2 * KB; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc0[j][i] = 0.f;
                if (MODE == kDkv) acc1[j][i] = 0.f;
            }
        // FWD: the sum of e^(s - ref), and the growth that moves the reference:
        // any for a row that has met no key, so that ref starts at a score
        float l[2] = {0.f, 0.f}, grow[2] = {-INFINITY, -INFINITY};
        float inner[2] = {0.f, 0.f};   // DQ: the sum of p dp

        // this warp's part of a chunk: its columns from (hf, w), their steps, and the addresses of
        // the first ones in a stage (and its tables, where a frame has one chunk, once a unit)
        Part part{0, 0, 0};
        int part_steps = 0, step = 0;
        uint32_t part_at = 0;
        float row_t[2] = {float(rt[0] - cur.bt.x), float(rt[1] - cur.bt.x)};   // frames ahead
        for (int it = 0; it < g.nt && ok; ++it) {
            const int t = cur.bt.x + it;
            // the frame's part of the score: -inf for a row that does not see it
            float far_t[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                far_t[i] = uint32_t(t - t_lo[i]) < uint32_t(t_n[i]) ? sl[0] * fabsf(row_t[i]) : -INFINITY;
                row_t[i] -= 1.f;
            }
            // no row of this warp sees the frame: its chunks are passed over
            const bool frame_seen = t < cur.bt.y && __any_sync(0xffffffffu, fmaxf(far_t[0], far_t[1]) > -INFINITY);
            if (!one_chunk) step = 0;   // of the frame's table
            for (int ih = 0; ih < g.nhc && ok; ++ih)
                for (int iw = 0; iw < g.nwc; ++iw) {
                    if (!(ok = sy.wait(sy.bar(s), turn))) break;
                    if (!one_chunk || it == 0) {
                        part = part_of(g, cur, mine, ih, iw);
                        step += part_steps;
                        if (iw == 0 && ih == 0) step = 0;
                        part_steps = part.n > 0 ? (part.n + 15) >> 4 : 0;
                        // ldmatrix addresses: the permutation of a row's chunks repeats every 8 rows, so a
                        // step moves them by 16 rows and a column block by an exclusive or
                        part_at = swizzled<HD>((part.hf - cur.bh.x - ih * g.cr) * g.cc + (lane & 15), hi, 0);
                    }
                    int n_steps = frame_seen ? part_steps : 0;
                    const float* lut_at = lut_row + step * 16;
                    const uint32_t* mask_at = mask + step * 8 + r0;
                    // documents: a comparison for each score where the chunk holds others than
                    // the rows', none where it does not, no work where no row's is there
                    bool mixed = false;
                    if ((DKV || docs) && has_frame(cur, t)) {
                        bool other = docs && (row_doc[0] != d0 || row_doc[1] != d0);
                        bool met = other;
                        const int n = DKV ? part_steps * 16 : part.n;   // statistics: with the last step's columns past the part
                        auto keep = [&](int i, int doc, const float2& x) {
                            if (docs) {
                                col_doc[i] = doc;
                                other = other || doc != d0;
                                met = met || (doc == d0 && (!DKV || i < part.n));
                            }
                            if (DKV) col_stat[i] = x;
                        };
#pragma unroll
                        for (int j = 0; j < PF; ++j)
                            if (lane + 32 * j < n) keep(lane + 32 * j, pre_doc[j], pre_stat[DKV ? j : 0]);
                        for (int i = lane + 32 * PF; i < n; i += 32) {
                            int d;
                            float2 x;
                            fetch(i, part, t, d, x);
                            keep(i, d, x);
                        }
                        if (docs) {
                            mixed = __any_sync(0xffffffffu, other);
                            if (!__any_sync(0xffffffffu, met)) n_steps = 0;
                        }
                        __syncwarp();
                        const bool row_end = iw + 1 == g.nwc, part_end = row_end && ih + 1 == g.nhc;
                        if (!part_end || it + 1 < g.nt) prefetch(it + part_end, part_end ? 0 : ih + row_end, row_end ? 0 : iw + 1);
                    }
                    const int* key_doc = col_doc;
                    const float2* stat = col_stat;
                    uint32_t a0 = base + g.off_x + 2 * s * x_bytes + part_at;
                    auto columns = [&](uint32_t at, int kk) { return (at + (kk >> 2) * x_region) ^ ((kk & 3) << 5); };
                    // In a step columns 0..7 have their scores in sc[0..3], 8..15 in sc[4..7]; value i is
                    // of row (i >> 1) & 1 and column 8 * (i >> 2) + 2 * c2 + (i & 1).
                    // Most chunks take plain steps, without a branch in one: those with the table, but for
                    // caps or slopes that want a running maximum and the polynomial. Taking the next
                    // step's scores ahead, or two steps at a time, measured 4 to 9 % slower here: what
                    // it saves in waiting costs more in registers.
                    if (MODE == kFwd && use_lut && (!capped || bounded)) {
                        uint32_t ak[KB];   // a column block's address; the next step's is 16 rows on
#pragma unroll
                        for (int kk = 0; kk < KB; ++kk) ak[kk] = columns(a0, kk);
                        auto plain = [&](auto cap_const, auto mix_const) {
                            constexpr bool CAP = decltype(cap_const)::value, MIX = decltype(mix_const)::value;
                            float sc[8] = {}, sv[8];
                            uint32_t f[4];
#pragma unroll
                            for (int kk = 0; kk < KB; ++kk) {
                                ldsm4(ak[kk], f);
                                mma16816(sc, fa[0][kk], f[0], f[2]);
                                mma16816(sc + 4, fa[0][kk], f[1], f[3]);
                            }
                            const uint64_t from[2] = {f2_dup(far_t[0] - ref[0]), f2_dup(far_t[1] - ref[1])};
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint64_t x = *reinterpret_cast<const uint64_t*>(lut_at + 8 * j);
                                const uint64_t y = same_hw ? x : *reinterpret_cast<const uint64_t*>(lut_at + 8 * g.lut_pitch + 8 * j);
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const int v = 4 * j + 2 * i;
                                    const uint64_t a = f2_pack(sc[v], sc[v + 1]), bias = f2_add(i ? y : x, from[i]);   // minus the reference
                                    uint64_t s;
                                    if (CAP) {
                                        // c tanh(a / c) = c - 2 c / (1 + e^(2 a / c)), c up to 66 here. The quotient
                                        // near 1/2 has half the exponential's 2^-22, the sum's 2^-24 and the
                                        // reciprocal's 2^-23: with the last rounding under 2^-21 of c, where p takes
                                        // half a step of bf16, 2^-8 of itself
                                        float e0, e1;
                                        f2_unpack(f2_mul(a, f2_dup(exp_scale)), e0, e1);
                                        f2_unpack(f2_add(f2_pack(ex2_approx(e0), ex2_approx(e1)), f2_dup(1.f)), e0, e1);
                                        s = f2_fma(f2_pack(rcp_approx(e0), rcp_approx(e1)), f2_dup(-2.f * to_log2), f2_add(bias, f2_dup(to_log2)));
                                    } else {
                                        s = f2_fma(a, f2_dup(kLog2e), bias);
                                    }
                                    f2_unpack(s, sv[v], sv[v + 1]);
                                    if (MIX) {
                                        const int* d = key_doc + 8 * j + 2 * c2;
                                        if (d[0] != row_doc[i]) sv[v] = -INFINITY;
                                        if (d[1] != row_doc[i]) sv[v + 1] = -INFINITY;
                                    }
                                }
                            }
                            if (!CAP) {
                                float top[2];
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    top[i] = fmaxf(max3f(sv[2 * i], sv[2 * i + 1], sv[4 + 2 * i]), sv[5 + 2 * i]);
                                if (__any_sync(0xffffffffu, top[0] > grow[0] || top[1] > grow[1])) {
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        const float x = move_reference(top[i], grow[i], ref[i], l[i], acc0, i);
#pragma unroll
                                        for (int j = 0; j < 4; ++j) sv[4 * (j >> 1) + 2 * i + (j & 1)] -= x;
                                    }
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) sv[i] = ex2_approx(sv[i]);
                            l[0] += (sv[0] + sv[1]) + (sv[4] + sv[5]);
                            l[1] += (sv[2] + sv[3]) + (sv[6] + sv[7]);
                            const uint32_t a[4] = {pack_bf16x2(sv[0], sv[1]), pack_bf16x2(sv[2], sv[3]),
                                                   pack_bf16x2(sv[4], sv[5]), pack_bf16x2(sv[6], sv[7])};
#pragma unroll
                            for (int kk = 0; kk < KB; ++kk) {
                                ldsm4t(ak[kk] + x_bytes, f);
                                mma16816(acc0[2 * kk], a, f[0], f[1]);
                                mma16816(acc0[2 * kk + 1], a, f[2], f[3]);
                                ak[kk] += 16 * HDB * 2;
                            }
                            lut_at += 16;
                            if (MIX) key_doc += 16;
                        };
                        auto run = [&](auto cap_const, auto mix_const) {
                            for (int k = 0; k < n_steps; ++k) plain(cap_const, mix_const);
                        };
                        const std::integral_constant<bool, true> yes{};
                        const std::integral_constant<bool, false> no{};
                        if (capped && mixed) run(yes, yes);
                        else if (capped) run(yes, no);
                        else if (mixed) run(no, yes);
                        else run(no, no);
                        n_steps = 0;
                    }
                    // ... those of the backward passes
                    if (MODE != kFwd && use_lut && (!capped || to_log2 <= 96.f)) {
                        uint32_t ak[KB];
#pragma unroll
                        for (int kk = 0; kk < KB; ++kk) ak[kk] = columns(a0, kk);
                        auto plain = [&](auto cap_const, auto mix_const) {
                            constexpr bool CAP = decltype(cap_const)::value, MIX = decltype(mix_const)::value;
                            float sc[8] = {}, dp[8] = {};
#pragma unroll
                            for (int kk = 0; kk < KB; ++kk) {
                                uint32_t f[4], e[4], a[4];
                                ldsm4(ak[kk], f);
                                if (NFR < NF) ldsm4(f_at + f_bytes + swizzled<HD>(frag_row, 2 * kk + hi, f_region), a);
                                ldsm4(ak[kk] + x_bytes, e);
                                mma16816(sc, fa[0][kk], f[0], f[2]);
                                mma16816(sc + 4, fa[0][kk], f[1], f[3]);
                                mma16816(dp, NFR < NF ? a : fa[NFR - 1][kk], e[0], e[2]);
                                mma16816(dp + 4, NFR < NF ? a : fa[NFR - 1][kk], e[1], e[3]);
                            }
                            uint64_t from[2] = {f2_dup(far_t[0] - ref[0]), f2_dup(far_t[1] - ref[1])};
                            uint32_t pr[4], ds[4];   // probabilities (DQ: what da's rounding leaves) and da, pairs: 2 * tile + row
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                uint64_t minus_ref = 0, minus_delta = 0;
                                if (DKV) {
                                    const float2 c0 = stat[8 * j + 2 * c2], c1 = stat[8 * j + 2 * c2 + 1];
                                    minus_ref = f2_pack(-c0.x, -c1.x);
                                    minus_delta = f2_pack(-c0.y, -c1.y);
                                }
                                const uint64_t x = *reinterpret_cast<const uint64_t*>(lut_at + 8 * j);
                                const uint64_t y = same_hw ? x : *reinterpret_cast<const uint64_t*>(lut_at + 8 * g.lut_pitch + 8 * j);
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const int v = 4 * j + 2 * i;
                                    uint64_t s = f2_add(i ? y : x, from[i]), slope = 0;
                                    if (DKV) s = f2_add(s, minus_ref);
                                    if (CAP) {
                                        // with r = 1 / (1 + e^(2 a / c)): tanh = 1 - 2 r, its derivative 4 r (1 - r)
                                        float e0, e1;
                                        f2_unpack(f2_mul(f2_pack(sc[v], sc[v + 1]), f2_dup(exp_scale)), e0, e1);
                                        f2_unpack(f2_add(f2_pack(ex2_approx(e0), ex2_approx(e1)), f2_dup(1.f)), e0, e1);
                                        const uint64_t r = f2_pack(rcp_approx(e0), rcp_approx(e1));
                                        s = f2_fma(r, f2_dup(-2.f * to_log2), f2_add(s, f2_dup(to_log2)));
                                        slope = f2_mul(r, f2_fma(r, f2_dup(-4.f), f2_dup(4.f)));
                                    } else {
                                        s = f2_fma(f2_pack(sc[v], sc[v + 1]), f2_dup(kLog2e), s);
                                    }
                                    float p0, p1, d0, d1;
                                    f2_unpack(s, p0, p1);
                                    if (MIX) {
                                        const int* d = key_doc + 8 * j + 2 * c2;
                                        if (d[0] != row_doc[i]) p0 = -INFINITY;
                                        if (d[1] != row_doc[i]) p1 = -INFINITY;
                                    }
                                    p0 = ex2_approx(p0);
                                    p1 = ex2_approx(p1);
                                    if (MODE == kDq) inner[i] = fmaf(p0, dp[v], fmaf(p1, dp[v + 1], inner[i]));
                                    uint64_t d = f2_add(f2_pack(dp[v], dp[v + 1]), DKV ? minus_delta : f2_dup(-delta[i]));
                                    d = f2_mul(d, f2_pack(p0, p1));
                                    if (CAP) d = f2_mul(d, slope);
                                    f2_unpack(d, d0, d1);
                                    ds[2 * j + i] = pack_bf16x2(d0, d1);
                                    pr[2 * j + i] = MODE == kDq ? left_over(d0, d1, ds[2 * j + i]) : pack_bf16x2(p0, p1);
                                }
                            }
#pragma unroll
                            for (int kk = 0; kk < KB; ++kk) {
                                uint32_t f[4];
                                if (DKV) {
                                    ldsm4t(ak[kk] + x_bytes, f);
                                    mma16816(acc1[DKV ? 2 * kk : 0], pr, f[0], f[1]);
                                    mma16816(acc1[DKV ? 2 * kk + 1 : 0], pr, f[2], f[3]);
                                }
                                ldsm4t(ak[kk], f);
                                mma16816(acc0[2 * kk], ds, f[0], f[1]);
                                mma16816(acc0[2 * kk + 1], ds, f[2], f[3]);
                                if (MODE == kDq) {
                                    mma16816(acc0[2 * kk], pr, f[0], f[1]);
                                    mma16816(acc0[2 * kk + 1], pr, f[2], f[3]);
                                }
                            }
#pragma unroll
                            for (int kk = 0; kk < KB; ++kk) ak[kk] += 16 * HDB * 2;
                            lut_at += 16;
                            stat += 16;
                            if (MIX) key_doc += 16;
                        };
                        auto run = [&](auto cap_const, auto mix_const) {
                            for (int k = 0; k < n_steps; ++k) plain(cap_const, mix_const);
                        };
                        const std::integral_constant<bool, true> yes{};
                        const std::integral_constant<bool, false> no{};
                        if (capped && mixed) run(yes, yes);
                        else if (capped) run(yes, no);
                        else if (mixed) run(no, yes);
                        else run(no, no);
                        n_steps = 0;
                    }
                    for (int k = 0; k < n_steps; ++k, a0 += 16 * HDB * 2, lut_at += 16, mask_at += 8, stat += 16, key_doc += 16) {
                        const uint32_t a1 = a0 + x_bytes;
                        float sc[8], dp[8] = {};
                        uint32_t f[4];
#pragma unroll
                        for (int i = 0; i < 8; ++i) sc[i] = 0.f;
#pragma unroll
                        for (int kk = 0; kk < KB; ++kk) {
                            ldsm4(columns(a0, kk), f);
                            mma16816(sc, fa[0][kk], f[0], f[2]);
                            mma16816(sc + 4, fa[0][kk], f[1], f[3]);
                            if (MODE != kFwd) {
                                uint32_t a[4];
                                if (NFR < NF) ldsm4(f_at + f_bytes + swizzled<HD>(frag_row, 2 * kk + hi, f_region), a);
                                ldsm4(columns(a1, kk), f);
                                mma16816(dp, NFR < NF ? a : fa[NFR - 1][kk], f[0], f[2]);
                                mma16816(dp + 4, NFR < NF ? a : fa[NFR - 1][kk], f[1], f[3]);
                            }
                        }
                        float2 cs[4];   // DKV: (log2 reference, delta) of the four columns
                        if (DKV) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) cs[j] = stat[8 * (j >> 1) + 2 * c2 + (j & 1)];
                        }
                        // bias minus reference, log2: pair 2 * tile + row
                        uint64_t s2[4];
                        const float from[2] = {far_t[0] - ref[0], far_t[1] - ref[1]};
                        uint32_t bits = 0;   // 0, 1, 8, 9: the columns of row r0; 16, 17, 24, 25: of r0 + 8
                        if (use_lut) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint64_t x = *reinterpret_cast<const uint64_t*>(lut_at + 8 * j);
                                const uint64_t y = same_hw ? x : *reinterpret_cast<const uint64_t*>(lut_at + 8 * g.lut_pitch + 8 * j);
                                s2[2 * j] = f2_add(x, f2_dup(from[0]));
                                s2[2 * j + 1] = f2_add(y, f2_dup(from[1]));
                            }
                        } else {
                            bits = *mask_at >> (2 * c2);
#pragma unroll
                            for (int j = 0; j < 4; ++j) s2[j] = f2_dup(from[j & 1]);
                            if (biased) {
                                const float at_h[2] = {float(part.hf - rh[0]), float(part.hf - rh[1])}, at_w = float(part.w - rw);
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const float4 x = *reinterpret_cast<const float4*>(hw + k * 16 + 8 * j + 2 * c2);
                                    const float d0 = fabsf(x.y + at_w), d1 = fabsf(x.w + at_w);
#pragma unroll
                                    for (int i = 0; i < 2; ++i)
                                        s2[2 * j + i] = f2_pack(fmaf(sl[1], fabsf(x.x + at_h[i]), fmaf(sl[2], d0, from[i])),
                                                                fmaf(sl[1], fabsf(x.z + at_h[i]), fmaf(sl[2], d1, from[i])));
                                }
                            }
                        }
                        if (DKV) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                s2[j] = f2_add(s2[j], f2_pack(-cs[2 * (j >> 1)].x, -cs[2 * (j >> 1) + 1].x));
                        }
                        uint64_t th[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) th[j] = f2_pack(sc[2 * j], sc[2 * j + 1]);
                        if (capped) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) th[j] = f2_mul(th[j], f2_dup(inv_cap));
                            tanh_all(th);
                        }
                        float sv[8];   // scores minus reference, log2; then probabilities
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            f2_unpack(f2_fma(th[j], f2_dup(to_log2), s2[j]), sv[2 * j], sv[2 * j + 1]);
                        if (mixed || !use_lut) {
                            uint32_t gone = 0;   // bit i: value i is masked
                            if (!use_lut) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    gone |= (~bits >> (8 * (i >> 2) + 16 * ((i >> 1) & 1) + (i & 1)) & 1u) << i;
                            }
                            if (mixed) {
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const int2 d = make_int2(key_doc[8 * j + 2 * c2], key_doc[8 * j + 2 * c2 + 1]);
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        gone |= uint32_t(row_doc[i >> 1] != ((i & 1) ? d.y : d.x)) << (4 * j + i);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (gone >> i & 1u) {   // 0 times what a masked row holds need not be 0
                                    sv[i] = -INFINITY;
                                    if (MODE != kFwd) dp[i] = 0.f;
                                }
                            }
                        }
                        if (MODE == kFwd) {
                            float top[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                top[i] = fmaxf(max3f(sv[2 * i], sv[2 * i + 1], sv[4 + 2 * i]), sv[5 + 2 * i]);
                            if (__any_sync(0xffffffffu, top[0] > grow[0] || top[1] > grow[1])) {
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const float x = move_reference(top[i], grow[i], ref[i], l[i], acc0, i);
#pragma unroll
                                    for (int j = 0; j < 4; ++j) sv[4 * (j >> 1) + 2 * i + (j & 1)] -= x;
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) sv[i] = ex2_approx(sv[i]);
                            l[0] += (sv[0] + sv[1]) + (sv[4] + sv[5]);
                            l[1] += (sv[2] + sv[3]) + (sv[6] + sv[7]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                sv[i] = ex2_approx(sv[i]);
                                if (MODE == kDq) inner[(i >> 1) & 1] = fmaf(sv[i], dp[i], inner[(i >> 1) & 1]);
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint64_t d = f2_add(f2_pack(dp[2 * j], dp[2 * j + 1]),
                                                    DKV ? f2_pack(-cs[2 * (j >> 1)].y, -cs[2 * (j >> 1) + 1].y)
                                                        : f2_dup(-delta[j & 1]));
                                d = f2_mul(d, f2_pack(sv[2 * j], sv[2 * j + 1]));
                                if (capped) d = f2_mul(d, f2_fma(f2_mul(th[j], f2_dup(-1.f)), th[j], f2_dup(1.f)));
                                f2_unpack(d, dp[2 * j], dp[2 * j + 1]);
                            }
                        }
                        // products: probabilities (FWD: with V; DKV: with dO) and da (with K or Q)
                        if (MODE != kDq) {
                            const uint32_t a[4] = {pack_bf16x2(sv[0], sv[1]), pack_bf16x2(sv[2], sv[3]),
                                                   pack_bf16x2(sv[4], sv[5]), pack_bf16x2(sv[6], sv[7])};
#pragma unroll
                            for (int kk = 0; kk < KB; ++kk) {
                                ldsm4t(columns(a1, kk), f);
                                mma16816(MODE == kFwd ? acc0[2 * kk] : acc1[MODE == kDkv ? 2 * kk : 0], a, f[0], f[1]);
                                mma16816(MODE == kFwd ? acc0[2 * kk + 1] : acc1[MODE == kDkv ? 2 * kk + 1 : 0], a, f[2], f[3]);
                            }
                        }
                        if (MODE != kFwd) {
                            const uint32_t a[4] = {pack_bf16x2(dp[0], dp[1]), pack_bf16x2(dp[2], dp[3]),
                                                   pack_bf16x2(dp[4], dp[5]), pack_bf16x2(dp[6], dp[7])};
                            uint32_t rest[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (MODE == kDq) rest[j] = left_over(dp[2 * j], dp[2 * j + 1], a[j]);
#pragma unroll
                            for (int kk = 0; kk < KB; ++kk) {
                                ldsm4t(columns(a0, kk), f);
                                mma16816(acc0[2 * kk], a, f[0], f[1]);
                                mma16816(acc0[2 * kk + 1], a, f[2], f[3]);
                                if (MODE == kDq) {
                                    mma16816(acc0[2 * kk], rest, f[0], f[1]);
                                    mma16816(acc0[2 * kk + 1], rest, f[2], f[3]);
                                }
                            }
                        }
                    }
                    // the stage's next chunk is S further on
                    if (last_done(s) && (!in_next || u + 1 < u1)) {
                        Unit of = cur;
                        if (in_next) next_unit<DKV>(p, g, of);
                        load_chunk(of, nt_i, nh_i, nw_i, s);
                    }
                    advance();
                    if (++s == S) {
                        s = 0;
                        turn ^= 1u;
                    }
                }
        }
        if (!ok) break;
        if (NFR < NF && last_done(S + fb) && u + FB < u1) load_fixed(unit_of<DKV>(p, g, u + FB), fb);

        // rows out; a row that is not finite throughout is computed again by itself
        uint32_t bad = 0;
        uint16_t* const out0 = MODE == kFwd ? p.out : MODE == kDq ? p.dq : p.dk;
        const int64_t ts0 = MODE == kFwd ? int64_t(p.NH) * HD : MODE == kDq ? p.dq_ts : p.dk_ts;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t token = token_of(p, o.b, rt[i], rh[i], rw);
            float inv = 1.f;
            float top = 0.f;   // the largest magnitude, NaN where there is one
            if (MODE == kFwd) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
                inv = l[i] == 0.f ? 0.f : 1.f / l[i];
                top = l[i];
                if (row_in[i] && c2 == 0 && p.lse)
                    p.lse[token * p.NH + head] = l[i] == 0.f ? -INFINITY : (ref[i] + log2f(l[i])) * kLn2;
            }
            if (MODE == kDq) {
                // what delta is without the rounding of out and of its probabilities: for DKV
                inner[i] += __shfl_xor_sync(0xffffffffu, inner[i], 1);
                inner[i] += __shfl_xor_sync(0xffffffffu, inner[i], 2);
                if (row_in[i] && c2 == 0) p.stat[stat_at(p, o.b, token, head)].y = inner[i];
            }
            uint16_t* const at0 = out0 + token * ts0 + int64_t(head) * HD + 2 * c2;
            uint16_t* const at1 = p.dv + token * p.dv_ts + int64_t(head) * HD + 2 * c2;
#pragma unroll
            for (int j = 0; j < 2 * KB; ++j) {
                float x = acc0[j][2 * i], y = acc0[j][2 * i + 1];
                if (MODE == kFwd) f2_unpack(f2_mul(f2_pack(x, y), f2_dup(inv)), x, y);
                top = max3_nan(top, x, y);
                if (row_in[i]) *reinterpret_cast<uint32_t*>(at0 + 8 * j) = pack_bf16x2(x, y);
                if (MODE == kDkv) {
                    top = max3_nan(top, acc1[j][2 * i], acc1[j][2 * i + 1]);
                    if (row_in[i]) *reinterpret_cast<uint32_t*>(at1 + 8 * j) = pack_bf16x2(acc1[j][2 * i], acc1[j][2 * i + 1]);
                }
            }
            if (row_in[i] && !(top < INFINITY)) bad |= 1u << i;
        }
        if (__any_sync(0xffffffffu, bad != 0u)) {
            for (int r = 0; r < 16; ++r) {
                if (!__ballot_sync(0xffffffffu, (bad >> (r >> 3) & 1u) && r0 == (r & 7))) continue;
                Pos q;
                q.b = o.b;
                q.w = o.w0 + r % g.sw;
                q.h = wh0 + r / g.sw % g.sh;
                q.t = o.t0 + r / n_hw;
                q.head = head;
                q.token = token_of(p, q.b, q.t, q.h, q.w);
                __syncwarp();
                if (MODE == kFwd) row_fwd<HD>(p, q, lane, sy.abort_flag + 1);
                else if (MODE == kDq) row_dq<HD>(p, q, lane, sy.abort_flag + 1);
                else row_dkv<HD>(p, q, lane, sy.abort_flag + 1);
            }
        }
        next_unit<DKV>(p, g, cur);
    }

    // every issued load lands before the block may exit: where all went well
    // each has been waited for
    __syncthreads();
    if (misc[0] && threadIdx.x == 0)
        for (int i = 0; i < S + FB; ++i)
            if (issued[i] && !mbar_wait_bounded(sy.bar(i), (issued[i] - 1u) & 1u, kDrainLimitNs))
                atomicOr(&g_scored_timeout_flag, 1u);
}

// (lse in log2 units, delta) of every row for the backward passes:
// delta_i = dout_i . out_i; a row that sees nothing gets (0, 0). The pass for
// dQ takes delta from here and leaves the sum of p dp, which is the same
// without the rounding of out, in its place for the one for dK and dV. A row
// takes HD / 8 lanes, 16 bytes each. Bound by its reads.
template <int HD>
__global__ void __launch_bounds__(256) scored_stat(const ScoredParams p, int64_t rows) {
    constexpr int L = HD / 8;
    dependents_may_start();
    const int64_t r = (int64_t(blockIdx.x) * 256 + threadIdx.x) / L;
    const int c = threadIdx.x % L;
    const bool live = r < rows;
    float d = 0.f;
    if (live) {
        const uint4 a = *reinterpret_cast<const uint4*>(p.out + r * HD + c * 8);
        const uint4 b = *reinterpret_cast<const uint4*>(p.dout + r * HD + c * 8);
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), d);
            d = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), d);
        }
    }
#pragma unroll
    for (int k = L / 2; k; k >>= 1) d += __shfl_xor_sync(0xffffffffu, d, k);
    if (live && c == 0) {
        const float lse = p.lse[r];
        const int64_t token = r / p.NH;
        const int b = int(token / (int64_t(p.T) * p.H * p.W));
        p.stat[stat_at(p, b, token, int(r - token * p.NH))] =
            lse == -INFINITY ? make_float2(0.f, 0.f) : make_float2(lse * kLog2e, d);
    }
}

// ------------------------------------------------------------------ launch

// The plan of a call; a thread keeps the last few, since the search takes
// some microseconds.
bool cached_plan(TileGeom* out, const ScoredParams& p, int hd, int mode, int sms) {
    struct Entry {
        int32_t key[13];
        TileGeom g;
    };
    static thread_local Entry cache[16] = {};
    static thread_local unsigned next = 0;
    const int32_t key[13] = {p.B, p.T, p.H, p.W, p.NH, p.KT, p.KH, p.KW, hd, mode, sms, p.doc != nullptr, p.softcap > 0.f};
    for (const Entry& e : cache)
        if (memcmp(e.key, key, sizeof key) == 0) {
            *out = e.g;
            return true;
        }
    if (!plan_tiles(out, p, hd, mode, sms)) return false;
    Entry& e = cache[next++ % 16];
    memcpy(e.key, key, sizeof key);
    e.g = *out;
    return true;
}

template <int HD, int MODE>
cudaError_t launch_tiles(const ScoredParams& p, int sms, cudaStream_t stream) {
    TileGeom g;
    if (!cached_plan(&g, p, HD, MODE, sms)) return cudaErrorInvalidValue;
    constexpr int HDB = HD > 64 ? 64 : HD;
    const int64_t row = int64_t(p.NH) * HD;
    struct Src { const void* ptr; int64_t ts; };
    const Src q{p.q, p.q_ts}, k{p.k, p.k_ts}, v{p.v, p.v_ts}, d{p.dout, row};
    const Src f0 = MODE == kDkv ? k : q, f1 = MODE == kFwd ? q : MODE == kDq ? d : v;
    const Src x0 = MODE == kDkv ? q : k, x1 = MODE == kDkv ? d : v;
    CUtensorMap mf0, mf1, mx0, mx1;
    auto fixed = [&](CUtensorMap* m, const Src& s) {
        return encode_map(m, s.ptr, p.B, p.T, p.H, p.W, p.NH, HD, s.ts, HDB, g.sw, g.bh, g.st);
    };
    auto streamed = [&](CUtensorMap* m, const Src& s) {
        return encode_map(m, s.ptr, p.B, p.T, p.H, p.W, p.NH, HD, s.ts, HDB, g.cc, g.cr, 1);
    };
    if (!fixed(&mf0, f0) || !fixed(&mf1, f1) || !streamed(&mx0, x0) || !streamed(&mx1, x1))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(scored_tiles<HD, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    const int64_t slots = int64_t(sms) * blocks_per_sm(HD, MODE);
    const int grid = int(g.units < slots ? g.units : slots);
    if (MODE == kFwd) {
        scored_tiles<HD, MODE><<<grid, g.nw * 32, g.smem, stream>>>(mf0, mf1, mx0, mx1, p, g);
        return cudaGetLastError();
    }
    // starts while the kernel before it, which lets it, still runs
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = dim3(grid);
    c.blockDim = dim3(g.nw * 32);
    c.dynamicSmemBytes = g.smem;
    c.stream = stream;
    c.attrs = &a;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, scored_tiles<HD, MODE>, mf0, mf1, mx0, mx1, p, g);
}

template <int HD>
cudaError_t bwd(const ScoredParams& p, int sms, cudaStream_t stream) {
    const int64_t rows = int64_t(p.B) * p.T * p.H * p.W * p.NH;
    const int64_t blocks = (rows * (HD / 8) + 255) / 256;
    if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    scored_stat<HD><<<unsigned(blocks), 256, 0, stream>>>(p, rows);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // The pass for dQ leaves the exact delta in the workspace. Over few keys the rounding of out, which
    // is in the first one, tells in dq: its error at unit scores is 2.8e-3 over three keys, 2.3e-3
    // (capped 2.7e-3) over five and 2.2e-3 over seven, of which 1.7e-3 is its own rounding. Up to five
    // a second pass takes the exact delta and leaves that alone. Gradients of (1,16,64,64,8,64) with a
    // cap, windows of (1,1,3) and (1,1,5): 281 and 245 us with one pass, 389 and 339 with two.
    const bool twice = int64_t(p.KT) * p.KH * p.KW <= 5;
    for (int i = 0; i < (twice ? 2 : 1); ++i) {
        e = launch_tiles<HD, kDq>(p, sms, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_tiles<HD, kDkv>(p, sms, stream);
}

}  // namespace

static std::atomic<bool> g_launched{false};

bool scored_planned(int hd, const ScoredParams& p, bool backward) {
    constexpr int kSms = 152;   // whether there is a plan does not depend on it
    TileGeom g;
    if (!backward) return cached_plan(&g, p, hd, kFwd, kSms);
    return cached_plan(&g, p, hd, kDq, kSms) && cached_plan(&g, p, hd, kDkv, kSms);
}

cudaError_t launch_scored_fwd(int hd, const ScoredParams& p, int sms, cudaStream_t stream) {
    g_launched = true;
    switch (hd) {
        case 16: return launch_tiles<16, kFwd>(p, sms, stream);
        case 32: return launch_tiles<32, kFwd>(p, sms, stream);
        case 64: return launch_tiles<64, kFwd>(p, sms, stream);
        case 128: return launch_tiles<128, kFwd>(p, sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_scored_bwd(int hd, const ScoredParams& p, int sms, cudaStream_t stream) {
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
__device__ unsigned int g_scored_status_slots[kStatusSlots];

__global__ void take_scored_flag(unsigned int slot) {
    g_scored_status_slots[slot] = atomicExch(&g_scored_timeout_flag, 0u);
}

cudaError_t take_scored_error(cudaStream_t stream, unsigned int* flag) {
    *flag = 0;
    if (!g_launched) return cudaSuccess;
    static std::atomic<unsigned int> next{0};
    const unsigned int slot = next.fetch_add(1u) % kStatusSlots;
    take_scored_flag<<<1, 1, 0, stream>>>(slot);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbolAsync(flag, g_scored_status_slots, sizeof(unsigned int), slot * sizeof(unsigned int),
                                  cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(stream);
}

}  // namespace na3d
