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
// One warp computes one row of one head, its lanes splitting the head dim;
// a masked key is skipped, so what it holds never reaches the row.
#include <cuda_bf16.h>

#include "na3d_scored.cuh"

namespace na3d {

namespace {

constexpr int kRowWarps = 8;

__device__ __forceinline__ int win_start(int i, int K, int N) {
    return max(0, min(i - K / 2, N - K));
}

// The queries whose windows hold position j of an axis: [first, last].
__device__ __forceinline__ int inv_first(int j, int K) { return j < K ? 0 : j - K / 2; }
__device__ __forceinline__ int inv_last(int j, int K, int N) { return j >= N - K ? N - 1 : j + K / 2; }

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

__device__ __forceinline__ Pos pos_of(const ScoredParams& p, int64_t row) {
    Pos o;
    o.head = int(row % p.NH);
    o.token = row / p.NH;
    int64_t r = o.token;
    o.w = int(r % p.W); r /= p.W;
    o.h = int(r % p.H); r /= p.H;
    o.t = int(r % p.T);
    o.b = int(r / p.T);
    return o;
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

// Forward row: a running maximum m, the sum l of e^(s - m) and the weighted
// sum of v, rescaled when m grows.
template <int HD>
__device__ void row_fwd(const ScoredParams& p, const Pos& o, int lane) {
    Row<HD> q, acc, x;
    q.load(p.q + o.token * p.q_ts + int64_t(o.head) * HD, lane);
    acc.zero();
    float slope[3], m = -INFINITY, l = 0.f, unused;
    load_slopes(p, o.head, slope);
    const int qdoc = p.doc ? p.doc[o.token] : 0, prefix = p.prefix ? p.prefix[o.b] : 0;
    const int t0 = win_start(o.t, p.KT, p.T), h0 = win_start(o.h, p.KH, p.H), w0 = win_start(o.w, p.KW, p.W);
    for (int t = t0; t < t0 + p.KT; ++t)
        for (int h = h0; h < h0 + p.KH; ++h)
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
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < Row<HD>::E; ++i) acc.x[i] *= inv;
    const int64_t row = o.token * p.NH + o.head;
    acc.store(p.out + row * HD, lane);
    if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

// Gradient of one query, and its delta.
template <int HD>
__device__ void row_dq(const ScoredParams& p, const Pos& o, int lane) {
    Row<HD> q, g, acc, x, y;
    const int64_t row = o.token * p.NH + o.head;
    q.load(p.q + o.token * p.q_ts + int64_t(o.head) * HD, lane);
    g.load(p.dout + row * HD, lane);
    y.load(p.out + row * HD, lane);
    const float lse = p.lse[row];
    // a row that sees nothing has no part in any gradient, whatever dout holds
    const float delta = lse == -INFINITY ? 0.f : g.dot(y);
    if (lane == 0) p.delta[row] = delta;
    acc.zero();
    float slope[3], ds;
    load_slopes(p, o.head, slope);
    const int qdoc = p.doc ? p.doc[o.token] : 0, prefix = p.prefix ? p.prefix[o.b] : 0;
    const int t0 = win_start(o.t, p.KT, p.T), h0 = win_start(o.h, p.KH, p.H), w0 = win_start(o.w, p.KW, p.W);
    if (lse != -INFINITY)
        for (int t = t0; t < t0 + p.KT; ++t)
            for (int h = h0; h < h0 + p.KH; ++h)
                for (int w = w0; w < w0 + p.KW; ++w) {
                    const int64_t tok = token_of(p, o.b, t, h, w);
                    if (!visible(p, qdoc, p.doc ? p.doc[tok] : 0, o.t, t, prefix)) continue;
                    x.load(p.k + tok * p.k_ts + int64_t(o.head) * HD, lane);
                    const float s = shape_score(p, q.dot(x), slope, o.t - t, o.h - h, o.w - w, &ds);
                    y.load(p.v + tok * p.v_ts + int64_t(o.head) * HD, lane);
                    acc.axpy(expf(s - lse) * (g.dot(y) - delta) * ds, x);
                }
    acc.store(p.dq + o.token * p.dq_ts + int64_t(o.head) * HD, lane);
}

// Gradients of one key and value, over the queries whose windows hold it.
template <int HD>
__device__ void row_dkv(const ScoredParams& p, const Pos& o, int lane) {
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
        for (int h = inv_first(o.h, p.KH); h <= h1; ++h)
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
                dk.axpy(e * (g.dot(v) - p.delta[row]) * ds, x);
            }
    dk.store(p.dk + o.token * p.dk_ts + int64_t(o.head) * HD, lane);
    dv.store(p.dv + o.token * p.dv_ts + int64_t(o.head) * HD, lane);
}

enum { kFwd, kDq, kDkv };

template <int HD, int MODE>
__global__ void __launch_bounds__(kRowWarps * 32) scored_rows(const ScoredParams p) {
    const int64_t rows = int64_t(p.B) * p.T * p.H * p.W * p.NH;
    const int lane = threadIdx.x & 31;
    for (int64_t r = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); r < rows;
         r += int64_t(gridDim.x) * kRowWarps) {
        const Pos o = pos_of(p, r);
        if (MODE == kFwd) row_fwd<HD>(p, o, lane);
        else if (MODE == kDq) row_dq<HD>(p, o, lane);
        else row_dkv<HD>(p, o, lane);
    }
}

int row_grid(const ScoredParams& p, int sms) {
    const int64_t rows = int64_t(p.B) * p.T * p.H * p.W * p.NH;
    const int64_t need = (rows + kRowWarps - 1) / kRowWarps;
    return int(need < int64_t(sms) * 8 ? need : int64_t(sms) * 8);
}

template <int HD>
cudaError_t fwd(const ScoredParams& p, int sms, cudaStream_t stream) {
    scored_rows<HD, kFwd><<<row_grid(p, sms), kRowWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int HD>
cudaError_t bwd(const ScoredParams& p, int sms, cudaStream_t stream) {
    scored_rows<HD, kDq><<<row_grid(p, sms), kRowWarps * 32, 0, stream>>>(p);
    scored_rows<HD, kDkv><<<row_grid(p, sms), kRowWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scored_fwd(int hd, const ScoredParams& p, int sms, cudaStream_t stream) {
    switch (hd) {
        case 16: return fwd<16>(p, sms, stream);
        case 32: return fwd<32>(p, sms, stream);
        case 64: return fwd<64>(p, sms, stream);
        case 128: return fwd<128>(p, sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_scored_bwd(int hd, const ScoredParams& p, int sms, cudaStream_t stream) {
    switch (hd) {
        case 16: return bwd<16>(p, sms, stream);
        case 32: return bwd<32>(p, sms, stream);
        case 64: return bwd<64>(p, sms, stream);
        case 128: return bwd<128>(p, sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace na3d
