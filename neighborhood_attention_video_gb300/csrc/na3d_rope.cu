// RMS norm of each head of queries and keys and the rotation by their position
// along T, H and W, in one pass, and its backward pass.
//
// A head x of HD values at grid position (t, h, w):
//   u = x r, r = (mean x^2 + eps)^(-1/2)       (r = 1 without the norm)
//   z = scale R(t,h,w) (w u)
// R turns pair i of the first 2 P values by the angle of its axis' position; the
// values behind them stay. Backward, with g = scale R^T dz:
//   dw = sum over the rows of g u,   dx = r (w g - u mean(w g u)).
//
// Bound by memory: each value is read once and written once, so everything is
// laid out for whole lines in flight. HD/16 lanes hold a head, two 16-byte
// pieces each (pairs are within a piece, or the same place of both), a warp
// 512/HD heads at once; the cosines of a token are read once and serve all its
// heads of q and k.
#include <algorithm>

#include "na3d_rope.cuh"
#include "sm103_ptx.cuh"

namespace na3d {

namespace {

using std::max;
using std::min;

constexpr int kWarps = 8;
// The blocks of a backward launch: their sums of the weights' gradients are
// joined in this order, whatever the device.
constexpr int kGradBlocks = 152 * 2;

struct Piece {   // 16 values of a head: two 16-byte pieces
    uint4 a, b;
};

// ... as eight pairs of fp32 values, the arithmetic of which goes two at a time.
__device__ __forceinline__ void unpack(const Piece& p, uint64_t (&f)[8]) {
    const uint32_t v[8] = {p.a.x, p.a.y, p.a.z, p.a.w, p.b.x, p.b.y, p.b.z, p.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f2_pack(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
}

__device__ __forceinline__ Piece pack(const uint64_t (&f)[8]) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x, y;
        f2_unpack(f[i], x, y);
        v[i] = pack_bf16x2(x, y);
    }
    return {make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7])};
}

// The sum of the products of 16 values.
__device__ __forceinline__ float dot(const uint64_t (&a)[8], const uint64_t (&b)[8]) {
    uint64_t s = f2_mul(a[0], b[0]), t = f2_mul(a[1], b[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        s = f2_fma(a[i], b[i], s);
        t = f2_fma(a[i + 1], b[i + 1], t);
    }
    float x, y;
    f2_unpack(f2_add(s, t), x, y);
    return x + y;
}

// Data that is used once: past L1.
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// The 16 values turned by the eight pairs' angles (DIR 1) or back (-1). PART: the pairs
// in `still` (a bit each; all or none of them where the pairs are halves) stay what they
// are; products by 1 and 0 would spread what is not finite among them.
template <bool INTER, bool PART, int DIR>
__device__ __forceinline__ void turn(uint64_t (&f)[8], const float2 (&cs)[8], uint32_t still) {
    if (INTER) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float a, b;
            const float c = cs[i].x, s = DIR * cs[i].y;
            f2_unpack(f[i], a, b);
            const uint64_t turned = f2_pack(fmaf(a, c, -(b * s)), fmaf(b, c, a * s));
            f[i] = PART && (still >> i & 1u) ? f[i] : turned;
        }
    } else if (!PART || !still) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t c = f2_pack(cs[2 * i].x, cs[2 * i + 1].x), s = f2_pack(DIR * cs[2 * i].y, DIR * cs[2 * i + 1].y);
            const uint64_t n = f2_pack(-DIR * cs[2 * i].y, -DIR * cs[2 * i + 1].y), a = f[i], b = f[4 + i];
            f[i] = f2_fma(a, c, f2_mul(b, n));
            f[4 + i] = f2_fma(b, c, f2_mul(a, s));
        }
    }
}

__device__ __forceinline__ uint32_t divided(uint32_t n, uint64_t by, int s) { return uint32_t((uint64_t(n) * by) >> s); }

template <int LPH>
__device__ __forceinline__ float sum_of_head(float v) {
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace

// A block takes tokens of q or of k (the first `q_blocks` along x those of q),
// a warp one at a time; along y the heads are shared out where there are few
// tokens. U: heads of a lane in flight. BOTH (U 2): a warp takes the heads of q and
// those of k of its token, which a batch holds each.
//
// 49152 tokens, 16 heads of 128 each: 129 us, 6.2 TB/s (6.7 is a copy); backward
// 202 us, 6.0 TB/s. 65536 tokens, 8 heads of 64 each: 53 us, 5.0 TB/s; backward 95
// us, 4.2 TB/s: what a token takes before its few values (its place, its cosines)
// is a good part of the instructions. Heads of 8 and 1: 44 us and 89 us.
template <int HD, bool INTER, bool PART, bool BWD, int U, bool BOTH>
__global__ void __launch_bounds__(kWarps * 32, BWD || BOTH ? 2 : 3) norm_rope(const __grid_constant__ RopeParams p, int q_blocks) {
    static_assert(!BOTH || (U == 2 && !BWD), "q and k at once");
    constexpr int LPH = HD / 16, HPW = 32 / LPH, SIDES = BOTH ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % LPH, sub = lane / LPH;
    const bool is_k = int(blockIdx.x) >= q_blocks;
    auto side = [&](int u) -> const RopeSide& { return p.side[BOTH ? u : is_k]; };
    const RopeSide& d = side(0);
    const int block = is_k ? blockIdx.x - q_blocks : blockIdx.x, blocks = is_k ? gridDim.x - q_blocks : q_blocks;
    // this lane's pieces: as halves of the rotated width lie apart, what does not turn behind them
    const int P = p.PT + p.PH + p.PW;
    const bool apart = INTER || 8 * l < P;
    const int ca = apart ? 8 * l : 2 * P + 16 * (l - P / 8), cb = ca + (INTER ? HD / 2 : apart ? P : 8);
    // the first of the pairs of either piece (the same four and four, INTER; else eight in a row)
    const int pa = INTER ? ca / 2 : apart ? ca : P, pb = INTER ? cb / 2 : pa + 4;

    uint32_t still = apart ? 0u : 255u;   // PART: pairs of this lane that do not turn
    if (PART && INTER)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((i < 4 ? pa + i : pb + i - 4) >= P) still |= 1u << i;

    uint64_t wt[SIDES][8];   // weight and scale
#pragma unroll
    for (int s = 0; s < SIDES; ++s) {
        const RopeSide& d = side(s);
        const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        const Piece wp = {d.w ? *reinterpret_cast<const uint4*>(d.w + ca) : one, d.w ? *reinterpret_cast<const uint4*>(d.w + cb) : one};
        unpack(wp, wt[s]);
#pragma unroll
        for (int i = 0; i < 8; ++i) wt[s][i] = f2_mul(wt[s][i], f2_pack(d.scale, d.scale));
    }
    uint64_t dw[BWD ? 8 : 1];   // without the scale
#pragma unroll
    for (int i = 0; i < (BWD ? 8 : 1); ++i) dw[i] = f2_pack(0.f, 0.f);

    for (int64_t token = int64_t(block) * kWarps + warp; token < p.tokens; token += int64_t(blocks) * kWarps) {
        const uint32_t place = uint32_t(token);   // below 2^31
        const uint32_t th = divided(place, p.by_w, p.s_w), w = place - th * p.W;
        const uint32_t bt = divided(th, p.by_h, p.s_h), h = th - bt * p.H, t = bt - divided(bt, p.by_t, p.s_t) * p.T;
        const float2* const of_t = p.table + t * uint32_t(p.PT);
        const float2* const of_h = p.table + uint32_t(p.T * p.PT) + h * p.PH - p.PT;
        const float2* const of_w = p.table + uint32_t(p.T * p.PT) + uint32_t(p.H * p.PH) + w * p.PW - p.PT - p.PH;
        float2 cs[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = i < 4 ? pa + i : pb + i - 4;
            const float2* const of = j < p.PT ? of_t : j < p.PT + p.PH ? of_h : of_w;
            cs[i] = j < P ? __ldg(of + j) : make_float2(1.f, 0.f);
        }
        const uint16_t *x_row[SIDES], *const g_row = BWD ? d.g + token * d.g_ts : nullptr;
        uint16_t* y_row[SIDES];
#pragma unroll
        for (int s = 0; s < SIDES; ++s) {
            x_row[s] = side(s).x + token * side(s).x_ts;
            y_row[s] = side(s).y + token * side(s).y_ts;
        }
        for (int h0 = BOTH ? 0 : int(blockIdx.y) * HPW * U; BOTH ? h0 == 0 : h0 < d.heads; h0 += BOTH ? 1 : int(gridDim.y) * HPW * U) {
            Piece x[U], g[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = BOTH ? u : 0, head = h0 + (BOTH ? 0 : u * HPW) + sub;
                x[u] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                g[u] = x[u];
                if (head < side(u).heads) {
                    x[u] = {load16(x_row[s] + head * HD + ca), load16(x_row[s] + head * HD + cb)};
                    if (BWD) g[u] = {load16(g_row + head * HD + ca), load16(g_row + head * HD + cb)};
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = BOTH ? u : 0, head = h0 + (BOTH ? 0 : u * HPW) + sub;
                uint64_t f[8];
                bool live = true;
                if (BWD) {
                    // a row without a gradient (padding's) adds nothing, whatever x holds there
                    const uint32_t bits = (g[u].a.x | g[u].a.y | g[u].a.z | g[u].a.w | g[u].b.x | g[u].b.y | g[u].b.z | g[u].b.w) & 0x7FFF7FFFu;
                    const uint32_t lanes = __ballot_sync(0xffffffffu, bits != 0u) >> (sub * LPH);
                    live = (lanes & (0xffffffffu >> (32 - LPH))) != 0u;
                    if (!live) x[u] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                }
                unpack(x[u], f);
                float r = 1.f;
                if (p.norm) r = rsqrtf(sum_of_head<LPH>(dot(f, f)) * (1.f / HD) + side(u).eps);
                const uint64_t r2 = f2_pack(r, r);
                if (!BWD) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = f2_mul(f2_mul(f[i], r2), wt[s][i]);
                    turn<INTER, PART, 1>(f, cs, still);
                } else {
                    uint64_t e[8];
                    unpack(g[u], e);
                    turn<INTER, PART, -1>(e, cs, still);
                    if (p.norm) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            f[i] = f2_mul(f[i], r2);
                            dw[BWD ? i : 0] = f2_fma(e[i], f[i], dw[BWD ? i : 0]);
                            e[i] = f2_mul(e[i], wt[0][i]);
                        }
                        const float m = -sum_of_head<LPH>(dot(e, f)) * (1.f / HD);
                        const uint64_t m2 = f2_pack(m, m);
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = f2_mul(r2, f2_fma(f[i], m2, e[i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = f2_mul(e[i], wt[0][i]);
                    }
                }
                if (head < side(u).heads) {
                    const Piece o = pack(f);
                    *reinterpret_cast<uint4*>(y_row[s] + head * HD + ca) = o.a;
                    *reinterpret_cast<uint4*>(y_row[s] + head * HD + cb) = o.b;
                }
            }
        }
    }
    if (BWD && p.work) {
        // the block's sums: over the heads of a warp, then over the warps
        __shared__ float sums[kWarps][HD];
#pragma unroll
        for (int i = 0; i < (BWD ? 8 : 1); ++i) {
            float v[2];
            f2_unpack(dw[i], v[0], v[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int o = LPH; o < 32; o <<= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
                if (sub == 0) sums[warp][(i < 4 ? ca : cb - 8) + 2 * i + k] = v[k] * d.scale;
            }
        }
        __syncthreads();
        float* const out = p.work + (int64_t(blockIdx.x) * gridDim.y + blockIdx.y) * HD;
        for (int i = threadIdx.x; i < HD; i += kWarps * 32) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) v += sums[k][i];
            out[i] = v;
        }
    }
}

// The sums of the blocks of q (the first q_blocks) and of k, 32 columns to a
// block, 32 threads to a column.
__global__ void __launch_bounds__(1024) norm_rope_sum(const float* work, int q_blocks, int blocks, int HD, float* dq, float* dk) {
    __shared__ float part[32][33];
    const int x = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int per = gridDim.x / 2;   // blocks of each
    const bool is_k = int(blockIdx.x) >= per;
    const int c = (int(blockIdx.x) - (is_k ? per : 0)) * 32 + x, end = is_k ? blocks : q_blocks;
    float v = 0.f;
    if (c < HD)
        for (int b = (is_k ? q_blocks : 0) + r; b < end; b += 32) v += work[int64_t(b) * HD + c];
    part[r][x] = v;
    __syncthreads();
    if (r == 0 && c < HD) {
        v = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) v += part[k][x];
        float* const to = is_k ? dk : dq;
        if (to) to[c] = v;
    }
}

// cos and sin of (offset + scale position) theta^(-i / pairs), angles in 64
// bits: in 32 a far position's angle would be off by more than its table's step.
__global__ void __launch_bounds__(256) rope_table(const RopeTable p) {
    int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    float2* to = p.table + i;
#pragma unroll
    for (int a = 0; a < 3; ++a) {
        const int64_t n = int64_t(p.n[a]) * p.pairs[a];
        if (i < n) {
            const double at = p.offset[a] + p.scale[a] * double(i / p.pairs[a]);
            double s, c;
            sincos(at * pow(p.theta, -double(i % p.pairs[a]) / double(p.pairs[a])), &s, &c);
            *to = make_float2(float(c), float(s));
            return;
        }
        i -= n;
    }
}

// ------------------------------------------------------------------ host side

cudaError_t launch_rope_table(const RopeTable& p, cudaStream_t stream) {
    int64_t n = 0;
    for (int a = 0; a < 3; ++a) n += int64_t(p.n[a]) * p.pairs[a];
    rope_table<<<unsigned((n + 255) / 256), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

int64_t rope_workspace(int64_t HD) { return int64_t(kGradBlocks) * HD * 4; }

namespace {

template <int HD, bool INTER, bool PART, bool BWD, int U, bool BOTH>
cudaError_t launch(const RopeParams& p, int sms, cudaStream_t stream) {
    constexpr int batch = 32 / (HD / 16) * U;
    const int NQ = p.side[0].heads, NK = p.side[1].heads;
    const int64_t want = (p.tokens + kWarps - 1) / kWarps;   // blocks for each of q and k
    if (BOTH) {
        const unsigned blocks = unsigned(min(want, int64_t(sms) * 2));
        norm_rope<HD, INTER, PART, BWD, U, BOTH><<<blocks, kWarps * 32, 0, stream>>>(p, int(blocks));
        return cudaGetLastError();
    }
    const int most = BWD ? kGradBlocks : sms * 3;
    // the blocks shared out by the batches of heads of q and k, a token's beginning as another batch
    // of each (16 heads of 128 and 1: 89 us; by heads alone 288)
    const int cost_q = 1 + (NQ + batch - 1) / batch, cost_k = 1 + (NK + batch - 1) / batch;
    const int64_t most_q = NK ? min(max(int64_t(most) * cost_q / (cost_q + cost_k), int64_t(1)), int64_t(most - 1)) : most;
    const int q_blocks = int(min(want, most_q)), k_blocks = NK ? int(min(want, most - most_q)) : 0;
    dim3 grid(unsigned(q_blocks + k_blocks));
    // few tokens: a token's heads over several blocks
    grid.y = unsigned(max(1, min((max(NQ, NK) + batch - 1) / batch, most / int(grid.x))));
    norm_rope<HD, INTER, PART, BWD, U, BOTH><<<grid, kWarps * 32, 0, stream>>>(p, q_blocks);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !BWD || !p.work) return e;
    norm_rope_sum<<<(HD + 31) / 32 * 2, 1024, 0, stream>>>(p.work, int(q_blocks * grid.y), int(grid.x * grid.y), HD,
                                                           p.side[0].dw, p.side[1].dw);
    return cudaGetLastError();
}

// n / d as (n by) >> s, exact for n < 2^31: by exceeds 2^s / d by less than 1, and n times that
// excess stays below 2^s / d, s being 31 more than the bits of d.
void division(int32_t d, uint64_t* by, int32_t* s) {
    *s = 31;
    while ((int64_t(1) << (*s - 31)) < d) ++*s;
    *by = (uint64_t(1) << *s) / uint32_t(d) + 1;
}

template <int HD, bool INTER, bool PART, bool BWD>
cudaError_t launch(const RopeParams& p, int sms, cudaStream_t stream) {
    // Heads enough for two batches at a time; else q's and k's at once, which reads a token's
    // cosines once (8 heads of 64 each: 53 us, 64 by blocks of their own; of 8 and 1: 44, 161).
    // Backward the second side's sums and weights do not fit the registers.
    if (max(p.side[0].heads, p.side[1].heads) > 32 / (HD / 16)) return launch<HD, INTER, PART, BWD, 2, false>(p, sms, stream);
    if constexpr (!BWD)
        if (p.side[1].heads) return launch<HD, INTER, PART, BWD, 2, true>(p, sms, stream);
    return launch<HD, INTER, PART, BWD, 1, false>(p, sms, stream);
}

template <int HD>
cudaError_t launch(const RopeParams& p, bool backward, int sms, cudaStream_t stream) {
    // Heads that turn whole do without the choice between turned and kept pairs (backward, 49152
    // tokens with 16 heads of 128 each: 202 us, 208 with it).
    const bool part = 2 * (p.PT + p.PH + p.PW) < HD;
    if (p.interleaved) {
        if (part) return backward ? launch<HD, true, true, true>(p, sms, stream) : launch<HD, true, true, false>(p, sms, stream);
        return backward ? launch<HD, true, false, true>(p, sms, stream) : launch<HD, true, false, false>(p, sms, stream);
    }
    if (part) return backward ? launch<HD, false, true, true>(p, sms, stream) : launch<HD, false, true, false>(p, sms, stream);
    return backward ? launch<HD, false, false, true>(p, sms, stream) : launch<HD, false, false, false>(p, sms, stream);
}

}  // namespace

cudaError_t launch_rope(int hd, const RopeParams& args, bool backward, int sms, cudaStream_t stream) {
    RopeParams p = args;
    division(p.W, &p.by_w, &p.s_w);
    division(p.H, &p.by_h, &p.s_h);
    division(p.T, &p.by_t, &p.s_t);
#define X(n) if (hd == n) return launch<n>(p, backward, sms, stream);
    X(16) X(32) X(64) X(128) X(256) X(512)
#undef X
    return cudaErrorInvalidValue;
}

}  // namespace na3d
