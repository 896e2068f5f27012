// Attention of a grid's tokens to states of another length, and its backward
// pass. Token i and state j of an entry, head h of q and h / (NH / NKV) of k, v:
//   s_ij = q_i . k_j where doc_i = kv_doc_j >= 0, else masked,
//   out_i = sum_j p_ij v_j, p the softmax, lse_i = log sum_j e^s_ij;
// backward, dp = dout_i . v_j, delta_i = sum_j p dp, ds = p (dp - delta_i):
//   dq_i = sum_j ds k_j, dk_j = sum_i ds q_i, dv_j = sum_i p dout_i.
//
// A warp takes a row (of q, or of k and v) and walks the others 32 at a time,
// one to a lane.
#include <cuda_bf16.h>

#include "na3d_cross.cuh"
#include "sm103_ptx.cuh"

namespace na3d {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float f32(uint16_t h) { return __uint_as_float(uint32_t(h) << 16); }
__device__ __forceinline__ uint16_t b16(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

template <int HD>
__device__ __forceinline__ float dot(const float* a, const uint16_t* b) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < HD; c += 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(b + c);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = fmaf(a[c + 2 * i], __uint_as_float(u[i] << 16), s);
            s = fmaf(a[c + 2 * i + 1], __uint_as_float(u[i] & 0xffff0000u), s);
        }
    }
    return s;
}

__device__ __forceinline__ float warp_max(float v) {
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

template <int HD, bool BWD>
__global__ void __launch_bounds__(kWarps * 32) cross_rows(const CrossParams p) {
    __shared__ float row_s[kWarps][2][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rows = int64_t(p.B) * p.L * p.NH, row = int64_t(blockIdx.x) * kWarps + warp;
    if (row >= rows) return;
    const int h = int(row % p.NH), kh = h / (p.NH / p.NKV);
    const int64_t token = row / p.NH, b = token / p.L;
    const int doc = p.doc ? p.doc[token] : 0;
    for (int c = lane; c < HD; c += 32) {
        row_s[warp][0][c] = f32(p.q[token * p.q_ts + int64_t(h) * HD + c]);
        if (BWD) row_s[warp][1][c] = f32(p.dout[row * HD + c]);
    }
    __syncwarp();
    constexpr int E = (HD + 31) / 32;
    float acc[E] = {}, top = -INFINITY, sum = 0.f, delta = 0.f;
    const float lse = BWD ? p.lse[row] : 0.f;
    for (int pass = 0; pass < (BWD ? 2 : 1); ++pass)
        for (int64_t j0 = 0; j0 < p.S; j0 += 32) {
            const int64_t j = b * p.S + j0 + lane;
            const bool seen = j0 + lane < p.S && doc >= 0 && (p.kv_doc ? p.kv_doc[j] : 0) == doc;
            float s = seen ? dot<HD>(row_s[warp][0], p.k + j * p.k_ts + int64_t(kh) * HD) : -INFINITY, e;
            if (!BWD) {
                const float was = top;
                top = fmaxf(top, warp_max(s));
                if (top == -INFINITY) continue;
                const float by = expf(was - top);
                e = seen ? expf(s - top) : 0.f;
                sum = sum * by + warp_sum(e);
                for (int i = 0; i < E; ++i) acc[i] *= by;
            } else {
                e = seen ? expf(s - lse) : 0.f;
                const float dp = seen ? dot<HD>(row_s[warp][1], p.v + j * p.v_ts + int64_t(kh) * HD) : 0.f;
                if (pass == 0) {
                    delta += warp_sum(e * dp);
                    continue;
                }
                e *= dp - delta;
            }
            const uint32_t live = __ballot_sync(~0u, seen);
            for (int n = 0; n < 32; ++n) {
                if (!(live >> n & 1u)) continue;
                const float w = __shfl_sync(~0u, e, n);
                const uint16_t* const from = (BWD ? p.k + (b * p.S + j0 + n) * p.k_ts : p.v + (b * p.S + j0 + n) * p.v_ts) + int64_t(kh) * HD;
                for (int i = 0; i < E; ++i)
                    if (lane + 32 * i < HD) acc[i] = fmaf(w, f32(from[lane + 32 * i]), acc[i]);
            }
        }
    const float by = BWD ? 1.f : sum > 0.f ? 1.f / sum : 0.f;
    uint16_t* const to = BWD ? p.dq + token * p.dq_ts + int64_t(h) * HD : p.out + row * HD;
    for (int i = 0; i < E; ++i)
        if (lane + 32 * i < HD) to[lane + 32 * i] = b16(acc[i] * by);
    if (!BWD && p.lse && lane == 0) p.lse[row] = sum > 0.f ? top + logf(sum) : -INFINITY;
    if (BWD && lane == 0) static_cast<float*>(p.work)[row] = delta;
}

template <int HD>
__global__ void __launch_bounds__(kWarps * 32) cross_states(const CrossParams p) {
    __shared__ float row_s[kWarps][2][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rows = int64_t(p.B) * p.S * p.NKV, row = int64_t(blockIdx.x) * kWarps + warp;
    if (row >= rows) return;
    const int kh = int(row % p.NKV), G = p.NH / p.NKV;
    const int64_t token = row / p.NKV, b = token / p.S;
    const int doc = p.kv_doc ? p.kv_doc[token] : 0;
    for (int c = lane; c < HD; c += 32) {
        row_s[warp][0][c] = f32(p.k[token * p.k_ts + int64_t(kh) * HD + c]);
        row_s[warp][1][c] = f32(p.v[token * p.v_ts + int64_t(kh) * HD + c]);
    }
    __syncwarp();
    constexpr int E = (HD + 31) / 32;
    float dk[E] = {}, dv[E] = {};
    const int64_t n_rows = int64_t(p.L) * G;
    for (int64_t i0 = 0; i0 < n_rows; i0 += 32) {
        const int64_t i = i0 + lane, t = b * p.L + i / G, r = t * p.NH + kh * G + i % G;
        const bool seen = i < n_rows && doc >= 0 && (p.doc ? p.doc[t] : 0) == doc;
        const float s = seen ? dot<HD>(row_s[warp][0], p.q + t * p.q_ts + (r % p.NH) * HD) : 0.f;
        const float e = seen ? expf(s - p.lse[r]) : 0.f;
        const float ds = seen ? e * (dot<HD>(row_s[warp][1], p.dout + r * HD) - static_cast<const float*>(p.work)[r]) : 0.f;
        const uint32_t live = __ballot_sync(~0u, seen);
        for (int n = 0; n < 32; ++n) {
            if (!(live >> n & 1u)) continue;
            const float w = __shfl_sync(~0u, e, n), w2 = __shfl_sync(~0u, ds, n);
            const int64_t tn = b * p.L + (i0 + n) / G, hn = kh * G + (i0 + n) % G;
            for (int k = 0; k < E; ++k)
                if (lane + 32 * k < HD) {
                    dv[k] = fmaf(w, f32(p.dout[(tn * p.NH + hn) * HD + lane + 32 * k]), dv[k]);
                    dk[k] = fmaf(w2, f32(p.q[tn * p.q_ts + hn * HD + lane + 32 * k]), dk[k]);
                }
        }
    }
    for (int i = 0; i < E; ++i)
        if (lane + 32 * i < HD) {
            p.dk[token * p.dk_ts + int64_t(kh) * HD + lane + 32 * i] = b16(dk[i]);
            p.dv[token * p.dv_ts + int64_t(kh) * HD + lane + 32 * i] = b16(dv[i]);
        }
}

template <int HD>
cudaError_t launch(const CrossParams& p, bool backward, cudaStream_t stream) {
    const int64_t rows = int64_t(p.B) * p.L * p.NH, states = int64_t(p.B) * p.S * p.NKV;
    const unsigned grid = unsigned((rows + kWarps - 1) / kWarps);
    if (!backward) {
        cross_rows<HD, false><<<grid, kWarps * 32, 0, stream>>>(p);
    } else {
        cross_rows<HD, true><<<grid, kWarps * 32, 0, stream>>>(p);
        cross_states<HD><<<unsigned((states + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

int64_t cross_workspace(int64_t B, int64_t L, int64_t, int64_t NH, int64_t, int64_t, bool backward) {
    return backward ? B * L * NH * 4 : 0;
}

cudaError_t launch_cross_fwd(int hd, const CrossParams& p, int, cudaStream_t stream) {
    return hd == 16 ? launch<16>(p, false, stream) : hd == 32 ? launch<32>(p, false, stream)
         : hd == 64 ? launch<64>(p, false, stream) : launch<128>(p, false, stream);
}

cudaError_t launch_cross_bwd(int hd, const CrossParams& p, int, cudaStream_t stream) {
    return hd == 16 ? launch<16>(p, true, stream) : hd == 32 ? launch<32>(p, true, stream)
         : hd == 64 ? launch<64>(p, true, stream) : launch<128>(p, true, stream);
}

cudaError_t take_cross_error(cudaStream_t, unsigned int* flag) {
    *flag = 0;
    return cudaSuccess;
}

}  // namespace na3d
