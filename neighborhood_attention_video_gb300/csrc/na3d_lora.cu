// The QKV projection with low-rank adapters of many requests, and its
// backward pass.
//
// Rows offsets[r] .. offsets[r+1] - 1 are request r's, with adapter
// a = adapter[r] (none where the id is not in 0 .. n_ad - 1):
//   t = scaling_a x A_a^T                     (rank R, fp32 sums)
//   qkv = s_n (x W^T + bias + t B_a^T)        (s_n = HD^-0.5 in the q block, else 1)
// Backward, with g = s_n dqkv:
//   u = scaling_a g B_a,  dx = g W + u A_a,
//   dA_a = sum over the adapter's rows of u^T x,  dB_a = sum of g^T t.
// The base weight and the scalings are frozen: they get no gradient.
#include <cuda_bf16.h>

#include "na3d_lora.cuh"

namespace na3d {

namespace {

__device__ __forceinline__ float f32(uint16_t h) { return __uint_as_float(uint32_t(h) << 16); }
__device__ __forceinline__ uint16_t b16(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// The adapter of a row, -1 for none: the last request that starts at or
// before the row, where it reaches that far.
__device__ __forceinline__ int adapter_of(const LoraParams& p, int m) {
    int lo = 0, hi = p.n_req;   // requests [0, lo) start at or before m
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.offsets[mid] <= m) lo = mid + 1;
        else hi = mid;
    }
    if (lo == 0 || m >= p.offsets[lo]) return -1;
    const int a = p.adapter[lo - 1];
    return a >= 0 && a < p.n_ad ? a : -1;
}

// t (from x and A) or u (from g and B) of every row: a warp per row.
template <bool BWD>
__global__ void __launch_bounds__(256) lora_down(const LoraParams p, float* t) {
    const int lane = threadIdx.x & 31;
    for (int m = blockIdx.x * 8 + (threadIdx.x >> 5); m < p.M; m += gridDim.x * 8) {
        const int a = adapter_of(p, m);
        for (int r = 0; r < p.R; ++r) {
            float s = 0.f;
            if (a >= 0 && !BWD) {
                const uint16_t *x = p.x + int64_t(m) * p.C, *ar = p.a + (int64_t(a) * p.R + r) * p.C;
                for (int c = lane; c < p.C; c += 32) s = fmaf(f32(x[c]), f32(ar[c]), s);
            } else if (a >= 0) {
                const uint16_t *g = p.dqkv + int64_t(m) * p.N, *br = p.b + int64_t(a) * p.N * p.R + r;
                for (int n = lane; n < p.N; n += 32)
                    s = fmaf(f32(g[n]) * (n < p.Nq ? p.q_scale : 1.f), f32(br[int64_t(n) * p.R]), s);
            }
#pragma unroll
            for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
            if (lane == 0) t[int64_t(m) * p.R + r] = a >= 0 ? s * p.scaling[a] : 0.f;
        }
    }
}

// A 64 x 64 tile of sum_k a(i, k) b(j, k), 4 x 4 values a thread.
template <class FA, class FB>
__device__ __forceinline__ void tile_product(FA fa, FB fb, int i0, int j0, int I, int J, int K, float (&acc)[4][4]) {
    __shared__ float sa[16][65], sb[16][65];
    const int ti = threadIdx.x >> 4, tj = threadIdx.x & 15;
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int e = threadIdx.x; e < 64 * 16; e += 256) {
            const int i = e >> 4, k = e & 15;
            sa[k][i] = i0 + i < I && k0 + k < K ? fa(i0 + i, k0 + k) : 0.f;
            sb[k][i] = j0 + i < J && k0 + k < K ? fb(j0 + i, k0 + k) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ti * 4 + i], sb[k][tj * 4 + j], acc[i][j]);
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256) lora_fwd_tile(const LoraParams p, const float* t) {
    float acc[4][4] = {};
    const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    tile_product([&](int m, int c) { return f32(p.x[int64_t(m) * p.C + c]); },
                 [&](int n, int c) { return f32(p.w[int64_t(n) * p.C + c]); }, i0, j0, p.M, p.N, p.C, acc);
    for (int i = 0; i < 4; ++i) {
        const int m = i0 + (threadIdx.x >> 4) * 4 + i;
        if (m >= p.M) break;
        const int a = adapter_of(p, m);
        for (int j = 0; j < 4; ++j) {
            const int n = j0 + (threadIdx.x & 15) * 4 + j;
            if (n >= p.N) break;
            float s = acc[i][j] + (p.bias ? f32(p.bias[n]) : 0.f);
            for (int r = 0; a >= 0 && r < p.R; ++r)
                s = fmaf(t[int64_t(m) * p.R + r], f32(p.b[(int64_t(a) * p.N + n) * p.R + r]), s);
            p.qkv[int64_t(m) * p.N + n] = b16(s * (n < p.Nq ? p.q_scale : 1.f));
        }
    }
}

__global__ void __launch_bounds__(256) lora_dx_tile(const LoraParams p, const float* u) {
    float acc[4][4] = {};
    const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    tile_product([&](int m, int n) { return f32(p.dqkv[int64_t(m) * p.N + n]) * (n < p.Nq ? p.q_scale : 1.f); },
                 [&](int c, int n) { return f32(p.w[int64_t(n) * p.C + c]); }, i0, j0, p.M, p.C, p.N, acc);
    for (int i = 0; i < 4; ++i) {
        const int m = i0 + (threadIdx.x >> 4) * 4 + i;
        if (m >= p.M) break;
        const int a = adapter_of(p, m);
        for (int j = 0; j < 4; ++j) {
            const int c = j0 + (threadIdx.x & 15) * 4 + j;
            if (c >= p.C) break;
            float s = acc[i][j];
            for (int r = 0; a >= 0 && r < p.R; ++r)
                s = fmaf(u[int64_t(m) * p.R + r], f32(p.a[(int64_t(a) * p.R + r) * p.C + c]), s);
            p.dx[int64_t(m) * p.C + c] = b16(s);
        }
    }
}

// dA[a][r][c] and dB[a][n][r]: a thread per value, over the rows of every
// request with the adapter, in their order.
template <bool B>
__global__ void __launch_bounds__(256) lora_dab(const LoraParams p, const float* tu) {
    const int64_t per = int64_t(p.R) * (B ? p.N : p.C);
    const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= per * p.n_ad) return;
    const int a = int(e / per);
    const int64_t f = e % per;
    const int r = B ? int(f % p.R) : int(f / p.C), c = B ? int(f / p.R) : int(f % p.C);
    float s = 0.f;
    for (int q = 0; q < p.n_req; ++q) {
        if (p.adapter[q] != a) continue;
        const int m1 = min(p.M, p.offsets[q + 1]);
        for (int m = max(0, p.offsets[q]); m < m1; ++m)
            s = fmaf(tu[int64_t(m) * p.R + r], f32(B ? p.dqkv[int64_t(m) * p.N + c] : p.x[int64_t(m) * p.C + c]), s);
    }
    if (B && c < p.Nq) s *= p.q_scale;
    (B ? p.db : p.da)[e] = b16(s);
}

unsigned ceil_div(int64_t a, int64_t b) { return unsigned((a + b - 1) / b); }

}  // namespace

int64_t lora_workspace(int64_t M, int64_t, int64_t, int64_t R, int64_t, int64_t, bool backward) {
    return M * R * 4 * (backward ? 2 : 1);
}

cudaError_t launch_lora_fwd(const LoraParams& p, int sms, cudaStream_t stream) {
    float* t = static_cast<float*>(p.work);
    lora_down<false><<<sms * 8, 256, 0, stream>>>(p, t);
    lora_fwd_tile<<<dim3(ceil_div(p.N, 64), ceil_div(p.M, 64)), 256, 0, stream>>>(p, t);
    return cudaGetLastError();
}

cudaError_t launch_lora_bwd(const LoraParams& p, int sms, cudaStream_t stream) {
    float *t = static_cast<float*>(p.work), *u = t + int64_t(p.M) * p.R;
    lora_down<false><<<sms * 8, 256, 0, stream>>>(p, t);
    lora_down<true><<<sms * 8, 256, 0, stream>>>(p, u);
    if (p.dx) lora_dx_tile<<<dim3(ceil_div(p.C, 64), ceil_div(p.M, 64)), 256, 0, stream>>>(p, u);
    lora_dab<false><<<ceil_div(int64_t(p.n_ad) * p.R * p.C, 256), 256, 0, stream>>>(p, u);
    lora_dab<true><<<ceil_div(int64_t(p.n_ad) * p.R * p.N, 256), 256, 0, stream>>>(p, t);
    return cudaGetLastError();
}

}  // namespace na3d
