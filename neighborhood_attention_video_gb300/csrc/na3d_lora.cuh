// Host/device interface of the projection with adapters.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace na3d {

struct LoraParams {
    int32_t M, C, N, Nq;         // tokens, channels, 3*NH*HD, NH*HD
    int32_t R, n_req, n_ad;      // rank, requests, adapters
    float q_scale;               // HD^-0.5, of the q block
    const uint16_t *x, *w, *bias;      // bf16 (M,C), (N,C), (N) or null
    const uint16_t *a, *b;             // bf16 (n_ad,R,C), (n_ad,N,R)
    const float* scaling;              // (n_ad)
    const int32_t *offsets, *adapter;  // (n_req+1), (n_req)
    uint16_t* qkv;                     // bf16 (M,N): output
    const uint16_t* dqkv;              // backward: bf16 (M,N)
    uint16_t *dx, *da, *db;            // backward outputs: (M,C) or null, as a, as b
    void* work;
};

// Bytes of workspace a forward or backward call uses.
int64_t lora_workspace(int64_t M, int64_t C, int64_t N, int64_t R, int64_t n_req, int64_t n_ad, bool backward);

cudaError_t launch_lora_fwd(const LoraParams& p, int sms, cudaStream_t stream);
cudaError_t launch_lora_bwd(const LoraParams& p, int sms, cudaStream_t stream);

// After the work already on `stream`, take (read and clear in one atomic
// step) these kernels' timeout flag, then synchronize `stream`. Nothing is
// done where the process has launched none of them.
cudaError_t take_lora_error(cudaStream_t stream, unsigned int* flag);

}  // namespace na3d
