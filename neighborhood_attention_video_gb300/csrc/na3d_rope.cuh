// Host/device interface of the norm and rotation of queries and keys.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace na3d {

// One of the two tensors of a call, tokens of `heads` heads.
struct RopeSide {
    const uint16_t* x;   // bf16, x_ts elements from token to token
    const uint16_t* g;   // backward: the gradient of the output, g_ts
    uint16_t* y;         // the output (backward: the gradient of x), y_ts
    const uint16_t* w;   // bf16 (HD) or null
    float* dw;           // backward: fp32 (HD) or null
    int64_t x_ts, g_ts, y_ts;
    int32_t heads;
    float eps, scale;
};

struct RopeParams {
    RopeSide side[2];         // q, k (no heads: none)
    const float2* table;      // cos and sin: (T, PT), (H, PH), (W, PW)
    int64_t tokens;
    int32_t T, H, W;
    int32_t PT, PH, PW;       // pairs that turn with each axis
    int32_t norm, interleaved;
    float* work;              // backward: the blocks' sums of the weights' gradients
    uint64_t by_w, by_h, by_t;   // n / W = (n by_w) >> s_w for n < 2^31, and so on (set by the launch)
    int32_t s_w, s_h, s_t;
};

// Bytes of workspace of the backward pass with gradients of the weights.
int64_t rope_workspace(int64_t HD);

struct RopeTable {
    float2* table;
    int32_t n[3], pairs[3];          // T, H, W and their pairs
    double theta, offset[3], scale[3];
};

cudaError_t launch_rope_table(const RopeTable& p, cudaStream_t stream);
cudaError_t launch_rope(int hd, const RopeParams& p, bool backward, int sms, cudaStream_t stream);

}  // namespace na3d
