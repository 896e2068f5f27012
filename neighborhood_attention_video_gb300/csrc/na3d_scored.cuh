// Host/device interface of the score-shaped attention kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace na3d {

struct ScoredParams {
    int32_t B, T, H, W, NH;
    int32_t KT, KH, KW;
    int64_t q_ts, k_ts, v_ts;      // token strides of q, k, v in elements
    int64_t dq_ts, dk_ts, dv_ts;   // and of their gradients
    const uint16_t *q, *k, *v;     // bf16
    uint16_t* out;                 // bf16 (B,T,H,W,NH,HD): written forward, read backward
    float* lse;                    // (B,T,H,W,NH) or null: written forward, read backward
    const uint16_t* dout;          // backward: bf16, as out
    uint16_t *dq, *dk, *dv;
    float2* stat;                  // backward workspace (B,T,H,W,NH): (lse, dout . out)
    float softcap;                 // 0: none
    const float* slopes;           // (NH, 3) or null
    const int32_t* doc;            // (B,T,H,W) or null
    const int32_t* prefix;         // (B) or null
};

// Is there a plan for the forward pass, or for both backward passes? (Sizes,
// the presence of documents and a cap count; host only.)
bool scored_planned(int hd, const ScoredParams& p, bool backward);

cudaError_t launch_scored_fwd(int hd, const ScoredParams& p, int sms, cudaStream_t stream);
cudaError_t launch_scored_bwd(int hd, const ScoredParams& p, int sms, cudaStream_t stream);

// After the work already on `stream`, take (read and clear in one atomic
// step) these kernels' timeout flag, then synchronize `stream`. Nothing is
// done where the process has launched none of them.
cudaError_t take_scored_error(cudaStream_t stream, unsigned int* flag);

}  // namespace na3d
