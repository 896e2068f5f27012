// Host/device interface of the attention to states of another length.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace na3d {

struct CrossParams {
    int32_t B, L, S, NH, NKV;        // entries, tokens and states of an entry, heads of q and of k
    int64_t q_ts, k_ts, v_ts, dq_ts, dk_ts, dv_ts;   // elements from token to token
    const uint16_t *q, *k, *v;       // bf16
    uint16_t* out;                   // bf16 (B, L, NH, HD)
    float* lse;                      // fp32 (B, L, NH) or null
    const uint16_t* dout;            // backward
    uint16_t *dq, *dk, *dv;
    const int32_t *doc, *kv_doc;     // (B, L), (B, S) or null: all 0
    void* work;
    bool withhold;                   // self-test: of each row tile's last token nothing is loaded, which its wait misses
};

// Bytes of workspace a forward or backward call uses.
int64_t cross_workspace(int64_t B, int64_t L, int64_t S, int64_t NH, int64_t NKV, int64_t HD, bool backward);

cudaError_t launch_cross_fwd(int hd, const CrossParams& p, int sms, cudaStream_t stream);
cudaError_t launch_cross_bwd(int hd, const CrossParams& p, int sms, cudaStream_t stream);

// After the work already on `stream`, take (read and clear in one atomic
// step) these kernels' timeout flag, then synchronize `stream`. Nothing is
// done where the process has launched none of them.
cudaError_t take_cross_error(cudaStream_t stream, unsigned int* flag);

}  // namespace na3d
