// ttt_join.cuh -- problem description of the join between two blocks (ttt_join.cu).
#pragma once

#include "ttt_common.cuh"

namespace ttt {

struct JoinArgs {
    const void *X, *Z, *gate;  // [B][T][D], [B][H][T][d] (NULL: the norm of X alone), [B][T][D] or NULL
    const float *scale, *gamma1, *beta1, *gamma2, *beta2;  // [D] each, or NULL
    void *R, *Hn;              // [B][T][D]; Hn may be NULL
    int B, H, T, d;
    float eps;
    bool bf16, z_bf16, rms, silu;
};

struct JoinBwdArgs {
    const void *R, *Z, *gate;
    const float *scale, *gamma1, *beta1, *gamma2;
    const float *dR, *dH;      // [B][T][D] fp32, either may be NULL
    float *dX, *dZ, *dGate;
    float *dscale, *dgamma1, *dbeta1, *dgamma2, *dbeta2;  // [D] each, NULL: not stored
    float *partials;           // workspace
    int B, H, T, d;
    float eps;
    bool bf16, z_bf16, rms, silu;
};

bool join_supported(int H, int d);
size_t join_bwd_workspace_bytes(int B, int H, int T, int d);
cudaError_t launch_join_fwd(const JoinArgs &a, cudaStream_t s);
cudaError_t launch_join_bwd(const JoinBwdArgs &a, cudaStream_t s);

}  // namespace ttt
