// ttt_delta.cuh -- what the gated delta rule's sources share: the problem
// description and the lay-out of packed sequences.
//
// The rule, per sequence and value head, row form, W [dk][dv] fp32:
//   Wd = exp(g_t) W,  rho_t = v_t - k_t Wd,  W = Wd + eta_t k_t^T rho_t,  z_t = c q_t W.
#pragma once

#include "ttt_common.cuh"

namespace ttt {

struct DeltaArgs {
    const void *Q, *K, *V;         // [B][Hk][T][dk], [B][Hk][T][dk], [B][H][T][dv]
    const float *eta, *g, *W0;     // [B][H][T], [B][H][T] or NULL (no decay), W0 or NULL (zero)
    void *Z;                       // [B][H][T][dv], fp32 or bf16
    float *W_out;                  // [N][H][dk][dv] or NULL
    const int *seq_start;          // [N + 1] on the device (packed, B == 1), or NULL
    int B, Hk, H, T, dk, dv, N;    // N sequences: B, or the packed ones
    float q_scale;
    bool bf16, w0_per_seq, z_bf16;
    void *workspace;
};

struct DeltaBwdArgs {
    DeltaArgs f;                   // the forward's inputs (Z, W_out unused)
    const float *dZ, *dW_out;      // [B][H][T][dv]; [N][H][dk][dv] or NULL
    float *dQ, *dK, *dV, *deta, *dg, *dW0;  // dg NULL without g, dW0 NULL without W0
};

constexpr int kDeltaC = 64;  // tokens per chunk of the chunked kernels

// First token and length of sequence n inside its batch row. The offsets live
// on the device, where the host cannot check them, so they are clamped: an
// offset outside [0, T], or one that runs backwards, never leads a kernel out
// of its arrays.
__host__ __device__ __forceinline__ void delta_span(const int *seq_start, int n, int T, int &t0,
                                                    int &len) {
    t0 = 0;
    len = T;
    if (seq_start) {
        int a = seq_start[n], b = seq_start[n + 1];
        a = a < 0 ? 0 : (a > T ? T : a);
        b = b < a ? a : (b > T ? T : b);
        t0 = a;
        len = b - a;
    }
}

bool delta_supported(int dk, int dv);
size_t delta_workspace_bytes(int B, int Hk, int H, int T, int dk, int dv, int N, bool packed,
                             bool bf16);
cudaError_t launch_delta_fwd(const DeltaArgs &a, cudaStream_t s);
size_t delta_bwd_workspace_bytes(int B, int Hk, int H, int T, int dk, int dv, int N, bool packed,
                                 bool bf16);
cudaError_t launch_delta_bwd(const DeltaBwdArgs &a, cudaStream_t s);

// Token-by-token kernel (ttt_delta.cu): the forward of at most 24 tokens, and
// decode of n tokens per row with the states in a pool.
cudaError_t launch_delta_recurrent(const DeltaArgs &a, cudaStream_t s);
cudaError_t launch_delta_decode(const DeltaArgs &a, float *W, const int *state_index, int n_slots,
                                cudaStream_t s);

}  // namespace ttt
