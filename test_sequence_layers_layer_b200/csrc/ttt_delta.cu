// ttt_delta.cu -- the gated delta rule token by token: decode with the states
// in a pool, and the forward of at most 24 tokens.
//
// Per token, with Wd = a W, a = exp(g): rho = v - k Wd, u = eta rho,
// W = Wd + k^T u, and z = c q W = c (a q W_old + (q.k) u): both products with
// the old weight are taken in one pass over it, so a token costs one
// reduction and one barrier.
// The columns of W are independent of one another. One block of 128 threads
// holds 32 columns of one state in registers for the whole call: thread
// (row group rg = tid / 8, lane quad column c4 = tid % 8) keeps rows
// rg * R .. rg * R + R - 1 (R = dk / 16) of columns 4 c4 .. 4 c4 + 3, loaded and
// stored as 16-byte vectors, every 8 lanes one 128-byte line. For one token the
// call is bound by reading and writing the state (8 dk dv bytes per head): 256
// rows of 16 heads of 128 x 128 take 95 us, 541 MB at 5.7 TB/s. Further tokens
// cost one reduction over the block and a barrier each, 0.4 - 0.8 us, whatever
// the number of rows up to about one block an SM partition; that chain, not
// memory, bounds longer calls, which is why they go chunk by chunk instead.
// Everything is held and added up in fp32; bf16 inputs are exact in it, and only
// a bf16 Z is rounded.
#include "../../include/ttt.h"
#include "ttt_delta.cuh"

namespace ttt {
namespace {

constexpr int kRecThreads = 128, kRecCols = 32;

struct RecArgs {
    const void *Q, *K, *V;
    const float *eta, *g;
    const float *W_in;       // start state, NULL: zero
    float *W_out;            // final state, NULL: not stored
    void *Z;
    const int *seq_start, *state_index;
    int Hk, H, T, dv, n_slots, w_heads;  // w_heads: 0 when W_in is shared by the sequences
    float q_scale;
    bool z_bf16;
};

// R consecutive elements of a row of Q or K.
template <int R>
__device__ __forceinline__ void load_row(float (&x)[R], const void *p, size_t i, bool bf16) {
    if (bf16) {
        const __nv_bfloat16 *b = reinterpret_cast<const __nv_bfloat16 *>(p) + i;
#pragma unroll
        for (int r = 0; r < R; r += 4) {
            const uint2 u = *reinterpret_cast<const uint2 *>(b + r);
            x[r] = __uint_as_float(u.x << 16);
            x[r + 1] = __uint_as_float(u.x & 0xFFFF0000u);
            x[r + 2] = __uint_as_float(u.y << 16);
            x[r + 3] = __uint_as_float(u.y & 0xFFFF0000u);
        }
    } else {
        const float *f = reinterpret_cast<const float *>(p) + i;
#pragma unroll
        for (int r = 0; r < R; r += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(f + r);
            x[r] = u.x;
            x[r + 1] = u.y;
            x[r + 2] = u.z;
            x[r + 3] = u.w;
        }
    }
}

template <int DK, bool BF16>
__global__ void __launch_bounds__(kRecThreads) delta_recurrent_kernel(RecArgs a) {
    constexpr int R = DK / 16;
    // per warp and token parity: k W (32 columns), q W (32 columns), q.k
    __shared__ float4 part[2][4][17];
    const int slices = a.dv / kRecCols;
    const int sl = blockIdx.x % slices, sh = blockIdx.x / slices;
    const int n = sh / a.H, h = sh % a.H;
    const int tid = threadIdx.x, warp = tid >> 5, rg = tid >> 3, c4 = tid & 7;

    long long slot = n;
    if (a.state_index) {
        slot = a.state_index[n];
        if (slot < 0 || slot >= a.n_slots) return;  // a padding row: nothing of it is touched
    }
    int t0, len;
    delta_span(a.seq_start, n, a.T, t0, len);
    const int b = a.seq_start ? 0 : n;
    const int col = sl * kRecCols + 4 * c4;
    const size_t hrow = ((size_t)b * a.H + h) * a.T + t0;
    const size_t krow = ((size_t)b * a.Hk + h / (a.H / a.Hk)) * a.T + t0;

    const size_t wrow = (size_t)(rg * R) * a.dv + col;
    const size_t state = (size_t)DK * a.dv;
    float4 W[R];
    if (a.W_in) {
        const float *w = a.W_in + ((a.w_heads ? slot * a.w_heads : 0) + h) * state + wrow;
#pragma unroll
        for (int r = 0; r < R; ++r) W[r] = *reinterpret_cast<const float4 *>(w + (size_t)r * a.dv);
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) W[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    float kn[R], qn[R], vn[4], en = 0.f, gn = 0.f;
    auto fetch = [&](int t) {
        load_row<R>(kn, a.K, (krow + t) * DK + rg * R, BF16);
        load_row<R>(qn, a.Q, (krow + t) * DK + rg * R, BF16);
        load_row<4>(vn, a.V, (hrow + t) * a.dv + col, BF16);
        en = a.eta[hrow + t];
        gn = a.g ? a.g[hrow + t] : 0.f;
    };
    if (len > 0) fetch(0);
    for (int t = 0; t < len; ++t) {
        float k[R], q[R], v[4];
#pragma unroll
        for (int r = 0; r < R; ++r) k[r] = kn[r], q[r] = qn[r];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = vn[c];
        const float eta = en, al = expf(gn);
        if (t + 1 < len) fetch(t + 1);

        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        float qk = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x.x = fmaf(k[r], W[r].x, x.x);
            x.y = fmaf(k[r], W[r].y, x.y);
            x.z = fmaf(k[r], W[r].z, x.z);
            x.w = fmaf(k[r], W[r].w, x.w);
            y.x = fmaf(q[r], W[r].x, y.x);
            y.y = fmaf(q[r], W[r].y, y.y);
            y.z = fmaf(q[r], W[r].z, y.z);
            y.w = fmaf(q[r], W[r].w, y.w);
            qk = fmaf(q[r], k[r], qk);
        }
        // the four row groups of the warp, then the four warps
#pragma unroll
        for (int o = 8; o <= 16; o <<= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
            x.z += __shfl_xor_sync(0xffffffffu, x.z, o);
            x.w += __shfl_xor_sync(0xffffffffu, x.w, o);
            y.x += __shfl_xor_sync(0xffffffffu, y.x, o);
            y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, o);
            y.w += __shfl_xor_sync(0xffffffffu, y.w, o);
            qk += __shfl_xor_sync(0xffffffffu, qk, o);
        }
        // two buffers in turn: a thread that writes token t + 2's sums has
        // passed token t + 1's barrier, behind which token t's are read
        float4(*p)[17] = part[t & 1];
        if ((tid & 31) < 8) {
            p[warp][c4] = x;
            p[warp][8 + c4] = y;
            if (c4 == 0) p[warp][16].x = qk;
        }
        __syncthreads();
        x = p[0][c4];
        y = p[0][8 + c4];
        qk = p[0][16].x;
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const float4 xw = p[w][c4], yw = p[w][8 + c4];
            x.x += xw.x, x.y += xw.y, x.z += xw.z, x.w += xw.w;
            y.x += yw.x, y.y += yw.y, y.z += yw.z, y.w += yw.w;
            qk += p[w][16].x;
        }
        const float4 u = make_float4(eta * (v[0] - al * x.x), eta * (v[1] - al * x.y),
                                     eta * (v[2] - al * x.z), eta * (v[3] - al * x.w));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            W[r].x = fmaf(k[r], u.x, al * W[r].x);
            W[r].y = fmaf(k[r], u.y, al * W[r].y);
            W[r].z = fmaf(k[r], u.z, al * W[r].z);
            W[r].w = fmaf(k[r], u.w, al * W[r].w);
        }
        if (tid < 8)
            store_z4(static_cast<float *>(a.Z), a.z_bf16, (hrow + t) * a.dv + col,
                     a.q_scale * fmaf(qk, u.x, al * y.x), a.q_scale * fmaf(qk, u.y, al * y.y),
                     a.q_scale * fmaf(qk, u.z, al * y.z), a.q_scale * fmaf(qk, u.w, al * y.w));
    }
    if (a.W_out) {
        float *w = a.W_out + ((size_t)slot * a.H + h) * state + wrow;
#pragma unroll
        for (int r = 0; r < R; ++r) *reinterpret_cast<float4 *>(w + (size_t)r * a.dv) = W[r];
    }
}

}  // namespace

namespace {
cudaError_t run_recurrent(const RecArgs &r, int N, int dk, bool bf16, cudaStream_t s) {
    const unsigned grid = (unsigned)((long long)N * r.H * (r.dv / kRecCols));
    if (dk == 64) {
        if (bf16) delta_recurrent_kernel<64, true><<<grid, kRecThreads, 0, s>>>(r);
        else delta_recurrent_kernel<64, false><<<grid, kRecThreads, 0, s>>>(r);
    } else {
        if (bf16) delta_recurrent_kernel<128, true><<<grid, kRecThreads, 0, s>>>(r);
        else delta_recurrent_kernel<128, false><<<grid, kRecThreads, 0, s>>>(r);
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}
}  // namespace

bool delta_supported(int dk, int dv) { return (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

cudaError_t launch_delta_recurrent(const DeltaArgs &a, cudaStream_t s) {
    const RecArgs r{a.Q, a.K, a.V, a.eta, a.g, a.W0, a.W_out, a.Z, a.seq_start, nullptr,
                    a.Hk, a.H, a.T, a.dv, 0, a.w0_per_seq ? a.H : 0, a.q_scale, a.z_bf16};
    return run_recurrent(r, a.N, a.dk, a.bf16, s);
}

cudaError_t launch_delta_decode(const DeltaArgs &a, float *W, const int *state_index, int n_slots,
                                cudaStream_t s) {
    const RecArgs r{a.Q, a.K, a.V, a.eta, a.g, W, W, a.Z, nullptr, state_index,
                    a.Hk, a.H, a.T, a.dv, n_slots, a.H, a.q_scale, a.z_bf16};
    return run_recurrent(r, a.B, a.dk, a.bf16, s);
}

}  // namespace ttt
