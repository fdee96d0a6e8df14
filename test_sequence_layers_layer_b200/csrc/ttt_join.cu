// ttt_join.cu -- the join between two blocks, forward and backward, one pass
// over memory each:
//   n = Norm_d(z) gamma1 + beta1  (per head),  r = x + s act(gate) n,
//   h = Norm_D(r) gamma2 + beta2.
// Norm is LayerNorm (population variance) or RMSNorm; z is head-major
// [B][H][T][d], everything else token-major [B][T][D], D = H d. h is the norm
// of r as it is stored, so that a backward that reads the stored r
// differentiates what the forward computed.
//
// Both directions are bound by memory (forward: 12 bytes per channel with bf16
// x, gate, r, h and fp32 z; 14 to 22 flops). A block keeps whole rows in registers, 8
// channels (16 bytes of bf16) per thread, so every tensor is read and written
// once and the row statistics are taken from registers, the mean before the
// squares. The norm of a head is a shuffle among its d / 8 threads; the norm
// of the row a block reduction. Sums and statistics are fp32.
//
// The backward's parameter gradients are column sums over all rows: each block
// adds up its own rows in registers (a thread keeps its 8 channels) and stores
// one partial row; a second kernel adds the partial rows in a fixed order.
#include "../../include/ttt.h"
#include "ttt_join.cuh"

namespace ttt {
namespace {

constexpr int kJoinMaxThreads = 512;  // D <= 4096
constexpr int kJoinParams = 5;        // scale, gamma1, beta1, gamma2, beta2

// Eight consecutive elements, 16-byte loads and stores.
template <bool BF16>
__device__ __forceinline__ void load8(float (&x)[8], const void *p, size_t i) {
    if (BF16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
        const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = f[0], b = f[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}
// Stores x and leaves in x the values as they were stored.
template <bool BF16>
__device__ __forceinline__ void store8(void *p, size_t i, float (&x)[8]) {
    if (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t *>(&b);
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) =
            make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}
__device__ __forceinline__ void param8(float (&x)[8], const float *p, int i, bool live, float dflt) {
    if (p && live) {
        load8<false>(x, p, i);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = dflt;
    }
}

// Sum over the block; `slots` holds a float per warp. The first barrier lets
// the readers of the sum before finish with the slots.
__device__ __forceinline__ float block_sum(float v, float *slots) {
    v = warp_sum(v);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < nw; ++w) s += slots[w];
    return s;
}
__device__ __forceinline__ float head_sum(float v, int lanes, float *slots) {
    if (lanes == 0) return block_sum(v, slots);  // one head: the whole row
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float sum8(const float (&x)[8]) {
    return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}
__device__ __forceinline__ float dot8(const float (&x)[8], const float (&y)[8]) {
    float s = x[0] * y[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) s = fmaf(x[j], y[j], s);
    return s;
}

// x <- (x - mean) / sqrt(mean square + eps), returns the factor. `sum` adds
// over the norm's n channels; a thread without channels holds zeros and
// passes live = false (its centred values must not count).
template <class Sum>
__device__ __forceinline__ float norm8(float (&x)[8], float inv_n, float eps, bool rms, bool live,
                                       Sum sum) {
    if (!rms) {
        const float m = sum(sum8(x)) * inv_n;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = live ? x[j] - m : 0.f;
    }
    // divided, not rsqrtf (2 ulp): one division per row costs nothing here
    const float i = 1.f / sqrtf(sum(dot8(x, x)) * inv_n + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= i;
    return i;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

template <bool BF16, bool ZBF16>
__global__ void __launch_bounds__(kJoinMaxThreads) join_fwd_kernel(JoinArgs a) {
    __shared__ float slots[kJoinMaxThreads / 32];
    const int D = a.H * a.d, c = threadIdx.x * 8;
    const bool live = c < D;
    const int h = c / a.d, cd = c - h * a.d;
    const int lanes = a.H == 1 ? 0 : a.d >> 3;
    const float inv_d = 1.f / (float)a.d, inv_D = 1.f / (float)D;
    float s[8], g1[8], b1[8], g2[8], b2[8];
    param8(s, a.scale, c, live, 1.f);
    param8(g1, a.gamma1, c, live, 1.f);
    param8(b1, a.beta1, c, live, 0.f);
    param8(g2, a.gamma2, c, live, 1.f);
    param8(b2, a.beta2, c, live, 0.f);
    auto hsum = [&](float v) { return head_sum(v, lanes, slots); };
    auto rsum = [&](float v) { return block_sum(v, slots); };
    const long long rows = (long long)a.B * a.T;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const size_t at = (size_t)row * D + c;
        float r[8] = {}, z[8] = {}, g[8] = {};
        if (live) load8<BF16>(r, a.X, at);
        if (a.Z) {
            const long long b = row / a.T, t = row - b * a.T;
            if (live) {
                load8<ZBF16>(z, a.Z, ((size_t)(b * a.H + h) * a.T + t) * a.d + cd);
                if (a.gate) load8<BF16>(g, a.gate, at);
            }
            norm8(z, inv_d, a.eps, a.rms, live, hsum);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float y = s[j] * fmaf(z[j], g1[j], b1[j]);
                if (a.gate) {
                    const float sg = sigmoid(g[j]);
                    y *= a.silu ? g[j] * sg : sg;
                }
                r[j] += y;
            }
            if (live) store8<BF16>(a.R, at, r);
        }
        if (a.Hn) {
            if (!live) {
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = 0.f;
            }
            norm8(r, inv_D, a.eps, a.rms, live, rsum);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = fmaf(r[j], g2[j], b2[j]);
            if (live) store8<BF16>(a.Hn, at, r);
        }
    }
}

template <bool BF16, bool ZBF16>
__global__ void __launch_bounds__(kJoinMaxThreads) join_bwd_kernel(JoinBwdArgs a) {
    __shared__ float slots[kJoinMaxThreads / 32];
    const int D = a.H * a.d, c = threadIdx.x * 8;
    const bool live = c < D;
    const int h = c / a.d, cd = c - h * a.d;
    const int lanes = a.H == 1 ? 0 : a.d >> 3;
    const float inv_d = 1.f / (float)a.d, inv_D = 1.f / (float)D;
    float s[8], g1[8], b1[8], g2[8];
    param8(s, a.scale, c, live, 1.f);
    param8(g1, a.gamma1, c, live, 1.f);
    param8(b1, a.beta1, c, live, 0.f);
    param8(g2, a.gamma2, c, live, 1.f);
    float acc[kJoinParams][8] = {};
    auto hsum = [&](float v) { return head_sum(v, lanes, slots); };
    auto rsum = [&](float v) { return block_sum(v, slots); };
    const long long rows = (long long)a.B * a.T;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const size_t at = (size_t)row * D + c;
        float dx[8] = {};
        if (a.dR && live) load8<false>(dx, a.dR, at);
        if (a.dH) {
            float r[8] = {}, dy[8] = {};
            if (live) {
                load8<BF16>(r, a.R, at);
                load8<false>(dy, a.dH, at);
            }
            const float i = norm8(r, inv_D, a.eps, a.rms, live, rsum);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc[3][j] = fmaf(dy[j], r[j], acc[3][j]);
                acc[4][j] += dy[j];
                dy[j] *= g2[j];
            }
            const float m1 = a.rms ? 0.f : rsum(sum8(dy)) * inv_D;
            const float m2 = rsum(dot8(dy, r)) * inv_D;
#pragma unroll
            for (int j = 0; j < 8; ++j) dx[j] += i * (dy[j] - m1 - r[j] * m2);
        }
        if (live) store8<false>(a.dX, at, dx);
        if (a.Z) {
            const long long b = row / a.T, t = row - b * a.T;
            const size_t zat = ((size_t)(b * a.H + h) * a.T + t) * a.d + cd;
            float z[8] = {}, g[8] = {}, dg[8];
            if (live) {
                load8<ZBF16>(z, a.Z, zat);
                if (a.gate) load8<BF16>(g, a.gate, at);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) dx[j] = 0.f;
            }
            const float i = norm8(z, inv_d, a.eps, a.rms, live, hsum);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = fmaf(z[j], g1[j], b1[j]);
                float act = 1.f, dact = 0.f;
                if (a.gate) {
                    const float sg = sigmoid(g[j]);
                    act = a.silu ? g[j] * sg : sg;
                    dact = a.silu ? sg * fmaf(g[j], 1.f - sg, 1.f) : sg * (1.f - sg);
                }
                acc[0][j] = fmaf(dx[j] * act, n, acc[0][j]);
                const float ds = dx[j] * s[j];
                dg[j] = ds * n * dact;
                const float dn = ds * act;
                acc[1][j] = fmaf(dn, z[j], acc[1][j]);
                acc[2][j] += dn;
                dx[j] = dn * g1[j];
            }
            if (a.gate && live) store8<false>(a.dGate, at, dg);
            const float m1 = a.rms ? 0.f : hsum(sum8(dx)) * inv_d;
            const float m2 = hsum(dot8(dx, z)) * inv_d;
#pragma unroll
            for (int j = 0; j < 8; ++j) dx[j] = i * (dx[j] - m1 - z[j] * m2);
            if (live) store8<false>(a.dZ, zat, dx);
        }
    }
    if (live) {
#pragma unroll
        for (int p = 0; p < kJoinParams; ++p)
            store8<false>(a.partials, ((size_t)blockIdx.x * kJoinParams + p) * D + c, acc[p]);
    }
}

// Adds the blocks' partial rows. Block: 32 channels x 8 threads, thread row y
// takes the partial rows y, y + 8, ... in order; the eight sums are added in order.
__global__ void __launch_bounds__(256) join_params_kernel(const float *partials, int nblocks, int D,
                                                          float *out0, float *out1, float *out2,
                                                          float *out3, float *out4) {
    __shared__ float sums[256];
    float *const outs[kJoinParams] = {out0, out1, out2, out3, out4};
    float *out = outs[blockIdx.y];
    if (!out) return;
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < D)
        for (int i = y; i < nblocks; i += 8)
            v += partials[((size_t)i * kJoinParams + blockIdx.y) * D + c];
    sums[threadIdx.x] = v;
    __syncthreads();
    if (y == 0 && c < D) {
        for (int i = 1; i < 8; ++i) v += sums[i * 32 + lane];
        out[c] = v;
    }
}

}  // namespace

#ifndef TTT_HOST_RUN  // launch code (a host build of the kernels for tests leaves it out)

bool join_supported(int H, int d) {
    const long long D = (long long)H * d;
    if (D > 8 * kJoinMaxThreads) return false;
    if (H == 1) return d % 8 == 0;
    return d == 16 || d == 32 || d == 64 || d == 128 || d == 256;
}

namespace {
int join_threads(int H, int d) { return (H * d / 8 + 31) / 32 * 32; }
// Blocks of the persistent backward: as many as are resident at 128 registers a
// thread (its accumulators), at most one per row. The count depends on the
// shape alone, so the order of the parameter sums is the same in every call.
int join_bwd_blocks(long long rows, int H, int d) {
    int per_sm = 512 / join_threads(H, d);
    if (per_sm > 8) per_sm = 8;
    const long long n = 148LL * (per_sm < 1 ? 1 : per_sm);
    return (int)(rows < n ? rows : n);
}
}  // namespace

size_t join_bwd_workspace_bytes(int B, int H, int T, int d) {
    return sizeof(float) * kJoinParams * (size_t)H * d * join_bwd_blocks((long long)B * T, H, d);
}

cudaError_t launch_join_fwd(const JoinArgs &a, cudaStream_t s) {
    const int nt = join_threads(a.H, a.d);
    const long long rows = (long long)a.B * a.T;
    const long long most = 148LL * (2048 / nt);
    const unsigned grid = (unsigned)(rows < most ? rows : most);
    if (a.bf16) {
        if (a.z_bf16) join_fwd_kernel<true, true><<<grid, nt, 0, s>>>(a);
        else join_fwd_kernel<true, false><<<grid, nt, 0, s>>>(a);
    } else {
        if (a.z_bf16) join_fwd_kernel<false, true><<<grid, nt, 0, s>>>(a);
        else join_fwd_kernel<false, false><<<grid, nt, 0, s>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}

cudaError_t launch_join_bwd(const JoinBwdArgs &a, cudaStream_t s) {
    const int nt = join_threads(a.H, a.d), D = a.H * a.d;
    const int grid = join_bwd_blocks((long long)a.B * a.T, a.H, a.d);
    if (a.bf16) {
        if (a.z_bf16) join_bwd_kernel<true, true><<<grid, nt, 0, s>>>(a);
        else join_bwd_kernel<true, false><<<grid, nt, 0, s>>>(a);
    } else {
        if (a.z_bf16) join_bwd_kernel<false, true><<<grid, nt, 0, s>>>(a);
        else join_bwd_kernel<false, false><<<grid, nt, 0, s>>>(a);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launch(s);
    if (!a.dscale && !a.dgamma1 && !a.dbeta1 && !a.dgamma2 && !a.dbeta2) return e;
    join_params_kernel<<<dim3((D + 31) / 32, kJoinParams), 256, 0, s>>>(
        a.partials, grid, D, a.dscale, a.dgamma1, a.dbeta1, a.dgamma2, a.dbeta2);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}
#endif  // TTT_HOST_RUN

}  // namespace ttt
