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
// squares; the next row's loads are on their way meanwhile. The norm of a head is a
// shuffle among its d / 8 threads; the norm of the row a block reduction with one
// barrier. Sums and statistics are fp32.
// 32,768 rows of 8 x 128, bf16 with fp32 z, RMS norms: forward 76 us (403 MB at
// 5.3 TB/s, 0.82 of the copy rate; issue slots used to 65 %), backward 160 us and 7 us
// for the parameters' sums (940 MB at 5.6 TB/s, 0.87). Without loads ahead, with exact
// divisions and two-barrier sums they took 170 and 257 us.
//
// The backward's parameter gradients are column sums over all rows: each block
// adds up its own rows in registers (a thread keeps its 8 channels) and stores
// one partial row; a second kernel adds the partial rows in a fixed order.
#include "../../include/ttt.h"
#include "ttt_join.cuh"

namespace ttt {
namespace {

// Threads of the largest blocks of an instance. The forward: up to 128 (rows of up to
// 1024 channels), four blocks an SM, and up to 512 (D <= 4096). The backward keeps the
// parameters in registers up to 384 threads (192: two blocks of 168 registers an SM, so
// three of 128 threads; 256 and 384: one block); the 512-thread blocks have 128 registers
// and read them again for each row.
constexpr int kJoinThreads = 128, kJoinBwdThreads = 192, kJoinMaxThreads = 512;
constexpr int kJoinParams = 5;        // scale, gamma1, beta1, gamma2, beta2

constexpr int V = 8;  // channels of a thread

// Eight consecutive elements as 4-byte words, as loaded (16 bytes at a time) and as floats.
template <bool BF16>
struct Raw {
    static constexpr int N = BF16 ? V / 2 : V;
    uint32_t w[N];
    __device__ __forceinline__ void load(const void *p, size_t i) {
        const char *q = static_cast<const char *>(p) + i * (BF16 ? 2 : 4);
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const uint4 u = reinterpret_cast<const uint4 *>(q)[j / 4];
            w[j] = u.x, w[j + 1] = u.y, w[j + 2] = u.z, w[j + 3] = u.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = 0;
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t u = w[BF16 ? j / 2 : j];
            x[j] = __uint_as_float(!BF16 ? u : (j & 1) ? u & 0xFFFF0000u : u << 16);
        }
    }
};
// Stores x and leaves in x the values as they were stored.
template <bool BF16>
__device__ __forceinline__ void store_v(void *p, size_t i, float (&x)[V]) {
    if (BF16) {
        uint32_t w[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t *>(&b);
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
        __nv_bfloat16 *q = static_cast<__nv_bfloat16 *>(p) + i;
        *reinterpret_cast<uint4 *>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
#pragma unroll
        for (int j = 0; j < V; j += 4) f[j / 4] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    }
}
__device__ __forceinline__ void param_v(float (&x)[V], const float *p, int i, bool live, float dflt) {
    if (p && live) {
        Raw<false> r;
        r.load(p, i);
        r.get(x);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = dflt;
    }
}

// Sums over the block and over a head. Two sets of 16 slots in turn: a thread that
// writes the sum after next has passed the next one's barrier, behind which this
// one's slots are read. Slots of warps that are not there stay zero.
struct Sums {
    float *slots;  // 32 floats, zeroed before the first use
    int nw, lanes; // warps; threads of a head (0: one head, the whole row)
    int turn;
    __device__ __forceinline__ float block(float v) {
        v = warp_sum(v);
        if (nw == 1) return v;
        float *p = slots + turn;
        turn ^= 16;
        if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
        __syncthreads();
        const float4 *q = reinterpret_cast<const float4 *>(p);
        float4 s = q[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            if (4 * i >= nw) break;
            const float4 u = q[i];
            s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
        }
        return (s.x + s.y) + (s.z + s.w);
    }
    __device__ __forceinline__ float head(float v) {
        if (lanes == 0) return block(v);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
        }
        return v;
    }
};
__device__ __forceinline__ float sum_v(const float (&x)[V]) {
    return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}
__device__ __forceinline__ float dot_v(const float (&x)[V], const float (&y)[V]) {
    float s = x[0] * y[0];
#pragma unroll
    for (int j = 1; j < V; ++j) s = fmaf(x[j], y[j], s);
    return s;
}

// x <- (x - mean) / sqrt(mean square + eps), returns the factor. `sum` adds
// over the norm's n channels; a thread without channels holds zeros and
// passes live = false (its centred values must not count).
template <class Sum>
__device__ __forceinline__ float norm_v(float (&x)[V], float inv_n, float eps, bool rms, bool live,
                                       Sum sum) {
    if (!rms) {
        const float m = sum(sum_v(x)) * inv_n;
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = live ? x[j] - m : 0.f;
    }
    // the fast root and one Newton step: within an ulp of the exact quotient. A sum of
    // squares above fp32's range gives a factor of 0 (the step would make it inf * 0); NaN stays.
    const float q = sum(dot_v(x, x)) * inv_n + eps, y = rsqrtf(q);
    const float i = q < INFINITY ? y * fmaf(-0.5f * q * y, y, 1.5f) : y;
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] *= i;
    return i;
}

// sigmoid(x) and 1 - sigmoid(x), neither by a subtraction, which would cancel where x is far
// from 0: with e = exp(-|x|) they are 1 / (1 + e) and e / (1 + e). The fast exponential
// is off by (2 + 1.173 |x|) 2^-23 of e at most and the fast reciprocal, its divisor being in
// [1, 2], by 2^-22: relative errors of 3e-6 at |x| = 20, a step of a bf16 gate being 4e-3
// of x. The exact forms cost four times the instructions, which at 12 bytes a channel
// bound the forward.
__device__ __forceinline__ void sigmoid(float x, float &s, float &rest) {
    const float e = __expf(-fabsf(x)), r = __fdividef(1.f, 1.f + e), er = e * r;
    s = x < 0.f ? er : r;
    rest = x < 0.f ? r : er;
}

// A block's rows are blockIdx.x, + gridDim.x, ...; a row's loads are on their way
// while the row before it is computed.
// Batch row and token of a block's rows, one after the other without divisions.
struct Rows {
    long long row, end;
    int b, t, T, db, dt;
    __device__ __forceinline__ Rows(long long rows, int T_) : row(blockIdx.x), end(rows), T(T_) {
        b = (int)(blockIdx.x / (unsigned)T);
        t = (int)(blockIdx.x - (unsigned)b * T);
        db = (int)(gridDim.x / (unsigned)T);
        dt = (int)(gridDim.x - (unsigned)db * T);
    }
    __device__ __forceinline__ bool live() const { return row < end; }
    __device__ __forceinline__ void next() {
        row += gridDim.x;
        b += db;
        t += dt;
        if (t >= T) t -= T, ++b;
    }
    // element of a head-major [B][H][T][d] array
    __device__ __forceinline__ size_t head_major(int H, int h, int d) const {
        return (((size_t)b * H + h) * T + t) * d;
    }
};

template <int NT, bool BF16, bool ZBF16>
__global__ void __launch_bounds__(NT, 512 / NT) join_fwd_kernel(JoinArgs a) {
    __shared__ __align__(16) float slots[32];
    const int D = a.H * a.d, c = threadIdx.x * V;
    const bool live = c < D;
    const int h = c / a.d, cd = c - h * a.d;
    if (threadIdx.x < 32) slots[threadIdx.x] = 0.f;
    __syncthreads();
    Sums sums{slots, (int)(blockDim.x >> 5), a.H == 1 ? 0 : a.d / V, 0};
    const float inv_d = 1.f / (float)a.d, inv_D = 1.f / (float)D;
    float s[V], g1[V], b1[V], g2[V], b2[V];
    param_v(s, a.scale, c, live, 1.f);
    param_v(g1, a.gamma1, c, live, 1.f);
    param_v(b1, a.beta1, c, live, 0.f);
    param_v(g2, a.gamma2, c, live, 1.f);
    param_v(b2, a.beta2, c, live, 0.f);
    auto hsum = [&](float v) { return sums.head(v); };
    auto rsum = [&](float v) { return sums.block(v); };
    const long long rows = (long long)a.B * a.T;
    Raw<BF16> xr, gr;
    Raw<ZBF16> zr;
    xr.zero(), gr.zero(), zr.zero();
    auto fetch = [&](const Rows &at) {
        if (!live) return;
        const size_t i = (size_t)at.row * D + c;
        xr.load(a.X, i);
        if (a.Z) {
            zr.load(a.Z, at.head_major(a.H, h, a.d) + cd);
            if (a.gate) gr.load(a.gate, i);
        }
    };
    Rows now(rows, a.T), ahead = now;
    if (ahead.live()) fetch(ahead);
    for (; now.live(); now.next()) {
        const size_t at = (size_t)now.row * D + c;
        float r[V], z[V], g[V];
        xr.get(r), zr.get(z), gr.get(g);
        ahead.next();
        if (ahead.live()) fetch(ahead);
        if (a.Z) {
            norm_v(z, inv_d, a.eps, a.rms, live, hsum);
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] = s[j] * fmaf(z[j], g1[j], b1[j]);
            if (a.gate) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float sg, rest;
                    sigmoid(g[j], sg, rest);
                    z[j] *= a.silu ? g[j] * sg : sg;
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) r[j] += z[j];
            if (live) store_v<BF16>(a.R, at, r);
        }
        if (a.Hn) {
            if (!live) {
#pragma unroll
                for (int j = 0; j < V; ++j) r[j] = 0.f;
            }
            norm_v(r, inv_D, a.eps, a.rms, live, rsum);
#pragma unroll
            for (int j = 0; j < V; ++j) r[j] = fmaf(r[j], g2[j], b2[j]);
            if (live) store_v<BF16>(a.Hn, at, r);
        }
    }
}

template <int NT, bool BF16, bool ZBF16>
__global__ void __launch_bounds__(NT, NT == kJoinBwdThreads ? 2 : 1) join_bwd_kernel(JoinBwdArgs a) {
    __shared__ __align__(16) float slots[32];
    const int D = a.H * a.d, c = threadIdx.x * V;
    const bool live = c < D;
    const int h = c / a.d, cd = c - h * a.d;
    if (threadIdx.x < 32) slots[threadIdx.x] = 0.f;
    __syncthreads();
    Sums sums{slots, (int)(blockDim.x >> 5), a.H == 1 ? 0 : a.d / V, 0};
    const float inv_d = 1.f / (float)a.d, inv_D = 1.f / (float)D;
    constexpr bool KEEP = NT < kJoinMaxThreads;  // else the parameters are read again for each row
    float ks[V], kg1[V], kb1[V], kg2[V];
    if (KEEP) {
        param_v(ks, a.scale, c, live, 1.f);
        param_v(kg1, a.gamma1, c, live, 1.f);
        param_v(kb1, a.beta1, c, live, 0.f);
        param_v(kg2, a.gamma2, c, live, 1.f);
    }
    float acc[kJoinParams][V] = {};
    auto hsum = [&](float v) { return sums.head(v); };
    auto rsum = [&](float v) { return sums.block(v); };
    const long long rows = (long long)a.B * a.T;
    Raw<BF16> rr, gr;
    Raw<ZBF16> zr;
    Raw<false> dr, hr;
    rr.zero(), gr.zero(), zr.zero(), dr.zero(), hr.zero();
    auto fetch = [&](const Rows &at) {
        if (!live) return;
        const size_t i = (size_t)at.row * D + c;
        if (a.dH) {
            rr.load(a.R, i);
            hr.load(a.dH, i);
        }
        if (a.dR) dr.load(a.dR, i);
        if (a.Z) {
            zr.load(a.Z, at.head_major(a.H, h, a.d) + cd);
            if (a.gate) gr.load(a.gate, i);
        }
    };
    Rows now(rows, a.T), ahead = now;
    if (ahead.live()) fetch(ahead);
    for (; now.live(); now.next()) {
        const size_t at = (size_t)now.row * D + c;
        float dx[V], z[V], g[V], r[V], dy[V];
        dr.get(dx), rr.get(r), hr.get(dy), zr.get(z), gr.get(g);
        ahead.next();
        if (ahead.live()) fetch(ahead);
        if (a.dH) {
            if (!KEEP) param_v(kg2, a.gamma2, c, live, 1.f);
            const float i = norm_v(r, inv_D, a.eps, a.rms, live, rsum);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                acc[3][j] = fmaf(dy[j], r[j], acc[3][j]);
                acc[4][j] += dy[j];
                dy[j] *= kg2[j];
            }
            const float m1 = a.rms ? 0.f : rsum(sum_v(dy)) * inv_D;
            const float m2 = rsum(dot_v(dy, r)) * inv_D;
#pragma unroll
            for (int j = 0; j < V; ++j) dx[j] += i * (dy[j] - m1 - r[j] * m2);
        }
        if (live) store_v<false>(a.dX, at, dx);
        if (a.Z) {
            const size_t zat = now.head_major(a.H, h, a.d) + cd;
            float dg[V];
            if (!KEEP) {
                param_v(ks, a.scale, c, live, 1.f);
                param_v(kg1, a.gamma1, c, live, 1.f);
                param_v(kb1, a.beta1, c, live, 0.f);
            }
            if (!live) {
#pragma unroll
                for (int j = 0; j < V; ++j) dx[j] = 0.f;
            }
            const float i = norm_v(z, inv_d, a.eps, a.rms, live, hsum);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = fmaf(z[j], kg1[j], kb1[j]);
                float act = 1.f, dact = 0.f;
                if (a.gate) {
                    float sg, rest;
                    sigmoid(g[j], sg, rest);
                    act = a.silu ? g[j] * sg : sg;
                    dact = a.silu ? sg * fmaf(g[j], rest, 1.f) : sg * rest;
                }
                acc[0][j] = fmaf(dx[j] * act, n, acc[0][j]);
                const float ds = dx[j] * ks[j];
                dg[j] = ds * n * dact;
                const float dn = ds * act;
                acc[1][j] = fmaf(dn, z[j], acc[1][j]);
                acc[2][j] += dn;
                dx[j] = dn * kg1[j];
            }
            if (a.gate && live) store_v<false>(a.dGate, at, dg);
            const float m1 = a.rms ? 0.f : hsum(sum_v(dx)) * inv_d;
            const float m2 = hsum(dot_v(dx, z)) * inv_d;
#pragma unroll
            for (int j = 0; j < V; ++j) dx[j] = i * (dx[j] - m1 - z[j] * m2);
            if (live) store_v<false>(a.dZ, zat, dx);
        }
    }
    if (live) {
#pragma unroll
        for (int p = 0; p < kJoinParams; ++p)
            store_v<false>(a.partials, ((size_t)blockIdx.x * kJoinParams + p) * D + c, acc[p]);
    }
}

// Adds the blocks' partial rows. Block: 8 channels x 32 threads, thread row y
// takes the partial rows y, y + 32, ... in order; the 32 sums are added in order.
__global__ void __launch_bounds__(256) join_params_kernel(const float *partials, int nblocks, int D,
                                                          float *out0, float *out1, float *out2,
                                                          float *out3, float *out4) {
    __shared__ float sums[32][9];
    const int p = blockIdx.y;
    float *out = p == 0 ? out0 : p == 1 ? out1 : p == 2 ? out2 : p == 3 ? out3 : out4;
    if (!out) return;
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3, c = blockIdx.x * 8 + x;
    float v = 0.f;
#pragma unroll 4
    for (int i = y; i < nblocks; i += 32) v += partials[((size_t)i * kJoinParams + p) * D + c];
    sums[y][x] = v;
    __syncthreads();
    if (y == 0) {
        for (int i = 1; i < 32; ++i) v += sums[i][x];
        out[c] = v;
    }
}

}  // namespace

bool join_supported(int H, int d) {
    const long long D = (long long)H * d;
    if (D > 8 * kJoinMaxThreads) return false;
    if (H == 1) return d % 8 == 0;
    return d == 16 || d == 32 || d == 64 || d == 128 || d == 256;
}

namespace {
int join_threads(int H, int d) { return (H * d / V + 31) / 32 * 32; }
// Blocks of the persistent kernels: as many as are resident at 128 registers a
// thread (168 in the backward's narrow blocks), at most one per row. Times of the kernels
// without the parameters' sums: 200,000 rows of 64 take 89 and 212 us (136 and 276 with
// eight blocks an SM), 6 heads of 64 and 65,536 rows 151 instead of 205, of which a third
// had to wait for a second round. The count depends
// on the shape alone, so the order of the parameter sums is the same in every call. Rows
// of more than 1536 channels leave one block an SM, whose phases overlap with nothing:
// 8192 rows of 4096, backward, 378 us at a floor of 146.
int join_blocks(long long rows, int nt, bool bwd) {
    const int per_sm = (bwd && nt <= 384 ? 384 : 512) / nt;
    const long long n = 148LL * (per_sm < 1 ? 1 : per_sm);
    return (int)(rows < n ? rows : n);
}

template <int NT>
void run_fwd(const JoinArgs &a, unsigned grid, int nt, cudaStream_t s) {
    if (a.bf16) {
        if (a.z_bf16) join_fwd_kernel<NT, true, true><<<grid, nt, 0, s>>>(a);
        else join_fwd_kernel<NT, true, false><<<grid, nt, 0, s>>>(a);
    } else {
        if (a.z_bf16) join_fwd_kernel<NT, false, true><<<grid, nt, 0, s>>>(a);
        else join_fwd_kernel<NT, false, false><<<grid, nt, 0, s>>>(a);
    }
}
template <int NT>
void run_bwd(const JoinBwdArgs &a, unsigned grid, int nt, cudaStream_t s) {
    if (a.bf16) {
        if (a.z_bf16) join_bwd_kernel<NT, true, true><<<grid, nt, 0, s>>>(a);
        else join_bwd_kernel<NT, true, false><<<grid, nt, 0, s>>>(a);
    } else {
        if (a.z_bf16) join_bwd_kernel<NT, false, true><<<grid, nt, 0, s>>>(a);
        else join_bwd_kernel<NT, false, false><<<grid, nt, 0, s>>>(a);
    }
}
}  // namespace

size_t join_bwd_workspace_bytes(int B, int H, int T, int d) {
    return sizeof(float) * kJoinParams * (size_t)H * d * join_blocks((long long)B * T, join_threads(H, d), true);
}

cudaError_t launch_join_fwd(const JoinArgs &a, cudaStream_t s) {
    const int nt = join_threads(a.H, a.d);
    const long long rows = (long long)a.B * a.T;
    const int grid = join_blocks(rows, nt, false);
    if (nt <= kJoinThreads) run_fwd<kJoinThreads>(a, grid, nt, s);
    else run_fwd<kJoinMaxThreads>(a, grid, nt, s);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}

cudaError_t launch_join_bwd(const JoinBwdArgs &a, cudaStream_t s) {
    const int nt = join_threads(a.H, a.d), D = a.H * a.d;
    const int grid = join_blocks((long long)a.B * a.T, nt, true);
    // 16,384 rows, us with the instance named and with that of 512 threads: 24 heads of 64
    // (192) 125 / 293, 16 of 128 (256) 200 / 332, 20 of 128 (384) 278 / 588
    if (nt <= kJoinBwdThreads) run_bwd<kJoinBwdThreads>(a, grid, nt, s);
    else if (nt <= 256) run_bwd<256>(a, grid, nt, s);
    else if (nt <= 384) run_bwd<384>(a, grid, nt, s);
    else run_bwd<kJoinMaxThreads>(a, grid, nt, s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launch(s);
    if (!a.dscale && !a.dgamma1 && !a.dbeta1 && !a.dgamma2 && !a.dbeta2) return e;
    join_params_kernel<<<dim3(D / 8, kJoinParams), 256, 0, s>>>(
        a.partials, grid, D, a.dscale, a.dgamma1, a.dbeta1, a.dgamma2, a.dbeta2);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}

}  // namespace ttt
