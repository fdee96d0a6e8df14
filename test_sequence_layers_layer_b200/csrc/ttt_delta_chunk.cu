// ttt_delta_chunk.cu -- chunked forward of the gated delta rule: the per-chunk
// preparation (all chunks at once) and the scan over the chunks.
//
// For a chunk of C = 64 tokens that starts from W, with G_i the sum of the decays
// up to token i, D = diag(exp G), Gam_ij = exp(G_i - G_j):
//   X = V - D K W,   (I + A) rho = X,   A_ij = Gam_ij (k_i.k_j) eta_j   (j < i)
//   Z = c D Q W + P rho,                P_ij = c Gam_ij (q_i.k_j) eta_j (j <= i)
//   W' = exp(G_C) W + sum_j exp(G_C - G_j) eta_j k_j^T rho_j.
// T = (I + A)^-1, P and the decays depend on q, k, eta and g alone, so one kernel
// forms them for all chunks in parallel; what is left to do one chunk after
// the other are four small products.
#include "../../include/ttt.h"
#include "ttt_delta_mma.cuh"

namespace ttt {
namespace delta {
namespace {

// ---------------------------------------------------------------- preparation

constexpr int kPrepThreads = 128;
constexpr int kLtStride = 68, kTmStride = 65;

struct PrepArgs {
    const void *Q, *K;
    const float *eta, *g;
    const int *seq_start;
    int B, Hk, H, T, N;
    float q_scale;
    Images im;
};

// Sequence and chunk of a slot; false for a slot that no chunk uses.
__device__ __forceinline__ bool find_chunk(const PrepArgs &a, int slot, int &n, int &t0, int &len) {
    int c;
    if (!a.seq_start) {
        const int per = (a.T + C - 1) / C;
        n = slot / per;
        c = slot - n * per;
        t0 = 0;
        len = a.T;
    } else {
        // the last sequence whose first slot is not behind this one
        int lo = 0, hi = a.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            int s, l;
            delta_span(a.seq_start, mid, a.T, s, l);
            if (s / C + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
        delta_span(a.seq_start, n, a.T, t0, len);
        c = slot - (t0 / C + n);
        if (c < 0) return false;
    }
    t0 += c * C;
    len -= c * C;
    len = len < C ? len : C;
    return len > 0;
}

// One 64-row image of Q or K: rows in global memory to scaled fp16 terms, in
// shared memory and in the workspace; inv[row] = 1 / scale.
template <int DK, bool BF16>
__device__ __forceinline__ void convert_rows(const void *src, size_t row0, int len, char *sm,
                                             char *gm, float *inv) {
    constexpr int LPR = DK / 8, RPP = kPrepThreads / LPR;  // lanes per row, rows per pass
    const int sub = threadIdx.x % LPR;
#pragma unroll
    for (int p = 0; p < C / RPP; ++p) {
        const int row = p * RPP + threadIdx.x / LPR;
        float x[8] = {};
        if (row < len) {
            const size_t at = (row0 + row) * DK + sub * 8;
            if (BF16) {
                const uint4 u = *reinterpret_cast<const uint4 *>(
                    static_cast<const __nv_bfloat16 *>(src) + at);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[2 * j] = __uint_as_float(w[j] << 16);
                    x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            } else {
                const float4 *f =
                    reinterpret_cast<const float4 *>(static_cast<const float *>(src) + at);
                const float4 u = f[0], v = f[1];
                x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
                x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
            }
        }
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float s, is;
        pow2_scale(m, s, is);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split_f16(x[2 * j] * s, x[2 * j + 1] * s, hi[j], lo[j]);
        const uint32_t o = img_off(row, sub * 8);
        const uint4 h = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(sm + o) = h;
        *reinterpret_cast<uint4 *>(gm + o) = h;
        if (!BF16) {
            const uint4 l = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            *reinterpret_cast<uint4 *>(sm + C * DK * 2 + o) = l;
            *reinterpret_cast<uint4 *>(gm + C * DK * 2 + o) = l;
        }
        if (sub == 0) inv[row] = is;
    }
}

template <int DK, bool BF16>
constexpr int prep_smem() {
    return 2 * C * DK * 2 * (BF16 ? 1 : 2) + 4 * (C * kLtStride + C * kTmStride) + 4 * 6 * C;
}

// One block per chunk and key head, its value heads one after the other.
// The inverse is a forward substitution in fp32: thread j < 64 holds column j of
// T in registers; step k takes x_i -= A_ik x_k for i > k, A's columns read as
// broadcasts.
template <int DK, bool BF16>
__global__ void __launch_bounds__(kPrepThreads) delta_prep_kernel(PrepArgs a) {
    extern __shared__ __align__(1024) char psm[];
    constexpr int IMG = C * DK * 2 * (BF16 ? 1 : 2);
    char *sK = psm, *sQ = sK + IMG;
    float *Lt = reinterpret_cast<float *>(sQ + IMG);  // A transposed: Lt[k][i] = A_ik
    float *Tm = Lt + C * kLtStride;
    float *iK = Tm + C * kTmStride, *iQ = iK + C, *Gh = iQ + C, *Gl = Gh + C, *eta = Gl + C;
    const int slot = blockIdx.x / a.Hk, hk = blockIdx.x % a.Hk;
    int n, t0, len;
    if (!find_chunk(a, slot, n, t0, len)) return;
    const int b = a.seq_start ? 0 : n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, q4 = lane & 3;
    const size_t kslot = (size_t)slot * a.Hk + hk;
    const size_t krow = ((size_t)b * a.Hk + hk) * a.T + t0;
    convert_rows<DK, BF16>(a.K, krow, len, sK, a.im.K + kslot * a.im.kimg, iK);
    convert_rows<DK, BF16>(a.Q, krow, len, sQ, a.im.Q + kslot * a.im.kimg, iQ);
    __syncthreads();

    // k_i.k_j and q_i.k_j of this warp's 16 rows i, columns j up to the diagonal
    float kk[8][4] = {}, qk[8][4] = {};
    const uint32_t uK = smem_u32(sK), uQ = smem_u32(sQ);
#pragma unroll
    for (int k = 0; k < DK; k += 16) {
        uint32_t ak[4], aq[4], akl[4], aql[4];
        ldsm_x4(ak, ldsm_addr(uK, 16 * warp, k, lane));
        ldsm_x4(aq, ldsm_addr(uQ, 16 * warp, k, lane));
        if (!BF16) {
            ldsm_x4(akl, ldsm_addr(uK + C * DK * 2, 16 * warp, k, lane));
            ldsm_x4(aql, ldsm_addr(uQ + C * DK * 2, 16 * warp, k, lane));
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            if (np > warp) break;
            uint32_t bb[4];
            load_b(bb, uK, 16 * np, k, lane);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                mma_f16(kk[2 * np + x], ak, bb[2 * x], bb[2 * x + 1]);
                mma_f16(qk[2 * np + x], aq, bb[2 * x], bb[2 * x + 1]);
                if (!BF16) {
                    mma_f16(kk[2 * np + x], akl, bb[2 * x], bb[2 * x + 1]);
                    mma_f16(qk[2 * np + x], aql, bb[2 * x], bb[2 * x + 1]);
                }
            }
            if (!BF16) {
                load_b(bb, uK + C * DK * 2, 16 * np, k, lane);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mma_f16(kk[2 * np + x], ak, bb[2 * x], bb[2 * x + 1]);
                    mma_f16(qk[2 * np + x], aq, bb[2 * x], bb[2 * x + 1]);
                }
            }
        }
    }

    const int rep = a.H / a.Hk;
    for (int r = 0; r < rep; ++r) {
        const int h = hk * rep + r;
        const size_t hrow = ((size_t)b * a.H + h) * a.T + t0;
        const size_t hslot = (size_t)slot * a.H + h;
        float *vec = reinterpret_cast<float *>(a.im.vec + hslot * kVecBytes);
        __syncthreads();  // the head before is done with the shared buffers
        if (warp == 0) {
            // sums of decays in double, handed on as two floats: differences of
            // sums stay exact to the last bit of the decays. A decay below -200
            // is a factor of zero in fp32 and is held there, so that no sum is
            // infinite and no difference NaN.
            double s[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int t = 2 * lane + x;
                float gt = a.g && t < len ? a.g[hrow + t] : 0.f;
                gt = gt < -200.f ? -200.f : gt;
                s[x] = (double)gt + (x ? s[0] : 0.0);
            }
            double base = s[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double u = __shfl_up_sync(0xffffffffu, base, o);
                if (lane >= o) base += u;
            }
            base -= s[1];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const double G = base + s[x];
                const float hi = (float)G;
                Gh[2 * lane + x] = hi;
                Gl[2 * lane + x] = (float)(G - (double)hi);
            }
        } else if (warp == 1) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int t = 2 * lane + x;
                eta[t] = t < len ? a.eta[hrow + t] : 0.f;
            }
        }
        __syncthreads();

        // A (transposed) and P from the products
        float pm[2] = {0.f, 0.f}, P[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * warp + gq + (e >> 1) * 8, j = 8 * nt + 2 * q4 + (e & 1);
                float av = 0.f, pv = 0.f;
                if (j <= i) {
                    const float gam = expf((Gh[i] - Gh[j]) + (Gl[i] - Gl[j])) * eta[j] * iK[j];
                    pv = a.q_scale * gam * (qk[nt][e] * iQ[i]);
                    if (j < i) av = gam * (kk[nt][e] * iK[i]);
                }
                Lt[j * kLtStride + i] = av;
                P[nt][e] = pv;
                pm[e >> 1] = fmaxf(pm[e >> 1], fabsf(pv));
            }
        float sp[2], ip[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) pow2_scale(quad_max(pm[x]), sp[x], ip[x]);
        char *gP = a.im.P + hslot * 2 * kImg;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t hi, lo;
                split_f16(P[nt][2 * x] * sp[x], P[nt][2 * x + 1] * sp[x], hi, lo);
                const uint32_t o = img_off(16 * warp + gq + 8 * x, 8 * nt) + 4 * q4;
                *reinterpret_cast<uint32_t *>(gP + o) = hi;
                *reinterpret_cast<uint32_t *>(gP + kImg + o) = lo;
            }
        if (q4 == 0) {
            vec[kVp * C + 16 * warp + gq] = ip[0];
            vec[kVp * C + 16 * warp + gq + 8] = ip[1];
        }
        if (tid < C) {
            const float G = Gh[tid] + Gl[tid], GC = Gh[C - 1];
            const float dec = expf(G), rest = expf((GC - Gh[tid]) + (Gl[C - 1] - Gl[tid]));
            vec[kVk * C + tid] = dec * iK[tid];
            vec[kVu * C + tid] = rest * eta[tid] * iK[tid];
            vec[kVq * C + tid] = a.q_scale * dec * iQ[tid];
            vec[kVeta * C + tid] = iK[tid];
            vec[kVspare * C + tid] = iQ[tid];
            vec[kVgam * C + tid] = expf(GC + Gl[C - 1]);
        }
        __syncthreads();

        if (tid < C) {
            float x[C];
#pragma unroll
            for (int i = 0; i < C; ++i) x[i] = i == tid ? 1.f : 0.f;
#pragma unroll
            for (int k = 0; k < C - 1; ++k) {
                const float xk = x[k];
#pragma unroll
                for (int i = (k + 1) & ~3; i < C; i += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(Lt + k * kLtStride + i);
                    if (i > k) x[i] = fmaf(-l.x, xk, x[i]);
                    if (i + 1 > k) x[i + 1] = fmaf(-l.y, xk, x[i + 1]);
                    if (i + 2 > k) x[i + 2] = fmaf(-l.z, xk, x[i + 2]);
                    if (i + 3 > k) x[i + 3] = fmaf(-l.w, xk, x[i + 3]);
                }
            }
#pragma unroll
            for (int i = 0; i < C; ++i) Tm[i * kTmStride + tid] = x[i];
        }
        __syncthreads();
        {
            const int row = tid >> 1, half = tid & 1;
            const float *t = Tm + row * kTmStride + 32 * half;
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(t[j]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            float s, is;
            pow2_scale(m, s, is);
            char *gT = a.im.T + hslot * 2 * kImg;
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    split_f16(t[j + 2 * e] * s, t[j + 2 * e + 1] * s, hi[e], lo[e]);
                const uint32_t o = img_off(row, 32 * half + j);
                *reinterpret_cast<uint4 *>(gT + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(gT + kImg + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            if (half == 0) vec[kVt * C + row] = is;
        }
    }
}

// ---------------------------------------------------------------- scan

struct ScanArgs {
    const void *V;
    const float *W0;
    void *Z;
    float *W_out;
    const int *seq_start;
    int B, Hk, H, T, dv, w_heads;  // w_heads: 0 when W0 is shared by the sequences
    int warps;                     // compute warps of a block, 16 columns of W each
    int stages;
    Images im;
    int *status;
};

constexpr int kScanStatus = 61;

// Bytes of one stage: K, Q, T (two terms), P (one or two), vectors.
template <int DK, bool BF16, bool ZF>
constexpr int scan_stage_bytes() {
    return 2 * C * DK * 2 * (BF16 ? 1 : 2) + 2 * kImg + (ZF ? 2 : 1) * kImg + kVecBytes;
}
template <bool BF16>
constexpr int v_tile_bytes() { return BF16 ? C * 32 : C * 20 * 4; }

// Scan over the chunks. A warp owns 16 columns of W for the whole sequence, as the
// rows of W^T [16][DK] in accumulator registers: accumulator fragments
// packed pairwise are A fragments, so W^T K^T, X^T T^T, rho^T P^T and
// rho^T K follow one another in registers, and no warp waits for another.
// The chunk's images come through a ring of shared-memory stages, filled with
// bulk copies that the first thread issues; V through registers, one chunk ahead.
// ZF: Z in fp32, its products with two terms.
template <int DK, bool BF16, bool ZF>
__global__ void __launch_bounds__(256, 1) delta_scan_kernel(ScanArgs a) {
    extern __shared__ __align__(1024) char ssm[];
    __shared__ uint64_t full[4], empty[4];
    __shared__ int abort_flag;
    constexpr int STAGE = scan_stage_bytes<DK, BF16, ZF>();
    constexpr int KIMG = C * DK * 2, KALL = KIMG * (BF16 ? 1 : 2);
    constexpr int NT = DK / 8;
    const int groups = a.dv / (16 * a.warps);
    const int grp = blockIdx.x % groups, sh = blockIdx.x / groups;
    const int n = sh / a.H, h = sh % a.H, hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int t0, len;
    delta_span(a.seq_start, n, a.T, t0, len);
    const int nchunk = (len + C - 1) / C;
    const int slot0 = first_slot(a.seq_start, n, a.T, t0);
    const int b = a.seq_start ? 0 : n;
    volatile int *abort = &abort_flag;

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], a.warps);
        }
        fence_mbar_init();
    }
    __syncthreads();

    // Fills the stage of chunk c (one thread): stages - 1 chunks ahead of the
    // one being worked on, once every warp has left the stage's last chunk.
    auto fill = [&](int c) {
        const int s = c % a.stages;
        if (c >= a.stages &&
            !mbar_wait(&empty[s], ((c / a.stages) & 1) ^ 1, abort, a.status, kScanStatus))
            return;
        char *d = ssm + s * STAGE;
        const size_t ks = (size_t)(slot0 + c) * a.Hk + hk, hs = (size_t)(slot0 + c) * a.H + h;
        mbar_arrive_expect_tx(&full[s], STAGE);
        bulk_load(d, a.im.K + ks * KALL, KALL, &full[s]);
        bulk_load(d + KALL, a.im.Q + ks * KALL, KALL, &full[s]);
        bulk_load(d + 2 * KALL, a.im.T + hs * 2 * kImg, 2 * kImg, &full[s]);
        bulk_load(d + 2 * KALL + 2 * kImg, a.im.P + hs * 2 * kImg, (ZF ? 2 : 1) * kImg, &full[s]);
        bulk_load(d + STAGE - kVecBytes, a.im.vec + hs * kVecBytes, kVecBytes, &full[s]);
    };
    if (tid == 0)
        for (int c = 0; c < nchunk && c < a.stages - 1; ++c) fill(c);

    const int gq = lane >> 2, q4 = lane & 3;
    const int v0 = (grp * a.warps + warp) * 16;
    const size_t vrow = ((size_t)b * a.H + h) * a.T + t0;
    char *vt = ssm + a.stages * STAGE + warp * v_tile_bytes<BF16>();
    constexpr int VU = BF16 ? 4 : 8;  // 16-byte units of V per lane
    uint4 vr[VU];
    auto fetch_v = [&](int c) {
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int u = lane + 32 * i, row = BF16 ? u >> 1 : u >> 2, part = BF16 ? u & 1 : u & 3;
            vr[i] = make_uint4(0, 0, 0, 0);
            if (c * C + row < len) {
                const size_t at = (vrow + c * C + row) * a.dv + v0;
                vr[i] = BF16 ? *reinterpret_cast<const uint4 *>(
                                   static_cast<const __nv_bfloat16 *>(a.V) + at + 8 * part)
                             : *reinterpret_cast<const uint4 *>(static_cast<const float *>(a.V) +
                                                                at + 4 * part);
            }
        }
    };
    // W^T: row gq (elements 0, 1) and gq + 8 (2, 3), columns 8 nt + 2 q4 + {0, 1}
    float S[NT][4];
    const size_t state = (size_t)DK * a.dv;
    const float *w0 =
        a.W0 ? a.W0 + ((size_t)n * a.w_heads + h) * state + v0 : nullptr;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[nt][e] = w0 ? w0[(size_t)(8 * nt + 2 * q4 + (e & 1)) * a.dv + gq + (e >> 1) * 8] : 0.f;
    if (nchunk > 0) fetch_v(0);

    for (int c = 0; c < nchunk; ++c) {
        const int s = c % a.stages;
        if (tid == 0 && c + a.stages - 1 < nchunk) fill(c + a.stages - 1);
        if (!mbar_wait_warp(&full[s], (c / a.stages) & 1, abort, a.status, kScanStatus)) {
            // copies in flight land before the block's shared memory goes
            if (tid == 0)
                for (int p = c; p < c + a.stages && p < nchunk; ++p)
                    mbar_drain(&full[p % a.stages], (p / a.stages) & 1);
            return;
        }
        const uint32_t uK = smem_u32(ssm + s * STAGE), uQ = uK + KALL, uT = uQ + KALL,
                       uP = uT + 2 * kImg;
        const float *vec = reinterpret_cast<const float *>(ssm + (s + 1) * STAGE - kVecBytes);

        // X^T = W^T K^T, Z^T = W^T Q^T (both still scaled)
        float X[8][4] = {}, Z[8][4] = {};
        float iS[2];
        {
            float sS[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float m = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    m = fmaxf(m, fmaxf(fabsf(S[nt][2 * x]), fabsf(S[nt][2 * x + 1])));
                pow2_scale(quad_max(m), sS[x], iS[x]);
            }
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int nt = 2 * kk + (r >> 1), x = r & 1;
                    split_f16(S[nt][2 * x] * sS[x], S[nt][2 * x + 1] * sS[x], hi[r], lo[r]);
                }
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t bk[4], bq[4];
                    load_b(bk, uK, 16 * np, 16 * kk, lane);
                    load_b(bq, uQ, 16 * np, 16 * kk, lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(X[2 * np + x], hi, bk[2 * x], bk[2 * x + 1]);
                        mma_f16(X[2 * np + x], lo, bk[2 * x], bk[2 * x + 1]);
                        mma_f16(Z[2 * np + x], hi, bq[2 * x], bq[2 * x + 1]);
                        if (ZF) mma_f16(Z[2 * np + x], lo, bq[2 * x], bq[2 * x + 1]);
                    }
                    if (!BF16) {
                        load_b(bk, uK + KIMG, 16 * np, 16 * kk, lane);
#pragma unroll
                        for (int x = 0; x < 2; ++x) mma_f16(X[2 * np + x], hi, bk[2 * x], bk[2 * x + 1]);
                        if (ZF) {
                            load_b(bq, uQ + KIMG, 16 * np, 16 * kk, lane);
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                mma_f16(Z[2 * np + x], hi, bq[2 * x], bq[2 * x + 1]);
                        }
                    }
                }
            }
        }

        // X = V - D K W
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int u = lane + 32 * i;
            // bf16: rows of 32 bytes, the halves of every other four rows swapped
            // (eight rows of an ldmatrix then meet all banks); fp32: 80 bytes
            const int row = BF16 ? u >> 1 : u >> 2, part = BF16 ? u & 1 : u & 3;
            char *d = BF16 ? vt + row * 32 + ((part ^ ((row >> 2) & 1)) << 4) : vt + row * 80 + part * 16;
            *reinterpret_cast<uint4 *>(d) = vr[i];
        }
        __syncwarp();
        if (c + 1 < nchunk) fetch_v(c + 1);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            float v[2][4];
            if (BF16) {
                uint32_t r[4];  // tokens 16 np + {0..7, 8..15} x columns {0..7, 8..15}
                const int row = 16 * np + (lane & 7) + ((lane >> 4) << 3), part = (lane >> 3) & 1;
                ldsm_x4_t(r, smem_u32(vt) + row * 32 + ((part ^ ((row >> 2) & 1)) << 4));
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        v[x][2 * y] = __uint_as_float(r[2 * x + y] << 16);
                        v[x][2 * y + 1] = __uint_as_float(r[2 * x + y] & 0xFFFF0000u);
                    }
            } else {
                const float *f = reinterpret_cast<const float *>(vt);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[x][e] = f[(16 * np + 8 * x + 2 * q4 + (e & 1)) * 20 + gq + (e >> 1) * 8];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float2 ck = *reinterpret_cast<const float2 *>(vec + kVk * C + 16 * np + 8 * x + 2 * q4);
                float(&X4)[4] = X[2 * np + x];
                X4[0] = v[x][0] - ck.x * (iS[0] * X4[0]);
                X4[1] = v[x][1] - ck.y * (iS[0] * X4[1]);
                X4[2] = v[x][2] - ck.x * (iS[1] * X4[2]);
                X4[3] = v[x][3] - ck.y * (iS[1] * X4[3]);
            }
        }
        __syncwarp();

        // rho^T = X^T T^T
        float rho[8][4] = {};
        {
            float sX[2], iX[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float m = 0.f;
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
                    m = fmaxf(m, fmaxf(fabsf(X[nt][2 * x]), fabsf(X[nt][2 * x + 1])));
                pow2_scale(quad_max(m), sX[x], iX[x]);
            }
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int nt = 2 * jj + (r >> 1), x = r & 1;
                    split_f16(X[nt][2 * x] * sX[x], X[nt][2 * x + 1] * sX[x], hi[r], lo[r]);
                }
#pragma unroll
                for (int np = jj; np < 4; ++np) {  // T_ij is zero for i < j
                    uint32_t th[4], tl[4];
                    load_b(th, uT, 16 * np, 16 * jj, lane);
                    load_b(tl, uT + kImg, 16 * np, 16 * jj, lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(rho[2 * np + x], hi, th[2 * x], th[2 * x + 1]);
                        mma_f16(rho[2 * np + x], lo, th[2 * x], th[2 * x + 1]);
                        mma_f16(rho[2 * np + x], hi, tl[2 * x], tl[2 * x + 1]);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 it = *reinterpret_cast<const float2 *>(vec + kVt * C + 8 * nt + 2 * q4);
                rho[nt][0] *= iX[0] * it.x;
                rho[nt][1] *= iX[0] * it.y;
                rho[nt][2] *= iX[1] * it.x;
                rho[nt][3] *= iX[1] * it.y;
            }
        }

        // Z^T += rho^T P^T
        {
            float sR[2], iR[2], Y[8][4] = {};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float m = 0.f;
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
                    m = fmaxf(m, fmaxf(fabsf(rho[nt][2 * x]), fabsf(rho[nt][2 * x + 1])));
                pow2_scale(quad_max(m), sR[x], iR[x]);
            }
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int nt = 2 * jj + (r >> 1), x = r & 1;
                    split_f16(rho[nt][2 * x] * sR[x], rho[nt][2 * x + 1] * sR[x], hi[r], lo[r]);
                }
#pragma unroll
                for (int np = jj; np < 4; ++np) {
                    uint32_t ph[4], pl[4];
                    load_b(ph, uP, 16 * np, 16 * jj, lane);
                    if (ZF) load_b(pl, uP + kImg, 16 * np, 16 * jj, lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(Y[2 * np + x], hi, ph[2 * x], ph[2 * x + 1]);
                        if (ZF) {
                            mma_f16(Y[2 * np + x], lo, ph[2 * x], ph[2 * x + 1]);
                            mma_f16(Y[2 * np + x], hi, pl[2 * x], pl[2 * x + 1]);
                        }
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 cq = *reinterpret_cast<const float2 *>(vec + kVq * C + 8 * nt + 2 * q4);
                const float2 ip = *reinterpret_cast<const float2 *>(vec + kVp * C + 8 * nt + 2 * q4);
                const float z0 = cq.x * (iS[0] * Z[nt][0]) + ip.x * (iR[0] * Y[nt][0]);
                const float z1 = cq.y * (iS[0] * Z[nt][1]) + ip.y * (iR[0] * Y[nt][1]);
                const float z2 = cq.x * (iS[1] * Z[nt][2]) + ip.x * (iR[1] * Y[nt][2]);
                const float z3 = cq.y * (iS[1] * Z[nt][3]) + ip.y * (iR[1] * Y[nt][3]);
                if (ZF) {
                    const int t = c * C + 8 * nt + 2 * q4;
                    float *z = static_cast<float *>(a.Z) + (vrow + t) * a.dv + v0 + gq;
                    if (t < len) z[0] = z0, z[8] = z2;
                    if (t + 1 < len) z[a.dv] = z1, z[a.dv + 8] = z3;
                } else {
                    // 8 x 8 blocks transposed between the lanes: a token per row
                    const __nv_bfloat162 p0 = __floats2bfloat162_rn(z0, z1);
                    const __nv_bfloat162 p1 = __floats2bfloat162_rn(z2, z3);
                    const uint32_t r0 = movt(*reinterpret_cast<const uint32_t *>(&p0));
                    const uint32_t r1 = movt(*reinterpret_cast<const uint32_t *>(&p1));
                    const int t = c * C + 8 * nt + gq;
                    if (t < len) {
                        uint32_t *z = reinterpret_cast<uint32_t *>(
                            static_cast<__nv_bfloat16 *>(a.Z) + (vrow + t) * a.dv + v0 + 2 * q4);
                        z[0] = r0;
                        z[4] = r1;
                    }
                }
            }
        }

        // W'^T = exp(G_C) W^T + (rho u)^T K
        {
            float sR[2], iR[2];
            float m0 = 0.f, m1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 cu = *reinterpret_cast<const float2 *>(vec + kVu * C + 8 * nt + 2 * q4);
                rho[nt][0] *= cu.x, rho[nt][1] *= cu.y, rho[nt][2] *= cu.x, rho[nt][3] *= cu.y;
                m0 = fmaxf(m0, fmaxf(fabsf(rho[nt][0]), fabsf(rho[nt][1])));
                m1 = fmaxf(m1, fmaxf(fabsf(rho[nt][2]), fabsf(rho[nt][3])));
            }
            pow2_scale(quad_max(m0), sR[0], iR[0]);
            pow2_scale(quad_max(m1), sR[1], iR[1]);
            uint32_t hi[4][4], lo[4][4];
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int nt = 2 * jj + (r >> 1), x = r & 1;
                    split_f16(rho[nt][2 * x] * sR[x], rho[nt][2 * x + 1] * sR[x], hi[jj][r], lo[jj][r]);
                }
            const float gam = vec[kVgam * C];
#pragma unroll
            for (int np = 0; np < DK / 16; ++np) {
                float U[2][4] = {};
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    uint32_t bk[4];
                    load_bt(bk, uK, 16 * jj, 16 * np, lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(U[x], hi[jj], bk[2 * x], bk[2 * x + 1]);
                        mma_f16(U[x], lo[jj], bk[2 * x], bk[2 * x + 1]);
                    }
                    if (!BF16) {
                        load_bt(bk, uK + KIMG, 16 * jj, 16 * np, lane);
#pragma unroll
                        for (int x = 0; x < 2; ++x) mma_f16(U[x], hi[jj], bk[2 * x], bk[2 * x + 1]);
                    }
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        S[2 * np + x][e] = fmaf(iR[e >> 1], U[x][e], gam * S[2 * np + x][e]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
    }

    if (a.W_out) {
        float *w = a.W_out + ((size_t)n * a.H + h) * state + v0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[(size_t)(8 * nt + 2 * q4 + (e & 1)) * a.dv + gq + (e >> 1) * 8] = S[nt][e];
    }
}

template <int DK, bool BF16>
cudaError_t prep_inst(const PrepArgs &r, int blocks, cudaStream_t s) {
    constexpr int smem = prep_smem<DK, BF16>();
    cudaError_t e = cudaFuncSetAttribute(delta_prep_kernel<DK, BF16>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    delta_prep_kernel<DK, BF16><<<blocks, kPrepThreads, smem, s>>>(r);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}

// Compute warps of a block: all of a head's columns when there are heads enough
// to fill the SMs, else half or a quarter of them, so that more SMs take part.
int scan_warps(long long heads, int dv) {
    int w = dv / 16;
    while (w > 2 && heads * (dv / (16 * w)) < 148) w /= 2;
    return w;
}

template <int DK, bool BF16, bool ZF>
cudaError_t scan_inst(ScanArgs r, int N, cudaStream_t s) {
    r.warps = scan_warps((long long)N * r.H, r.dv);
    constexpr int stage = scan_stage_bytes<DK, BF16, ZF>();
    const int vbytes = r.warps * v_tile_bytes<BF16>();
    r.stages = (226 * 1024 - vbytes) / stage;
    r.stages = r.stages > 3 ? 3 : r.stages;
    const int smem = r.stages * stage + vbytes;
    cudaError_t e = cudaFuncSetAttribute(delta_scan_kernel<DK, BF16, ZF>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((long long)N * r.H * (r.dv / (16 * r.warps)));
    delta_scan_kernel<DK, BF16, ZF><<<grid, 32 * r.warps, smem, s>>>(r);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}

}  // namespace

Images images_at(const Plan &p, void *workspace) {
    char *w = static_cast<char *>(workspace);
    return Images{w + p.oK, w + p.oQ, w + p.oT, w + p.oP, w + p.oV, p.kimg};
}

cudaError_t launch_prep(const DeltaArgs &a, const Plan &p, const Images &im, cudaStream_t s) {
    const PrepArgs r{a.Q, a.K, a.eta, a.g, a.seq_start, a.B, a.Hk, a.H, a.T, a.N, a.q_scale, im};
    const int blocks = p.slots * a.Hk;
    if (a.dk == 64) return a.bf16 ? prep_inst<64, true>(r, blocks, s) : prep_inst<64, false>(r, blocks, s);
    return a.bf16 ? prep_inst<128, true>(r, blocks, s) : prep_inst<128, false>(r, blocks, s);
}

}  // namespace delta

using namespace delta;

size_t delta_workspace_bytes(int B, int Hk, int H, int T, int dk, int dv, int N, bool packed,
                             bool bf16) {
    (void)dv;
    return make_plan(B, Hk, H, T, dk, N, packed, bf16).end;
}

cudaError_t launch_delta_fwd(const DeltaArgs &a, cudaStream_t s) {
    const Plan p = make_plan(a.B, a.Hk, a.H, a.T, a.dk, a.N, a.seq_start != nullptr, a.bf16);
    const Images im = images_at(p, a.workspace);
    cudaError_t e = launch_prep(a, p, im, s);
    if (e != cudaSuccess) return e;
    const ScanArgs r{a.V, a.W0, a.Z, a.W_out, a.seq_start, a.B, a.Hk, a.H, a.T, a.dv,
                     a.w0_per_seq ? a.H : 0, 0, 0, im, device_status_word()};
    if (a.dk == 64) {
        if (a.bf16) return a.z_bf16 ? scan_inst<64, true, false>(r, a.N, s) : scan_inst<64, true, true>(r, a.N, s);
        return a.z_bf16 ? scan_inst<64, false, false>(r, a.N, s) : scan_inst<64, false, true>(r, a.N, s);
    }
    if (a.bf16) return a.z_bf16 ? scan_inst<128, true, false>(r, a.N, s) : scan_inst<128, true, true>(r, a.N, s);
    return a.z_bf16 ? scan_inst<128, false, false>(r, a.N, s) : scan_inst<128, false, true>(r, a.N, s);
}

}  // namespace ttt
