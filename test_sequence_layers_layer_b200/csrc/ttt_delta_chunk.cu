// ttt_delta_chunk.cu -- chunked forward of the gated delta rule: the per-chunk
// preparation (all chunks at once) and the scan over the chunks.
//
// For a chunk of C = 64 tokens that starts from W, with G_i the sum of the decays
// up to token i, D = diag(exp G), Gam_ij = exp(G_i - G_j):
//   X = V - D K W,   (I + A) rho = X,   A_ij = Gam_ij (k_i.k_j) eta_j   (j < i)
//   Z = c D Q W + P rho,                P_ij = c Gam_ij (q_i.k_j) eta_j (j <= i)
//   W' = exp(G_C) W + sum_j u_j k_j^T rho_j,  u_j = exp(G_C - G_j) eta_j.
// T = (I + A)^-1, P and the decays depend on q, k, eta and g alone, and rho = T X
// is linear in X, so one kernel forms
//   M = P T [64][64] and H = T^T diag(u) K [64][dk]
// for all chunks in parallel. One chunk after the other remains
//   X = V - D K W,   Z = c D Q W + M X,   W' = exp(G_C) W + H^T X:
// two products deep instead of three, and X is the only operand besides W that
// has to be brought into operand form on the way.
//
// Chunks of 64: the products per token grow with C (C (dk + dv) and C^2 / 3 for the
// inverse) and the chain has T / C steps, each of which costs latency more than
// products; 64 is also the largest whose images, twice over, fit beside one another in
// shared memory at dk = 128. The products are warp-level MMAs: tiles of 16 x 64 x 32
// that follow one another through registers, of which the tensor pipe is busy 12 - 38 %
// of the time; a tcgen05 instruction costs about 150 cycles of the chain whatever its
// width, and its accumulators would have to come back from tensor memory at each of the
// chain's two turns. The forward's bytes (4 dk + 4 dv + 8 a token and head with bf16 in
// and out) are no bound: 4 x 32768 x 8 heads of 128 need 166 us at the copy rate and
// take 2215, 730 in the preparation and 1485 in the scan.
#include "../../include/ttt.h"
#include "ttt_delta_mma.cuh"

namespace ttt {
namespace delta {
namespace {

// ---------------------------------------------------------------- preparation

constexpr int kPrepThreads = 256;

struct PrepArgs {
    const void *Q, *K;
    const float *eta, *g;
    const int *seq_start;
    int B, Hk, H, T, N;
    float q_scale;
    Images im;
};

// A 64-row image of Q or K by 128 threads: rows in global memory to scaled fp16
// terms, in shared memory and in the workspace; inv[row] = 1 / scale. All loads
// are on their way before the first is used.
template <int DK, bool BF16>
__device__ __forceinline__ void convert_rows(const void *src, size_t row0, int len, char *sm,
                                             char *gm, float *inv, int tid) {
    constexpr int LPR = DK / 8, RPP = 128 / LPR, NP = C / RPP;  // lanes per row, rows per pass
    const int sub = tid % LPR;
    uint4 raw[NP][BF16 ? 1 : 2];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + tid / LPR;
        const size_t at = (row0 + row) * DK + sub * 8;
#pragma unroll
        for (int y = 0; y < (BF16 ? 1 : 2); ++y) {
            raw[p][y] = make_uint4(0, 0, 0, 0);
            if (row < len)
                raw[p][y] = BF16 ? *reinterpret_cast<const uint4 *>(
                                       static_cast<const __nv_bfloat16 *>(src) + at)
                                 : *reinterpret_cast<const uint4 *>(
                                       static_cast<const float *>(src) + at + 4 * y);
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + tid / LPR;
        float x[8];
        const uint32_t w[8] = {raw[p][0].x, raw[p][0].y, raw[p][0].z, raw[p][0].w,
                               raw[p][BF16 ? 0 : 1].x, raw[p][BF16 ? 0 : 1].y,
                               raw[p][BF16 ? 0 : 1].z, raw[p][BF16 ? 0 : 1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = __uint_as_float(!BF16 ? w[j] : (j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
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

constexpr int kLd = 68;  // row stride of the fp32 64 x 64 matrices (floats)

// Vectors of the preparation: 1 / scales of K and Q, sums of decays as two floats,
// eta / sK, and of the decays what the triangle needs (below), u, 1 / scales of T.
enum PrepVec { kPiK, kPiQ, kPGh, kPGl, kPek, kProw, kPcol, kPu = kPcol + 3, kPiT, kPrepVecs };

// Shared memory: K and Q images, A and T in fp32; the images that go out take
// the places of what is no longer needed (T's terms and then M over A, H's high
// terms over Q, its low terms over T).
template <int DK, bool BF16>
constexpr int prep_smem() {
    return 2 * C * DK * 2 * (BF16 ? 1 : 2) + 2 * 4 * C * kLd + 4 * kPrepVecs * C + 4 * 32 * 36;
}

// T = (I + L)^-1 for L strictly lower triangular, in fp32, by 128 threads (named
// barrier `bar`): the four 16 x 16 diagonal blocks by forward substitution (a lane per
// column), then twice T_21 = -T_22 (L_21 T_11): for the two pairs of 16-blocks, and for
// the pair of 32-blocks that they make. Writes the lower blocks and what lies above
// the diagonal inside the 32 x 32 ones; Y: 32 x 36 floats.
__device__ __forceinline__ void invert(const float *L, float *T, float *Y, int tid, int bar) {
    const int warp = tid >> 5, lane = tid & 31;
    if (lane < 16) {
        const float *l = L + 16 * warp * kLd + 16 * warp;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == lane ? 1.f : 0.f;
#pragma unroll
        for (int i = 1; i < 16; ++i) {  // row i of L as vectors: the same for all lanes
            float y = 0.f;              // two chains
#pragma unroll
            for (int k4 = 0; k4 < i; k4 += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(l + i * kLd + k4);
                x[i] = fmaf(-v.x, x[k4], x[i]);
                if (k4 + 1 < i) y = fmaf(v.y, x[k4 + 1], y);
                if (k4 + 2 < i) x[i] = fmaf(-v.z, x[k4 + 2], x[i]);
                if (k4 + 3 < i) y = fmaf(v.w, x[k4 + 3], y);
            }
            x[i] -= y;
        }
        float *t = T + 16 * warp * kLd + 16 * warp + lane;
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i * kLd] = x[i];
        if (!(warp & 1))  // above the pair's lower block: zeros, so that 32-blocks are whole
#pragma unroll
            for (int i = 0; i < 16; ++i) t[i * kLd + 16] = 0.f;
    }
    named_bar(bar, 128);
    constexpr int kY = 36;
    // R rows, four columns a thread: out = sign * X[rows][0 .. K) W[0 .. K)[cols]
    auto product = [&](const float *X, int ldx, const float *W, int ldw, float *out, int ldo, int K,
                       int r0, int rows, float sign) {
        float acc[2][4] = {};
#pragma unroll 4
        for (int k = 0; k < K; k += 4) {
            float4 x[2];
#pragma unroll
            for (int y = 0; y < 2; ++y)
                if (y < rows) x[y] = *reinterpret_cast<const float4 *>(X + (r0 + y) * ldx + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 w = *reinterpret_cast<const float4 *>(W + (k + e) * ldw);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    if (y >= rows) continue;
                    const float f = e == 0 ? x[y].x : e == 1 ? x[y].y : e == 2 ? x[y].z : x[y].w;
                    acc[y][0] = fmaf(f, w.x, acc[y][0]), acc[y][1] = fmaf(f, w.y, acc[y][1]);
                    acc[y][2] = fmaf(f, w.z, acc[y][2]), acc[y][3] = fmaf(f, w.w, acc[y][3]);
                }
            }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
            if (y < rows)
                *reinterpret_cast<float4 *>(out + (r0 + y) * ldo) = make_float4(
                    sign * acc[y][0], sign * acc[y][1], sign * acc[y][2], sign * acc[y][3]);
    };
    {  // two pairs of 16-blocks: 64 threads each, a row and four columns
        const int pair = tid >> 6, r = (tid & 63) >> 2, c = (tid & 3) * 4, o = 32 * pair;
        float *y = Y + 16 * pair * kY + c;
        product(L + (o + 16) * kLd + o, kLd, T + o * kLd + o + c, kLd, y, kY, 16, r, 1, 1.f);
        named_bar(bar, 128);
        product(T + (o + 16) * kLd + o + 16, kLd, y, kY, T + (o + 16) * kLd + o + c, kLd, 16, r, 1, -1.f);
        named_bar(bar, 128);
    }
    {  // the pair of 32-blocks: two rows and four columns a thread
        const int r = (tid >> 3) * 2, c = (tid & 7) * 4;
        product(L + 32 * kLd, kLd, T + c, kLd, Y + c, kY, 32, r, 2, 1.f);
        named_bar(bar, 128);
        product(T + 32 * kLd + 32, kLd, Y + c, kY, T + 32 * kLd + c, kLd, 32, r, 2, -1.f);
        named_bar(bar, 128);
    }
}

// One block per chunk and key head, its value heads one after the other. Warps
// 0..3 work for Z (q_i.k_j, P, T's terms, M), warps 4..7 for the weight (k_i.k_j, A, T,
// H), 16 rows each. The decays Gam_ij of a block below the diagonal come as
// products of two factors that are at most 1, around the last token r before the rows'
// block: exp(G_i - G_r) exp(G_r - G_j); only the diagonal blocks take an exponential
// an element.
// What bounds it is latency: a block is a row of dependent phases (rows to images,
// k.k and the gates, A, the inverse, T's terms, M and H: 24,000 cycles at dk = 128), and
// two blocks an SM are all that registers (128 a thread) and shared memory hold. Issue
// slots are used to 43 %, shared memory to 50 %, DRAM to 22 %, the tensor pipe to
// 12 %; barriers are the largest stall. 16,384 chunks of 64 x 128 (bf16) take
// 730 us, 45 ns each. Four warps a block took 1168, eight that all did the same 895, an
// inverse of one level with the gates loaded where they are used 772.
template <int DK, bool BF16>
__global__ void __launch_bounds__(kPrepThreads, 2) delta_prep_kernel(PrepArgs a) {
    extern __shared__ __align__(128) char psm[];
    constexpr int KIMG = C * DK * 2, IMG = KIMG * (BF16 ? 1 : 2);
    char *sK = psm, *sQ = sK + IMG;
    float *L = reinterpret_cast<float *>(sQ + IMG);  // A of the chunk, row-major
    float *T = L + C * kLd;
    float *pv = T + C * kLd, *Y = pv + kPrepVecs * C;
    const float *iK = pv + kPiK * C, *iQ = pv + kPiQ * C, *Gh = pv + kPGh * C, *Gl = pv + kPGl * C,
                *ek = pv + kPek * C, *it = pv + kPiT * C, *u = pv + kPu * C;
    char *sT = reinterpret_cast<char *>(L);   // T's two terms, then M's
    char *sHl = reinterpret_cast<char *>(T);  // H's low terms; its high terms over Q
    const int slot = blockIdx.x / a.Hk, hk = blockIdx.x % a.Hk;
    int n, t0, len;
    if (!ChunkSearch{a.seq_start, a.T, a.N}.find(slot, n, t0, len)) return;
    const int b = a.seq_start ? 0 : n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, q4 = lane & 3;
    const int mt = warp & 3;
    const bool forw = warp >= 4;  // works for the weight
    const size_t kslot = (size_t)slot * a.Hk + hk;
    const size_t krow = ((size_t)b * a.Hk + hk) * a.T + t0;
    const int rep = a.H / a.Hk;
    // the gates of a head: loaded a head ahead (the first with the rows)
    float g2[2] = {0.f, 0.f}, eta1 = 0.f;
    auto load_gates = [&](int h) {
        const size_t hrow = ((size_t)b * a.H + h) * a.T + t0;
        if (warp == 0)
#pragma unroll
            for (int x = 0; x < 2; ++x) g2[x] = a.g && 2 * lane + x < len ? a.g[hrow + 2 * lane + x] : 0.f;
        if (tid < 2 * C) eta1 = (tid & 63) < len ? a.eta[hrow + (tid & 63)] : 0.f;
    };
    load_gates(hk * rep);
    // Sums of decays in double, handed on as two floats: differences of sums stay
    // exact to the last bit of the decays. A decay below -200 is a factor of zero in
    // fp32 and is held there, so that no sum is infinite and no difference NaN.
    auto sum_gates = [&]() {
        double s[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            s[x] = (double)(g2[x] < -200.f ? -200.f : g2[x]) + (x ? s[0] : 0.0);
        double base = s[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double v = __shfl_up_sync(0xffffffffu, base, o);
            if (lane >= o) base += v;
        }
        base -= s[1];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const double G = base + s[x];
            const float hi = (float)G;
            pv[kPGh * C + 2 * lane + x] = hi;
            pv[kPGl * C + 2 * lane + x] = (float)(G - (double)hi);
        }
    };
    if (forw)
        convert_rows<DK, BF16>(a.K, krow, len, sK, a.im.K + kslot * a.im.kimg, pv + kPiK * C, tid & 127);
    else
        convert_rows<DK, BF16>(a.Q, krow, len, sQ, a.im.Q + kslot * a.im.kimg, pv + kPiQ * C, tid);
    if (warp == 0) sum_gates();
    __syncthreads();

    // k_i.k_j or q_i.k_j of this warp's 16 rows i, columns j up to the diagonal; products
    // of low terms in sums of their own (the tensor cores cut off what is below a
    // sum's last bit, once a product)
    float kk[8][4] = {}, small[BF16 ? 1 : 8][4] = {};
    const uint32_t uK = smem_u32(sK), uA = forw ? uK : smem_u32(sQ);
#pragma unroll
    for (int k = 0; k < DK; k += 16) {
        uint32_t ah[4], al[4];
        ldsm_x4(ah, ldsm_addr(uA, 16 * mt, k, lane));
        if (!BF16) ldsm_x4(al, ldsm_addr(uA + KIMG, 16 * mt, k, lane));
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            if (np > mt) break;
            uint32_t bb[4];
            load_b(bb, uK, 16 * np, k, lane);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                mma_f16(kk[2 * np + x], ah, bb[2 * x], bb[2 * x + 1]);
                if (!BF16) mma_f16(small[BF16 ? 0 : 2 * np + x], al, bb[2 * x], bb[2 * x + 1]);
            }
            if (!BF16) {
                load_b(bb, uK + KIMG, 16 * np, k, lane);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    mma_f16(small[BF16 ? 0 : 2 * np + x], ah, bb[2 * x], bb[2 * x + 1]);
            }
        }
    }
    if (!BF16)
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) kk[nt][e] += small[BF16 ? 0 : nt][e];

    for (int r = 0; r < rep; ++r) {
        const int h = hk * rep + r;
        const size_t hslot = (size_t)slot * a.H + h;
        float *vec = reinterpret_cast<float *>(a.im.vec + hslot * kVecBytes);
        if (r > 0) {
            if (tid == 0 || tid == 128) bulk_wait_read<0>();  // the head before has gone out
            if (warp == 0) sum_gates();
            __syncthreads();
        }
        if (tid < 2 * C) {
            const int j = tid & 63;
            const float hj = Gh[j], lj = Gl[j];
            auto from = [&](int i) { return expf((Gh[i] - hj) + (Gl[i] - lj)); };
            const float e = eta1 * iK[j];
            if (tid < C) {
                const float dec = expf(hj + lj);
                pv[kPek * C + j] = e;
                const int q = j < 16 ? j : (j & ~15) - 1;
                pv[kProw * C + j] = expf((hj - Gh[q]) + (lj - Gl[q]));
                pv[kPu * C + j] = from(C - 1) * e;
                vec[kVk * C + j] = dec * iK[j];
                vec[kVq * C + j] = a.q_scale * dec * iQ[j];
                if (j == 0) vec[kVs * C] = expf(Gh[C - 1] + Gl[C - 1]);
            } else {
#pragma unroll
                for (int y = 0; y < 3; ++y)  // around the last token before block y + 1
                    pv[(kPcol + y) * C + j] = j < 16 * (y + 1) ? from(16 * y + 15) * e : 0.f;
                vec[kVik * C + j] = iK[j];
                vec[kViq * C + j] = iQ[j];
                vec[kVgh * C + j] = hj;
                vec[kVgl * C + j] = lj;
            }
        }
        if (r + 1 < rep) load_gates(h + 1);
        __syncthreads();

        // A (to shared memory) or P (kept) from the products
        float P[8][4];
        {
            const int i0 = 16 * mt + gq, i1 = i0 + 8;
            const float si[2] = {forw ? iK[i0] : a.q_scale * iQ[i0], forw ? iK[i1] : a.q_scale * iQ[i1]};
            const float ri[2] = {si[0] * pv[kProw * C + i0], si[1] * pv[kProw * C + i1]};
            const float hi2[2] = {Gh[i0], Gh[i1]}, li2[2] = {Gl[i0], Gl[i1]};
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) P[nt][e] = 0.f;
                const int j0 = 8 * nt + 2 * q4;
                if (nt < 2 * mt) {  // below the diagonal blocks
                    const float2 cj = *reinterpret_cast<const float2 *>(pv + (kPcol + mt - 1) * C + j0);
                    P[nt][0] = kk[nt][0] * ri[0] * cj.x, P[nt][1] = kk[nt][1] * ri[0] * cj.y;
                    P[nt][2] = kk[nt][2] * ri[1] * cj.x, P[nt][3] = kk[nt][3] * ri[1] * cj.y;
                } else if (nt < 2 * mt + 2) {
                    const float2 hj = *reinterpret_cast<const float2 *>(Gh + j0);
                    const float2 lj = *reinterpret_cast<const float2 *>(Gl + j0);
                    const float2 ej = *reinterpret_cast<const float2 *>(ek + j0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = e < 2 ? i0 : i1, j = j0 + (e & 1);
                        const float d = (hi2[e >> 1] - (e & 1 ? hj.y : hj.x)) + (li2[e >> 1] - (e & 1 ? lj.y : lj.x));
                        const float f = kk[nt][e] * si[e >> 1] * (e & 1 ? ej.y : ej.x) * expf(d);
                        // above the diagonal the exponential may be infinite: chosen, not multiplied
                        P[nt][e] = (forw ? j < i : j <= i) ? f : 0.f;
                    }
                }
                if (forw && nt < 2 * mt + 2) {
                    float *l = L + i0 * kLd + j0;
                    *reinterpret_cast<float2 *>(l) = make_float2(P[nt][0], P[nt][1]);
                    *reinterpret_cast<float2 *>(l + 8 * kLd) = make_float2(P[nt][2], P[nt][3]);
                }
            }
        }

        if (forw) {
            named_bar(2, 128);  // A is there
            invert(L, T, Y, tid & 127, 2);
            named_arrive(3, 256);  // T is there
            // H = T^T diag(u) K: rows j of this warp, summed over tokens i >= j
            // (T^T's elements are read twice, once for the rows' scales: registers are short)
            float Hc[DK / 8][4] = {}, sA[2], iA[2];
            auto tile = [&](int nt, float(&A)[4]) {
                const int i = 8 * nt + 2 * q4;
                const float2 ui = *reinterpret_cast<const float2 *>(u + i);
                const float *t = T + i * kLd + 16 * mt + gq;
                // inside the diagonal block T holds zeros above the diagonal
                A[0] = ui.x * t[0], A[1] = ui.y * t[kLd];
                A[2] = ui.x * t[8], A[3] = ui.y * t[kLd + 8];
            };
            {
                float m[2] = {0.f, 0.f};
#pragma unroll
                for (int nt = 0; nt < 8; ++nt) {
                    if (nt < 2 * mt) continue;
                    float A[4];
                    tile(nt, A);
                    m[0] = fmaxf(m[0], fmaxf(fabsf(A[0]), fabsf(A[1])));
                    m[1] = fmaxf(m[1], fmaxf(fabsf(A[2]), fabsf(A[3])));
                }
                pow2_scale(quad_max(m[0]), sA[0], iA[0]);
                pow2_scale(quad_max(m[1]), sA[1], iA[1]);
            }
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                if (kb < mt) continue;
                uint32_t hi[4], lo[4];
                float A0[4], A1[4];
                tile(2 * kb, A0);
                tile(2 * kb + 1, A1);
                a_terms(A0, A1, sA, hi, lo);
#pragma unroll
                for (int np = 0; np < DK / 16; ++np) {
                    uint32_t bb[4];
                    load_bt(bb, uK, 16 * kb, 16 * np, lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(Hc[2 * np + x], hi, bb[2 * x], bb[2 * x + 1]);
                        mma_f16(Hc[2 * np + x], lo, bb[2 * x], bb[2 * x + 1]);
                    }
                    if (!BF16) {
                        load_bt(bb, uK + KIMG, 16 * kb, 16 * np, lane);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            mma_f16(Hc[2 * np + x], hi, bb[2 * x], bb[2 * x + 1]);
                    }
                }
            }
            // one scale for the 16 rows: they are one step of the sums over tokens
            float m[2] = {0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < DK / 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e >> 1] = fmaxf(m[e >> 1], fabsf(Hc[nt][e]));
            float mm = fmaxf(m[0] * iA[0], m[1] * iA[1]), sH, iH;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
            pow2_scale(mm, sH, iH);
            if (lane == 0) vec[kVs * C + 1 + mt] = iH;
            const float sHr[2] = {iA[0] * sH, iA[1] * sH};
            named_bar(4, 256);  // T is read, by both sides
#pragma unroll
            for (int nt = 0; nt < DK / 8; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t hi, lo;
                    split_f16(Hc[nt][2 * x] * sHr[x], Hc[nt][2 * x + 1] * sHr[x], hi, lo);
                    const uint32_t o = img_off(16 * mt + gq + 8 * x, 8 * nt) + 4 * q4;
                    *reinterpret_cast<uint32_t *>(sQ + o) = hi;
                    *reinterpret_cast<uint32_t *>(sHl + o) = lo;
                }
            fence_async_smem();
            named_bar(2, 128);
            if (tid == 128) {
                bulk_store(a.im.H + hslot * a.im.himg, sQ, KIMG);
                bulk_store(a.im.H + hslot * a.im.himg + KIMG, sHl, KIMG);
                bulk_commit();
            }
        } else {
            named_bar(3, 256);  // T is there
            // T's terms, row by row, over A
            {
                const int row = tid >> 1, side = tid & 1;
                const float *t = T + row * kLd + 32 * side;
                float v[32], m = 0.f;
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(t + j);
                    v[j] = w.x, v[j + 1] = w.y, v[j + 2] = w.z, v[j + 3] = w.w;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (32 * side + j > row) v[j] = 0.f;
                    m = fmaxf(m, fabsf(v[j]));
                }
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                float s, is;
                pow2_scale(m, s, is);
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        split_f16(v[j + 2 * e] * s, v[j + 2 * e + 1] * s, hi[e], lo[e]);
                    const uint32_t o = img_off(row, 32 * side + j);
                    const uint4 h4 = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    const uint4 l4 = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    *reinterpret_cast<uint4 *>(sT + o) = h4;
                    *reinterpret_cast<uint4 *>(sT + kImg + o) = l4;
                    if (a.im.T) {
                        char *gT = a.im.T + hslot * 2 * kImg;
                        *reinterpret_cast<uint4 *>(gT + o) = h4;
                        *reinterpret_cast<uint4 *>(gT + kImg + o) = l4;
                    }
                }
                if (side == 0) pv[kPiT * C + row] = is, vec[kVit * C + row] = is;
            }
            named_bar(1, 128);
            named_arrive(4, 256);  // T is read on this side
            // M = P T: rows i of this warp; T's row scales go into P's columns
            float M[8][4] = {}, sM[2], iM[2], sP[2], iP[2];
            const uint32_t uT = smem_u32(sT);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 t2 = *reinterpret_cast<const float2 *>(it + 8 * nt + 2 * q4);
                P[nt][0] *= t2.x, P[nt][1] *= t2.y, P[nt][2] *= t2.x, P[nt][3] *= t2.y;
            }
            row_scales<8>(P, sP, iP);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                if (jj > mt) break;
                uint32_t hi[4], lo[4];
                a_terms(P[2 * jj], P[2 * jj + 1], sP, hi, lo);
#pragma unroll
                for (int np = 0; np <= jj; ++np) {
                    uint32_t th[4], tl[4];
                    load_bt(th, uT, 16 * jj, 16 * np, lane);
                    load_bt(tl, uT + kImg, 16 * jj, 16 * np, lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(M[2 * np + x], hi, th[2 * x], th[2 * x + 1]);
                        mma_f16(M[2 * np + x], lo, th[2 * x], th[2 * x + 1]);
                        mma_f16(M[2 * np + x], hi, tl[2 * x], tl[2 * x + 1]);
                    }
                }
            }
            row_scales<8>(M, sM, iM);
            if (q4 == 0) {
                vec[kVm * C + 16 * mt + gq] = iP[0] * iM[0];
                vec[kVm * C + 16 * mt + gq + 8] = iP[1] * iM[1];
            }
            named_bar(1, 128);  // T's terms are read
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t hi, lo;
                    split_f16(M[nt][2 * x] * sM[x], M[nt][2 * x + 1] * sM[x], hi, lo);
                    const uint32_t o = img_off(16 * mt + gq + 8 * x, 8 * nt) + 4 * q4;
                    *reinterpret_cast<uint32_t *>(sT + o) = hi;
                    *reinterpret_cast<uint32_t *>(sT + kImg + o) = lo;
                }
            fence_async_smem();
            named_bar(1, 128);
            if (tid == 0) {
                bulk_store(a.im.M + hslot * 2 * kImg, sT, 2 * kImg);
                bulk_commit();
            }
        }
    }
    if (tid == 0 || tid == 128) bulk_wait_read<0>();  // shared memory is read; the writes end with the kernel
}

// ---------------------------------------------------------------- scan

struct ScanArgs {
    const void *V;
    const float *W0;
    void *Z;
    float *W_out;
    const int *seq_start;
    int B, Hk, H, T, dv, w_heads;  // w_heads: 0 when W0 is shared by the sequences
    int stages, zstages;           // of the chain's ring and of Z's
    Images im;
    float *saveS, *saveX;          // kSave: [slot][H][DK][dv] and [slot][H][64][dv]
    int *status;
};

// Bytes of a stage of the chain's ring (K, H with two terms, vectors) and of Z's (Q, M
// with two terms, vectors).
template <int DK, bool BF16>
constexpr int chain_stage_bytes() { return ((BF16 ? 1 : 2) + 2) * C * DK * 2 + kHalfVecBytes; }
template <int DK, bool BF16, int MODE>
constexpr int z_stage_bytes() {
    return MODE == kSave ? 0 : (BF16 ? 1 : 2) * C * DK * 2 + 2 * kImg + kHalfVecBytes;
}
// Where the 16-byte unit `part` of a token's 16 columns of V stands: rows of 32 bytes
// (bf16) with the halves of every other four swapped, so that the eight rows of an
// ldmatrix meet all banks, or of 64 (fp32) with the quarters turned by row pairs.
template <bool BF16>
__device__ __forceinline__ uint32_t v_off(int row, int part) {
    return BF16 ? row * 32 + ((part ^ ((row >> 2) & 1)) << 4)
                : row * 64 + ((part ^ ((row >> 1) & 3)) << 4);
}
// V of a block of 16 tokens as two tiles of V^T: columns gq (x, y) and gq + 8 (z, w) of
// tokens 8 x + 2 q4 + {0, 1}.
template <bool BF16>
__device__ __forceinline__ void load_v(float4 (&v)[2], const char *vt, int row0, int lane) {
    if (BF16) {
        uint32_t r[4];
        ldsm_x4_t(r, smem_u32(vt) + v_off<BF16>(row0 + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1));
#pragma unroll
        for (int x = 0; x < 2; ++x)
            v[x] = make_float4(__uint_as_float(r[2 * x] << 16), __uint_as_float(r[2 * x] & 0xFFFF0000u),
                               __uint_as_float(r[2 * x + 1] << 16),
                               __uint_as_float(r[2 * x + 1] & 0xFFFF0000u));
    } else {
        const int gq = lane >> 2, q4 = lane & 3;
        auto at = [&](int row, int col) {
            return *reinterpret_cast<const float *>(vt + v_off<BF16>(row, col >> 2) + (col & 3) * 4);
        };
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int t = row0 + 8 * x + 2 * q4;
            v[x] = make_float4(at(t, gq), at(t + 1, gq), at(t, gq + 8), at(t + 1, gq + 8));
        }
    }
}

// Behind the stages: the four warps' shares of X [to][from][2 tiles], and, twice for
// the chunks in turn, V [64][16], the terms of X [4 blocks][hi, lo], 1 / their
// scales and those of W^T, the terms of W^T [DK / 16][hi, lo].
template <bool BF16>
constexpr int scan_v_bytes() { return C * 16 * (BF16 ? 2 : 4); }
template <int DK, bool BF16, int MODE>
constexpr int scan_turn_bytes() {
    return scan_v_bytes<BF16>() + 4096 + 512 + (MODE == kSave ? 0 : DK / 16 * 512 * 2);
}
template <int DK, bool BF16, int MODE, int MT>
constexpr int scan_area_bytes() { return MT * (16 * 1024 + 2 * scan_turn_bytes<DK, BF16, MODE>()); }

// Scan over the chunks. Four warps own 16 MT columns of W for the whole sequence,
// as the rows of W^T [16 MT][DK] in accumulator registers, a quarter of DK each:
// accumulator fragments packed pairwise are A fragments, so W^T K^T and X^T H
// follow one another in registers. Twice a chunk the four meet:
//   1. each has its quarter's share of W^T K^T for all 64 tokens and hands the
//      others theirs; warp p then forms X of the 16 tokens of block p, and brings it
//      into operand form under that block's own row scales;
//   2. each takes the operand X of all blocks and updates its quarter of W.
// This chain is what bounds the scan, so all else is off it. Four more warps, a block
// of tokens each, form Z up to two chunks behind, from the operand forms of W^T and
// X that the chain leaves in shared memory (a quarter's rows under its own scales:
// the sums over the quarters and blocks are put together in fp32). One brings V to
// shared memory up to two chunks ahead. The chunks' images come by bulk copies
// through two rings of stages, K and H for the chain, Q and M for Z, so that the
// chain's next images need not wait for Z; one thread of a warp of its own fills
// each ring. The last warp, the gate, does the chain's waiting: a wait on an
// mbarrier costs a warp about 150 cycles even when nothing is waited for.
// Latency is the bound, the chain's and, where Z is formed, that of the four warps behind it:
// 1.5 us a chunk at dk = 128 and 1.2 us at 64 with 16 columns (2.9 and 2.2 with 32; the
// saving scan 1.25), of which the products are a third; shared memory is busy 53 %, the
// tensor pipe 38 %, DRAM 14 %. 4 x 32768 x 8 heads of 128 (bf16, bf16 Z): 1485 us; 8 x
// 2048 x 12 of 64: 114 us; the saving scan of 2 x 8192 x 8 of 128 160 us. A bf16 Z takes
// the products of an fp32 one and is rounded once: with one fp16 term an operand the
// first of these took 1240 us, and Z was off by 2^-11 of its terms' sizes, more than its own
// rounding where they cancel. Measured and not taken (Z with one term): two or one warps
// a group (1516, 2076 us for the first of these, Z on the chain), eight (2142: more exchange
// than products), two groups of 16 a block (1380), Z's stores on the chain (+ 193 cycles
// a chunk).
template <int DK, bool BF16, int MODE, int MT>
__global__ void __launch_bounds__(384, 1) delta_scan_kernel(ScanArgs a) {
    extern __shared__ __align__(128) char ssm[];
    __shared__ uint64_t full[4], empty[4], zfull[4], zempty[4];
    __shared__ uint64_t tready[2], zready[2];  // for the chunks in turn
    __shared__ int abort_flag;
    constexpr bool SAVE = MODE == kSave;
    constexpr int STAGE = chain_stage_bytes<DK, BF16>(), ZSTAGE = z_stage_bytes<DK, BF16, MODE>();
    constexpr int KIMG = C * DK * 2, KALL = KIMG * (BF16 ? 1 : 2);
    constexpr int NT = DK / 32, KK = DK / 64;  // 8-column tiles and 16-deep steps of a quarter
    const int groups = a.dv / (16 * MT);
    const int grp = blockIdx.x % groups, sh = blockIdx.x / groups;
    const int n = sh / a.H, h = sh % a.H, hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, p = warp & 3;
    int t0, len;
    delta_span(a.seq_start, n, a.T, t0, len);
    const int nchunk = (len + C - 1) / C;
    const int slot0 = first_slot(a.seq_start, n, a.T, t0);
    const int b = a.seq_start ? 0 : n;
    volatile int *abort = &abort_flag;

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < 4; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&zfull[s], 1);
            mbar_init(&zempty[s], 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&tready[t], SAVE ? 32 : 36);  // V is there (a warp), the four Z warps are done
            mbar_init(&zready[t], 4);
        }
        fence_mbar_init();
    }
    __syncthreads();

    const int gq = lane >> 2, q4 = lane & 3;
    const int v0 = grp * 16 * MT;
    const size_t vrow = ((size_t)b * a.H + h) * a.T + t0;
    char *zst = ssm + a.stages * STAGE, *area = zst + a.zstages * ZSTAGE;
    auto wait = [&](uint64_t *bar, int parity) {
        return mbar_wait_warp(bar, parity, abort, a.status, kScanStatus);
    };

    // what the chunks in turn keep for 16 columns: V, X's terms, 1 / scales, W^T's terms
    constexpr int VB = scan_v_bytes<BF16>();
    auto turn_at = [&](int turn, int m) {
        return area + MT * 16 * 1024 + (turn * MT + m) * scan_turn_bytes<DK, BF16, MODE>();
    };

    if (warp == 11) {  // ------------------------------------------------ the gate
        // Waits for all that a chunk needs and then meets the chain, which so waits on
        // nothing but barriers; at the next meeting the chain is done with the stage.
        Ring ring(a.stages);
        int last = 0;
        for (int c = 0; c < nchunk; ++c, ring.next()) {
            const bool ok = wait(&full[ring.s], ring.ph) && wait(&tready[c & 1], (c >> 1) & 1);
            if (named_bar_or(2, 160, !ok)) return;
            if (c > 0 && lane == 0) mbar_arrive(&empty[last]);
            last = ring.s;
        }
        return;
    }
    if (warp == 10) {  // ------------------------------------------------ V ahead
        // Rows of 16 columns by 16-byte asynchronous copies, zeros behind the sequence;
        // each lane's arrival follows its copies.
        constexpr int U = BF16 ? 4 : 8, PER = BF16 ? 2 : 4;  // units of a lane, of a row
        const size_t v_at = (vrow * a.dv + v0) * (BF16 ? 2 : 4);
        const char *src = static_cast<const char *>(a.V) + v_at;
        const size_t ld = (size_t)a.dv * (BF16 ? 2 : 4);
        for (int c = 0; c < nchunk; ++c) {
            // X of the chunk two before is formed: its V has been read
            if (c >= 2 && !wait(&zready[c & 1], ((c >> 1) & 1) ^ 1)) break;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t d = smem_u32(turn_at(c & 1, m));
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int u = lane + 32 * i, row = u / PER, part = u % PER, t = c * C + row;
                    const bool in = t < len;
                    cp_async16(d + v_off<BF16>(row, part),
                               src + (in ? t * ld : 0) + (m * PER + part) * 16, in);
                }
            }
            cp_async_arrive(&tready[c & 1]);
        }
        cp_async_wait_all();
        return;
    }
    if (warp >= 8) {  // ------------------------------------------------ the rings
        auto chain_copy = [&](int c, int s, uint64_t *bar) {
            char *d = ssm + s * STAGE;
            const size_t ks = (size_t)(slot0 + c) * a.Hk + hk, hs = (size_t)(slot0 + c) * a.H + h;
            mbar_arrive_expect_tx(bar, STAGE);
            bulk_load(d, a.im.K + ks * KALL, KALL, bar);
            bulk_load(d + KALL, a.im.H + hs * 2 * KIMG, 2 * KIMG, bar);
            bulk_load(d + STAGE - kHalfVecBytes, a.im.vec + hs * kVecBytes, kHalfVecBytes, bar);
        };
        auto z_copy = [&](int c, int s, uint64_t *bar) {
            char *d = zst + s * ZSTAGE;
            const size_t ks = (size_t)(slot0 + c) * a.Hk + hk, hs = (size_t)(slot0 + c) * a.H + h;
            mbar_arrive_expect_tx(bar, ZSTAGE);
            bulk_load(d, a.im.Q + ks * KALL, KALL, bar);
            bulk_load(d + KALL, a.im.M + hs * 2 * kImg, 2 * kImg, bar);
            bulk_load(d + ZSTAGE - kHalfVecBytes, a.im.vec + hs * kVecBytes + kHalfVecBytes,
                      kHalfVecBytes, bar);
        };
        if (lane == 0 && warp == 8) {
            Filler<decltype(chain_copy)> f(full, empty, a.stages, nchunk, abort, a.status, chain_copy);
            f.run();
        }
        if (lane == 0 && warp == 9 && !SAVE) {
            Filler<decltype(z_copy)> f(zfull, zempty, a.zstages, nchunk, abort, a.status, z_copy);
            f.run();
        }
        return;
    }

    if (warp >= 4) {  // ------------------------------------------------ Z behind
        if (SAVE) return;
        if (lane == 0) mbar_arrive(&tready[0]), mbar_arrive(&tready[1]);  // nothing to be done with yet
        Ring ring(a.zstages);
        for (int c = 0; c < nchunk; ++c, ring.next()) {
            const int turn = c & 1;
            const uint32_t uQ = smem_u32(zst + ring.s * ZSTAGE), uM = uQ + KALL;
            // the enum's order, counted from kVq on
            const float *vec = reinterpret_cast<const float *>(zst + (ring.s + 1) * ZSTAGE - kHalfVecBytes) - kVq * C;
            if (!wait(&zfull[ring.s], ring.ph) || !wait(&zready[turn], (c >> 1) & 1)) return;
#pragma unroll
            for (int m = 0; m < MT; ++m) {  // 16 columns
                const char *at = turn_at(turn, m);
                const uint4 *xfr = reinterpret_cast<const uint4 *>(at + VB) + lane;        // [block][hi, lo][32]
                const float *iXs = reinterpret_cast<const float *>(at + VB + 4096), *iSs = iXs + 64;
                const uint4 *sfr = reinterpret_cast<const uint4 *>(at + VB + 4096 + 512) + lane;  // [step][hi, lo][32]
                float Z[2][4] = {}, ZM[2][4] = {};
                // (Q W)^T of block p, quarter by quarter
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float z[2][4] = {};
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const uint4 *d = sfr + 64 * (w * KK + kk);
                        const uint4 fh = d[0], fl = d[32];
                        const uint32_t hi[4] = {fh.x, fh.y, fh.z, fh.w}, lo[4] = {fl.x, fl.y, fl.z, fl.w};
                        uint32_t bb[4];
                        load_b(bb, uQ, 16 * p, w * (DK / 4) + 16 * kk, lane);
#pragma unroll
                        for (int x = 0; x < 2; ++x) mma_f16(z[x], hi, bb[2 * x], bb[2 * x + 1]);
#pragma unroll
                        for (int x = 0; x < 2; ++x) mma_f16(z[x], lo, bb[2 * x], bb[2 * x + 1]);
                        if (!BF16) {
                            load_b(bb, uQ + KIMG, 16 * p, w * (DK / 4) + 16 * kk, lane);
#pragma unroll
                            for (int x = 0; x < 2; ++x) mma_f16(z[x], hi, bb[2 * x], bb[2 * x + 1]);
                        }
                    }
                    const float i0 = iSs[16 * w + gq], i1 = iSs[16 * w + gq + 8];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) Z[x][e] = fmaf(e < 2 ? i0 : i1, z[x][e], Z[x][e]);
                }
                // (M X)^T
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    if (jj > p) continue;  // M_ij is zero for i < j; the same for the whole warp
                    const uint4 fh = xfr[32 * (2 * jj)], fl = xfr[32 * (2 * jj + 1)];
                    const uint32_t hi[4] = {fh.x, fh.y, fh.z, fh.w}, lo[4] = {fl.x, fl.y, fl.z, fl.w};
                    const float i0 = iXs[16 * jj + gq], i1 = iXs[16 * jj + gq + 8];
                    float z[2][4] = {};
                    uint32_t bm[4];
                    load_b(bm, uM, 16 * p, 16 * jj, lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(z[x], hi, bm[2 * x], bm[2 * x + 1]);
                        mma_f16(z[x], lo, bm[2 * x], bm[2 * x + 1]);
                    }
                    load_b(bm, uM + kImg, 16 * p, 16 * jj, lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) mma_f16(z[x], hi, bm[2 * x], bm[2 * x + 1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) ZM[x][e] = fmaf(e < 2 ? i0 : i1, z[x][e], ZM[x][e]);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = 16 * p + 8 * x + 2 * q4;
                    const float2 cq = *reinterpret_cast<const float2 *>(vec + kVq * C + i);
                    const float2 im = *reinterpret_cast<const float2 *>(vec + kVm * C + i);
                    float(&z)[4] = Z[x], (&u)[4] = ZM[x];
                    z[0] = cq.x * z[0] + im.x * u[0], z[1] = cq.y * z[1] + im.y * u[1];
                    z[2] = cq.x * z[2] + im.x * u[2], z[3] = cq.y * z[3] + im.y * u[3];
                }
                // everything is read: the arrivals do not wait for the stores behind them
                __syncwarp();
                if (m == MT - 1 && lane == 0) {
                    mbar_arrive(&tready[turn]);
                    mbar_arrive(&zempty[ring.s]);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = c * C + 16 * p + 8 * x;
                    const float(&z)[4] = Z[x];
                    if (MODE == kZ32) {
                        const int t = i + 2 * q4;
                        float *o = static_cast<float *>(a.Z) + (vrow + t) * a.dv + v0 + 16 * m + gq;
                        if (t < len) o[0] = z[0], o[8] = z[2];
                        if (t + 1 < len) o[a.dv] = z[1], o[a.dv + 8] = z[3];
                    } else {
                        // 8 x 8 blocks transposed between the lanes: a token per row
                        const __nv_bfloat162 p0 = __floats2bfloat162_rn(z[0], z[1]);
                        const __nv_bfloat162 p1 = __floats2bfloat162_rn(z[2], z[3]);
                        const uint32_t r0 = movt(*reinterpret_cast<const uint32_t *>(&p0));
                        const uint32_t r1 = movt(*reinterpret_cast<const uint32_t *>(&p1));
                        const int t = i + gq;
                        if (t < len) {
                            uint32_t *o = reinterpret_cast<uint32_t *>(
                                static_cast<__nv_bfloat16 *>(a.Z) + (vrow + t) * a.dv + v0 + 16 * m + 2 * q4);
                            o[0] = r0;
                            o[4] = r1;
                        }
                    }
                }
            }
        }
        return;
    }

    // -------------------------------------------------------------- the chain
    float4 *part = reinterpret_cast<float4 *>(area) + lane;  // [16 columns][to][from][tile][32]
    // W^T: row gq (elements 0, 1) and gq + 8 (2, 3), columns k0 + 8 nt + 2 q4 + {0, 1}
    const int k0 = p * (DK / 4);
    float S[MT][NT][4];
    const size_t state = (size_t)DK * a.dv, mine = (size_t)(k0 + 2 * q4) * a.dv + v0 + gq;
    const float *w0 = a.W0 ? a.W0 + ((size_t)n * a.w_heads + h) * state + mine : nullptr;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[m][nt][e] = w0 ? w0[(size_t)(8 * nt + (e & 1)) * a.dv + 16 * m + (e >> 1) * 8] : 0.f;

    // W at the start of chunk c
    auto save = [&](int c) {
        float *ws = a.saveS + ((size_t)(slot0 + c) * a.H + h) * state + mine;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    ws[(size_t)(8 * nt + (e & 1)) * a.dv + 16 * m + (e >> 1) * 8] = S[m][nt][e];
    };
    if (SAVE && nchunk > 0) save(0);

    Ring ring(a.stages);
    for (int c = 0; c < nchunk; ++c, ring.next()) {
        const int turn = c & 1;
        const uint32_t uK = smem_u32(ssm + ring.s * STAGE), uH = uK + KALL;
        const float *vec = reinterpret_cast<const float *>(ssm + (ring.s + 1) * STAGE - kHalfVecBytes);
        if (named_bar_or(2, 160, false)) return;  // with the gate; it says when a wait has run out
        // W^T K^T over this warp's quarter of DK, W^T's terms left for Z
        {
            float X[MT][8][4] = {}, sS[MT][2], iS[MT][2];
            uint32_t bb[KK][4][4];
            auto load_k = [&](uint32_t(&b)[4][4], uint32_t u, int kk) {
#pragma unroll
                for (int np = 0; np < 4; ++np) load_b(b[np], u, 16 * np, k0 + 16 * kk, lane);
            };
            if (MT == 1) {  // all on their way; with 32 columns the registers are short
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) load_k(bb[kk], uK, kk);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) row_scales<NT>(S[m], sS[m], iS[m]);
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                uint32_t(&b)[4][4] = bb[MT == 1 ? kk : 0];
                uint32_t hi[MT][4];
                if (MT > 1) load_k(b, uK, kk);
                auto add = [&](float(&x)[8][4], const uint32_t(&t)[4]) {
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt)
                        mma_f16(x[nt], t, b[nt >> 1][2 * (nt & 1)], b[nt >> 1][2 * (nt & 1) + 1]);
                };
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint32_t lo[4];
                    a_terms(S[m][2 * kk], S[m][2 * kk + 1], sS[m], hi[m], lo);
                    add(X[m], hi[m]);
                    add(X[m], lo);
                    if (!SAVE) {
                        uint4 *d = reinterpret_cast<uint4 *>(turn_at(turn, m) + VB + 4096 + 512) + lane +
                                   64 * (p * KK + kk);
                        d[0] = make_uint4(hi[m][0], hi[m][1], hi[m][2], hi[m][3]);
                        d[32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                if (!BF16) {
                    load_k(b, uK + KIMG, kk);
#pragma unroll
                    for (int m = 0; m < MT; ++m) add(X[m], hi[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (!SAVE && q4 == 0) {
                    float *iSs = reinterpret_cast<float *>(turn_at(turn, m) + VB + 4096) + 64;
                    iSs[16 * p + gq] = iS[m][0], iSs[16 * p + gq + 8] = iS[m][1];
                }
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
                    part[1024 * m + 32 * (8 * (nt >> 1) + 2 * p + (nt & 1))] =
                        make_float4(iS[m][0] * X[m][nt][0], iS[m][0] * X[m][nt][1],
                                    iS[m][1] * X[m][nt][2], iS[m][1] * X[m][nt][3]);
            }
        }
        named_bar(1, 128);  // the first meeting
        // X of block p, in operand form
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            char *at = turn_at(turn, m);
            uint4 *xfr = reinterpret_cast<uint4 *>(at + VB) + lane;
            float *iXs = reinterpret_cast<float *>(at + VB + 4096);
            const float4 *in = part + 1024 * m;
            float X[2][4];
            float4 v4[2];
            load_v<BF16>(v4, at, 16 * p, lane);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float2 ck = *reinterpret_cast<const float2 *>(vec + kVk * C + 16 * p + 8 * x + 2 * q4);
                const float4 o0 = in[32 * (8 * p + x)], o1 = in[32 * (8 * p + 2 + x)],
                             o2 = in[32 * (8 * p + 4 + x)], o3 = in[32 * (8 * p + 6 + x)];
                const float4 v = v4[x];
                X[x][0] = v.x - ck.x * ((o0.x + o1.x) + (o2.x + o3.x));
                X[x][1] = v.y - ck.y * ((o0.y + o1.y) + (o2.y + o3.y));
                X[x][2] = v.z - ck.x * ((o0.z + o1.z) + (o2.z + o3.z));
                X[x][3] = v.w - ck.y * ((o0.w + o1.w) + (o2.w + o3.w));
            }
            float sX[2], iX[2];
            uint32_t hi[4], lo[4];
            row_scales<2>(X, sX, iX);
            a_terms(X[0], X[1], sX, hi, lo);
            xfr[32 * (2 * p)] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            xfr[32 * (2 * p + 1)] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (q4 == 0) iXs[16 * p + gq] = iX[0], iXs[16 * p + gq + 8] = iX[1];
            if (m == MT - 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&zready[turn]);
            }
            if (SAVE) {
                float *wx = a.saveX + (((size_t)(slot0 + c) * a.H + h) * C + 16 * p + 2 * q4) * a.dv + v0 + 16 * m + gq;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        wx[(size_t)(8 * x + (e & 1)) * a.dv + (e >> 1) * 8] = X[x][e];
            }
        }
        // H's first fragments, in the shadow of the meeting
        constexpr int HA = 2;  // blocks of tokens whose fragments are at hand
        uint32_t bh[HA][KK][4], bl[HA][KK][4];
        auto load_h = [&](int y, int jj) {
#pragma unroll
            for (int np = 0; np < KK; ++np) {
                load_bt(bh[y][np], uH, 16 * jj, k0 + 16 * np, lane);
                load_bt(bl[y][np], uH + KIMG, 16 * jj, k0 + 16 * np, lane);
            }
        };
#pragma unroll
        for (int jj = 0; jj < HA; ++jj) load_h(jj, jj);
        const float gam = vec[kVs * C];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[m][nt][e] *= gam;
        named_bar(1, 128);  // the second meeting

        // W'^T = exp(G_C) W^T + X^T H
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const float iH = vec[kVs * C + 1 + jj];
            uint32_t(&h2)[KK][4] = bh[jj % HA], (&l2)[KK][4] = bl[jj % HA];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const char *at = turn_at(turn, m);
                const uint4 *xfr = reinterpret_cast<const uint4 *>(at + VB) + lane;
                const float *iXs = reinterpret_cast<const float *>(at + VB + 4096);
                const uint4 fh = xfr[32 * (2 * jj)], fl = xfr[32 * (2 * jj + 1)];
                const uint32_t hi[4] = {fh.x, fh.y, fh.z, fh.w}, lo[4] = {fl.x, fl.y, fl.z, fl.w};
                const float u0 = iXs[16 * jj + gq] * iH, u1 = iXs[16 * jj + gq + 8] * iH;
                float U[NT][4] = {};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16(U[nt], hi, h2[nt >> 1][2 * (nt & 1)], h2[nt >> 1][2 * (nt & 1) + 1]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16(U[nt], lo, h2[nt >> 1][2 * (nt & 1)], h2[nt >> 1][2 * (nt & 1) + 1]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16(U[nt], hi, l2[nt >> 1][2 * (nt & 1)], l2[nt >> 1][2 * (nt & 1) + 1]);
                if (m == MT - 1 && jj + HA < 4) load_h(jj % HA, jj + HA);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    S[m][nt][0] = fmaf(u0, U[nt][0], S[m][nt][0]);
                    S[m][nt][1] = fmaf(u0, U[nt][1], S[m][nt][1]);
                    S[m][nt][2] = fmaf(u1, U[nt][2], S[m][nt][2]);
                    S[m][nt][3] = fmaf(u1, U[nt][3], S[m][nt][3]);
                }
            }
        }
        if (SAVE && c + 1 < nchunk) save(c + 1);
    }

    if (a.W_out) {
        float *w = a.W_out + ((size_t)n * a.H + h) * state + mine;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[(size_t)(8 * nt + (e & 1)) * a.dv + 16 * m + (e >> 1) * 8] = S[m][nt][e];
    }
}

template <int DK, bool BF16>
cudaError_t prep_inst(const PrepArgs &r, int blocks, cudaStream_t s) {
    constexpr int smem = prep_smem<DK, BF16>();
    static SmemOnce once;
    cudaError_t e = once.allow(delta_prep_kernel<DK, BF16>, smem);
    if (e != cudaSuccess) return e;
    delta_prep_kernel<DK, BF16><<<blocks, kPrepThreads, smem, s>>>(r);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}

template <int DK, bool BF16, int MODE, int MT>
constexpr bool scan_fits() {
    return 2 * chain_stage_bytes<DK, BF16>() + z_stage_bytes<DK, BF16, MODE>() +
               scan_area_bytes<DK, BF16, MODE, MT>() <= kScanSmem;
}

template <int DK, bool BF16, int MODE, int MT>
cudaError_t scan_run(ScanArgs r, int N, cudaStream_t s) {
    constexpr int stage = chain_stage_bytes<DK, BF16>(), zstage = z_stage_bytes<DK, BF16, MODE>();
    constexpr int area = scan_area_bytes<DK, BF16, MODE, MT>();
    // two stages of the chain's ring at least (the gate frees one when the chain has
    // met it for the next), two of Z's or a third of the chain's where there is room
    static_assert(scan_fits<DK, BF16, MODE, MT>(), "shared memory");
    r.stages = 2;
    r.zstages = 2 * (stage + zstage) + area <= kScanSmem ? 2 : 1;
    if (3 * stage + 2 * zstage + area <= kScanSmem) r.stages = 3;
    const int smem = r.stages * stage + r.zstages * zstage + area;
    static SmemOnce once;
    cudaError_t e = once.allow(delta_scan_kernel<DK, BF16, MODE, MT>, kScanSmem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((long long)N * r.H * (r.dv / (16 * MT)));
    delta_scan_kernel<DK, BF16, MODE, MT><<<grid, 384, smem, s>>>(r);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}

template <int DK, bool BF16, int MODE>
cudaError_t scan_inst(const ScanArgs &r, int N, cudaStream_t s) {
    // 16 columns a block, or 32 where that saves rounds over the SMs: the fragments of K
    // and H are loaded once for both, but the chain's and Z's warps have twice the work. A
    // chunk of 32 takes 1.6 - 1.8 times one of 16 at d_k = 64, so 32 pay from a ratio of
    // rounds of 9 : 5 on, and 1.95 times at 128, where they pay if they halve the rounds.
    // T 2048, bf16 in and out, us with 16 / 32 columns:
    //   d 64:   64 heads (2 rounds / 1) 87 / 71   96 (3 / 2) 127 / 133   148 (4 / 2) 169 / 135
    //           400 (11 / 6) 445 / 387
    //   d 128:  24 heads (2 rounds / 1) 102 / 97  48 (3 / 2) 149 / 194   148 (8 / 4) 391 / 385
    //           200 (11 / 6) 527 / 567
    // The saving scan, whose stores of W bound it, takes 16 (16 heads of 128, T 8192: 159 / 389).
    if constexpr (MODE != kSave && scan_fits<DK, BF16, MODE, 2>()) {
        const long long blocks = (long long)N * r.H * (r.dv / 16);
        const long long rounds16 = (blocks + 147) / 148, rounds32 = (blocks / 2 + 147) / 148;
        if (DK == 128 ? 2 * rounds32 <= rounds16 : 9 * rounds32 < 5 * rounds16)
            return scan_run<DK, BF16, MODE, 2>(r, N, s);
    }
    return scan_run<DK, BF16, MODE, 1>(r, N, s);
}

template <int DK, bool BF16>
cudaError_t scan_mode(const ScanArgs &r, int N, int mode, cudaStream_t s) {
    return mode == kZ16   ? scan_inst<DK, BF16, kZ16>(r, N, s)
           : mode == kZ32 ? scan_inst<DK, BF16, kZ32>(r, N, s)
                          : scan_inst<DK, BF16, kSave>(r, N, s);
}

}  // namespace

Images images_at(const Plan &p, void *workspace, bool bwd) {
    char *w = static_cast<char *>(workspace);
    return Images{w + p.oK, w + p.oQ, w + p.oM, w + p.oH, bwd ? w + p.oT : nullptr, w + p.oV,
                  p.kimg, p.himg};
}

cudaError_t launch_prep(const DeltaArgs &a, const Plan &p, const Images &im, cudaStream_t s) {
    const PrepArgs r{a.Q, a.K, a.eta, a.g, a.seq_start, a.B, a.Hk, a.H, a.T, a.N, a.q_scale, im};
    const int blocks = p.slots * a.Hk;
    if (a.dk == 64) return a.bf16 ? prep_inst<64, true>(r, blocks, s) : prep_inst<64, false>(r, blocks, s);
    return a.bf16 ? prep_inst<128, true>(r, blocks, s) : prep_inst<128, false>(r, blocks, s);
}

cudaError_t launch_scan(const DeltaArgs &a, const Images &im, int mode, float *saveS, float *saveX,
                        cudaStream_t s) {
    const ScanArgs r{a.V, a.W0, a.Z, a.W_out, a.seq_start, a.B, a.Hk, a.H, a.T, a.dv,
                     a.w0_per_seq ? a.H : 0, 0, 0, im, saveS, saveX, device_status_word()};
    if (a.dk == 64)
        return a.bf16 ? scan_mode<64, true>(r, a.N, mode, s) : scan_mode<64, false>(r, a.N, mode, s);
    return a.bf16 ? scan_mode<128, true>(r, a.N, mode, s) : scan_mode<128, false>(r, a.N, mode, s);
}

}  // namespace delta

using namespace delta;

// Short calls go token by token: one launch instead of two, no chunk to prepare and no
// workspace. Both sides, us of kernel time (token by token / chunked):
//   B 1, H 4, d 64, bf16:     T 8: 12 / 24    T 24: 19 / 23     T 32: 23 / 23
//   B 4, H 8, d 128, fp32:    T 8: 11 / 32    T 24: 19 / 32     T 48: 29 / 32
//   B 128, H 8, d 128, bf16:  T 8: 69 / 272   T 24: 180 / 276   T 48: 342 / 279
static bool token_by_token(int T) { return T <= 24; }

size_t delta_workspace_bytes(int B, int Hk, int H, int T, int dk, int dv, int N, bool packed,
                             bool bf16) {
    (void)dv;
    if (token_by_token(T)) return 0;
    return make_plan(B, Hk, H, T, dk, N, packed, bf16, false).end;
}

cudaError_t launch_delta_fwd(const DeltaArgs &a, cudaStream_t s) {
    if (token_by_token(a.T)) return launch_delta_recurrent(a, s);
    const Plan p = make_plan(a.B, a.Hk, a.H, a.T, a.dk, a.N, a.seq_start != nullptr, a.bf16, false);
    const Images im = images_at(p, a.workspace, false);
    const cudaError_t e = launch_prep(a, p, im, s);
    if (e != cudaSuccess) return e;
    return launch_scan(a, im, a.z_bf16 ? kZ16 : kZ32, nullptr, nullptr, s);
}

}  // namespace ttt
