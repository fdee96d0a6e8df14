// ttt_delta_bwd.cu -- backward of the gated delta rule, chunked.
//
// With the chunk's X = V - D K W, rho = T X, Z = c D Q W + M X,
// W' = exp(G_C) W + H^T X (ttt_delta_chunk.cu) and Om = dL/dW':
//   dX = M^T dZ + H Om = dV
//   dL/dW = exp(G_C) Om + c Q^T D dZ - K^T D dX          (the reverse scan)
// and per chunk, all chunks at once,
//   phi_ij = c Gam_ij (dZ_i.rho_j) (j <= i),  eps_ij = -Gam_ij (dX_i.rho_j) (j < i)
//   dQ = c D dZ W^T + (phi eta) K
//   dK = -D dX W^T + diag(exp(G_C - G) eta) rho Om^T + (phi eta)^T Q + (E + E^T) K,
//        E_ij = eps_ij eta_j
//   deta_j = sum_i phi_ij (q_i.k_j) + sum_i eps_ij (k_i.k_j) + exp(G_C - G_j) k_j.(Om rho_j)
//   dg_t = sum_{i >= t} (q_i.(c D_i W dZ_i) - k_i.(D_i W dX_i))
//          + sum_{j < t <= i} eta_j (phi_ij q_i.k_j + eps_ij k_i.k_j)
//          + sum_{j < t} eta_j exp(G_C - G_j) k_j.(Om rho_j) + exp(G_C) <W, Om>:
// what g_t scales, no sums of dL/dG_i from t on (those hold every pair j, i >= t twice with
// opposite signs). The pairs across t come one token after the other: t + 1 gains those
// of column t below the diagonal and loses those of row t left of it, in double, so that
// a pair that has left leaves nothing: in fp32 the decays of tokens behind a forgetting were off
// by 2^-24 of the largest pair in front of it.
// The forward scan runs again first and keeps W at the start of each chunk and
// X; the reverse scan keeps Om at its end. Everything is fp32, its products two
// fp16 terms an operand (ttt_delta_mma.cuh). No atomics: every sum has one order.
#include "../../include/ttt.h"
#include "ttt_delta_mma.cuh"

namespace ttt {
namespace delta {
namespace {

// ---------------------------------------------------------------- reverse scan

struct RevArgs {
    const float *dZ, *dW_out;
    float *dV, *dW0;               // dW0 [N][H][DK][dv] or NULL
    const int *seq_start;
    int B, Hk, H, T, dv, stages, zstages;
    Images im;
    float *saveO;                  // [slot][H][DK][dv]
    int *status;
};

// Bytes of a stage of the chain's ring (K, H, vectors) and of the helpers' (Q, M, vectors).
template <int DK, bool BF16>
constexpr int rev_stage_bytes() { return ((BF16 ? 1 : 2) + 2) * C * DK * 2 + kHalfVecBytes; }
template <int DK, bool BF16>
constexpr int rev_zstage_bytes() { return (BF16 ? 1 : 2) * C * DK * 2 + 2 * kImg + kHalfVecBytes; }
// Shares of dX [to 4][from 4][2 tiles], the terms of dX [4 blocks][hi, lo] and of dZ
// [4 blocks][for M, for Q][hi, lo] with 1 / their scales; twice, for the chunks in turn,
// what the helpers leave: (M^T dZ)^T [4 blocks][2 tiles], (c D Q)^T dZ transposed [DK / 8 tiles].
template <int DK>
constexpr int rev_turn_bytes() { return 4096 + DK / 8 * 512; }
// Two turns, so that the helpers may run ahead; one where shared memory is short.
template <int DK, bool BF16>
constexpr int rev_turns() { return DK == 128 && !BF16 ? 1 : 2; }
template <int DK, bool BF16>
constexpr int rev_area_bytes() {
    return 16 * 1024 + 4096 + 8192 + 768 + rev_turns<DK, BF16>() * rev_turn_bytes<DK>();
}

// The mirror of the forward scan: four warps own 16 columns of Om, as the rows of
// Om^T in registers, a quarter of DK each. Before the first meeting each hands out its
// quarter's share of Om^T H^T; warp p puts dX of block p together, and after the second
// meeting each updates its quarter of Om. What dZ adds does not depend on Om: four
// helper warps form M^T dZ (a block of tokens each) and (c D Q)^T dZ (a quarter of DK
// each), up to two chunks ahead. Two more warps fill the rings of stages, and one, the
// gate, does the chain's waiting. Bound by the chain's latency as the forward's scan is:
// 2 x 8192 x 8 heads of 128 in 250 us, 1.95 us a chunk (337 with dZ's parts on the
// chain); shared memory busy 57 %, the tensor pipe 28 %, DRAM 17 %.
template <int DK, bool BF16>
__global__ void __launch_bounds__(352, 1) delta_rev_kernel(RevArgs a) {
    extern __shared__ __align__(128) char ssm[];
    __shared__ uint64_t full[4], empty[4], zfull[4], zempty[4], zready[2], zfree[2];
    __shared__ int abort_flag;
    constexpr int STAGE = rev_stage_bytes<DK, BF16>(), ZSTAGE = rev_zstage_bytes<DK, BF16>();
    constexpr int KIMG = C * DK * 2, KALL = KIMG * (BF16 ? 1 : 2);
    constexpr int NT = DK / 32, KK = DK / 64, TURNS = rev_turns<DK, BF16>();
    const int groups = a.dv / 16;
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
            mbar_init(&zready[t], 4);
            mbar_init(&zfree[t], 1);
        }
        fence_mbar_init();
    }
    __syncthreads();

    const int gq = lane >> 2, q4 = lane & 3;
    const int v0 = grp * 16;
    const size_t vrow = ((size_t)b * a.H + h) * a.T + t0;
    char *zst = ssm + a.stages * STAGE, *area = zst + a.zstages * ZSTAGE;
    auto wait = [&](uint64_t *bar, int parity) {
        return mbar_wait_warp(bar, parity, abort, a.status, kScanStatus);
    };
    uint4 *const zfr = reinterpret_cast<uint4 *>(area + 20 * 1024) + lane;  // [block][M hi, lo, Q hi, lo][32]
    float *const iXs = reinterpret_cast<float *>(area + 28 * 1024), *const iZm = iXs + 64, *const iZq = iZm + 64;
    auto turn_at = [&](int turn) { return area + 28 * 1024 + 768 + turn * rev_turn_bytes<DK>(); };

    // step i works on chunk nchunk - 1 - i
    if (warp == 10) {  // ------------------------------------------------ the gate
        // Waits for all that a step needs and then meets the chain, which so waits on
        // nothing but barriers; at the next meeting the chain is done with what it had.
        Ring ring(a.stages);
        int last = 0;
        for (int i = 0; i < nchunk; ++i, ring.next()) {
            const bool ok = wait(&full[ring.s], ring.ph) && wait(&zready[i % TURNS], (i / TURNS) & 1);
            if (named_bar_or(3, 160, !ok)) return;
            if (i > 0 && lane == 0) {
                mbar_arrive(&empty[last]);
                if (TURNS == 2) mbar_arrive(&zfree[(i - 1) % TURNS]);
            }
            last = ring.s;
        }
        return;
    }
    if (warp >= 8) {  // ------------------------------------------------ the rings
        auto chain_copy = [&](int i, int s, uint64_t *bar) {
            char *d = ssm + s * STAGE;
            const size_t c = slot0 + nchunk - 1 - i, ks = c * a.Hk + hk, hs = c * a.H + h;
            mbar_arrive_expect_tx(bar, STAGE);
            bulk_load(d, a.im.H + hs * 2 * KIMG, 2 * KIMG, bar);
            bulk_load(d + 2 * KIMG, a.im.K + ks * KALL, KALL, bar);
            bulk_load(d + STAGE - kHalfVecBytes, a.im.vec + hs * kVecBytes, kHalfVecBytes, bar);
        };
        auto z_copy = [&](int i, int s, uint64_t *bar) {
            char *d = zst + s * ZSTAGE;
            const size_t c = slot0 + nchunk - 1 - i, ks = c * a.Hk + hk, hs = c * a.H + h;
            mbar_arrive_expect_tx(bar, ZSTAGE);
            bulk_load(d, a.im.Q + ks * KALL, KALL, bar);
            bulk_load(d + KALL, a.im.M + hs * 2 * kImg, 2 * kImg, bar);
            bulk_load(d + ZSTAGE - kHalfVecBytes, a.im.vec + hs * kVecBytes + kHalfVecBytes,
                      kHalfVecBytes, bar);
        };
        if (lane == 0) {
            if (warp == 8) {
                Filler<decltype(chain_copy)> f(full, empty, a.stages, nchunk, abort, a.status, chain_copy);
                f.run();
            } else {
                Filler<decltype(z_copy)> f(zfull, zempty, a.zstages, nchunk, abort, a.status, z_copy);
                f.run();
            }
        }
        return;
    }
    if (warp >= 4) {  // ------------------------------------------------ dZ's parts
        // dZ of this lane's places in block p
        float z[2][4];
        const size_t zlane = (vrow + 16 * p + 2 * q4) * a.dv + v0 + gq;
        auto fetch_z = [&](int c) {
            const size_t at = zlane + (size_t)c * C * a.dv;
            const int t = c * C + 16 * p + 2 * q4;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z[x][e] = t + 8 * x + (e & 1) < len
                                  ? a.dZ[at + (8 * x + (e & 1)) * a.dv + (e >> 1) * 8] : 0.f;
        };
        if (nchunk > 0) fetch_z(nchunk - 1);
        Ring ring(a.zstages);
        for (int i = 0; i < nchunk; ++i, ring.next()) {
            const int turn = i % TURNS, c = nchunk - 1 - i;
            const uint32_t uQ = smem_u32(zst + ring.s * ZSTAGE), uM = uQ + KALL;
            // the enum's order, counted from kVq on
            const float *vec = reinterpret_cast<const float *>(zst + (ring.s + 1) * ZSTAGE - kHalfVecBytes) - kVq * C;
            float4 *zm = reinterpret_cast<float4 *>(turn_at(turn)) + lane;  // [block][tile][32]
            float4 *uq = zm + 256;                                         // [DK / 8][32]
            bool ok = wait(&zfull[ring.s], ring.ph);
            if (i >= TURNS) ok = ok && wait(&zfree[turn], ((i / TURNS) & 1) ^ 1);
            if (ok) {
                // dZ of block p as an operand for M (M's row scales in it) and for c D Q
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float A[2][4], sA[2], iA[2];
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float2 f = *reinterpret_cast<const float2 *>(
                            vec + (y ? kVq : kVm) * C + 16 * p + 8 * x + 2 * q4);
                        A[x][0] = z[x][0] * f.x, A[x][1] = z[x][1] * f.y;
                        A[x][2] = z[x][2] * f.x, A[x][3] = z[x][3] * f.y;
                    }
                    row_scales<2>(A, sA, iA);
                    a_terms(A[0], A[1], sA, hi, lo);
                    zfr[32 * (4 * p + 2 * y)] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    zfr[32 * (4 * p + 2 * y + 1)] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    float *q = y ? iZq : iZm;
                    if (q4 == 0) q[16 * p + gq] = iA[0], q[16 * p + gq + 8] = iA[1];
                }
                if (i + 1 < nchunk) fetch_z(c - 1);
            }
            if (named_bar_or(2, 128, !ok)) return;
            float D[2][4] = {}, Q[NT][4] = {};
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                if (jj >= p) {  // (M^T dZ)^T of block p: M_ij is zero for i < j
                    const uint4 fh = zfr[32 * (4 * jj)], fl = zfr[32 * (4 * jj + 1)];
                    const uint32_t hi[4] = {fh.x, fh.y, fh.z, fh.w}, lo[4] = {fl.x, fl.y, fl.z, fl.w};
                    const float i0 = iZm[16 * jj + gq], i1 = iZm[16 * jj + gq + 8];
                    uint32_t bh[4], bl[4];
                    float d[2][4] = {}, e2[2][4] = {};
                    load_bt(bh, uM, 16 * jj, 16 * p, lane);
                    load_bt(bl, uM + kImg, 16 * jj, 16 * p, lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(d[x], hi, bh[2 * x], bh[2 * x + 1]);
                        mma_f16(e2[x], lo, bh[2 * x], bh[2 * x + 1]);
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) mma_f16(e2[x], hi, bl[2 * x], bl[2 * x + 1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            D[x][e] = fmaf(e < 2 ? i0 : i1, d[x][e] + e2[x][e], D[x][e]);
                }
                // dZ^T (c D Q) of quarter p of DK
                const uint4 fh = zfr[32 * (4 * jj + 2)], fl = zfr[32 * (4 * jj + 3)];
                const uint32_t hi[4] = {fh.x, fh.y, fh.z, fh.w}, lo[4] = {fl.x, fl.y, fl.z, fl.w};
                const float i0 = iZq[16 * jj + gq], i1 = iZq[16 * jj + gq + 8];
                uint32_t bb[KK][4];
                float U[NT][4] = {};
#pragma unroll
                for (int np = 0; np < KK; ++np) load_bt(bb[np], uQ, 16 * jj, p * (DK / 4) + 16 * np, lane);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16(U[nt], hi, bb[nt >> 1][2 * (nt & 1)], bb[nt >> 1][2 * (nt & 1) + 1]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16(U[nt], lo, bb[nt >> 1][2 * (nt & 1)], bb[nt >> 1][2 * (nt & 1) + 1]);
                if (!BF16) {
#pragma unroll
                    for (int np = 0; np < KK; ++np)
                        load_bt(bb[np], uQ + KIMG, 16 * jj, p * (DK / 4) + 16 * np, lane);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(U[nt], hi, bb[nt >> 1][2 * (nt & 1)], bb[nt >> 1][2 * (nt & 1) + 1]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        Q[nt][e] = fmaf(e < 2 ? i0 : i1, U[nt][e], Q[nt][e]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) zm[32 * (2 * p + x)] = make_float4(D[x][0], D[x][1], D[x][2], D[x][3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                uq[32 * (p * NT + nt)] = make_float4(Q[nt][0], Q[nt][1], Q[nt][2], Q[nt][3]);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&zready[turn]);
                mbar_arrive(&zempty[ring.s]);
            }
            named_bar(2, 128);  // dZ's terms are read
        }
        return;
    }

    // -------------------------------------------------------------- the chain
    float4 *part = reinterpret_cast<float4 *>(area) + lane;           // [to][from][tile][32]
    uint4 *xfr = reinterpret_cast<uint4 *>(area + 16 * 1024) + lane;  // [block][hi, lo][32]
    const int k0 = p * (DK / 4);
    float S[NT][4];
    const size_t state = (size_t)DK * a.dv, mine = (size_t)(k0 + 2 * q4) * a.dv + v0 + gq;
    const float *w0 = a.dW_out ? a.dW_out + ((size_t)n * a.H + h) * state + mine : nullptr;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[nt][e] = w0 ? w0[(size_t)(8 * nt + (e & 1)) * a.dv + (e >> 1) * 8] : 0.f;

    // Om at the end of chunk c
    auto save = [&](int c) {
        float *ws = a.saveO + ((size_t)(slot0 + c) * a.H + h) * state + mine;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                ws[(size_t)(8 * nt + (e & 1)) * a.dv + (e >> 1) * 8] = S[nt][e];
    };
    if (nchunk > 0) save(nchunk - 1);

    Ring ring(a.stages);
    for (int i = 0; i < nchunk; ++i, ring.next()) {
        const int turn = i % TURNS, c = nchunk - 1 - i;
        const uint32_t uH = smem_u32(ssm + ring.s * STAGE), uK = uH + 2 * KIMG;
        const float *vec = reinterpret_cast<const float *>(ssm + (ring.s + 1) * STAGE - kHalfVecBytes);
        const float4 *zm = reinterpret_cast<const float4 *>(turn_at(turn)) + lane, *uq = zm + 256;
        if (named_bar_or(3, 160, false)) return;  // with the gate; it says when a wait has run out
        // Om^T H^T over this warp's quarter of DK
        {
            float X[8][4] = {}, sS[2], iS[2];
            uint32_t bh[KK][4][4], bl[KK][4][4];
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    load_b(bh[kk][np], uH, 16 * np, k0 + 16 * kk, lane);
                    load_b(bl[kk][np], uH + KIMG, 16 * np, k0 + 16 * kk, lane);
                }
            row_scales<NT>(S, sS, iS);
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                uint32_t hi[4], lo[4];
                a_terms(S[2 * kk], S[2 * kk + 1], sS, hi, lo);
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
                    mma_f16(X[nt], hi, bh[kk][nt >> 1][2 * (nt & 1)], bh[kk][nt >> 1][2 * (nt & 1) + 1]);
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
                    mma_f16(X[nt], lo, bh[kk][nt >> 1][2 * (nt & 1)], bh[kk][nt >> 1][2 * (nt & 1) + 1]);
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
                    mma_f16(X[nt], hi, bl[kk][nt >> 1][2 * (nt & 1)], bl[kk][nt >> 1][2 * (nt & 1) + 1]);
            }
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
                part[32 * (8 * (nt >> 1) + 2 * p + (nt & 1))] = make_float4(
                    iS[0] * X[nt][0], iS[0] * X[nt][1], iS[1] * X[nt][2], iS[1] * X[nt][3]);
        }
        named_bar(1, 128);  // the first meeting
        // dX of block p
        float X[2][4];
        {
            const float iH = vec[kVs * C + 1 + p];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float4 o0 = part[32 * (8 * p + x)], o1 = part[32 * (8 * p + 2 + x)],
                             o2 = part[32 * (8 * p + 4 + x)], o3 = part[32 * (8 * p + 6 + x)];
                const float4 m = zm[32 * (2 * p + x)];
                X[x][0] = fmaf(iH, (o0.x + o1.x) + (o2.x + o3.x), m.x);
                X[x][1] = fmaf(iH, (o0.y + o1.y) + (o2.y + o3.y), m.y);
                X[x][2] = fmaf(iH, (o0.z + o1.z) + (o2.z + o3.z), m.z);
                X[x][3] = fmaf(iH, (o0.w + o1.w) + (o2.w + o3.w), m.w);
            }
            float A[2][4], sX[2], iX[2];
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float2 ck = *reinterpret_cast<const float2 *>(vec + kVk * C + 16 * p + 8 * x + 2 * q4);
                A[x][0] = -ck.x * X[x][0], A[x][1] = -ck.y * X[x][1];
                A[x][2] = -ck.x * X[x][2], A[x][3] = -ck.y * X[x][3];
            }
            row_scales<2>(A, sX, iX);
            a_terms(A[0], A[1], sX, hi, lo);
            xfr[32 * (2 * p)] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            xfr[32 * (2 * p + 1)] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (q4 == 0) iXs[16 * p + gq] = iX[0], iXs[16 * p + gq + 8] = iX[1];
        }
        // in the shadow of the meeting: what goes out, and all that does not wait for X
        uint32_t bk[4][KK][4];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
            for (int np = 0; np < KK; ++np) load_bt(bk[jj][np], uK, 16 * jj, k0 + 16 * np, lane);
        const float gam = vec[kVs * C];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float4 u = uq[32 * (p * NT + nt)];
            S[nt][0] = fmaf(gam, S[nt][0], u.x), S[nt][1] = fmaf(gam, S[nt][1], u.y);
            S[nt][2] = fmaf(gam, S[nt][2], u.z), S[nt][3] = fmaf(gam, S[nt][3], u.w);
        }
        named_bar(1, 128);  // the second meeting
        // with one turn the gate cannot give it back: it waits for the next step's
        if (TURNS == 1 && tid == 0) mbar_arrive(&zfree[0]);

        // Om^T <- exp(G_C) Om^T + dZ^T (c D Q) - dX^T (D K)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const uint4 fh = xfr[32 * (2 * jj)], fl = xfr[32 * (2 * jj + 1)];
            const uint32_t hi[4] = {fh.x, fh.y, fh.z, fh.w}, lo[4] = {fl.x, fl.y, fl.z, fl.w};
            const float i0 = iXs[16 * jj + gq], i1 = iXs[16 * jj + gq + 8];
            float U[NT][4] = {};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_f16(U[nt], hi, bk[jj][nt >> 1][2 * (nt & 1)], bk[jj][nt >> 1][2 * (nt & 1) + 1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_f16(U[nt], lo, bk[jj][nt >> 1][2 * (nt & 1)], bk[jj][nt >> 1][2 * (nt & 1) + 1]);
            if (!BF16) {
                uint32_t bb[KK][4];
#pragma unroll
                for (int np = 0; np < KK; ++np) load_bt(bb[np], uK + KIMG, 16 * jj, k0 + 16 * np, lane);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16(U[nt], hi, bb[nt >> 1][2 * (nt & 1)], bb[nt >> 1][2 * (nt & 1) + 1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                S[nt][0] = fmaf(i0, U[nt][0], S[nt][0]);
                S[nt][1] = fmaf(i0, U[nt][1], S[nt][1]);
                S[nt][2] = fmaf(i1, U[nt][2], S[nt][2]);
                S[nt][3] = fmaf(i1, U[nt][3], S[nt][3]);
            }
        }
        if (c > 0) save(c - 1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int t = c * C + 16 * p + 8 * x + 2 * q4;
            float *d = a.dV + (vrow + t) * a.dv + v0 + gq;
            if (t < len) d[0] = X[x][0], d[8] = X[x][2];
            if (t + 1 < len) d[a.dv] = X[x][1], d[a.dv + 8] = X[x][3];
        }
    }

    if (a.dW0) {
        float *w = a.dW0 + ((size_t)n * a.H + h) * state + mine;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[(size_t)(8 * nt + (e & 1)) * a.dv + (e >> 1) * 8] = S[nt][e];
    }
}

// ---------------------------------------------------------------- per-chunk gradients

struct GradArgs {
    const float *dZ, *dV;          // [B][H][T][dv]; dV = dX
    const float *eta;
    const float *saveS, *saveX, *saveO;
    float *dQ, *dK, *deta, *dg;    // dg NULL without a gate
    const int *seq_start;
    int B, Hk, H, T, N;
    float q_scale;
    Images im;
};

constexpr int kGradThreads = 512;

// Shared memory: K and Q images; a region that first holds X and T, then W, dZ
// and dX, then W and Om, then the three 64 x 64 images; rho; vectors and partial
// sums.
template <int DK, int DV, bool BF16>
struct GradSmem {
    static constexpr int IMG = C * DK * 2 * (BF16 ? 1 : 2);
    static constexpr int W = DK * DV * 2 * 2;          // W (or Om), two terms
    static constexpr int R = C * DV * 2 * 2;           // rho (or X, dZ, dX), two terms
    static constexpr int big1 = W + (W > 2 * R ? W : 2 * R), big2 = R + 2 * kImg, big3 = 6 * kImg;
    static constexpr int big = big1 > big2 ? (big1 > big3 ? big1 : big3) : (big2 > big3 ? big2 : big3);
    static constexpr int oBig = 2 * IMG, oR = oBig + big, oF = oR + R;
    // floats: Gh, Gl, eta, iR, iT (5 x 64), iS (128), iZ or iO (128), sums over warps (128:
    // X's maxima 32, <W, Om> 16, 1 / scales of X 4)
    static constexpr int bytes = oF + 4 * (5 * C + 128 + 128 + 128);
};

// Row (c0 .. c0 + 7) units of an fp32 matrix row, scaled to two fp16 terms.
__device__ __forceinline__ void put8(const float (&x)[8], float s, char *hi, char *lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split_f16(x[2 * j] * s, x[2 * j + 1] * s, h[j], l[j]);
    *reinterpret_cast<uint4 *>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void get8(float (&x)[8], const float *p) {
    const float4 u = reinterpret_cast<const float4 *>(p)[0], v = reinterpret_cast<const float4 *>(p)[1];
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
}
__device__ __forceinline__ float max8(const float (&x)[8]) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
    return m;
}
__device__ __forceinline__ float2 h2f(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// One block per chunk and key head, its value heads one after the other; dQ and
// dK of the chunk stay in registers and are added up over them. Warp (mt, hf)
// holds the rows of tokens 16 mt .. 16 mt + 15 and a quarter of the columns.
// Reads 272 KB and writes 64 KB a chunk at 128 x 128 (bf16), more than a block's
// shared memory, so one block an SM, whose loads and products take turns. 2048 chunks of
// 128 x 128 take 448 us (32 us a block; 107 us at the copy rate): issue slots used to
// 34 %, shared memory 57 %, tensor pipe 27 %, DRAM 18 %; the stalls are waits for loads,
// shared memory and barriers. One scale for X of a chunk and one an image of phi and E
// took 435: tokens behind a forgetting lost their bits to those in front of it. Eight warps of 255 registers instead of sixteen of 128, with
// dZ and dX as fragments from global memory, took 17 % longer, W asked for before rho is
// formed 3 %. The low terms' products in the same sums as the high ones' would take 8 %
// less, and double the gradients' errors (8e-7 of a gradient's norm instead of 4.5e-7): the
// tensor cores cut off what is below a sum's last bit, once a product.
template <int DK, int DV, bool BF16>
__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(GradArgs a) {
    extern __shared__ __align__(128) char gsm[];
    using SM = GradSmem<DK, DV, BF16>;
    constexpr int IMG = SM::IMG, KIMG = C * DK * 2;
    constexpr int NK = DK / 32;  // 8-column tiles of a quarter of DK
    constexpr int NV = DV / 32;
    constexpr int KV = DV / 16;  // 16-deep steps over DV
    char *sK = gsm, *sQ = sK + IMG, *big = gsm + SM::oBig, *sR = gsm + SM::oR;
    float *Gh = reinterpret_cast<float *>(gsm + SM::oF), *Gl = Gh + C, *eta = Gl + C, *iR = eta + C,
          *iTs = iR + C, *iS = iTs + C, *iZ = iS + 128, *iO = iZ, *rmax = iS, *red = iZ + 128;
    // partial sums over the warps, in the place of rho once it is read
    double *rowp = reinterpret_cast<double *>(sR), *colp = rowp + 4 * C, *upto = colp + 4 * C;
    float *dotp = reinterpret_cast<float *>(upto + C), *decp = dotp + 4 * C, *diag = decp + 4 * C, *from = diag + C;
    // largest sizes of the rows and columns of phi eta and E, and the three images' row scales
    float *p_row = from + C, *p_col = p_row + 4 * C, *e_row = p_col + 4 * C, *e_col = e_row + 4 * C, *isc = e_col + 4 * C;
    static_assert((9 * 8 + 29 * 4) * C <= SM::R, "partial sums");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, q4 = lane & 3;
    const int mt = warp & 3, hf = warp >> 2;
    const int slot = blockIdx.x / a.Hk, hk = blockIdx.x % a.Hk;
    int n, t0, len;
    if (!ChunkSearch{a.seq_start, a.T, a.N}.find(slot, n, t0, len)) return;
    const int b = a.seq_start ? 0 : n;
    const size_t kslot = (size_t)slot * a.Hk + hk;
    const uint32_t uK = smem_u32(sK), uQ = smem_u32(sQ);
    for (int u = tid; u < IMG / 16; u += kGradThreads) {
        cp_async16(uK + 16 * u, a.im.K + kslot * IMG + 16 * (size_t)u, true);
        cp_async16(uQ + 16 * u, a.im.Q + kslot * IMG + 16 * (size_t)u, true);
    }
    const uint32_t uB = smem_u32(big), uR = smem_u32(sR);
    float dQ[NK][4] = {}, dK[NK][4] = {};
    const int rep = a.H / a.Hk;
    const int row[2] = {16 * mt + gq, 16 * mt + gq + 8};
    const int n0 = hf * (DK / 4);  // this warp's columns of DK
    // this lane's places in an image for fragments of A (rows of block mt), of B with rows as
    // n (from row 0) and as k (columns from 0): steps of 16 rows are 2048 bytes, of 16
    // columns step16()
    const uint32_t oA = ldsm_addr(0, 16 * mt, 0, lane);
    const int rB = ((lane >> 4) << 3) + (lane & 7), cB = ((lane >> 3) & 1) * 8;
    const int rT = (lane & 7) + ((lane >> 3) & 1) * 8, cT = (lane >> 4) * 8;
    const uint32_t oB = img_off(rB, cB), oX = img_off(rT, hf * (DV / 4) + cT), oK = img_off(rT, n0 + cT);

    for (int r = 0; r < rep; ++r) {
        const int h = hk * rep + r;
        const size_t hrow = ((size_t)b * a.H + h) * a.T + t0;
        const size_t hslot = (size_t)slot * a.H + h;
        const float *vec = reinterpret_cast<const float *>(a.im.vec + hslot * kVecBytes);
        // what the head needs later is fetched into L2 meanwhile
        if (lane == 0 && warp < 4) {
            const float *src = warp == 0   ? a.saveS + hslot * DK * DV
                               : warp == 1 ? a.saveO + hslot * DK * DV
                               : warp == 2 ? a.dZ + hrow * DV
                                           : a.dV + hrow * DV;
            bulk_prefetch_l2(src, (warp < 2 ? DK : len) * DV * 4);
        }
        __syncthreads();  // the head before is done with shared memory
        if (tid < C) {
            Gh[tid] = vec[kVgh * C + tid];
            Gl[tid] = vec[kVgl * C + tid];
            iTs[tid] = vec[kVit * C + tid];
            eta[tid] = tid < len ? a.eta[hrow + tid] : 0.f;
        }
        // X, 16 tokens under one scale, and T
        {
            constexpr int U = C * DV / 8 / kGradThreads;
            constexpr int RW = 256 / DV, GW = 16 / RW;  // rows of a warp's units, warps of 16 rows
            const float *gx = a.saveX + hslot * C * DV;
            float x[U][8];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                get8(x[i], gx + (size_t)(tid + kGradThreads * i) * 8);
                float m = max8(x[i]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (lane == 0) red[16 * i + warp] = m;
            }
            for (int u = tid; u < 2 * kImg / 16; u += kGradThreads)
                reinterpret_cast<uint4 *>(big + SM::R)[u] =
                    reinterpret_cast<const uint4 *>(a.im.T + hslot * 2 * kImg)[u];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = tid + kGradThreads * i, rw = u / (DV / 8), col = (u % (DV / 8)) * 8;
                float m = 0.f, s, is;
#pragma unroll
                for (int w = 0; w < GW; ++w) m = fmaxf(m, red[16 * i + (warp & ~(GW - 1)) + w]);
                pow2_scale(m, s, is);
                char *d = big + img_off(rw, col);
                put8(x[i], s, d, d + C * DV * 2);
                if (lane == 0 && (warp & (GW - 1)) == 0) red[48 + (rw >> 4)] = is;
            }
        }
        __syncthreads();
        constexpr int LPR = DV / 8, RPP = kGradThreads / LPR;
        const int srow = tid / LPR, scol = (tid % LPR) * 8;
        // rho = T X: 16 tokens, a quarter of DV
        {
            float rho[NV][4] = {};
            const uint32_t uT = uB + SM::R;
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                if (jj > mt) break;
                float acc[NV][4] = {}, small[NV][4] = {};
                uint32_t th[4], tl[4];
                ldsm_x4(th, step16(uT + oA, jj));
                ldsm_x4(tl, step16(uT + oA, jj) + kImg);
#pragma unroll
                for (int np = 0; np < NV / 2; ++np) {
                    uint32_t xh[4], xl[4];
                    ldsm_x4_t(xh, step16(uB + oX, np) + 2048 * jj);
                    ldsm_x4_t(xl, step16(uB + oX, np) + 2048 * jj + C * DV * 2);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(acc[2 * np + x], th, xh[2 * x], xh[2 * x + 1]);
                        mma_f16(small[2 * np + x], tl, xh[2 * x], xh[2 * x + 1]);
                        mma_f16(small[2 * np + x], th, xl[2 * x], xl[2 * x + 1]);
                    }
                }
                const float is = red[48 + jj];
#pragma unroll
                for (int nt = 0; nt < NV; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) rho[nt][e] = fmaf(is, acc[nt][e] + small[nt][e], rho[nt][e]);
            }
            float m[2] = {0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < NV; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    rho[nt][e] *= iTs[row[e >> 1]];
                    m[e >> 1] = fmaxf(m[e >> 1], fabsf(rho[nt][e]));
                }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                m[x] = quad_max(m[x]);
                if (q4 == 0) rmax[hf * C + row[x]] = m[x];
            }
            __syncthreads();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float s, is;
                pow2_scale(fmaxf(fmaxf(rmax[row[x]], rmax[C + row[x]]),
                                 fmaxf(rmax[2 * C + row[x]], rmax[3 * C + row[x]])),
                           s, is);
                if (q4 == 0 && hf == 0) iR[row[x]] = is;
#pragma unroll
                for (int nt = 0; nt < NV; ++nt) {
                    uint32_t hi, lo;
                    split_f16(rho[nt][2 * x] * s, rho[nt][2 * x + 1] * s, hi, lo);
                    const uint32_t o = img_off(row[x], hf * (DV / 4) + 8 * nt) + 4 * q4;
                    *reinterpret_cast<uint32_t *>(sR + o) = hi;
                    *reinterpret_cast<uint32_t *>(sR + C * DV * 2 + o) = lo;
                }
            }
        }
        // 1 / scales of K and Q: of this thread's rows, and K's of all over T's (read above)
        const float iKr[2] = {vec[kVik * C + row[0]], vec[kVik * C + row[1]]};
        const float iQr[2] = {vec[kViq * C + row[0]], vec[kViq * C + row[1]]};
        float *iKs = iTs;
        if (tid < C) iKs[tid] = vec[kVik * C + tid];
        __syncthreads();  // the row maxima are read
        // W row by row (rows of DK), dZ and dX token by token
        auto stage = [&](const float(&w)[8], int rw, char *img, float *inv) {
            float m = max8(w);
#pragma unroll
            for (int x = 1; x < LPR; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            float s, is;
            // 64 rows an image, its two terms behind one another
            char *d = img + (rw >> 6) * SM::R + img_off(rw & 63, scol);
            pow2_scale(m, s, is);
            put8(w, s, d, d + C * DV * 2);
            if (tid % LPR == 0) inv[rw] = is;
        };
        char *sO = big + SM::W;  // dZ and dX, later Om
        {
            float w[DK / RPP][8], z[2 * C / RPP][8] = {};
#pragma unroll
            for (int p = 0; p < DK / RPP; ++p)
                get8(w[p], a.saveS + hslot * DK * DV + (size_t)(p * RPP + srow) * DV + scol);
#pragma unroll
            for (int p = 0; p < 2 * C / RPP; ++p) {
                const int t = (p * RPP + srow) & (C - 1);
                if (t < len) get8(z[p], (p * RPP < C ? a.dZ : a.dV) + (hrow + t) * DV + scol);
            }
#pragma unroll
            for (int p = 0; p < DK / RPP; ++p) stage(w[p], p * RPP + srow, big, iS);
#pragma unroll
            for (int p = 0; p < 2 * C / RPP; ++p) stage(z[p], p * RPP + srow, sO, iZ);
        }
        cp_async_wait_all();  // K and Q, asked for at the start
        __syncthreads();

        const float GC = Gh[C - 1], GCl = Gl[C - 1];
        float dec[2], rest[2];  // exp(G_i), exp(G_C - G_i) of this thread's two rows
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            dec[x] = expf(Gh[row[x]] + Gl[row[x]]);
            rest[x] = expf((GC - Gh[row[x]]) + (GCl - Gl[row[x]]));
        }
        // rows n0 .. of W and of Om
        const uint32_t uW = uB + (n0 >> 6) * SM::R + (n0 & 63) * 128, uO = uW + SM::W;
        float phi[2][4] = {}, eps[2][4] = {};  // tokens 16 hf + ..
        float dot[2] = {0.f, 0.f}, ktp[2] = {0.f, 0.f};
        // dZ, then dX, against W and rho
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            const uint32_t uZ = uB + SM::W + pass * SM::R;
            const float iz[2] = {iZ[pass * C + row[0]], iZ[pass * C + row[1]]};
            float(&cc)[2][4] = pass ? eps : phi;
            float cs[2][4] = {};
#pragma unroll
            for (int np = 0; np < NK / 2; ++np) {
                float N[2][4] = {}, Ns[2][4] = {};
#pragma unroll 4  // DV 128, all eight: more loads ahead than registers (297 bytes spilled, 36 us)
                for (int kk = 0; kk < KV; ++kk) {
                    uint32_t hi[4], lo[4], wh[4], wl[4];
                    ldsm_x4(hi, step16(uZ + oA, kk));
                    ldsm_x4(lo, step16(uZ + oA, kk) + C * DV * 2);
                    ldsm_x4(wh, step16(uW + oB, kk) + 2048 * np);
                    ldsm_x4(wl, step16(uW + oB, kk) + 2048 * np + C * DV * 2);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(N[x], hi, wh[2 * x], wh[2 * x + 1]);
                        mma_f16(Ns[x], lo, wh[2 * x], wh[2 * x + 1]);
                        mma_f16(Ns[x], hi, wl[2 * x], wl[2 * x + 1]);
                    }
                    if (np == 0 && hf <= mt) {  // not above the diagonal
                        ldsm_x4(wh, step16(uR + oB + 2048 * hf, kk));
                        ldsm_x4(wl, step16(uR + oB + 2048 * hf, kk) + C * DV * 2);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            mma_f16(cc[x], hi, wh[2 * x], wh[2 * x + 1]);
                            mma_f16(cs[x], lo, wh[2 * x], wh[2 * x + 1]);
                            mma_f16(cs[x], hi, wl[2 * x], wl[2 * x + 1]);
                        }
                    }
                }
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int nt = 2 * np + y, col = n0 + 8 * nt + 2 * q4;
                        const float w = (pass ? -dec[x] : a.q_scale * dec[x]) * iz[x];
                        const float y0 = w * (N[y][2 * x] + Ns[y][2 * x]) * iS[col], y1 = w * (N[y][2 * x + 1] + Ns[y][2 * x + 1]) * iS[col + 1];
                        const uint32_t o = img_off(row[x], n0 + 8 * nt) + 4 * q4;
                        const char *im = pass ? sK : sQ;
                        float2 kq = h2f(*reinterpret_cast<const uint32_t *>(im + o));
                        if (!BF16) {
                            const float2 l = h2f(*reinterpret_cast<const uint32_t *>(im + KIMG + o));
                            kq.x += l.x, kq.y += l.y;
                        }
                        const float inv = pass ? iKr[x] : iQr[x];
                        dot[x] = fmaf(inv, fmaf(kq.x, y0, kq.y * y1), dot[x]);
                        float *d = pass ? &dK[nt][2 * x] : &dQ[nt][2 * x];
                        d[0] += y0, d[1] += y1;
                    }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    cc[nt][e] = (cc[nt][e] + cs[nt][e]) *
                                (iz[e >> 1] * iR[16 * hf + 8 * nt + 2 * q4 + (e & 1)]);
        }
        __syncthreads();  // dZ and dX are read: Om takes their place
        // Om, and <W, Om> with W as it was staged
        {
            float o[DK / RPP][8], wo = 0.f;
#pragma unroll
            for (int p = 0; p < DK / RPP; ++p)
                get8(o[p], a.saveO + hslot * DK * DV + (size_t)(p * RPP + srow) * DV + scol);
#pragma unroll
            for (int p = 0; p < DK / RPP; ++p) {
                const int rw = p * RPP + srow;
                const char *d = big + (rw >> 6) * SM::R + img_off(rw & 63, scol);
                const uint4 h = *reinterpret_cast<const uint4 *>(d);
                const uint4 l = *reinterpret_cast<const uint4 *>(d + C * DV * 2);
                const uint32_t hh[4] = {h.x, h.y, h.z, h.w}, ll[4] = {l.x, l.y, l.z, l.w};
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 u = h2f(hh[j]), v = h2f(ll[j]);
                    s = fmaf(u.x + v.x, o[p][2 * j], s);
                    s = fmaf(u.y + v.y, o[p][2 * j + 1], s);
                }
                wo = fmaf(s, iS[rw], wo);
                stage(o[p], rw, sO, iO);
            }
            wo = warp_sum(wo);
            if (lane == 0) red[32 + warp] = wo;
        }
        __syncthreads();
        // rho against Om
#pragma unroll
        for (int np = 0; np < NK / 2; ++np) {
            float N[2][4] = {}, Ns[2][4] = {};
#pragma unroll 4
            for (int kk = 0; kk < KV; ++kk) {
                uint32_t hi[4], lo[4], wh[4], wl[4];
                ldsm_x4(hi, step16(uR + oA, kk));
                ldsm_x4(lo, step16(uR + oA, kk) + C * DV * 2);
                ldsm_x4(wh, step16(uO + oB, kk) + 2048 * np);
                ldsm_x4(wl, step16(uO + oB, kk) + 2048 * np + C * DV * 2);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mma_f16(N[x], hi, wh[2 * x], wh[2 * x + 1]);
                    mma_f16(Ns[x], lo, wh[2 * x], wh[2 * x + 1]);
                    mma_f16(Ns[x], hi, wl[2 * x], wl[2 * x + 1]);
                }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int nt = 2 * np + y, col = n0 + 8 * nt + 2 * q4;
                    const float w = rest[x] * iR[row[x]];
                    const float y0 = w * (N[y][2 * x] + Ns[y][2 * x]) * iO[col], y1 = w * (N[y][2 * x + 1] + Ns[y][2 * x + 1]) * iO[col + 1];
                    const uint32_t o = img_off(row[x], n0 + 8 * nt) + 4 * q4;
                    float2 kq = h2f(*reinterpret_cast<const uint32_t *>(sK + o));
                    if (!BF16) {
                        const float2 l = h2f(*reinterpret_cast<const uint32_t *>(sK + KIMG + o));
                        kq.x += l.x, kq.y += l.y;
                    }
                    const float inv = iKr[x];
                    ktp[x] = fmaf(inv, fmaf(kq.x, y0, kq.y * y1), ktp[x]);
                    dK[nt][2 * x] = fmaf(eta[row[x]], y0, dK[nt][2 * x]);
                    dK[nt][2 * x + 1] = fmaf(eta[row[x]], y1, dK[nt][2 * x + 1]);
                }
        }
        // the triangle: q_i.k_j and k_i.k_j of this warp's 16 x 16 block
        float kk2[2][4] = {}, qk2[2][4] = {};
        if (hf <= mt) {
            float ks[2][4] = {}, qs[2][4] = {};
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                uint32_t ak[4], aq[4], bb[4];
                ldsm_x4(ak, step16(uK + oA, k));
                ldsm_x4(aq, step16(uQ + oA, k));
                ldsm_x4(bb, step16(uK + oB + 2048 * hf, k));
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mma_f16(kk2[x], ak, bb[2 * x], bb[2 * x + 1]);
                    mma_f16(qk2[x], aq, bb[2 * x], bb[2 * x + 1]);
                }
                if (!BF16) {
                    uint32_t akl[4], aql[4], bl[4];
                    ldsm_x4(akl, step16(uK + oA, k) + KIMG);
                    ldsm_x4(aql, step16(uQ + oA, k) + KIMG);
                    ldsm_x4(bl, step16(uK + oB + 2048 * hf, k) + KIMG);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(ks[x], akl, bb[2 * x], bb[2 * x + 1]);
                        mma_f16(qs[x], aql, bb[2 * x], bb[2 * x + 1]);
                        mma_f16(ks[x], ak, bl[2 * x], bl[2 * x + 1]);
                        mma_f16(qs[x], aq, bl[2 * x], bl[2 * x + 1]);
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) kk2[x][e] += ks[x][e], qk2[x][e] += qs[x][e];
        }
        __syncthreads();  // rho, W and Om are read
        // The sums over pairs in double: a pair comes into the running sum of dg with its
        // column and leaves it with its row, and what stays may be 2^30 smaller (behind a
        // forgetting). eta_j times the pair is exact in 48 bits.
        double rs[2] = {0.0, 0.0};
        float pm[2] = {0.f, 0.f}, em[2] = {0.f, 0.f};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            double cs[2] = {0.0, 0.0};
            float qm[2] = {0.f, 0.f}, fm[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = row[e >> 1], j = 16 * hf + 8 * nt + 2 * q4 + (e & 1);
                float p = 0.f, q = 0.f;
                if (j <= i) {
                    const float gam = expf((Gh[i] - Gh[j]) + (Gl[i] - Gl[j]));
                    const float ikj = iKs[j], iqi = iQr[e >> 1], iki = iKr[e >> 1];
                    p = a.q_scale * gam * phi[nt][e];
                    if (j < i) q = -gam * eps[nt][e];
                    const float w = ikj * (p * qk2[nt][e] * iqi + q * kk2[nt][e] * iki);
                    if (j < i) {
                        cs[e & 1] += w;
                        rs[e >> 1] = fma((double)eta[j], (double)w, rs[e >> 1]);
                    } else
                        diag[i] = w;
                    p *= eta[j];
                    q *= eta[j];
                    // as operands: the rows of K and Q they meet carry their scales
                    pm[e >> 1] = fmaxf(pm[e >> 1], fabsf(p * ikj));
                    qm[e & 1] = fmaxf(qm[e & 1], fabsf(p * iqi));
                    em[e >> 1] = fmaxf(em[e >> 1], fabsf(q * ikj));
                    fm[e & 1] = fmaxf(fm[e & 1], fabsf(q * iki));
                }
                phi[nt][e] = p;
                eps[nt][e] = q;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) {
                    cs[x] += __shfl_xor_sync(0xffffffffu, cs[x], o);
                    qm[x] = fmaxf(qm[x], __shfl_xor_sync(0xffffffffu, qm[x], o));
                    fm[x] = fmaxf(fm[x], __shfl_xor_sync(0xffffffffu, fm[x], o));
                }
                const int at = mt * C + 16 * hf + 8 * nt + 2 * q4 + x;
                if (gq == 0) colp[at] = cs[x], p_col[at] = qm[x], e_col[at] = fm[x];
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float d = dot[x], k2 = ktp[x];
            double w = rs[x];
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                d += __shfl_xor_sync(0xffffffffu, d, o);
                w += __shfl_xor_sync(0xffffffffu, w, o);
                k2 += __shfl_xor_sync(0xffffffffu, k2, o);
            }
            pm[x] = quad_max(pm[x]), em[x] = quad_max(em[x]);
            const int at = hf * C + row[x];
            if (q4 == 0) decp[at] = d, rowp[at] = w, dotp[at] = k2, p_row[at] = pm[x], e_row[at] = em[x];
        }
        __syncthreads();  // sums and maxima are there
        // a scale a row of what is multiplied: of phi eta, of its transpose, of E + E^T
        if (tid < 3 * C) {
            const int y = tid >> 6, i = tid & 63;
            auto max4 = [&](const float *v) { return fmaxf(fmaxf(v[i], v[C + i]), fmaxf(v[2 * C + i], v[3 * C + i])); };
            float s, is;
            pow2_scale(y == 0 ? max4(p_row) : y == 1 ? max4(p_col) : fmaxf(max4(e_row), max4(e_col)), s, is);
            isc[tid] = s;
        }
        __syncthreads();
        char *i1 = big, *i2 = big + 2 * kImg, *i3 = big + 4 * kImg;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const int j0 = 16 * hf + 8 * nt + 2 * q4;
            const float k0 = iKs[j0], k1 = iKs[j0 + 1];
            const float q0 = isc[C + j0], q1 = isc[C + j0 + 1], f0 = isc[2 * C + j0], f1 = isc[2 * C + j0 + 1];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = row[x];
                const float qi = iQr[x], ki = iKr[x];
                const float p0 = phi[nt][2 * x], p1 = phi[nt][2 * x + 1];
                const float e0 = eps[nt][2 * x], e1 = eps[nt][2 * x + 1];
                const uint32_t o = img_off(i, 16 * hf + 8 * nt) + 4 * q4;
                uint32_t hi, lo;
                split_f16(p0 * k0 * isc[i], p1 * k1 * isc[i], hi, lo);
                *reinterpret_cast<uint32_t *>(i1 + o) = hi;
                *reinterpret_cast<uint32_t *>(i1 + kImg + o) = lo;
                split_f16(p0 * qi * q0, p1 * qi * q1, hi, lo);
                *reinterpret_cast<uint32_t *>(i2 + o) = hi;
                *reinterpret_cast<uint32_t *>(i2 + kImg + o) = lo;
                // E + E^T: the element below the diagonal, and its mirror
                uint32_t uh, ul;
                split_f16(e0 * k0 * isc[2 * C + i], e1 * k1 * isc[2 * C + i], hi, lo);
                split_f16(e0 * ki * f0, e1 * ki * f1, uh, ul);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int j = j0 + y;
                    if (j > i) continue;
                    const uint32_t ol = img_off(i, j & ~7) + 2 * (j & 7);
                    *reinterpret_cast<uint16_t *>(i3 + ol) = (uint16_t)(hi >> (16 * y));
                    *reinterpret_cast<uint16_t *>(i3 + kImg + ol) = (uint16_t)(lo >> (16 * y));
                    if (j == i) continue;
                    const uint32_t ou = img_off(j, i & ~7) + 2 * (i & 7);
                    *reinterpret_cast<uint16_t *>(i3 + ou) = (uint16_t)(uh >> (16 * y));
                    *reinterpret_cast<uint16_t *>(i3 + kImg + ou) = (uint16_t)(ul >> (16 * y));
                }
            }
        }
        if (tid < C) {
            auto sum4 = [&](const auto *v) {
                return (v[tid] + v[C + tid]) + (v[2 * C + tid] + v[3 * C + tid]);
            };
            const double cs = sum4(colp);
            const float k2 = sum4(dotp);
            if (tid < len) a.deta[hrow + tid] = ((float)cs + diag[tid]) + k2;
            from[tid] = sum4(decp);
            upto[tid] = eta[tid] * (cs + k2) - sum4(rowp);
        }
        __syncthreads();
        if (a.dg && warp == 15) {
            // sums over tokens in double. Lane l holds tokens 2 l, 2 l + 1.
            const double a0 = from[2 * lane], a1 = from[2 * lane + 1];
            const double b0 = upto[2 * lane], b1 = upto[2 * lane + 1];
            double s = a0 + a1, u = b0 + b1, d = lane < 16 ? (double)red[32 + lane] : 0.0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_down_sync(0xffffffffu, s, o);
                if (lane + o < 32) s += v;
                const double w = __shfl_up_sync(0xffffffffu, u, o);
                if (lane >= o) u += w;
                d += __shfl_xor_sync(0xffffffffu, d, o);
            }
            // s: from token 2 l on, u: up to token 2 l + 1
            const double later = __shfl_down_sync(0xffffffffu, s, 1);
            const double before = __shfl_up_sync(0xffffffffu, u, 1);
            const double c0 = lane > 0 ? before : 0.0, wo = (double)expf(GC + GCl) * d;
            if (2 * lane < len) a.dg[hrow + 2 * lane] = (float)(s + c0 + wo);
            if (2 * lane + 1 < len)
                a.dg[hrow + 2 * lane + 1] = (float)(a1 + (lane < 31 ? later : 0.0) + (c0 + b0) + wo);
        }
        // dQ += (phi eta) K, dK += (phi eta)^T Q + (E + E^T) K
        float ix[3][2];
#pragma unroll
        for (int y = 0; y < 3; ++y)
#pragma unroll
            for (int x = 0; x < 2; ++x) ix[y][x] = inv_pow2(isc[y * C + row[x]]);
        const uint32_t u1 = smem_u32(i1), u2 = smem_u32(i2), u3 = smem_u32(i3);
        const uint32_t oAt = img_off(rB, 16 * mt + cB);  // A read across
#pragma unroll
        for (int np = 0; np < NK / 2; ++np) {
            float q[2][4] = {}, k[2][4] = {}, e[2][4] = {};
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                uint32_t bk[4], bq[4], bkl[4], bql[4], ah[4], al[4];
                ldsm_x4_t(bk, step16(uK + oK, np) + 2048 * jj);
                ldsm_x4_t(bq, step16(uQ + oK, np) + 2048 * jj);
                if (!BF16) {
                    ldsm_x4_t(bkl, step16(uK + oK, np) + 2048 * jj + KIMG);
                    ldsm_x4_t(bql, step16(uQ + oK, np) + 2048 * jj + KIMG);
                }
                auto add = [&](float(&acc)[2][4], const uint32_t(&bh)[4], const uint32_t(&bl)[4]) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mma_f16(acc[x], ah, bh[2 * x], bh[2 * x + 1]);
                        mma_f16(acc[x], al, bh[2 * x], bh[2 * x + 1]);
                        if (!BF16) mma_f16(acc[x], ah, bl[2 * x], bl[2 * x + 1]);
                    }
                };
                if (jj <= mt) {
                    ldsm_x4(ah, step16(u1 + oA, jj));
                    ldsm_x4(al, step16(u1 + oA, jj) + kImg);
                    add(q, bk, bkl);
                }
                if (jj >= mt) {  // A = (phi eta)^T: read across
                    ldsm_x4_t(ah, u2 + oAt + 2048 * jj);
                    ldsm_x4_t(al, u2 + oAt + 2048 * jj + kImg);
                    add(k, bq, bql);
                }
                ldsm_x4(ah, step16(u3 + oA, jj));
                ldsm_x4(al, step16(u3 + oA, jj) + kImg);
                add(e, bk, bkl);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    dQ[2 * np + x][y] = fmaf(ix[0][y >> 1], q[x][y], dQ[2 * np + x][y]);
                    dK[2 * np + x][y] += fmaf(ix[1][y >> 1], k[x][y], ix[2][y >> 1] * e[x][y]);
                }
        }
    }
    const size_t krow = ((size_t)b * a.Hk + hk) * a.T + t0;
#pragma unroll
    for (int x = 0; x < 2; ++x)
        if (row[x] < len)
#pragma unroll
            for (int nt = 0; nt < NK; ++nt) {
                const size_t at = (krow + row[x]) * DK + n0 + 8 * nt + 2 * q4;
                *reinterpret_cast<float2 *>(a.dQ + at) = make_float2(dQ[nt][2 * x], dQ[nt][2 * x + 1]);
                *reinterpret_cast<float2 *>(a.dK + at) = make_float2(dK[nt][2 * x], dK[nt][2 * x + 1]);
            }
}

// Sum over the sequences of a shared start weight's gradient, in order, sixteen loads
// on their way. Bound by their latency, the order being fixed: 512 sequences of 16 heads of
// 128 x 128, 537 MB, in 111 us, of 2 heads in 97 (124 and 113 in blocks of 256, one by one).
constexpr int kSumThreads = 64;
__global__ void __launch_bounds__(kSumThreads) delta_sum_kernel(const float *per_seq, float *out,
                                                                int N, size_t n4) {
    const size_t i = (size_t)blockIdx.x * kSumThreads + threadIdx.x;
    if (i >= n4) return;
    const float4 *p = reinterpret_cast<const float4 *>(per_seq) + i;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 &v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
    int k = 0;
    for (; k + 16 <= N; k += 16, p += 16 * n4) {
        float4 v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = p[j * n4];
#pragma unroll
        for (int j = 0; j < 16; ++j) add(v[j]);
    }
    for (; k < N; ++k, p += n4) add(*p);
    reinterpret_cast<float4 *>(out)[i] = s;
}

// Zero gradients for the tokens in front of the first packed sequence and behind the
// last, a head by the blocks of one x: bound by its stores (a buffer of 262,144 tokens,
// half of them behind the last sequence, 8 heads of 128: 1.6 GB in 280 us).
__global__ void __launch_bounds__(256) delta_outside_kernel(float *dQ, float *dK, float *dV,
                                                            float *deta, float *dg,
                                                            const int *seq_start, int N, int Hk,
                                                            int H, int T, int dk, int dv) {
    int first, last, len;
    delta_span(seq_start, 0, T, first, len);
    delta_span(seq_start, N - 1, T, last, len);
    last += len;
    if (last < first) last = first;
    const int h = blockIdx.x, out = first + (T - last), lane = threadIdx.x & 31;
    auto row = [&](int t) { return (size_t)h * T + (t < first ? t : t - first + last); };
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    // a token a warp: its rows of 64 or 128
    for (int t = blockIdx.y * 8 + (threadIdx.x >> 5); t < out; t += gridDim.y * 8) {
        const size_t r = row(t);
        if (4 * lane < dv) reinterpret_cast<float4 *>(dV + r * dv)[lane] = zero;
        if (h < Hk && 4 * lane < dk) {
            reinterpret_cast<float4 *>(dQ + r * dk)[lane] = zero;
            reinterpret_cast<float4 *>(dK + r * dk)[lane] = zero;
        }
        if (lane == 0) deta[r] = 0.f;
        if (lane == 1 && dg) dg[r] = 0.f;
    }
}

struct BwdPlan {
    Plan p;
    size_t oS, oO, oX, oW, end;
};
BwdPlan bwd_plan(int B, int Hk, int H, int T, int dk, int dv, int N, bool packed, bool bf16) {
    BwdPlan q;
    q.p = make_plan(B, Hk, H, T, dk, N, packed, bf16, true);
    const size_t st = up256((size_t)q.p.slots * H * dk * dv * 4);
    q.oS = q.p.end;
    q.oO = q.oS + st;
    q.oX = q.oO + st;
    q.oW = q.oX + up256((size_t)q.p.slots * H * C * dv * 4);
    q.end = q.oW + up256((size_t)N * H * dk * dv * 4);
    return q;
}

template <int DK, bool BF16>
cudaError_t rev_inst(RevArgs r, int N, cudaStream_t s) {
    constexpr int stage = rev_stage_bytes<DK, BF16>(), zstage = rev_zstage_bytes<DK, BF16>();
    constexpr int area = rev_area_bytes<DK, BF16>();
    // two stages of the chain's ring at least (the gate frees one when the chain has
    // met it for the next), two of the helpers' or a third of the chain's where there is room
    static_assert(2 * stage + zstage + area <= kScanSmem, "shared memory");
    r.stages = 2;
    r.zstages = 2 * (stage + zstage) + area <= kScanSmem ? 2 : 1;
    if (3 * stage + 2 * zstage + area <= kScanSmem) r.stages = 3;
    const int smem = r.stages * stage + r.zstages * zstage + area;
    static SmemOnce once;
    cudaError_t e = once.allow(delta_rev_kernel<DK, BF16>, kScanSmem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((long long)N * r.H * (r.dv / 16));
    delta_rev_kernel<DK, BF16><<<grid, 352, smem, s>>>(r);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}

template <int DK, int DV, bool BF16>
cudaError_t grad_inst(const GradArgs &r, int blocks, cudaStream_t s) {
    constexpr int smem = GradSmem<DK, DV, BF16>::bytes;
    static_assert(smem <= 227 * 1024, "shared memory");
    static SmemOnce once;
    cudaError_t e = once.allow(delta_grad_kernel<DK, DV, BF16>, smem);
    if (e != cudaSuccess) return e;
    delta_grad_kernel<DK, DV, BF16><<<blocks, kGradThreads, smem, s>>>(r);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(s);
    return e;
}
template <int DK, int DV>
cudaError_t grad_type(const GradArgs &r, bool bf16, int blocks, cudaStream_t s) {
    return bf16 ? grad_inst<DK, DV, true>(r, blocks, s) : grad_inst<DK, DV, false>(r, blocks, s);
}

}  // namespace
}  // namespace delta

using namespace delta;

size_t delta_bwd_workspace_bytes(int B, int Hk, int H, int T, int dk, int dv, int N, bool packed,
                                 bool bf16) {
    return bwd_plan(B, Hk, H, T, dk, dv, N, packed, bf16).end;
}

cudaError_t launch_delta_bwd(const DeltaBwdArgs &g, cudaStream_t s) {
    DeltaArgs a = g.f;
    const BwdPlan q = bwd_plan(a.B, a.Hk, a.H, a.T, a.dk, a.dv, a.N, a.seq_start != nullptr, a.bf16);
    char *ws = static_cast<char *>(a.workspace);
    const Images im = images_at(q.p, ws, true);
    float *saveS = reinterpret_cast<float *>(ws + q.oS), *saveO = reinterpret_cast<float *>(ws + q.oO),
          *saveX = reinterpret_cast<float *>(ws + q.oX), *sums = reinterpret_cast<float *>(ws + q.oW);
    a.Z = nullptr;
    a.W_out = nullptr;
    cudaError_t e = launch_prep(a, q.p, im, s);
    if (e != cudaSuccess) return e;
    e = launch_scan(a, im, kSave, saveS, saveX, s);
    if (e != cudaSuccess) return e;
    const bool sum = g.dW0 && !a.w0_per_seq;
    const RevArgs r{g.dZ, g.dW_out, g.dV, sum ? sums : g.dW0, a.seq_start, a.B, a.Hk, a.H, a.T,
                    a.dv, 0, 0, im, saveO, device_status_word()};
    if (a.dk == 64) e = a.bf16 ? rev_inst<64, true>(r, a.N, s) : rev_inst<64, false>(r, a.N, s);
    else e = a.bf16 ? rev_inst<128, true>(r, a.N, s) : rev_inst<128, false>(r, a.N, s);
    if (e != cudaSuccess) return e;
    const GradArgs d{g.dZ, g.dV, a.eta, saveS, saveX, saveO, g.dQ, g.dK, g.deta, g.dg, a.seq_start,
                     a.B, a.Hk, a.H, a.T, a.N, a.q_scale, im};
    const int blocks = q.p.slots * a.Hk;
    if (a.dk == 64)
        e = a.dv == 64 ? grad_type<64, 64>(d, a.bf16, blocks, s) : grad_type<64, 128>(d, a.bf16, blocks, s);
    else
        e = a.dv == 64 ? grad_type<128, 64>(d, a.bf16, blocks, s) : grad_type<128, 128>(d, a.bf16, blocks, s);
    if (e != cudaSuccess) return e;
    if (sum) {
        const size_t n4 = (size_t)a.H * a.dk * a.dv / 4;
        delta_sum_kernel<<<(unsigned)((n4 + kSumThreads - 1) / kSumThreads), kSumThreads, 0, s>>>(
            sums, g.dW0, a.N, n4);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        count_launch(s);
    }
    if (a.seq_start) {
        const unsigned slices = (unsigned)((a.T + 511) / 512);
        delta_outside_kernel<<<dim3(a.H, slices < 128 ? slices : 128), 256, 0, s>>>(g.dQ, g.dK, g.dV, g.deta, g.dg, a.seq_start, a.N,
                                                 a.Hk, a.H, a.T, a.dk, a.dv);
        e = cudaGetLastError();
        if (e == cudaSuccess) count_launch(s);
    }
    return e;
}

}  // namespace ttt
