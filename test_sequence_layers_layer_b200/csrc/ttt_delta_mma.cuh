// ttt_delta_mma.cuh -- the operand form of the chunked gated delta rule.
//
// An fp32 operand goes to the tensor cores as two fp16 terms under a
// power-of-two scale of its row (of what the tokens bring, 16 tokens' values of a column, or of
// all columns in the gradients' X, may share one): with the row's largest size brought into
// [2^13, 2^14), x s = hi + lo + e, hi = fp16(x s), lo = fp16(x s - hi) and |e| <= 2^-22
// of |x s| (2^-25 absolute for the elements more than 2^17 below the largest): the
// precision of fp32 products, in two or three fp16 products (lo lo is left
// out) instead of the three or six that bf16 terms would take for the same bits. Where a
// sum runs over many steps, hi hi and the others go to accumulators of their own: the
// tensor cores cut a sum off below its last bit at every step, and so a third as often. A
// bf16 operand is one term, exact in fp16 (8 bits of 11) down to 2^-27 of its
// row's largest size. The scales are taken out again in fp32, where the rows of
// the result are scaled anyway.
#pragma once

#include "sm100.cuh"
#include "ttt_delta.cuh"

#include <cuda_fp16.h>

#include <atomic>

namespace ttt {
namespace delta {
using namespace sm100;
}  // namespace delta
}  // namespace ttt

#include "ttt_delta_ring.cuh"

namespace ttt {
namespace delta {

constexpr int C = kDeltaC;
constexpr int kImg = C * C * 2;  // bytes of a 64 x 64 fp16 image

// Per chunk and value head: vectors of 64 floats; sX is the scale of row j of image
// X. The scans' chains read the first two, the warps beside them the next two.
enum Vec {
    kVk,   // exp(G_j) / sK_j
    kVs,   // [0] exp(G_C), [1 + b] 1 / sH of the 16 rows of block b (one scale for them)
    kVq,   // c exp(G_i) / sQ_i
    kVm,   // 1 / sM_i
    kVik,  // 1 / sK_j
    kViq,  // 1 / sQ_i
    kVgh,  // G_j as the sum of two floats
    kVgl,
    kVit,  // 1 / sT_i
    kVecs
};
constexpr int kVecBytes = kVecs * C * 4, kHalfVecBytes = 2 * C * 4;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Power of two s that brings amax into [2^13, 2^14), and 1 / s; both stay normal
// numbers for any amax (zero, subnormal, infinity, NaN).
__device__ __forceinline__ void pow2_scale(float amax, float &s, float &inv) {
    const int e = (__float_as_int(amax) >> 23) & 255;
    int f = 267 - e;
    f = f > 253 ? 253 : f;
    s = __int_as_float(f << 23);
    inv = __int_as_float((254 - f) << 23);
}

// 1 / s of a scale that pow2_scale gave.
__device__ __forceinline__ float inv_pow2(float s) {
    return __int_as_float((254 << 23) - __float_as_int(s));
}

__device__ __forceinline__ uint32_t h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// hi and lo terms of a pair already scaled.
__device__ __forceinline__ void split_f16(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = h2(a - f.x, b - f.y);
}

// Byte offset of the 16-byte unit (row, col .. col + 7) of a 64-row fp16 image:
// 128-byte swizzled rows, 64 columns after one another.
__device__ __forceinline__ uint32_t img_off(int row, int col) {
    return (uint32_t)((col >> 6) * (C * 128) + (row >> 3) * 1024 + (row & 7) * 128 +
                      ((((col & 63) >> 3) ^ (row & 7)) << 4));
}

// An address inside an image, k steps of 16 columns on. The steps must not carry into a bit
// that the first column has; images stand at multiples of 128 bytes.
__device__ __forceinline__ uint32_t step16(uint32_t at, int k) {
    return (at ^ ((k & 3) << 5)) + (k >> 2) * (C * 128);
}

// Shared address of this lane's row for an ldmatrix.x4 of a 16 x 16 block at
// (row, col). Plain, as A: registers a0..a3. Plain, as B with the rows as n and
// the columns as k: {b0, b1} of the first 8 rows, then of the next 8 (order 0, 2 / 1, 3).
__device__ __forceinline__ uint32_t ldsm_addr(uint32_t img, int row, int col, int lane) {
    return img + img_off(row + (lane & 15), col + (lane >> 4) * 8);
}
// B with rows as n: b0, b1 of rows row .. row + 7 in r[0], r[1], of the next 8 in r[2], r[3].
__device__ __forceinline__ void load_b(uint32_t (&r)[4], uint32_t img, int row, int col, int lane) {
    ldsm_x4(r, img + img_off(row + ((lane >> 4) << 3) + (lane & 7), col + ((lane >> 3) & 1) * 8));
}
// B with rows as k: b0, b1 of columns col .. col + 7 in r[0], r[1], of the next 8 in r[2], r[3].
__device__ __forceinline__ void load_bt(uint32_t (&r)[4], uint32_t img, int row, int col,
                                        int lane) {
    ldsm_x4_t(r, img + img_off(row + (lane & 15), col + (lane >> 4) * 8));
}

// Largest size over the four lanes that share a row.
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// A fragments of a 16 x 16 block held as two accumulator tiles (columns 0..7 and
// 8..15), both terms; s: the scales of rows gq and gq + 8.
__device__ __forceinline__ void a_terms(const float (&t0)[4], const float (&t1)[4],
                                        const float (&s)[2], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split_f16(t0[0] * s[0], t0[1] * s[0], hi[0], lo[0]);
    split_f16(t0[2] * s[1], t0[3] * s[1], hi[1], lo[1]);
    split_f16(t1[0] * s[0], t1[1] * s[0], hi[2], lo[2]);
    split_f16(t1[2] * s[1], t1[3] * s[1], hi[3], lo[3]);
}
// Scales of a warp's two rows over N accumulator tiles.
template <int N>
__device__ __forceinline__ void row_scales(const float (&t)[N][4], float (&s)[2], float (&inv)[2]) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, fmaxf(fabsf(t[i][2 * x]), fabsf(t[i][2 * x + 1])));
        pow2_scale(quad_max(m), s[x], inv[x]);
    }
}

__device__ __forceinline__ void named_bar(int id, int nthreads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

constexpr int kScanSmem = 231936;  // dynamic shared memory a scan may take (227 KB less its barriers)

// Counts this warp in at a barrier that others wait at.
__device__ __forceinline__ void named_arrive(int id, int nthreads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// What a scan writes: Z as bf16, Z as fp32, or (for the backward) the weight
// each chunk starts from and X.
enum ScanMode { kZ16, kZ32, kSave };

// Workspace: per chunk slot and head, the images that the scans read.
//   K, Q [key head]: the chunk's rows, one fp16 term (bf16 inputs) or two
//   M, H [value head], two terms each: M = P T [64][64], H = T^T diag(u) K [64][dk]
//   T [value head], two terms, only for the backward
//   vec [value head]: the vectors above
struct Plan {
    int slots;          // chunk slots of all sequences
    size_t kimg, himg;  // bytes of one chunk's K (or Q), and H
    size_t oK, oQ, oM, oH, oT, oV, end;
};
inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
inline Plan make_plan(int B, int Hk, int H, int T, int dk, int N, bool packed, bool bf16,
                      bool bwd) {
    Plan p;
    // packed: sequence n starts at slot start / 64 + n, so that the slots of two
    // sequences never meet, whatever the offsets
    p.slots = packed ? T / C + N : B * ((T + C - 1) / C);
    p.kimg = (size_t)C * dk * 2 * (bf16 ? 1 : 2);
    p.himg = (size_t)C * dk * 2 * 2;
    size_t o = 0;
    auto take = [&](size_t n) {
        const size_t at = o;
        o += up256(n);
        return at;
    };
    p.oK = take((size_t)p.slots * Hk * p.kimg);
    p.oQ = take((size_t)p.slots * Hk * p.kimg);
    p.oM = take((size_t)p.slots * H * 2 * kImg);
    p.oH = take((size_t)p.slots * H * p.himg);
    p.oV = take((size_t)p.slots * H * kVecBytes);
    p.oT = o;
    if (bwd) take((size_t)p.slots * H * 2 * kImg);
    p.end = o;
    return p;
}

// Where the kernels find the images of a chunk; T is NULL in the forward.
struct Images {
    char *K, *Q, *M, *H, *T, *vec;
    size_t kimg, himg;
};

__device__ __forceinline__ int first_slot(const int *seq_start, int n, int T, int t0) {
    return seq_start ? t0 / C + n : n * ((T + C - 1) / C);
}

// Sequence of a slot, and its chunk's first token (inside the batch row) and
// length; false for a slot that no chunk uses.
struct ChunkSearch {
    const int *seq_start;
    int T, N;
    __device__ __forceinline__ bool find(int slot, int &n, int &t0, int &len) const {
        int c;
        if (!seq_start) {
            const int per = (T + C - 1) / C;
            n = slot / per;
            c = slot - n * per;
            t0 = 0;
            len = T;
        } else {
            // the last sequence whose first slot is not behind this one
            int lo = 0, hi = N - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                int s, l;
                delta_span(seq_start, mid, T, s, l);
                if (s / C + mid <= slot) lo = mid;
                else hi = mid - 1;
            }
            n = lo;
            delta_span(seq_start, n, T, t0, len);
            c = slot - (t0 / C + n);
            if (c < 0) return false;
        }
        t0 += c * C;
        len -= c * C;
        len = len < C ? len : C;
        return len > 0;
    }
};

// Lets a kernel take `bytes` of dynamic shared memory, asked of the runtime once
// per device (the request costs about a microsecond). Two threads may both ask.
struct SmemOnce {
    std::atomic<bool> done[64] = {};
    template <class K>
    cudaError_t allow(K *kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
        return e;
    }
};

// The shared part of the chunk preparation's launch (ttt_delta_chunk.cu).
cudaError_t launch_prep(const DeltaArgs &a, const Plan &p, const Images &im, cudaStream_t s);
Images images_at(const Plan &p, void *workspace, bool bwd);
cudaError_t launch_scan(const DeltaArgs &a, const Images &im, int mode, float *saveS, float *saveX,
                        cudaStream_t s);

}  // namespace delta
}  // namespace ttt
