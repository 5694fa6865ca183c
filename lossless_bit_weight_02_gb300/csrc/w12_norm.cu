// Residual addition + root-mean-square norm, BF16 or 8-bit output: what
// stands between two GEMMs of a decoder layer (SpecPilot, arXiv 2611.02501,
// describes the GEMMs of a verify pass; the published RMS norm, Zhang and
// Sennrich 2019, is written out here because the pages do not).
//
//     h = x + r,   t_k = h_k rsqrt(mean(h^2) + eps) w_k
//     h_out = BF16(h), y = BF16(t), q8 = e4m3(t / s_g), s_g = max_g |t| / 448
//
// One CTA owns one row: every thread loads its 8-column chunks of x and r
// (16 bytes each, all in flight at once), keeps h in FP32 registers, and the
// row's sum of squares goes through one shuffle tree and one shared-memory
// step; nothing is read twice and nothing but the outputs is written.  A row
// is one pass, so the kernel is bound by HBM for many rows and by the
// load-reduce-store latency for few: 16383 rows of 5120 with a residual (671
// MB) take 96.5 us, 6.9 TB/s; one row takes 2.1 us.  The 16 threads that hold
// the chunks of a 128-column group are neighbours in one half-warp, so the
// group's maximum takes four shuffles.
//
// The number of chunks per thread is a rule on K alone (launch_rmsnorm), so the
// order of the sum, and with it every bit of the result, does not depend on M.
#include <cstdint>
#include <cuda_runtime.h>

#include "w12_device.cuh"
#include "w12_internal.h"
#include "w12_stream.cuh"

namespace w12 {
namespace {

struct NormArgs {
    const uint16_t *x, *r, *w;
    int64_t ldx, ldr;
    uint16_t *h, *y;
    int64_t ldh, ldy;
    uint8_t *q8;
    int64_t ldq;
    float *scale;
    int64_t lds;
    int K;
    float eps, inv_k;
};

__device__ __forceinline__ float bf2f(uint32_t b) { return __uint_as_float(b << 16); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// two e4m3 codes, lower column in the low byte; finite values beyond 448 saturate
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 columns of a row (zeros past K).  Rows that do not begin on 16 bytes are
// moved in aligned pairs of words or words, shifted by half a word where they
// begin between two (10000 rows of 3001 with a residual: 60 us, column by
// column 126).
template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t *row, int k, int K, uint32_t v[4]) {
    if (VEC) {
        const uint4 u = *reinterpret_cast<const uint4 *>(row + k);
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
        return;
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
    if ((at & 7) == 0 && k + 8 <= K) {
        const uint2 *w = reinterpret_cast<const uint2 *>(at);
        const uint2 a = w[0], b = w[1];
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else if (k > 0 && k + 8 < K) {  // the words at both ends lie in the row too
        const uint32_t *w = reinterpret_cast<const uint32_t *>(at & ~(uintptr_t)3);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = w[j];
        if (at & 2) {
            const uint32_t last = w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __funnelshift_r(v[j], j < 3 ? v[j + 1] : last, 16);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = k + 2 * j < K ? row[k + 2 * j] : 0, hi = k + 2 * j + 1 < K ? row[k + 2 * j + 1] : 0;
            v[j] = lo | hi << 16;
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint16_t *row, int k, int K, const float t[8]) {
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pack_bf16(t[2 * j], t[2 * j + 1]);
    if (VEC) {
        *reinterpret_cast<uint4 *>(row + k) = make_uint4(v[0], v[1], v[2], v[3]);
        return;
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
    if ((at & 7) == 0 && k + 8 <= K) {
        uint2 *w = reinterpret_cast<uint2 *>(at);
        w[0] = make_uint2(v[0], v[1]), w[1] = make_uint2(v[2], v[3]);
    } else if (k + 8 <= K) {
        const bool odd = at & 2;
        if (odd) {
            row[k] = (uint16_t)v[0];
            row[k + 7] = (uint16_t)(v[3] >> 16);
        }
        uint32_t *w = reinterpret_cast<uint32_t *>(row + k + odd);
#pragma unroll
        for (int j = 0; j < 3; ++j) w[j] = odd ? __funnelshift_r(v[j], v[j + 1], 16) : v[j];
        if (!odd) w[3] = v[3];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k + j < K) row[k + j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
    }
}

// C chunks per thread; RES / QUANT: a residual is added / 8-bit output.
template <int C, bool VEC, bool RES, bool QUANT>
__global__ __launch_bounds__(1024) void k_rmsnorm(NormArgs a) {
    __shared__ float part[32];
    const int T = blockDim.x, tid = threadIdx.x, K = a.K;
    const int64_t m = blockIdx.x;
    const uint16_t *x = a.x + m * a.ldx, *r = RES ? a.r + m * a.ldr : nullptr;
    uint32_t xv[C][4], rv[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = 8 * (tid + c * T);
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[c][j] = rv[c][j] = 0;
        if (k < K) {
            load8<VEC>(x, k, K, xv[c]);
            if (RES) load8<VEC>(r, k, K, rv[c]);
        }
    }
    float h[C][8], ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[c][2 * j] = bf2f(xv[c][j]);
            h[c][2 * j + 1] = __uint_as_float(xv[c][j] & 0xFFFF0000u);
            if (RES) {
                h[c][2 * j] += bf2f(rv[c][j]);
                h[c][2 * j + 1] += __uint_as_float(rv[c][j] & 0xFFFF0000u);
            }
            ss = fmaf(h[c][2 * j], h[c][2 * j], ss);
            ss = fmaf(h[c][2 * j + 1], h[c][2 * j + 1], ss);
        }
    // the weights and h_out do not wait for the sum
    uint32_t wv[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = 8 * (tid + c * T);
#pragma unroll
        for (int j = 0; j < 4; ++j) wv[c][j] = 0;
        if (k < K) {
            load8<VEC>(a.w, k, K, wv[c]);
            if (a.h) store8<VEC>(a.h + m * a.ldh, k, K, h[c]);
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) ss += __shfl_xor_sync(kFull, ss, s);
    if (T > 32) {
        if ((tid & 31) == 0) part[tid >> 5] = ss;
        __syncthreads();
        ss = (tid & 31) < (T >> 5) ? part[tid & 31] : 0.f;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) ss += __shfl_xor_sync(kFull, ss, s);
    }
    const float rstd = rsqrtf(fmaf(ss, a.inv_k, a.eps));
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = 8 * (tid + c * T);
        float t[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            t[2 * j] = h[c][2 * j] * rstd * bf2f(wv[c][j]);
            t[2 * j + 1] = h[c][2 * j + 1] * rstd * __uint_as_float(wv[c][j] & 0xFFFF0000u);
        }
        if (a.y && k < K) store8<VEC>(a.y + m * a.ldy, k, K, t);
        if (QUANT) {  // T is a multiple of 32: a group's 16 chunks are one half-warp
            uint32_t top = 0;  // bits of |t|: NaN compares above Inf, Inf above every number
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = k + j < K ? __float_as_uint(t[j]) & 0x7FFFFFFFu : 0u;
                top = u > top ? u : top;
            }
#pragma unroll
            for (int s = 8; s > 0; s >>= 1) {
                const uint32_t o = __shfl_xor_sync(kFull, top, s);
                top = o > top ? o : top;
            }
            const float amax = __uint_as_float(top);
            float sc = amax / 448.0f;
            if (sc == 0.f) sc = 1.f;
            if (k < K) {
                if ((tid & 15) == 0) a.scale[m * a.lds + k / 128] = sc;
                // one reciprocal per group; where it could overflow (or amax is not finite), divisions
                uint32_t q[4];
                if (amax > 1e-30f && amax < 1e30f) {
                    const float inv = 448.0f / amax;
#pragma unroll
                    for (int j = 0; j < 4; ++j) q[j] = pack_e4m3(t[2 * j] * inv, t[2 * j + 1] * inv);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) q[j] = pack_e4m3(t[2 * j] / sc, t[2 * j + 1] / sc);
                }
                uint8_t *row = a.q8 + m * a.ldq;
                if (VEC) {
                    *reinterpret_cast<uint2 *>(row + k) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (k + j < K) row[k + j] = (uint8_t)(q[j >> 1] >> (8 * (j & 1)));
                }
            }
        }
    }
}

template <int C, bool VEC>
cudaError_t launch_c(const NormArgs &a, int64_t M, int threads, cudaStream_t s) {
    const dim3 grid((unsigned)M), block(threads);
    if (a.r) {
        if (a.q8) k_rmsnorm<C, VEC, true, true><<<grid, block, 0, s>>>(a);
        else k_rmsnorm<C, VEC, true, false><<<grid, block, 0, s>>>(a);
    } else {
        if (a.q8) k_rmsnorm<C, VEC, false, true><<<grid, block, 0, s>>>(a);
        else k_rmsnorm<C, VEC, false, false><<<grid, block, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <bool VEC>
cudaError_t launch_v(const NormArgs &a, int64_t M, int C, int threads, cudaStream_t s) {
    switch (C) {
        case 2: return launch_c<2, VEC>(a, M, threads, s);
        case 4: return launch_c<4, VEC>(a, M, threads, s);
        default: return launch_c<8, VEC>(a, M, threads, s);
    }
}

bool at(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

cudaError_t launch_rmsnorm(const uint16_t *x, int64_t ldx, const uint16_t *r, int64_t ldr, const uint16_t *w, float eps,
                           int64_t M, int64_t K, uint16_t *h, int64_t ldh, uint16_t *y, int64_t ldy, uint8_t *q8,
                           int64_t ldq, float *scale, int64_t lds, cudaStream_t s) {
    NormArgs a{x, r, w, ldx, ldr, h, y, ldh, ldy, q8, ldq, scale, lds, (int)K, eps, 1.0f / (float)K};
    const bool vec = K % 8 == 0 && at(x, 16) && ldx % 8 == 0 && at(w, 16) && (!r || (at(r, 16) && ldr % 8 == 0)) &&
                     (!h || (at(h, 16) && ldh % 8 == 0)) && (!y || (at(y, 16) && ldy % 8 == 0)) &&
                     (!q8 || (at(q8, 8) && ldq % 8 == 0));
    // Two chunks of 8 columns a thread, more where a CTA of 1024 would not hold the row.  K = 5120, 16383 rows
    // and one: two chunks 96.6 and 2.1 us; one chunk 99.2 and 2.4 (twice the warps to reduce over and to wait
    // for); four 97.6 and 2.3.  Rows of more than 32768 columns take eight chunks, which do not fit the 64
    // registers of a CTA of 1024 threads (250 to 580 bytes a thread are spilled): 1280 rows of 65536 with a
    // residual run at 3.9 TB/s, 2560 of 32768 with four chunks at 6.8.
    const int64_t chunks = (K + 7) / 8;
    const int C = chunks <= 2048 ? 2 : chunks <= 4096 ? 4 : 8;
    const int threads = (int)(((chunks + C - 1) / C + 31) / 32 * 32);
    return vec ? launch_v<true>(a, M, C, threads, s) : launch_v<false>(a, M, C, threads, s);
}

}  // namespace w12
