// Rotary positions on queries and keys, with one position per axis for image
// and video tokens, optional per-head norms, and the write of keys and values
// into a paged cache: what stands between the QKV GEMM and the attention of a
// decoder layer (SpecPilot, arXiv 2611.02501, names the layers of a verify
// pass only; the published rotary embedding, Su et al. 2021).
//
//     (x_a, x_b) -> (x_a cos - x_b sin, x_b cos + x_a sin),  angle = pos_axis(j) inv_freq_j
//
// The angle is kept as a fraction of a turn: pos * (inv_freq / 2 pi) is formed
// exactly (product and its rounding error by FMA, 1 / 2 pi in two floats), its
// whole turns dropped, and CUDA's sincospif evaluated on what is left, so a
// position of a million is as accurate as one of ten.
//
// A CTA takes TOK tokens: its threads evaluate the TOK * rot/2 sines and
// cosines once into shared memory, then dim/16 neighbouring lanes take a head:
// each lane holds the two 16-byte chunks whose columns pair up (j and
// j + rot/2; for interleaved pairs two chunks in a row), so the rotation needs
// no exchange, and a head's mean square takes a few shuffles.  Every element is
// read once and written once: HBM bound for many tokens.
#include <cstdint>
#include <cuda_runtime.h>

#include "w12_device.cuh"
#include "w12_internal.h"

namespace w12 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxHalf = 128;  // rot / 2 <= dim / 2

struct RopeArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv;
    uint16_t *qo, *ko;
    int64_t ldqo, ldko;
    int64_t n;
    int Hq, Hkv, rot;  // Hq = 0 without q, and no k heads without k
    const int32_t *pos;
    int64_t ld_pos;
    const float *inv_freq;
    const uint16_t *qn, *kn;
    float eps;
    uint16_t *ck, *cv;  // cache (null: not written)
    const int64_t *slots;
    int64_t n_slots;
    int32_t page_tokens;
    int64_t page_stride, token_stride, head_stride;
    uint8_t axis[kMaxHalf];
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// p * f / (2 pi) without its whole turns, |p| < 2^24
__device__ __forceinline__ float turns(float p, float fh, float fl) {
    const float t = p * fh;
    const float e = fmaf(p, fh, -t);
    return (t - rintf(t)) + fmaf(p, fl, e);
}

__device__ __forceinline__ void unpack8(uint4 u, float x[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float x[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

template <int D, int TOK, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void k_rope(const __grid_constant__ RopeArgs a) {
    constexpr int L = D / 16;  // lanes per head
    __shared__ __align__(16) float cs[TOK][kMaxHalf], sn[TOK][kMaxHalf];
    const int tid = threadIdx.x, half = a.rot / 2;
    const int64_t i0 = (int64_t)blockIdx.x * TOK;
    for (int x = tid; x < TOK * half; x += kRopeThreads) {
        const int t = TOK == 1 ? 0 : x / half, j = x - t * half;
        if (i0 + t < a.n) {
            const int32_t p = a.pos[a.axis[j] * a.ld_pos + i0 + t];
            // 1 / (2 pi) = ch + cl; the frequency in turns per position, in two floats
            const float ch = 0.15915494309189535f, cl = (float)(0.15915494309189535 - (double)0.15915494309189535f);
            const float f = a.inv_freq[j];
            const float fh = f * ch, fl = fmaf(f, cl, fmaf(f, ch, -fh));
            // a position in two parts that FP32 holds exactly
            const float r = turns((float)(p & ~4095), fh, fl) + turns((float)(p & 4095), fh, fl);
            sincospif(2.0f * r, &sn[t][j], &cs[t][j]);
        }
    }
    __syncthreads();
    const int lane = tid % L;
    const int heads = a.Hq + (a.k ? a.Hkv : 0) + (a.cv ? a.Hkv : 0);
    const int lr = a.rot / 16;  // lanes whose chunks turn
    const bool turn = lane < lr;
    // the two chunks of this lane
    const int c0 = INTER ? 2 * lane : (turn ? lane : 2 * lr + 2 * (lane - lr));
    const int c1 = INTER ? 2 * lane + 1 : (turn ? lane + lr : c0 + 1);
    const int items = TOK * heads, step = kRopeThreads / L;
    const uint32_t group = ((1u << L) - 1u) << (tid % 32 / L * L);  // the lanes of this head
    for (int it = tid / L; it < items; it += step) {
        const int t = TOK == 1 ? 0 : it / heads, hd = it - t * heads;
        const int64_t i = i0 + t;
        if (i >= a.n) break;  // the same for every lane of the head
        const bool is_q = hd < a.Hq, is_k = !is_q && hd < a.Hq + (a.k ? a.Hkv : 0);
        const int h = is_q ? hd : is_k ? hd - a.Hq : hd - a.Hq - (a.k ? a.Hkv : 0);
        const uint16_t *src = (is_q ? a.q + i * a.ldq : is_k ? a.k + i * a.ldk : a.v + i * a.ldv) + h * D;
        uint4 u0 = *reinterpret_cast<const uint4 *>(src + 8 * c0);
        uint4 u1 = *reinterpret_cast<const uint4 *>(src + 8 * c1);
        const int64_t slot = !is_q && a.ck ? a.slots[i] : -1;
        if (is_q || is_k) {
            const uint16_t *nw = is_q ? a.qn : a.kn;
            const bool norm = nw != nullptr;
            if (norm || turn) {
                float x[8], y[8];
                unpack8(u0, x);
                unpack8(u1, y);
                if (norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
                    for (int s = L / 2; s > 0; s >>= 1) ss += __shfl_xor_sync(group, ss, s);
                    const float rstd = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
                    float wx[8], wy[8];
                    unpack8(*reinterpret_cast<const uint4 *>(nw + 8 * c0), wx);
                    unpack8(*reinterpret_cast<const uint4 *>(nw + 8 * c1), wy);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[j] *= rstd * wx[j];
                        y[j] *= rstd * wy[j];
                    }
                }
                if (turn) {
                    const float *C = cs[t], *S = sn[t];
                    if (INTER) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float ca = C[8 * lane + j], sa = S[8 * lane + j];
                            const float cb = C[8 * lane + 4 + j], sb = S[8 * lane + 4 + j];
                            const float xa = x[2 * j], xb = x[2 * j + 1], ya = y[2 * j], yb = y[2 * j + 1];
                            x[2 * j] = fmaf(xa, ca, -xb * sa);
                            x[2 * j + 1] = fmaf(xb, ca, xa * sa);
                            y[2 * j] = fmaf(ya, cb, -yb * sb);
                            y[2 * j + 1] = fmaf(yb, cb, ya * sb);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float c = C[8 * lane + j], s = S[8 * lane + j];
                            const float xa = x[j], xb = y[j];
                            x[j] = fmaf(xa, c, -xb * s);
                            y[j] = fmaf(xb, c, xa * s);
                        }
                    }
                }
                u0 = pack8(x);
                u1 = pack8(y);
            }
        }
        uint16_t *dst = is_q ? a.qo + i * a.ldqo + h * D : (is_k && a.ko) ? a.ko + i * a.ldko + h * D : nullptr;
        if (dst) {
            *reinterpret_cast<uint4 *>(dst + 8 * c0) = u0;
            *reinterpret_cast<uint4 *>(dst + 8 * c1) = u1;
        }
        if (slot >= 0 && slot < a.n_slots) {
            const int64_t page = slot / a.page_tokens, tok = slot - page * a.page_tokens;
            uint16_t *c = (is_k ? a.ck : a.cv) + page * a.page_stride + tok * a.token_stride + h * a.head_stride;
            *reinterpret_cast<uint4 *>(c + 8 * c0) = u0;
            *reinterpret_cast<uint4 *>(c + 8 * c1) = u1;
        }
    }
}

template <int D, int TOK>
cudaError_t launch_t(const RopeArgs &a, bool inter, cudaStream_t s) {
    const unsigned grid = (unsigned)((a.n + TOK - 1) / TOK);
    if (inter) k_rope<D, TOK, true><<<grid, kRopeThreads, 0, s>>>(a);
    else k_rope<D, TOK, false><<<grid, kRopeThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const RopeArgs &a, bool inter, cudaStream_t s) {
    // few tokens: one CTA each, for the latency; many: four, so that the
    // CTA's threads all have a sine to evaluate
    return a.n <= 4 * W12_PLAN_SMS ? launch_t<D, 1>(a, inter, s) : launch_t<D, 4>(a, inter, s);
}

}  // namespace

cudaError_t launch_rope(const w12_rope_args &r, cudaStream_t s) {
    RopeArgs a{};
    a.q = r.q, a.k = r.k, a.v = r.v;
    a.ldq = r.ldq, a.ldk = r.ldk, a.ldv = r.ldv;
    a.qo = r.q_out, a.ko = r.k_out;
    a.ldqo = r.ldqo, a.ldko = r.ldko;
    a.n = r.n;
    a.Hq = r.q ? r.q_heads : 0;
    a.Hkv = r.kv_heads;
    a.rot = r.rot;
    a.pos = r.pos;
    a.ld_pos = r.ld_pos;
    a.inv_freq = r.inv_freq;
    a.qn = r.q_norm, a.kn = r.k_norm;
    a.eps = r.eps;
    if (r.slots) {
        const w12_kv_cache &c = *r.cache;
        a.ck = c.k, a.cv = c.v;
        a.slots = r.slots;
        a.n_slots = c.pages * c.page_tokens;
        a.page_tokens = c.page_tokens;
        a.page_stride = c.page_stride, a.token_stride = c.token_stride, a.head_stride = c.head_stride;
    }
    if (r.axis)
        for (int j = 0; j < r.rot / 2; ++j) a.axis[j] = r.axis[j];
    const bool inter = r.interleaved != 0;
    return r.dim == 64 ? launch_d<64>(a, inter, s) : r.dim == 128 ? launch_d<128>(a, inter, s) : launch_d<256>(a, inter, s);
}

}  // namespace w12
