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
// position of millions is as accurate as one of ten.
//
// A CTA takes TOK tokens: its threads evaluate the TOK * rot/2 sines and
// cosines once into shared memory, then dim/16 neighbouring lanes take a head:
// each lane holds the two 16-byte chunks whose columns pair up (j and
// j + rot/2; for interleaved pairs two chunks in a row), so the rotation needs
// no exchange, and a head's mean square takes a few shuffles.  Every element is
// read once and written once.  12345 tokens of 40 + 8 + 8 heads of 128 with
// three axes, norms and the cache (354 MB) take 64.8 us, 5.5 TB/s: issue slots
// are 74% busy and HBM 60%, so what is left is the unpacking, the norms and the
// rotation, 80 instructions for 32 bytes.  (With one head ahead 71.4 us: four
// CTAs of 256 did not keep enough loads in flight.)  256 tokens take 3.5 us.
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

// One head of one token (or a value row), in one register: its place in the
// CTA's tokens, q 0 / k 1 / v 2, the head.
struct HeadAt {
    int id;
    __device__ __forceinline__ bool none() const { return id < 0; }
    __device__ __forceinline__ int t() const { return id >> 18; }
    __device__ __forceinline__ int what() const { return id >> 16 & 3; }
    __device__ __forceinline__ int h() const { return id & 0xFFFF; }
};

template <int D, int TOK, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void k_rope(const __grid_constant__ RopeArgs a) {
    constexpr int L = D / 16;  // lanes per head
    constexpr int AHEAD = TOK == 1 ? 1 : 2;
    __shared__ __align__(16) float cs[TOK][kMaxHalf], sn[TOK][kMaxHalf];
    __shared__ int64_t place[TOK];  // where a token's slot begins in the cache, -1: nowhere
    const int tid = threadIdx.x, half = a.rot / 2;
    const int64_t i0 = (int64_t)blockIdx.x * TOK;
    const int lane = tid % L;
    const int hk = a.k ? a.Hkv : 0, heads = a.Hq + hk + (a.cv ? a.Hkv : 0);
    const int lr = a.rot / 16;  // lanes whose chunks turn
    const bool turn = lane < lr;
    // the two chunks of this lane
    const int c0 = INTER ? 2 * lane : (turn ? lane : 2 * lr + 2 * (lane - lr));
    const int c1 = INTER ? 2 * lane + 1 : (turn ? lane + lr : c0 + 1);
    const int step = kRopeThreads / L;
    const uint32_t group = ((1u << L) - 1u) << (tid % 32 / L * L);  // the lanes of this head
    int t_at = 0, h_at = tid / L;  // (token, head) of the item to locate next, advanced without a division
    auto locate = [&]() {
        while (h_at >= heads) h_at -= heads, ++t_at;
        const int what = h_at < a.Hq ? 0 : h_at < a.Hq + hk ? 1 : 2;
        const HeadAt x{t_at < TOK && i0 + t_at < a.n
                           ? t_at << 18 | what << 16 | (h_at - (what == 0 ? 0 : what == 1 ? a.Hq : a.Hq + hk))
                           : -1};
        h_at += step;
        return x;
    };
    auto load = [&](const HeadAt &x, uint4 &u, uint4 &v) {
        if (x.none()) return;
        const int64_t i = i0 + x.t();
        const uint16_t *src =
            (x.what() == 0 ? a.q + i * a.ldq : x.what() == 1 ? a.k + i * a.ldk : a.v + i * a.ldv) + x.h() * D;
        u = *reinterpret_cast<const uint4 *>(src + 8 * c0);
        v = *reinterpret_cast<const uint4 *>(src + 8 * c1);
    };
    // the chunks of the next heads (AHEAD of them) are on their way while one is turned, the first while the
    // sines are evaluated
    HeadAt next[AHEAD];
    uint4 n0[AHEAD], n1[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) load(next[j] = locate(), n0[j], n1[j]);
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
    if (a.ck && tid < TOK && i0 + tid < a.n) {
        const int64_t slot = a.slots[i0 + tid];
        const int64_t page = slot / a.page_tokens;
        place[tid] = slot >= 0 && slot < a.n_slots ? page * a.page_stride + (slot - page * a.page_tokens) * a.token_stride : -1;
    }
    __syncthreads();
    while (!next[0].none()) {  // the same for every lane of the head; past the last token there is none
        const HeadAt at = next[0];
        uint4 u0 = n0[0], u1 = n1[0];
#pragma unroll
        for (int j = 0; j + 1 < AHEAD; ++j) next[j] = next[j + 1], n0[j] = n0[j + 1], n1[j] = n1[j + 1];
        load(next[AHEAD - 1] = locate(), n0[AHEAD - 1], n1[AHEAD - 1]);
        const bool is_q = at.what() == 0, is_k = at.what() == 1;
        const int64_t i = i0 + at.t();
        const int h = at.h();
        const int64_t slot = !is_q && a.ck ? place[at.t()] : -1;
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
                    const float4 *C = reinterpret_cast<const float4 *>(cs[at.t()] + 8 * lane);
                    const float4 *S = reinterpret_cast<const float4 *>(sn[at.t()] + 8 * lane);
                    const float4 ca = C[0], cb = C[1], sa = S[0], sb = S[1];
                    const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
                    const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
                    if (INTER) {  // pairs 8 lane .. 8 lane + 7 are neighbours in x, then in y
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float xa = x[2 * j], xb = x[2 * j + 1], ya = y[2 * j], yb = y[2 * j + 1];
                            x[2 * j] = fmaf(xa, c[j], -xb * s[j]);
                            x[2 * j + 1] = fmaf(xb, c[j], xa * s[j]);
                            y[2 * j] = fmaf(ya, c[j + 4], -yb * s[j + 4]);
                            y[2 * j + 1] = fmaf(yb, c[j + 4], ya * s[j + 4]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float xa = x[j], xb = y[j];
                            x[j] = fmaf(xa, c[j], -xb * s[j]);
                            y[j] = fmaf(xb, c[j], xa * s[j]);
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
        if (slot >= 0) {
            uint16_t *c = (is_k ? a.ck : a.cv) + slot + h * a.head_stride;
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
    // Few tokens: one CTA each, for the latency; many: four, so that the CTA's threads all have a sine to
    // evaluate and two heads are on their way.  40 + 8 heads of 128: 256 tokens 3.8 us with one, 6.2 with four;
    // 608 5.1 and 6.7; 1216 7.9 and 7.7; 12345 76 and 60.5.
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
