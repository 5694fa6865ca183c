// The gated delta rule over long sequences: chunks of 64 tokens, the products on
// the tensor cores (tcgen05).
//
// Within a chunk that begins with the state S0, with gamma_t the product of
// alpha up to t, G_tj that of alpha after j up to t, and f_t the coefficient
// vectors (S = gamma S0 + sum G f k^T, see w12_gdn.cu),
//     (I + A) F = diag(beta) X,   X = V - diag(gamma) K S0^T,   A_tj = beta_t G_tj k_t.k_j (j < t)
//     O = diag(gamma) Q S0^T + M F,   M_tj = G_tj q_t.k_j (j <= t)
//     S = gamma_C S0 + (G_C. F)^T K
// With T = (I + A)^-1 diag(beta), which does not depend on S0, this is two
// products with X: G_C. F = (diag(G_C.) T) X, and M F = (M T) X.  One kernel makes
// diag(G_C.) T and M T of all chunks, another goes through a head's chunks.
//
// FP32 operands of tensor-core products are sums of two BF16 numbers (the
// nearest, and the nearest to what remains), which leaves 2^-18 of them; without the
// second part an output of 16 bits would come out 1.4 times as far off as its
// rounding, and the states, which are kept in 32 bits, 2^-9.  As it is the
// states of independent keys are 6e-6 to 8e-6 off their norm (token by token 3e-7), with
// equal keys 5e-5; where that would not hold a head is left to k_scan_redo (see kMaxColumn).
//
// One prompt of 8191 tokens, 32 heads of 128 over 16: 361 us (68 and 293), where
// its bytes take 31; four of 8192 548 us (about 240 and 305).  Token by token the
// first takes 5.4 ms.
#include <cstdint>
#include <cuda_runtime.h>

#include "w12_gdn_scan.cuh"
#include "w12_stream.cuh"
#include "w12_tc.cuh"
#include "w12_tmap.cuh"

namespace w12 {
namespace {

using namespace tc;

constexpr int C = 64;                            // tokens of a chunk
constexpr uint32_t kTile = C * 128;              // 64 rows of 64 BF16, swizzled
constexpr uint32_t kImageBytes = 4 * kTile;      // G T high, M T high, G T low, M T low parts

__host__ __device__ inline int64_t slot_of(int64_t start, int64_t r) { return start / C + r; }  // r's first chunk
inline int64_t slots_of(int64_t n, int64_t R) { return n / C + R; }
inline size_t cond_bytes(size_t units) { return (2 * units + 3) / 4 * 4; }
// The request that a slot is searched for: the last whose first slot is not behind it.  (Without `start` there is one.)
__device__ __forceinline__ int request_of(const ScanArgs &a, int64_t slot) {
    int lo = 0, hi = a.R - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (slot_of(a.start[mid], mid) <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
// Whether that search leads to r from all slots of [s0, s1]: where `start` descends somewhere it may not, and their
// images are not r's.  The places that it looks at are those on the way to r, whatever is there.
__device__ __forceinline__ bool found(const ScanArgs &a, int r, int64_t s0, int64_t s1) {
    bool ok = true;
    int lo = 0, hi = a.R - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int64_t s = slot_of(a.start[mid], mid);
        if (mid <= r) ok &= s <= s0, lo = mid;
        else ok &= s > s1, hi = mid - 1;
    }
    return ok;
}

// Two FP32 values as BF16 pairs: the nearest, and the nearest to what remains (lower column in the low half).  (The
// conversions and the unpacking take two cycles of a warp each; packed FP32 operations did not help: 8191 tokens 382 us
// with them, then 360 without.)
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
    hi = pack2(x.x, x.y);
    lo = pack2(x.x - __uint_as_float(hi << 16), x.y - __uint_as_float(hi & 0xFFFF0000u));
}

// ---------------------------------------------------------------------------
// T and M T of every chunk and head, as the tiles that k_scan_main's products read.  A CTA takes a chunk of a key head
// and its value heads one after the other.
//
// (I + A)^-1 by blocks of 16: the four diagonal blocks by substitution (a lane a column); then warp J finds the rest
// of the J-th block column on the tensor cores, transposed, so that one product's result is the next one's operand
// in the same registers, and the tiles lie transposed (a row a token j, columns the tokens t):
//     U_i = (T_iJ)^T = -(sum_{J <= k < i} U_k A_ik^T) T_ii^T,    ((M T)_IJ)^T = sum_{J <= s <= I} U_s M_Is^T.
// Operands are sums of two BF16 numbers, products of the two low ones are left out (2^-16 of a term).  The columns of
// a result's two 8-wide tiles stand for the tokens 4 q, 4 q + 1 and 4 q + 2, 4 q + 3 (q: the lane's place in its
// four), so that a lane's four values are neighbours; a position's token is tok(), and A, M and T are stored by
// position.
//
// What bounds it: four CTAs of four warps a multiprocessor wait for loads, for
// one another at barriers and for their own results; 37% of the issue slots are
// used.  Of 76 us for 8191 tokens 20 were loads, 7 K K^T and Q K^T, 18 decays and the
// conversion of A and M, 12 the diagonal blocks, 13 the block columns and 6 their
// stores (loads by cp.async, with the decays under them, took 6 off; A and M as the
// blocks that are there instead of squares, 46 KB of shared memory instead of 53, 4
// more: four prompts of 8192 553 us before, 539 after, on one GPU).  Two heads in every
// phase, three CTAs a multiprocessor, took 430 us instead of 422 for 16 x 1999 tokens;
// the diagonal blocks of two heads in one phase 447.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 128;
// Conditioning: a head with a chunk in which a column of a diagonal block's inverse has a larger sum of absolute values is
// computed token by token (k_scan_redo).  Keys of norm 1, beta <= 1 and alpha <= 1 never come to that: what a token writes is
// only taken down by the later ones, the squares of a column's entries below the diagonal add up to 1 at most, their absolute
// values to sqrt(15), 4.9 with the diagonal.  Where beta |k|^2 stays near 2 and the keys are alike, every write
// flips what is there, nothing decays, a column's sum goes to 31, and products of operands of 16 bits leave nothing
// of the states (heads of 64, 2000 equal keys of beta = 2: 36% off, by token 4e-6).  Below the limit the states were 2e-4
// off at most.  The whole chunk's columns would say a little more (keys that come back every 8 tokens, beta = 2 and no decay:
// 4e-4 in an emulation) and cost 4 us of 8191 tokens more than this, which with the words it writes, their reading and
// k_scan_redo's launch costs 6.
constexpr float kMaxColumn = 6.f;
constexpr int kGroup = 2;  // value heads whose decays are taken together, a warp each
constexpr int kPitch = 24;  // of a 16 x 16 block of BF16: its rows start in eight different groups of banks

struct PrepHead {  // of a value head; l = sums of log2 alpha
    float lh[C], ll[C];  // l: its multiple of 2^-8, and the rest
    float from_ref[C];   // 2^(l_t - l at the end of the 16 tokens before t's), times beta
    float from_ref_m[C]; // the same without beta
    float to_ref[3][C];  // 2^(l at the end of the first 16, 32, 48 tokens - l_j)
    float beta[C], bad[C], to_end[C];
};
using PrepBlock = uint16_t[16][kPitch];
__host__ __device__ constexpr int blk_a(int i, int k) { return i * (i - 1) / 2 + k; }  // k < i
__host__ __device__ constexpr int blk_m(int i, int k) { return i * (i + 1) / 2 + k; }  // k <= i
struct PrepBlocks {  // of A and M, in high and low parts
    PrepBlock A[2][6], M[2][10];
};
union PrepDiag {  // a diagonal block of A, transposed; then of T, transposed, high and low parts
    float At[16][20];
    PrepBlock T[2];
};
template <int D>
struct PrepTiles {
    uint16_t k[C][D + 8], q[C][D + 8];
};
template <int D>
struct PrepSmem {
    union {
        PrepTiles<D> in;  // read before A and M are written
        PrepBlocks b;
    };
    PrepDiag diag[4];
    PrepHead head[kGroup];
};

__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t r[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_addr(p))
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t r[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_addr(p))
                 : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Frag {  // a 16 x 16 operand in two parts
    uint32_t hi[4], lo[4];
};
__device__ __forceinline__ Frag frag_of(const float c[2][4]) {  // of a result
    Frag f;
    split2(make_float2(c[0][0], c[0][1]), f.hi[0], f.lo[0]);
    split2(make_float2(c[0][2], c[0][3]), f.hi[1], f.lo[1]);
    split2(make_float2(c[1][0], c[1][1]), f.hi[2], f.lo[2]);
    split2(make_float2(c[1][2], c[1][3]), f.hi[3], f.lo[3]);
    return f;
}
__device__ __forceinline__ int tok(int pos) { return 4 * ((pos & 7) >> 1) + (pos & 1) + 2 * (pos >> 3); }
// acc += X B; b: this lane's address in the 16 x 16 matrix B^T (trans: B), its low part `gap` elements on
template <bool TRANS>
__device__ __forceinline__ void mul(float acc[2][4], const Frag &x, const uint16_t *b, int gap) {
    uint32_t h[4], l[4];
    if (TRANS) ldsm4_t(h, b), ldsm4_t(l, b + gap);
    else ldsm4(h, b), ldsm4(l, b + gap);
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        mma16816(acc[nt], x.hi, h[2 * nt], h[2 * nt + 1]);
        mma16816(acc[nt], x.lo, h[2 * nt], h[2 * nt + 1]);
        mma16816(acc[nt], x.hi, l[2 * nt], l[2 * nt + 1]);
    }
}
// Where this lane's four values of row r go in 16 columns of a tile: at put_at(r) ^ 32 * (which 16).
__device__ __forceinline__ uint32_t put_at(int r, int q4) {
    return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + (((q4 >> 1) ^ (r & 7)) << 4) + 8 * (q4 & 1));
}
// x, y (and their low parts one tile, or `gap` bytes, on): a row's values of tokens 4 q4 .. 4 q4 + 3
__device__ __forceinline__ void put4(uint8_t *at, uint32_t gap, float2 x, float2 y) {
    uint2 h, l;
    split2(x, h.x, l.x);
    split2(y, h.y, l.y);
    *reinterpret_cast<uint2 *>(at) = h;
    *reinterpret_cast<uint2 *>(at + gap) = l;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) { return fma2(x, y, make_float2(0.f, 0.f)); }

// The sums of log2 alpha of a head's 64 tokens, by a warp.  As whole numbers (2^-40): a decay of 0 (2^-200 here)
// leaves no error in the differences behind it.
__device__ __forceinline__ void prep_decays(const ScanArgs &a, PrepHead &p, int h, int row0, int m, int lane, float *gamma) {
    long long s[2];
    bool bad[2];
    float beta[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int t = 2 * lane + u;
        const float al = t < m ? a.alpha[(int64_t)(row0 + t) * a.H + h] : 1.f;
        beta[u] = t < m ? a.beta[(int64_t)(row0 + t) * a.H + h] : 0.f;
        bad[u] = !(al >= 0.f && al < INFINITY);
        s[u] = __float2ll_rn(fmaxf(log2f(bad[u] ? 1.f : al), -200.f) * 0x1p40f);
    }
    s[1] += s[0];
    bad[1] |= bad[0];
    long long sum = s[1];
    int any = bad[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(kFull, sum, d);
        const int ob = __shfl_up_sync(kFull, any, d);
        if (lane >= d) sum += o, any |= ob;
    }
    const long long before = sum - s[1], all = __shfl_sync(kFull, sum, 31);
    const bool bad_before = __shfl_up_sync(kFull, any, 1) && lane > 0, bad_all = __shfl_sync(kFull, any, 31) != 0;
    const float nan = __int_as_float(0x7FC00000);
    const long long ref_up = __shfl_sync(kFull, sum, ((lane & 24) + 31) & 31), ref = lane < 8 ? 0 : ref_up;  // end of the 16 before
    long long refs[3];
#pragma unroll
    for (int b = 0; b < 3; ++b) refs[b] = __shfl_sync(kFull, sum, 8 * b + 7);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int t = 2 * lane + u;
        const long long x = before + s[u], hi = (x + (1LL << 31)) >> 32;
        const float b = bad_before || bad[u] ? nan : 0.f;
        p.lh[t] = (float)hi * 0x1p-8f;
        p.ll[t] = (float)(x - (hi << 32)) * 0x1p-40f;
        p.beta[t] = beta[u];
        p.bad[t] = b;
        const float e = exp2_fast((float)(x - ref) * 0x1p-40f) + b;
        p.from_ref_m[t] = e;
        p.from_ref[t] = e * beta[u];
#pragma unroll
        for (int k = 0; k < 3; ++k) p.to_ref[k][t] = t < 16 * (k + 1) ? exp2_fast((float)(refs[k] - x) * 0x1p-40f) : 0.f;
        p.to_end[t] = t < m ? exp2_fast((float)(all - x) * 0x1p-40f) + (bad_all ? nan : 0.f) : 0.f;
        gamma[t] = exp2_fast((float)x * 0x1p-40f) + b;
    }
}

template <int D>
__global__ __launch_bounds__(kPrepThreads, 4) void k_scan_prep(const __grid_constant__ ScanArgs a) {
    extern __shared__ __align__(16) uint8_t smem_prep[];
    PrepSmem<D> &sm = *reinterpret_cast<PrepSmem<D> *>(smem_prep);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
    const int key_heads = a.H / a.per_key;
    grid_dep_launch();  // k_scan_main's start and its first loads run under the end of this
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.redo[0] = 0;
    if (blockIdx.y == (unsigned)key_heads) {  // one CTA more a column of the grid: only the first is of use
        if (blockIdx.x == 0 && a.status) check_all(a);
        return;
    }
    const int slot = blockIdx.x, hk = blockIdx.y;
    const int r = request_of(a, slot);
    const Seq seq = seq_of(a, r);
    const int64_t c = slot - slot_of(seq.first, r);
    if (!seq.ok || c < 0 || c * C >= seq.len) return;
    const int row0 = seq.first + (int)c * C, m = min(C, seq.len - (int)c * C);
    // 64 rows of a key head, zeros from `rows` on
    auto tile = [&](uint16_t (*to)[D + 8], const uint16_t *from, int64_t ld, int64_t row, int rows) {
#pragma unroll
        for (int it = 0; it < C * (D / 8) / kPrepThreads; ++it) {
            const int x = tid + it * kPrepThreads, t = x / (D / 8), ch = x % (D / 8);
            const uint16_t *src = t < rows ? from + (row + t) * ld + hk * D + 8 * ch : from;  // (0 bytes of it: zeros)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(&to[t][8 * ch])), "l"(src),
                         "r"(t < rows ? 16 : 0)
                         : "memory");
        }
    };
    // this lane's row and columns of a 16 x 16 operand: the left one, the right one by rows of its transpose, the same
    // from the matrix itself
    const int la = lane & 15, lac = (lane >> 4) * 8, lb = tok((lane & 7) + ((lane >> 4) << 3)), lbc = ((lane >> 3) & 1) * 8;
    const int lt = tok(lane & 15), ltc = (lane >> 4) * 8;
    auto decays = [&](int h0) {
        if (warp < kGroup && h0 + warp < a.per_key) {
            const int h = hk * a.per_key + h0 + warp;
            prep_decays(a, sm.head[warp], h, row0, m, lane, a.gamma + ((int64_t)slot * a.H + h) * C);
        }
    };
    tile(sm.in.k, a.k, a.ldk, row0, m);
    if (a.q) tile(sm.in.q, a.q, a.ldq, row0, m);
    decays(0);  // while they come
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // K K^T and Q K^T, the 16 x 16 blocks on and below the diagonal: (bi, bj) of warp w's n-th
    auto block_of = [&](int n, int &bi, int &bj) {  // 2, 2, 3, 3 of them
        const int at = warp == 0 ? n : warp == 1 ? 2 + n : warp == 2 ? 4 + n : 7 + n;
        bi = at < 1 ? 0 : at < 3 ? 1 : at < 6 ? 2 : 3;
        bj = at - bi * (bi + 1) / 2;
        return n < (warp < 2 ? 2 : 3);
    };
    float kk_[3][2][4] = {}, qk_[3][2][4] = {};
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        int bi, bj;
        if (!block_of(n, bi, bj)) continue;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t f[4], b[4];
            ldsm4(b, &sm.in.k[16 * bj + lb][16 * kk + lbc]);
            ldsm4(f, &sm.in.k[16 * bi + la][16 * kk + lac]);
            mma16816(kk_[n][0], f, b[0], b[1]);
            mma16816(kk_[n][1], f, b[2], b[3]);
            if (a.q) {
                ldsm4(f, &sm.in.q[16 * bi + la][16 * kk + lac]);
                mma16816(qk_[n][0], f, b[0], b[1]);
                mma16816(qk_[n][1], f, b[2], b[3]);
            }
        }
    }
    for (int h0 = 0; h0 < a.per_key; h0 += kGroup) {
        if (h0 > 0) {
            __syncthreads();  // the heads before are no longer read
            decays(h0);
        }
        for (int hn = 0; hn < kGroup && h0 + hn < a.per_key; ++hn) {
            const PrepHead &p = sm.head[hn];
            const int h = hk * a.per_key + h0 + hn;
            uint8_t *img = a.image + ((int64_t)slot * a.H + h) * kImageBytes;
            __syncthreads();  // the decays are there; the tiles, or A, M and T of the head before, are no longer read
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                int bi, bj;
                if (!block_of(n, bi, bj)) continue;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int j = 16 * bj + 4 * q4 + 2 * nt, pos = 8 * nt + 2 * q4;
                    float x[2][2], y[2][2];
                    if (bi == bj) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int t = 16 * bi + g + 8 * u;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float G = exp2_fast((p.lh[t] - p.lh[j + e]) + (p.ll[t] - p.ll[j + e])) + p.bad[t];
                                x[u][e] = j + e < t ? p.beta[t] * G * kk_[n][nt][2 * u + e] : 0.f;
                                y[u][e] = j + e <= t ? G * qk_[n][nt][2 * u + e] : 0.f;
                                sm.diag[bi].At[j + e - 16 * bj][t - 16 * bi] = x[u][e];
                            }
                        }
                    } else {  // the product of two decays, each at most 1
                        const float2 f = *reinterpret_cast<const float2 *>(&p.to_ref[bi - 1][j]);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int t = 16 * bi + g + 8 * u;
                            const float e = p.from_ref[t], em = p.from_ref_m[t];
                            x[u][0] = kk_[n][nt][2 * u] * f.x * e, x[u][1] = kk_[n][nt][2 * u + 1] * f.y * e;
                            y[u][0] = qk_[n][nt][2 * u] * f.x * em, y[u][1] = qk_[n][nt][2 * u + 1] * f.y * em;
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t h2, l2;
                        if (bi != bj) {
                            split2(make_float2(x[u][0], x[u][1]), h2, l2);
                            *reinterpret_cast<uint32_t *>(&sm.b.A[0][blk_a(bi, bj)][g + 8 * u][pos]) = h2;
                            *reinterpret_cast<uint32_t *>(&sm.b.A[1][blk_a(bi, bj)][g + 8 * u][pos]) = l2;
                        }
                        split2(make_float2(y[u][0], y[u][1]), h2, l2);
                        *reinterpret_cast<uint32_t *>(&sm.b.M[0][blk_m(bi, bj)][g + 8 * u][pos]) = h2;
                        *reinterpret_cast<uint32_t *>(&sm.b.M[1][blk_m(bi, bj)][g + 8 * u][pos]) = l2;
                    }
                }
            }
            __syncthreads();
            if (warp < 2) {  // two diagonal blocks: column `lane & 15` of (I + A)^-1
                const int col = lane & 15;
                PrepDiag &d = sm.diag[2 * warp + (lane >> 4)];
                float x[16];
#pragma unroll
                for (int t = 0; t < 16; ++t) x[t] = t == col ? 1.f : 0.f;
#pragma unroll
                for (int s = 0; s < 15; ++s) {
                    const float xs = x[s];
                    float w[16];
#pragma unroll
                    for (int t4 = (s + 1) / 4; t4 < 4; ++t4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&d.At[s][4 * t4]);
                        w[4 * t4] = f.x, w[4 * t4 + 1] = f.y, w[4 * t4 + 2] = f.z, w[4 * t4 + 3] = f.w;
                    }
#pragma unroll
                    for (int t = s + 1; t < 16; ++t) x[t] = fmaf(-w[t], xs, x[t]);
                }
                float sum[4] = {};
#pragma unroll
                for (int t = 0; t < 16; ++t) sum[t & 3] += fabsf(x[t]);
                const bool large = __any_sync(kFull, !((sum[0] + sum[1]) + (sum[2] + sum[3]) <= kMaxColumn));  // (NaN too)
                if (lane == 0) a.cond[((int64_t)slot * a.H + h) * 2 + warp] = large;
                uint32_t h2[8], l2[8];  // by position: 0 1 4 5 8 9 12 13, 2 3 6 7 ...
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int t = 4 * (k & 3) + 2 * (k >> 2);
                    split2(make_float2(x[t], x[t + 1]), h2[k], l2[k]);
                }
                __syncwarp();  // T goes where A was
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    *reinterpret_cast<uint4 *>(&d.T[0][col][8 * k]) = make_uint4(h2[4 * k], h2[4 * k + 1], h2[4 * k + 2], h2[4 * k + 3]);
                    *reinterpret_cast<uint4 *>(&d.T[1][col][8 * k]) = make_uint4(l2[4 * k], l2[4 * k + 1], l2[4 * k + 2], l2[4 * k + 3]);
                }
            } else {  // meanwhile: zeros above the diagonal, rows j of tokens before their block
                const int x = tid - 64, rr = x & 15;
                uint8_t *to = img + (x >> 4) * kTile + (rr >> 3) * 1024 + (rr & 7) * 128;
#pragma unroll
                for (int b = 1; b < 4; ++b)
#pragma unroll
                    for (int ch = 0; ch < 2 * b; ++ch)
                        *reinterpret_cast<uint4 *>(to + b * 2048 + ((ch ^ (rr & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            }
            __syncthreads();
            // block column J = warp of T and of M T
            const int J = warp;
            const float be0 = p.beta[16 * J + g], be1 = p.beta[16 * J + g + 8];
            const uint32_t at0 = put_at(16 * J + g, q4);
            // a transposed 16 x 16 block: rows 16 J .. of a tile and its low part, columns (tokens) 16 I ..
            auto put = [&](uint8_t *tile, int I, const float x[2][4], float4 s) {
                uint8_t *to = tile + (at0 ^ 32 * I);
                const float2 s0 = make_float2(s.x, s.y), s1 = make_float2(s.z, s.w);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float2 be = u ? make_float2(be1, be1) : make_float2(be0, be0);
                    put4(to + 1024 * u, 2 * kTile, mul2(make_float2(x[0][2 * u], x[0][2 * u + 1]), mul2(be, s0)),
                         mul2(make_float2(x[1][2 * u], x[1][2 * u + 1]), mul2(be, s1)));
                }
            };
            auto ends = [&](int I) { return *reinterpret_cast<const float4 *>(&p.to_end[16 * I + 4 * q4]); };
            Frag U[4];
            {
                ldsm4(U[0].hi, &sm.diag[J].T[0][la][lac]);
                ldsm4(U[0].lo, &sm.diag[J].T[1][la][lac]);
                float own[2][4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    own[x >> 1][2 * (x & 1)] = __uint_as_float(U[0].hi[x] << 16) + __uint_as_float(U[0].lo[x] << 16);
                    own[x >> 1][2 * (x & 1) + 1] = __uint_as_float(U[0].hi[x] & 0xFFFF0000u) + __uint_as_float(U[0].lo[x] & 0xFFFF0000u);
                }
                put(img, J, own, ends(J));
            }
#pragma unroll
            for (int d = 1; d < 4; ++d) {
                if (J + d > 3) break;
                const int i = J + d;
                float w[2][4] = {}, y[2][4] = {};
#pragma unroll
                for (int e = 0; e < d; ++e) mul<false>(w, U[e], &sm.b.A[0][blk_a(i, J + e)][lb][lbc], 6 * 16 * kPitch);
                mul<true>(y, frag_of(w), &sm.diag[i].T[0][lt][ltc], 16 * kPitch);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[nt][e] = -y[nt][e];
                U[d] = frag_of(y);
                put(img, i, y, ends(i));
            }
            if (a.q) {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    if (J + d > 3) break;
                    const int i = J + d;
                    float y[2][4] = {};
#pragma unroll
                    for (int e = 0; e <= d; ++e) mul<false>(y, U[e], &sm.b.M[0][blk_m(i, J + e)][lb][lbc], 10 * 16 * kPitch);
                    const int t = 16 * i + 4 * q4;
                    put(img + kTile, i, y, make_float4(t < m ? 1.f : 0.f, t + 1 < m ? 1.f : 0.f, t + 2 < m ? 1.f : 0.f, t + 3 < m ? 1.f : 0.f));
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The chunks of a (request, head), one after the other: a CTA.  The products
// are taken transposed: a TMEM lane is a row of S, the tokens are columns, so
// that a thread turns what one product left in its lane into the next one's
// operand in the same lane: S (in registers, FP32) as BF16 parts -> K S^T and Q S^T
// -> X -> F' -> the increment of S, which is added in registers.  Eight warps do
// that, half a row each; four write the outputs, one issues the products (in
// halves, as operands come), one the copies.
//
// What bounds it: a chunk is a chain of 4400 cycles: S as BF16 parts 600, K S^T
// 700, X 750, F' 600, its parts 350, the increment 650, its sum 250, and six
// hand-overs.  The tensor cores are busy 53% of it; conversions and unpacking are
// half-rate instructions, and fill the stages between products.  Sixteen warps
// instead of eight took as long (313 us and 305 for 8191 tokens), halves of X and
// F' handed over as they come longer (379 us with the inverses, without 360).
// ---------------------------------------------------------------------------
constexpr int kStateWarps = 8, kMmaWarp = 12, kLoadWarp = 13, kCondWarp = 14;  // outputs: 8 .. 11
constexpr int kMainThreads = 512;
constexpr int kStages = 2;
constexpr uint32_t kTmemCols = 512;
// Columns: S as BF16 high and low parts, Q S^T, K S^T and then X in its place, F' as FP32 and then as BF16 parts, M T X,
// the state's increment.  X and F' take the columns that their own warp has just read: 32 tokens' 16 columns of high
// parts, then 16 of low ones.
constexpr uint32_t kColSH = 0, kColSL = 64, kColQ = 128, kColX = 192, kColF = 256, kColO = 320, kColU = 384;
__device__ __forceinline__ uint32_t part_col(int kk) { return (kk >> 1) * 32 + (kk & 1) * 8; }  // of the kk-th 16 tokens

template <int D>
struct MainSizes {
    static constexpr int kHalves = D / 64;
    static constexpr uint32_t kKQ = 2 * kHalves * kTile;  // K, Q of the first 64 columns, then of the others
    static constexpr uint32_t kV = kHalves * kTile;
    static constexpr uint32_t kStage = kKQ + kV + kImageBytes;
};
template <int D>
constexpr size_t main_smem_bytes() {
    return 1024 + kStages * ((size_t)MainSizes<D>::kStage + C * 4) + 8 * (2 * kStages + 12) + 32;
}

struct MainMaps {
    CUtensorMap k, q, v;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// A wait gave up: what there is of this CTA's head is not its result.
template <int D>
__device__ __noinline__ void all_nan(const ScanArgs &a) {
    const float nan = __int_as_float(0x7FC00000);
    const int r = (int)blockIdx.x / a.H, h = (int)blockIdx.x - r * a.H;
    const Seq seq = seq_of(a, r);
    float4 *S = reinterpret_cast<float4 *>(a.S_out + (int64_t)blockIdx.x * D * D);
    for (int x = threadIdx.x; x < D * D / 4; x += kMainThreads) S[x] = make_float4(nan, nan, nan, nan);
    for (int64_t x = threadIdx.x; a.o && x < (int64_t)seq.len * D; x += kMainThreads) {
        const int64_t to = (seq.first + x / D) * a.ldo + h * D + x % D;
        if (a.o32) static_cast<float *>(a.o)[to] = nan;
        else static_cast<uint16_t *>(a.o)[to] = 0x7FC0;
    }
    __syncwarp();
}

template <int D>
__global__ __launch_bounds__(kMainThreads, 1) void k_scan_main(const __grid_constant__ ScanArgs a,
                                                               const __grid_constant__ MainMaps maps) {
    using Z = MainSizes<D>;
    constexpr int COLS = D / 2;  // columns of S that a state thread holds
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    float *gam = reinterpret_cast<float *>(base + kStages * Z::kStage);  // [kStages][C]
    uint64_t *full = reinterpret_cast<uint64_t *>(gam + kStages * C), *empty = full + kStages;
    uint64_t *s_ready = empty + kStages, *p_full = s_ready + 2, *x_ready = p_full + 1, *f_full = x_ready + 1,
             *f_ready = f_full + 1, *u_full = f_ready + 1, *o_full = u_full + 2, *o_free = o_full + 1, *fin = o_free + 1,
             *known = fin + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(known + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1), *redo = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = (int)blockIdx.x / a.H, h = (int)blockIdx.x - r * a.H, hk = h / a.per_key;
    Seq seq = seq_of(a, r);
    if (seq.len > 0 && !found(a, r, slot_of(seq.first, r), slot_of(seq.first, r) + (seq.len - 1) / C)) seq.len = 0;
    const int64_t state = ((int64_t)r * a.H + h) * D * D;
    if (seq.len == 0) {
        if (a.S != a.S_out)
            for (int x = threadIdx.x; x < D * D / 4; x += kMainThreads)
                reinterpret_cast<float4 *>(a.S_out + state)[x] = reinterpret_cast<const float4 *>(a.S + state)[x];
        grid_dep_wait();
        return;
    }
    const int chunks = (seq.len + C - 1) / C;
    const bool outs = a.q != nullptr;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1 + kStateWarps + (outs ? 4 : 0));
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_ready + i, kStateWarps);
            mbar_init(u_full + i, 1);
        }
        mbar_init(p_full, 1);
        mbar_init(x_ready, kStateWarps);
        mbar_init(f_full, 1);
        mbar_init(f_ready, kStateWarps);
        mbar_init(o_full, 1);
        mbar_init(o_free, 4);
        mbar_init(fin, 1);
        mbar_init(known, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    int32_t *err = a.err;
    int issued = 0;  // chunks whose copies were handed out (the loading lane's)
    // The launch's registers (128 x 512) are split anew: 152 x 256 + 104 x 256.
    if (warp < kStateWarps) {
        // -------------------------------------------------------------- the state, and what is made of it
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        const int part = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;  // part: which tokens, which columns
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
        const bool live = row < D;
        float2 S[COLS / 2];
#pragma unroll
        for (int j = 0; j < COLS; j += 4) {
            const float4 x = live ? *reinterpret_cast<const float4 *>(a.S + state + (int64_t)row * D + part * COLS + j)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            S[j / 2] = make_float2(x.x, x.y), S[j / 2 + 1] = make_float2(x.z, x.w);
        }
        auto hand_over = [&](uint64_t *bar) {
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            const uint32_t ph = (c >> 1) & 1, par = c & 1;
            uint8_t *stage = base + st * Z::kStage;
            // S as two BF16 numbers, handed over 32 columns at a time
#pragma unroll
            for (int b = 0; b < COLS; b += 32) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) split2(S[b / 2 + j], hi[j], lo[j]);
                tmem_st16(lane_base + kColSH + part * (COLS / 2) + b / 2, hi);
                tmem_st16(lane_base + kColSL + part * (COLS / 2) + b / 2, lo);
                hand_over(s_ready + b / 32);
            }
            ok = warp_wait(full + st, ph, abort_flag, err);
            if (!ok) break;
            const int left = seq.len - c * C;  // tokens from here on
            // this row of V of the part's 32 tokens
            float v[32];
            {
                const uint8_t *vt = stage + Z::kKQ + (row / 64 % Z::kHalves) * kTile + part * 4096 + (row & 7) * 2;
                const int ch = (row & 63) >> 3;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(vt + (j >> 3) * 1024 + (j & 7) * 128 + ((ch ^ (j & 7)) << 4)) << 16);
            }
            ok = warp_wait(p_full, par, abort_flag, err);
            if (!ok) break;
            fence_after();
            {
                float p[32];
                tmem_ld32(lane_base + kColX + 32 * part, p);
                uint32_t hi[16], lo[16];
                const float4 *gm = reinterpret_cast<const float4 *>(gam + st * C + 32 * part);
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 ga = gm[j / 4];
                    p[j] = fmaf(-ga.x, p[j], v[j]), p[j + 1] = fmaf(-ga.y, p[j + 1], v[j + 1]);
                    p[j + 2] = fmaf(-ga.z, p[j + 2], v[j + 2]), p[j + 3] = fmaf(-ga.w, p[j + 3], v[j + 3]);
                }
                if (left < C)  // rows behind the sequence are another's
#pragma unroll
                    for (int j = 0; j < 32; ++j) p[j] = 32 * part + j < left ? p[j] : 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) split2(make_float2(p[2 * j], p[2 * j + 1]), hi[j], lo[j]);
                tmem_st16(lane_base + kColX + 32 * part, hi);
                tmem_st16(lane_base + kColX + 32 * part + 16, lo);
            }
            if (left < C) {  // their keys too: the state's product sums over the rows
                for (int x = threadIdx.x; x < (C - left) * (D / 8); x += 32 * kStateWarps) {
                    const int t = left + x / (D / 8), ch = x % (D / 8);
                    *reinterpret_cast<uint4 *>(stage + (ch >> 3) * 2 * kTile + swz(t, ch & 7)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
            }
            hand_over(x_ready);
            ok = warp_wait(f_full, par, abort_flag, err);
            if (!ok) break;
            fence_after();
            {
                float f[32];
                tmem_ld32(lane_base + kColF + 32 * part, f);
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) split2(make_float2(f[2 * j], f[2 * j + 1]), hi[j], lo[j]);
                tmem_st16(lane_base + kColF + 32 * part, hi);
                tmem_st16(lane_base + kColF + 32 * part + 16, lo);
            }
            hand_over(f_ready);
            const float gc = gam[st * C + C - 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + st);
            ok = warp_wait(u_full + part, par, abort_flag, err);
            if (!ok) break;
            fence_after();
#pragma unroll
            for (int b = 0; b < COLS; b += 32) {
                float u[32];
                tmem_ld32(lane_base + kColU + part * COLS + b, u);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    S[b / 2 + j] = make_float2(fmaf(gc, S[b / 2 + j].x, u[2 * j]), fmaf(gc, S[b / 2 + j].y, u[2 * j + 1]));
            }
            fence_before();
        }
        ok = ok && warp_wait(known, 0, abort_flag, err);
        if (ok && live && !*redo)
#pragma unroll
            for (int j = 0; j < COLS; j += 4)
                *reinterpret_cast<float4 *>(a.S_out + state + (int64_t)row * D + part * COLS + j) =
                    make_float4(S[j / 2].x, S[j / 2].y, S[j / 2 + 1].x, S[j / 2 + 1].y);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp < kMmaWarp) {
            // ---------------------------------------------------------- outputs
            const int quarter = warp & 3, row = 32 * quarter + lane;
            const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
            for (int c = 0; outs && c < chunks; ++c) {
                const int st = c & 1;
                if (!warp_wait(full + st, (c >> 1) & 1, abort_flag, err)) break;
                if (!warp_wait(o_full, c & 1, abort_flag, err)) break;
                fence_after();
                const int left = min(C, seq.len - c * C);
                const int64_t to = (int64_t)(seq.first + c * C) * a.ldo + h * D + row;
                float y[C];
#pragma unroll
                for (int b = 0; b < C; b += 32) {
                    float x[32];
                    tmem_ld32(lane_base + kColQ + b, x);
                    tmem_ld32(lane_base + kColO + b, y + b);
                    const float4 *gm = reinterpret_cast<const float4 *>(gam + st * C + b);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 ga = gm[j / 4];
                        y[b + j] = fmaf(ga.x, x[j], y[b + j]), y[b + j + 1] = fmaf(ga.y, x[j + 1], y[b + j + 1]);
                        y[b + j + 2] = fmaf(ga.z, x[j + 2], y[b + j + 2]), y[b + j + 3] = fmaf(ga.w, x[j + 3], y[b + j + 3]);
                    }
                }
                // read before anything is stored: the next chunk's products wait for these columns
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(o_free);
                    mbar_arrive(empty + st);
                }
                if (row >= D) continue;
                if (a.o32) {
                    float *o = static_cast<float *>(a.o) + to;
#pragma unroll
                    for (int j = 0; j < C; ++j, o += a.ldo)
                        if (j < left) *o = y[j];
                } else {
                    uint16_t *o = static_cast<uint16_t *>(a.o) + to;
                    if (left == C) {
#pragma unroll
                        for (int j = 0; j < C; ++j, o += a.ldo) *o = f32_to_bf16_rn(y[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < C; ++j, o += a.ldo)
                            if (j < left) *o = f32_to_bf16_rn(y[j]);
                    }
                }
            }
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------- products
            constexpr uint32_t kF = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);  // FP32 += BF16 BF16, 128 rows
            constexpr uint32_t id_t = kF | ((uint32_t)(C >> 3) << 17);              // 64 tokens
            constexpr uint32_t id_u = kF | (1u << 16) | ((64u >> 3) << 17);         // 64 columns, B is MN-major
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const uint32_t ph = (c >> 1) & 1, par = c & 1;
                const uint32_t kq = (smem_addr(base + st * Z::kStage) >> 4) & 0x3FFFu;
                const uint32_t img = (smem_addr(base + st * Z::kStage + Z::kKQ + Z::kV) >> 4) & 0x3FFFu;
                constexpr uint32_t T16 = kTile >> 4;
                if (!warp_wait(full + st, ph, abort_flag, err)) break;
                bool ok = true;
                // d += S b^T over the g-th 32 columns of either half of S
                auto with_state = [&](uint32_t d, uint32_t b, int g) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int kk = (i >> 1) * (D / 32) + 2 * g + (i & 1);
                            umma_ts(tmem + d, tmem + (x ? kColSL : kColSH) + 8 * kk, desc_of(b + (kk / 4) * 2 * T16 + (kk % 4) * 2, 16),
                                    id_t, g || x || i);
                        }
                };
                auto with_x = [&](uint32_t d, uint32_t b) {  // d = X b^T, all but low x low
#pragma unroll
                    for (int x = 0; x < 3; ++x)
#pragma unroll
                        for (int kk = 0; kk < C / 16; ++kk)
                            umma_ts(tmem + d, tmem + kColX + (x == 1 ? 16 : 0) + part_col(kk),
                                    desc_of(b + (x == 2 ? 2 * T16 : 0) + (2048 >> 4) * kk, kTile), id_u, x || kk);
                };
#pragma unroll
                for (int g = 0; g < D / 64; ++g) {
                    ok = ok && warp_wait(s_ready + g, par, abort_flag, err);
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) {
                        with_state(kColX, kq, g);
                        if (g == D / 64 - 1) commit(p_full);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (outs) {
                    if (c > 0 && !warp_wait(o_free, (c - 1) & 1, abort_flag, err)) break;
                    fence_after();
                    if (elect_one())
#pragma unroll
                        for (int g = 0; g < D / 64; ++g) with_state(kColQ, kq + T16, g);
                    __syncwarp();
                }
                if (!warp_wait(x_ready, par, abort_flag, err)) break;
                fence_after();
                if (elect_one()) {
                    with_x(kColF, img);
                    commit(f_full);
                    if (outs) {
                        with_x(kColO, img + T16);
                        commit(o_full);
                    }
                }
                __syncwarp();
                if (!warp_wait(f_ready, par, abort_flag, err)) break;
                fence_after();
                if (elect_one()) {  // 64 columns at a time: the state's first half is read under the other's product
#pragma unroll
                    for (int y = 0; y < Z::kHalves; ++y) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int kk = 0; kk < C / 16; ++kk)
                                umma_ts(tmem + kColU + 64 * y, tmem + kColF + 16 * x + part_col(kk),
                                        desc_of(kq + y * 2 * T16 + (2048 >> 4) * kk, 2 * kTile), id_u, x || kk);
                        commit(u_full + y);
                    }
                    if (Z::kHalves == 1) commit(u_full + 1);
                    commit(empty + st);
                }
                __syncwarp();
            }
        } else if (warp == kCondWarp) {
            // ---------------------------------------------------------- is any chunk ill-conditioned?  Then S_out stays as it is
            // (S, where they are the same), the outputs will be written again, and the head is handed to k_scan_redo.
            grid_dep_wait();
            const uint16_t *cond = reinterpret_cast<const uint16_t *>(a.cond) + slot_of(seq.first, r) * a.H + h;
            uint32_t any = 0;
            for (int c = lane; c < chunks; c += 32) any |= cond[(int64_t)c * a.H];
            any = __any_sync(kFull, any != 0);
            if (lane == 0) {
                *redo = any;
                mbar_arrive(known);
            }
        } else if (warp == kLoadWarp) {
            // ---------------------------------------------------------- loads
            const int64_t slot0 = slot_of(seq.first, r);
            if (a.stall) grid_dep_wait();
            for (int c = 0; c < chunks && !a.stall; ++c) {
                const int st = c & 1;
                if (c >= kStages && !warp_wait(empty + st, ((c >> 1) - 1) & 1, abort_flag, err)) break;
                if (lane == 0) {
                    uint64_t *bar = full + st;
                    const uint32_t at = smem_addr(base + st * Z::kStage);
                    const int row = seq.first + c * C;
                    const int64_t sh = (slot0 + c) * a.H + h;
                    mbar_expect_tx(bar, (outs ? Z::kKQ : Z::kKQ / 2) + Z::kV + (outs ? kImageBytes : kImageBytes / 2) + C * 4);
                    for (int x = 0; x < Z::kHalves; ++x) {
                        tma_load_2d(at + 2 * x * kTile, &maps.k, hk * D + 64 * x, row, bar);
                        if (outs) tma_load_2d(at + (2 * x + 1) * kTile, &maps.q, hk * D + 64 * x, row, bar);
                    }
                    for (int x = 0; x < Z::kHalves; ++x)
                        tma_load_2d(at + Z::kKQ + x * kTile, &maps.v, h * D + 64 * x, row, bar);
                    if (c == 0) grid_dep_wait();  // what follows k_scan_prep has made
                    for (int x = 0; x < 4; x += outs ? 1 : 2)
                        bulk_load(at + Z::kKQ + Z::kV + x * kTile, a.image + sh * kImageBytes + x * kTile, kTile, bar);
                    bulk_load(smem_addr(gam + st * C), a.gamma + sh * C, C * 4, bar);
                }
                ++issued;
                __syncwarp();
            }
        }
    }
    __syncthreads();
    if (*abort_flag) all_nan<D>(a);
    else if (threadIdx.x == 0 && *redo) a.redo[1 + atomicAdd(a.redo, 1)] = blockIdx.x;
    // every copy and every MMA that was issued has completed before shared memory and TMEM go
    if (warp == kLoadWarp && lane == 0)
        for (int c = max(0, issued - kStages); c < issued; ++c) mbar_drain(full + (c & 1), (c >> 1) & 1, err);
    if (warp == kMmaWarp) {
        if (elect_one()) commit(fin);
        __syncwarp();
        mbar_drain(fin, 0, err);
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int D>
cudaError_t launch_d(const ScanArgs &a, const MainMaps &m, int64_t slots, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_scan_prep<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(PrepSmem<D>));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(k_scan_main<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)main_smem_bytes<D>());
    if (e != cudaSuccess) return e;
    k_scan_prep<D><<<dim3((unsigned)slots, (unsigned)(a.H / a.per_key) + (a.status ? 1 : 0)), kPrepThreads, sizeof(PrepSmem<D>), s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)a.R * a.H));
    cfg.blockDim = dim3(kMainThreads);
    cfg.dynamicSmemBytes = main_smem_bytes<D>();
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    // The early start gains 2 us (3 x 1000 tokens 45 us, without 47), and costs long sequences more than that by the
    // places that it finds for the CTAs (8191 tokens 382 us, without 360).
    cfg.numAttrs = a.n <= 1024LL * a.R ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_scan_main<D>, a, m);
}

}  // namespace

size_t scan_chunk_bytes(int64_t n, int64_t R, int H) {
    const size_t units = (size_t)slots_of(n, R) * H;
    return 256 + units * (kImageBytes + C * 4) + cond_bytes(units) + (size_t)(1 + R * H) * 4;
}

cudaError_t launch_scan_chunks(ScanArgs &a, const w12_gdn_scan_args &x, void *workspace, cudaStream_t s) {
    MainMaps m;
    const int64_t kd[2] = {(int64_t)x.key_heads * x.D, x.n}, vd[2] = {(int64_t)x.H * x.D, x.n};
    const int box[2] = {64, C};
    if (!encode_tmap(&m.k, x.k, 2, kd, &x.ldk, box) || !encode_tmap(&m.v, x.v, 2, vd, &x.ldv, box)) return cudaErrorNotSupported;
    if (x.q && !encode_tmap(&m.q, x.q, 2, kd, &x.ldq, box)) return cudaErrorNotSupported;
    if (!x.q) m.q = m.k;
    const int64_t slots = slots_of(x.n, x.R);
    a.stall = x.mode & W12_GDN_TEST_STALL;
    a.err = x.status ? x.status : static_cast<int32_t *>(workspace);
    a.image = static_cast<uint8_t *>(workspace) + 256;
    a.gamma = reinterpret_cast<float *>(a.image + (size_t)slots * x.H * kImageBytes);
    a.cond = reinterpret_cast<uint8_t *>(a.gamma + (size_t)slots * x.H * C);
    a.redo = reinterpret_cast<int32_t *>(a.cond + cond_bytes((size_t)slots * x.H));
    return x.D == 64 ? launch_d<64>(a, m, slots, s) : launch_d<128>(a, m, slots, s);
}

}  // namespace w12
