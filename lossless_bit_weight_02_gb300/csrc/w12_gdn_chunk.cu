// The gated delta rule over long sequences: chunks of 64 tokens, the products on
// the tensor cores (tcgen05).
//
// Within a chunk that begins with the state S0, with gamma_t the product of
// alpha up to t, G_tj that of alpha after j up to t, and f_t the coefficient
// vectors (S = gamma S0 + sum G f k^T, see w12_gdn.cu),
//     (I + A) F = diag(beta) X,   X = V - diag(gamma) K S0^T,   A_tj = beta_t G_tj k_t.k_j (j < t)
//     O = diag(gamma) Q S0^T + M F,   M_tj = G_tj q_t.k_j (j <= t)
//     S = gamma_C S0 + (G_C. F)^T K
// With T = (I + A)^-1 diag(beta), which does not depend on S0, this is two products with
// X: G_C. F = (diag(G_C.) T) X, and M F = (M T) X.
#include <cstdint>
#include <cuda_runtime.h>

#include "w12_gdn_scan.cuh"
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

// Two FP32 values as BF16 pairs: the nearest, and the nearest to what remains (lower column in the low half).
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
    hi = pack2(x.x, x.y);
    const float2 rest = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)), make_float2(-1.f, -1.f), x);
    lo = pack2(rest.x, rest.y);
}

// ---------------------------------------------------------------------------
// T and M T of every chunk and head, as the tiles that k_scan_main's products read.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr int kP = C + 4;  // pitch of a 64 x 64 FP32 matrix

template <int D>
struct PrepSmem {
    uint16_t k[C][D + 8], q[C][D + 8];
    float A[C][kP], M[C][kP], T[C][kP];
    float Y[C][kP / 2];
    long long lg[C];  // sums of log2 alpha in 2^-40
    float beta[C], bad[C];
};

__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fixed(long long d) {  // 2^(d 2^-40)
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((float)d * 0x1p-40f));
    return y;
}

template <int D>
__global__ __launch_bounds__(kPrepThreads, 2) void k_scan_prep(const __grid_constant__ ScanArgs a) {
    extern __shared__ __align__(16) uint8_t smem_prep[];
    PrepSmem<D> &sm = *reinterpret_cast<PrepSmem<D> *>(smem_prep);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
    if (blockIdx.y == (unsigned)a.H) {  // one CTA more a column of the grid: only the first is of use
        if (blockIdx.x == 0 && a.status) check_all(a);
        return;
    }
    const int slot = blockIdx.x, h = blockIdx.y, hk = h / a.per_key;
    int lo = 0, hi = a.R - 1;  // the last request whose first slot is not behind this one
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (slot_of(a.start[mid], mid) <= slot) lo = mid;
        else hi = mid - 1;
    }
    const int r = lo;
    const Seq seq = seq_of(a, r);
    const int64_t c = slot - slot_of(a.start[r], r);
    if (!seq.ok || c < 0 || c * C >= seq.len) return;
    const int row0 = seq.first + (int)c * C, m = min(C, seq.len - (int)c * C);
    // rows of keys and queries, zeros behind the sequence
    for (int x = tid; x < C * (D / 8); x += kPrepThreads) {
        const int t = x / (D / 8), ch = x % (D / 8);
        uint4 kv = make_uint4(0, 0, 0, 0), qv = kv;
        if (t < m) {
            kv = *reinterpret_cast<const uint4 *>(a.k + (int64_t)(row0 + t) * a.ldk + hk * D + 8 * ch);
            if (a.q) qv = *reinterpret_cast<const uint4 *>(a.q + (int64_t)(row0 + t) * a.ldq + hk * D + 8 * ch);
        }
        *reinterpret_cast<uint4 *>(&sm.k[t][8 * ch]) = kv;
        *reinterpret_cast<uint4 *>(&sm.q[t][8 * ch]) = qv;
    }
    if (warp == 0) {
        // Sums of logarithms, as whole numbers: a decay of 0 (2^-200 here) leaves no error in the differences behind it.
        long long s[2];
        bool bad[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = 2 * lane + u;
            const float al = t < m ? a.alpha[(int64_t)(row0 + t) * a.H + h] : 1.f;
            bad[u] = !(al >= 0.f && al < INFINITY);
            s[u] = __float2ll_rn(fmaxf(log2f(bad[u] ? 1.f : al), -200.f) * 0x1p40f);
            sm.beta[t] = t < m ? a.beta[(int64_t)(row0 + t) * a.H + h] : 0.f;
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
        const long long before = sum - s[1];
        const bool bad_before = __shfl_up_sync(kFull, any, 1) && lane > 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            sm.lg[2 * lane + u] = before + s[u];
            sm.bad[2 * lane + u] = bad_before || bad[u] ? __int_as_float(0x7FC00000) : 0.f;
        }
    }
    __syncthreads();
    float *gamma = a.gamma + ((int64_t)slot * a.H + h) * C;
    if (tid < C) gamma[tid] = exp2_fixed(sm.lg[tid]) + sm.bad[tid];
    // A and M: 16 x 16 blocks on and below the diagonal, a warp one of K K^T or Q K^T at a time
    {
        const uint32_t *K32 = reinterpret_cast<const uint32_t *>(sm.k);
        constexpr int RW = (D + 8) / 2;
        for (int x = warp; x < (a.q ? 20 : 10); x += kPrepThreads / 32) {
            const int y = x % 10, bi = y < 1 ? 0 : y < 3 ? 1 : y < 6 ? 2 : 3, bj = y - bi * (bi + 1) / 2;
            const bool isq = x >= 10;
            const uint32_t *X32 = isq ? reinterpret_cast<const uint32_t *>(sm.q) : K32;
            float acc[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int w0 = 8 * kk + q4;
                const uint32_t af[4] = {X32[(16 * bi + g) * RW + w0], X32[(16 * bi + g + 8) * RW + w0],
                                        X32[(16 * bi + g) * RW + w0 + 4], X32[(16 * bi + g + 8) * RW + w0 + 4]};
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int rn = 16 * bj + 8 * nt + g;
                    mma16816(acc[nt], af, K32[rn * RW + w0], K32[rn * RW + w0 + 4]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * bi + g + 8 * (e >> 1), j = 16 * bj + 8 * nt + 2 * q4 + (e & 1);
                    const float G = exp2_fixed(sm.lg[t] - sm.lg[j]) + sm.bad[t];
                    if (isq) sm.M[t][j] = j <= t ? G * acc[nt][e] : 0.f;
                    else sm.A[t][j] = j < t ? sm.beta[t] * G * acc[nt][e] : 0.f;
                }
        }
    }
    // zeros above the diagonal blocks of M and T
    for (int x = tid; x < 6 * 256; x += kPrepThreads) {
        const int y = x >> 8, bj = y < 1 ? 1 : y < 3 ? 2 : 3, bi = y - bj * (bj - 1) / 2, i = 16 * bi + (x >> 4 & 15), j = 16 * bj + (x & 15);
        sm.M[i][j] = 0.f;
        sm.T[i][j] = 0.f;
    }
    __syncthreads();
    // (I + A)^-1: diagonal blocks of 16 by substitution, a lane a column
    if (warp < 4 && lane < 16) {
        const int b = 16 * warp;
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int s = 0; s < t; s += 2) {
                s0 = fmaf(sm.A[b + t][b + s], x[s], s0);
                if (s + 1 < t) s1 = fmaf(sm.A[b + t][b + s + 1], x[s + 1], s1);
            }
            x[t] = t == lane ? 1.f : t > lane ? -(s0 + s1) : 0.f;
        }
#pragma unroll
        for (int t = 0; t < 16; ++t) sm.T[b + t][b + lane] = x[t];
    }
    __syncthreads();
    // blocks of twice the size: T21 = -T22 (A21 T11)
    for (int half = 16; half < C; half *= 2) {
        const int pairs = C / (2 * half), outs = pairs * half * half;
        for (int x = tid; x < outs; x += kPrepThreads) {
            const int p = x / (half * half), i = x / half % half, j = x % half, b = 2 * half * p;
            float s = 0.f;
            for (int k = j; k < half; ++k) s = fmaf(sm.A[b + half + i][b + k], sm.T[b + k][b + j], s);
            sm.Y[p * half + i][j] = s;
        }
        __syncthreads();
        for (int x = tid; x < outs; x += kPrepThreads) {
            const int p = x / (half * half), i = x / half % half, j = x % half, b = 2 * half * p;
            float s = 0.f;
            for (int k = 0; k <= i; ++k) s = fmaf(sm.T[b + half + i][b + half + k], sm.Y[p * half + k][j], s);
            sm.T[b + half + i][b + j] = -s;
        }
        __syncthreads();
    }
    // out: rows t of G_C T beta and of M T beta, eight columns at a time
    uint8_t *img = a.image + ((int64_t)slot * a.H + h) * kImageBytes;
    for (int x = tid; x < 2 * C * (C / 8); x += kPrepThreads) {
        const int what = x / (C * (C / 8)), t = x / (C / 8) % C, ch = x % (C / 8);
        if (what && !a.q) break;
        float y[8];
        if (what == 0) {
            const float e = exp2_fixed(sm.lg[C - 1] - sm.lg[t]) + sm.bad[C - 1];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = e * sm.T[t][8 * ch + j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = 0.f;
            for (int s = 8 * ch; s <= t; ++s) {
                const float w = sm.M[t][s];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fmaf(w, sm.T[s][8 * ch + j], y[j]);
            }
        }
        uint32_t hi4[4], lo4[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const int col = 8 * ch + j;
            // nothing above the diagonal, and nothing behind the sequence
            const float u = col <= t && t < m ? y[j] * sm.beta[col] : 0.f, v = col + 1 <= t && t < m ? y[j + 1] * sm.beta[col + 1] : 0.f;
            split2(make_float2(u, v), hi4[j / 2], lo4[j / 2]);
        }
        *reinterpret_cast<uint4 *>(img + what * kTile + swz(t, ch)) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
        *reinterpret_cast<uint4 *>(img + (2 + what) * kTile + swz(t, ch)) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
    }
}

// ---------------------------------------------------------------------------
// The chunks of a (request, head), one after the other: a CTA.  The products
// are taken transposed: a TMEM lane is a row of S, the tokens are columns.
// ---------------------------------------------------------------------------
constexpr int kStateWarps = 8, kMmaWarp = 12, kLoadWarp = 13;  // outputs: 8 .. 11
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
             *f_ready = f_full + 1, *u_full = f_ready + 1, *o_full = u_full + 2, *o_free = o_full + 1, *fin = o_free + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fin + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = (int)blockIdx.x / a.H, h = (int)blockIdx.x - r * a.H, hk = h / a.per_key;
    const Seq seq = seq_of(a, r);
    const int64_t state = ((int64_t)r * a.H + h) * D * D;
    if (seq.len == 0) {
        if (a.S != a.S_out)
            for (int x = threadIdx.x; x < D * D / 4; x += kMainThreads)
                reinterpret_cast<float4 *>(a.S_out + state)[x] = reinterpret_cast<const float4 *>(a.S + state)[x];
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
                    const float2 x = fma2(make_float2(-ga.x, -ga.y), make_float2(p[j], p[j + 1]), make_float2(v[j], v[j + 1]));
                    const float2 y = fma2(make_float2(-ga.z, -ga.w), make_float2(p[j + 2], p[j + 3]), make_float2(v[j + 2], v[j + 3]));
                    p[j] = x.x, p[j + 1] = x.y, p[j + 2] = y.x, p[j + 3] = y.y;
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
                    S[b / 2 + j] = fma2(make_float2(gc, gc), S[b / 2 + j], make_float2(u[2 * j], u[2 * j + 1]));
            }
            fence_before();
        }
        if (ok && live)
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
                        const float2 u = fma2(make_float2(ga.x, ga.y), make_float2(x[j], x[j + 1]), make_float2(y[b + j], y[b + j + 1]));
                        const float2 w = fma2(make_float2(ga.z, ga.w), make_float2(x[j + 2], x[j + 3]), make_float2(y[b + j + 2], y[b + j + 3]));
                        y[b + j] = u.x, y[b + j + 1] = u.y, y[b + j + 2] = w.x, y[b + j + 3] = w.y;
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
                            umma_ts(tmem + d, tmem + kColX + (x == 1 ? 16 : 0) + part_col(kk), desc_of(b + (x == 2 ? 2 * T16 : 0) + kk * 2, 16),
                                    id_t, x || kk);
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
        } else if (warp == kLoadWarp && !a.stall) {
            // ---------------------------------------------------------- loads
            const int64_t slot0 = slot_of(seq.first, r);
            for (int c = 0; c < chunks; ++c) {
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
                    for (int x = 0; x < 4; x += outs ? 1 : 2)
                        bulk_load(at + Z::kKQ + Z::kV + x * kTile, a.image + sh * kImageBytes + x * kTile, kTile, bar);
                    bulk_load(smem_addr(gam + st * C), a.gamma + sh * C, C * 4, bar);
                }
                ++issued;
                __syncwarp();
            }
        }
    }
    // every copy and every MMA that was issued has completed before shared memory and TMEM go
    __syncthreads();
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
    k_scan_prep<D><<<dim3((unsigned)slots, (unsigned)a.H + (a.status ? 1 : 0)), kPrepThreads, sizeof(PrepSmem<D>), s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_scan_main<D><<<(unsigned)((int64_t)a.R * a.H), kMainThreads, main_smem_bytes<D>(), s>>>(a, m);
    return cudaGetLastError();
}

}  // namespace

size_t scan_chunk_bytes(int64_t n, int64_t R, int H) {
    return 256 + (size_t)slots_of(n, R) * H * (kImageBytes + C * 4);
}

cudaError_t launch_scan_chunks(ScanArgs a, const w12_gdn_scan_args &x, void *workspace, cudaStream_t s) {
    MainMaps m;
    const int64_t kd[2] = {(int64_t)x.key_heads * x.D, x.n}, vd[2] = {(int64_t)x.H * x.D, x.n};
    const int box[2] = {64, C};
    if (!encode_tmap(&m.k, x.k, 2, kd, &x.ldk, box) || !encode_tmap(&m.v, x.v, 2, vd, &x.ldv, box)) return cudaErrorNotSupported;
    if (x.q && !encode_tmap(&m.q, x.q, 2, kd, &x.ldq, box)) return cudaErrorNotSupported;
    if (!x.q) m.q = m.k;
    const int64_t slots = slots_of(x.n, x.R);
    a.err = x.status ? x.status : static_cast<int32_t *>(workspace);
    a.image = static_cast<uint8_t *>(workspace) + 256;
    a.gamma = reinterpret_cast<float *>(a.image + (size_t)slots * x.H * kImageBytes);
    return x.D == 64 ? launch_d<64>(a, m, slots, s) : launch_d<128>(a, m, slots, s);
}

}  // namespace w12
