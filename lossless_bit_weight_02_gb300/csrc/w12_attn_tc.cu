// Attention of draft-tree nodes over a paged cache, many rows per key/value
// head: tcgen05.mma with scores, weights and outputs in TMEM.
//
// A CTA (one per SM, persistent over its range of the work line) runs two
// streams of 128 query rows through the same machinery:
//   * an item of more than 128 rows ("pair"): the streams are its two row
//     tiles, and every key block serves both;
//   * an item of at most 128 rows ("split"): both streams hold the same rows
//     and take the key blocks in turn; their (max, sum, O) join in TMEM at
//     the end, where a row's two halves lie in the same lane.
// Step u of an item belongs to stream u & 1.  Per step the MMA warp issues
//     S = Q K^T        (M = 128 rows, N = 128 keys, both operands in shared memory)
//     O += P V         (P in TMEM over the first half of S, V in shared memory, MN-major)
// in the order S(0) S(1) | O(0) S(2) | O(1) S(3) | ..., so the tensor cores
// work on one stream while the softmax warps work on the other.  Warps 0-3
// and 4-7 are the streams' softmax: thread = row = TMEM lane, so maxima and
// sums need no exchange.  The row maximum is the largest seen rounded up
// lazily: O is rescaled only when a block's maximum exceeds the reference by
// more than 8 (a factor 256 of FP32's range), which after the first blocks
// almost never happens.
//
// Keys and values arrive in a ring of [128 keys x D] tiles.  Blocks that every
// row sees whole come by TMA (a copy per page and 64 columns); blocks with
// anything masked (the end of the cache, the tree, the window's edge) are
// gathered by two warps with plain loads: absent keys become zeros, and
// values that are not finite are left out of the product and added at the end
// to the rows that see them, so that 0 * Inf cannot reach a row.
//
// Rate: a step is 8.4 MFLOP at D = 128, about 1050 tensor cycles; its 64 KB of
// keys and values take about 1500 cycles of HBM at an SM's share.  So a split
// item is bound by HBM and a pair item by the tensor cores or the softmax.
//
// Every wait is bounded (about a second): a CTA that gives up sets the
// workspace's timeout word, drains its copies and MMAs and frees its TMEM.
#include <cstdint>
#include <cuda_runtime.h>
#include <mutex>
#include <type_traits>

#include "w12_attn.cuh"
#include "w12_tc.cuh"

namespace w12 {
namespace {

using namespace tc;

constexpr int kRows = 128;     // of a stream
constexpr int kKeys = kAttnTcBlock;  // of a block
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 10, kLoadWarps = 2;  // MMA: one warp per stream
constexpr int kTcThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 per stream
constexpr float kLazy = 8.0f;               // log2 of the growth that an unscaled O may carry
constexpr int kPoison = 8;                  // masked blocks of a segment (at most 3 at the window's edge, 4 at the end)

template <int D>
struct TcSizes {
    static constexpr uint32_t kSlot = kKeys * D * 2;
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr uint32_t kQ = kRows * D * 2;
};

constexpr int kQuarters = kKeys / 32;
struct Poison {  // per 32 rows of a block: masked blocks whose V rows hold values that are not finite
    int n;
    int key[kPoison];
    uint32_t rows[kPoison];
};

template <int D>
constexpr size_t tc_smem_bytes() {
    return 1024 + (size_t)TcSizes<D>::kSlots * TcSizes<D>::kSlot + 2 * TcSizes<D>::kQ + 8 * (2 * TcSizes<D>::kSlots + 13) +
           2 * kQuarters * sizeof(Poison) + 16 + 16 * ((TcSizes<D>::kSlots + 3) / 4) +
           (kTcThreads / 32) * sizeof(SegWalk);
}
static_assert(tc_smem_bytes<128>() <= 227 * 1024, "one CTA's shared memory");

// A position in the ring as slot and phase.
template <int NS>
struct RingPos {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void advance(uint32_t d, uint32_t laps = 0) {  // d <= NS
        slot += d;
        phase ^= laps;
        if (slot >= NS) {
            slot -= NS;
            phase ^= 1u;
        }
    }
};

// The order in which tiles enter the ring: that in which the MMAs need them.
// pair: K0 V0 K1 V1 ...; split: K0 K1 V0 K2 V1 ... V(n-2) V(n-1).
__device__ __forceinline__ void load_at(bool pair, int nb, int l, bool &is_v, int &j) {
    if (pair) {
        is_v = l & 1;
        j = l >> 1;
    } else if (l == 2 * nb - 1) {
        is_v = true;
        j = nb - 1;
    } else if (l == 0) {
        is_v = false;
        j = 0;
    } else {
        is_v = !(l & 1);
        j = is_v ? (l - 2) / 2 : (l + 1) / 2;
    }
}

__device__ __forceinline__ int key_of(const Seg &s, int j) { return s.key0 + j * kKeys; }
// every row of the request sees every key of the block, and all are cached
__device__ __forceinline__ bool seen_whole(const Seg &s, int key) {
    return key >= s.lo_max && key + kKeys <= s.ctx;
}
// bits below n
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Which of the keys [key, key + 32) a row sees: cached ones from lo on, and
// the ranks of its mask.
__device__ __forceinline__ uint32_t seen_word(int key, int ctx, int lo, const uint32_t *mask) {
    uint32_t w = below(ctx - key) & ~below(lo - key);
    const int rk = key - ctx;  // rank of the first key
    if (rk > -32 && rk < kAttnMaxNodes) {
        const int i = rk >> 5;  // floor
        const uint32_t lo_w = i >= 0 ? mask[i] : 0u, hi_w = i + 1 < kMaskWords ? mask[i + 1] : 0u;
        w |= __funnelshift_r(lo_w, hi_w, rk & 31);
    }
    return w;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int D, bool CAP>
__global__ __launch_bounds__(kTcThreads, 1) void k_attn_tc(const __grid_constant__ AttnArgs a,
                                                           const __grid_constant__ CUtensorMap kmap,
                                                           const __grid_constant__ CUtensorMap vmap, const int use_tma) {
    using Z = TcSizes<D>;
    constexpr int NS = Z::kSlots;
    constexpr uint32_t kHalf = kKeys * 128;  // 64 columns of a tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = base, *qs = base + NS * Z::kSlot;
    SegWalk *walks = reinterpret_cast<SegWalk *>(qs + 2 * Z::kQ);  // [warps]
    uint64_t *full = reinterpret_cast<uint64_t *>(walks + kTcThreads / 32);
    uint64_t *empty = full + NS, *q_full = empty + NS, *q_free = q_full + 1, *s_full = q_free + 1, *p_full = s_full + 2,
             *p_half = p_full + 2, *pv_done = p_half + 2, *o_free = pv_done + 2, *ml_ready = o_free + 1;
    uint64_t *fin = ml_ready + 1;  // every MMA of the CTA has completed
    Poison *poison = reinterpret_cast<Poison *>(fin + 1);  // [2][quarters]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(poison + 2 * kQuarters);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile uint32_t *granted = tmem_slot + 2;  // ring positions up to here may be filled by the gather warps
    uint32_t *issued = tmem_slot + 3;  // [NS]: the ring position last handed to the TMA unit, + 1

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, kLoadWarps);
            mbar_init(empty + i, 2);  // both streams are done with it
            issued[i] = 0;
        }
        mbar_init(q_full, kLoadWarps);
        mbar_init(q_free, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(p_half + i, 4);
            mbar_init(pv_done + i, 1);
        }
        mbar_init(o_free, kSoftWarps);
        mbar_init(ml_ready, kSoftWarps);
        mbar_init(fin, 2);
        *abort_flag = 0;
        *granted = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == kLoadWarp && lane == 0 && use_tma) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    int32_t *err = a.ws.timeout;
    grid_dep_wait();
    grid_dep_launch();

    // The launch's registers (168 x 384) are split anew, 216 x 256 + 72 x 128, per warpgroup.
    // (a warp's segment lies in shared memory: the registers are for the scores)
    SegWalk &walk = walks[warp];
    Seg &sg = walk.sg;
    const Geometry geo{kAttnTcRows, kKeys, kRows, kAttnTcPair, kAttnTcOne};
    if (lane == 0) walk.begin(a, geo);
    __syncwarp();
    if (warp < kSoftWarps) {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int st = warp >> 2, quarter = warp & 3;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t tS = lane_base + kColS + 128 * st;
        const float sl2 = a.scale * kLog2e, cap2 = CAP ? 2.0f * kLog2e * a.scale / a.softcap : 0.f,
                    capl = CAP ? a.softcap * kLog2e : 0.f;
        uint32_t n_s = 0, n_pv[2] = {0, 0}, n_ml = 0;
        int seg = 0;
        for (; walk.next(a, geo); ++seg) {
            const int row0 = (sg.pair ? st * kRows : 0) + 32 * quarter + lane;  // row of the item
            const int rowi = sg.t * kAttnTcRows + row0, rank = rowi / a.group;
            const bool live = row0 < sg.rows;
            const int at = sg.start + (live ? rank : 0);
            const uint32_t *mrow = a.ws.mask + (int64_t)at * kMaskWords;
            const int lo_key = a.window > 0 ? sg.ctx + a.ws.depth[at] - a.window : 0;
            float m = -INFINITY, l = 0.f;  // reference maximum (log2 domain), sum
            bool ok = true;
            // One step: the row's 128 scores of S(u), read once into registers, become weights, which
            // go over the first half of S.
            auto step = [&](bool first, int key, auto masked_) {
                constexpr bool masked = decltype(masked_)::value;
                float v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_start(tS + 32 * c, v[c]);
                uint32_t see[4];
                float t0 = -INFINITY, t1 = t0, t2 = t0, t3 = t0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (masked) see[c] = seen_word(key + 32 * c, sg.ctx, lo_key, mrow);
                    float *x = v[c];
                    tmem_ld32_wait(x);
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = see[c] >> j & 1u ? x[j] : -INFINITY;
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        t0 = max3(t0, x[j], x[j + 1]);
                        t1 = max3(t1, x[j + 2], x[j + 3]);
                        t2 = max3(t2, x[j + 4], x[j + 5]);
                        t3 = max3(t3, x[j + 6], x[j + 7]);
                    }
                }
                float top = fmaxf(max3(t0, t1, t2), t3);
                top = CAP ? cap_score(top, cap2, capl) : top * sl2;  // both grow with the score
                const bool grow = top > m + kLazy || (m == -INFINITY && top > m);
                if (__any_sync(kFull, grow)) {
                    const float mn = grow ? top : m, f = grow ? exp2_approx(m - mn) : 1.0f;
                    l *= f;
                    m = mn;
                    if (!first) {  // what was summed so far; the stream's last product is complete (s_full)
#pragma unroll 1
                        for (int c = 0; c < D; c += 8) tmem_scale8(lane_base + kColO + 128 * st + c, f);
                    }
                }
                const float m0 = m == -INFINITY ? 0.f : m;
                const float2 sc = make_float2(sl2, sl2), mm = make_float2(-m0, -m0);
                auto weights = [&](int c) {
                    float *x = v[c];
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float2 y = make_float2(x[j], x[j + 1]);
                        if (CAP) y = make_float2(cap_score(y.x, cap2, capl) - m0, cap_score(y.y, cap2, capl) - m0);
                        else y = fma2(y, sc, mm);
                        x[j] = exp2_approx(y.x);
                        x[j + 1] = exp2_approx(y.y);
                        if (masked) {
                            x[j] = see[c] >> j & 1u ? x[j] : 0.f;
                            x[j + 1] = see[c] >> (j + 1) & 1u ? x[j + 1] : 0.f;
                        }
                        p[j / 2] = pack_bf16(x[j], x[j + 1]);
                    }
                    tmem_st16(tS + 16 * c, p);
                };
                weights(0);
                weights(1);
                wait_st();  // the first 64 keys' weights, and O
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_half + st);
                weights(2);
                weights(3);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + st);
                // the sum, while the products run
                float2 s0 = make_float2(0.f, 0.f), s1 = s0, s2 = s0, s3 = s0;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        s0 = add2(s0, make_float2(v[c][j], v[c][j + 1]));
                        s1 = add2(s1, make_float2(v[c][j + 2], v[c][j + 3]));
                        s2 = add2(s2, make_float2(v[c][j + 4], v[c][j + 5]));
                        s3 = add2(s3, make_float2(v[c][j + 6], v[c][j + 7]));
                    }
                s0 = add2(add2(s0, s1), add2(s2, s3));
                l += s0.x + s0.y;
            };
            {
                const int lo_max = sg.lo_max, whole_end = sg.ctx - kKeys;  // keys of blocks that every row sees whole
                const int U = sg.pair ? 2 * sg.nb : sg.nb, key_step = sg.pair ? kKeys : 2 * kKeys;
                int key = sg.key0 + (sg.pair ? 0 : st * kKeys);
                for (int u = st; u < U; u += 2, key += key_step) {
                    const bool whole = key >= lo_max && key <= whole_end;
                    ok = warp_wait(s_full + st, n_s & 1, abort_flag, err);
                    if (!ok) break;
                    ++n_s;
                    fence_after();
                    if (whole) step(u < 2, key, std::false_type{});
                    else step(u < 2, key, std::true_type{});
                }
            }
            if (!ok) break;
            // ---- the end of the segment: join (split) and write
            const bool two = sg.pair || sg.nb > 1;
            float f0 = 1.0f, f1 = 0.0f;
            if (sg.pair) {  // (stream 1 waits for both: its next wait for stream 0's may be one segment on)
                if (!warp_wait(pv_done, n_pv[0] & 1, abort_flag, err)) break;
                if (st && !warp_wait(pv_done + 1, n_pv[1] & 1, abort_flag, err)) break;
                fence_after();
            } else {
                if (!warp_wait(pv_done, n_pv[0] & 1, abort_flag, err)) break;
                if (two && !warp_wait(pv_done + 1, n_pv[1] & 1, abort_flag, err)) break;
                // the other stream's (max, sum) of this row, through the unused half of S
                fence_after();
                tmem_st2(tS + 64, m, l);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_ready);
                if (!warp_wait(ml_ready, n_ml & 1, abort_flag, err)) break;
                ++n_ml;
                fence_after();
                const float2 o = tmem_ld2(lane_base + kColS + 128 * (st ^ 1) + 64);
                const float ma = st ? o.x : m, la = st ? o.y : l, mb = st ? m : o.x, lb = st ? l : o.y;
                m = fmaxf(ma, mb);
                const float m0 = m == -INFINITY ? 0.f : m;
                f0 = exp2_approx(ma - m0);
                f1 = two ? exp2_approx(mb - m0) : 0.f;
                l = two ? fmaf(lb, f1, la * f0) : la * f0;
            }
            ++n_pv[0];
            n_pv[1] += two;
            const float inv = sg.whole ? 1.0f / l : 1.0f;
            f0 *= inv;
            f1 *= inv;
            const int node = a.ws.order[at];
            const int head = sg.h * a.group + (rowi - rank * a.group);
            uint16_t *orow = a.o + (int64_t)node * a.ldo + (int64_t)head * D;
            const int64_t prow = (int64_t)sg.slot * kAttnTcRows + row0;
            // neighbouring lanes (rows) write neighbouring addresses
            float *part = a.ws.part + ((int64_t)sg.slot * (D / 4) * kAttnTcRows + row0) * 4;
            const Poison *po = poison + (seg & 1) * kQuarters;
            const bool any_odd = po[0].n | po[1].n | po[2].n | po[3].n;
            const int cbeg = sg.pair ? 0 : st * (D / 64), cend = sg.pair ? D / 32 : cbeg + D / 64;
            for (int c = cbeg; c < cend; ++c) {
                float v[32];
                tmem_ld32(lane_base + kColO + (sg.pair ? 128 * st : 0) + 32 * c, v);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= f0;
                if (!sg.pair && two) {
                    float w[32];
                    tmem_ld32(lane_base + kColO + 128 + 32 * c, w);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = fmaf(w[j], f1, v[j]);
                }
                if (any_odd) {
                    for (int g = 0; g < kQuarters; ++g)
                        for (int i = 0; i < po[g].n; ++i) {
                            for (uint32_t rest = po[g].rows[i]; rest; rest &= rest - 1) {
                                const int key = po[g].key[i] + 32 * g + __ffs(rest) - 1;
                                if (!(seen_word(key, sg.ctx, lo_key, mrow) & 1u)) continue;
                                const uint16_t *vr;
                                if (key >= sg.ctx) {
                                    vr = a.v + (int64_t)a.ws.order[sg.start + key - sg.ctx] * a.ldv + sg.h * D;
                                } else {
                                    int tok;
                                    const int64_t pg = page_of(a, sg.r, key, tok);
                                    vr = a.cv + pg * a.page_stride + tok * a.token_stride + sg.h * a.head_stride;
                                }
#pragma unroll
                                for (int j = 0; j < 32; ++j) {
                                    const float x = __uint_as_float((uint32_t)vr[32 * c + j] << 16);
                                    if (!isfinite(x)) v[j] += x;
                                }
                            }
                        }
                }
                if (live) {
                    if (sg.whole) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            *reinterpret_cast<uint4 *>(orow + 32 * c + j) =
                                make_uint4(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]),
                                           pack_bf16(v[j + 4], v[j + 5]), pack_bf16(v[j + 6], v[j + 7]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4 *>(part + (int64_t)(8 * c + j / 4) * (4 * kAttnTcRows)) =
                                make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    }
                }
            }
            if (live && !sg.whole && (sg.pair || st == 0)) a.ws.ml[prow] = make_float2(m, l);
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp < kLoadWarp) {
            // -------------------------------------------------------- MMA issue, one warp per stream
            constexpr uint32_t kF = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kRows >> 4) << 24);  // FP32 += BF16 BF16
            constexpr uint32_t id_s = kF | ((uint32_t)(kKeys >> 3) << 17);
            constexpr uint32_t id_o = kF | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // B is MN-major
            // What the loop needs is kept warp-uniform (shuffles from lane 0 say so to the compiler) and
            // advanced, not recomputed: these warps' own instructions are on the path of every step.  The
            // MMA unit queues about four instructions (256 cycles); one warp for both streams left it
            // idle for 700 of 1750 cycles a step, so each stream has its own.
            const int st = warp - kMmaWarp;
            const uint32_t ring_lo = __shfl_sync(kFull, (smem_addr(ring) >> 4) & 0x3FFFu, 0);
            const uint32_t q_lo = __shfl_sync(kFull, (smem_addr(qs) >> 4) & 0x3FFFu, 0);
            const uint32_t tm = __shfl_sync(kFull, tmem, 0);
            const uint32_t tS = tm + kColS + 128 * st, tO = tm + kColO + 128 * st;
            // The next ring position to wait for: every one in its turn, the other stream's too, and none is
            // free for the loader before both have had it (a parity wait must not miss a phase).
            RingPos<NS> seen;
            uint32_t ph = 0;   // of the stream's weights
            bool ok = true;
            for (int seg = 0; ok && walk.next(a, geo); ++seg) {
                const bool pair = __shfl_sync(kFull, sg.pair, 0) != 0;
                const int nb = __shfl_sync(kFull, sg.nb, 0);
                const int steps = pair ? nb : (nb + 1 - st) / 2;  // of this stream
                ok = warp_wait(q_full, seg & 1, abort_flag, err);
                if (ok && seg > 0) ok = warp_wait(o_free, (seg - 1) & 1, abort_flag, err);
                if (!ok) break;
                fence_after();
                int upto = 0;  // positions of the segment that have been waited for
                auto arrived = [&](int n) {  // the segment's first n tiles are there
                    for (; ok && upto < n; ++upto) {
                        ok = warp_wait(full + seen.slot, seen.phase, abort_flag, err);
                        if (ok && !pair) {  // a tile of the other stream: this one is done with it
                            bool is_v;
                            int j;
                            load_at(false, nb, upto, is_v, j);
                            if ((j & 1) != st && lane == 0) mbar_arrive(empty + seen.slot);
                            __syncwarp();
                        }
                        seen.advance(1);
                    }
                };
                // the slot of the segment's tile number n, of which `upto` have been waited for
                auto slot_at = [&](int n) { return (seen.slot + 2 * NS * 16 - (uint32_t)(upto - n)) % NS; };
                const uint32_t q0 = q_lo + (pair && st ? Z::kQ >> 4 : 0u);
                auto issue_s = [&](uint32_t kslot, bool last) {  // one lane
                    const uint32_t k0 = ring_lo + kslot * (Z::kSlot >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk / 4) * kHalf + (kk % 4) * 32) >> 4;
                        umma_ss(tS, desc_of(q0 + off, 16), desc_of(k0 + off, 16), id_s, kk != 0);
                    }
                    commit(s_full + st);
                    commit(empty + kslot);
                    if (last) commit(q_free);
                };
                auto issue_o = [&](uint32_t vslot, int hf, bool first) {  // one lane; a half of the keys
                    const uint32_t v0 = ring_lo + vslot * (Z::kSlot >> 4);
#pragma unroll
                    for (int kk = 0; kk < kKeys / 32; ++kk) {
                        const int k = hf * (kKeys / 32) + kk;
                        umma_ts(tO, tS + 8 * k, desc_of(v0 + (2048 >> 4) * k, kHalf), id_o, !first || k != 0);
                    }
                };
                if (steps == 0) {  // a split item of one block leaves stream 1 without a step
                    if (lane == 0) mbar_arrive(q_free);
                    __syncwarp();
                    arrived(2 * nb);
                    continue;
                }
                // Ring numbers of this stream's i-th tiles (load_at): K, and V behind it.
                auto num_k = [&](int i) { return pair ? 2 * i : (2 * i + st == 0 ? 0 : 2 * (2 * i + st) - 1); };
                auto num_v = [&](int i) { return pair ? 2 * i + 1 : (2 * i + st == nb - 1 ? 2 * nb - 1 : 2 * (2 * i + st) + 2); };
                arrived(num_k(0) + 1);
                if (!ok) break;
                uint32_t kslot = slot_at(num_k(0));
                fence_after();
                if (elect_one()) issue_s(kslot, steps == 1);
                __syncwarp();
                arrived(num_v(0) + 1);
                uint32_t vslot = slot_at(num_v(0));
                // Step i: the product with V, then the scores of step i + 1.  Waits and ring positions are
                // taken care of while the first half's products run.
                for (int i = 0; ok && i < steps; ++i) {
                    const bool more = i + 1 < steps;
                    ok = warp_wait(p_half + st, ph, abort_flag, err);
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) issue_o(vslot, 0, i == 0);
                    __syncwarp();
                    uint32_t vnext = 0;
                    if (more) {
                        arrived(num_k(i + 1) + 1);
                        kslot = slot_at(num_k(i + 1));
                    }
                    if (ok) ok = warp_wait(p_full + st, ph, abort_flag, err);
                    if (!ok) break;
                    ph ^= 1u;
                    fence_after();
                    if (elect_one()) {
                        issue_o(vslot, 1, false);
                        commit(empty + vslot);
                        if (more) issue_s(kslot, i + 2 == steps);
                        else commit(pv_done + st);
                    }
                    __syncwarp();
                    if (more) {
                        arrived(num_v(i + 1) + 1);
                        vnext = slot_at(num_v(i + 1));
                    }
                    vslot = vnext;
                }
                arrived(2 * nb);
            }
        } else {
            // -------------------------------------------------------- loads
            // Whole blocks by TMA (warp 0 of the two), queries and masked blocks by both.
            // Warp 0 alone waits for the slots to come free, position by position: a parity wait tells a
            // phase from the next one only, so whoever skipped positions could take an old phase for the
            // one it needs.  What the other warp is to fill with it it learns from `granted`.
            const int gw = warp - kLoadWarp;
            constexpr int CH = D / 8, RPI = 32 / CH, IT = 32 / RPI;  // chunks of a row, rows per pass, passes of 32 rows
            const int ch = lane % CH, sub = lane / CH;
            uint32_t pos = 0;
            bool ok = true;
            const int per = a.page < kKeys ? a.page : kKeys;  // tokens of a copy (use_tma: a power of two, 16 at least)
            // rows 32 qt .. 32 qt + 31 of a tile: `ptr` is lane's row (null: zeros)
            auto fill = [&](uint8_t *tile, int qt, const uint16_t *ptr) {
                const uint32_t t = smem_addr(tile) + (ch >> 3) * kHalf;
#pragma unroll 4
                for (int i = 0; i < IT; ++i) {
                    const int row = i * RPI + sub;
                    const uint64_t src = __shfl_sync(kFull, reinterpret_cast<uint64_t>(ptr), row);
                    cp_async16(t + swz(32 * qt + row, ch & 7),
                               reinterpret_cast<const uint4 *>(src ? src : reinterpret_cast<uint64_t>(a.q)) + ch, src ? 16 : 0);
                }
            };
            // once they are there: values that are not finite become 0; returns the rows that had one
            auto clean = [&](uint8_t *tile, int qt) -> uint32_t {
                uint32_t odd = 0;
                uint8_t *t = tile + (ch >> 3) * kHalf;
#pragma unroll 1
                for (int i = 0; i < IT; ++i) {
                    uint4 *at = reinterpret_cast<uint4 *>(t + swz(32 * qt + i * RPI + sub, ch & 7));
                    uint4 x = *at;
                    uint32_t *w = &x.x;
                    bool nf = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if ((w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xFFFF0000u, nf = true;
                        if ((w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0xFFFFu, nf = true;
                    }
                    const uint32_t ball = __ballot_sync(kFull, nf);
                    if (ball) {
                        if (nf) *at = x;
#pragma unroll
                        for (int k = 0; k < RPI; ++k)
                            if (ball >> (k * CH) & ((1u << CH) - 1u)) odd |= 1u << (i * RPI + k);
                    }
                }
                return odd;
            };
            for (int seg = 0; ok && walk.next(a, geo); ++seg) {
                if (seg > 0) ok = warp_wait(q_free, (seg - 1) & 1, abort_flag, err);
                if (!ok) break;
                Poison *po = poison + (seg & 1) * kQuarters;
                if (lane == 0)
                    for (int qt = gw; qt < kQuarters; qt += kLoadWarps) po[qt].n = 0;
                for (int q = gw; q < (sg.pair ? 2 : 1) * kQuarters; q += kLoadWarps) {
                    const int row0 = 32 * q + lane, rowi = sg.t * kAttnTcRows + row0, rank = rowi / a.group;
                    const uint16_t *ptr = nullptr;
                    if (row0 < sg.rows)
                        ptr = a.q + (int64_t)a.ws.order[sg.start + rank] * a.ldq +
                              (int64_t)(sg.h * a.group + (rowi - rank * a.group)) * D;
                    fill(qs + q / kQuarters * Z::kQ, q % kQuarters, ptr);
                }
                bool q_there = false;
                auto give_q = [&]() {  // once the queries have arrived
                    cp_async_wait_all();
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_full);
                    q_there = true;
                };
                if (gw != 0) give_q();
                for (int l = 0; ok && l < 2 * sg.nb; ++l) {
                    bool is_v;
                    int j;
                    load_at(sg.pair, sg.nb, l, is_v, j);
                    const int key = key_of(sg, j);
                    const bool masked = !seen_whole(sg, key), whole = !masked && use_tma;
                    if (whole && gw != 0) continue;
                    const uint32_t p = pos + l, slot = p % NS;
                    if (whole) {
                        // pages of the block, one per lane
                        int tok = 0;
                        int32_t page = 0;
                        if (lane * per < kKeys) page = (int32_t)page_of(a, sg.r, key + lane * per, tok);
                        if (!q_there && l >= 2) give_q();  // (the first tiles' copies go out while the queries come in)
                        if (p >= NS) ok = warp_wait(empty + slot, (p / NS - 1) & 1, abort_flag, err);
                        if (!ok) break;
                        const uint32_t dst = smem_addr(ring) + slot * Z::kSlot;
                        if (elect_one()) {
                            issued[slot] = p + 1;
                            mbar_arrive(full + slot, kLoadWarps - 1);
                            mbar_expect_tx(full + slot, Z::kSlot);
                        }
                        for (int i = 0; i * per < kKeys; ++i) {
                            const int pg = __shfl_sync(kFull, page, i), tk = __shfl_sync(kFull, tok, i);
                            if (elect_one()) {
#pragma unroll
                                for (int hf = 0; hf < D / 64; ++hf)
                                    tma_load_4d(dst + hf * kHalf + i * per * 128, is_v ? &vmap : &kmap, 64 * hf, tk, sg.h,
                                                pg, full + slot);
                            }
                            __syncwarp();
                        }
                        continue;
                    }
                    const uint16_t *ptr[kQuarters / kLoadWarps];
#pragma unroll
                    for (int i = 0; i < kQuarters / kLoadWarps; ++i) {
                        const int mine = key + 32 * (gw + i * kLoadWarps) + lane;
                        ptr[i] = nullptr;
                        if (mine >= sg.ctx) {
                            if (mine < sg.ctx + sg.cnt) {
                                const int64_t node = a.ws.order[sg.start + mine - sg.ctx];
                                ptr[i] = (is_v ? a.v + node * a.ldv : a.k + node * a.ldk) + sg.h * D;
                            }
                        } else if (mine >= sg.key_lo) {
                            int tok;
                            const int64_t pg = page_of(a, sg.r, mine, tok);
                            ptr[i] = (is_v ? a.cv : a.ck) + pg * a.page_stride + tok * a.token_stride + sg.h * a.head_stride;
                        }
                    }
                    if (gw == 0) {
                        if (!q_there) give_q();
                        if (p >= NS) ok = warp_wait(empty + slot, (p / NS - 1) & 1, abort_flag, err);
                        if (!ok) break;
                        __threadfence_block();
                        if (lane == 0) *granted = p + 1;
                        __syncwarp();
                    } else {
                        ok = warp_wait_count(granted, p + 1, abort_flag, err);
                        if (!ok) break;
                    }
                    uint8_t *tile = ring + slot * Z::kSlot;
#pragma unroll 1
                    for (int i = 0; i < kQuarters / kLoadWarps; ++i) fill(tile, gw + i * kLoadWarps, ptr[i]);
                    cp_async_wait_all();
                    if (is_v && masked) {
                        __syncwarp();
                        for (int qt = gw; qt < kQuarters; qt += kLoadWarps) {
                            const uint32_t odd = clean(tile, qt);
                            if (odd && lane == 0 && po[qt].n < kPoison) {
                                po[qt].key[po[qt].n] = key;
                                po[qt].rows[po[qt].n] = odd;
                                po[qt].n += 1;
                            }
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full + slot);
                }
                if (ok && !q_there) give_q();
                pos += 2 * sg.nb;
            }
        }
    }
    // every copy and every MMA that was issued has completed before TMEM and shared memory go (the
    // copies of a CTA that did not give up have all been read)
    __syncthreads();
    if (warp == kLoadWarp && lane == 0 && *abort_flag)
        for (int i = 0; i < NS; ++i)
            if (issued[i]) mbar_drain(full + i, (issued[i] - 1) / NS & 1, err);
    if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        if (elect_one()) commit(fin);
        __syncwarp();
    }
    if (warp == kMmaWarp) {
        mbar_drain(fin, 0, err);
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// The driver's tensor-map encoder, looked up once.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// The cache as [page][head][token][dim], a box of 64 columns of the tokens of
// one page (at most a block's).  False where the layout has no tensor map;
// every block is then gathered.
bool cache_map(const AttnArgs &a, const uint16_t *p, int D, CUtensorMap *map) {
    const auto enc = encoder();
    if (!enc || a.page_shift < 4 || a.pages < 1 || !p) return false;
    const int64_t st[3] = {a.token_stride, a.head_stride, a.page_stride};
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        if (st[i] <= 0 || st[i] * 2 >= (1LL << 40)) return false;
        strides[i] = (cuuint64_t)st[i] * 2;
    }
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.page, (cuuint64_t)a.H, (cuuint64_t)a.pages};
    const cuuint32_t box[4] = {64, (cuuint32_t)(a.page < kKeys ? a.page : kKeys), 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool CAP>
cudaError_t launch_tc(const AttnArgs &a, int max_ctas, bool overlap, cudaStream_t s) {
    CUtensorMap km{}, vm{};
    const int use_tma = cache_map(a, a.ck, D, &km) && cache_map(a, a.cv, D, &vm);
    const size_t smem = tc_smem_bytes<D>();
    cudaError_t e = cudaFuncSetAttribute(k_attn_tc<D, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int grid = max_ctas > 0 && max_ctas < a.G ? max_ctas : a.G;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_attn_tc<D, CAP>, a, km, vm, use_tma);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, int D, int max_ctas, bool overlap, cudaStream_t s) {
    const bool cap = a.softcap > 0.f;
    if (D == 64) return cap ? launch_tc<64, true>(a, max_ctas, overlap, s) : launch_tc<64, false>(a, max_ctas, overlap, s);
    return cap ? launch_tc<128, true>(a, max_ctas, overlap, s) : launch_tc<128, false>(a, max_ctas, overlap, s);
}

}  // namespace w12
