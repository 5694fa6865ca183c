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
// Step u of an item belongs to stream u & 1.  Each stream has a warp that issues its
//     S = Q K^T        (M = 128 rows, N = 128 keys, both operands in shared memory)
//     O += P V         (P in TMEM over the first half of S, V in shared memory, MN-major)
// and four softmax warps: thread = row = TMEM lane, so maxima and sums need no
// exchange.  The streams take turns at the tensor cores, so one's products run
// under the other's softmax.  The reference of a row's weights is its maximum
// when it was last raised: O is rescaled only when a block's maximum exceeds it
// by more than 8 (a factor 256 of FP32's range; to put the rescale off like this
// is a published technique of attention kernels), which after the first blocks
// almost never happens.  Weights are rounded to BF16 for the product, as every
// operand of it is; their sum is taken before.
//
// Everything arrives by TMA: the cache in a ring of [128 keys x D] tiles, a copy
// per page and 64 columns; the nodes' own keys and values, which may lie anywhere
// in the call's order, four rows at a time (gather4), or 32 where they follow
// one another; the queries, the heads of a group of one node, or of several, at
// a time.  (Gathering rows with cp.async was limited by the loads that an SM
// keeps outstanding: 4000 cycles a tile, 19000 for the queries of an item, with
// HBM busy.)  Values of a block with anything masked (the end of the cache, the
// tree, the window's edge) pass through one warp first: rows that nobody sees
// become zeros, and values that are not finite are left out of the product and
// added at the end to the rows that see them, so that 0 * Inf cannot reach a row.
//
// What bounds it.  A pair block (D = 128) is 32 MMAs of 64 cycles, 2048 cycles,
// and 1024 for the exponentials of a quarter of an SM; its tiles take 1500 at
// an SM's share of HBM.  It takes 3300 to 3600: a stream's chain is 1100 cycles
// of products, 1500 of softmax (400 to read the scores and find the maximum,
// 900 for the weights: one warp alone keeps neither the exponential unit nor
// the others full) and 600 of barriers and of instructions that wait for their
// turn.  Measured and left: 16 softmax warps, half a row each (3200 cycles a
// pair block, 225 us for 8 x 256 nodes over 8k, but slower for the smaller
// calls and 218 instead of 208 for 64 nodes over 128k: fewer registers for the
// loads); weights against the last block's reference while the maximum is
// taken (263 instead of 248 then).  The code's size counts: the softmax loop of
// half the instructions made up for reading the scores twice.
//
// Times of ten calls in one CUDA graph.  8 x 256 nodes over up to 8192 tokens,
// 40 heads of 128 over 8 (234 GFLOP): 233-237 us, 1.0 PFLOP/s, tensor pipe 51%
// busy, 226 with the plan of the call before.  64 nodes over 131072 (172
// GFLOP, 538 MB): 205-209 us; its 320 rows are two items, so the cache is read
// twice, 1.07 GB at 5.2 TB/s.
//
// Every wait is bounded (about a second): a CTA that gives up sets the
// workspace's timeout word, drains its copies and MMAs and frees its TMEM.
#include <cstdint>
#include <cuda_runtime.h>

#include "w12_attn.cuh"
#include "w12_tc.cuh"
#include "w12_tmap.cuh"

namespace w12 {
namespace {

using namespace tc;

constexpr int kRows = 128;     // of a stream
constexpr int kKeys = kAttnTcBlock;  // of a block
constexpr int kMmaWarp = 0, kLoadWarp = 2, kSoftWarp = 4, kSoftWarps = 8;  // MMA: one warp per stream
constexpr int kTcThreads = 32 * (kSoftWarp + kSoftWarps);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 per stream
constexpr float kLazy = 8.0f;               // log2 of the growth that an unscaled O may carry
constexpr int kNodeRows = 32;               // nodes of a copy, where they follow one another
constexpr int kSegs = 4;                    // segments that the loads may be ahead
constexpr int kPoison = 8;                  // masked blocks of a segment (at most 3 at the window's edge, 3 at the end)

template <int D>
struct TcSizes {
    static constexpr uint32_t kSlot = kKeys * D * 2;
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr uint32_t kQ = kRows * D * 2;
};

struct Poison {  // masked blocks with values that are not finite: the first key, and the rows that have one
    int n;
    int key[kPoison];
    uint32_t rows[kPoison][kKeys / 32];
};

// Tensor maps of a call: the cache's pages, the nodes' rows, the queries (all heads of a group, one head).
// Where a request's nodes follow one another in the call, several rows (nb*, qb: kNodeRows rows, q_nodes nodes) go
// in one copy.
struct TcMaps {
    CUtensorMap ck, cv, nk, nv, qg, q1, kb, vb, qb;
};
static_assert(sizeof(TcMaps) == sizeof(AttnTcMaps), "handed through the launch interface as bytes");

template <int D>
constexpr size_t tc_smem_bytes() {
    return 1024 + (size_t)TcSizes<D>::kSlots * TcSizes<D>::kSlot + 2 * TcSizes<D>::kQ + 8 * (3 * TcSizes<D>::kSlots + 15) +
           2 * sizeof(Poison) + 16 + 4 * (TcSizes<D>::kSlots + 1) +
           kSegs * (sizeof(Seg) + 16) + sizeof(Seg) + sizeof(SegWalk);
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

__device__ __forceinline__ int tree_key(int ctx) { return (ctx + kKeys - 1) & -kKeys; }  // the first node's number

// bits below n
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Which of the keys [key, key + 32) a row sees: cached ones from lo on, and
// the ranks of its mask.
__device__ __forceinline__ uint32_t seen_word(int key, int ctx, int lo, const uint32_t *mask) {
    uint32_t w = below(ctx - key) & ~below(lo - key);
    const int rk = key - tree_key(ctx);  // rank of the first key
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
                                                           const __grid_constant__ TcMaps maps) {
    using Z = TcSizes<D>;
    constexpr int NS = Z::kSlots;
    constexpr uint32_t kHalf = kKeys * 128;  // 64 columns of a tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = base, *qs = base + NS * Z::kSlot;
    Seg *segs = reinterpret_cast<Seg *>(qs + 2 * Z::kQ);  // [kSegs], and one of no work
    SegWalk &walk = *reinterpret_cast<SegWalk *>(segs + kSegs + 1);
    uint64_t *full = reinterpret_cast<uint64_t *>(&walk + 1);
    uint64_t *empty = full + NS, *q_full = empty + NS, *q_free = q_full + 1, *s_full = q_free + 1, *p_full = s_full + 2,
             *p_half = p_full + 2, *pv_done = p_half + 2, *o_free = pv_done + 2, *ml_ready = o_free + 1;
    uint64_t *fin = ml_ready + 1;  // every MMA of the CTA has completed
    uint64_t *turn = fin + 1;      // [2]: the other stream's products are queued
    uint64_t *seg_full = turn + 2, *seg_free = seg_full + kSegs;
    uint64_t *raw = seg_free + kSegs;  // [NS]: values of a masked block, before they are looked over
    Poison *poison = reinterpret_cast<Poison *>(raw + NS);  // [2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(poison + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    uint32_t *issued = tmem_slot + 2;  // [NS + 1]: copies last handed to the TMA unit for a slot, for Q: 1 | parity << 1 | raw << 2

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        Seg none{};  // a block of no keys before the first one, a row
        none.nb = 1, none.key0 = -kKeys, none.lo_max = -2 * kKeys, none.rows = 1;
        segs[kSegs] = none;
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(raw + i, 1);
            mbar_init(empty + i, 2);  // both streams are done with it
            issued[i] = 0;
        }
        issued[NS] = 0;
        mbar_init(q_full, 1);
        mbar_init(q_free, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(p_half + i, 4);
            mbar_init(pv_done + i, 1);
            mbar_init(turn + i, 1);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(seg_full + i, 1);
            mbar_init(seg_free + i, kTcThreads / 32 - 1);
        }
        mbar_init(o_free, kSoftWarps);
        mbar_init(ml_ready, kSoftWarps);
        mbar_init(fin, 2);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == kLoadWarp && lane == 0) {
        prefetch_tmap(&maps.ck);
        prefetch_tmap(&maps.cv);
        prefetch_tmap(&maps.qg);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    int32_t *err = a.ws.timeout;
    // While the plan is made, the loading warps go through their code once without loading: a CTA's first tile
    // was asked for 7000 cycles after the plan, most of them spent on fetching instructions (256 nodes of 8
    // requests: 59.5 -> 58.1 us; 3 x 200 chained: 41.5 -> 41.0).
    const bool loads = warp >= kLoadWarp && warp < kSoftWarp;
    if (!loads) {
        grid_dep_wait();
        grid_dep_launch();
    }

    // The launch's registers (168 x 384) are split anew, 200 x 256 + 104 x 128, per warpgroup.
    // The ring's loader walks the CTA's segments and hands them on through shared memory (the registers are
    // for the scores): a warp's own walk cost it 2000 cycles a segment.
    int seg_at = 0;
    uint32_t seg_ph = 0;
    auto next_seg = [&]() { return warp_wait(seg_full + seg_at, seg_ph, abort_flag, err) && segs[seg_at].nb > 0; };
    auto done_seg = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_free + seg_at);
        if (++seg_at == kSegs) seg_at = 0, seg_ph ^= 1u;
    };
    if (warp >= kSoftWarp) {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int st = (warp - kSoftWarp) >> 2, quarter = warp & 3;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t tS = lane_base + kColS + 128 * st;
        const float sl2 = a.scale * kLog2e, cap2 = CAP ? 2.0f * kLog2e * a.scale / a.softcap : 0.f,
                    capl = CAP ? a.softcap * kLog2e : 0.f;
        uint32_t n_s = 0, n_pv[2] = {0, 0}, n_ml = 0;
        int seg = 0;
        for (; next_seg(); ++seg, done_seg()) {
            const Seg &sg = segs[seg_at];
            const int row0 = (sg.pair ? st * kRows : 0) + 32 * quarter + lane;  // row of the item
            const int rowi = sg.t * kAttnTcRows + row0, rank = rowi / a.group;
            const bool live = row0 < sg.rows;
            const int at = sg.start + (live ? rank : 0);
            const uint32_t *mrow = a.ws.mask + (int64_t)at * kMaskWords;
            const int lo_key = a.window > 0 ? sg.ctx + a.ws.depth[at] - a.window : 0;
            const int node = a.ws.order[at];
            asm volatile("prefetch.global.L1 [%0];" ::"l"(mrow));
            float m = -INFINITY, l = 0.f;  // reference maximum (log2 domain), sum
            bool ok = true;
            // One step: the row's 128 scores of S(u) become weights, which go over the first half of S.  They
            // are read twice, for the maximum and for the weights, 64 at a time.
            auto raise = [&](float top, bool first) {  // the reference, if a block's maximum asks for it
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
            };
            auto hand_over = [&](uint64_t *bar) {  // weights (and O) written so far
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + st);
            };
            auto step = [&](bool first) {
                float va[32], vb[32];
                tmem_ld32_start(tS, va);
                tmem_ld32_start(tS + 32, vb);
                float t0 = -INFINITY, t1 = t0, t2 = t0, t3 = t0;
                auto top_of = [&](float *x) {
                    tmem_ld32_wait(x);
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        t0 = max3(t0, x[j], x[j + 1]);
                        t1 = max3(t1, x[j + 2], x[j + 3]);
                        t2 = max3(t2, x[j + 4], x[j + 5]);
                        t3 = max3(t3, x[j + 6], x[j + 7]);
                    }
                };
#pragma unroll 1
                for (int c = 64; c < 192; c += 64) {  // the last two loads are the first two again
                    top_of(va);
                    tmem_ld32_start(tS + (c & 64), va);
                    top_of(vb);
                    tmem_ld32_start(tS + (c & 64) + 32, vb);
                }
                raise(fmaxf(max3(t0, t1, t2), t3), first);
                const float m0 = m == -INFINITY ? 0.f : m;
                const float2 sc = make_float2(sl2, sl2), mm = make_float2(-m0, -m0);
                float2 s0 = make_float2(0.f, 0.f), s1 = s0;
                auto weights = [&](float *x, uint32_t to) {
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float2 y = make_float2(x[j], x[j + 1]);
                        if (CAP) y = make_float2(cap_score(y.x, cap2, capl) - m0, cap_score(y.y, cap2, capl) - m0);
                        else y = fma2(y, sc, mm);
                        y.x = exp2_approx(y.x);
                        y.y = exp2_approx(y.y);
                        p[j / 2] = pack_bf16(y.x, y.y);
                        if (j & 2) s1 = add2(s1, y);
                        else s0 = add2(s0, y);
                    }
                    tmem_st16(to, p);
                };
                uint64_t *bar = p_half;
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    tmem_ld32_wait(va);
                    tmem_ld32_wait(vb);
                    weights(va, tS + c / 2);
                    if (c == 0) tmem_ld32_start(tS + 64, va);
                    weights(vb, tS + c / 2 + 16);
                    if (c == 0) tmem_ld32_start(tS + 96, vb);
                    hand_over(bar);
                    bar = p_full;
                }
                s0 = add2(s0, s1);
                l += s0.x + s0.y;
            };
            // The same for a block with something masked: a few of them per item, so the code is kept short
            // rather than fast; a kernel this size starts with cold instruction caches.  (One body for both
            // left the compiler less to overlap: 257 us instead of 234 for 8 x 256 nodes over 8k.)
            auto step_masked = [&](bool first, int key) {
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const uint32_t see = seen_word(key + 32 * c, sg.ctx, lo_key, mrow);
                    float x[32];
                    tmem_ld32(tS + 32 * c, x);
#pragma unroll
                    for (int j = 0; j < 32; ++j) top = fmaxf(top, see >> j & 1u ? x[j] : -INFINITY);
                }
                raise(top, first);
                const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    const uint32_t see = seen_word(key + 32 * c, sg.ctx, lo_key, mrow);
                    float x[32];
                    uint32_t p[16];
                    tmem_ld32(tS + 32 * c, x);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        x[j] = exp2_approx(CAP ? cap_score(x[j], cap2, capl) - m0 : fmaf(x[j], sl2, -m0));
                        x[j] = see >> j & 1u ? x[j] : 0.f;
                        l += x[j];
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
                    tmem_st16(tS + 16 * c, p);
                    if (c & 1) hand_over(c == 1 ? p_half : p_full);
                }
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
                    if (whole) step(u < 2);
                    else step_masked(u < 2, key);
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
            const int head = sg.h * a.group + (rowi - rank * a.group);
            uint16_t *orow = a.o + (int64_t)node * a.ldo + (int64_t)head * D;
            const int64_t prow = (int64_t)sg.slot * kAttnTcRows + row0;
            // neighbouring lanes (rows) write neighbouring addresses
            float *part = a.ws.part + ((int64_t)sg.slot * (D / 4) * kAttnTcRows + row0) * 4;
            const Poison &po = poison[seg & 1];
            const int n_odd = po.n;
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
                for (int i = 0; i < n_odd; ++i)
                    for (int g = 0; g < kKeys / 32; ++g)
                        for (uint32_t rest = po.rows[i][g]; rest; rest &= rest - 1) {
                            const int key = po.key[i] + 32 * g + __ffs(rest) - 1, rk = key - tree_key(sg.ctx);
                            if (!(seen_word(key, sg.ctx, lo_key, mrow) & 1u)) continue;
                            const uint16_t *vr;
                            if (rk >= 0) {
                                vr = a.v + (int64_t)a.ws.order[sg.start + rk] * a.ldv + sg.h * D;
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
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
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
            bool mine = st == 0;  // the turn
            uint32_t turn_ph = 0;
            bool ok = true;
            for (int seg = 0; ok && next_seg(); ++seg, done_seg()) {
                const Seg &sg = segs[seg_at];
                const bool pair = __shfl_sync(kFull, sg.pair, 0) != 0;
                const int nb = __shfl_sync(kFull, sg.nb, 0);
                const int steps = pair ? nb : (nb + 1 - st) / 2;  // of this stream
                const int other = pair ? nb : (nb + st) / 2;      // of the other
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
                uint32_t vslot = 0;
                // Step i: the product with V, then the scores of step i + 1.  Waits and ring positions are
                // taken care of while the first half's products run.
                for (int i = -1; ok && i < steps; ++i) {
                    const bool more = i + 1 < steps;
                    if (i >= 0) {
                        ok = warp_wait(p_half + st, ph, abort_flag, err);
                        if (!ok) break;
                        fence_after();
                        if (elect_one()) issue_o(vslot, 0, i == 0);
                        __syncwarp();
                    }
                    if (more) arrived(num_k(i + 1) + 1);
                    const uint32_t kslot = slot_at(num_k(i + 1));
                    if (ok && i >= 0) {
                        ok = warp_wait(p_full + st, ph, abort_flag, err);
                        if (ok && !mine) {
                            ok = warp_wait(turn + st, turn_ph, abort_flag, err);
                            turn_ph ^= 1u;
                        }
                        ph ^= 1u;
                    }
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) {
                        if (i >= 0) {
                            issue_o(vslot, 1, false);
                            commit(empty + vslot);
                        }
                        if (more) issue_s(kslot, i + 2 == steps);
                        else commit(pv_done + st);
                    }
                    __syncwarp();
                    if (i >= 0) {
                        mine = st == 0 && i >= other;
                        if (!mine && lane == 0) mbar_arrive(turn + (st ^ 1));
                    }
                    if (more) {
                        arrived(num_v(i + 1) + 1);
                        vslot = slot_at(num_v(i + 1));
                    }
                }
                arrived(2 * nb);
            }
        } else {
            // -------------------------------------------------------- loads
            // Copies are issued by many lanes at once, each with coordinates of its own: what a single warp
            // spends on its instructions is on the path of every tile (with one lane issuing in a loop a
            // tile took 2000 cycles, an item's queries 20000 and more).
            constexpr int HB = D / 64;                                                   // copies across a row
            const int per_sh = a.page_shift < 0 ? 0 : a.page_shift < 7 ? a.page_shift : 7;  // 2^per_sh tokens of a copy
            const int lane_c = lane / HB, lane_x = 64 * (lane % HB);                     // this lane's copy of a round, and its columns
            const uint32_t lane_d = (lane % HB) * kHalf;
            constexpr int kRound = 32 / HB;                                              // copies of a round
            bool ok = true;
            if (warp == kLoadWarp) {
                // The ring.  This warp waits for every slot in its turn: a parity wait tells a phase from the
                // next one only.
                RingPos<NS> at;
                uint32_t laps = 0, raw_phase = 0;  // positions used (up to NS); one bit per slot
                const uint32_t ring_a = smem_addr(ring);
                // The first segment is ready in the workspace; the walk begins when it is needed, behind the
                // first tiles.
                const uint4 *ready = reinterpret_cast<const uint4 *>(a.ws.range + blockIdx.x);
                bool first = true, begun = false;
                for (int seg = -1;; ++seg) {
                    const bool dry = seg < 0;
                    if (seg == 0) {
                        grid_dep_wait();
                        at = RingPos<NS>();
                        laps = 0;
                        if (lane < sizeof(Seg) / 16) reinterpret_cast<uint4 *>(segs)[lane] = ready[lane];
                        __syncwarp();
                        first = segs[0].nb > 0;
                        if (first && lane == 0) mbar_arrive(seg_full);
                    }
                    bool there = true;
                    if (seg > 0 || !first) {
                        const Geometry geo{kAttnTcRows, kKeys, kRows, kAttnTcPair, kAttnTcOne, kAttnTcBlock, *a.ws.extra};
                        if (!begun && lane == 0) {
                            walk.begin(a, geo);
                            if (first) walk.more = 1;
                        }
                        begun = true;
                        there = walk.next(a, geo);
                        if (seg >= kSegs) ok = warp_wait(seg_free + seg_at, seg_ph ^ 1u, abort_flag, err);
                        if (!ok) break;
                        if (!there && lane == 0) walk.sg.nb = 0;
                        __syncwarp();
                        if (lane < sizeof(Seg) / 16)
                            reinterpret_cast<uint4 *>(segs + seg_at)[lane] = reinterpret_cast<const uint4 *>(&walk.sg)[lane];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(seg_full + seg_at);
                    }
                    const Seg &sg = segs[dry ? kSegs : seg_at];
                    if (!dry && ++seg_at == kSegs) seg_at = 0, seg_ph ^= 1u;
                    if (!there) break;
                    const int nb = sg.nb, key0 = sg.key0, lo_max = sg.lo_max, ctx = sg.ctx, key_lo = sg.key_lo, h = sg.h;
                    const int cnt = sg.cnt, tree0 = tree_key(ctx), r = sg.r;
                    const bool pair = sg.pair;
                    const int32_t *order = a.ws.order + sg.start;
                    const bool seq = sg.node0 >= 0;  // the nodes follow one another from node0
                    const int node0 = sg.node0;
                    const bool one_round = kKeys >> per_sh <= kRound;
                    // this lane's page of the block at `key` (one round), asked for a tile ahead
                    auto ask = [&](int key) -> int {
                        const int k = key + (lane_c << per_sh);
                        int tok;
                        return k >= key_lo - (1 << per_sh) && k >= 0 && k < ctx ? (int)page_of(a, r, k, tok) : 0;
                    };
                    int page_k = one_round ? ask(key0) : 0, page_v = page_k;
                    for (int l = 0; ok && l < 2 * nb; ++l) {
                        bool is_v;
                        int j;
                        load_at(pair, nb, l, is_v, j);
                        const int key = key0 + j * kKeys;
                        const bool tree = key >= tree0, look = is_v && (key < lo_max || key + kKeys > ctx);
                        // first and last copy: of keys that some row may see
                        const int end = tree ? cnt - (key - tree0) : ctx - key, keys = end < kKeys ? end : kKeys;
                        const int sh = tree ? (seq ? 5 : 2) : per_sh;
                        const int c0 = tree || key >= key_lo ? 0 : (key_lo - key) >> sh,
                                  c1 = dry ? 0 : (keys + (1 << sh) - 1) >> sh;
                        int n0 = 0, n1 = 0, n2 = 0, n3 = 0;
                        if (tree && !seq && lane_c < c1) {  // past the last node the last one again: nobody sees those rows
                            const int rk = key - tree0 + 4 * lane_c;
                            n0 = order[rk], n1 = order[min(rk + 1, cnt - 1)], n2 = order[min(rk + 2, cnt - 1)],
                            n3 = order[min(rk + 3, cnt - 1)];
                        }
                        if (laps == NS) ok = warp_wait(empty + at.slot, at.phase ^ 1u, abort_flag, err);
                        else ++laps;
                        if (!ok) break;
                        uint64_t *bar = (look ? raw : full) + at.slot;
                        const uint32_t dst = ring_a + at.slot * Z::kSlot + lane_d;
                        if (elect_one() && !dry) {
                            issued[at.slot] = look ? 5u | (raw_phase >> at.slot & 1u) << 1 : 1u | at.phase << 1;
                            mbar_expect_tx(bar, (uint32_t)(c1 - c0) << sh << (D == 128 ? 8 : 7));
                        }
                        __syncwarp();
                        if (look) raw_phase ^= 1u << at.slot;
                        if (tree && seq) {
                            if (lane_c < c1)
                                tma_load_2d(dst + lane_c * (kNodeRows * 128), is_v ? &maps.vb : &maps.kb, h * D + lane_x,
                                            node0 + key - tree0 + lane_c * kNodeRows, bar);
                        } else if (tree) {
                            const CUtensorMap *map = is_v ? &maps.nv : &maps.nk;
                            for (int c = lane_c; c < c1; c += kRound) {
                                if (c >= kRound) {
                                    const int rk = key - tree0 + 4 * c;
                                    n0 = order[rk], n1 = order[min(rk + 1, cnt - 1)], n2 = order[min(rk + 2, cnt - 1)],
                                    n3 = order[min(rk + 3, cnt - 1)];
                                }
                                tma_gather4(dst + c * 512, map, h * D + lane_x, n0, n1, n2, n3, bar);
                            }
                        } else {
                            const CUtensorMap *map = is_v ? &maps.cv : &maps.ck;
                            for (int c = lane_c; c < c1; c += kRound) {
                                const int k = key + (c << per_sh);
                                int pg = is_v ? page_v : page_k, tok = k & (a.page - 1);
                                if (!one_round) pg = (int)page_of(a, r, k, tok);
                                if (c >= c0) tma_load_4d(dst + (c << per_sh) * 128, map, lane_x, tok, h, pg, bar);
                            }
                            if (one_round) {
                                if (is_v) page_v = ask(key + kKeys);
                                else page_k = ask(key + kKeys);
                            }
                        }
                        __syncwarp();
                        at.advance(1);
                    }
                }
            } else {
                // The queries, and the values of masked blocks.
                uint32_t pos = 0, raw_phase = 0;  // one bit per slot
                for (int seg = -1; ok; ++seg) {
                    const bool dry = seg < 0;
                    if (seg == 0) grid_dep_wait();
                    if (seg > 0) done_seg();
                    if (!dry && !next_seg()) break;
                    const Seg &sg = segs[dry ? kSegs : seg_at];
                    const int nb = sg.nb, key0 = sg.key0, lo_max = sg.lo_max, ctx = sg.ctx, key_lo = sg.key_lo, h = sg.h;
                    const int cnt = sg.cnt, tree0 = tree_key(ctx), group = a.group;
                    const bool pair = sg.pair;
                    // Q of the last segment and the list of the one before it are no longer read
                    if (seg > 0) ok = warp_wait(q_free, (seg - 1) & 1, abort_flag, err);
                    if (!ok) break;
                    Poison &po = poison[seg & 1];
                    if (lane == 0) po.n = 0;
                    if (a.stall) continue;  // (tests: the wait for the queries runs out)
                    if (elect_one() && !dry) {
                        issued[NS] = 1u | (uint32_t)(seg & 1) << 1;
                        mbar_expect_tx(q_full, (uint32_t)sg.rows * (D * 2));
                    }
                    __syncwarp();
                    const int first_row = sg.t * kAttnTcRows, rank0 = first_row / group, rows = sg.rows;
                    const int g0 = first_row - rank0 * group;  // the item may begin inside a node's group of heads
                    const uint32_t q_a = smem_addr(qs) + lane_d;
                    // nodes [i, i + q_nodes) of the item by one copy where they follow one another, their heads' rows
                    // are all in the item and in one of its tiles; else node by node
                    const int node0 = sg.node0, many = node0 >= 0 ? a.q_nodes : 1;
                    const int32_t *order = a.ws.order + sg.start + rank0;
                    auto node_at = [&](int i) { return node0 >= 0 ? node0 + rank0 + i : i * group - g0 < rows ? order[i] : 0; };
                    int ahead = node_at(lane_c * many);  // a load ahead: the loop waits for none of its own
                    for (int i0 = lane_c * many; i0 * group - g0 < rows; i0 += kRound * many) {
                        const int rb0 = i0 * group - g0, rb1 = rb0 + many * group;
                        const int first = ahead;
                        ahead = node_at(i0 + kRound * many);
                        if (dry) continue;
                        if (many > 1 && rb0 >= 0 && rb1 <= rows && rb0 / kRows == (rb1 - 1) / kRows) {
                            tma_load_3d(q_a + rb0 / kRows * Z::kQ + rb0 % kRows * 128, &maps.qb, lane_x, h * group, first,
                                        q_full);
                            continue;
                        }
                        for (int i = i0; i < i0 + many && i * group - g0 < rows; ++i) {  // node rank0 + i
                            const int node = first + (i - i0);
                            const int b0 = i * group - g0, ra = b0 < 0 ? 0 : b0, rb = b0 + group < rows ? b0 + group : rows;
                            const int head = h * group;
                            if (rb - ra == group && ra / kRows == (rb - 1) / kRows && group <= 256) {
                                tma_load_3d(q_a + ra / kRows * Z::kQ + ra % kRows * 128, &maps.qg, lane_x, head, node, q_full);
                            } else {
                                for (int x = ra; x < rb; ++x)
                                    tma_load_3d(q_a + x / kRows * Z::kQ + x % kRows * 128, &maps.q1, lane_x, head + x - b0,
                                                node, q_full);
                            }
                        }
                    }
                    __syncwarp();
                    if (dry) continue;
                    for (int l = 0; ok && l < 2 * nb; ++l) {
                        bool is_v;
                        int j;
                        load_at(pair, nb, l, is_v, j);
                        const int key = key0 + j * kKeys;
                        if (!is_v || (key >= lo_max && key + kKeys <= ctx)) continue;
                        const uint32_t slot = (pos + l) % NS;
                        ok = warp_wait(raw + slot, raw_phase >> slot & 1u, abort_flag, err);
                        if (!ok) break;
                        raw_phase ^= 1u << slot;
                        // rows [r0, r1) of the tile hold keys; zeros in the others
                        const bool tree = key >= tree0;
                        const int r0 = tree || key >= key_lo ? 0 : key_lo - key;
                        const int r1 = tree ? cnt - (key - tree0) : ctx - key;
                        constexpr int CH = D / 8, RPI = 32 / CH;
                        const int ch = lane % CH, sub = lane / CH;
                        uint8_t *t = ring + slot * Z::kSlot + (ch >> 3) * kHalf;
                        // eight rows at a time (their swizzle repeats); 0 * x adds up to NaN if any x is not finite
                        constexpr int PASS = 8 / RPI;
                        uint32_t acc = 0;
#pragma unroll 2
                        for (int r8 = 0; r8 < kKeys; r8 += 8) {
#pragma unroll
                            for (int i = 0; i < PASS; ++i) {
                                const int rr = i * RPI + sub, r = r8 + rr;
                                uint4 *at = reinterpret_cast<uint4 *>(t + r8 * 128 + swz(rr, ch & 7));
                                if (r >= r0 && r < r1) {
                                    const uint4 x = *at;
                                    acc = fma_bf16x2(x.x, 0u, acc);
                                    acc = fma_bf16x2(x.y, 0u, acc);
                                    acc = fma_bf16x2(x.z, 0u, acc);
                                    acc = fma_bf16x2(x.w, 0u, acc);
                                } else {
                                    *at = make_uint4(0, 0, 0, 0);
                                }
                            }
                        }
                        if (__any_sync(kFull, (acc & 0x7F80u) == 0x7F80u || (acc & 0x7F800000u) == 0x7F800000u)) {
                            const int slot_n = po.n;
                            const bool room = slot_n < kPoison;
#pragma unroll 1
                            for (int i = 0; i < kKeys / RPI; ++i) {
                                const int r = i * RPI + sub;
                                uint4 *at = reinterpret_cast<uint4 *>(t + swz(r, ch & 7));
                                uint4 x = *at;
                                uint32_t *w = &x.x;
                                bool nf = false;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if ((w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xFFFF0000u, nf = true;
                                    if ((w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0xFFFFu, nf = true;
                                }
                                const uint32_t ball = __ballot_sync(kFull, nf);
                                if (nf) *at = x;
                                if (lane == 0 && room) {
                                    uint32_t rows = 0;
#pragma unroll
                                    for (int k = 0; k < RPI; ++k)
                                        if (ball >> (k * CH) & ((1u << CH) - 1u)) rows |= 1u << k;
                                    uint32_t &out = po.rows[slot_n][i * RPI / 32];
                                    out = (i * RPI % 32 == 0 ? 0u : out) | rows << (i * RPI % 32);
                                }
                            }
                            if (lane == 0 && room) {
                                po.key[slot_n] = key;
                                po.n = slot_n + 1;
                            }
                        }
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full + slot);
                    }
                    pos += 2 * nb;
                }
            }
        }
    }
    // every copy and every MMA that was issued has completed before TMEM and shared memory go (the
    // copies of a CTA that did not give up have all been read)
    __syncthreads();
    if (warp == kLoadWarp && lane == 0 && *abort_flag)
        for (int i = 0; i <= NS; ++i)
            if (issued[i]) mbar_drain(i == NS ? q_full : (issued[i] & 4 ? raw : full) + i, issued[i] >> 1 & 1, err);
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

template <int D, bool CAP>
cudaError_t launch_tc(const AttnArgs &a, const TcMaps &maps, int max_ctas, bool overlap, cudaStream_t s) {
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
    return cudaLaunchKernelEx(&cfg, k_attn_tc<D, CAP>, a, maps);
}

}  // namespace

bool attn_tc_maps(const AttnArgs &a, int D, AttnTcMaps *out) {
    TcMaps &m = *reinterpret_cast<TcMaps *>(out);
    const int per = a.page_shift < 0 ? 1 : a.page < kKeys ? a.page : kKeys;
    const int64_t cd[4] = {D, a.page, a.H, a.pages}, cs[3] = {a.token_stride, a.head_stride, a.page_stride};
    const int cb[4] = {64, per, 1, 1};
    const int64_t nd[2] = {(int64_t)a.H * D, a.n}, ks[1] = {a.ldk}, vs[1] = {a.ldv};
    const int nb[2] = {64, 1};
    const int64_t qd[3] = {D, a.Hq, a.n}, qst[2] = {D, a.ldq};
    const int gb[3] = {64, a.group < 256 ? a.group : 256, 1}, ob[3] = {64, 1, 1};
    const int rb[2] = {64, kNodeRows}, mb[3] = {64, gb[1], a.q_nodes};
    return encode_tmap(&m.kb, a.k, 2, nd, ks, rb) && encode_tmap(&m.vb, a.v, 2, nd, vs, rb) && encode_tmap(&m.qb, a.q, 3, qd, qst, mb) &&
           encode_tmap(&m.ck, a.ck, 4, cd, cs, cb) && encode_tmap(&m.cv, a.cv, 4, cd, cs, cb) && encode_tmap(&m.nk, a.k, 2, nd, ks, nb) &&
           encode_tmap(&m.nv, a.v, 2, nd, vs, nb) && encode_tmap(&m.qg, a.q, 3, qd, qst, gb) && encode_tmap(&m.q1, a.q, 3, qd, qst, ob);
}

cudaError_t launch_attn_tc(const AttnArgs &a, const AttnTcMaps &b, int D, int max_ctas, bool overlap, cudaStream_t s) {
    const TcMaps &m = *reinterpret_cast<const TcMaps *>(&b);
    const bool cap = a.softcap > 0.f;
    if (D == 64)
        return cap ? launch_tc<64, true>(a, m, max_ctas, overlap, s) : launch_tc<64, false>(a, m, max_ctas, overlap, s);
    return cap ? launch_tc<128, true>(a, m, max_ctas, overlap, s) : launch_tc<128, false>(a, m, max_ctas, overlap, s);
}

}  // namespace w12
