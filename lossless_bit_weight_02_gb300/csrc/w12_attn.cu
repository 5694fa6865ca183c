// Attention of draft-tree nodes over a paged cache: the tree's analysis, the
// kernel for few rows, and the join of partial results (w12_attn_tc.cu has
// the kernel for many rows).  Tree verification checks every drafted node in
// one pass (SpecPilot, arXiv 2611.02501: the news article's part (2)); an
// attention layer then lets a node see the cached tokens and its own
// ancestors.
//
//     x_j = scale q.k_j  (capped: c tanh(x_j / c)),  o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m)
//
// in one pass over the keys with the running maximum m and sum (Milakov and
// Gimelshein 2018): when m grows, what was summed is multiplied by
// e^(m_old - m_new).  Partial (m, sum, output) triples of any split of the
// keys join by the same rule.
#include <cstdint>
#include <cuda_runtime.h>

#include "w12_attn.cuh"

namespace w12 {
namespace {

// ---------------------------------------------------------------------------
// The plan.  One CTA per request lists its nodes (in the order of the call,
// by ballots, so the list does not depend on timing), finds every node's
// ancestors by doubling (after s rounds a node's mask holds the 2^s - 1 nodes
// above it and it jumps 2^s up), and checks the tree, the length and the
// pages.  The last CTA adds the requests' units up, cuts the line into ranges
// and writes down every range's first segment and the joins.
//
// Nothing here is work (a few KB are read): the kernel is a chain of round
// trips of 700 cycles and of barriers, 9.7k cycles (5 us) for one token, 17k
// for eight trees of 256 nodes, of which 3.5k to 5.5k are the ranges.  The
// kernel behind it is launched meanwhile, and the layers of one verify step
// share one plan (W12_ATTN_REUSE_PLAN).
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 256;
constexpr int kAhead = 8;        // passes over the nodes whose loads are in flight
constexpr int kCumShared = 512;  // requests that the last CTA keeps in shared memory

struct PlanArgs {
    AttnArgs a;
    Geometry g;
    int extra;  // Geometry::extra, if the work is enough
};

__device__ __forceinline__ ReqInfo load_req(const ReqInfo *p) {  // written by another CTA of this launch
    static_assert(sizeof(ReqInfo) == 32, "two 16-byte loads");
    ReqInfo r;
    reinterpret_cast<int4 *>(&r)[0] = __ldcg(reinterpret_cast<const int4 *>(p));
    reinterpret_cast<int4 *>(&r)[1] = __ldcg(reinterpret_cast<const int4 *>(p) + 1);
    return r;
}

__global__ __launch_bounds__(kPlanThreads) void k_attn_plan(const __grid_constant__ PlanArgs p) {
    const AttnArgs &a = p.a;
    __shared__ int list[kAttnMaxNodes], plist[kAttnMaxNodes];  // nodes, their parents
    __shared__ int jump[2][kAttnMaxNodes];
    __shared__ uint32_t mask[2][kMaskWords][kAttnMaxNodes];
    __shared__ int dep[2][kAttnMaxNodes];
    __shared__ uint32_t wcount[kPlanThreads / 32];
    __shared__ int s_before, s_bad, s_last, s_deep, s_joins;
    __shared__ int64_t cum_s[kCumShared], wsum[kPlanThreads / 32];
    __shared__ ReqInfo req_s[kCumShared];
    grid_dep_launch();
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // every load that needs no other's answer goes out at once: a round trip is 700 cycles
    const int ctx = a.ctx_len[r];
    int qs[kAhead], pars[kAhead];
    auto read = [&](int base, int &q, int &par) {
        const int i = base + tid;
        q = i < a.n ? (a.req ? a.req[i] : 0) : -2;
        par = i < a.n && a.parent ? a.parent[i] : -1;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) read(k * kPlanThreads, qs[k], pars[k]);
    if (tid == 0) s_before = s_bad = s_deep = s_joins = 0;
    const bool len_bad = ctx < 0 || ctx > (int64_t)a.width * a.page;
    // first cached token that a node sees; only its page and those after it are checked and read
    const int first = !len_bad && a.window > 0 && ctx >= a.window ? ctx - a.window + 1 : 0;
    const int pg0 = first / a.page, pg1 = !len_bad && ctx > first ? (ctx - 1) / a.page : -1;
    auto page_at = [&](int g) { return g <= pg1 ? a.table[r * a.ld_table + g] : 0; };
    const int32_t page0 = page_at(pg0 + tid);
    __syncthreads();

    // nodes of request r in order; how many belong to earlier requests
    int cnt = 0, before = 0, stray = 0;
    for (int base = 0; base < a.n; base += kPlanThreads) {
        const int i = base + tid, q = qs[0], par = pars[0];
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) qs[k] = qs[k + 1], pars[k] = pars[k + 1];
        read(base + kAhead * kPlanThreads, qs[kAhead - 1], pars[kAhead - 1]);
        const bool mine = q == r;
        before += q >= 0 && q < r;
        if (i < a.n && (q < 0 || q >= a.R)) {
            stray = 1;
            if (r == 0) a.ws.pos[i] = -1;
        }
        const uint32_t ball = __ballot_sync(kFull, mine);
        if (lane == 0) wcount[warp] = __popc(ball);
        __syncthreads();
        int at = cnt + __popc(ball & ((1u << lane) - 1u)), all = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const int c = wcount[w];
            at += w < warp ? c : 0;
            all += c;
        }
        if (mine && at < kAttnMaxNodes) {
            list[at] = i;
            plist[at] = par;
        }
        cnt += all;
        __syncthreads();
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) before += __shfl_xor_sync(kFull, before, s);
    if (lane == 0 && before) atomicAdd(&s_before, before);
    bool page_bad = page0 < 0 || (page0 >= a.pages && pg1 >= pg0 + tid);
#pragma unroll 4
    for (int g = pg0 + tid + kPlanThreads; g <= pg1; g += kPlanThreads) {
        const int32_t pg = page_at(g);
        page_bad |= pg < 0 || pg >= a.pages;
    }
    if (page_bad || len_bad || cnt > kAttnMaxNodes) s_bad = 1;
    __syncthreads();
    const int start = s_before;
    const bool bad = s_bad != 0;
    const int m = cnt < kAttnMaxNodes ? cnt : kAttnMaxNodes;

    // parents by rank: an earlier node of the same list, else the node is in error
    bool node_bad = false;
    if (tid < m) {
        const int par = plist[tid];
        int up = -1;
        if (par != -1) {
            int lo = 0, hi = tid;  // the list ascends
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (list[mid] < par) lo = mid + 1;
                else hi = mid;
            }
            if (lo < tid && list[lo] == par) up = lo;
            else node_bad = true;
        }
        jump[0][tid] = up;
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w)
            if (w <= warp) mask[0][w][tid] = w == warp ? 1u << lane : 0u;  // no ancestor has a higher rank
        dep[0][tid] = node_bad ? 0 : 1;
    }
    int cur = 0;
    while (__syncthreads_or(tid < m && jump[cur][tid] >= 0)) {
        if (tid < m) {
            const int j = jump[cur][tid];
            int d = dep[cur][tid];
#pragma unroll
            for (int w = 0; w < kMaskWords; ++w)
                if (w <= warp) {
                    uint32_t u = mask[cur][w][tid];
                    if (j >= 0 && w <= j / 32) u |= mask[cur][w][j];
                    mask[cur ^ 1][w][tid] = u;
                }
            jump[cur ^ 1][tid] = j >= 0 ? jump[cur][j] : -1;
            if (j >= 0 && dep[cur][j] == 0) d = 0;  // an ancestor is in error
            dep[cur ^ 1][tid] = d;
        }
        cur ^= 1;
    }
    if (tid < m && dep[cur][tid]) {
        int d = 0;
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w)
            if (w <= warp) d += __popc(mask[cur][w][tid]);
        dep[cur][tid] = d;
        atomicMax(&s_deep, d);
    }
    __syncthreads();
    if (tid < m) {
        const int i = list[tid], at = start + tid, d = dep[cur][tid];
        a.ws.order[at] = i;
        a.ws.pos[i] = at;
        a.ws.depth[at] = bad ? 0 : d;
        node_bad = d == 0;
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) {
            uint32_t u = w <= warp ? mask[cur][w][tid] : 0u;
            if (a.window > 0 && a.window < d) {  // drop the ancestors beyond the window
                for (uint32_t rest = u; rest; rest &= rest - 1) {
                    const int b = __ffs(rest) - 1;
                    if (d - dep[cur][32 * w + b] >= a.window) u &= ~(1u << b);
                }
            }
            a.ws.mask[(int64_t)at * kMaskWords + w] = u;
        }
    }
    // nodes beyond the limit have no place in the list
    if (cnt > kAttnMaxNodes) {
        for (int i = tid; i < a.n; i += kPlanThreads)
            if ((a.req ? a.req[i] : 0) == r && i > list[kAttnMaxNodes - 1]) a.ws.pos[i] = -1;
    }
    const int any = __syncthreads_or(node_bad || bad || (r == 0 && stray));
    ReqInfo q{};
    if (tid == 0) {
        q.start = start;
        q.cnt = bad ? 0 : m;
        q.ctx = bad ? 0 : ctx;
        const int tree0 = p.g.tree0(q.ctx);
        q.k0 = first < q.ctx || p.g.tree_align < p.g.BN ? first & -p.g.BN : tree0;  // (BN: a power of two)
        q.kb = q.cnt ? (int)((uint32_t)(tree0 + q.cnt - q.k0 + p.g.BN - 1) / (uint32_t)p.g.BN) : 0;
        q.tiles = (q.cnt * a.group + p.g.IM - 1) / p.g.IM;
        q.lo_max = a.window > 0 && q.ctx + s_deep > a.window ? q.ctx + s_deep - a.window : 0;
        q.flags = (any ? kReqBad : 0) | (m > 0 && list[m - 1] - list[0] == m - 1 ? 2 * (list[0] + 1) : 0);
        a.ws.req[r] = q;
        if (a.R > 1) {
            __threadfence();
            s_last = atomicAdd(a.ws.ticket, 1) == a.R - 1;
        } else {
            s_last = 1;
        }
    }
    __syncthreads();
    if (!s_last) return;

    // the last CTA: blocks before every request, then the ranges
    if (a.R > 1) __threadfence();
    if (a.R > 1 && tid < a.R) q = load_req(a.ws.req + tid);  // (of one request: thread 0's own)
    Geometry geo = p.g;
    if (p.extra > 0) {  // where every range is long enough for it, an item's end has a cost of its own
        int64_t mine = tid < a.R ? ItemAt::units(geo, a.group, a.H, q) : 0;
        for (int i = tid + kPlanThreads; i < a.R; i += kPlanThreads)
            mine += ItemAt::units(geo, a.group, a.H, load_req(a.ws.req + i));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) mine += __shfl_xor_sync(kFull, mine, s);
        if (lane == 0) wsum[warp] = mine;
        __syncthreads();
        int64_t all = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) all += wsum[w];
        __syncthreads();
        if (all >= (int64_t)a.G * (geo.least() + p.extra)) geo.extra = p.extra;
    }
    int64_t carry = 0;
    int err = 0;
    for (int base = 0; base < a.R; base += kPlanThreads) {
        const int i = base + tid;
        int64_t x = 0;
        if (i < a.R) {
            if (base > 0) q = load_req(a.ws.req + i);
            x = ItemAt::units(geo, a.group, a.H, q);
            err |= q.flags & kReqBad;
        }
        int64_t sum = x;  // inclusive over the warp
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int64_t y = __shfl_up_sync(kFull, sum, s);
            if (lane >= s) sum += y;
        }
        if (lane == 31) wsum[warp] = sum;
        __syncthreads();
        int64_t before_w = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            before_w += w < warp ? wsum[w] : 0;
            all += wsum[w];
        }
        if (i < a.R) {
            const int64_t c = carry + before_w + sum - x;
            a.ws.cum[i] = c;
            if (i < kCumShared) {
                cum_s[i] = c;
                req_s[i] = q;
            }
        }
        carry += all;
        __syncthreads();
    }
    err = __syncthreads_or(err);
    if (tid == 0) {
        a.ws.cum[a.R] = carry;
        *a.ws.err = err;
        *a.ws.ticket = 0;
        *a.ws.extra = geo.extra;
    }
    __syncthreads();  // cum is this CTA's own: visible to all its threads
    auto cum_at = [&](int i) { return i < kCumShared ? cum_s[i] : a.ws.cum[i]; };
    const Cut cut(carry, a.G, geo.least());
    for (int c = tid; c < a.G; c += kPlanThreads) {
        Seg seg{};
        if (carry > 0 && c < cut.G) {
            const int64_t x = cut.begin(c);
            int lo = 0, hi = a.R - 1;  // the last request that begins at or before x: x is one of its units
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cum_at(mid) <= x) lo = mid;
                else hi = mid - 1;
            }
            const ReqInfo ri = lo < kCumShared ? req_s[lo] : load_req(a.ws.req + lo);
            seg = segment_at(geo, a.group, a.window, ri, lo, cum_at(lo), c, x, x, cut.begin(c + 1));
            const ItemAt it(geo, a.group, ri, cum_at(lo), x);
            const int own = cut.of((ri.kb == 1 ? it.end : it.begin + it.w) - 1), end = cut.of(it.end - 1);
            if (it.begin < x && own == c - 1 && end >= c) {
                // (their order in the list is of no consequence)
                a.ws.join[atomicAdd(&s_joins, 1)] =
                    JoinInfo{lo, it.h, it.t, c, end, 2 * own + (it.begin >= cut.begin(own) ? 1 : 0), {0, 0}};
            }
        }
        a.ws.range[c] = seg;
    }
    __syncthreads();
    if (tid == 0) *a.ws.joins = s_joins;
}

// ---------------------------------------------------------------------------
// Few rows (IM = 16): every warp walks 16 keys of each 64-key block on its own
// with mma.sync: S = Q K^T (Q in registers), softmax, O += P V, with a private
// ring of cp.async copies, so no barrier inside the walk.  The four warps'
// results join at the end of the item in shared memory.
//
// With at most 16 rows per key/value head an element of the cache takes 16
// multiply-adds at most: the kernel has to keep the copies coming, and HBM
// bounds it.  64 requests of one token over up to 16384 tokens (3.17 GB) take
// 474-490 us on different GPUs, 6.5-6.7 TB/s.  Two CTAs an SM with three stages
// of 16 keys per warp keep 192 KB on their way.
// ---------------------------------------------------------------------------
constexpr int kRowWarps = 4;
constexpr int kRowBlock = 16 * kRowWarps;
constexpr int kRowStages = 3;
constexpr int kRowCtasPerSm = 2;

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int D>
constexpr int row_smem_bytes() {
    return kRowWarps * kRowStages * 2 * 16 * D * 2 + kRowWarps * 16 * 8;
}

// 16 rows of D BF16, 16-byte chunks swizzled by the row so that eight rows of
// one chunk lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t row_chunk(int row, int chunk) {
    return (uint32_t)(row * (D * 2) + ((chunk ^ (row & 7)) << 4));
}

template <int D, bool CAP>
__global__ __launch_bounds__(32 * kRowWarps, kRowCtasPerSm) void k_attn_rows(const __grid_constant__ AttnArgs a) {
    constexpr int KS = D / 16;        // k-steps of Q K^T
    constexpr int CH = D / 8;         // 16-byte chunks of a row
    constexpr int PER = 16 * CH / 32; // chunks a lane copies per 16 keys
    constexpr uint32_t kTile = 16 * D * 2;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
    uint8_t *ring = smem + warp * (kRowStages * 2 * kTile);
    const uint32_t ring_s = smem_u32(ring);
    float2 *ml_s = reinterpret_cast<float2 *>(smem + kRowWarps * kRowStages * 2 * kTile);  // [warps][16]
    __shared__ SegWalk walks[kRowWarps];
    SegWalk &walk = walks[warp];
    const Seg &sg = walk.sg;
    const Geometry geo{16, kRowBlock, 16, 1, 1, 1, 0};
    grid_dep_wait();
    grid_dep_launch();
    if (lane == 0) walk.begin(a, geo);
    const float sl2 = a.scale * kLog2e, cap2 = CAP ? 2.0f * kLog2e * a.scale / a.softcap : 0.f,
                capl = CAP ? a.softcap * kLog2e : 0.f;

    {
        while (walk.next(a, geo)) {
            const int nb = sg.nb, h = sg.h, t = sg.t, r = sg.r, ctx = sg.ctx, cnt = sg.cnt, start = sg.start;
            // this lane's two query rows (g and g + 8 of the tile)
            const uint32_t *mrow[2];
            int lo_key[2];
            bool live[2];
            uint32_t qf[KS][4];
            int lo_max = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int row = t * 16 + g + 8 * u, rank = row / a.group;
                live[u] = rank < cnt;
                const int at = start + (live[u] ? rank : 0);
                mrow[u] = a.ws.mask + (int64_t)at * kMaskWords;
                const int d = a.ws.depth[at];
                lo_key[u] = a.window > 0 ? ctx + d - a.window : 0;  // cached tokens from here on
                lo_max = lo_key[u] > lo_max ? lo_key[u] : lo_max;
                const uint32_t *qp = reinterpret_cast<const uint32_t *>(
                    a.q + (int64_t)a.ws.order[at] * a.ldq + (int64_t)(h * a.group + (row - rank * a.group)) * D);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    qf[s][u] = live[u] ? qp[8 * s + q4] : 0u;
                    qf[s][2 + u] = live[u] ? qp[8 * s + 4 + q4] : 0u;
                }
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) lo_max = max(lo_max, __shfl_xor_sync(kFull, lo_max, s));
            const int end = ctx + cnt, key_lo = sg.key_lo;
            // keys of step i: the segment's first + 64 i + 16 warp ...
            const int steps = nb;
            const int key0 = sg.key0 + warp * 16;
            auto fetch_page = [&](int i, int &tok) -> int64_t {  // lane's key of step i: page of a cached token
                const int key = key0 + i * kRowBlock + (lane & 15);
                if (i < steps && key >= key_lo && key < ctx) return page_of(a, r, key, tok);
                return -1;
            };
            int tok_n = 0;
            int64_t page_n = fetch_page(0, tok_n);
            auto issue = [&](int i) {
                if (i < steps) {
                    const int key = key0 + i * kRowBlock + (lane & 15);
                    const uint16_t *kp = a.k, *vp = a.v;  // 0 bytes of it: zeros
                    uint32_t bytes = 0;
                    if (key >= ctx && key < end) {
                        const int64_t node = a.ws.order[start + key - ctx];
                        kp = a.k + node * a.ldk + h * D;
                        vp = a.v + node * a.ldv + h * D;
                        bytes = 16;
                    } else if (page_n >= 0) {
                        const int64_t off = page_n * a.page_stride + tok_n * a.token_stride + h * a.head_stride;
                        kp = a.ck + off;
                        vp = a.cv + off;
                        bytes = 16;
                    }
                    page_n = fetch_page(i + 1, tok_n);
                    const uint32_t st = ring_s + (uint32_t)(i % kRowStages) * 2 * kTile;
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const int ch = lane % CH, row = lane / CH + j * (32 / CH);
                        const uint64_t ks = __shfl_sync(kFull, reinterpret_cast<uint64_t>(kp), row);
                        const uint64_t vs = __shfl_sync(kFull, reinterpret_cast<uint64_t>(vp), row);
                        const uint32_t nb = __shfl_sync(kFull, bytes, row);
                        const uint32_t dst = st + row_chunk<D>(row, ch);
                        cp_async16(dst, reinterpret_cast<const uint8_t *>(ks) + 16 * ch, nb);
                        cp_async16(dst + kTile, reinterpret_cast<const uint8_t *>(vs) + 16 * ch, nb);
                    }
                }
                cp_commit();
            };
            float O[D / 8][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[j][e] = 0.f;
#pragma unroll
            for (int i = 0; i < kRowStages - 1; ++i) issue(i);
            for (int i = 0; i < steps; ++i) {
                cp_wait<kRowStages - 2>();
                __syncwarp();
                const uint32_t st = ring_s + (uint32_t)(i % kRowStages) * 2 * kTile;
                float S[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[j][e] = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s) {  // keys 0-7 and 8-15, chunks 2s and 2s + 1
                    uint32_t b[4];
                    ldsm4(b, st + row_chunk<D>((lane & 7) + ((lane >> 4) << 3), 2 * s + ((lane >> 3) & 1)));
                    mma16(S[0], qf[s], b[0], b[1]);
                    mma16(S[1], qf[s], b[2], b[3]);
                }
                issue(i + kRowStages - 1);  // the stage read in step i - 1 is free
                const int kbase = key0 + i * kRowBlock;
                const bool inner = kbase >= lo_max && kbase + 16 <= ctx;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[j][e] = CAP ? cap_score(S[j][e], cap2, capl) : S[j][e] * sl2;
                if (!inner) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int u = e >> 1, key = kbase + 8 * j + 2 * q4 + (e & 1), rk = key - ctx;
                            const bool see = key < ctx ? key >= lo_key[u] : key < end && (mrow[u][rk >> 5] >> (rk & 31) & 1u);
                            if (!see || !live[u]) S[j][e] = -INFINITY;
                        }
                }
                float P[2][4];
                bool grew = false;
                float mn[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float top = fmaxf(fmaxf(S[0][2 * u], S[0][2 * u + 1]), fmaxf(S[1][2 * u], S[1][2 * u + 1]));
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
                    mn[u] = fmaxf(mx[u], top);
                    grew |= mn[u] != mx[u];
                }
                if (__any_sync(kFull, grew)) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float f = mn[u] == mx[u] ? 1.0f : exp2_approx(mx[u] - mn[u]);
                        sum[u] *= f;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            O[j][2 * u] *= f;
                            O[j][2 * u + 1] *= f;
                        }
                        mx[u] = mn[u];
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float m0 = mx[u] == -INFINITY ? 0.f : mx[u];  // nothing seen yet: every weight is 0
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            P[j][2 * u + e] = exp2_approx(S[j][2 * u + e] - m0);
                            sum[u] += P[j][2 * u + e];
                        }
                }
                // 0 * Inf: an unseen key's V must not reach the product.  Rows of a block with
                // masked keys are looked over; a row that is not finite is taken out of the
                // product and added where it is seen, with a weight that underflowed to 0 too
                // (0 * Inf is then NaN, as in a block without masked keys).
                uint32_t odd = 0;
                if (!inner) {
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const int ch = lane % CH, row = lane / CH + j * (32 / CH);
                        const uint4 u = *reinterpret_cast<const uint4 *>(ring + (i % kRowStages) * 2 * kTile + kTile +
                                                                         row_chunk<D>(row, ch));
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                        bool nf = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            nf |= (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
                        const uint32_t ball = __ballot_sync(kFull, nf);
#pragma unroll
                        for (int k = 0; k < 32 / CH; ++k)
                            if (ball >> (k * CH) & ((CH == 32 ? 0u : 1u << CH) - 1u)) odd |= 1u << (k + j * (32 / CH));
                    }
                }
                if (odd) {
                    for (int k = 0; k < 16; ++k) {
                        if (!(odd >> k & 1u)) continue;
                        // the weights of key k for this lane's rows
                        const int src = (lane & ~3) | ((k & 7) >> 1), e = k & 1;
                        const int key = kbase + k, rk = key - ctx;
                        float w[2];
                        bool see[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float lo = __shfl_sync(kFull, k < 8 ? P[0][2 * u] : P[1][2 * u], src);
                            const float hi = __shfl_sync(kFull, k < 8 ? P[0][2 * u + 1] : P[1][2 * u + 1], src);
                            w[u] = e ? hi : lo;
                            see[u] = live[u] && (key < ctx ? key >= lo_key[u] : key < end && (mrow[u][rk >> 5] >> (rk & 31) & 1u));
                        }
                        uint8_t *vt = ring + (i % kRowStages) * 2 * kTile + kTile;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            const uint32_t v2 = *reinterpret_cast<const uint32_t *>(vt + row_chunk<D>(k, j) + 4 * q4);
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                if (see[u]) {
                                    O[j][2 * u] = fmaf(w[u], __uint_as_float(v2 << 16), O[j][2 * u]);
                                    O[j][2 * u + 1] = fmaf(w[u], __uint_as_float(v2 & 0xFFFF0000u), O[j][2 * u + 1]);
                                }
                        }
                        __syncwarp();
                        if (lane < CH) *reinterpret_cast<uint4 *>(vt + row_chunk<D>(k, lane)) = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
                const uint32_t pa[4] = {pack_bf16(P[0][0], P[0][1]), pack_bf16(P[0][2], P[0][3]),
                                        pack_bf16(P[1][0], P[1][1]), pack_bf16(P[1][2], P[1][3])};
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {  // columns 16j .. 16j + 15
                    uint32_t b[4];
                    ldsm4t(b, st + kTile + row_chunk<D>(lane & 15, 2 * j + (lane >> 4)));
                    mma16(O[2 * j], pa, b[0], b[1]);
                    mma16(O[2 * j + 1], pa, b[2], b[3]);
                }
                __syncwarp();
            }
            cp_wait<0>();
            // join the warps: (max, sum) and O to shared memory, over the ring
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                sum[u] += __shfl_xor_sync(kFull, sum[u], 1);
                sum[u] += __shfl_xor_sync(kFull, sum[u], 2);
            }
            __syncthreads();
            float *Os = reinterpret_cast<float *>(smem);  // [warps][16][D + 4]
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (q4 == 0) ml_s[warp * 16 + g + 8 * u] = make_float2(mx[u], sum[u]);
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    *reinterpret_cast<float2 *>(Os + (warp * 16 + g + 8 * u) * (D + 4) + 8 * j + 2 * q4) =
                        make_float2(O[j][2 * u], O[j][2 * u + 1]);
            }
            __syncthreads();
            {
                const int row = tid >> 3, c0 = (tid & 7) * (D / 8);
                float m = -INFINITY, l = 0.f, f[kRowWarps];
#pragma unroll
                for (int w = 0; w < kRowWarps; ++w) m = fmaxf(m, ml_s[w * 16 + row].x);
                const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int w = 0; w < kRowWarps; ++w) {
                    f[w] = exp2_approx(ml_s[w * 16 + row].x - m0);
                    l = fmaf(ml_s[w * 16 + row].y, f[w], l);
                }
                const int rowg = t * 16 + row, rank = rowg / a.group;
                const bool whole = sg.whole;
                const float inv = whole ? 1.0f / l : 1.0f;
                float out[D / 8];
#pragma unroll
                for (int j = 0; j < D / 8; j += 4) {
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kRowWarps; ++w) {
                        const float4 v = *reinterpret_cast<const float4 *>(Os + (w * 16 + row) * (D + 4) + c0 + j);
                        s.x = fmaf(v.x, f[w], s.x);
                        s.y = fmaf(v.y, f[w], s.y);
                        s.z = fmaf(v.z, f[w], s.z);
                        s.w = fmaf(v.w, f[w], s.w);
                    }
                    out[j] = s.x * inv, out[j + 1] = s.y * inv, out[j + 2] = s.z * inv, out[j + 3] = s.w * inv;
                }
                if (rank < cnt) {
                    if (whole) {
                        uint16_t *o = a.o + (int64_t)a.ws.order[start + rank] * a.ldo +
                                      (int64_t)(h * a.group + rowg - rank * a.group) * D + c0;
#pragma unroll
                        for (int j = 0; j < D / 8; j += 8)
                            *reinterpret_cast<uint4 *>(o + j) =
                                make_uint4(pack_bf16(out[j], out[j + 1]), pack_bf16(out[j + 2], out[j + 3]),
                                           pack_bf16(out[j + 4], out[j + 5]), pack_bf16(out[j + 6], out[j + 7]));
                    } else {
                        const int64_t slot = sg.slot;
                        if (c0 == 0) a.ws.ml[slot * 16 + row] = make_float2(m, l);
                        float *o = a.ws.part + (slot * (D / 4) * 16 + row) * 4;
#pragma unroll
                        for (int j = 0; j < D / 8; j += 4)
                            *reinterpret_cast<float4 *>(o + (c0 + j) * 16) =
                                make_float4(out[j], out[j + 1], out[j + 2], out[j + 3]);
                    }
                }
            }
            __syncthreads();  // the ring is written again
        }
    }
}

// ---------------------------------------------------------------------------
// The join of the items that several ranges share: a CTA takes some rows and
// columns of one.  Thread = (row, a few columns): the partials are read along
// the rows, the first 16 loads with those of the sums.  The nodes that the plan
// found in error get NaN here.
// ---------------------------------------------------------------------------
template <int D, int IM>
struct JoinShape {
    // Few rows: a few items share all ranges, so their columns go to several CTAs, and 16 partials' loads are
    // in flight (one token over 4000: 28.3 -> 23.0 us).  Many rows: many items of a few partials each, so few
    // and large CTAs (8 x 256 nodes over 8k: 234-237 us; slices of 64 columns 243, 8 loads ahead 247).
    static constexpr int kRows = IM < 32 ? IM : 64;            // of a CTA
    static constexpr int kCols = IM < 32 ? 32 : D;             // of a CTA
    static constexpr int kPer = IM < 32 ? 1 : D / 32;          // float4 columns of a thread
    static constexpr int kAhead = IM < 32 ? 16 : 4;            // partials whose loads go out together
    static constexpr int kLanes = kCols / 4 / kPer;            // threads of a row
    static constexpr int kThreads = kRows * kLanes;
    static constexpr int kSlices = D / kCols;
};

template <int D, int IM, int GMAX>
__global__ __launch_bounds__(JoinShape<D, IM>::kThreads) void k_attn_join(const __grid_constant__ AttnArgs a) {
    using J = JoinShape<D, IM>;
    constexpr int RB = J::kRows, PAR = J::kLanes, PER = J::kPer, T = J::kThreads;
    __shared__ float f_s[GMAX + 1][RB];
    __shared__ float m_s[PAR][RB], l_s[PAR][RB];
    __shared__ __align__(16) uint2 out_s[RB][J::kCols / 4 + 2];
    const int tid = threadIdx.x, row = tid % RB, grp = tid / RB;
    const int row0 = (int)blockIdx.y / J::kSlices * RB, col0 = (int)blockIdx.y % J::kSlices * J::kCols;
    // (the plan's results are there before the wait: the kernel between has waited for them)
    const bool bad = *a.ws.err != 0, none = (int)blockIdx.x >= *a.ws.joins;
    JoinInfo ri{};
    ReqInfo rq{};
    if (!none) {
        ri = a.ws.join[blockIdx.x];
        rq = a.ws.req[ri.r];
    }
    const int c = ri.c;
    grid_dep_wait();
    if (none && !bad) return;
    if (bad) {
        const int64_t all = (int64_t)a.n * a.Hq, step = (int64_t)gridDim.x * gridDim.y;
        for (int64_t w = (int64_t)blockIdx.y * gridDim.x + blockIdx.x; w < all; w += step) {
            const int i = (int)(w / a.Hq), hq = (int)(w - (int64_t)i * a.Hq);
            const int p = a.ws.pos[i];
            if (p >= 0 && a.ws.depth[p] != 0) continue;
            for (int d = tid; d < D; d += T) a.o[(int64_t)i * a.ldo + (int64_t)hq * D + d] = 0x7FC0;
        }
        if (none) return;
    }
    const int rows = min(rq.cnt * a.group - ri.t * IM - row0, RB);  // of this CTA
    if (rows <= 0) return;
    const int n = ri.last - c + 2;  // partials: that of the range before, then this range's and the next ones' first pieces
    auto slot = [&](int j) { return j == 0 ? (int64_t)ri.first : (int64_t)2 * (c - 1 + j); };
    const float4 *part = reinterpret_cast<const float4 *>(a.ws.part) + (int64_t)(col0 / 4 + grp) * IM + row0 + row;
    const bool live = row < rows;  // nobody has written the others
    auto at = [&](int j, int k) { return part[(slot(j) * (D / 4) + k * PAR) * IM]; };
    // Loads go out in batches: one after the other they would take the L2's latency each.
    constexpr int AHEAD = J::kAhead;
    float4 v[AHEAD][PER];
    auto load = [&](int j0) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
#pragma unroll
            for (int k = 0; k < PER; ++k) v[j][k] = live && j0 + j < n ? at(j0 + j, k) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);  // with the loads of the sums
    constexpr int SUMS = 4;
    float m = -INFINITY;
    for (int j0 = grp; j0 < n; j0 += SUMS * PAR) {
        float2 ml[SUMS];
#pragma unroll
        for (int i = 0; i < SUMS; ++i)
            ml[i] = live && j0 + i * PAR < n ? a.ws.ml[slot(j0 + i * PAR) * IM + row0 + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < SUMS; ++i) {
            if (j0 + i * PAR < n) {
                f_s[j0 + i * PAR][row] = ml[i].x;
            }
            m = fmaxf(m, ml[i].x);
        }
    }
    m_s[grp][row] = m;
    __syncthreads();
#pragma unroll
    for (int g = 0; g < PAR; ++g) m = fmaxf(m, m_s[g][row]);
    const float m0 = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int j0 = grp; j0 < n; j0 += SUMS * PAR) {
        float w[SUMS];
#pragma unroll
        for (int i = 0; i < SUMS; ++i)
            w[i] = live && j0 + i * PAR < n ? a.ws.ml[slot(j0 + i * PAR) * IM + row0 + row].y : 0.f;
#pragma unroll
        for (int i = 0; i < SUMS; ++i)
            if (j0 + i * PAR < n) {
                float &f = f_s[j0 + i * PAR][row];
                f = exp2_approx(f - m0);
                l = fmaf(w[i], f, l);
            }
    }
    l_s[grp][row] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int g = 0; g < PAR; ++g) l += l_s[g][row];
    float4 acc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < n; j0 += AHEAD) {
        if (j0 > 0) load(j0);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const float f = j0 + j < n ? f_s[j0 + j][row] : 0.f;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                acc[k].x = fmaf(v[j][k].x, f, acc[k].x);
                acc[k].y = fmaf(v[j][k].y, f, acc[k].y);
                acc[k].z = fmaf(v[j][k].z, f, acc[k].z);
                acc[k].w = fmaf(v[j][k].w, f, acc[k].w);
            }
        }
    }
    const float inv = 1.0f / l;
#pragma unroll
    for (int k = 0; k < PER; ++k)
        out_s[row][grp + k * PAR] =
            make_uint2(pack_bf16(acc[k].x * inv, acc[k].y * inv), pack_bf16(acc[k].z * inv, acc[k].w * inv));
    __syncthreads();
    for (int w = tid; w < rows * (J::kCols / 8); w += T) {  // 16 bytes each
        const int rr = w / (J::kCols / 8), ch = w % (J::kCols / 8);
        const int rowi = ri.t * IM + row0 + rr, rank = rowi / a.group, at = rq.start + rank;
        if (bad && a.ws.depth[at] == 0) continue;
        uint16_t *o = a.o + (int64_t)a.ws.order[at] * a.ldo + (int64_t)(ri.h * a.group + (rowi - rank * a.group)) * D + col0;
        reinterpret_cast<uint4 *>(o)[ch] = *reinterpret_cast<const uint4 *>(&out_s[rr][2 * ch]);
    }
}

template <typename... A>
cudaError_t launch_after(void (*k)(A...), dim3 grid, int threads, size_t smem, bool overlap, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

template <int D, int IM, int GMAX>
cudaError_t launch_join(const AttnArgs &a, cudaStream_t s) {
    using J = JoinShape<D, IM>;
    // no more than the boundaries of ranges, nor than there are items
    const int64_t items = a.H * (a.R + (int64_t)a.n * a.group / IM);
    const int joins = items < GMAX ? (int)items : GMAX;
    return launch_after(k_attn_join<D, IM, GMAX>, dim3(joins, IM / J::kRows * J::kSlices), J::kThreads, 0, true, s, a);
}

template <int D, bool CAP>
cudaError_t launch_rows(const AttnArgs &a, int max_ctas, bool overlap, cudaStream_t s) {
    const int smem = row_smem_bytes<D>();
    cudaError_t e = cudaFuncSetAttribute(k_attn_rows<D, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = max_ctas > 0 && max_ctas < a.G ? max_ctas : a.G;
    return launch_after(k_attn_rows<D, CAP>, dim3(grid), 32 * kRowWarps, smem, overlap, s, a);
}

constexpr AttnShape kRowsShape{16, kRowBlock, kRowCtasPerSm * W12_PLAN_SMS, false};
constexpr AttnShape kTcShape{kAttnTcRows, kAttnTcBlock, W12_PLAN_SMS, true};
// Up to 16 rows per key/value head and request on average: the kernel for few rows; more: the tcgen05 kernel,
// whose tiles hold 128.  40 heads over 8, us for few rows / tcgen05: 1 token over 1000 16.8 / 21.4; 64 x 1 over
// 16k 487 / 504; 64 x 3 (15 rows) over 4000 143 / 153; 4 nodes (20 rows) over 16k 37 / 31, over 128k 132 / 109;
// 16 x 4 over 8k 126 / 89; 64 nodes over 16k 155 / 50.  The average is all that is known on the host: a large
// tree beside many requests of few nodes or none goes to the kernel for few rows (64 nodes over 16k beside 63 of
// one node over 1000: 219 us; 200 nodes over 16k in a table of 64 requests 454, alone 80).
AttnShape attn_shape(int64_t n, int64_t R, int group) { return n * group > 16 * R ? kTcShape : kRowsShape; }

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Pointers into the workspace; returns its size.
size_t attn_layout(char *base, int64_t n, int64_t R, int D, const AttnShape &sh, AttnWs *ws) {
    size_t off = 256;
    auto take = [&](size_t bytes) {
        char *p = base + off;
        off = up256(off + bytes);
        return p;
    };
    AttnWs w;
    w.err = reinterpret_cast<int32_t *>(base);
    w.ticket = w.err + 1;
    w.timeout = w.err + 2;
    w.extra = w.err + 3;
    w.joins = w.err + 4;
    w.req = reinterpret_cast<ReqInfo *>(take(sizeof(ReqInfo) * (size_t)R));
    w.cum = reinterpret_cast<int64_t *>(take(8 * (size_t)(R + 1)));
    w.range = reinterpret_cast<Seg *>(take(sizeof(Seg) * (size_t)sh.G));
    w.join = reinterpret_cast<JoinInfo *>(take(sizeof(JoinInfo) * (size_t)sh.G));
    w.order = reinterpret_cast<int32_t *>(take(4 * (size_t)n));
    w.pos = reinterpret_cast<int32_t *>(take(4 * (size_t)n));
    w.depth = reinterpret_cast<int32_t *>(take(4 * (size_t)n));
    w.mask = reinterpret_cast<uint32_t *>(take(4 * (size_t)kMaskWords * (size_t)n));
    w.ml = reinterpret_cast<float2 *>(take(8 * (size_t)(2 * sh.G) * sh.IM));
    w.part = reinterpret_cast<float *>(take(4 * (size_t)(2 * sh.G) * sh.IM * D));
    if (ws) *ws = w;
    return off;
}

}  // namespace

size_t attn_workspace_bytes(int64_t n, int64_t R, int q_heads, int heads, int D) {
    const size_t rows = attn_layout(nullptr, n, R, D, kRowsShape, nullptr);
    const size_t own = attn_layout(nullptr, n, R, D, attn_shape(n, R, q_heads / heads), nullptr);
    return own > rows ? own : rows;
}

cudaError_t launch_tree_attn(const w12_attn_args &x, const w12_kv_cache &c, void *workspace, cudaStream_t s) {
    const int D = c.dim, group = x.q_heads / c.heads;
    AttnArgs a{};
    a.q = x.q, a.k = x.k, a.v = x.v;
    a.ldq = x.ldq, a.ldk = x.ldk, a.ldv = x.ldv;
    a.o = x.o;
    a.ldo = x.ldo;
    a.n = (int)x.n, a.R = (int)x.R, a.Hq = x.q_heads, a.H = c.heads, a.group = group;
    a.ck = c.k, a.cv = c.v;
    a.pages = c.pages;
    a.page_stride = c.page_stride, a.token_stride = c.token_stride, a.head_stride = c.head_stride;
    a.page = c.page_tokens;
    a.page_shift = -1;
    for (int b = 0; b < 31; ++b)
        if (c.page_tokens == 1 << b) a.page_shift = b;
    a.table = x.block_table;
    a.ld_table = x.ld_table;
    a.width = x.width;
    a.ctx_len = x.ctx_len, a.parent = x.parent, a.req = x.req;
    a.scale = x.scale > 0.f ? x.scale : (D == 64 ? 0.125f : 0.08838834764831845f);
    a.softcap = x.softcap;
    a.window = x.window;
    a.stall = x.flags & W12_ATTN_TEST_STALL;
    AttnShape sh = attn_shape(x.n, x.R, group);
    // rows of a copy of queries: up to 64, so that most of an item's go by such copies whatever the group
    a.q_nodes = group < 64 ? 64 / group : 1;
    AttnTcMaps maps;
    if (sh.tc && !attn_tc_maps(a, D, &maps)) sh = kRowsShape;
    a.G = sh.G;
    attn_layout(static_cast<char *>(workspace), x.n, x.R, D, sh, &a.ws);
    cudaError_t e = cudaSuccess;
    const bool plan = !(x.flags & W12_ATTN_REUSE_PLAN);
    if (plan) {
        PlanArgs p;
        p.a = a;
        p.g = sh.tc ? Geometry{sh.IM, sh.BN, kAttnTcRows / 2, kAttnTcPair, kAttnTcOne, kAttnTcBlock, 0}
                    : Geometry{sh.IM, sh.BN, sh.IM, 1, 1, 1, 0};
        p.extra = sh.tc ? kAttnTcExtra : 0;
        k_attn_plan<<<(unsigned)a.R, kPlanThreads, 0, s>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const bool cap = a.softcap > 0.f;
    if (sh.tc)
        e = launch_attn_tc(a, maps, D, x.max_ctas, plan, s);
    else if (D == 64)
        e = cap ? launch_rows<64, true>(a, x.max_ctas, plan, s) : launch_rows<64, false>(a, x.max_ctas, plan, s);
    else
        e = cap ? launch_rows<128, true>(a, x.max_ctas, plan, s) : launch_rows<128, false>(a, x.max_ctas, plan, s);
    if (e != cudaSuccess) return e;
    if (sh.tc) return D == 64 ? launch_join<64, kAttnTcRows, W12_PLAN_SMS>(a, s) : launch_join<128, kAttnTcRows, W12_PLAN_SMS>(a, s);
    return D == 64 ? launch_join<64, 16, kRowCtasPerSm * W12_PLAN_SMS>(a, s)
                   : launch_join<128, 16, kRowCtasPerSm * W12_PLAN_SMS>(a, s);
}

}  // namespace w12
