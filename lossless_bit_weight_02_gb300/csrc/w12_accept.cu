// Which drafted nodes a verify step accepts, and the token that follows
// (SpecPilot, arXiv 2611.02501, verifies draft trees but does not write the
// rule out; the published rejection rule of speculative sampling, Leviathan et
// al. 2023, applied to a node's children one after the other).
//
// At a place of the tree (the root, then the node last accepted) p is the
// target's softmax of that place's row of logits.  Its children are tried in
// the order of the list: token y with its random number u is accepted where
//     u q(y) < p(y),   else   p <- max(p - q, 0) / sum,
// q the distribution that y was drawn from (a point mass where the drafter
// only proposed it).  Where none is accepted the walk ends, and the token after
// it is argmax p(t) / e(t), e exponential noise: an exact draw from p.
//
// What it costs is the rows of the places that the walk visits.  Not every
// node's row is read: of 8 requests with 32 nodes each about 35 rows of 264 are
// needed (each request visits one row more than it accepts nodes).  A cluster
// of up to 8 CTAs takes a request, each CTA a slice of the vocabulary.  Every
// warp hands its (maximum, sum, first maximum) of a row to all CTAs of the
// cluster by asynchronous stores that count down a barrier there; every warp waits
// for its own CTA's, joins the parts, in the same order, and takes the same
// decisions from the same numbers, a lane a child, without another barrier.  (With
// cluster barriers, which wait for the stores first, a round took 0.6 us more.)  The root's row is on its way
// while the tree is looked over, and the children's numbers while the warps wait
// for one another.
#include <cooperative_groups.h>

#include <cstdint>
#include <cuda_runtime.h>

#include "w12_device.cuh"
#include "w12_internal.h"
#include "w12_tc.cuh"

namespace w12 {
namespace {

namespace cg = cooperative_groups;
using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::smem_addr;
using tc::warp_wait;

constexpr int kAccNodes = W12_TREE_MAX_BUDGET;  // of a request
constexpr int kRoot = kAccNodes;                // the root's place among them
constexpr int kNone = kAccNodes + 1;
constexpr int kMaxParts = 8 * 16;               // warps of a cluster
constexpr int kChunk = 8;                       // logits of one load
constexpr int kDeep = 4;                        // chunks of a thread in flight
constexpr int kMaxCluster = 8;
constexpr float kLog2eF = 1.4426950408889634f;

struct AcceptArgs {
    const void *logits;
    int64_t ldl, rows;
    int V;
    const int32_t *token, *parent, *req, *row, *root_row;
    int n, R;
    const float *temperature;
    float temperature1;
    const float *uniform, *noise;
    int64_t ld_noise;
    const float *draft;
    int64_t ldd, draft_rows;
    const int32_t *draft_row;
    int max_depth;
    int32_t *count, *nodes, *next;
    int64_t ld_nodes;
    int stall;  // tests only
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Eight values of a row, as they were loaded; -inf outside [0, n).  Whole chunks begin on 16 bytes.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
    uint4 u;
    __device__ __forceinline__ void load(const uint16_t *row, int i0, int n) {
        if (i0 >= 0 && i0 + kChunk <= n) {
            u = *reinterpret_cast<const uint4 *>(row + i0);
            return;
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + 2 * j;
            w[j] = (i >= 0 && i < n ? row[i] : 0xFF80u) | (uint32_t)(i + 1 >= 0 && i + 1 < n ? row[i + 1] : 0xFF80u) << 16;
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void none() { u = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
    __device__ __forceinline__ void get(float x[kChunk]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
};
template <>
struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *row, int i0, int n) {
        if (i0 >= 0 && i0 + kChunk <= n) {
            a = *reinterpret_cast<const float4 *>(row + i0);
            b = *reinterpret_cast<const float4 *>(row + i0 + 4);
            return;
        }
        float x[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) x[j] = i0 + j >= 0 && i0 + j < n ? row[i0 + j] : -INFINITY;
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ __forceinline__ void none() { a = b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    __device__ __forceinline__ void get(float x[kChunk]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
// The same of a second row, whose alignment may be another: whole groups of 16 bytes, then the shift (the same for
// every thread); `fill` outside.
__device__ __forceinline__ void load8_any(const float *row, int i0, int n, float x[kChunk], float fill) {
    const int sh = (int)((reinterpret_cast<uintptr_t>(row + i0) >> 2) & 3);
    if (i0 - sh >= 0 && i0 - sh + 12 <= n) {
        const float4 *p = reinterpret_cast<const float4 *>(row + i0 - sh);
        const float4 a = p[0], b = p[1];
        if (sh == 0) {
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
            return;
        }
        const float4 c = p[2];
        if (sh == 1) x[0] = a.y, x[1] = a.z, x[2] = a.w, x[3] = b.x, x[4] = b.y, x[5] = b.z, x[6] = b.w, x[7] = c.x;
        else if (sh == 2) x[0] = a.z, x[1] = a.w, x[2] = b.x, x[3] = b.y, x[4] = b.z, x[5] = b.w, x[6] = c.x, x[7] = c.y;
        else x[0] = a.w, x[1] = b.x, x[2] = b.y, x[3] = b.z, x[4] = b.w, x[5] = c.x, x[6] = c.y, x[7] = c.z;
        return;
    }
#pragma unroll
    for (int j = 0; j < kChunk; ++j) x[j] = i0 + j >= 0 && i0 + j < n ? row[i0 + j] : fill;
}

__device__ __forceinline__ float value(const uint16_t *row, int i) { return __uint_as_float((uint32_t)row[i] << 16); }
__device__ __forceinline__ float value(const float *row, int i) { return row[i]; }

// A row's statistics: its maximum, the sum of exp((x - maximum) / T), the first place of the maximum.  With a NaN among
// the values the maximum is NaN: every probability is then, no place is the first, and no child is accepted.
struct Stat {
    float m, s;
    int at;
};
__device__ __forceinline__ float max_nan(float x, float y) {  // (fmaxf would pass over a NaN; this costs the same)
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}
__device__ __forceinline__ float weight(float x, float m, float c) {  // exp((x - m) / T) of a finite maximum
    return ex2((x - m) * c);
}
// An infinite maximum leaves the values that equal it, each with weight 1.
__device__ __forceinline__ float weight_any(float x, float m, float c) {
    return isinf(m) ? (x == m ? 1.f : 0.f) : weight(x, m, c);
}
// x times f, where no x is no matter what f is
__device__ __forceinline__ float scaled(float x, float f) { return x > 0.f ? x * f : x; }  // (NaN stays)

struct Best {  // of a draw: the highest score, the lowest token of that score
    float score;
    int at;
};
__device__ __forceinline__ Best better(const Best &a, const Best &b) {
    return b.score > a.score || (b.score == a.score && b.at < a.at) ? b : a;
}

struct Shared {
    uint4 part[2][kMaxParts];                 // from every warp of the cluster, by the parity of the round
    uint64_t bar[2];
    int node[kAccNodes];                   // the request's nodes, ascending: index in the call's list,
    int par[kAccNodes], tok[kAccNodes];    // parent's there, token,
    int up[kAccNodes];                     // parent's place among them
    int gone[kAccNodes];                   // children refused at the place (written by every warp, the same values)
    int off[16];
    int total, bad, gave_up;
    int32_t err;                           // (a wait that gave up)
};

template <typename T, int kAccThreads>
__global__ __launch_bounds__(kAccThreads, 2) void k_accept(const __grid_constant__ AcceptArgs a) {
    constexpr int kAccWarps = kAccThreads / 32, kParts = kMaxCluster * kAccWarps;
    static_assert(kParts <= kMaxParts, "shared memory");
    __shared__ Shared sm;
    cg::cluster_group cl = cg::this_cluster();
    const int nc = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int r = (int)blockIdx.x / nc, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int V = a.V, parts = nc * kAccWarps, me = rank * kAccWarps + warp;
    const T *logits = static_cast<const T *>(a.logits);
    const float temp = a.temperature ? a.temperature[r] : a.temperature1;
    const bool greedy = !(temp > 0.f);
    const float c = greedy ? kLog2eF : fminf(fmaxf(kLog2eF / temp, 1e-30f), 1e30f);  // of any temperature: no 0 * inf
    const float *noise = greedy ? nullptr : a.noise + (int64_t)r * a.ld_noise;
    if (tid == 0) {
        sm.gave_up = 0, sm.err = 0;
        sm.total = 0, sm.bad = 0;  // (before the barrier: without nodes there is no other before they are read)
        for (int i = 0; i < 2; ++i) {
            mbar_init(sm.bar + i, 1);
            mbar_expect_tx(sm.bar + i, parts * 16);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    cl.barrier_arrive();  // every CTA of the cluster runs before any writes into another's shared memory

    // The chunks of a row begin on 16 bytes: chunk k holds elements 8 k - (what lies before the row's start).  This
    // CTA's are [k0, k1).
    struct Row {
        const T *p;
        int lead, k0, k1;
    };
    auto row_at = [&](int64_t i) {
        Row x;
        x.p = logits + i * a.ldl;
        x.lead = (int)((reinterpret_cast<uintptr_t>(x.p) & 15) / sizeof(T));
        const int all = (V + x.lead + kChunk - 1) / kChunk, per = (all + nc - 1) / nc;
        x.k0 = rank * per;
        x.k1 = min(all, x.k0 + per);
        return x;
    };
    auto fetch = [&](const Row &x, int k, Chunk<T> v[kDeep]) {
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int kk = k + d * kAccThreads;
            if (kk < x.k1) v[d].load(x.p, kk * kChunk - x.lead, V);
            else v[d].none();
        }
    };
    // the root's row, and this CTA's part of the noise (wanted at the end)
    const int64_t root = a.root_row ? a.root_row[r] : (int64_t)a.n + r;
    const bool root_ok = root >= 0 && root < a.rows;
    const Row root_row = row_at(root_ok ? root : 0);
    Chunk<T> ahead[kDeep];
    if (root_ok) fetch(root_row, root_row.k0 + tid, ahead);
    if (!greedy) {
        const int per = (V + nc - 1) / nc;
        for (int i = rank * per + 32 * tid; i < min(V, (rank + 1) * per); i += 32 * kAccThreads)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + i));
    }

    // ---- the request's nodes, in their order, and what is wrong with them
    if (tid == 0 && !root_ok) sm.bad = 1;
    for (int i0 = 0; i0 < a.n; i0 += kAccThreads) {
        const int i = i0 + tid;
        int rq = -1, par = 0, y = 0;
        bool ok = true;
        if (i < a.n) {  // (all of it asked for at once)
            rq = a.req ? a.req[i] : 0;
            par = a.parent[i];
            y = a.token[i];
            const int64_t rw = a.row ? a.row[i] : i, d = a.draft ? a.draft_row[i] : 0;
            ok = par >= -1 && par < i && y >= 0 && y < V && rw >= 0 && rw < a.rows && (!a.draft || (d >= 0 && d < a.draft_rows));
        }
        const bool mine = rq == r;
        const uint32_t ball = __ballot_sync(kFull, mine);
        if (lane == 0) sm.off[warp] = __popc(ball);
        if (!__syncthreads_or(mine)) continue;
        if (mine) {
            int at = sm.total;
            for (int w = 0; w < warp; ++w) at += sm.off[w];
            at += __popc(ball & ((1u << lane) - 1u));
            if (at < kAccNodes) sm.node[at] = i, sm.par[at] = ok ? par : -2, sm.tok[at] = y;
        }
        __syncthreads();
        if (tid == 0) {
            int at = sm.total;
            for (int w = 0; w < kAccWarps; ++w) at += sm.off[w];
            sm.total = at;
        }
        __syncthreads();
    }
    const int total = min(sm.total, kAccNodes);
    if (sm.total > kAccNodes && tid == 0) sm.bad = 1;
    auto row_of = [&](int place) -> int64_t {
        if (place == kRoot) return root;
        const int i = sm.node[place];
        return a.row ? a.row[i] : i;
    };
    static_assert(kAccThreads >= kAccNodes, "a thread a node");
    int up = kNone;
    if (tid < total) {
        const int p = sm.par[tid];
        bool ok = p >= -1;
        up = kRoot;
        if (p >= 0) {  // the parent's place in the list, if it is this request's
            int lo = 0, hi = tid;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sm.node[mid] < p) lo = mid + 1;
                else hi = mid;
            }
            ok = lo < tid && sm.node[lo] == p;
            up = lo;
        }
        if (!ok) sm.bad = 1;
    }
    if (tid < kAccNodes) sm.up[tid] = up;
    cl.barrier_wait();
    __syncthreads();
    int32_t *nodes = a.nodes + (int64_t)r * a.ld_nodes;
    if (sm.bad) {  // the same for every CTA of the cluster
        if (rank == 0) {
            if (tid == 0) a.count[r] = -1, a.next[r] = -1;
            for (int d = tid; d < a.max_depth; d += kAccThreads) nodes[d] = -1;
        }
        return;
    }

    // ---- What a warp has of a round goes to all CTAs (or to the first one): 16 bytes each.  A round's buffer is written
    // again two rounds on, by warps that have had the round between from every warp: all have read it by then.
    int round = 0;
    bool ok = true;
    auto send = [&](uint4 x, int to) {
        if (a.stall && round == 1 && me == parts - 1) return;
        if (lane < to) {
            uint32_t dst, bar;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_addr(&sm.part[round & 1][me])), "r"(lane));
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_addr(&sm.bar[round & 1])), "r"(lane));
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                         "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(bar)
                         : "memory");
        }
    };
    auto receive = [&](uint4 x[kParts / 32]) {  // (past its limit a wait gives up, and the request with it)
        ok = warp_wait<true>(sm.bar + (round & 1), (round >> 1) & 1, &sm.gave_up, &sm.err) && ok;
#pragma unroll
        for (int i = 0; i < kParts / 32; ++i) x[i] = sm.part[round & 1][min(lane + 32 * i, parts - 1)];
        __syncwarp();
        if (ok && tid == 0) mbar_expect_tx(sm.bar + (round & 1), parts * 16);  // for the round after the next
        ++round;
    };
    // the sum of one number from every warp
    auto total_of = [&](float s) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
        send(make_uint4(__float_as_uint(s), 0, 0, 0), nc);
        uint4 x[kParts / 32];
        receive(x);
        s = 0.f;
#pragma unroll
        for (int i = 0; i < kParts / 32; ++i) s += lane + 32 * i < parts ? __uint_as_float(x[i].x) : 0.f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
        return s;
    };
    // ---- statistics of a place's row, in two steps: this CTA's, handed to all; everybody's, joined by every warp
    auto stats_begin = [&](int place) {
        const bool is_root = place == kRoot;
        const Row row = is_root ? root_row : row_at(row_of(place));
        float m = -INFINITY, sum = 0.f;
        int first = INT32_MAX;
        for (int k = row.k0 + tid; k < row.k1; k += kDeep * kAccThreads) {
            Chunk<T> v[kDeep];
            if (is_root && k == row.k0 + tid) {
#pragma unroll
                for (int d = 0; d < kDeep; ++d) v[d] = ahead[d];
            } else {
                fetch(row, k, v);
            }
            float top = m;
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                float x[kChunk];
                v[d].get(x);
#pragma unroll
                for (int j = 0; j < kChunk; ++j) top = max_nan(top, x[j]);
            }
            if (!(top <= m)) {
                sum = scaled(sum, weight_any(m, top, c));
                m = top;
                first = INT32_MAX;
                if (greedy) {
#pragma unroll
                    for (int d = kDeep - 1; d >= 0; --d) {
                        float x[kChunk];
                        v[d].get(x);
#pragma unroll
                        for (int j = kChunk - 1; j >= 0; --j)
                            if (x[j] == m) first = (k + d * kAccThreads) * kChunk - row.lead + j;
                    }
                }
            }
            if (!isinf(m)) {
                if (!greedy) {
                    // exp((x - m) / T) as 2^(x c - m c); what m c was rounded by is made good in the sum
                    const float mc = m * c, off = fmaf(m, c, -mc);
                    float s[4] = {};
                    if (fabsf(mc) < 1048576.f) {
#pragma unroll
                        for (int d = 0; d < kDeep; ++d) {
                            float x[kChunk];
                            v[d].get(x);
#pragma unroll
                            for (int j = 0; j < kChunk; ++j) s[j & 3] += ex2(fmaf(x[j], c, -mc));
                        }
                        sum += ((s[0] + s[1]) + (s[2] + s[3])) * ex2(-off);
                    } else {
#pragma unroll
                        for (int d = 0; d < kDeep; ++d) {
                            float x[kChunk];
                            v[d].get(x);
#pragma unroll
                            for (int j = 0; j < kChunk; ++j) sum += weight(x[j], m, c);
                        }
                    }
                }
            } else {  // +inf somewhere, or nothing but -inf: those count that equal it
#pragma unroll
                for (int d = 0; d < kDeep; ++d) {
                    float x[kChunk];
                    v[d].get(x);
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) {
                        const int kk = k + d * kAccThreads, i = kk * kChunk - row.lead + j;
                        if (kk < row.k1 && i >= 0 && i < V && x[j] == m) {
                            sum += 1.f;
                            first = min(first, i);
                        }
                    }
                }
            }
        }
        float M = m;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) M = max_nan(M, __shfl_xor_sync(kFull, M, s));
        first = __reduce_min_sync(kFull, m == M ? first : INT32_MAX);
        sum = m == M ? sum : scaled(sum, weight_any(m, M, c));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
        send(make_uint4(__float_as_uint(M), __float_as_uint(sum), (uint32_t)first, 0), nc);
    };
    auto stats_end = [&]() {
        uint4 got[kParts / 32];
        receive(got);
        Stat x[kParts / 32];
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < kParts / 32; ++i) {
            x[i] = lane + 32 * i < parts ? Stat{__uint_as_float(got[i].x), __uint_as_float(got[i].y), (int)got[i].z}
                                         : Stat{-INFINITY, 0.f, INT32_MAX};
            M = max_nan(M, x[i].m);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) M = max_nan(M, __shfl_xor_sync(kFull, M, s));
        float sum = 0.f;
        int first = INT32_MAX;
#pragma unroll
        for (int i = 0; i < kParts / 32; ++i) {
            sum += x[i].m == M ? x[i].s : scaled(x[i].s, weight_any(x[i].m, M, c));
            first = min(first, x[i].m == M ? x[i].at : INT32_MAX);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
        first = __reduce_min_sync(kFull, first);
        return Stat{M, sum, first};
    };

    // ---- p of the place after the `gone` children refused there, for every token of this CTA's slice; inv_mine: one
    // over the sum after the g-th
    float inv_mine = 0.f;  // lane g: of the g-th
    auto each_left = [&](int place, int gone, const Stat &st, auto f) {  // f(first of eight tokens, p left of them, p; 0 outside the row)
        const Row row = row_at(row_of(place));
        const float inv_s = 1.f / st.s;
        // one row of q for all refused children (they were drawn from the same one), or another for each
        const int64_t d0 = a.draft_row[sm.node[sm.gone[0]]];
        bool same = true;
        for (int g = 1; g < gone; ++g) same &= a.draft_row[sm.node[sm.gone[g]]] == d0;
        const float *q0 = a.draft + d0 * a.ldd;
        for (int k = row.k0 + tid;; k += kAccThreads) {
            const bool live = k < row.k1;
            if (!__any_sync(kFull, live)) break;  // the shuffles below need the whole warp
            Chunk<T> v;
            float x[kChunk], q[kChunk];
            const int i0 = k * kChunk - row.lead;
            if (live) {
                v.load(row.p, i0, V);
                load8_any(q0, i0, V, q, 0.f);
            } else {
                v.none();
#pragma unroll
                for (int j = 0; j < kChunk; ++j) q[j] = 0.f;
            }
            v.get(x);
            float p0[kChunk], p[kChunk];
#pragma unroll
            for (int j = 0; j < kChunk; ++j) p[j] = p0[j] = i0 + j >= 0 && i0 + j < V ? weight_any(x[j], st.m, c) * inv_s : 0.f;
            for (int g = 0; g < gone; ++g) {
                const float scale = g > 0 ? __shfl_sync(kFull, inv_mine, g - 1) : 1.f;
                const float *qg = same ? nullptr : a.draft + (int64_t)a.draft_row[sm.node[sm.gone[g]]] * a.ldd;
#pragma unroll
                for (int j = 0; j < kChunk; ++j) {
                    const int i = i0 + j;
                    const float qj = same ? q[j] : live && i >= 0 && i < V ? qg[i] : 0.f;
                    p[j] = fmaxf(fmaf(scale, p[j], -qj), 0.f);
                }
            }
            if (live) f(i0, p, p0);
        }
    };

    // ---- the walk
    int place = kRoot, depth = 0, gone = 0;
    Stat st{};
    for (;;) {
        const T *row = logits + row_of(place) * a.ldl;
        int taken = kNone;
        gone = 0;
        float left = 1.f;  // of p, where given tokens are taken out of it
        // The children, 32 nodes at a time, a lane a node, in the order of the list; what they need of the row and of the
        // random numbers is asked for before the row's statistics are waited for.
        bool begun = false;
        for (int w = 0; !begun || (w < total && taken == kNone); w += 32) {
            bool is = w + lane < total && sm.up[w + lane] == place && depth < a.max_depth;
            uint32_t kids = __ballot_sync(kFull, is);
            if (begun && !kids) continue;
            const int y = is ? sm.tok[w + lane] : -1 - lane, node = is ? sm.node[w + lane] : 0;
            float x = 0.f, u = 1.f, q = 1.f;
            if (is && !greedy) {
                x = value(row, y);
                u = a.uniform[node];
                if (a.draft) q = a.draft[(int64_t)a.draft_row[node] * a.ldd + y];
            }
            if (!begun) {
                begun = true;
                stats_begin(place);
                st = stats_end();
                if (!ok) break;
            }
            if (greedy) {
                const uint32_t hit = __ballot_sync(kFull, is && y == st.at);
                if (hit) taken = w + __ffs(hit) - 1;
                continue;
            }
            float p = is ? weight_any(x, st.m, c) / st.s : 0.f;
            if (!a.draft) {
                // a token that was refused before has nothing left
                bool again = (__match_any_sync(kFull, y) & ((1u << lane) - 1u)) != 0;
                for (int g = 0; g < gone; ++g) again |= sm.tok[sm.gone[g]] == y;
                if (again) p = 0.f;
                __syncwarp();
                for (; kids; kids &= kids - 1) {
                    const int j = __ffs(kids) - 1;
                    const float pj = __shfl_sync(kFull, p, j);
                    if (__shfl_sync(kFull, u, j) * left < pj) {
                        taken = w + j;
                        break;
                    }
                    left -= pj;
                    if (lane == 0) sm.gone[gone] = w + j;
                    ++gone;
                }
                __syncwarp();
                continue;
            }
            for (int g = 0; g < gone; ++g) {  // what the nodes before have left of it
                const float scale = g > 0 ? __shfl_sync(kFull, inv_mine, g - 1) : 1.f;
                const float qg = is ? a.draft[(int64_t)a.draft_row[sm.node[sm.gone[g]]] * a.ldd + y] : 0.f;
                p = fmaxf(fmaf(scale, p, -qg), 0.f);
            }
            for (; kids && gone < 32; kids &= kids - 1) {
                // (p is what the refused ones have left of it, unscaled since the last)
                const int j = __ffs(kids) - 1;
                const float scale = gone > 0 ? __shfl_sync(kFull, inv_mine, gone - 1) : 1.f;
                const float pj = __shfl_sync(kFull, p, j) * scale;
                if (__shfl_sync(kFull, u, j) * __shfl_sync(kFull, q, j) < pj) {
                    taken = w + j;
                    break;
                }
                // refused: p <- max(p - q, 0) / sum
                const float qi = is ? a.draft[(int64_t)a.draft_row[sm.node[w + j]] * a.ldd + y] : 0.f;
                p = fmaxf(fmaf(scale, p, -qi), 0.f);
                if (lane == 0) sm.gone[gone] = w + j;
                __syncwarp();
                ++gone;
                // the sum is needed only where another child follows
                bool more = (kids & (kids - 1)) != 0;
                for (int v = w + 32; v < total && !more; v += 32) more = __any_sync(kFull, v + lane < total && sm.up[v + lane] == place);
                if (!more || gone == 32) break;
                float s = 0.f;
                each_left(place, gone, st, [&](int, const float *pl, const float *) {
#pragma unroll
                    for (int z = 0; z < kChunk; ++z) s += pl[z];
                });
                s = total_of(s);
                if (!ok) break;
                if (lane == gone - 1) inv_mine = s > 0.f ? 1.f / s : 0.f;
            }
            if (gone == 32 || !ok) break;
        }
        if (taken == kNone || !ok) break;
        if (rank == 0 && tid == 0) nodes[depth] = sm.node[taken];
        place = taken;
        ++depth;
    }
    // ---- the token after the last accepted one
    int token = st.at;
    if (!greedy && ok) {
        // `all`: where rounding left nothing of p, the draw is from p as it was
        Best best{-INFINITY, INT32_MAX}, all = best;
        if (a.draft && gone > 0) {
            each_left(place, gone, st, [&](int i0, const float *p, const float *p0) {
                float e[kChunk];
                load8_any(noise, i0, V, e, 1.f);
#pragma unroll
                for (int j = 0; j < kChunk; ++j) {
                    const float score = p[j] > 0.f ? __fdividef(p[j], e[j]) : -INFINITY;
                    if (score > best.score) best = Best{score, i0 + j};
                    const float score0 = p0[j] > 0.f ? __fdividef(p0[j], e[j]) : -INFINITY;
                    if (score0 > all.score) all = Best{score0, i0 + j};
                }
            });
        } else {
            // the logarithm of p / e, up to a constant; refused tokens are left out
            const Row row = row_at(row_of(place));
            const bool inf = isinf(st.m);
            for (int k = row.k0 + tid; k < row.k1; k += 2 * kAccThreads) {
                Chunk<T> v[2];
                float e[2][kChunk];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const int kk = k + d * kAccThreads;
                    if (kk < row.k1) {
                        v[d].load(row.p, kk * kChunk - row.lead, V);
                        load8_any(noise, kk * kChunk - row.lead, V, e[d], INFINITY);
                    } else {
                        v[d].none();
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) e[d][j] = INFINITY;
                    }
                }
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    float x[kChunk];
                    v[d].get(x);
                    const int i0 = (k + d * kAccThreads) * kChunk - row.lead;
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) {
                        const float lp = inf ? (x[j] == st.m ? 0.f : -INFINITY) : (x[j] - st.m) * c;
                        x[j] = lp - lg2(e[d][j]);
                    }
                    for (int g = 0; g < gone; ++g) {
                        const int j = sm.tok[sm.gone[g]] - i0;
                        if (j >= 0 && j < kChunk) {
#pragma unroll
                            for (int z = 0; z < kChunk; ++z)
                                if (z == j) {
                                    if (x[z] > -INFINITY) all = better(all, Best{x[z], i0 + z});  // (in the order of the list)
                                    x[z] = -INFINITY;
                                }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) top = fmaxf(top, x[j]);
                    if (top > best.score) {
                        int at = 0;
#pragma unroll
                        for (int j = kChunk - 1; j >= 0; --j) at = x[j] == top ? j : at;
                        best = Best{top, i0 + at};
                    }
                }
            }
        }
        auto over = [&](Best &b) {
#pragma unroll
            for (int s = 16; s > 0; s >>= 1)
                b = better(b, Best{__shfl_xor_sync(kFull, b.score, s), __shfl_xor_sync(kFull, b.at, s)});
        };
        over(best);
        over(all);
        send(make_uint4(__float_as_uint(best.score), (uint32_t)best.at, __float_as_uint(all.score), (uint32_t)all.at), 1);
        if (rank == 0 && warp == 0) {
            uint4 x[kParts / 32];
            receive(x);
            for (int w = 0; w < 2 && (w == 0 || token == INT32_MAX); ++w) {
                best = Best{-INFINITY, INT32_MAX};
#pragma unroll
                for (int i = 0; i < kParts / 32; ++i)
                    best = better(best, w ? Best{__uint_as_float(x[i].z), (int)x[i].w} : Best{__uint_as_float(x[i].x), (int)x[i].y});
                over(best);
                token = best.at;
            }
        }
    }
    if (rank == 0 && warp == 0) {
        if (!ok) depth = -1;  // a wait gave up: nothing of the walk stands, the nodes that it has written either
        if (lane == 0) {
            a.count[r] = depth;
            a.next[r] = depth < 0 ? -1 : token >= 0 && token < V ? token : 0;
        }
        __syncwarp();
        for (int d = max(depth, 0) + lane; d < a.max_depth; d += 32) nodes[d] = -1;
    }
    // others may still be sending to a warp that gave up: it stays until they have ended
    if (!ok) cl.sync();
}

}  // namespace

cudaError_t launch_tree_accept(const w12_accept_args &x, cudaStream_t s) {
    AcceptArgs a{};
    a.logits = x.logits;
    a.ldl = x.ldl, a.rows = x.rows;
    a.V = (int)x.V;
    a.token = x.token, a.parent = x.parent, a.req = x.req, a.row = x.row, a.root_row = x.root_row;
    a.n = (int)x.n, a.R = (int)x.R;
    a.temperature = x.temperature;
    a.temperature1 = x.temperature1;
    a.uniform = x.uniform, a.noise = x.noise;
    a.ld_noise = x.ld_noise;
    a.draft = x.draft;
    a.ldd = x.ldd, a.draft_rows = x.draft_rows;
    a.draft_row = x.draft_row;
    a.max_depth = x.max_depth & ~W12_ACCEPT_TEST_STALL;
    a.stall = x.max_depth & W12_ACCEPT_TEST_STALL;
    a.count = x.count, a.nodes = x.nodes, a.next = x.next;
    a.ld_nodes = x.ld_nodes;
    // As large a cluster as two CTAs a multiprocessor allow, each with 4096 tokens at least.  Few requests: CTAs of 256,
    // whose waits cost less (4 tokens of 32000 greedy, in a graph: 9.7 us, with 512 12.3); many: of 512, which keep more of the rows on
    // their way with 64 registers a thread (64 chains of 7 over 131072: 65 us, with 256 81; clusters of 8 for all 83).
    int nc = 1;
    while (nc < kMaxCluster && x.V > (int64_t)nc * 4096 && x.R * nc * 2 <= 2 * W12_PLAN_SMS) nc *= 2;
    const bool few = x.R <= 16;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(x.R * nc));
    cfg.blockDim = dim3(few ? 256 : 512);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = nc;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (x.logits32) return few ? cudaLaunchKernelEx(&cfg, k_accept<float, 256>, a) : cudaLaunchKernelEx(&cfg, k_accept<float, 512>, a);
    return few ? cudaLaunchKernelEx(&cfg, k_accept<uint16_t, 256>, a) : cudaLaunchKernelEx(&cfg, k_accept<uint16_t, 512>, a);
}

}  // namespace w12
