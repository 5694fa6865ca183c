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
// of up to 8 CTAs takes a request, each CTA a slice of the vocabulary, every
// thread 32 logits in registers; the CTAs hand their (maximum, sum, first
// maximum) to each other through distributed shared memory, one cluster barrier a
// round, and then all take the same decisions from the same numbers.  A round
// may take further rows of the path that is most likely next (first children)
// along with the place's own, which saves a round's latency where they are
// needed and costs a row's bytes where they are not.
#include <cooperative_groups.h>

#include <cstdint>
#include <cuda_runtime.h>

#include "w12_device.cuh"
#include "w12_internal.h"

namespace w12 {
namespace {

namespace cg = cooperative_groups;

constexpr int kAccThreads = 512;
constexpr int kAccWarps = kAccThreads / 32;
constexpr int kAccNodes = W12_TREE_MAX_BUDGET;  // of a request
constexpr int kChunk = 8;                       // logits of one load
constexpr int kDeep = 4;                        // chunks of a thread in flight
constexpr int kMaxCluster = 8;
constexpr int kMaxAhead = 8;                    // rows of a round
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
    int max_depth, ahead;
    int32_t *count, *nodes, *next;
    int64_t ld_nodes;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Eight values from element i0 on; -inf outside [0, n).  `vec`: the address of
// i0 is aligned to 16 bytes (the same for every chunk of a row).
__device__ __forceinline__ void load8(const uint16_t *row, int i0, int n, float x[kChunk]) {
    if (i0 >= 0 && i0 + kChunk <= n) {
        const uint4 u = *reinterpret_cast<const uint4 *>(row + i0);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
        x[j] = i0 + j >= 0 && i0 + j < n ? __uint_as_float((uint32_t)row[i0 + j] << 16) : -INFINITY;
}
__device__ __forceinline__ void load8(const float *row, int i0, int n, float x[kChunk]) {
    if (i0 >= 0 && i0 + kChunk <= n) {
        const float4 a = *reinterpret_cast<const float4 *>(row + i0), b = *reinterpret_cast<const float4 *>(row + i0 + 4);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        return;
    }
#pragma unroll
    for (int j = 0; j < kChunk; ++j) x[j] = i0 + j >= 0 && i0 + j < n ? row[i0 + j] : -INFINITY;
}
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

// A row's statistics: its maximum, the sum of exp((x - maximum) / T), the first place of the maximum.
struct Stat {
    float m, s;
    int at;
};
__device__ __forceinline__ float weight(float x, float m, float c) {  // exp((x - m) / T) of a finite maximum
    return ex2((x - m) * c);
}
// An infinite maximum leaves the values that equal it, each with weight 1.
__device__ __forceinline__ float weight_any(float x, float m, float c) {
    return isinf(m) ? (x == m ? 1.f : 0.f) : weight(x, m, c);
}
__device__ __forceinline__ Stat join(const Stat &a, const Stat &b, float c) {
    Stat r;
    r.m = fmaxf(a.m, b.m);
    r.s = a.s * (a.m == r.m ? 1.f : weight_any(a.m, r.m, c)) + b.s * (b.m == r.m ? 1.f : weight_any(b.m, r.m, c));
    r.at = a.m == b.m ? min(a.at, b.at) : a.m > b.m ? a.at : b.at;
    return r;
}

struct Best {  // of a draw: the highest score, the lowest token of that score
    float score;
    int at;
};
__device__ __forceinline__ Best better(const Best &a, const Best &b) {
    return b.score > a.score || (b.score == a.score && b.at < a.at) ? b : a;
}

struct Shared {
    Stat part[2][kMaxAhead][kMaxCluster];  // written by the cluster's CTAs, by the parity of the round
    Best best[2][kMaxCluster];
    float sums[2][kMaxCluster];
    Stat warp_part[kMaxAhead][kAccWarps];
    Best warp_best[2][kAccWarps];
    float warp_sum[kAccWarps];
    Stat stat[kAccNodes + 1];              // of the rows done; the last is the root's
    uint8_t have[kAccNodes + 1];
    int node[kAccNodes];                   // the request's nodes, ascending
    int up[kAccNodes], tok[kAccNodes], first[kAccNodes + 1];
    float px[kAccNodes], u[kAccNodes], q[kAccNodes];  // of the children of the place
    uint32_t kids[kAccNodes / 32];
    int off[kAccWarps + 1];
    int todo[kMaxAhead];
    int gone[kAccNodes];                   // children refused at the place
    float inv[kAccNodes];                  // 1 / sum after each
    int n_todo, n_gone, taken, total, bad;
};

template <typename T>
__global__ __launch_bounds__(kAccThreads, 1) void k_accept(const __grid_constant__ AcceptArgs a) {
    __shared__ Shared sm;
    cg::cluster_group cl = cg::this_cluster();
    const int nc = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int r = (int)blockIdx.x / nc, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int V = a.V;
    const T *logits = static_cast<const T *>(a.logits);
    const float temp = a.temperature ? a.temperature[r] : a.temperature1;
    const bool greedy = !(temp > 0.f);
    const float c = greedy ? kLog2eF : fminf(fmaxf(kLog2eF / temp, 1e-30f), 1e30f);  // of any temperature: no 0 * inf
    const float *noise = greedy ? nullptr : a.noise + (int64_t)r * a.ld_noise;

    cl.barrier_arrive();  // every CTA of the cluster runs before any writes into another's shared memory
    if (!greedy) {        // this CTA's part of the noise, wanted at the end
        const int per = (V + nc - 1) / nc;
        for (int i = rank * per + 32 * tid; i < min(V, (rank + 1) * per); i += 32 * kAccThreads)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + i));
    }

    // ---- the request's nodes, in their order, and what is wrong with them
    if (tid == 0) sm.total = 0, sm.bad = 0;
    for (int i = tid; i <= kAccNodes; i += kAccThreads) sm.first[i] = kAccNodes, sm.have[i] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < a.n; i0 += kAccThreads) {
        const int i = i0 + tid;
        const bool mine = i < a.n && (a.req ? a.req[i] : 0) == r;
        const uint32_t ball = __ballot_sync(kFull, mine);
        if (lane == 0) sm.off[warp] = __popc(ball);
        __syncthreads();
        if (tid == 0) {
            int at = sm.total;
            for (int w = 0; w < kAccWarps; ++w) {
                const int k = sm.off[w];
                sm.off[w] = at;
                at += k;
            }
            sm.total = at;
        }
        __syncthreads();
        if (mine) {
            const int at = sm.off[warp] + __popc(ball & ((1u << lane) - 1u));
            if (at < kAccNodes) sm.node[at] = i;
        }
        __syncthreads();
    }
    const int total = min(sm.total, kAccNodes);
    if (sm.total > kAccNodes && tid == 0) sm.bad = 1;
    auto row_of = [&](int local) -> int64_t {  // kAccNodes: the root
        if (local == kAccNodes) return a.root_row ? a.root_row[r] : (int64_t)a.n + r;
        const int i = sm.node[local];
        return a.row ? a.row[i] : i;
    };
    if (tid < total) {
        const int i = sm.node[tid], p = a.parent[i], y = a.token[i];
        int up = kAccNodes;
        bool ok = p >= -1 && p < i && y >= 0 && y < V;
        if (p >= 0 && ok) {  // the parent's place in the list, if it is this request's
            int lo = 0, hi = tid;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sm.node[mid] < p) lo = mid + 1;
                else hi = mid;
            }
            ok = lo < tid && sm.node[lo] == p;
            up = lo;
        }
        const int64_t rw = row_of(tid);
        ok = ok && rw >= 0 && rw < a.rows;
        if (a.draft) {
            const int64_t d = a.draft_row[i];
            ok = ok && d >= 0 && d < a.draft_rows;
        }
        sm.up[tid] = up;
        sm.tok[tid] = y;
        if (ok) atomicMin(&sm.first[up], tid);
        else sm.bad = 1;
    }
    if (tid == 0) {
        const int64_t rw = row_of(kAccNodes);
        if (rw < 0 || rw >= a.rows) sm.bad = 1;
    }
    __syncthreads();
    cl.barrier_wait();
    int32_t *nodes = a.nodes + (int64_t)r * a.ld_nodes;
    if (sm.bad) {  // the same for every CTA of the cluster
        if (rank == 0) {
            if (tid == 0) a.count[r] = -1, a.next[r] = -1;
            for (int d = tid; d < a.max_depth; d += kAccThreads) nodes[d] = -1;
        }
        return;
    }

    // The chunks of a row begin on 16 bytes: chunk k holds elements 8 k - (what lies before the row's start).
    auto lead_of = [&](const T *row) {
        return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    };
    auto range_of = [&](int lead, int &k0, int &k1) {
        const int all = (V + lead + kChunk - 1) / kChunk, per = (all + nc - 1) / nc;
        k0 = rank * per;
        k1 = min(all, k0 + per);
    };

    // ---- statistics of the rows of a round
    int round = 0;
    auto stats_round = [&]() {
        const int todo = sm.n_todo;
        for (int b = 0; b < todo; ++b) {
            const T *row = logits + row_of(sm.todo[b]) * a.ldl;
            const int lead = lead_of(row);
            int k0, k1;
            range_of(lead, k0, k1);
            Stat st{-INFINITY, 0.f, INT32_MAX};
            for (int k = k0 + tid; k < k1; k += kDeep * kAccThreads) {
                float x[kDeep][kChunk];
#pragma unroll
                for (int d = 0; d < kDeep; ++d) {
                    const int kk = k + d * kAccThreads;
                    if (kk < k1) load8(row, kk * kChunk - lead, V, x[d]);
                    else
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) x[d][j] = -INFINITY;
                }
                float m = st.m;
#pragma unroll
                for (int d = 0; d < kDeep; ++d)
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) m = fmaxf(m, x[d][j]);
                if (m > st.m) {
                    if (st.s > 0.f) st.s *= weight_any(st.m, m, c);
                    st.at = INT32_MAX;
                    if (greedy) {
#pragma unroll
                        for (int d = kDeep - 1; d >= 0; --d)
#pragma unroll
                            for (int j = kChunk - 1; j >= 0; --j)
                                if (x[d][j] == m) st.at = (k + d * kAccThreads) * kChunk - lead + j;
                    }
                    st.m = m;
                }
                if (!isinf(m)) {
#pragma unroll
                    for (int d = 0; d < kDeep; ++d)
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) st.s += weight(x[d][j], m, c);
                } else {  // +inf somewhere, or nothing but -inf: those count that equal it
                    for (int d = 0; d < kDeep; ++d)
                        for (int j = 0; j < kChunk; ++j) {
                            const int kk = k + d * kAccThreads, i = kk * kChunk - lead + j;
                            if (kk < k1 && i >= 0 && i < V && x[d][j] == m) {
                                st.s += 1.f;
                                st.at = min(st.at, i);
                            }
                        }
                }
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) {
                Stat o;
                o.m = __shfl_xor_sync(kFull, st.m, s);
                o.s = __shfl_xor_sync(kFull, st.s, s);
                o.at = __shfl_xor_sync(kFull, st.at, s);
                st = (lane & s) ? join(o, st, c) : join(st, o, c);
            }
            if (lane == 0) sm.warp_part[b][warp] = st;
        }
        __syncthreads();
        // one warp a row joins the warps' and hands the CTA's to every CTA of the cluster
        if (warp < todo) {
            Stat st = lane < kAccWarps ? sm.warp_part[warp][lane] : Stat{-INFINITY, 0.f, INT32_MAX};
#pragma unroll
            for (int s = 8; s > 0; s >>= 1) {
                Stat o;
                o.m = __shfl_xor_sync(kFull, st.m, s);
                o.s = __shfl_xor_sync(kFull, st.s, s);
                o.at = __shfl_xor_sync(kFull, st.at, s);
                st = (lane & s) ? join(o, st, c) : join(st, o, c);
            }
            st.m = __shfl_sync(kFull, st.m, 0);
            st.s = __shfl_sync(kFull, st.s, 0);
            st.at = __shfl_sync(kFull, st.at, 0);
            if (lane < nc) *cl.map_shared_rank(&sm.part[round & 1][warp][rank], lane) = st;
        }
        cl.sync();
        if (tid < todo) {
            Stat st = sm.part[round & 1][tid][0];
            for (int k = 1; k < nc; ++k) st = join(st, sm.part[round & 1][tid][k], c);
            sm.stat[sm.todo[tid]] = st;
            sm.have[sm.todo[tid]] = 1;
        }
        ++round;
        __syncthreads();
    };

    // ---- p of the place after the children refused there, for every token of this CTA's slice
    int sums_done = 0;
    // One row of q for all refused children (they were drawn from the same one) or another for each.
    auto one_row = [&](int n_gone) {
        for (int g = 1; g < n_gone; ++g)
            if (a.draft_row[sm.node[sm.gone[g]]] != a.draft_row[sm.node[sm.gone[0]]]) return false;
        return true;
    };
    // calls f(token, p left of it, p) for the slice
    auto each_left = [&](int place, int n_gone, auto f) {
        const T *row = logits + row_of(place) * a.ldl;
        const int lead = lead_of(row);
        int k0, k1;
        range_of(lead, k0, k1);
        const Stat st = sm.stat[place];
        const float inv_s = 1.f / st.s;
        const bool same = one_row(n_gone);
        const float *q0 = a.draft + (int64_t)a.draft_row[sm.node[sm.gone[0]]] * a.ldd;
        for (int k = k0 + tid; k < k1; k += kAccThreads) {
            float x[kChunk], q[kChunk];
            const int i0 = k * kChunk - lead;
            load8(row, i0, V, x);
            load8_any(q0, i0, V, q, 0.f);
#pragma unroll
            for (int j = 0; j < kChunk; ++j) {
                const int i = i0 + j;
                if (i < 0 || i >= V) continue;
                const float p0 = weight_any(x[j], st.m, c) * inv_s;
                float p = p0;
                for (int g = 0; g < n_gone; ++g) {
                    const float qg = same ? q[j] : a.draft[(int64_t)a.draft_row[sm.node[sm.gone[g]]] * a.ldd + i];
                    p = fmaxf(fmaf(g > 0 ? sm.inv[g - 1] : 1.f, p, -qg), 0.f);
                }
                f(i, p, p0);
            }
        }
    };

    // ---- the walk
    int place = kAccNodes, depth = 0;
    for (;;) {
        // a round of rows if this place's is not there yet: its own, and the first children's below it
        if (!sm.have[place]) {
            if (tid == 0) {
                int k = 0, at = place;
                const int most = min(a.ahead, a.max_depth + 1 - depth);
                while (k < most && at != kAccNodes + 1) {
                    sm.todo[k++] = at;
                    at = sm.first[at] < kAccNodes ? sm.first[at] : kAccNodes + 1;
                }
                sm.n_todo = k;
            }
            __syncthreads();
            stats_round();
        }
        const Stat st = sm.stat[place];
        // the children, each with its token's probability
        if (tid < kAccNodes) {
            const bool kid = tid < total && sm.up[tid] == place && depth < a.max_depth;
            const uint32_t ball = __ballot_sync(kFull, kid);
            if (lane == 0) sm.kids[warp] = ball;
            if (kid) {
                const int i = sm.node[tid], y = sm.tok[tid];
                if (greedy) {
                    sm.px[tid] = y == st.at ? 1.f : 0.f;
                } else {
                    sm.px[tid] = weight_any(value(logits + row_of(place) * a.ldl, y), st.m, c) / st.s;
                    sm.u[tid] = a.uniform[i];
                    sm.q[tid] = a.draft ? a.draft[(int64_t)a.draft_row[i] * a.ldd + y] : 1.f;
                }
            }
        }
        __syncthreads();
        // one after the other; every CTA goes the same way
        int n_gone = 0, from = 0;
        for (;;) {
            if (tid == 0) {
                int taken = -1, stop = 0;
                double left = 1.0;  // of p where tokens are taken out of it
                for (int w = from >> 5; w < kAccNodes / 32 && taken < 0 && !stop; ++w) {
                    uint32_t bits = sm.kids[w];
                    if (w == from >> 5) bits &= ~0u << (from & 31);
                    for (; bits; bits &= bits - 1) {
                        const int k = 32 * w + __ffs(bits) - 1;
                        float p = sm.px[k];
                        if (greedy) {
                            if (p > 0.f) {
                                taken = k;
                                break;
                            }
                            continue;
                        }
                        if (a.draft) {
                            const int y = sm.tok[k];
                            for (int g = 0; g < n_gone; ++g) {
                                const float qg = a.draft[(int64_t)a.draft_row[sm.node[sm.gone[g]]] * a.ldd + y];
                                p = fmaxf(fmaf(g > 0 ? sm.inv[g - 1] : 1.f, p, -qg), 0.f);
                            }
                            if (n_gone > 0) p *= sm.inv[n_gone - 1];
                            if (sm.u[k] * sm.q[k] < p) {
                                taken = k;
                                break;
                            }
                            sm.gone[n_gone++] = k;
                            // the sum of what is left is needed only where another child follows
                            uint32_t more = bits & (bits - 1);
                            for (int v = w + 1; v < kAccNodes / 32; ++v) more |= sm.kids[v];
                            if (more) stop = k + 1;
                            break;
                        }
                        for (int g = 0; g < n_gone; ++g)
                            if (sm.tok[sm.gone[g]] == sm.tok[k]) p = 0.f;
                        if ((double)sm.u[k] * left < (double)p) {
                            taken = k;
                            break;
                        }
                        sm.gone[n_gone++] = k;
                        left -= (double)p;
                    }
                }
                sm.taken = taken;
                sm.n_gone = n_gone;
                sm.off[0] = stop;
            }
            __syncthreads();
            n_gone = sm.n_gone;
            from = sm.off[0];
            if (from == 0) break;
            // p <- max(p - q, 0) / sum: the sum, over the cluster
            float s = 0.f;
            if (tid == 0) sm.inv[n_gone - 1] = 1.f;
            each_left(place, n_gone, [&](int, float p, float) { s += p; });
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
            if (lane == 0) sm.warp_sum[warp] = s;
            __syncthreads();
            if (warp == 0) {
                s = lane < kAccWarps ? sm.warp_sum[lane] : 0.f;
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
                s = __shfl_sync(kFull, s, 0);
                if (lane < nc) *cl.map_shared_rank(&sm.sums[sums_done & 1][rank], lane) = s;
            }
            cl.sync();
            if (tid == 0) {
                float all = 0.f;
                for (int k = 0; k < nc; ++k) all += sm.sums[sums_done & 1][k];
                sm.inv[n_gone - 1] = all > 0.f ? 1.f / all : 0.f;
            }
            ++sums_done;
            __syncthreads();
        }
        if (sm.taken < 0) break;
        if (rank == 0 && tid == 0) nodes[depth] = sm.node[sm.taken];
        place = sm.taken;
        ++depth;
        __syncthreads();
    }
    // ---- the token after the last accepted one
    const Stat st = sm.stat[place];
    int token = st.at;
    if (!greedy) {
        const int n_gone = sm.n_gone;
        // `all`: where rounding left nothing of p, the draw is from p as it was
        Best best{-INFINITY, INT32_MAX}, all = best;
        if (a.draft && n_gone > 0) {
            each_left(place, n_gone, [&](int i, float p, float p0) {
                const float e = noise[i], score = p > 0.f ? __fdividef(p, e) : -INFINITY;
                if (score > best.score) best = Best{score, i};
                const float score0 = __fdividef(p0, e);
                if (score0 > all.score) all = Best{score0, i};
            });
        } else {
            // the logarithm of p / e, up to a constant; refused tokens are left out
            const T *row = logits + row_of(place) * a.ldl;
            const int lead = lead_of(row);
            int k0, k1;
            range_of(lead, k0, k1);
            const bool inf = isinf(st.m);
            for (int k = k0 + tid; k < k1; k += 2 * kAccThreads) {
                float x[2][kChunk], e[2][kChunk];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const int kk = k + d * kAccThreads;
                    if (kk < k1) {
                        load8(row, kk * kChunk - lead, V, x[d]);
                        load8_any(noise, kk * kChunk - lead, V, e[d], INFINITY);
                    } else {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) x[d][j] = -INFINITY, e[d][j] = INFINITY;
                    }
                }
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) {
                        const float lp = inf ? (x[d][j] == st.m ? 0.f : -INFINITY) : (x[d][j] - st.m) * c;
                        const float score = lp - __log2f(e[d][j]);
                        if (score > best.score) {
                            const int i = (k + d * kAccThreads) * kChunk - lead + j;
                            bool out = false;
                            for (int g = 0; g < n_gone; ++g) out |= sm.tok[sm.gone[g]] == i;
                            if (i < 0 || i >= V) continue;
                            if (!out) best = Best{score, i};
                            else if (score > all.score) all = Best{score, i};
                        }
                    }
            }
        }
        auto over = [&](Best &b, int width) {
            for (int s = width / 2; s > 0; s >>= 1)
                b = better(b, Best{__shfl_xor_sync(kFull, b.score, s), __shfl_xor_sync(kFull, b.at, s)});
        };
        over(best, 32);
        over(all, 32);
        if (lane == 0) sm.warp_best[0][warp] = best, sm.warp_best[1][warp] = all;
        __syncthreads();
        if (warp < 2) {
            best = lane < kAccWarps ? sm.warp_best[warp][lane] : Best{-INFINITY, INT32_MAX};
            over(best, kAccWarps);
            if (lane == 0) *cl.map_shared_rank(&sm.best[warp][rank], 0) = best;
        }
        cl.sync();
        if (rank == 0) {
            for (int w = 0; w < 2 && (w == 0 || token == INT32_MAX); ++w) {
                best = sm.best[w][0];
                for (int k = 1; k < nc; ++k) best = better(best, sm.best[w][k]);
                token = best.at;
            }
        }
    }
    if (rank == 0) {
        if (tid == 0) {
            a.count[r] = depth;
            a.next[r] = token >= 0 && token < V ? token : 0;
        }
        for (int d = depth + tid; d < a.max_depth; d += kAccThreads) nodes[d] = -1;
    }
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
    a.max_depth = x.max_depth;
    a.ahead = 1;
    a.count = x.count, a.nodes = x.nodes, a.next = x.next;
    a.ld_nodes = x.ld_nodes;
    int nc = 1;
    while (nc < kMaxCluster && x.V > (int64_t)nc * 4096) nc *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(x.R * nc));
    cfg.blockDim = dim3(kAccThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = nc;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return x.logits32 ? cudaLaunchKernelEx(&cfg, k_accept<float>, a) : cudaLaunchKernelEx(&cfg, k_accept<uint16_t>, a);
}

}  // namespace w12
