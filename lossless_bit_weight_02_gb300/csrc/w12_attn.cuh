// What the kernels of the tree attention share: the workspace, the cut of the
// work, and who sees what.
//
// Keys of request r are numbered: its ctx cached tokens from 0, then, from ctx
// rounded up to `tree_align`, its cnt tree nodes in the order of the call
// ("rank").  They are walked in blocks of BN keys from k0, the first key that
// any of its nodes sees rounded down to a block.  Query rows of a key/value head are (rank, head of the
// group), rank first; an item is IM rows of one (request, head), with kb
// blocks to walk.
//
// The work is a line of units, in the order (request, head, row tile, block):
// a block of an item costs more where it feeds two streams of the tcgen05
// kernel (more than 128 rows), and the last of an item more than the others.
// The line is cut into ranges of equal length whatever the requests' lengths; a range is one CTA's work,
// and a block belongs to the range of its last unit.  An item inside one range
// is finished there; of an item that several ranges share each leaves a
// partial (running maximum, sum and FP32 output of its blocks), and a last
// kernel joins them in the order of the ranges.  The cut depends on the inputs
// alone, so the grid never changes a result.
#pragma once

#include <cstdint>

#include "w12_device.cuh"
#include "w12_internal.h"
#include "w12_stream.cuh"

namespace w12 {

constexpr int kAttnMaxNodes = W12_TREE_MAX_BUDGET;  // per request
constexpr int kMaskWords = kAttnMaxNodes / 32;
constexpr int kAttnTcRows = 256;  // query rows of an item of the tcgen05 kernel
constexpr int kAttnTcBlock = 128; // keys of its blocks
// Units of a block that feeds two streams' rows, and of another (64 nodes over 128k tokens: 212 us; 4 : 3 227,
// 1 : 1 223), and of an item's end, its epilogue and masked blocks, where every range is at least that long
// (8 x 256 nodes over 8k 242.6 us, without 246.0; four windowed requests 41.9, without 43.4).
constexpr int kAttnTcPair = 8, kAttnTcOne = 7;
constexpr int kAttnTcExtra = 20;
constexpr float kLog2e = 1.4426950408889634f;

struct alignas(16) ReqInfo {
    int32_t start;  // its nodes: order[start .. start + cnt)
    int32_t cnt;    // nodes (0 if the request is in error)
    int32_t ctx;    // cached tokens
    int32_t k0;     // first key walked, a multiple of BN
    int32_t kb;     // blocks per item
    int32_t tiles;  // items per head
    int32_t lo_max; // from this key on every node sees every cached token
    int32_t flags;  // kReqBad, and twice (1 + its first node) if its nodes follow one another in the call
};
constexpr int kReqBad = 1;  // a node of the request, or the request, is in error

// A segment: the blocks of one item that fall into one range.
struct alignas(16) Seg {
    int32_t start, cnt, ctx, lo_max;  // of the request (ReqInfo)
    int32_t r, h, t, rows;            // item: request, head, row tile, rows
    int32_t nb, key0, key_lo, slot;   // blocks; the first one's first key; no key before key_lo is read; of its partial
    int32_t pair, whole;              // more than one stream's rows; all blocks of its item
    int64_t next;                     // the unit after it
    int32_t node0, pad[3];            // the first node, if the request's nodes follow one another, else -1
};

// An item that several ranges share: its partials are those from slot `first`
// and of the ranges c .. last.
struct alignas(16) JoinInfo {
    int32_t r, h, t, c;
    int32_t last, first, pad[2];
};

// Workspace: [0, 256) error word, ticket, timeout word, Geometry::extra, number of
// joins | ReqInfo [R] | cum
// [R + 1] | Seg [G] |
// JoinInfo [G] | order, pos, depth [n] | masks [n][8] | (max, sum)
// of the partials | partials.  A partial lies as [D / 4][IM][4], so that
// threads of neighbouring rows read and write neighbouring addresses.
struct AttnWs {
    int32_t *err, *ticket, *timeout, *extra, *joins;
    ReqInfo *req;
    int64_t *cum;      // blocks before request r
    Seg *range;        // the first segment of every range (nb = 0: it has none)
    JoinInfo *join;
    int32_t *order;    // node at sorted position p
    int32_t *pos;      // sorted position of node i, -1: in no request
    int32_t *depth;    // by sorted position; 0: the node is in error
    uint32_t *mask;    // by sorted position: ranks it sees
    float2 *ml;        // [2G][IM]
    float *part;       // [2G][D / 4][IM][4]
};

// The variant of a call: a rule on sizes alone (attn_shape).
struct AttnShape {
    int IM;  // query rows of an item
    int BN;  // keys of a block
    int G;   // ranges
    bool tc;
};

struct AttnArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv;
    uint16_t *o;
    int64_t ldo;
    int n, R, Hq, H, group;
    const uint16_t *ck, *cv;
    int64_t pages, page_stride, token_stride, head_stride;
    int page, page_shift;  // page_shift: log2 of page, or -1
    const int32_t *table;
    int64_t ld_table;
    int width;
    const int32_t *ctx_len, *parent, *req;
    float scale, softcap;
    int window;
    AttnWs ws;
    int G;
    int q_nodes;  // nodes of one copy of queries
    int stall;    // W12_ATTN_TEST_STALL
};

// x / y for x >= 0, y > 0: a 64-bit division takes several times a 32-bit one,
// and unit counts beyond 32 bits are rare.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// Range c holds the units [begin(c), begin(c + 1)); at least `least` units
// each: with a block's cost a range between two others of an item has a block
// of it.
struct Cut {
    int64_t q;
    int rem, G;
    __device__ __forceinline__ Cut(int64_t total, int most, int least) {
        G = total >= (int64_t)least * most ? most : (total >= least ? (int)quotient(total, least) : 1);
        q = quotient(total, G);
        rem = (int)(total - q * G);
    }
    __device__ __forceinline__ int64_t begin(int c) const { return q * c + (c < rem ? c : rem); }
    __device__ __forceinline__ int of(int64_t x) const {  // the range of unit x
        return x < (q + 1) * rem ? (int)quotient(x, q + 1) : rem + (int)quotient(x - (q + 1) * rem, q);
    }
};

// Geometry of a variant's items.
struct Geometry {
    int IM, BN, pair_rows;  // rows of an item; keys of a block; an item of more rows feeds two streams
    int w_pair, w_one;      // units of a block of such an item, and of another
    int tree_align;         // the number of a request's first node is a multiple of this power of two
    int extra;              // units of an item's last block beyond the others'
    __device__ __forceinline__ int tree0(int ctx) const { return (ctx + tree_align - 1) & -tree_align; }
    __device__ __forceinline__ int least() const { return extra + (IM > pair_rows ? w_pair : w_one); }
    // complete blocks in the first z units of an item
    __device__ __forceinline__ int blocks(int64_t z, int w, int kb) const {
        const int b = (int)quotient(z, w);
        return z >= (int64_t)w * kb + extra ? kb : b < kb - 1 ? b : kb - 1;
    }
};

// The item of unit x of request r (ri, whose units begin at cum): its head and
// tile, where it begins and what a block of it costs.
struct ItemAt {
    int h, t, w, rows;
    int64_t begin, end;
    __device__ __forceinline__ ItemAt(const Geometry &g, int group, const ReqInfo &ri, int64_t cum, int64_t x) {
        const int all = ri.cnt * group, left = all - (ri.tiles - 1) * g.IM;  // rows; of the last tile
        const int wf = g.IM > g.pair_rows ? g.w_pair : g.w_one, wl = left > g.pair_rows ? g.w_pair : g.w_one;
        const int64_t full = (int64_t)wf * ri.kb + g.extra, per_head = full * (ri.tiles - 1) + (int64_t)wl * ri.kb + g.extra;
        const int64_t y = x - cum;
        h = (int)quotient(y, per_head);
        const int64_t z = y - h * per_head;
        t = (int)quotient(z, full);
        if (t > ri.tiles - 1) t = ri.tiles - 1;
        w = t < ri.tiles - 1 ? wf : wl;
        rows = t < ri.tiles - 1 ? g.IM : left;
        begin = cum + h * per_head + t * full;
        end = begin + (int64_t)w * ri.kb + g.extra;
    }
    static __device__ __forceinline__ int64_t units(const Geometry &g, int group, int H, const ReqInfo &ri) {
        if (ri.cnt == 0) return 0;
        const int left = ri.cnt * group - (ri.tiles - 1) * g.IM;
        return (int64_t)H * ri.kb *
                   ((ri.tiles - 1) * (g.IM > g.pair_rows ? g.w_pair : g.w_one) + (left > g.pair_rows ? g.w_pair : g.w_one)) +
               (int64_t)H * ri.tiles * g.extra;
    }
};

// The segment of range c (its units [x_beg, x_end)) at unit x; nb may be 0
// (the last unit of its block may lie in the next range).
__device__ __forceinline__ Seg segment_at(const Geometry &g, int group, int window, const ReqInfo &ri, int r, int64_t cum,
                                          int c, int64_t x, int64_t x_beg, int64_t x_end) {
    const ItemAt it(g, group, ri, cum, x);
    const int64_t end = x_end < it.end ? x_end : it.end;
    const int b0 = g.blocks(x - it.begin, it.w, ri.kb), b1 = g.blocks(end - it.begin, it.w, ri.kb);
    Seg s;
    s.start = ri.start, s.cnt = ri.cnt, s.ctx = ri.ctx, s.lo_max = ri.lo_max;
    s.r = r, s.h = it.h, s.t = it.t, s.rows = it.rows;
    s.nb = b1 - b0;
    s.key0 = ri.k0 + b0 * g.BN;
    s.key_lo = window > 0 && ri.ctx >= window ? ri.ctx - window + 1 : 0;
    s.slot = 2 * c + (it.begin >= x_beg ? 1 : 0);
    s.pair = it.rows > g.pair_rows;
    s.whole = s.nb == ri.kb;
    s.next = end;
    s.node0 = (ri.flags >> 1) - 1;
    return s;
}

// Walks the segments of a CTA's ranges blockIdx.x, blockIdx.x + gridDim.x, ...
struct SegWalk {
    int64_t cut_q;
    int cut_rem, cut_G, c, more;
    Seg sg;
    __device__ __forceinline__ int64_t at(int c_) const { return cut_q * c_ + (c_ < cut_rem ? c_ : cut_rem); }
    __device__ __forceinline__ void begin(const AttnArgs &a, const Geometry &g) {
        c = blockIdx.x;
        sg = a.ws.range[c];  // (the grid is no larger than the number of ranges)
        const int64_t total = a.ws.cum[a.R];
        const Cut cut(total, a.G, g.least());
        cut_q = cut.q;
        cut_rem = cut.rem;
        cut_G = total > 0 ? cut.G : 0;
        more = 2;  // the first one is there
    }
    // The next segment that has blocks into sg; false: there is none.
    __device__ bool step(const AttnArgs &a, const Geometry &g) {
        for (;;) {
            if (more == 2) {
                more = 1;
                if (c >= cut_G) return false;
            } else if (!more) {  // the next range: its first segment is ready
                c += gridDim.x;
                if (c >= cut_G) return false;
                sg = a.ws.range[c];
                more = 1;
            } else {
                const int64_t x = sg.next, x_end = at(c + 1);
                if (x >= x_end) {
                    more = 0;
                    continue;
                }
                int r = sg.r;
                while (a.ws.cum[r + 1] <= x) ++r;
                const ReqInfo ri = a.ws.req[r];
                sg = segment_at(g, a.group, a.window, ri, r, a.ws.cum[r], c, x, at(c), x_end);
            }
            if (sg.nb > 0) return true;
        }
    }
    // the same by the whole warp (the walk lies in shared memory)
    __device__ bool next(const AttnArgs &a, const Geometry &g) {
        __syncwarp();
        int ok = 0;
        if ((threadIdx.x & 31) == 0) ok = step(a, g);
        return __shfl_sync(kFull, ok, 0) != 0;
    }
};

// A page's index, whatever the table holds (the plan has already put requests
// with pages outside the cache in error; this keeps every access inside).
__device__ __forceinline__ int64_t page_of(const AttnArgs &a, int r, int key, int &tok) {
    const int p = a.page_shift >= 0 ? key >> a.page_shift : key / a.page;
    tok = key - p * a.page;
    const uint32_t g = (uint32_t)a.table[r * a.ld_table + p];
    return g < (uint64_t)a.pages ? (int64_t)g : a.pages - 1;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// softcap * tanh(x / softcap) * log2(e), with cap2 = 2 log2(e) / softcap and
// capl = softcap log2(e): tanh(u) = 1 - 2 / (1 + e^(2u)).  The absolute error
// is that of the reciprocal, below 1e-6 of the cap.
__device__ __forceinline__ float cap_score(float x, float cap2, float capl) {
    const float e = exp2_approx(x * cap2);
    return fmaf(-2.0f * capl, __fdividef(1.0f, 1.0f + e), capl);
}

// The kernel for many rows (w12_attn_tc.cu).
// The call's tensor maps (as bytes: the driver's types stay in that file);
// false where a layout has none, and the kernel for few rows does the work.
struct alignas(64) AttnTcMaps {
    unsigned char bytes[9 * 128];
};
bool attn_tc_maps(const AttnArgs &a, int D, AttnTcMaps *maps);
cudaError_t launch_attn_tc(const AttnArgs &a, const AttnTcMaps &maps, int D, int max_ctas, bool overlap, cudaStream_t s);

}  // namespace w12
