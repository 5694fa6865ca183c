// What the kernels of the tree attention share: the workspace, the cut of the
// work, and who sees what.
//
// Keys of request r are numbered 0 .. ctx + cnt: its ctx cached tokens, then
// its cnt tree nodes in the order of the call ("rank").  They are walked in
// blocks of BN keys from k0, the first key that any of its nodes sees rounded
// down to a block.  Query rows of a key/value head are (rank, head of the
// group), rank first; an item is IM rows of one (request, head), with kb
// blocks to walk.  All blocks of all items form one line, in the order
// (request, head, row tile, block), that is cut into G ranges of equal length
// whatever the requests' lengths; a range is one CTA's work.  An item inside
// one range is finished there; of an item that several ranges share each
// leaves a partial (running maximum, sum and FP32 output of its blocks), and
// a last kernel joins them in the order of the ranges.  The cut depends on the
// inputs alone, so the grid never changes a result.
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
constexpr float kLog2e = 1.4426950408889634f;

struct alignas(16) ReqInfo {
    int32_t start;  // its nodes: order[start .. start + cnt)
    int32_t cnt;    // nodes (0 if the request is in error)
    int32_t ctx;    // cached tokens
    int32_t k0;     // first key walked, a multiple of BN
    int32_t kb;     // blocks per item
    int32_t tiles;  // items per head
    int32_t lo_max; // from this key on every node sees every cached token
    int32_t bad;    // a node of the request, or the request, is in error
};

// A range: the request in which it begins, and the join it stands for: if it
// begins inside an item that the range before it begins, that item (h, t) is
// joined from ranges c - 1 .. last; else last is -1.
struct alignas(16) RangeInfo {
    int32_t r, h, t, last;
};

// Workspace: [0, 256) error word, ticket, timeout word | ReqInfo [R] | cum
// [R + 1] | RangeInfo [G] | order, pos, depth [n] | masks [n][8] | (max, sum)
// of the partials | partials.  A partial lies as [D / 4][IM][4], so that
// threads of neighbouring rows read and write neighbouring addresses.
struct AttnWs {
    int32_t *err, *ticket, *timeout;
    ReqInfo *req;
    int64_t *cum;      // blocks before request r
    RangeInfo *range;
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
};

// Range c holds the blocks [begin(c), begin(c + 1)).
struct Cut {
    int64_t q;
    int rem;
    __device__ __forceinline__ Cut(int64_t total, int G) {
        q = total / G;
        rem = (int)(total - q * G);
    }
    __device__ __forceinline__ int64_t begin(int c) const { return q * c + (c < rem ? c : rem); }
    __device__ __forceinline__ int of(int64_t x) const {  // the range of block x
        return x < (q + 1) * rem ? (int)(x / (q + 1)) : rem + (int)((x - (q + 1) * rem) / q);
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
cudaError_t launch_attn_tc(const AttnArgs &a, int D, int max_ctas, bool overlap, cudaStream_t s);

}  // namespace w12
