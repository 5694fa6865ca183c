// What the kernels of w12_gdn_scan share.
#pragma once

#include <cstdint>

#include "w12_device.cuh"
#include "w12_internal.h"

namespace w12 {

struct ScanArgs {
    const float *S;
    float *S_out;
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float *alpha, *beta;
    void *o;
    int64_t ldo;
    int o32;
    const int32_t *start, *rows, *count;
    int64_t ld_rows;
    int width;
    int n, R, H, per_key;  // per_key: value heads of a key head
    int32_t *status;  // or null
    // in chunks
    int32_t *err;      // where a wait that gave up leaves a mark: status, or a word of the workspace that nobody reads
                       // (the head's outputs and state are NaN then)
    uint8_t *image;    // what k_scan_prep makes for k_scan_main: kImageBytes a chunk and head
    float *gamma;      // [chunks][H][64]
    uint8_t *cond;     // [chunks][H][2]: whether half a chunk's inverses are too large for the chunks' arithmetic
    int32_t *redo;     // [1 + R * H]: how many heads (r * H + h) have such chunks, and which; k_scan_path computes them
    int stall;         // tests only
};

// The tokens of request r: `len` of them, the t-th in row first + t, or list[t].
struct Seq {
    int first, len;
    const int32_t *list;
    bool ok;
};
__device__ __forceinline__ Seq seq_of(const ScanArgs &a, int r) {
    Seq s;
    if (!a.count) {
        const int b = a.start ? a.start[r] : 0, e = a.start ? a.start[r + 1] : a.n;
        s.ok = b >= 0 && b <= e && e <= a.n;
        s.first = b;
        s.len = s.ok ? e - b : 0;
        s.list = nullptr;
    } else {
        const int c = a.count[r];
        s.ok = c >= 0 && c <= a.width;
        s.first = 0;
        s.len = s.ok ? c : 0;
        s.list = a.rows + (int64_t)r * a.ld_rows;
    }
    return s;
}
__device__ __forceinline__ bool list_ok(const ScanArgs &a, const Seq &s, int from, int step) {
    bool ok = true;
    if (s.list)
        for (int t = from; t < s.len; t += step) ok &= s.list[t] >= 0 && s.list[t] < a.n;
    return ok;
}

// Whether any sequence breaks a rule: written by one CTA of a call, so that the word needs no clearing.
__device__ __forceinline__ void check_all(const ScanArgs &a) {
    bool bad = false;
    for (int r = threadIdx.x; r < a.R; r += blockDim.x) {
        const Seq s = seq_of(a, r);
        bad |= !s.ok || !list_ok(a, s, 0, 1);
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.status = any ? 1 : 0;
}

__device__ __forceinline__ float bf2f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// In chunks (w12_gdn_chunk.cu).
size_t scan_chunk_bytes(int64_t n, int64_t R, int H);
// cudaErrorNotSupported: the rows do not fit a tensor map (nothing was launched).
// Sets a.redo: the heads there are left to k_scan_redo.
cudaError_t launch_scan_chunks(ScanArgs &a, const w12_gdn_scan_args &x, void *workspace, cudaStream_t s);

}  // namespace w12
