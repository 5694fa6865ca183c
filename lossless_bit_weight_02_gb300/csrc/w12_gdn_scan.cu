// The gated delta rule over sequences: outputs of every token and the states
// after the last (SpecPilot, arXiv 2611.02501, names the recurrent layers of
// hybrid targets, the news article's part (2); the published gated delta rule,
// as w12_gdn.cu has it for the nodes of draft trees).
//
// Per head, with the state S a D x D FP32 matrix (row = value index, column =
// key index), every token t of a sequence applies
//     S <- alpha_t S (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
// that is, with u = S k_t and f = beta_t (v_t - alpha_t u),
//     S <- alpha_t S + f k_t^T,      o_t = S q_t.
//
// Token by token (k_scan_path).  The rows of S do not touch one another, so a
// CTA takes some rows of a (request, head) and a thread 16 columns of one, two or
// four of them in registers: D/16 neighbouring lanes hold a row, a product with k
// or q is 16 multiply-adds and log2(D/16) shuffles.  Tokens come eight at a time
// through shared memory, the next eight while these are applied.  A state is read
// once and written once, whatever the number of tokens: for one token a request
// that is all the kernel does (64 requests, 32 heads of 128: 42.9 us, 6.3 TB/s;
// one request 3.4 us in a graph, 10 a call through the binding).  Up to 12 accepted nodes of 8 requests: 13.9 us (19.5 with every
// token's rows loaded a token ahead, two latencies each).
#include <cstdint>
#include <cuda_runtime.h>

#include "w12_device.cuh"
#include "w12_gdn_scan.cuh"
#include "w12_stream.cuh"

namespace w12 {
namespace {

constexpr int kPathThreads = 128;
constexpr int kAhead = 8;  // tokens of a load

template <int D, int ROWS>
struct PathTokens {
    __align__(16) uint16_t k[kAhead][D], q[kAhead][D], v[kAhead][ROWS];
    float al[kAhead], be[kAhead];
    int row[kAhead];
};
__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(void *to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

template <int D, int RPT>
struct PathSizes {
    static constexpr int L = D / 16;                     // lanes of a row
    static constexpr int ROWS = kPathThreads / L * RPT;  // of a CTA
    static constexpr int SPLIT = D / ROWS;
    static_assert(SPLIT >= 1 && ROWS * SPLIT == D, "whole CTAs a head");
    using Tokens = PathTokens<D, ROWS>[2];
};

// Rows part * ROWS .. of head rh's (r * H + h) state.
template <int D, int RPT>
__device__ __forceinline__ void path_of(const ScanArgs &a, int rh, int part, typename PathSizes<D, RPT>::Tokens &tokens) {
    constexpr int L = PathSizes<D, RPT>::L, ROWS = PathSizes<D, RPT>::ROWS;
    const int r = rh / a.H, h = rh - r * a.H;
    const int tid = threadIdx.x, lane = tid % L, row0 = part * ROWS + tid / L * RPT;
    const uint32_t group = ((1u << L) - 1u) << (tid % 32 / L * L);
    const int64_t at = ((int64_t)rh * D + row0) * D + 4 * lane;  // this thread's columns: 4 lane + 4 L m + 0 .. 3
    float S[RPT][16];
#pragma unroll
    for (int j = 0; j < RPT; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 x = *reinterpret_cast<const float4 *>(a.S + at + j * D + 4 * L * m);
            S[j][4 * m] = x.x, S[j][4 * m + 1] = x.y, S[j][4 * m + 2] = x.z, S[j][4 * m + 3] = x.w;
        }
    Seq seq = seq_of(a, r);
    if (seq.list) {
        const int ok = __syncthreads_and(list_ok(a, seq, tid, kPathThreads));
        if (!ok) seq.len = 0;
    }
    const int hk = h / a.per_key;
    // kAhead tokens at a time through shared memory, the next ones on their way
    auto load = [&](int t0, PathTokens<D, ROWS> &x) {
        const int m = min(kAhead, seq.len - t0);
        auto row_at = [&](int j) -> int64_t { return seq.list ? seq.list[t0 + j] : seq.first + t0 + j; };
        for (int i = tid; i < m * (D / 8); i += kPathThreads) {
            const int j = i / (D / 8), ch = i % (D / 8);
            const int64_t row = row_at(j);
            copy16(&x.k[j][8 * ch], a.k + row * a.ldk + hk * D + 8 * ch);
            if (a.q) copy16(&x.q[j][8 * ch], a.q + row * a.ldq + hk * D + 8 * ch);
        }
        for (int i = tid; i < m * (ROWS / 8); i += kPathThreads) {
            const int j = i / (ROWS / 8), ch = i % (ROWS / 8);
            copy16(&x.v[j][8 * ch], a.v + row_at(j) * a.ldv + h * D + part * ROWS + 8 * ch);
        }
        if (tid < m) {
            const int64_t row = row_at(tid);
            x.row[tid] = (int)row;
            copy4(&x.al[tid], a.alpha + row * a.H + h);
            copy4(&x.be[tid], a.beta + row * a.H + h);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto unpack = [](const uint16_t *p, float x[16]) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p + 4 * L * m);
            x[4 * m] = __uint_as_float(u.x << 16);
            x[4 * m + 1] = __uint_as_float(u.x & 0xFFFF0000u);
            x[4 * m + 2] = __uint_as_float(u.y << 16);
            x[4 * m + 3] = __uint_as_float(u.y & 0xFFFF0000u);
        }
    };
    // row j of S times x, the same on every lane of the row
    auto dots = [&](const float x[16], float y[RPT]) {
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            float p0 = 0.f, p1 = 0.f;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                p0 = fmaf(S[j][e], x[e], p0);
                p1 = fmaf(S[j][e + 1], x[e + 1], p1);
            }
            y[j] = p0 + p1;
        }
#pragma unroll
        for (int s = L / 2; s > 0; s >>= 1)
#pragma unroll
            for (int j = 0; j < RPT; ++j) y[j] += __shfl_xor_sync(group, y[j], s);
    };
    if (seq.len > 0) load(0, tokens[0]);
    for (int t0 = 0; t0 < seq.len; t0 += kAhead) {
        const PathTokens<D, ROWS> &now = tokens[t0 / kAhead & 1];
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        if (t0 + kAhead < seq.len) load(t0 + kAhead, tokens[(t0 / kAhead & 1) ^ 1]);
        const int m = min(kAhead, seq.len - t0);
        for (int t = 0; t < m; ++t) {
            const float al = now.al[t], be = now.be[t];
            float x[16], y[RPT];
            unpack(now.k[t] + 4 * lane, x);
            dots(x, y);
#pragma unroll
            for (int j = 0; j < RPT; ++j) {
                const float f = be * (bf2f(now.v[t][tid / L * RPT + j]) - al * y[j]);
#pragma unroll
                for (int e = 0; e < 16; ++e) S[j][e] = fmaf(f, x[e], al * S[j][e]);
            }
            if (a.q) {
                unpack(now.q[t] + 4 * lane, x);
                dots(x, y);
                float mine = y[0];  // lane j writes row j
#pragma unroll
                for (int j = 1; j < RPT; ++j) mine = lane == j ? y[j] : mine;
                if (lane < RPT) {
                    const int64_t to = (int64_t)now.row[t] * a.ldo + h * D + row0 + lane;
                    if (a.o32) static_cast<float *>(a.o)[to] = mine;
                    else static_cast<uint16_t *>(a.o)[to] = f32_to_bf16_rn(mine);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < RPT; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m)
            *reinterpret_cast<float4 *>(a.S_out + at + j * D + 4 * L * m) =
                make_float4(S[j][4 * m], S[j][4 * m + 1], S[j][4 * m + 2], S[j][4 * m + 3]);
}

template <int D, int RPT>
__global__ __launch_bounds__(kPathThreads) void k_scan_path(const __grid_constant__ ScanArgs a) {
    constexpr int SPLIT = PathSizes<D, RPT>::SPLIT;
    __shared__ typename PathSizes<D, RPT>::Tokens tokens;
    if (blockIdx.x == (int64_t)a.R * a.H * SPLIT) check_all(a);
    else path_of<D, RPT>(a, (int)(blockIdx.x / SPLIT), (int)(blockIdx.x % SPLIT), tokens);
}

// The heads that the chunked kernels have left: a.redo says how many, and which, in any order.
template <int D, int RPT>
__global__ __launch_bounds__(kPathThreads) void k_scan_redo(const __grid_constant__ ScanArgs a) {
    constexpr int SPLIT = PathSizes<D, RPT>::SPLIT;
    __shared__ typename PathSizes<D, RPT>::Tokens tokens;
    grid_dep_wait();
    const int64_t todo = (int64_t)a.redo[0] * SPLIT;
    for (int64_t u = blockIdx.x; u < todo; u += gridDim.x) {
        path_of<D, RPT>(a, a.redo[1 + u / SPLIT], (int)(u % SPLIT), tokens);
        __syncthreads();  // its tokens are no longer read
    }
}

template <int D>
cudaError_t launch_path(const ScanArgs &a, bool redo, cudaStream_t s) {
    constexpr int L = D / 16;
    const int64_t heads = (int64_t)a.R * a.H;
    auto grid = [&](int rpt) { return (unsigned)(heads * (D / (kPathThreads / L * rpt)) + (a.status ? 1 : 0)); };
    if (redo) {  // rarely any: no more CTAs than run at once, its start under the end of the chunks
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)min((int64_t)4 * W12_PLAN_SMS, heads * (D / (kPathThreads / L))));
        cfg.blockDim = dim3(kPathThreads);
        cfg.stream = s;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, k_scan_redo<D, 1>, a);
    }
    // Few states: a row a thread, for as many CTAs as there are multiprocessors and the shorter way of a token through a
    // thread; many: as many rows as registers hold, so that k and q are unpacked once for all of them.
    if (heads * D * L <= 2LL * W12_PLAN_SMS * kPathThreads * 2) k_scan_path<D, 1><<<grid(1), kPathThreads, 0, s>>>(a);
    else k_scan_path<D, D == 128 ? 4 : 2><<<grid(D == 128 ? 4 : 2), kPathThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Token by token or in chunks, by the average length: a chunk costs the same whatever is in it (us, by token / in
// chunks; 32 heads of 128, 64 requests of 23 tokens 183 / 176, of 36 267 / 178; one request of 32 14.7 / 21.6, of 48
// 20.3 / 21.6, of 64 26 / 22; 16 heads of 64, 64 requests of 36 52 / 65, of 64 81 / 66).  One choice for the whole call:
// where the lengths differ much neither serves all of it, and two calls do.
bool gdn_scan_chunks(int64_t n, int64_t R, int H, int D) { return n >= (D == 128 && R * H >= 128 ? 24 : 48) * R; }

size_t gdn_scan_workspace_bytes(int64_t n, int64_t R, int H, int, bool chunks) {
    return chunks ? scan_chunk_bytes(n, R, H) : 0;
}

cudaError_t launch_gdn_scan(const w12_gdn_scan_args &x, void *workspace, bool chunks, cudaStream_t s) {
    ScanArgs a{};
    a.S = x.S, a.S_out = x.S_out;
    a.q = x.q, a.k = x.k, a.v = x.v;
    a.ldq = x.ldq, a.ldk = x.ldk, a.ldv = x.ldv;
    a.alpha = x.alpha, a.beta = x.beta;
    a.o = x.o;
    a.ldo = x.ldo;
    a.o32 = x.o32;
    a.start = x.start, a.rows = x.rows, a.count = x.count;
    a.ld_rows = x.ld_rows;
    a.width = x.width;
    a.n = (int)x.n, a.R = (int)x.R, a.H = x.H, a.per_key = x.H / x.key_heads;
    a.status = x.status;
    if (chunks && x.n > 0) {
        const cudaError_t e = launch_scan_chunks(a, x, workspace, s);
        if (e == cudaSuccess) return x.D == 64 ? launch_path<64>(a, true, s) : launch_path<128>(a, true, s);
        if (e != cudaErrorNotSupported) return e;
    }
    return x.D == 64 ? launch_path<64>(a, false, s) : launch_path<128>(a, false, s);
}

}  // namespace w12
