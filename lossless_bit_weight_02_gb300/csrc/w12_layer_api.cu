// C-ABI layer of the operators between the GEMMs of a decoder layer: norm,
// rotary positions + cache write, tree attention.  Argument validation and
// launches, as w12_api.cu does it for the others.
#include <cstdint>

#include "w12.h"
#include "w12_device.cuh"
#include "w12_internal.h"

namespace {

using namespace w12;

bool at(const void *p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }

w12_status cuda_status(cudaError_t e) { return e == cudaSuccess ? W12_OK : W12_ERR_CUDA; }

w12_status check_cache(const w12_kv_cache *c) {
    if (!c || c->pages < 0 || c->page_tokens < 1 || c->heads < 1 || c->dim < 1) return W12_ERR_INVALID;
    if (c->pages > INT32_MAX || c->heads > 1024) return W12_ERR_INVALID;
    if (c->pages > 0 && (!c->k || !c->v)) return W12_ERR_INVALID;
    if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0) return W12_ERR_INVALID;
    if (!at(c->k, 16) || !at(c->v, 16) || c->page_stride % 8 || c->token_stride % 8 || c->head_stride % 8)
        return W12_ERR_ALIGN;
    return W12_OK;
}

}  // namespace

extern "C" {

w12_status w12_rmsnorm(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr, const uint16_t *weight,
                       float eps, int64_t M, int64_t K, uint16_t *h_out, int64_t ldh, uint16_t *y, int64_t ldy,
                       uint8_t *q8, int64_t ldq, float *scale, int64_t lds, w12_stream_t stream) {
    if (M < 0 || M > INT32_MAX || K < 1 || K > W12_NORM_MAX_K || !(eps >= 0.f)) return W12_ERR_INVALID;
    if ((q8 == nullptr) != (scale == nullptr)) return W12_ERR_INVALID;
    if (M == 0) return W12_OK;
    if (!x || !weight || ldx < K || (residual && ldr < K) || (h_out && ldh < K) || (y && ldy < K) ||
        (q8 && (ldq < K || lds < (K + 127) / 128)))
        return W12_ERR_INVALID;
    if (!at(x, 2) || !at(residual, 2) || !at(weight, 2) || !at(h_out, 2) || !at(y, 2) || !at(scale, 4))
        return W12_ERR_ALIGN;
    if (!h_out && !y && !q8) return W12_OK;
    return cuda_status(launch_rmsnorm(x, ldx, residual, ldr, weight, eps, M, K, h_out, ldh, y, ldy, q8, ldq, scale, lds,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

w12_status w12_rope_append(const w12_rope_args *a, w12_stream_t stream) {
    if (!a) return W12_ERR_INVALID;
    if (a->n < 0 || a->n > INT32_MAX || (a->dim != 64 && a->dim != 128 && a->dim != 256)) return W12_ERR_INVALID;
    if (a->rot < 0 || a->rot > a->dim || a->rot % 16 != 0 || (a->interleaved != 0 && a->interleaved != 1) ||
        !(a->eps >= 0.f))
        return W12_ERR_INVALID;
    if (a->q && (a->q_heads < 1 || a->q_heads > 4096)) return W12_ERR_INVALID;
    if ((a->k || a->slots) && (a->kv_heads < 1 || a->kv_heads > 1024)) return W12_ERR_INVALID;
    if (a->rot > 0) {
        if (a->n_axes < 1 || a->n_axes > W12_ROPE_MAX_AXES || !a->inv_freq) return W12_ERR_INVALID;
        if (a->axis)
            for (int j = 0; j < a->rot / 2; ++j)
                if (a->axis[j] >= a->n_axes) return W12_ERR_INVALID;
        if (a->n_axes > 1 && a->ld_pos < a->n) return W12_ERR_INVALID;
    }
    if (a->slots) {
        const w12_status st = check_cache(a->cache);
        if (st != W12_OK) return st;
        if (a->cache->heads != a->kv_heads || a->cache->dim != a->dim) return W12_ERR_INVALID;
    }
    if (a->n == 0) return W12_OK;
    if (a->rot > 0 && !a->pos) return W12_ERR_INVALID;
    if ((a->q == nullptr) != (a->q_out == nullptr) || (!a->k && a->k_out)) return W12_ERR_INVALID;
    if (a->slots ? (!a->k || !a->v) : (a->k && !a->k_out)) return W12_ERR_INVALID;
    if (!a->q && !a->k) return W12_ERR_INVALID;
    const int64_t wq = (int64_t)a->q_heads * a->dim, wk = (int64_t)a->kv_heads * a->dim;
    if ((a->q && (a->ldq < wq || a->ldqo < wq)) || (a->k && a->ldk < wk) || (a->k_out && a->ldko < wk) ||
        (a->slots && a->ldv < wk))
        return W12_ERR_INVALID;
    if (!at(a->q, 16) || !at(a->k, 16) || !at(a->q_out, 16) || !at(a->k_out, 16) || (a->slots && !at(a->v, 16)) ||
        !at(a->q_norm, 16) || !at(a->k_norm, 16) || !at(a->pos, 4) || !at(a->inv_freq, 4) || !at(a->slots, 8) ||
        (a->q && (a->ldq % 8 || a->ldqo % 8)) || (a->k && a->ldk % 8) || (a->k_out && a->ldko % 8) ||
        (a->slots && a->ldv % 8))
        return W12_ERR_ALIGN;
    return cuda_status(launch_rope(*a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t w12_tree_attn_workspace_bytes(int64_t n, int64_t R, int32_t q_heads, int32_t heads, int32_t dim) {
    if (n < 0 || n > W12_ATTN_MAX_NODES || R < 1 || R > W12_ATTN_MAX_REQUESTS || heads < 1 || heads > 1024 ||
        q_heads < 1 || q_heads > 4096 || q_heads % heads || (dim != 64 && dim != 128))
        return 0;
    return attn_workspace_bytes(n, R, q_heads, heads, dim);
}

w12_status w12_tree_attn(const w12_attn_args *a, const w12_kv_cache *cache, void *workspace, size_t ws_bytes,
                         w12_stream_t stream) {
    if (!a) return W12_ERR_INVALID;
    const w12_status st = check_cache(cache);
    if (st != W12_OK) return st;
    const size_t need = w12_tree_attn_workspace_bytes(a->n, a->R, a->q_heads, cache->heads, cache->dim);
    if (need == 0) return W12_ERR_INVALID;
    if (a->window < 0 || a->max_ctas < 0 || (a->flags & ~(W12_ATTN_REUSE_PLAN | W12_ATTN_TEST_STALL)) || a->width < 0 || !(a->scale >= 0.f) ||
        !(a->softcap >= 0.f && a->softcap <= W12_ATTN_MAX_SOFTCAP) || a->ld_table < a->width || (int64_t)a->width * cache->page_tokens > INT32_MAX - 512)
        return W12_ERR_INVALID;
    if (!workspace || ws_bytes < need) return W12_ERR_CAPACITY;
    if (!at(workspace, 256)) return W12_ERR_ALIGN;
    if (a->n == 0) return W12_OK;
    const int64_t wq = (int64_t)a->q_heads * cache->dim, wk = (int64_t)cache->heads * cache->dim;
    if (!a->q || !a->k || !a->v || !a->o || !a->ctx_len || (a->width > 0 && !a->block_table) || a->ldq < wq ||
        a->ldo < wq || a->ldk < wk || a->ldv < wk)
        return W12_ERR_INVALID;
    if (!at(a->q, 16) || !at(a->k, 16) || !at(a->v, 16) || !at(a->o, 16) || a->ldq % 8 || a->ldk % 8 || a->ldv % 8 ||
        a->ldo % 8 || !at(a->block_table, 4) || !at(a->ctx_len, 4) || !at(a->parent, 4) || !at(a->req, 4))
        return W12_ERR_ALIGN;
    return cuda_status(launch_tree_attn(*a, *cache, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

w12_status w12_tree_attn_status(void *workspace, size_t ws_bytes, w12_stream_t stream) {
    if (!workspace || ws_bytes < 256) return W12_ERR_INVALID;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int32_t w[3] = {0, 0, 0};  // tree error, ticket, timeout
    if (cudaMemcpyAsync(w, workspace, sizeof w, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return W12_ERR_CUDA;
    if (w[2] != 0) {
        if (cudaMemsetAsync(static_cast<char *>(workspace) + 8, 0, 4, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess)
            return W12_ERR_CUDA;
        return W12_ERR_TIMEOUT;
    }
    return w[0] == 0 ? W12_OK : W12_ERR_INVALID;
}

}  // extern "C"
