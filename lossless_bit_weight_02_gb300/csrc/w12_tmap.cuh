// Tensor maps of BF16 tensors for TMA copies with the 128-byte swizzle.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

namespace w12 {

// The driver's tensor-map encoder, looked up once.
inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
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

// A tensor of BF16 with `rank` dimensions, the first contiguous; a stride
// (elements) of a dimension of one is not used and any value will do.
inline bool encode_tmap(CUtensorMap *map, const uint16_t *p, int rank, const int64_t *dim, const int64_t *stride, const int *box) {
    const auto enc = tmap_encoder();
    if (!enc || !p) return false;
    cuuint64_t d[4], st[3];
    cuuint32_t b[4], es[4];
    for (int i = 0; i < rank; ++i) {
        if (dim[i] < 1 || dim[i] > (1LL << 32)) return false;
        d[i] = (cuuint64_t)dim[i];
        b[i] = (cuuint32_t)box[i];
        es[i] = 1;
        if (i > 0) {
            const int64_t s = dim[i] == 1 ? 8 * ((dim[0] + 7) / 8) : stride[i - 1];
            if (s <= 0 || s * 2 >= (1LL << 40)) return false;
            st[i - 1] = (cuuint64_t)s * 2;
        }
    }
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<uint16_t *>(p), d, st, b, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace w12
