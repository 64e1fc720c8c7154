// tensor_map.h: tensor maps of [rows, heads, head dim] arrays of 16-bit or 8-bit elements for the kernels' TMA copies.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "pa_internal.h"

namespace pa {

static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> cached{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = cached.load(std::memory_order_relaxed);
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            cached.store(fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr), std::memory_order_relaxed);
    }
    return fn;
}

// The map of a contiguous [rows, heads, hd] array of elements of `bytes` bytes with boxes of box_rows x box_heads x box_cols.
static bool encode_elements_3d(CUtensorMap *m, const void *base, CUtensorMapDataType type, int bytes, int heads, int hd,
                               long long rows, int box_heads, int box_rows, int box_cols, CUtensorMapSwizzle swizzle,
                               CUtensorMapL2promotion fill) {
    const auto fn = tensor_map_encoder();
    if (!fn || rows <= 0) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hd) * bytes, static_cast<cuuint64_t>(heads) * hd * bytes};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_heads),
                               static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[3] = {1, 1, 1};
    const auto make = [&] {
        return fn(m, type, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, fill,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (make()) return true;
    // A thread that has made no call of the runtime yet has no context, which this driver call needs; setting
    // the device that is current binds one.
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && make();
}

// of 16-bit elements
[[maybe_unused]] static bool encode_rows_3d(CUtensorMap *m, const void *base, pa_dtype dt, int heads, int hd, long long rows,
                                            int box_heads, int box_rows, int box_cols, CUtensorMapSwizzle swizzle,
                                            CUtensorMapL2promotion fill) {
    return encode_elements_3d(m, base, dt == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                              heads, hd, rows, box_heads, box_rows, box_cols, swizzle, fill);
}

// of e4m3 elements, whole rows of 64 or 128 bytes of one head, one after the other or swizzled over as many bytes
[[maybe_unused]] static bool encode_rows_e4m3(CUtensorMap *m, const void *base, int heads, int hd, long long rows, int box_rows,
                                              bool swizzled) {
    return encode_elements_3d(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, heads, hd, rows, 1, box_rows, hd,
                              !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
}

}  // namespace pa
