// tensor_map.cuh -- host side of the tiled copies: tensor maps and the device's size.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

namespace ep {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library links no driver library).
inline EncodeTiled encoder() {
    static std::atomic<EncodeTiled> found{nullptr};
    EncodeTiled e = found.load(std::memory_order_acquire);
    if (e) return e;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    e = reinterpret_cast<EncodeTiled>(fn);
    found.store(e, std::memory_order_release);
    return e;
}

// A tensor of `rank` dimensions (innermost first, strides in elements of dimensions 1..) of
// `size` bytes an element, read in boxes with zeros outside.
inline bool make_map(CUtensorMap *m, CUtensorMapDataType type, int size, const void *base, int rank, const uint64_t *dims,
                     const uint64_t *strides, const uint32_t *box, CUtensorMapSwizzle swizzle) {
    EncodeTiled enc = encoder();
    if (!enc) return false;
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        one[i] = 1;
        if (i > 0) s[i - 1] = strides[i - 1] * size;
    }
    return enc(m, type, (cuuint32_t)rank, const_cast<void *>(base), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16, with the 128-byte swizzle.
inline bool make_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                     const uint32_t *box) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, rank, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// [groups][rows][cols] read in boxes of 64 columns and box_rows rows.
inline bool make_map3(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint64_t groups, uint32_t box_rows) {
    const uint64_t dims[3] = {cols, rows, groups}, strides[2] = {cols, cols * rows};
    const uint32_t box[3] = {64, box_rows, 1};
    return make_map(m, base, 3, dims, strides, box);
}

// The multiprocessor count of the current device.
inline cudaError_t sm_count(int *out) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && (*out = cached[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < kMaxDevices) cached[dev].store(*out, std::memory_order_relaxed);
    return e;
}

}  // namespace ep
