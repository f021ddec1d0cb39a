// tma_host.h -- host-side construction of TMA tensor maps (2D, 128-byte
// swizzle), through the driver entry point obtained from the runtime.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace csa {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};   // by any thread
    PFN_cuTensorMapEncodeTiled_v12000 fn = known;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            known = fn = (PFN_cuTensorMapEncodeTiled_v12000)p;
    }
    return fn;
}

// Encodes a 2D map. The encoder refuses a thread without a current context,
// which one has whose first CUDA call this is (queries give it none): such a
// thread is given its device's before a second try.
inline bool encode_tmap(CUtensorMap *m, CUtensorMapDataType dt, const void *base,
                        const cuuint64_t (&dims)[2], const cuuint64_t (&strides)[1],
                        const cuuint32_t (&box)[2], CUtensorMapSwizzle swizzle)
{
    const auto enc = tensor_map_encoder();
    if (!enc)
        return false;
    const cuuint32_t estr[2] = {1, 1};
    for (int tries = 0; tries < 2; tries++) {
        int dev = 0;
        if (tries && (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess))
            return false;
        if (enc(m, dt, 2, const_cast<void *>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
            return true;
    }
    return false;
}

// Row-major [rows, cols] matrix of `esize`-byte elements, read in boxes of
// box_rows x (128 / esize) elements with the 128-byte swizzle; out-of-range
// rows read as zero. Rows lie `row_bytes` apart (0: cols * esize, packed).
// Returns false when the map cannot be encoded.
inline bool make_tmap_2d(CUtensorMap *m, const void *base, CUtensorMapDataType dt, int esize,
                         uint64_t rows, uint64_t cols, uint32_t box_rows, uint64_t row_bytes = 0)
{
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(row_bytes ? row_bytes : cols * esize)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / esize), (cuuint32_t)box_rows};
    return encode_tmap(m, dt, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Row-major [rows, row_bytes] bytes (rows `stride` bytes apart) read in
// unswizzled boxes of box_rows x box_bytes; out-of-range rows read as zero.
inline bool make_tmap_bytes(CUtensorMap *m, const void *base, uint64_t rows, uint64_t row_bytes,
                            uint64_t stride, uint32_t box_rows, uint32_t box_bytes)
{
    const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {box_bytes, box_rows};
    return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace csa
