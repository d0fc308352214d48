// tq_tmap.cu -- tensor-map encoding through the driver entry point (resolved
// once through the runtime, so libtq needs no link-time libcuda dependency).
#include <mutex>

#include "tq_tmap.h"

namespace tq {

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn(cudaError_t *err) {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    static cudaError_t status = cudaSuccess;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        status = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                  cudaEnableDefault, &q);
        if (status == cudaSuccess && (q != cudaDriverEntryPointSuccess || p == nullptr))
            status = cudaErrorSymbolNotFound;
        fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    *err = status;
    return fn;
}

// Encode.  A thread that has made no CUDA call of its own has no context yet, and the driver's
// encoder wants one: the current device's is then made current, and the encoder asked again.
cudaError_t encode(CUtensorMap *out, CUtensorMapDataType dtype, uint32_t rank, const void *base, const cuuint64_t *dims,
                   const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle) {
    cudaError_t e = cudaSuccess;
    EncodeTiledFn fn = encode_fn(&e);
    if (e != cudaSuccess) return e;
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    const auto ask = [&] {
        return fn(out, dtype, rank, const_cast<void *>(base), dims, strides, box, elem_strides,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = ask();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess || (e = cudaSetDevice(dev)) != cudaSuccess) return e;
        r = ask();
    }
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t make_tmap_2d(CUtensorMap *out, CUtensorMapDataType dtype, const void *base,
                         uint64_t inner, uint64_t rows, uint64_t row_stride_bytes,
                         uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_stride_bytes)};
    const cuuint32_t box[2] = {box_inner, box_rows};
    return encode(out, dtype, 2, base, dims, strides, box, swizzle);
}

cudaError_t make_codes_tmap_3d(CUtensorMap *out, const void *base, uint64_t row_bytes, uint64_t rows) {
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(row_bytes / 128), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {128, static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[3] = {128, 2, 16};
    return encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace tq
