// tma.cu -- host-side encoding of TMA tensor maps.  The driver entry point is
// fetched through the runtime (cudaGetDriverEntryPoint), so the library does
// not link libcuda directly.
#include <mutex>

#include "common.cuh"

namespace infllmv2 {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

}  // namespace

// bf16 tensor of rank 4, 128-byte swizzle, zero fill outside the tensor.
// dims: innermost first; strides_bytes: of dims 1..3; box: tile extent per dim.
int make_tmap_bf16_4d(CUtensorMap* map, const void* base, const uint64_t dims[4],
                      const uint64_t strides_bytes[3], const uint32_t box[4]) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return INFLLMV2_ERR_CUDA;
  const cuuint32_t elem_strides[4] = {1, 1, 1, 1};
  auto encode = [&] {
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
              strides_bytes, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    // The runtime binds a thread to its device's context with the thread's first
    // call that needs it, and this driver call may come before: bind it here.
    int d = 0;
    if (cudaGetDevice(&d) == cudaSuccess && cudaSetDevice(d) == cudaSuccess) r = encode();
  }
  return r == CUDA_SUCCESS ? INFLLMV2_OK : INFLLMV2_ERR_CUDA;
}

}  // namespace infllmv2
