// dense.cu -- tensor maps of the dense products (dense.cuh).
#include <cudaTypedefs.h>

#include <mutex>

#include "dense.cuh"
#include "entry.h"

namespace moe {
namespace dense {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}
}  // namespace

int32_t make_map(CUtensorMap* m, const void* base, Elem type, int64_t rows, int64_t cols, int64_t ld,
                 int box_cols, int box_rows, Swizzle swizzle) {
  auto fn = encoder();
  if (!fn) return entry_fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
  const int64_t bytes = type == Elem::kF32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m,
                        type == Elem::kBf16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                        : type == Elem::kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                        2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swizzle == Swizzle::k128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return entry_fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) rows=%lld cols=%lld ld=%lld",
                      static_cast<int>(r), static_cast<long long>(rows), static_cast<long long>(cols),
                      static_cast<long long>(ld));
  return MOE_OK;
}

}  // namespace dense
}  // namespace moe
