// kd_tmap.cu -- TMA descriptor encoding through the driver entry point (no
// link-time dependency on libcuda).
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kd_tmap.h"

namespace kd {

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

bool make_tmap_bthd(CUtensorMap* m, const void* base, int es, int B, int T, int H, int D, int box_d,
                    bool swizzle128, int box_t) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t e = static_cast<cuuint64_t>(es);
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T),
                        static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {D * e, static_cast<cuuint64_t>(H) * D * e,
                           static_cast<cuuint64_t>(T) * H * D * e};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(box_d), 1u, static_cast<cuuint32_t>(box_t), 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  const auto encode = [&] {
    return fn(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r != CUDA_SUCCESS) {
    // a thread that has made no runtime call yet (an autograd worker) has no
    // current context, which the driver call wants: bind the device's own
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encode();
  }
  return r == CUDA_SUCCESS;
}

}  // namespace kd
