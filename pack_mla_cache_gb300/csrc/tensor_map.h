// tensor_map.h -- the driver's tensor map encoder, found through the runtime (the library
// links no driver stub).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace mla {

using TensorMapEncode = decltype(&cuTensorMapEncodeTiled);

// Null where the driver has none.
inline TensorMapEncode tensor_map_encode() {
  static const TensorMapEncode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    (void)cudaGetLastError();
    return reinterpret_cast<TensorMapEncode>(f);
  }();
  return encode;
}

}  // namespace mla
