// paged_shared_f16_64.cu -- attention behind shared rows (paged_shared.cuh) of f16 heads
// of 64: a file a type and head size, compiled side by side.
#include "paged_shared.cuh"

namespace exattn {

cudaError_t launch_paged_shared_f16_64(const PagedLines& a, cudaStream_t stream) {
  return launch_paged_lines<__half, 64>(a, stream);
}

}  // namespace exattn
