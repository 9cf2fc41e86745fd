// paged_shared_bf16_64.cu -- attention behind shared rows (paged_shared.cuh) of bf16 heads
// of 64: a file a type and head size, compiled side by side.
#include "paged_shared.cuh"

namespace exattn {

cudaError_t launch_paged_shared_bf16_64(const PagedLines& a, cudaStream_t stream) {
  return launch_paged_lines<__nv_bfloat16, 64>(a, stream);
}

}  // namespace exattn
