// paged_decode.cu -- the launches of paged_decode.cuh's kernel.
#include "paged_decode.cuh"

namespace exattn {

namespace {

template <typename T, int D, int NC>
__global__ void __launch_bounds__(PdCfg<D, NC>::THREADS, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedArgs a) {
  using C = PdCfg<D, NC>;
  using Bars = PdBars<C::K_STAGES, C::V_STAGES>;
  static_assert(sizeof(Bars) <= 1024, "barrier block too large");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PagedCursor<false> cur{};
  PagedSeq seq{};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 32) {
    paged_decode_init<Bars, C::K_STAGES, C::V_STAGES>(bars);
    fence_barrier_init();
  }
  if (warp == C::S_WARP) {
    tmem_alloc(&bars->tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  if (warp == C::V_WARP && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  paged_decode_clear<C>(smem);
  // Up to here this CTA may run beside the stream's last kernel.  The walking warp
  // finds its place in the line.
  if (warp == C::K_WARP) paged_touch(a);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == C::K_WARP) cur = paged_start(a, a.tile_tokens, lane, &seq);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  paged_decode_run<T, D, NC, false>(tm_q, tm_k, tm_v, a, static_cast<int>(blockIdx.x), cur, seq, smem, bars);
  if (warp == C::S_WARP) tmem_dealloc(bars->tmem_base, C::TM_COLS);
}

template <typename T, int D, int NC>
cudaError_t launch_n(const PagedArgs& a, cudaStream_t stream) {
  using C = PdCfg<D, NC>;
  auto kern = paged_decode_kernel<T, D, NC>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, a.device);
  if (e != cudaSuccess) return e;
  return launch_dependent("paged decode kernel launch", kern, a.ctas, C::THREADS, C::SMEM_BYTES, stream, *a.tm_q, *a.tm_k,
                          *a.tm_v, a);
}

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t stream) {
  switch (a.cols) {
    case 4: return launch_n<T, D, 4>(a, stream);
    case 8: return launch_n<T, D, 8>(a, stream);
    case 16: return launch_n<T, D, 16>(a, stream);
    case 32: return launch_n<T, D, 32>(a, stream);
    default: return note_cuda(cudaErrorInvalidValue, "paged decode kernel (columns)");
  }
}

}  // namespace

cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t stream) {
  if (a.dtype == kF16) return a.d == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_t<__nv_bfloat16, 64>(a, stream) : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
