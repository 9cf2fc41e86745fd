// paged_shared.cuh -- attention over a paged cache behind rows that several sequences
// share, for sm_103a.
//
// The rows that a group of sequences has on the same pages are seen by all its new
// tokens, so these attend to them as one sequence's: one line of units (paged_sched.cuh)
// goes over the groups' shared rows, a second one over each sequence's own rows, and the
// softmax's parts add up by their masses (paged_join.cu).  K and V of the shared rows are
// read once a group and 256 query rows, where attn_fwd_paged reads them once a sequence.
//
// Both lines run in one launch: a CTA reads the tables, weighs both, and takes its place
// in one of them, as many CTAs a line as its share of the time.  (As two launches, the
// second one's CTAs had to wait for those of the first that had nothing to do: they began
// 7 us in, and its last ones ended 4 us after its work.)  The lines' kernels are those of
// attn_fwd_paged: groups of more than 32 query rows take the forward kernel
// (paged_fwd.cuh), smaller ones the decode kernel with 8, 16 or 32 columns; own rows the one
// that their count of new tokens asks for.  What does not depend on the line is done
// before the CTA knows it, beside the stream's last kernel: both lines' barriers, TMEM.
//
// 71 chats behind four prompts of up to 16,384 rows, 32 heads on 4 of 128, 87 us where
// attn_fwd_paged takes 231 (429 MB of keys and values: 62 at the copy's rate): the own
// rows' CTAs stream some 46 GB/s each, 192 KB in flight, whatever the others do, so the
// SMs on the shared rows, bound by their products, are bandwidth lost.  16 samples behind
// 8,192 rows, 32 heads on 8, 28 us (48): tables and place 2, the first tile 5, a CTA's six tiles
// of 1.9 (a query tile alone is a chain of product, softmax, product), its end 2, stragglers
// 3, the join and its launch 6.  Two behind 512 rows 12 us (9): not worth sharing.  Chunks of
// prompts, bound by products either way, gain nothing: six of 264 tokens behind 16,384 rows 346 us
// (350).
#pragma once
#include "paged_decode.cuh"
#include "paged_fwd.cuh"

namespace exattn {

// A line's CTAs: the forward kernel's (NC = 0) or the decode kernel's.
template <typename T, int D, int NC>
struct LineKernel {
  using C = PdCfg<D, NC>;
  using Bars = PdBars<C::K_STAGES, C::V_STAGES>;
  static constexpr int SMEM = C::SMEM_BYTES - 1024;  // the barriers lie elsewhere
  __device__ __forceinline__ static void init(Bars* bars) { paged_decode_init<Bars, C::K_STAGES, C::V_STAGES>(bars); }
  __device__ __forceinline__ static void clear(uint8_t* smem) { paged_decode_clear<C>(smem); }
  __device__ __forceinline__ static void run(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedArgs& a,
                                             int cta, const PagedCursor<true>& cur, const PagedSeq& seq, uint8_t* smem, Bars* bars) {
    paged_decode_run<T, D, NC, true>(q, k, v, a, cta, cur, seq, smem, bars);
  }
};
template <typename T, int D>
struct LineKernel<T, D, 0> {
  using C = PfCfg<D>;
  using Bars = PfBars<C::STAGES>;
  static constexpr int SMEM = C::SMEM_BYTES - 1024;
  __device__ __forceinline__ static void init(Bars* bars) { paged_fwd_init<Bars, C::STAGES, C::ISSUERS>(bars); }
  __device__ __forceinline__ static void clear(uint8_t*) {}
  __device__ __forceinline__ static void run(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedArgs& a,
                                             int cta, const PagedCursor<true>& cur, const PagedSeq& seq, uint8_t* smem, Bars* bars) {
    paged_fwd_run<T, D, true>(q, k, v, a, cta, cur, seq, smem, bars);
  }
};

template <typename T, int D, int NS, int NO>
__global__ void __launch_bounds__(512, 1)
    paged_shared_kernel(const __grid_constant__ CUtensorMap tm_qs, const __grid_constant__ CUtensorMap tm_qo,
                        const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedLines p) {
  using KS = LineKernel<T, D, NS>;
  using KO = LineKernel<T, D, NO>;
  // The role of this CTA is not known yet: both lines' barriers, and all of TMEM.
  __shared__ typename KS::Bars bars_s;
  __shared__ typename KO::Bars bars_o;
  __shared__ int weight_s[2];
  __shared__ PagedCursor<true> cur_s;
  __shared__ PagedSeq seq_s;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = static_cast<int>(blockIdx.x);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 32 * 2) {
    KS::init(&bars_s);
    if (NS != NO) KO::init(&bars_o);
    fence_barrier_init();
  }
  if (warp == 3) {
    tmem_alloc(&bars_s.tmem_base, 512);
    tmem_relinquish();
  }
  KS::clear(smem);
  if (NS != NO) KO::clear(smem);
  // Up to here this CTA may run beside the stream's last kernel.
  if (warp < 2) paged_touch(p.line[warp]);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  PagedLine<true> line{};
  if (warp < 2) {
    line = paged_line<true>(p.line[warp], p.line[warp].share.unit_tokens[warp], lane);
    if (lane == 0) weight_s[warp] = line.W;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars_s.tmem_base;
  if (NS != NO && threadIdx.x == 0) bars_o.tmem_base = tmem;
  const PagedShare& s = p.line[0].share;
  const int first = shared_ctas(s, weight_s[0], weight_s[1]), own = min(s.sms - first, s.ctas[1]);
  const int role = cta < first ? 0 : 1, at = role ? cta - first : cta;
  if (cta < first + own) {
    if (warp == role) {
      PagedSeq seq;
      const PagedCursor<true> cur =
          paged_place<true>(p.line[role], p.line[role].share.unit_tokens[role], lane, at, role ? own : first, line, &seq);
      if (lane == 0) {
        cur_s = cur;
        seq_s = seq;
      }
    }
    __syncthreads();
    if constexpr (NS == NO) {  // one copy of the code
      KS::run(role ? tm_qo : tm_qs, tm_k, tm_v, p.line[role], at, cur_s, seq_s, smem, &bars_s);
    } else {
      if (role == 0) KS::run(tm_qs, tm_k, tm_v, p.line[0], at, cur_s, seq_s, smem, &bars_s);
      else KO::run(tm_qo, tm_k, tm_v, p.line[1], at, cur_s, seq_s, smem, &bars_o);
    }
  }
  if (warp == 3) tmem_dealloc(tmem, 512);
}

template <typename T, int D, int NS, int NO>
cudaError_t launch_lines(const PagedLines& a, cudaStream_t stream) {
  constexpr int smem = std::max(LineKernel<T, D, NS>::SMEM, LineKernel<T, D, NO>::SMEM);
  auto kern = paged_shared_kernel<T, D, NS, NO>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem, a.line[0].device);
  if (e != cudaSuccess) return e;
  return launch_dependent("paged shared kernel launch", kern, a.line[0].share.sms, 512, smem, stream, *a.line[0].tm_q,
                          *a.line[1].tm_q, *a.line[0].tm_k, *a.line[0].tm_v, a);
}

template <typename T, int D, int NS>
cudaError_t launch_own(const PagedLines& a, cudaStream_t stream) {
  switch (a.line[1].cols) {
    case 4: return launch_lines<T, D, NS, 4>(a, stream);
    case 8: return launch_lines<T, D, NS, 8>(a, stream);
    case 16: return launch_lines<T, D, NS, 16>(a, stream);
    case 32: return launch_lines<T, D, NS, 32>(a, stream);
    default: return note_cuda(cudaErrorInvalidValue, "paged shared kernel (columns)");
  }
}

template <typename T, int D>
cudaError_t launch_paged_lines(const PagedLines& a, cudaStream_t stream) {
  if (a.line[0].cols == 8)
    return a.line[1].cols == 4 ? launch_lines<T, D, 8, 4>(a, stream) : launch_lines<T, D, 8, 8>(a, stream);
  if (a.line[0].cols == 16)
    return a.line[1].cols == 4   ? launch_lines<T, D, 16, 4>(a, stream)
           : a.line[1].cols == 8 ? launch_lines<T, D, 16, 8>(a, stream)
                                 : launch_lines<T, D, 16, 16>(a, stream);
  if (a.line[0].cols) return launch_own<T, D, 32>(a, stream);
  return a.line[1].cols ? launch_own<T, D, 0>(a, stream) : launch_lines<T, D, 0, 0>(a, stream);
}

}  // namespace exattn
