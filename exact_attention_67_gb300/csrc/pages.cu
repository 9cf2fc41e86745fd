// pages.cu -- copies whole pages of a paged key/value cache, for sm_103a:
// page dst[i] of every slab (a layer's K or V) becomes a copy of page src[i].
//
// The page numbers come from the host, where page tables are kept, and travel
// in the kernel's parameters: no copy to the device and no workspace, and a
// captured graph holds its own list.  The C ABI has checked that no
// destination occurs twice or is a source, so the copies are independent.
//
// Bound by HBM: a block copies 16 KB, all of its loads before its stores, past the
// caches' reuse.  1,500 pages of 32 KB in 32 slabs 458 us (6.9 TB/s), 7 pages in 64
// slabs 5.2 us (5.7 TB/s).  A smaller page leaves threads idle: 1,000 pages of 8, 4
// and 2 KB in 64 slabs 7.0, 6.4 and 4.0 TB/s.
#include "paged.cuh"

namespace exattn {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kPiece = kThreads * kUnroll * 16;  // bytes a block: one piece of one page

template <int N>
struct Pairs {
  int src[N], dst[N];
};

template <int N>
__global__ void __launch_bounds__(kThreads) page_copy_kernel(const __grid_constant__ Pairs<N> p, char* pool,
                                                             long long slab_stride, long long page_stride,
                                                             long long page_bytes, int pieces) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int pair = static_cast<int>(blockIdx.x) / pieces, piece = static_cast<int>(blockIdx.x) % pieces;
  char* slab = pool + blockIdx.y * slab_stride;
  const char* src = slab + p.src[pair] * page_stride;
  char* dst = slab + p.dst[pair] * page_stride;
  const long long o0 = static_cast<long long>(piece) * kPiece + threadIdx.x * 16;
  uint4 x[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long o = o0 + u * (kThreads * 16);
    if (o < page_bytes) x[u] = __ldcs(reinterpret_cast<const uint4*>(src + o));
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long o = o0 + u * (kThreads * 16);
    if (o < page_bytes) __stcs(reinterpret_cast<uint4*>(dst + o), x[u]);
  }
}

template <int N>
cudaError_t launch_n(const CopyArgs& a, int at, int n, cudaStream_t stream) {
  Pairs<N> p;
  for (int i = 0; i < N; ++i) {
    p.src[i] = i < n ? a.src[at + i] : 0;
    p.dst[i] = i < n ? a.dst[at + i] : 0;
  }
  const int pieces = static_cast<int>((a.page_bytes + kPiece - 1) / kPiece);
  const dim3 grid(static_cast<unsigned>(n) * pieces, a.slabs);
  return launch_dependent("page copy kernel launch", page_copy_kernel<N>, grid, kThreads, 0, stream, p, a.pool,
                          a.slab_stride, a.page_stride, a.page_bytes, pieces);
}

}  // namespace

cudaError_t launch_page_copy(const CopyArgs& a, cudaStream_t stream) {
  constexpr int kFew = 64, kMany = 1024;  // pairs a launch: 512 bytes of parameters, or 8 KB
  for (int at = 0; at < a.n;) {
    const int n = a.n - at;
    const cudaError_t e = n <= kFew ? launch_n<kFew>(a, at, n, stream)
                                    : launch_n<kMany>(a, at, n < kMany ? n : kMany, stream);
    if (e != cudaSuccess) return e;
    at += n < kMany ? n : kMany;
  }
  return cudaSuccess;
}

}  // namespace exattn
