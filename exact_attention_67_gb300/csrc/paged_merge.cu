// paged_merge.cu -- joins the pieces of the units of a paged attention whose
// keys ended up on several CTAs (paged_sched.cuh), for sm_103a.
//
// With a piece's O_s (normalised within it) and logsumexp L_s, lse = log sum_s
// exp(L_s) and O = sum_s exp(L_s - lse) O_s, the combination the online
// softmax makes inside one CTA.  One block for each boundary between two
// chunks and a few rows; the first boundary inside a unit joins that unit, any
// other block returns at once.  Launched as a programmatic dependent of the
// kernel that wrote the pieces.
#include "paged.cuh"
#include "paged_sched.cuh"

namespace exattn {

namespace {

// RPB rows a block of eight warps, 8 / RPB warps a row: one warp a row for the
// forward kernel's 256 rows (few pieces each), all eight for the decode
// kernel's rows, whose pieces can be as many as there are CTAs.
template <typename T, int D, int RPB>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PagedArgs a, int rows, int UT) {
  constexpr int WPR = 8 / RPB;   // warps a row
  constexpr int V = D / 32;      // columns a lane
  __shared__ float red[8];
  __shared__ float acc_s[8][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = static_cast<int>(blockIdx.x) + 1;  // boundary between CTAs g - 1 and g
  const int* plan = a.plan + g * 8;
  if (!plan[0] || plan[4] == 0) return;  // no chunk starts here, or it starts a unit
  const long long chunk = (static_cast<long long>(plan[6]) << 31) | plan[5];
  const int pos = plan[4];
  if (pos > chunk) return;  // an earlier boundary is inside the unit too
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = static_cast<int>(blockIdx.y) * RPB + warp / WPR, part = warp % WPR;
  const PagedSeq s = paged_seq(a, plan[1]);
  const int h = plan[2], t0 = plan[3] * UT, t1 = min(s.n, t0 + UT);
  int lo, hi;
  paged_keys(a, s, t0, t1, &lo, &hi);
  const int k0 = lo / kKeyTile, k1 = hi > lo ? (hi + kKeyTile - 1) / kKeyTile : k0;
  const int w = k1 - k0 + a.unit_cost;
  // Pieces: CTA g - 1 + i has weights [i chunk - lead, (i + 1) chunk - lead) of
  // the unit, lead those of its chunk that lie before it.
  const long long lead = chunk - pos;
  const int pieces = static_cast<int>((w + lead + chunk - 1) / chunk);
  auto tiles_before = [&](long long x) {  // key tiles in the unit's first x weights
    return static_cast<int>(max(0ll, min(static_cast<long long>(w), x) - a.unit_cost));
  };
  auto empty = [&](int i) { return tiles_before((i + 1) * chunk - lead) <= tiles_before(i * chunk - lead); };
  // All its key tiles on one CTA: that CTA has written the rows itself.
  int used = 0;
  for (int i = 0; i < pieces && used < 2; ++i) used += !empty(i);
  if (used < 2) return;
  // Row r of the unit lies in query tile r / 128 at the forward kernel (tiles
  // of tile_tokens G rows), in the only one at the decode kernel.
  const int tile = row / 128, tr = row % 128;
  const int tok = t0 + tile * a.tile_tokens + tr / a.G;
  const bool live = row < rows && tr < a.tile_tokens * a.G && tok < t1;
  auto at = [&](int i) {
    const int first = tiles_before(i * chunk - lead) == 0;
    return (static_cast<long long>(g - 1 + i) * 2 + first) * rows + row;
  };
  float m = -INFINITY;
  if (live)
    for (int i = part * 32 + lane; i < pieces; i += 32 * WPR)
      if (!empty(i)) m = fmaxf(m, a.part_lse[at(i)]);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if constexpr (WPR > 1) {
    if (lane == 0) red[warp] = m;
    __syncthreads();
    for (int i = 0; i < WPR; ++i) m = fmaxf(m, red[warp - part + i]);
  }
  float acc[V] = {}, sum = 0.f;
  if (live && m != -INFINITY) {
    for (int i = part; i < pieces; i += WPR) {
      if (empty(i)) continue;
      const long long r = at(i);
      const float l = a.part_lse[r];
      if (l == -INFINITY) continue;
      const float e = expf(l - m);
      sum += e;
      const float* po = a.part_o + r * D + lane * V;
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(po);
        acc[0] = fmaf(e, x.x, acc[0]);
        acc[1] = fmaf(e, x.y, acc[1]);
        acc[2] = fmaf(e, x.z, acc[2]);
        acc[3] = fmaf(e, x.w, acc[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(po);
        acc[0] = fmaf(e, x.x, acc[0]);
        acc[1] = fmaf(e, x.y, acc[1]);
      }
    }
  }
  if constexpr (WPR > 1) {
    __syncthreads();
    if (lane == 0) red[warp] = sum;
#pragma unroll
    for (int c = 0; c < V; ++c) acc_s[warp][lane * V + c] = acc[c];
    __syncthreads();
    if (part != 0) return;
    for (int i = 1; i < WPR; ++i) {
      sum += red[warp + i];
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] += acc_s[warp + i][lane * V + c];
    }
  }
  if (!live) return;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int head = h * a.G + tr % a.G, prow = s.row0 + tok;
  T* out = static_cast<T*>(a.o) + prow * a.so.n + head * a.so.h + lane * V;
#pragma unroll
  for (int c = 0; c < V; c += 2)
    *reinterpret_cast<uint32_t*>(out + c) = Elem<T>::pack(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0) a.lse[static_cast<long long>(head) * a.nt.total + prow] = sum > 0.f ? m + logf(sum) : -INFINITY;
}

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t stream) {
  const int rows = a.rows;
  const bool few = a.cols > 0;
  const int UT = few ? a.tile_tokens : 2 * a.tile_tokens;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas - 1, few ? a.cols : rows / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, D, 1>, a, rows, UT)
                            : cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, D, 8>, a, rows, UT);
  const cudaError_t last = cudaGetLastError();
  return note_cuda(e != cudaSuccess ? e : last, "paged merge kernel launch");
}

}  // namespace

cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t stream) {
  if (a.ctas < 2) return cudaSuccess;
  if (a.dtype == kF16) return a.d == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_t<__nv_bfloat16, 64>(a, stream) : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
