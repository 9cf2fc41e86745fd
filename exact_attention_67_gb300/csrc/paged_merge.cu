// paged_merge.cu -- joins the pieces of the units of a paged attention whose
// keys ended up on several CTAs (paged_sched.cuh), for sm_103a.
//
// With a piece's O_s (normalised within it) and mass l_s 2^(m_s), m_s its reference,
// the whole mass is M = sum_s l_s 2^(m_s) and O = sum_s l_s 2^(m_s) O_s / M, the
// combination the online softmax makes inside one CTA.  (By the pieces' logsumexps,
// rounded to 32 bits, a piece's weight was off by 2^-24 |lse|: 1 in 1,000 at scores of
// 20,000.)  One block for each boundary between two
// chunks and a few rows; the first boundary inside a unit joins that unit, any
// other block returns at once.  Launched as a programmatic dependent of the
// kernel that wrote the pieces.
#include "paged.cuh"
#include "paged_sched.cuh"

namespace exattn {

namespace {

// The decode kernel's rows: two a block, WPR warps each, so that a row of few
// long sequences, with a piece on every CTA, is not one chain of loads.  Four
// warps with at most 8 columns, else two.  Whole calls with 2, 4 and 8 warps: 8
// units of 4 pieces 9.2, 9.5, 9.8 us; one unit of 147 pieces 21.1, 16.2, 14.4;
// 192 units of 1 to 3 pieces 141.1, 140.8, 142.8.
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(64 * WPR) paged_merge_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int V = D / 32;      // columns a lane
  constexpr int BATCH = 4;       // pieces a warp loads at once
  __shared__ float2 red[2 * WPR];  // reference, mass
  __shared__ float acc_s[2 * WPR][D];
  // The next kernel of the stream may set itself up; this one waits for the pieces.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = static_cast<int>(blockIdx.x) + 1;  // boundary between CTAs g - 1 and g
  const PagedPlan p = a.plan[g];
  // No unit across this boundary, or one that an earlier boundary joins.
  if (p.pos == 0 || p.pos > p.chunk) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = static_cast<int>(blockIdx.y) * 2 + warp / WPR, part = warp % WPR;
  const int tok = row / a.G;
  const bool live = tok < p.ntok;
  // Pieces: CTA g - 1 + i has the weights [i chunk - lead, (i + 1) chunk - lead)
  // of the unit, lead those of its chunk that lie before it.
  const int w = p.tiles + p.cost, lead = p.chunk - p.pos;
  const int pieces = min((w + lead + p.chunk - 1) / p.chunk, a.ctas - g + 1);
  auto tiles_before = [&](int x) { return max(0, min(w, x) - p.cost); };  // in the unit's first x weights
  auto from = [&](int i) { return tiles_before(i * p.chunk - lead); };
  // All its key tiles on one CTA: that CTA has written the rows itself.
  int used = 0;
  for (int i = 0; i < pieces && used < 2; ++i) used += from(i + 1) > from(i);
  if (used < 2) return;
  // One pass with a running maximum, a batch of pieces' loads all at once.
  float m = -INFINITY, sum = 0.f, acc[V] = {};
  for (int i0 = part; live && i0 < pieces; i0 += BATCH * WPR) {
    float2 l[BATCH];  // references and masses
    float x[BATCH][V];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int i = i0 + u * WPR;
      l[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int c = 0; c < V; ++c) x[u][c] = 0.f;
      if (i >= pieces || from(i + 1) <= from(i)) continue;
      const long long r = (static_cast<long long>(g - 1 + i) * 2 + (from(i) == 0)) * a.rows + row;
      l[u] = a.part_sum[r];
      const float* po = a.part_o + r * D + lane * V;
      if constexpr (V == 4) {
        const float4 y = *reinterpret_cast<const float4*>(po);
        x[u][0] = y.x;
        x[u][1] = y.y;
        x[u][2] = y.z;
        x[u][3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(po);
        x[u][0] = y.x;
        x[u][1] = y.y;
      }
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) top = fmaxf(top, l[u].x);
    // (A NaN is in no maximum, but in the sums, and stays there.)
    const float keep = m == -INFINITY ? 0.f : ex2(m - top);
    sum *= keep;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] *= keep;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const float e = l[u].y == 0.f ? 0.f : l[u].y * ex2(l[u].x - top);
      sum += e;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = fmaf(e, x[u][c], acc[c]);
    }
    m = top;
  }
  // The row's warps, in order.
  if (lane == 0) red[warp] = make_float2(m, sum);
#pragma unroll
  for (int c = 0; c < V; ++c) acc_s[warp][lane * V + c] = acc[c];
  __syncthreads();
  if (part != 0 || !live) return;
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < WPR; ++i) m = fmaxf(m, red[warp + i].x);
  sum = 0.f;
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = 0.f;
#pragma unroll
  for (int i = 0; i < WPR; ++i) {
    const float2 w_i = red[warp + i];
    const float e = w_i.x == -INFINITY ? 0.f : ex2(w_i.x - m);
    sum = fmaf(e, w_i.y, sum);
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = fmaf(e, acc_s[warp + i][lane * V + c], acc[c]);
  }
  const float inv = sum == 0.f ? 0.f : sum_inverse(sum);
  const int head = p.h * a.G + row % a.G, prow = p.row + tok;
  T* out = static_cast<T*>(a.o) + prow * a.so.n + head * a.so.h + lane * V;
#pragma unroll
  for (int c = 0; c < V; c += 2)
    *reinterpret_cast<uint32_t*>(out + c) = Elem<T>::pack(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0) a.lse[static_cast<long long>(head) * a.nt.total + prow] = sum == 0.f ? -INFINITY : (m + sum_log2(sum)) * 0.6931471805599453f;
}

// The forward kernel's rows: a block takes 32 of a query tile, a lane each (their
// partial results lie side by side), and 32 columns, 8 a warp.  One pass with a
// running maximum over the pieces, two at a time (most units have two or three;
// four at a time take more registers and leave fewer blocks an SM: a windowed
// batch of 6 chunks 34.2 us with them, 32.6 with two).  Reading and joining the
// pieces, mostly in L2, is latency: 2 to 5 us a call, 2 % of a long chunk's time.
template <typename T, int D>
__global__ void __launch_bounds__(128) paged_merge_rows_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int C4 = 2, BATCH = 2;  // 4-column vectors a thread, pieces at once
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = static_cast<int>(blockIdx.x) + 1;
  const PagedPlan p = a.plan[g];
  if (p.pos == 0 || p.pos > p.chunk) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.y) >> 2, row = (static_cast<int>(blockIdx.y) & 3) * 32 + lane;
  const int c0 = static_cast<int>(blockIdx.z) * 8 + warp * C4;  // first 4-column vector
  const int row_tok = row / a.G, tok = t * a.tile_tokens + row_tok;
  const int w = p.tiles + p.cost, lead = p.chunk - p.pos;
  const int pieces = min((w + lead + p.chunk - 1) / p.chunk, a.ctas - g + 1);
  auto tiles_before = [&](int x) { return max(0, min(w, x) - p.cost); };
  auto from = [&](int i) { return tiles_before(i * p.chunk - lead); };
  int used = 0;
  for (int i = 0; i < pieces && used < 2; ++i) used += from(i + 1) > from(i);
  if (used < 2) return;
  if (row_tok >= a.tile_tokens || tok >= p.ntok) return;
  float4 acc[C4];
#pragma unroll
  for (int c = 0; c < C4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, sum = 0.f;
  for (int i0 = 0; i0 < pieces; i0 += BATCH) {
    float2 l[BATCH];
    float4 x[BATCH][C4];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int i = i0 + u;
      l[u] = make_float2(-INFINITY, 0.f);
      if (i >= pieces || from(i + 1) <= from(i)) continue;
      const long long part = (static_cast<long long>(g - 1 + i) * 2 + (from(i) == 0)) * 2 + t;
      l[u] = a.part_sum[part * 128 + row];
      const float4* po = reinterpret_cast<const float4*>(a.part_o + part * 128 * D) + c0 * 128 + row;
#pragma unroll
      for (int c = 0; c < C4; ++c) x[u][c] = po[c * 128];
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) top = fmaxf(top, l[u].x);
    const float keep = m == -INFINITY ? 0.f : ex2(m - top);
    sum *= keep;
#pragma unroll
    for (int c = 0; c < C4; ++c)
      acc[c] = make_float4(acc[c].x * keep, acc[c].y * keep, acc[c].z * keep, acc[c].w * keep);
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (l[u].y == 0.f) continue;  // a piece that this row saw no key of: its O may not be written
      const float e = l[u].y * ex2(l[u].x - top);
      sum += e;
#pragma unroll
      for (int c = 0; c < C4; ++c)
        acc[c] = make_float4(fmaf(e, x[u][c].x, acc[c].x), fmaf(e, x[u][c].y, acc[c].y), fmaf(e, x[u][c].z, acc[c].z),
                             fmaf(e, x[u][c].w, acc[c].w));
    }
    m = top;
  }
  const float inv = sum == 0.f ? 0.f : sum_inverse(sum);
  const int head = p.h * a.G + row % a.G, prow = p.row + tok;
  T* out = static_cast<T*>(a.o) + prow * a.so.n + head * a.so.h + c0 * 4;
  *reinterpret_cast<uint4*>(out) =
      make_uint4(Elem<T>::pack(acc[0].x * inv, acc[0].y * inv), Elem<T>::pack(acc[0].z * inv, acc[0].w * inv),
                 Elem<T>::pack(acc[1].x * inv, acc[1].y * inv), Elem<T>::pack(acc[1].z * inv, acc[1].w * inv));
  if (c0 == 0) a.lse[static_cast<long long>(head) * a.nt.total + prow] = sum == 0.f ? -INFINITY : (m + sum_log2(sum)) * 0.6931471805599453f;
}

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t stream) {
  const bool few = a.cols > 0, deep = few && a.cols <= 8;
  const dim3 grid(a.ctas - 1, few ? a.cols / 2 : 8, few ? 1 : D / 32), block(deep ? 256 : 128);
  const char* what = "paged merge kernel launch";
  return deep  ? launch_dependent(what, paged_merge_kernel<T, D, 4>, grid, block, 0, stream, a)
         : few ? launch_dependent(what, paged_merge_kernel<T, D, 2>, grid, block, 0, stream, a)
               : launch_dependent(what, paged_merge_rows_kernel<T, D>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t stream) {
  if (a.ctas < 2) return cudaSuccess;
  if (a.dtype == kF16) return a.d == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_t<__nv_bfloat16, 64>(a, stream) : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
