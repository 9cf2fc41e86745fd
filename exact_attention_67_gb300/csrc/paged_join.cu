// paged_join.cu -- joins what the two lines of an attention behind shared rows left of
// every query row (PagedShare), for sm_103a.
//
// A row's keys lie in pieces: its own in one (the row buffer) or in several (slots of
// consecutive CTAs, when its unit was cut), and so the shared ones.  With a piece's O_s
// (normalised within it) and mass l_s 2^(m_s), O = sum_s l_s 2^(m_s) O_s / M, M the sum
// of the masses, as in paged_merge.cu.  The records say where the pieces are.  They are
// this library's own, but rows that the tables leave out of every group have none: what
// lies there instead is checked before it is used as a place.
//
// LPR lanes a row and head: a whole warp, and four of them that share its pieces out
// where there are few rows, or eight lanes, four rows a warp, where there are many.  A
// chain of three loads (record, mass, O), so what counts is how many rows are in flight:
// 50,624 rows of 128 (76 MB read) 19.7 us, 3.7 TB/s; a few rows 2 to 3 us.
#include "paged.cuh"
#include "paged_sched.cuh"

namespace exattn {

namespace {

struct JoinLine {
  const PagedRecord* rec;
  const float* part_o;
  const float2* part_sum;
  const PagedPlan* plan;
  long long rows_at;
  int rows, slots;  // of a piece; of all
};

struct JoinArgs {
  JoinLine line[2];
  void* o;
  Strides so;
  float* lse;
  NewTokens nt;
  const int* prefix;  // shared rows of a sequence, as the lines take them
  int Hq, max_q, max_k;
};

// Where piece i of a line's row is.
struct JoinPieces {
  int count;  // 0: none; whole: 1, in the row buffer
  int first;  // slot, or -1: the row buffer
  float2 whole;
};
__device__ __forceinline__ JoinPieces pieces_of(const JoinLine& l, const PagedRecord& r, int chunk) {
  JoinPieces p{1, -1, make_float2(r.ref, r.mass)};
  if (r.rest <= 0) return p;
  p.count = 2 + (min(r.rest, 1 << 24) - 1) / max(chunk, 1);
  p.first = r.part;
  // CTA c's pieces: slot 2 c continues a unit, 2 c + 1 begins one.
  const long long last = r.part + (2ll * p.count - 3) * l.rows;
  if (r.part < 0 || last >= l.slots) p.count = 0;
  return p;
}

// WPR warps a row, or (WPR = 1) LPR lanes.
template <typename T, int D, int LPR, int WPR>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ JoinArgs a) {
  static_assert(WPR == 1 || LPR == 32, "several warps, or a part of one");
  constexpr int V = D / LPR, V4 = V / 4 > 0 ? V / 4 : 1, BATCH = V > 4 ? 2 : 4;  // columns a lane; pieces at once
  constexpr int HEADS = 256 / LPR / WPR;                                          // of a block
  __shared__ float2 red[8];  // reference, mass
  __shared__ float acc_s[WPR > 1 ? 8 : 1][D];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = threadIdx.x % LPR, part = WPR > 1 ? warp % WPR : 0;
  const int row = blockIdx.x, head = static_cast<int>(blockIdx.y) * HEADS + static_cast<int>(threadIdx.x) / (LPR * WPR);
  bool live = head < a.Hq;
  const long long at = static_cast<long long>(row) * a.Hq + (live ? head : 0);
  // Records, chunks and the row's place among its sequence's tokens.
  const PagedRecord r0 = a.line[0].rec[at], r1 = a.line[1].rec[at];
  const int chunk0 = a.line[0].plan->chunk, chunk1 = a.line[1].plan->chunk;
  int b = 0;
  if (a.nt.cu_seqlens) {
    for (int b0 = 0; b0 < a.nt.B; b0 += 32)
      b += __popc(__ballot_sync(0xffffffffu, b0 + lane < a.nt.B && a.nt.cu_seqlens[b0 + lane + 1] <= row));
    const int i = b < a.nt.B ? row - a.nt.cu_seqlens[b] : -1;
    live = live && i >= 0 && i < a.max_q;
  } else {
    b = row / a.nt.each;
    live = live && row - b * a.nt.each < a.max_q;
  }
  // (Rows of a group that shares nothing have no record in the shared line.)
  const bool shares = live && min(a.prefix[b], a.max_k) >= kKeyTile;
  JoinPieces p0 = pieces_of(a.line[0], r0, chunk0);
  const JoinPieces p1 = pieces_of(a.line[1], r1, chunk1);
  if (!shares) p0.count = 0;
  const int count = live ? p0.count + p1.count : 0;
  float m = -INFINITY, sum = 0.f, acc[V] = {};
  for (int i0 = part; i0 < count; i0 += BATCH * WPR) {
    float2 l[BATCH];
    float x[BATCH][V];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int i = i0 + u * WPR;
      l[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int c = 0; c < V; ++c) x[u][c] = 0.f;
      if (i >= count) continue;
      const bool shared = i < p0.count;
      const JoinLine& ln = a.line[shared ? 0 : 1];
      const JoinPieces& p = shared ? p0 : p1;
      const int j = shared ? i : i - p0.count;
      long long from = ln.rows_at + at * D;
      if (p.first >= 0) {
        const long long slot = p.first + (j ? (2ll * j - 1) * ln.rows : 0);
        l[u] = ln.part_sum[slot];
        from = slot * D;
      } else {
        l[u] = p.whole;
      }
      if constexpr (V == 2) {
        const float2 y = *reinterpret_cast<const float2*>(ln.part_o + from + sub * V);
        x[u][0] = y.x;
        x[u][1] = y.y;
      } else {
        const float4* po = reinterpret_cast<const float4*>(ln.part_o + from) + sub;  // vectors LPR apart
#pragma unroll
        for (int c = 0; c < V4; ++c) {
          const float4 y = po[c * LPR];
          x[u][4 * c] = y.x;
          x[u][4 * c + 1] = y.y;
          x[u][4 * c + 2] = y.z;
          x[u][4 * c + 3] = y.w;
        }
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
      if (l[u].y == 0.f) continue;  // a piece that this row saw no key of: its O may not be written
      const float e = l[u].y * ex2(l[u].x - top);
      sum += e;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = fmaf(e, x[u][c], acc[c]);
    }
    m = top;
  }
  if constexpr (WPR > 1) {  // the row's warps, in order
    if (lane == 0) red[warp] = make_float2(m, sum);
#pragma unroll
    for (int c = 0; c < V; ++c) acc_s[warp][lane * V + c] = acc[c];
    __syncthreads();
    if (part != 0) return;
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < WPR; ++i) m = fmaxf(m, red[warp + i].x);
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) {
      const float2 w = red[warp + i];
      if (w.y == 0.f) continue;
      const float e = ex2(w.x - m);
      sum = fmaf(e, w.y, sum);
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = fmaf(e, acc_s[warp + i][lane * V + c], acc[c]);
    }
  }
  if (!live) return;
  const float inv = sum == 0.f ? 0.f : sum_inverse(sum);
  T* out = static_cast<T*>(a.o) + row * a.so.n + head * a.so.h;
  if constexpr (V == 2) {
    reinterpret_cast<uint32_t*>(out)[sub] = Elem<T>::pack(acc[0] * inv, acc[1] * inv);
  } else {
#pragma unroll
    for (int c = 0; c < V4; ++c)
      reinterpret_cast<uint2*>(out)[sub + c * LPR] = make_uint2(Elem<T>::pack(acc[4 * c] * inv, acc[4 * c + 1] * inv),
                                                                Elem<T>::pack(acc[4 * c + 2] * inv, acc[4 * c + 3] * inv));
  }
  if (sub == 0)
    a.lse[static_cast<long long>(head) * a.nt.total + row] = sum == 0.f ? -INFINITY : (m + sum_log2(sum)) * 0.6931471805599453f;
}

template <typename T, int D>
cudaError_t launch_t(const JoinArgs& a, cudaStream_t stream) {
  // Few rows have many pieces each; many have few.
  const long long rows = static_cast<long long>(a.nt.total) * a.Hq;
  const int heads = rows <= 1024 ? 2 : rows <= 8192 ? 8 : 32;
  const dim3 grid(a.nt.total, (a.Hq + heads - 1) / heads);
  auto kern = heads == 2 ? paged_join_kernel<T, D, 32, 4> : heads == 8 ? paged_join_kernel<T, D, 32, 1> : paged_join_kernel<T, D, 8, 1>;
  return launch_dependent("paged join kernel launch", kern, grid, 256, 0, stream, a);
}

}  // namespace

cudaError_t launch_paged_join(const PagedArgs& shared, const PagedArgs& own, cudaStream_t stream) {
  JoinArgs a{};
  const PagedArgs* lines[2] = {&shared, &own};
  for (int i = 0; i < 2; ++i) {
    const PagedArgs& l = *lines[i];
    a.line[i] = JoinLine{l.share.rec, l.part_o, l.part_sum, l.plan, l.share.rows_at, l.rows, l.ctas * 2 * l.rows};
  }
  a.o = own.o;
  a.so = own.so;
  a.lse = own.lse;
  a.nt = own.nt;
  a.Hq = own.Hkv * own.G;
  a.max_q = own.max_q;
  a.max_k = own.max_k;
  a.prefix = own.share.prefix;
  if (own.dtype == kF16) return own.d == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return own.d == 64 ? launch_t<__nv_bfloat16, 64>(a, stream) : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
