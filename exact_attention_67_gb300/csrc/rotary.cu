// rotary.cu -- rotary positions and the append of new tokens to a paged
// key/value cache, for sm_103a.
//
// Rotary positions turn each pair (x1, x2) of the first `rot` elements of a
// head by the angle a = p f_i (position p, frequency f_i of pair i):
//     y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a),
// with the caller's factor m; the other elements are copied.  Pairs are
// (i, i + rot / 2) or, interleaved, (2 i, 2 i + 1).  The map is m times an
// orthogonal one, so its gradient is the same kernel with the angle negated.
//
// Angles.  p f_i in 32 bits is wrong by p 2^-24 radians (0.06 at p = 10^6), and
// only its fraction of a turn matters.  Frequencies arrive in 64 bits and are
// taken as turns a token in 64-bit fixed point, F = frac(f / 2 pi) 2^64; then
// p F mod 2^64 is the angle's fraction of a turn, with no range reduction, from
// one integer product, whose upper 32 bits sincospi takes as an fp32 number of half
// turns.  Errors: |p f| 2^-53 radians from 1 / 2 pi to 53 bits; in turns |p| 2^-64 from
// F cut off at 64 bits, 2^-32 from keeping the upper half and 2^-26 from its conversion
// to fp32: together below |p f| 2^-53 + 2^-23 radians.  (p f formed in 64-bit floating
// point is off by |p f| 2^-53 too.)  The turned values are rounded once, to the
// output's type.
//
// A block takes a few consecutive tokens: it forms cos and sin of their rot / 2
// angles once, in shared memory, for all heads of Q and K; a thread turns one item
// of 2 V elements (two 16-byte vectors at V = 8) of one token in every few heads,
// the next one's loads in flight, the first of them while the tokens are looked up
// and the angles formed.  V is the widest vector that divides rot / 2 (interleaved:
// half of an item's run), so rot a multiple of 16 moves 16-byte vectors.
//
// Bound by memory traffic, every element read and written once, and near it by
// instructions: 8,192 tokens of 16 + 16 heads of 128, head-major, 23.8 us (5.6
// TB/s; a plain elementwise map of these bytes 21.3 us), 16,380 tokens of 32 + 8
// heads of 64 28.8 us (5.8 TB/s; 26.0), 9,838 appended tokens of 32 + 8 + 8 heads
// of 128 42.5 us (5.7 TB/s; 36.4).  Before: angles by FP64, divisions and a
// thread's angles kept in registers 26.5, 32.5 and 46.6 us.  Narrower vectors move
// the copied part of a head, and V, too: the first case with rot 24, 20 and 6 (8, 4
// and 2 bytes) 25.4, 32.1 and 71.0 us, the append with rot 20 and 6 53.9 and 129.7.
#include "rotary.cuh"

#include <limits.h>

#include <algorithm>

namespace exattn {

namespace {

template <typename T, int D, int V, bool IL, bool APPEND>
__global__ void __launch_bounds__(kRotaryThreads, 5) rotary_kernel(const __grid_constant__ RotaryArgs a,
                                                          const __grid_constant__ Deal deal) {
  constexpr int S = D / (2 * V);  // items a head
  __shared__ AngleTable<D> angles;
  __shared__ Token tk[kRotaryTokens];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned t0 = blockIdx.x << deal.tok_shift;
  const int nt = static_cast<int>(min(1u << deal.tok_shift, deal.rows - t0));

  // This thread: item `slot` of the heads hl, hl + HL, ... (of Q, K, V in order) of
  // one token.  Of the tokens and heads of a block, neighbouring threads take those
  // that lie side by side.
  using VT = typename Vec<V>::type;
  using I = Item<V>;
  constexpr int ROWS = kRotaryThreads / S;
  const int half = a.inv_freq ? a.rot >> 1 : 0;
  const int heads = a.Hq + a.Hk + (APPEND ? a.Hk : 0), HL = ROWS >> deal.tok_shift;
  const int slot = tid % S, r = tid / S;
  const int t = deal.head_major ? r & ((1 << deal.tok_shift) - 1) : r / HL;
  const int hl = deal.head_major ? r >> deal.tok_shift : r & (HL - 1);
  const bool live = t < nt;
  const unsigned row = t0 + (live ? t : 0), b = APPEND ? 0 : deal.length(row);
  const unsigned n = APPEND ? row : row - b * deal.length.d;
  auto at = [&](const Strides& st) { return (APPEND ? 0 : b * st.b) + n * st.n; };
  const int pairs0 = slot * V;
  const bool turned = pairs0 < half;
  // The item's two vectors: its pairs' halves, or (interleaved, and past the
  // turned part) 2 V consecutive elements.  V is copied whole: the same places.
  const int e1 = !IL && turned ? pairs0 : 2 * pairs0;
  const int e2 = !IL && turned ? pairs0 + half : 2 * pairs0 + V;
  // Places of head h: base + h * stride, each tensor's heads counted on.
  const int hk = a.Hq, hv = APPEND ? a.Hq + a.Hk : INT_MAX;
  auto load = [&](int h, I& x) {
    if (!live || h >= heads) return;
    const T* src;
    if (h < hk) src = static_cast<const T*>(a.q) + at(a.sq) + h * a.sq.h;
    else if (h < hv) src = static_cast<const T*>(a.k) + at(a.sk) + (h - hk) * a.sk.h;
    else src = static_cast<const T*>(a.v) + at(a.sv) + (h - hv) * a.sv.h;
    x.p1.v = *reinterpret_cast<const VT*>(src + e1);
    x.p2.v = *reinterpret_cast<const VT*>(src + e2);
  };
  // The first item is on its way while the tokens are looked up and their angles
  // formed.
  I x;
  load(hl, x);

  read_frequencies<D>(a, half, angles);
  // Each token by one warp (kRotaryTokens <= warps).
  if (warp < nt) {
    const Token k = find_token<APPEND>(a, deal, t0 + warp, lane);
    if (lane == 0) tk[warp] = k;
  }
  __syncthreads();
  form_angles<D, V>(a, half, nt, tk, angles);
  __syncthreads();
  if (!live) return;
  const int flags = APPEND ? tk[t].flags : 3;
  using E = Elem<T>;
  for (int h = hl; h < heads; h += HL) {
    I y;
    load(h + HL, y);
    if (turned && h < hv) {
      float c[V], s[V];
      angle_load<D, V>(angles.cos + t * (D / 2), slot, c);
      angle_load<D, V>(angles.sin + t * (D / 2), slot, s);
      if constexpr (V == 1) {
        const float x1 = E::unpack(x.p1.w[0]).x, x2 = E::unpack(x.p2.w[0]).x;
        x.p1.w[0] = E::pack(x1 * c[0] - x2 * s[0], 0.f);
        x.p2.w[0] = E::pack(x2 * c[0] + x1 * s[0], 0.f);
      } else if constexpr (!IL) {
#pragma unroll
        for (int i = 0; i < I::W; ++i) {
          const float2 x1 = E::unpack(x.p1.w[i]), x2 = E::unpack(x.p2.w[i]);
          const float2 cc = make_float2(c[2 * i], c[2 * i + 1]), ss = make_float2(s[2 * i], s[2 * i + 1]);
          const float2 y1 = ffma2(x2, make_float2(-ss.x, -ss.y), fmul2(x1, cc)), y2 = ffma2(x1, ss, fmul2(x2, cc));
          x.p1.w[i] = E::pack(y1.x, y1.y);
          x.p2.w[i] = E::pack(y2.x, y2.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {  // pair i is one word
          uint32_t& w = i < I::W ? x.p1.w[i] : x.p2.w[i - I::W];
          const float2 z = E::unpack(w);
          const float2 r = ffma2(make_float2(z.y, z.x), make_float2(-s[i], s[i]), fmul2(z, make_float2(c[i], c[i])));
          w = E::pack(r.x, r.y);
        }
      }
    }
    T* dst;
    if (h < hk) dst = static_cast<T*>(a.q_out) + at(a.sqo) + h * a.sqo.h;
    else if (!APPEND) dst = static_cast<T*>(a.k_out) + at(a.sko) + (h - hk) * a.sko.h;
    else if (h < hv) dst = static_cast<T*>(a.k_out) + tk[t].k + (h - hk) * a.sko.h;
    else dst = static_cast<T*>(a.v_out) + tk[t].v + (h - hv) * a.svo.h;
    if (flags & (h < hk ? 1 : 2)) {
      *reinterpret_cast<VT*>(dst + e1) = x.p1.v;
      *reinterpret_cast<VT*>(dst + e2) = x.p2.v;
    }
    x = y;
  }
}

template <typename T, int D, int V, bool IL>
cudaError_t launch_t(const RotaryArgs& a, cudaStream_t stream) {
  // Several tokens a block (a power of two) once that still leaves eight blocks an
  // SM: 8,192 tokens with four 23.5 us, two (sixteen blocks) 25.3, one 29.
  constexpr int kRows = kRotaryThreads / (D / (2 * V));
  Deal deal{};
  deal.rows = a.append ? a.nt.total : static_cast<unsigned>(a.B) * a.N;
  while ((1 << deal.tok_shift) < std::min(kRotaryTokens, kRows) && deal.rows >> (deal.tok_shift + 1) >= 152 * 8)
    ++deal.tok_shift;
  deal.head_major = a.Hq > 0 ? a.sq.n < a.sq.h : a.sk.n < a.sk.h;
  deal.length = Divide(!a.append ? a.N : a.nt.each > 0 ? a.nt.each : 1);
  const unsigned grid = (deal.rows + (1u << deal.tok_shift) - 1) >> deal.tok_shift;
  auto kern = a.append ? rotary_kernel<T, D, V, IL, true> : rotary_kernel<T, D, V, IL, false>;
  return launch_dependent("rotary kernel launch", kern, grid, kRotaryThreads, 0, stream, a, deal);
}

template <typename T, int D>
cudaError_t launch_d(const RotaryArgs& a, cudaStream_t stream) {
  const int rot = a.inv_freq ? a.rot : D;
  const int v = rot % 16 == 0 ? 8 : rot % 8 == 0 ? 4 : rot % 4 == 0 ? 2 : 1;
  if (a.interleaved) {
    if (v == 8) return launch_t<T, D, 8, true>(a, stream);
    if (v == 4) return launch_t<T, D, 4, true>(a, stream);
    if (v == 2) return launch_t<T, D, 2, true>(a, stream);
    return launch_t<T, D, 1, true>(a, stream);
  }
  if (v == 8) return launch_t<T, D, 8, false>(a, stream);
  if (v == 4) return launch_t<T, D, 4, false>(a, stream);
  if (v == 2) return launch_t<T, D, 2, false>(a, stream);
  return launch_t<T, D, 1, false>(a, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t stream) {
  if (a.dtype == kF16) return a.d == 64 ? launch_d<__half, 64>(a, stream) : launch_d<__half, 128>(a, stream);
  return a.d == 64 ? launch_d<__nv_bfloat16, 64>(a, stream) : launch_d<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
