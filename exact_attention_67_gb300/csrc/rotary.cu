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
#include "paged.cuh"
#include "ptx.cuh"

#include <limits.h>

#include <algorithm>

namespace exattn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;  // tokens a block at most
static_assert(kMaxTok <= kThreads / 32, "a warp looks up each token");

template <int V>
struct Vec;
template <>
struct Vec<8> { using type = uint4; };
template <>
struct Vec<4> { using type = uint2; };
template <>
struct Vec<2> { using type = uint32_t; };
template <>
struct Vec<1> { using type = uint16_t; };

// One item: two vectors of V elements, as 32-bit words of two (V = 1: one
// element in a word's low half).
template <int V>
struct Item {
  static constexpr int W = V > 1 ? V / 2 : 1;
  union Half {
    typename Vec<V>::type v;
    uint32_t w[W];
    __device__ Half() : w{} {}
  } p1, p2;
};

template <int Q>
struct alignas(4 * Q) Angles {
  float a[Q];
};

// x / d for x below 2^31 and 0 < d < 2^31 by a product: d in (2^(l-1), 2^l],
// magic = ceil(2^(31 + l) / d), x magic >> (31 + l).  magic exceeds 2^(31 + l) / d by
// less than 1, so the product x / d by less than x / 2^(31 + l) < 2^-l <= 1 / d: too
// little to reach the next integer.
struct Divide {
  unsigned d = 1, magic = 1u << 31;
  int shift = 31;

  Divide() = default;
  explicit Divide(unsigned by) : d(by) {
    int l = 0;
    while ((1u << l) < d) ++l;
    shift = 31 + l;
    magic = static_cast<unsigned>(((1ull << shift) + d - 1) / d);
  }
  __device__ unsigned operator()(unsigned x) const {
    return static_cast<unsigned>(static_cast<unsigned long long>(x) * magic >> shift);
  }
};

// How the work is dealt out.
struct Deal {
  unsigned rows;     // tokens
  int tok_shift;     // log2 of the tokens a block
  bool head_major;   // a head's tokens lie side by side
  Divide length;     // rows of a batch entry or sequence
};

// Where a token goes, found once a block.
struct Token {
  long long k, v;  // append: element offsets of head 0 in the caches
  int pos;
  int flags;       // bit 0: a row of some sequence; bit 1: its cache row exists
};

// frac(f / 2 pi) in 64-bit fixed point, by integers alone: FP64 units are few.
// f = m 2^e, finite, with m below 2^53; C is 1 / 2 pi in double precision, as an
// integer.
__device__ __forceinline__ unsigned long long turns_of(double f) {
  constexpr unsigned long long C = static_cast<unsigned long long>(0.15915494309189535 * 73786976294838206464.0);  // 2^66
  const long long bits = __double_as_longlong(f);
  const int field = static_cast<int>(bits >> 52) & 2047;
  const unsigned long long m = (bits & ((1ll << 52) - 1)) | (field ? 1ull << 52 : 0);
  const unsigned long long hi = __umul64hi(m, C), lo = m * C;
  const int s = 1077 - max(field, 1);  // F = m C 2^-s
  const unsigned long long F = s >= 128  ? 0
                               : s >= 64 ? hi >> (s - 64)
                               : s > 0   ? lo >> s | hi << (64 - s)
                               : s > -64 ? lo << -s
                                         : 0;
  return bits < 0 ? 0 - F : F;
}

// The sequence of packed row t: the first b with cu[b + 1] > t (B if none),
// counted by a whole warp with independent loads.
__device__ __forceinline__ int sequence_of(const int* cu, int B, int t, int lane) {
  int n = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    n += __popc(__ballot_sync(0xffffffffu, b < B && cu[b + 1] <= t));
  }
  return n;
}

template <typename T, int D, int V, bool IL, bool APPEND>
__global__ void __launch_bounds__(kThreads, 5) rotary_kernel(const __grid_constant__ RotaryArgs a,
                                                          const __grid_constant__ Deal deal) {
  constexpr int S = D / (2 * V);  // items a head
  constexpr int Q = V < 4 ? V : 4;  // angles a vector load
  __shared__ alignas(16) float cos_s[kMaxTok * (D / 2)], sin_s[kMaxTok * (D / 2)];
  __shared__ unsigned long long turns_s[D / 2];
  __shared__ float factor_s[D / 2];  // of a pair's cos and sin: NaN where its frequency is not finite
  __shared__ Token tk[kMaxTok];
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
  constexpr int ROWS = kThreads / S;
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

  for (int f = tid; f < half; f += kThreads) {
    const double freq = a.inv_freq[f];
    turns_s[f] = turns_of(freq);
    factor_s[f] = isfinite(freq) ? a.factor : __int_as_float(0x7fffffff);
  }
  // Each token by one warp (kMaxTok <= warps).
  if (warp < nt) {
    const unsigned t = t0 + warp;
    Token k{};
    if constexpr (APPEND) {
      int b, i, n;
      if (a.nt.cu_seqlens) {
        b = sequence_of(a.nt.cu_seqlens, a.nt.B, static_cast<int>(t), lane);
        i = n = 0;
        if (b < a.nt.B) {
          const int c0 = a.nt.cu_seqlens[b];
          i = static_cast<int>(t) - c0;
          n = a.nt.cu_seqlens[b + 1] - c0;
        }
      } else {
        b = static_cast<int>(deal.length(t));
        n = a.nt.each;
        i = static_cast<int>(t) - b * n;
      }
      if (b < a.nt.B && i >= 0) {  // a row of some sequence
        k.flags = 1;
        k.pos = a.nt.seqlens[b] - n + i;
        const int slot = k.pos >> a.pv.page_shift;
        if (k.pos >= 0 && slot < a.pv.max_pages) {
          const int page = a.pv.table[b * a.pv.table_stride + slot];
          if (page >= 0 && page < a.pv.num_pages) {
            const int row = k.pos & (a.pv.page_size - 1);
            k.k = page * a.sko.b + row * a.sko.n;
            k.v = page * a.svo.b + row * a.svo.n;
            k.flags = 3;
          }
        }
      }
    } else {
      const unsigned b = deal.length(t);
      k.pos = a.positions[b * a.pos_stride + (t - b * deal.length.d)];
    }
    if (lane == 0) tk[warp] = k;
  }
  __syncthreads();
  for (int i = tid; i < nt * half; i += kThreads) {
    const int tt = i / half, f = i - tt * half;
    const unsigned long long angle = static_cast<unsigned long long>(static_cast<long long>(tk[tt].pos)) * turns_s[f];
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    // Runs of Q angles of neighbouring items side by side: the items' vector
    // loads below then meet no bank twice.
    const int at = tt * (D / 2) + f % V / Q * (S * Q) + f / V * Q + f % Q;
    cos_s[at] = c * factor_s[f];
    sin_s[at] = (a.inverse ? -s : s) * factor_s[f];
  }
  __syncthreads();
  if (!live) return;
  const int flags = APPEND ? tk[t].flags : 3;
  using E = Elem<T>;
  for (int h = hl; h < heads; h += HL) {
    I y;
    load(h + HL, y);
    if (turned && h < hv) {
      float c[V], s[V];
#pragma unroll
      for (int i = 0; i < V / Q; ++i) {
        const int at = t * (D / 2) + i * (S * Q) + slot * Q;
        const Angles<Q> cc = *reinterpret_cast<const Angles<Q>*>(&cos_s[at]);
        const Angles<Q> ss = *reinterpret_cast<const Angles<Q>*>(&sin_s[at]);
#pragma unroll
        for (int j = 0; j < Q; ++j) {
          c[i * Q + j] = cc.a[j];
          s[i * Q + j] = ss.a[j];
        }
      }
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
  constexpr int kRows = kThreads / (D / (2 * V));
  Deal deal{};
  deal.rows = a.append ? a.nt.total : static_cast<unsigned>(a.B) * a.N;
  while ((1 << deal.tok_shift) < std::min(kMaxTok, kRows) && deal.rows >> (deal.tok_shift + 1) >= 152 * 8)
    ++deal.tok_shift;
  deal.head_major = a.Hq > 0 ? a.sq.n < a.sq.h : a.sk.n < a.sk.h;
  deal.length = Divide(!a.append ? a.N : a.nt.each > 0 ? a.nt.each : 1);
  const unsigned grid = (deal.rows + (1u << deal.tok_shift) - 1) >> deal.tok_shift;
  auto kern = a.append ? rotary_kernel<T, D, V, IL, true> : rotary_kernel<T, D, V, IL, false>;
  return launch_dependent("rotary kernel launch", kern, grid, kThreads, 0, stream, a, deal);
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
