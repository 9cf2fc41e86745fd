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
// one integer product (error below |p| 2^-54 turns from the 53 bits of f, and
// 2^-33 from keeping the upper 32 bits), which sincospi takes in 32 bits.
// The turned values are rounded once, to the output's type.
//
// A block takes a few consecutive tokens: it forms cos and sin of their
// rot / 2 angles once, in shared memory, for all heads of Q and K; a thread
// turns one item of 2 V elements (two 16-byte vectors at V = 8), whose cos and sin
// it keeps, of every few heads, two items in flight, the first of them while the
// angles are formed.  Bound by memory traffic: every element is read once and
// written once.  V is the widest vector that divides rot / 2 (interleaved: half
// of an item's run), so rot a multiple of 16 moves 16-byte vectors.
#include "paged.cuh"
#include "ptx.cuh"

namespace exattn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;  // tokens a block at most
constexpr int kBatch = 2;   // items a thread has in flight
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

// What a block knows of each of its tokens.
struct Token {
  long long q, qo, k, ko, v, vo;  // element offsets of head 0
  int pos;
  int flags;  // bit 0: the token exists; bit 1: its cache row does
};

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
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryArgs a, int tok_per_block,
                                                          long long tokens) {
  constexpr int S = D / (2 * V);  // items a head
  constexpr int Q = V < 4 ? V : 4;  // angles a vector load
  __shared__ alignas(16) float cos_s[kMaxTok * (D / 2)], sin_s[kMaxTok * (D / 2)];
  __shared__ Token tk[kMaxTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long t0 = static_cast<long long>(blockIdx.x) * tok_per_block;
  const int nt = static_cast<int>(min(static_cast<long long>(tok_per_block), tokens - t0));

  // Each token by one warp (kMaxTok <= warps).
  if (warp < nt) {
    const long long t = t0 + warp;
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
        b = static_cast<int>(t / a.nt.each);
        i = static_cast<int>(t % a.nt.each);
        n = a.nt.each;
      }
      if (b < a.nt.B && i >= 0) {  // a row of some sequence
        k.flags = 1;
        k.pos = a.nt.seqlens[b] - n + i;
        const int slot = k.pos >> a.pv.page_shift;
        if (k.pos >= 0 && slot < a.pv.max_pages) {
          const int page = a.pv.table[b * a.pv.table_stride + slot];
          if (page >= 0 && page < a.pv.num_pages) {
            const int row = k.pos & (a.pv.page_size - 1);
            k.ko = page * a.sko.b + row * a.sko.n;
            k.vo = page * a.svo.b + row * a.svo.n;
            k.flags = 3;
          }
        }
      }
      k.q = t * a.sq.n;
      k.qo = t * a.sqo.n;
      k.k = t * a.sk.n;
      k.v = t * a.sv.n;
    } else {
      const int b = static_cast<int>(t / a.N);
      const int n = static_cast<int>(t - static_cast<long long>(b) * a.N);
      k.pos = a.positions[b * a.pos_stride + n];
      k.flags = 3;
      k.q = b * a.sq.b + n * a.sq.n;
      k.qo = b * a.sqo.b + n * a.sqo.n;
      k.k = b * a.sk.b + n * a.sk.n;
      k.ko = b * a.sko.b + n * a.sko.n;
    }
    if (lane == 0) tk[warp] = k;
  }
  __syncthreads();

  // This thread: item `slot` of the heads hl, hl + HL, ... of one token.
  using VT = typename Vec<V>::type;
  using I = Item<V>;
  const int half = a.inv_freq ? a.rot >> 1 : 0;
  const int heads = a.Hq + a.Hk + (APPEND ? a.Hk : 0);
  const int slot = tid % S, t = tid / S & (tok_per_block - 1), hl = tid / S / tok_per_block;
  const int HL = kThreads / S / tok_per_block;
  const bool live = t < nt;
  const Token k = live ? tk[t] : Token{};
  const int pairs0 = slot * V;
  const bool turned = pairs0 < half;
  // The item's two vectors: its pairs' halves, or (interleaved, and past the
  // turned part) 2 V consecutive elements.  V is copied whole: the same places.
  const int e1 = !IL && turned ? pairs0 : 2 * pairs0;
  const int e2 = !IL && turned ? pairs0 + half : 2 * pairs0 + V;
  I x[kBatch];
  T* dst[kBatch];
  auto load = [&](int h, I& x, T*& dst) {
    dst = nullptr;
    if (!live || h >= heads) return;
    const T* src;
    if (h < a.Hq) {
      if (!(k.flags & 1)) return;
      src = static_cast<const T*>(a.q) + (k.q + h * a.sq.h);
      dst = static_cast<T*>(a.q_out) + (k.qo + h * a.sqo.h);
    } else {
      if (!(k.flags & 2)) return;
      const int g = h - a.Hq;
      if (!APPEND || g < a.Hk) {
        src = static_cast<const T*>(a.k) + (k.k + g * a.sk.h);
        dst = static_cast<T*>(a.k_out) + (k.ko + g * a.sko.h);
      } else {
        src = static_cast<const T*>(a.v) + (k.v + (g - a.Hk) * a.sv.h);
        dst = static_cast<T*>(a.v_out) + (k.vo + (g - a.Hk) * a.svo.h);
      }
    }
    x.p1.v = *reinterpret_cast<const VT*>(src + e1);
    x.p2.v = *reinterpret_cast<const VT*>(src + e2);
  };
  // The first items are on their way while the angles are formed.
#pragma unroll
  for (int u = 0; u < kBatch; ++u) load(hl + u * HL, x[u], dst[u]);
  for (int i = tid; i < nt * half; i += kThreads) {
    const int tt = i / half, f = i - tt * half;
    double turns = a.inv_freq[f] * 0.15915494309189535;  // 1 / 2 pi
    turns -= floor(turns);
    const unsigned long long F = __double2ull_rn(turns * 18446744073709551616.0);
    const unsigned long long angle = static_cast<unsigned long long>(static_cast<long long>(tk[tt].pos)) * F;
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    // Runs of Q angles of neighbouring items side by side: the items' vector
    // loads below then meet no bank twice.
    const int at = tt * (D / 2) + f % V / Q * (S * Q) + f / V * Q + f % Q;
    cos_s[at] = c * a.factor;
    sin_s[at] = (a.inverse ? -s : s) * a.factor;
  }
  __syncthreads();
  float c[V] = {}, s[V] = {};
  if (turned) {
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
  }
  using E = Elem<T>;
  for (int h = hl; h < heads; h += kBatch * HL) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (dst[u] == nullptr) continue;
      I& y = x[u];
      const bool turn = turned && (!APPEND || h + u * HL < a.Hq + a.Hk);
      if (turn) {
        if constexpr (V == 1) {
          const float x1 = E::unpack(y.p1.w[0]).x, x2 = E::unpack(y.p2.w[0]).x;
          y.p1.w[0] = E::pack(x1 * c[0] - x2 * s[0], 0.f);
          y.p2.w[0] = E::pack(x2 * c[0] + x1 * s[0], 0.f);
        } else if constexpr (!IL) {
#pragma unroll
          for (int i = 0; i < I::W; ++i) {
            const float2 x1 = E::unpack(y.p1.w[i]), x2 = E::unpack(y.p2.w[i]);
            const float2 cc = make_float2(c[2 * i], c[2 * i + 1]), ss = make_float2(s[2 * i], s[2 * i + 1]);
            const float2 y1 = ffma2(x2, make_float2(-ss.x, -ss.y), fmul2(x1, cc)), y2 = ffma2(x1, ss, fmul2(x2, cc));
            y.p1.w[i] = E::pack(y1.x, y1.y);
            y.p2.w[i] = E::pack(y2.x, y2.y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) {  // pair i is one word
            uint32_t& w = i < I::W ? y.p1.w[i] : y.p2.w[i - I::W];
            const float2 z = E::unpack(w);
            const float2 r = ffma2(make_float2(z.y, z.x), make_float2(-s[i], s[i]), fmul2(z, make_float2(c[i], c[i])));
            w = E::pack(r.x, r.y);
          }
        }
      }
      *reinterpret_cast<VT*>(dst[u] + e1) = y.p1.v;
      *reinterpret_cast<VT*>(dst[u] + e2) = y.p2.v;
      load(h + (kBatch + u) * HL, y, dst[u]);  // its successor, while the other item is turned
    }
  }
}

template <typename T, int D, int V, bool IL>
cudaError_t launch_t(const RotaryArgs& a, cudaStream_t stream) {
  const long long tokens = a.append ? a.nt.total : static_cast<long long>(a.B) * a.N;
  // Several tokens a block (a power of two, at most a block's rows of items)
  // once that still leaves sixteen blocks an SM.
  constexpr int kRows = kThreads / (D / (2 * V));
  int tok = 1;
  while (tok < kMaxTok && tok < kRows && tokens / (2 * tok) >= 152 * 16) tok *= 2;
  const long long grid = (tokens + tok - 1) / tok;
  auto kern = a.append ? rotary_kernel<T, D, V, IL, true> : rotary_kernel<T, D, V, IL, false>;
  return launch_dependent("rotary kernel launch", kern, static_cast<unsigned>(grid), kThreads, 0, stream, a, tok, tokens);
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
