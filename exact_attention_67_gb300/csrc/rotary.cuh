// rotary.cuh -- what the kernels that turn heads to their positions share (rotary.cu,
// norm_rotary.cu): the deal of tokens and heads to threads, the place of a token, its
// angles.
#pragma once
#include "paged.cuh"
#include "ptx.cuh"

namespace exattn {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryTokens = 8;  // tokens a block at most
static_assert(kRotaryTokens <= kRotaryThreads / 32, "a warp looks up each token");

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

// Where token t (packed row, or row of [B, N]) stands, found by a whole warp.
template <bool APPEND>
__device__ __forceinline__ Token find_token(const RotaryArgs& a, const Deal& deal, unsigned t, int lane) {
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
  return k;
}

// Shared memory of a block's angles: cos and sin by token, each token's in the order
// of angle_at.
template <int D>
struct AngleTable {
  alignas(16) float cos[kRotaryTokens * (D / 2)], sin[kRotaryTokens * (D / 2)];
  unsigned long long turns[D / 2];
  float factor[D / 2];  // of a pair's cos and sin: NaN where its frequency is not finite
};

// Place of value f (of D / 2): runs of Q values of neighbouring items side by side, so
// that the items' vector loads meet no bank twice.
template <int D, int V>
__device__ __forceinline__ int angle_at(int f) {
  constexpr int S = D / (2 * V), Q = V < 4 ? V : 4;
  return f % V / Q * (S * Q) + f / V * Q + f % Q;
}

// V values of item `slot` from `table` (a token's, in the order of angle_at).
template <int D, int V>
__device__ __forceinline__ void angle_load(const float* table, int slot, float (&out)[V]) {
  constexpr int S = D / (2 * V), Q = V < 4 ? V : 4;
#pragma unroll
  for (int i = 0; i < V / Q; ++i) {
    const Angles<Q> x = *reinterpret_cast<const Angles<Q>*>(&table[i * (S * Q) + slot * Q]);
#pragma unroll
    for (int j = 0; j < Q; ++j) out[i * Q + j] = x.a[j];
  }
}

// Frequencies, by the whole block; a barrier goes between this and form_angles.
template <int D>
__device__ __forceinline__ void read_frequencies(const RotaryArgs& a, int half, AngleTable<D>& s) {
  for (int f = threadIdx.x; f < half; f += kRotaryThreads) {
    const double freq = a.inv_freq[f];
    s.turns[f] = turns_of(freq);
    s.factor[f] = isfinite(freq) ? a.factor : __int_as_float(0x7fffffff);
  }
}

// cos and sin of nt tokens' angles, by the whole block, value f of token t to place(t, f).
template <int D, typename Place>
__device__ __forceinline__ void form_angles(const RotaryArgs& a, int half, int nt, const Token* tk, AngleTable<D>& s,
                                            const Place& place) {
  for (int i = threadIdx.x; i < nt * (D / 2); i += kRotaryThreads) {
    const int t = i / (D / 2), f = i % (D / 2);  // idle threads cost less than a division
    if (f >= half) continue;
    const unsigned long long angle = static_cast<unsigned long long>(static_cast<long long>(tk[t].pos)) * s.turns[f];
    float sn, c;
    sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 4.656612873077393e-10f, &sn, &c);  // 2^-31: half turns
    const int at = place(t, f);
    s.cos[at] = c * s.factor[f];
    s.sin[at] = (a.inverse ? -sn : sn) * s.factor[f];
  }
}
template <int D, int V>
__device__ __forceinline__ void form_angles(const RotaryArgs& a, int half, int nt, const Token* tk, AngleTable<D>& s) {
  form_angles<D>(a, half, nt, tk, s, [](int t, int f) { return t * (D / 2) + angle_at<D, V>(f); });
}

}  // namespace exattn
