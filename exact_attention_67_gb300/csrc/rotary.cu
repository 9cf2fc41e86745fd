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
// rot / 2 angles once, in shared memory, for all heads of Q and K; then
// each thread turns items of 2 V elements (two 16-byte vectors at V = 8), four
// items in flight.  Bound by memory traffic: every element is read once and
// written once.  V is the widest vector that divides rot / 2 (interleaved: half
// of an item's run), so rot a multiple of 16 moves 16-byte vectors.
#include "paged.cuh"
#include "ptx.cuh"

namespace exattn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;  // tokens a block at most

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

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

// V elements of one type in registers.
template <typename T, int V>
union Pack {
  typename Vec<V>::type v;
  T e[V];
  __device__ Pack() {}
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
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a, int tok_per_block,
                                                          long long tokens, unsigned head_magic) {
  constexpr int S = D / (2 * V);  // items a head
  __shared__ float2 cs[kMaxTok * (D / 2)];
  __shared__ Token tk[kMaxTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const int half = a.inv_freq ? a.rot >> 1 : 0;
  for (int x = tid; x < nt * half; x += kThreads) {
    const int t = x / half, f = x - t * half;
    double turns = a.inv_freq[f] * 0.15915494309189535;  // 1 / 2 pi
    turns -= floor(turns);
    const unsigned long long F = __double2ull_rn(turns * 18446744073709551616.0);
    const unsigned long long angle = static_cast<unsigned long long>(static_cast<long long>(tk[t].pos)) * F;
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    cs[t * (D / 2) + f] = make_float2(c * a.factor, (a.inverse ? -s : s) * a.factor);
  }
  __syncthreads();

  using VT = typename Vec<V>::type;
  const int heads = a.Hq + a.Hk + (APPEND ? a.Hk : 0);
  const int items = nt * heads * S;
  constexpr int U = 4;
  for (int x0 = tid; x0 < items; x0 += U * kThreads) {
    Pack<T, V> p1[U], p2[U];
    T* dst[U];
    int e1[U], e2[U], tok[U];
    bool turn[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = x0 + u * kThreads;
      dst[u] = nullptr;
      if (x >= items) continue;
      const int slot = x % S, row = x / S;
      const int t = static_cast<int>(__umulhi(static_cast<unsigned>(row), head_magic));
      int h = row - t * heads;
      const Token& k = tk[t];
      const T* src;
      turn[u] = true;
      if (h < a.Hq) {
        if (!(k.flags & 1)) continue;
        src = static_cast<const T*>(a.q) + k.q + h * a.sq.h;
        dst[u] = static_cast<T*>(a.q_out) + k.qo + h * a.sqo.h;
      } else {
        if (!(k.flags & 2)) continue;
        h -= a.Hq;
        if (!APPEND || h < a.Hk) {
          src = static_cast<const T*>(a.k) + k.k + h * a.sk.h;
          dst[u] = static_cast<T*>(a.k_out) + k.ko + h * a.sko.h;
        } else {
          h -= a.Hk;
          src = static_cast<const T*>(a.v) + k.v + h * a.sv.h;
          dst[u] = static_cast<T*>(a.v_out) + k.vo + h * a.svo.h;
          turn[u] = false;
        }
      }
      // The item's two vectors: a pair's halves, or (interleaved, and past the
      // turned part) 2 V consecutive elements.
      const int pairs0 = slot * V;
      turn[u] = turn[u] && pairs0 < half;
      e1[u] = !IL && turn[u] ? pairs0 : 2 * pairs0;
      e2[u] = !IL && turn[u] ? pairs0 + half : 2 * pairs0 + V;
      tok[u] = t * (D / 2) + pairs0;
      p1[u].v = *reinterpret_cast<const VT*>(src + e1[u]);
      p2[u].v = *reinterpret_cast<const VT*>(src + e2[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u] == nullptr) continue;
      if (turn[u]) {
        if constexpr (!IL) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 w = cs[tok[u] + e];
            const float x1 = to_f<T>(p1[u].e[e]), x2 = to_f<T>(p2[u].e[e]);
            p1[u].e[e] = from_f<T>(x1 * w.x - x2 * w.y);
            p2[u].e[e] = from_f<T>(x2 * w.x + x1 * w.y);
          }
        } else {
          T e[2 * V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            e[i] = p1[u].e[i];
            e[V + i] = p2[u].e[i];
          }
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 w = cs[tok[u] + i];
            const float x1 = to_f<T>(e[2 * i]), x2 = to_f<T>(e[2 * i + 1]);
            e[2 * i] = from_f<T>(x1 * w.x - x2 * w.y);
            e[2 * i + 1] = from_f<T>(x2 * w.x + x1 * w.y);
          }
#pragma unroll
          for (int i = 0; i < V; ++i) {
            p1[u].e[i] = e[i];
            p2[u].e[i] = e[V + i];
          }
        }
      }
      *reinterpret_cast<VT*>(dst[u] + e1[u]) = p1[u].v;
      *reinterpret_cast<VT*>(dst[u] + e2[u]) = p2[u].v;
    }
  }
}

template <typename T, int D, int V, bool IL>
cudaError_t launch_t(const RotaryArgs& a, cudaStream_t stream) {
  const long long tokens = a.append ? a.nt.total : static_cast<long long>(a.B) * a.N;
  const int heads = a.Hq + a.Hk + (a.append ? a.Hk : 0);
  // Several tokens a block once that still leaves eight blocks an SM.
  int tok = 1;
  while (tok < kMaxTok && tokens / (2 * tok) >= 152 * 8) tok *= 2;
  const long long grid = (tokens + tok - 1) / tok;
  const unsigned magic = static_cast<unsigned>(((1ull << 32) + heads - 1) / heads);
  auto kern = a.append ? rotary_kernel<T, D, V, IL, true> : rotary_kernel<T, D, V, IL, false>;
  kern<<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a, tok, tokens, magic);
  return note_cuda(cudaGetLastError(), "rotary kernel launch");
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
