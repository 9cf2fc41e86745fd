// norm_rotary.cu -- the norm of each head of queries and keys with the rotary turn in
// one pass, its gradient, and the same on the way into a paged cache, for sm_103a.
//
// A row x (a token's head of d elements) becomes
//     y = m R(p) (g x / s),   s = sqrt(mean x^2 + eps),
// with the gains g of d elements (one vector for all heads of Q, one for K), the turn
// R(p) of the first `rot` elements as in rotary.cu and the caller's factor m.
// Gradient: with h = m R(p)^T dy, e = x / s and u = g h,
//     dg = sum over rows of h e,      dx = (u - e mean(u e)) / s.
// s is formed again from x, which the gradient reads anyway: nothing is kept between
// the passes.  Sums, statistics and products are fp32, rounded once, to the output's
// type.
//
// The lanes that hold a row's items (rotary.cuh: 2 V elements each) add its squares up
// by exchanges; everything else stays in a thread.  Items arrive by asynchronous copies
// into shared memory (Feed), asked for before the block looks up its tokens and forms
// their angles; 1 / s, the last thing to be known, is applied behind the turn.  The
// gradient's blocks run through token groups, a thread summing h e of its places over the
// heads of Q in registers, then of K, and at the end the block's threads in order; the
// blocks' sums go to the workspace and a second kernel adds them up.  No atomics: results
// do not vary from run to run.
//
// Bound by memory traffic and, nearly as much, by instructions (67 % of the issue slots
// in the forward, 55 in the gradient): 8,192 tokens of 32 + 8 heads of 128, head-major, bf16,
// 29.7 us (5.6 TB/s), the gradient 50.9 (4.9 TB/s); 16,380 tokens of 32 + 8 heads of 64,
// token-major, f16, half turned in pairs, 30.5 and 50.2; 9,837 tokens of 32 + 4 + 4 heads of 64
// into the cache 22.6 (4.5 TB/s).  A token of each of 64 sequences into the cache, a launch
// and a chain of loads, 3.9.  With items in registers, one ahead, these were 34.7, 67.3,
// 34.2, 67.3 and 27.7; three to five items on their way instead of two 30.2 to 33.5; four or
// six blocks an SM instead of five 29.7 and 33.5; blocks that run through groups in the
// forward too 38.5.
#include "rotary.cuh"

#include <limits.h>

#include <algorithm>

namespace exattn {

namespace {

// Blocks an SM, and items of a thread on their way (Feed).
constexpr int kNormBlocks = 5, kNormDepth = 2, kNormGradBlocks = kNormParts / 152, kNormGradDepth = 2;

template <int D, int V>
struct NormCfg {
  static constexpr int S = D / (2 * V);          // items a head
  static constexpr int K = S > 32 ? S / 32 : 1;  // of a thread: a head's lanes are of one warp
  static constexpr int SL = S / K;               // lanes a head
  static constexpr int ROWS = kRotaryThreads / SL;
  static constexpr int W = Item<V>::W;
};

// Gains in shared memory by tensor and half of an item, each in the order of angle_at.
template <int D>
struct GainTable {
  alignas(16) float g[2][2][D / 2];
};

// First elements of an item's two vectors (as in rotary.cu).
template <int V, bool IL>
__device__ __forceinline__ int first_of(int item, int half) {
  return !IL && item * V < half ? item * V : 2 * item * V;
}
template <int V, bool IL>
__device__ __forceinline__ int second_of(int item, int half) {
  return !IL && item * V < half ? item * V + half : 2 * item * V + V;
}

__device__ __forceinline__ float gain_of(const void* g, int dtype, int i) {
  if (!g) return 1.f;
  if (dtype == kF32) return static_cast<const float*>(g)[i];
  if (dtype == kF16) return __half2float(static_cast<const __half*>(g)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(g)[i]);
}

template <int D, int V, bool IL>
__device__ __forceinline__ void read_gains(const NormArgs& a, int half, GainTable<D>& s) {
  for (int i = threadIdx.x; i < 2 * D; i += kRotaryThreads) {
    const int which = i / D, part = i / (D / 2) & 1, f = i % (D / 2), item = f / V;
    const int e = (part ? second_of<V, IL>(item, half) : first_of<V, IL>(item, half)) + f % V;
    s.g[which][part][angle_at<D, V>(f)] = gain_of(which ? a.k_gain : a.q_gain, a.gain_dtype, e);
  }
}

// V values of a table as pairs (V = 1: the second of the pair 0).
template <int D, int V>
__device__ __forceinline__ void pairs_load(const float* table, int item, float2 (&out)[Item<V>::W]) {
  float x[V];
  angle_load<D, V>(table, item, x);
#pragma unroll
  for (int i = 0; i < Item<V>::W; ++i) out[i] = make_float2(x[V > 1 ? 2 * i : 0], V > 1 ? x[(2 * i + 1) % V] : 0.f);
}

// An item's values turned: pairs are (x1, x2) of the same place or, interleaved, the
// two of a word.
template <int D, int V, bool IL>
__device__ __forceinline__ void turn(const float* cos, const float* sin, int item, float2 (&x1)[Item<V>::W],
                                     float2 (&x2)[Item<V>::W]) {
  constexpr int W = Item<V>::W;
  if constexpr (!IL || V == 1) {
    float2 c[W], s[W];
    pairs_load<D, V>(cos, item, c);
    pairs_load<D, V>(sin, item, s);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 y1 = ffma2(fmul2(x2[i], make_float2(-1.f, -1.f)), s[i], fmul2(x1[i], c[i]));
      x2[i] = ffma2(x1[i], s[i], fmul2(x2[i], c[i]));
      x1[i] = y1;
    }
  } else {
    float c[V], s[V];
    angle_load<D, V>(cos, item, c);
    angle_load<D, V>(sin, item, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float2& z = i < W ? x1[i] : x2[i - W];
      z = ffma2(make_float2(z.y, z.x), make_float2(-s[i], s[i]), fmul2(z, make_float2(c[i], c[i])));
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void unpack_item(const Item<V>& x, float2 (&x1)[Item<V>::W], float2 (&x2)[Item<V>::W]) {
#pragma unroll
  for (int i = 0; i < Item<V>::W; ++i) {
    x1[i] = Elem<T>::unpack(x.p1.w[i]);
    x2[i] = Elem<T>::unpack(x.p2.w[i]);
  }
}

// Sum over the SL lanes of a head, the same in each.
template <int SL>
__device__ __forceinline__ float head_sum(float x, unsigned mask) {
#pragma unroll
  for (int o = SL / 2; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
  return x;
}

// This thread's part of a block: items item(0..K-1) of the heads hl, hl + HL, ... of
// token t of the group.  Of the tokens and heads of a block, neighbouring threads take
// those that lie side by side.
template <int D, int V>
struct Part {
  int slot, t, hl, HL;
  unsigned mask;  // the head's lanes
  __device__ explicit Part(const Deal& deal) {
    using C = NormCfg<D, V>;
    const int tid = threadIdx.x, lane = tid & 31, r = tid / C::SL;
    HL = C::ROWS >> deal.tok_shift;
    slot = tid % C::SL;
    t = deal.head_major ? r & ((1 << deal.tok_shift) - 1) : r / HL;
    hl = deal.head_major ? r >> deal.tok_shift : r & (HL - 1);
    mask = C::SL == 32 ? ~0u : ((1u << C::SL) - 1) << (lane & ~(C::SL - 1));
  }
  __device__ int item(int k) const { return slot + k * NormCfg<D, V>::SL; }
};

// The items that a thread is about to work on, DEPTH of N tensors' each, on their way in
// shared memory: asynchronous copies, so that they hold no registers and are under way
// while the block looks up its tokens and forms their angles.  A thread reads what it has
// itself asked for: no barriers.
template <int V, int K, int N, int DEPTH>
struct Feed {
  using VT = typename Vec<V>::type;
  VT data[DEPTH][N][K][2][kRotaryThreads];

  // Item k's halves of tensor n, from `a` and `b`, into slot s.  `spread`: the lanes' halves
  // lie side by side; else an item's two do, and the second finds its 32-byte sector in L1
  // (through L2 alone 38.7 us instead of 30.5 for 16,380 tokens of 40 heads of 64).
  __device__ __forceinline__ void ask(int s, int n, int k, const void* a, const void* b, bool spread) {
    const void* from[2] = {a, b};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      VT* to = &data[s][n][k][i][threadIdx.x];
      if (V == 8 && spread) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from[i]) : "memory");
      } else if constexpr (V >= 2) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from[i]), "n"(2 * V)
                     : "memory");
      } else {
        *to = *static_cast<const VT*>(from[i]);  // two bytes: too few for a copy
      }
    }
  }
  __device__ __forceinline__ static void asked() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // The oldest but DEPTH - 1 of the groups asked for.
  __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
  __device__ __forceinline__ void read(int s, int n, Item<V> (&x)[K]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k].p1.v = data[s][n][k][0][threadIdx.x];
      x[k].p2.v = data[s][n][k][1][threadIdx.x];
    }
  }
};

template <int D, int V>
struct NormGradShared {
  alignas(16) Feed<V, NormCfg<D, V>::K, 2, kNormGradDepth> feed;
  AngleTable<D> angles;
  GainTable<D> gains;
  Token tk[kRotaryTokens];
  float sums[2][NormCfg<D, V>::K][2][V][kRotaryThreads];  // h e by tensor, item, half, place and thread
};

template <typename T, int D, int V, bool IL, bool APPEND>
__global__ void __launch_bounds__(kRotaryThreads, kNormBlocks) norm_rotary_kernel(const __grid_constant__ NormArgs na,
                                                                                 const __grid_constant__ Deal deal) {
  using C = NormCfg<D, V>;
  using VT = typename Vec<V>::type;
  constexpr int K = C::K, W = C::W, DEPTH = kNormDepth;
  __shared__ AngleTable<D> angles;
  __shared__ GainTable<D> gains;
  __shared__ Token tk[kRotaryTokens];
  __shared__ alignas(16) Feed<V, K, 1, DEPTH> feed;
  const RotaryArgs& a = na.r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned t0 = blockIdx.x << deal.tok_shift;
  const int nt = static_cast<int>(min(1u << deal.tok_shift, deal.rows - t0));
  const int half = a.inv_freq ? a.rot >> 1 : 0;
  const int heads = a.Hq + a.Hk + (APPEND ? a.Hk : 0);
  const Part<D, V> p(deal);
  const int t = p.t;
  const bool live = t < nt;
  const unsigned row = t0 + (live ? t : 0), b = APPEND ? 0 : deal.length(row);
  const unsigned n = APPEND ? row : row - b * deal.length.d;
  auto at = [&](const Strides& st) { return (APPEND ? 0 : b * st.b) + n * st.n; };
  const int hk = a.Hq, hv = APPEND ? a.Hq + a.Hk : INT_MAX;
  const bool spread = !IL && 2 * half == D;
  auto ask = [&](int h, int s) {
    if (live && h < heads) {
      const T* src;
      if (h < hk) src = static_cast<const T*>(a.q) + at(a.sq) + h * a.sq.h;
      else if (h < hv) src = static_cast<const T*>(a.k) + at(a.sk) + (h - hk) * a.sk.h;
      else src = static_cast<const T*>(a.v) + at(a.sv) + (h - hv) * a.sv.h;
#pragma unroll
      for (int k = 0; k < K; ++k) feed.ask(s, 0, k, src + first_of<V, IL>(p.item(k), half), src + second_of<V, IL>(p.item(k), half), spread);
    }
    feed.asked();
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) ask(p.hl + i * p.HL, i);
  read_frequencies<D>(a, half, angles);
  read_gains<D, V, IL>(na, half, gains);
  if (warp < nt) {
    const Token k = find_token<APPEND>(a, deal, t0 + warp, lane);
    if (lane == 0) tk[warp] = k;
  }
  __syncthreads();
  form_angles<D, V>(a, half, nt, tk, angles);
  __syncthreads();
  if (!live) return;
  const int flags = APPEND ? tk[t].flags : 3;
  int s = 0;
  for (int h = p.hl; h < heads; h += p.HL) {
    Item<V> x[K];
    feed.wait();
    feed.read(s, 0, x);
    if (h < hv) {
      float2 x1[K][W], x2[K][W], sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        unpack_item<T, V>(x[k], x1[k], x2[k]);
#pragma unroll
        for (int i = 0; i < W; ++i) sum = ffma2(x1[k][i], x1[k][i], ffma2(x2[k][i], x2[k][i], sum));
      }
      const float r = rsqrtf(fmaf(head_sum<C::SL>(sum.x + sum.y, p.mask), 1.f / D, na.eps));
      const float2 rr = make_float2(r, r);
      const float(*g)[D / 2] = gains.g[h < hk ? 0 : 1];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int item = p.item(k);
        float2 w[W];
        pairs_load<D, V>(g[0], item, w);
#pragma unroll
        for (int i = 0; i < W; ++i) x1[k][i] = fmul2(x1[k][i], w[i]);
        pairs_load<D, V>(g[1], item, w);
#pragma unroll
        for (int i = 0; i < W; ++i) x2[k][i] = fmul2(x2[k][i], w[i]);
        if (item * V < half) turn<D, V, IL>(angles.cos + t * (D / 2), angles.sin + t * (D / 2), item, x1[k], x2[k]);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float2 y1 = fmul2(x1[k][i], rr), y2 = fmul2(x2[k][i], rr);
          x[k].p1.w[i] = Elem<T>::pack(y1.x, y1.y);
          x[k].p2.w[i] = Elem<T>::pack(y2.x, y2.y);
        }
      }
    }
    T* dst;
    if (h < hk) dst = static_cast<T*>(a.q_out) + at(a.sqo) + h * a.sqo.h;
    else if (!APPEND) dst = static_cast<T*>(a.k_out) + at(a.sko) + (h - hk) * a.sko.h;
    else if (h < hv) dst = static_cast<T*>(a.k_out) + tk[t].k + (h - hk) * a.sko.h;
    else dst = static_cast<T*>(a.v_out) + tk[t].v + (h - hv) * a.svo.h;
    if (flags & (h < hk ? 1 : 2)) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        *reinterpret_cast<VT*>(dst + first_of<V, IL>(p.item(k), half)) = x[k].p1.v;
        *reinterpret_cast<VT*>(dst + second_of<V, IL>(p.item(k), half)) = x[k].p2.v;
      }
    }
    ask(h + DEPTH * p.HL, s);
    s = s + 1 == DEPTH ? 0 : s + 1;
  }
}

// The gradient.  A block takes the token groups blockIdx.x, + gridDim.x, ...; a thread sums
// h e of its places over its heads of Q, then of K, in registers, and over the token groups
// in shared memory.
template <typename T, int D, int V, bool IL>
__global__ void __launch_bounds__(kRotaryThreads, kNormGradBlocks) norm_rotary_grad_kernel(const __grid_constant__ NormArgs na,
                                                                                          const __grid_constant__ Deal deal) {
  using C = NormCfg<D, V>;
  using VT = typename Vec<V>::type;
  constexpr int K = C::K, W = C::W, DEPTH = kNormGradDepth;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  NormGradShared<D, V>& sm = *reinterpret_cast<NormGradShared<D, V>*>(smem_raw);
  auto& feed = sm.feed;
  const RotaryArgs& a = na.r;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int half = a.rot >> 1, heads = a.Hq + a.Hk, hk = a.Hq;
  const Part<D, V> p(deal);
  const int t = p.t;
  const bool spread = !IL && 2 * half == D;
  // A group's tokens are looked up while the group before is worked on.
  auto look_up = [&](unsigned t0) {
    const unsigned tok = t0 + warp;
    return tok < deal.rows && warp < 1 << deal.tok_shift ? find_token<false>(a, deal, tok, lane) : Token{};
  };
  Token next = look_up(blockIdx.x << deal.tok_shift);
#pragma unroll
  for (int i = 0; i < 4 * K * V; ++i) (&sm.sums[0][0][0][0][0])[i * kRotaryThreads + tid] = 0.f;
  bool first = true;
  for (unsigned t0 = blockIdx.x << deal.tok_shift; t0 < deal.rows; t0 += gridDim.x << deal.tok_shift) {
    const int nt = static_cast<int>(min(1u << deal.tok_shift, deal.rows - t0));
    const bool live = t < nt;
    const unsigned row = t0 + (live ? t : 0), b = deal.length(row), n = row - b * deal.length.d;
    auto at = [&](const Strides& st) { return b * st.b + n * st.n; };
    auto ask = [&](int h, int s) {
      if (live && h < heads) {
        const bool q = h < hk;
        const T* xs = static_cast<const T*>(q ? a.q : a.k) + at(q ? a.sq : a.sk) + (q ? h * a.sq.h : (h - hk) * a.sk.h);
        const T* gs = static_cast<const T*>(q ? na.dq : na.dk) + at(q ? na.sdq : na.sdk) + (q ? h * na.sdq.h : (h - hk) * na.sdk.h);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int e1 = first_of<V, IL>(p.item(k), half), e2 = second_of<V, IL>(p.item(k), half);
          feed.ask(s, 0, k, xs + e1, xs + e2, spread);
          feed.ask(s, 1, k, gs + e1, gs + e2, spread);
        }
      }
      feed.asked();
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) ask(p.hl + i * p.HL, i);
    if (first) {
      read_frequencies<D>(a, half, sm.angles);
      read_gains<D, V, IL>(na, half, sm.gains);
      first = false;
    } else {
      __syncthreads();  // the last group's angles are used up
    }
    if (warp < nt && lane == 0) sm.tk[warp] = next;
    __syncthreads();
    next = look_up(t0 + (gridDim.x << deal.tok_shift));
    form_angles<D, V>(a, half, nt, sm.tk, sm.angles);
    __syncthreads();
    if (!live) continue;
    float2 s1[K][W], s2[K][W];  // this thread's sums of h e for one tensor
    int which = p.hl < hk ? 0 : 1, s = 0;
    auto clear = [&]() {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) s1[k][i] = s2[k][i] = make_float2(0.f, 0.f);
    };
    auto flush = [&]() {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sm.sums[which][k][0][i][tid] += i & 1 ? s1[k][i / 2].y : s1[k][i / 2].x;
          sm.sums[which][k][1][i][tid] += i & 1 ? s2[k][i / 2].y : s2[k][i / 2].x;
        }
    };
    clear();
    for (int h = p.hl; h < heads; h += p.HL) {
      if (which == 0 && h >= hk) {
        flush();
        clear();
        which = 1;
      }
      Item<V> x[K], g[K];
      feed.wait();
      feed.read(s, 0, x);
      feed.read(s, 1, g);
      float2 x1[K][W], x2[K][W], h1[K][W], h2[K][W], sq = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
      const float(*gain)[D / 2] = sm.gains.g[which];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int item = p.item(k);
        unpack_item<T, V>(x[k], x1[k], x2[k]);
        unpack_item<T, V>(g[k], h1[k], h2[k]);
        if (item * V < half) turn<D, V, IL>(sm.angles.cos + t * (D / 2), sm.angles.sin + t * (D / 2), item, h1[k], h2[k]);
        float2 w[W];
        pairs_load<D, V>(gain[0], item, w);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          sq = ffma2(x1[k][i], x1[k][i], sq);
          dot = ffma2(fmul2(h1[k][i], w[i]), x1[k][i], dot);
        }
        pairs_load<D, V>(gain[1], item, w);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          sq = ffma2(x2[k][i], x2[k][i], sq);
          dot = ffma2(fmul2(h2[k][i], w[i]), x2[k][i], dot);
        }
      }
      const float r = rsqrtf(fmaf(head_sum<C::SL>(sq.x + sq.y, p.mask), 1.f / D, na.eps));
      const float mean = head_sum<C::SL>(dot.x + dot.y, p.mask) * r * (1.f / D);  // of g h e
      const float2 rr = make_float2(r, r), mm = make_float2(-mean, -mean);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float2 w[W];
        pairs_load<D, V>(gain[0], p.item(k), w);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float2 e = fmul2(x1[k][i], rr);
          s1[k][i] = ffma2(h1[k][i], e, s1[k][i]);
          const float2 dx = fmul2(ffma2(e, mm, fmul2(h1[k][i], w[i])), rr);
          x[k].p1.w[i] = Elem<T>::pack(dx.x, dx.y);
        }
        pairs_load<D, V>(gain[1], p.item(k), w);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float2 e = fmul2(x2[k][i], rr);
          s2[k][i] = ffma2(h2[k][i], e, s2[k][i]);
          const float2 dx = fmul2(ffma2(e, mm, fmul2(h2[k][i], w[i])), rr);
          x[k].p2.w[i] = Elem<T>::pack(dx.x, dx.y);
        }
      }
      T* dst = h < hk ? static_cast<T*>(a.q_out) + at(a.sqo) + h * a.sqo.h
                      : static_cast<T*>(a.k_out) + at(a.sko) + (h - hk) * a.sko.h;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        *reinterpret_cast<VT*>(dst + first_of<V, IL>(p.item(k), half)) = x[k].p1.v;
        *reinterpret_cast<VT*>(dst + second_of<V, IL>(p.item(k), half)) = x[k].p2.v;
      }
      ask(h + DEPTH * p.HL, s);
      s = s + 1 == DEPTH ? 0 : s + 1;
    }
    flush();
  }
  __syncthreads();
  // The block's sums, a value a thread, its rows in order.
  for (int i = tid; i < 2 * D; i += kRotaryThreads) {
    const int which = i / D, part = i / (D / 2) & 1, j = i % (D / 2) / C::S, item = i % C::S;
    const float* from = sm.sums[which][item / C::SL][part][j] + item % C::SL;
    float sum = 0.f;
#pragma unroll 8
    for (int r = 0; r < C::ROWS; ++r) sum += from[r * C::SL];
    const int e = (part ? second_of<V, IL>(item, half) : first_of<V, IL>(item, half)) + j;
    na.partial[static_cast<long long>(blockIdx.x) * 2 * D + which * D + e] = sum;
  }
}

// Gains' gradients: the blocks' sums added up, 32 columns a block, a warp every 32nd row
// (all of a lane's loads at once: the rows are in L2, so that what counts is how often it
// waits), then the warps in order.
template <int D>
__global__ void __launch_bounds__(1024) norm_gains_kernel(const __grid_constant__ NormArgs a) {
  constexpr int LOADS = (kNormParts + 31) / 32;
  __shared__ float s[32][33];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float x[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = run + 32 * i;
    x[i] = r < a.parts ? a.partial[static_cast<long long>(r) * 2 * D + col] : 0.f;
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < LOADS; ++i) sum += x[i];
  s[run][lane] = sum;
  __syncthreads();
  if (run) return;
  sum = 0.f;
#pragma unroll
  for (int r = 0; r < 32; ++r) sum += s[r][lane];
  void* out = col < D ? a.q_dgain : a.k_dgain;
  const int i = col % D;
  if (!out) return;
  if (a.gain_dtype == kF32) static_cast<float*>(out)[i] = sum;
  else if (a.gain_dtype == kF16) static_cast<__half*>(out)[i] = __float2half_rn(sum);
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(sum);
}

template <typename T, int D, int V, bool IL>
cudaError_t launch_t(const NormArgs& na, cudaStream_t stream) {
  const RotaryArgs& a = na.r;
  using C = NormCfg<D, V>;
  Deal deal{};
  deal.rows = a.append ? a.nt.total : static_cast<unsigned>(a.B) * a.N;
  if (!na.partial) {
    // Several tokens a block (a power of two) once that still leaves eight blocks an SM:
    // 8,192 tokens of 40 heads of 128 with four 29.5 us, two 33, eight (four blocks) 31.1.
    while ((1 << deal.tok_shift) < std::min(kRotaryTokens, C::ROWS) && deal.rows >> (deal.tok_shift + 1) >= 152 * 8)
      ++deal.tok_shift;
  } else {
    // As many as take the least time, in items of a thread, each group costing two more.
    long long best = LLONG_MAX;
    for (int shift = 0; 1 << shift <= std::min(kRotaryTokens, C::ROWS); ++shift) {
      const long long groups = (deal.rows + (1ll << shift) - 1) >> shift;
      const long long items = ((static_cast<long long>(a.Hq + a.Hk) << shift) + C::ROWS - 1) / C::ROWS;
      const long long time = (groups + kNormParts - 1) / kNormParts * (items + 2);
      if (time < best) {
        best = time;
        deal.tok_shift = shift;
      }
    }
  }
  deal.head_major = a.Hq > 0 ? a.sq.n < a.sq.h : a.sk.n < a.sk.h;
  deal.length = Divide(!a.append ? a.N : a.nt.each > 0 ? a.nt.each : 1);
  const unsigned groups = (deal.rows + (1u << deal.tok_shift) - 1) >> deal.tok_shift;
  if (!na.partial) {
    auto kern = a.append ? norm_rotary_kernel<T, D, V, IL, true> : norm_rotary_kernel<T, D, V, IL, false>;
    return launch_dependent("norm kernel launch", kern, groups, kRotaryThreads, 0, stream, na, deal);
  }
  NormArgs g = na;
  g.parts = static_cast<int>(std::min<unsigned>(groups, kNormParts));
  auto grad = norm_rotary_grad_kernel<T, D, V, IL>;
  constexpr int smem = sizeof(NormGradShared<D, V>);
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(grad), smem, na.device);
  if (e != cudaSuccess) return e;
  e = launch_dependent("norm gradient kernel launch", grad, g.parts, kRotaryThreads, smem, stream, g, deal);
  if (e != cudaSuccess || (!g.q_dgain && !g.k_dgain)) return e;
  return launch_dependent("gains' gradient kernel launch", norm_gains_kernel<D>, 2 * D / 32, 1024, 0, stream, g);
}

template <typename T, int D>
cudaError_t launch_d(const NormArgs& a, cudaStream_t stream) {
  const int rot = a.r.inv_freq ? a.r.rot : D;
  const int v = rot % 16 == 0 ? 8 : rot % 8 == 0 ? 4 : rot % 4 == 0 ? 2 : 1;
  if (a.r.interleaved) {
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

cudaError_t launch_norm_rotary(const NormArgs& a, cudaStream_t stream) {
  if (a.r.dtype == kF16) return a.r.d == 64 ? launch_d<__half, 64>(a, stream) : launch_d<__half, 128>(a, stream);
  return a.r.d == 64 ? launch_d<__nv_bfloat16, 64>(a, stream) : launch_d<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
