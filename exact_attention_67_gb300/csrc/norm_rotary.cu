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
// type; a row whose squares would leave fp32's range is scaled by a power of two first
// (scale_far: a branch that is not taken as a rule).
//
// A lane holds an item of a row, two vectors of 8 elements, whatever part of the head is
// turned: its pairs' halves (`rot` a multiple of 16), or 16 consecutive elements, whose
// pairs are its own (interleaved) or go through shared memory (Turn).  The row's lanes
// add its squares up by exchanges.  Items arrive by asynchronous copies
// into shared memory (Feed), asked for before the block looks up its tokens and forms
// their angles; 1 / s, the last thing to be known, is applied behind the turn.  The
// gradient's blocks run through token groups, a thread summing h e of its places over the
// heads of Q in registers, then of K, and at the end the block's threads in order; the
// blocks' sums go to the workspace and a second kernel adds them up.  No atomics: results
// do not vary from run to run.
//
// Bound by memory traffic and, nearly as much, by instructions (71 % of the issue slots
// in the forward, 56 in the gradient, whose blocks also take their token groups in rounds,
// the last one filled in part, and let their items run out at each group's end): 8,192 tokens of 32 + 8 heads of 128, head-major, bf16,
// 29.9 us (5.6 TB/s), the gradient 51.6 (4.9 TB/s); interleaved, whatever part is turned, 34.5
// and 54.5 to 57 (a lane's two vectors side by side); 20 or 6 of 128 elements turned as halves
// 37.9 and 36.0, 62.7 and 58.8.  16,380 tokens of 32 + 8 heads of 64, token-major, f16, half
// turned in pairs, 31.3 and 50.9; 9,837 tokens of 32 + 4 + 4 heads of 64 into the cache 22.4 (4.5
// TB/s; without a turn 21.6, the turn without the norms 21.4): 1,230 blocks on 760 places, whose
// second round is thin.  A token of each of 64 sequences into the cache, a launch and a chain of
// loads, 3.8.
// With items in registers, one ahead, the first were 34.7 and 67.3; three to five items on
// their way instead of two 30.2 to 33.5; blocks that run through groups in the forward too
// 38.5; narrower vectors for other turned parts (4 bytes for 20, 2 for 6) 45.4 and 69.3,
// their gradients 113.6 and 167.3.
#include "rotary.cuh"

#include <limits.h>

#include <algorithm>

namespace exattn {

namespace {

// Items of a thread on their way (Feed), and the gradient's blocks an SM.
constexpr int kNormDepth = 2, kNormGradDepth = 2, kNormGradBlocks = kNormParts / 152;

// Where a head's pairs are.
enum Turn : int {
  kHalves,    // (i, i + rot / 2), rot / 2 a multiple of 8: a lane's two vectors are its pairs' halves
  kPairs,     // (2 i, 2 i + 1)
  kAnywhere,  // (i, i + rot / 2): exchanged in shared memory
};

// The forward's blocks an SM: five where that spills next to nothing (four 30.8 us instead of
// 29.7 for 8,192 tokens of 40 heads of 128), else four (five 35.6 and 42.0 instead of 33.7 and
// 36.9, in pairs and with 20 elements turned).
__host__ __device__ constexpr int norm_blocks(Turn m) { return m == kHalves ? 5 : 4; }

constexpr int V = 8;  // elements a vector
using Vector = typename Vec<V>::type;
constexpr int W = Item<V>::W;

template <int D>
struct NormCfg {
  static constexpr int S = D / (2 * V);  // lanes a head
  static constexpr int ROWS = kRotaryThreads / S;
};

// Gains in shared memory by tensor and half of an item, each in the order of angle_at.
template <int D>
struct GainTable {
  alignas(16) float g[2][2][D / 2];
};

// A row's elements on the way between their lanes and their pairs, one row a head that the
// block works on; padded so that the rows of a warp meet no bank twice.
template <int D, Turn M>
struct RowTable {
  static constexpr int STRIDE = D + D / 16;
  alignas(16) float x[M == kAnywhere ? NormCfg<D>::ROWS * STRIDE : 4];
};

// First elements of an item's two vectors.
template <Turn M>
__device__ __forceinline__ int first_of(int item, int half) {
  return M == kHalves && item * V < half ? item * V : 2 * item * V;
}
template <Turn M>
__device__ __forceinline__ int second_of(int item, int half) {
  return M == kHalves && item * V < half ? item * V + half : 2 * item * V + V;
}

__device__ __forceinline__ float gain_of(const void* g, int dtype, int i) {
  if (!g) return 1.f;
  if (dtype == kF32) return static_cast<const float*>(g)[i];
  if (dtype == kF16) return __half2float(static_cast<const __half*>(g)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(g)[i]);
}

template <int D, Turn M>
__device__ __forceinline__ void read_gains(const NormArgs& a, int half, GainTable<D>& s) {
  for (int i = threadIdx.x; i < 2 * D; i += kRotaryThreads) {
    const int which = i / D, part = i / (D / 2) & 1, f = i % (D / 2), item = f / V;
    const int e = (part ? second_of<M>(item, half) : first_of<M>(item, half)) + f % V;
    s.g[which][part][angle_at<D, V>(f)] = gain_of(which ? a.k_gain : a.q_gain, a.gain_dtype, e);
  }
}

// An item's V values of a table, as pairs.
template <int D>
__device__ __forceinline__ void pairs_load(const float* table, int item, float2 (&out)[W]) {
  float x[V];
  angle_load<D, V>(table, item, x);
#pragma unroll
  for (int i = 0; i < W; ++i) out[i] = make_float2(x[2 * i], x[2 * i + 1]);
}

// cos and sin in the order in which the turn reads them; pair by pair, a token's begin 8
// banks after the last one's.
template <int D>
__device__ __forceinline__ int pair_at(int t, int f) {
  return t * (D / 2) + ((f + 8 * t) & (D / 2 - 1));
}
template <int D, Turn M>
__device__ __forceinline__ void norm_angles(const RotaryArgs& a, int half, int nt, const Token* tk, AngleTable<D>& s) {
  if constexpr (M == kAnywhere) form_angles<D>(a, half, nt, tk, s, [](int t, int f) { return pair_at<D>(t, f); });
  else form_angles<D, V>(a, half, nt, tk, s);
}

// An item's values turned by the angles of the group's token t; `row`: its head's row of the RowTable,
// `mask` the head's lanes.
template <int D, Turn M>
__device__ __forceinline__ void turn(const AngleTable<D>& angles, int t, float* row, int item, int half, unsigned mask,
                                     float2 (&x1)[W], float2 (&x2)[W]) {
  const float *cos = angles.cos + t * (D / 2), *sin = angles.sin + t * (D / 2);
  if constexpr (M == kHalves) {
    if (item * V >= half) return;
    float2 c[W], s[W];
    pairs_load<D>(cos, item, c);
    pairs_load<D>(sin, item, s);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 y1 = ffma2(fmul2(x2[i], make_float2(-1.f, -1.f)), s[i], fmul2(x1[i], c[i]));
      x2[i] = ffma2(x1[i], s[i], fmul2(x2[i], c[i]));
      x1[i] = y1;
    }
  } else if constexpr (M == kPairs) {
    if (item * V >= half) return;
    float c[V], s[V];
    angle_load<D, V>(cos, item, c);
    angle_load<D, V>(sin, item, s);
    // (Of a pair by scalars: packed, its halves would have to change places.)
    auto turned = [&](int i) {
      const float2 z = i < W ? x1[i] : x2[i - W];
      return make_float2(fmaf(z.x, c[i], -z.y * s[i]), fmaf(z.y, c[i], z.x * s[i]));
    };
    const int last = half - item * V;  // pairs from here on are past the turned part
    if (last >= V) {
#pragma unroll
      for (int i = 0; i < V; ++i) (i < W ? x1[i] : x2[i - W]) = turned(i);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < last) (i < W ? x1[i] : x2[i - W]) = turned(i);
    }
  } else {
    constexpr int S = NormCfg<D>::S;
    const bool mine = 2 * V * item < 2 * half;
    float4* at = reinterpret_cast<float4*>(row + 2 * V * item);
    if (mine) {
#pragma unroll
      for (int i = 0; i < W; i += 2) {
        at[i / 2] = make_float4(x1[i].x, x1[i].y, x1[i + 1].x, x1[i + 1].y);
        at[W / 2 + i / 2] = make_float4(x2[i].x, x2[i].y, x2[i + 1].x, x2[i + 1].y);
      }
    }
    __syncwarp(mask);
    for (int f = item; f < half; f += S) {
      const int at_f = pair_at<D>(t, f);
      const float u = row[f], v = row[f + half], c = angles.cos[at_f], sn = angles.sin[at_f];
      row[f] = u * c - v * sn;
      row[f + half] = v * c + u * sn;
    }
    __syncwarp(mask);
    if (mine) {
#pragma unroll
      for (int i = 0; i < W; i += 2) {
        const float4 a = at[i / 2], b = at[W / 2 + i / 2];
        x1[i] = make_float2(a.x, a.y);
        x1[i + 1] = make_float2(a.z, a.w);
        x2[i] = make_float2(b.x, b.y);
        x2[i + 1] = make_float2(b.z, b.w);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void unpack_item(const Item<V>& x, float2 (&x1)[W], float2 (&x2)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    x1[i] = Elem<T>::unpack(x.p1.w[i]);
    x2[i] = Elem<T>::unpack(x.p2.w[i]);
  }
}

// Sum over the S lanes of a head, the same in each.
template <int S>
__device__ __forceinline__ float head_sum(float x, unsigned mask) {
#pragma unroll
  for (int o = S / 2; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
  return x;
}

// A row whose mean square (+ eps) t is outside this range is far: its squares may have left
// fp32's, or its products with gains would.  (Of f16 rows only those of zeros could be.)
template <typename T>
__device__ __forceinline__ bool far_from_one(float t) {
  return Elem<T>::kFmt != Elem<__half>::kFmt && !(t >= 0x1p-64f && t <= 0x1p64f);
}

// A far row by 2^k, exactly, so that the larger of its greatest element and sqrt(eps) is near 1:
// g x / s stays what it is with eps by 2^2k, and 1 / s is 2^k times the scaled row's, which
// together may be past fp32.  Gives the scaled mean square (+ eps).
// (Rows that are not far pay for the branch: the forward of 8,192 tokens of 40 heads of 128 0.1 us,
// in pairs and by a row in shared memory 0.7 to 1.2, the gradient 0.7 to 2.5.  Forming y of a far
// row once more behind the loop's own 36.9 instead of 30.7, in a function of its own 31.9.)
template <int D>
__device__ __forceinline__ float scale_far(float2 (&x1)[W], float2 (&x2)[W], float eps, unsigned mask, float* scale) {
  constexpr int S = NormCfg<D>::S;
  float m = sqrtf(eps);
#pragma unroll
  for (int i = 0; i < W; ++i)
    m = fmaxf(fmaxf(m, fmaxf(fabsf(x1[i].x), fabsf(x1[i].y))), fmaxf(fabsf(x2[i].x), fabsf(x2[i].y)));
#pragma unroll
  for (int o = S / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
  const float k = __int_as_float(min(max(254 - (__float_as_int(m) >> 23), 1), 253) << 23);  // 2^-126 to 2^126
  const float2 kk = make_float2(k, k);
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    x1[i] = fmul2(x1[i], kk);
    x2[i] = fmul2(x2[i], kk);
    sum = ffma2(x1[i], x1[i], ffma2(x2[i], x2[i], sum));
  }
  *scale = k;
  return fmaf(head_sum<S>(sum.x + sum.y, mask), 1.f / D, eps * k * k);
}

// This thread's part of a block: item `item` of the heads hl, hl + HL, ... of token t of
// the group.  Of the tokens and heads of a block, neighbouring threads take those that lie
// side by side.
template <int D>
struct Part {
  int item, t, hl, HL;
  int row;        // of the block's
  unsigned mask;  // the head's lanes
  __device__ explicit Part(const Deal& deal) {
    using C = NormCfg<D>;
    const int tid = threadIdx.x, lane = tid & 31;
    row = tid / C::S;
    HL = C::ROWS >> deal.tok_shift;
    item = tid % C::S;
    t = deal.head_major ? row & ((1 << deal.tok_shift) - 1) : row / HL;
    hl = deal.head_major ? row >> deal.tok_shift : row & (HL - 1);
    mask = ((1u << C::S) - 1) << (lane & ~(C::S - 1));
  }
};

// The items that a thread is about to work on, DEPTH of N tensors' each, on their way in
// shared memory: asynchronous copies, so that they hold no registers and are under way
// while the block looks up its tokens and forms their angles.  A thread reads what it has
// itself asked for: no barriers.
template <int N, int DEPTH>
struct Feed {
  Vector data[DEPTH][N][2][kRotaryThreads];

  // An item's vectors of tensor n, from `a` and `b`, into slot s.  `spread`: the lanes'
  // vectors lie side by side; else an item's two do, and the second finds its 32-byte sector
  // in L1 (through L2 alone 38.7 us instead of 30.5 for 16,380 tokens of 40 heads of 64).
  __device__ __forceinline__ void ask(int s, int n, const void* a, const void* b, bool spread) {
    const void* from[2] = {a, b};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t to = smem_u32(&data[s][n][i][threadIdx.x]);
      if (spread) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from[i]) : "memory");
      else asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from[i]) : "memory");
    }
  }
  __device__ __forceinline__ static void asked() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // The oldest but DEPTH - 1 of the groups asked for.
  __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
  __device__ __forceinline__ void read(int s, int n, Item<V>& x) const {
    x.p1.v = data[s][n][0][threadIdx.x];
    x.p2.v = data[s][n][1][threadIdx.x];
  }
};

template <int D, Turn M>
struct NormGradShared {
  alignas(16) Feed<2, kNormGradDepth> feed;
  AngleTable<D> angles;
  GainTable<D> gains;
  RowTable<D, M> rows;
  Token tk[kRotaryTokens];
  float sums[2][2][V][kRotaryThreads];  // h e by tensor, half, place and thread
};

template <typename T, int D, Turn M, bool APPEND>
__global__ void __launch_bounds__(kRotaryThreads, norm_blocks(M))
    norm_rotary_kernel(const __grid_constant__ NormArgs na, const __grid_constant__ Deal deal) {
  constexpr int DEPTH = kNormDepth;
  __shared__ AngleTable<D> angles;
  __shared__ GainTable<D> gains;
  __shared__ RowTable<D, M> rows;
  __shared__ Token tk[kRotaryTokens];
  __shared__ alignas(16) Feed<1, DEPTH> feed;
  const RotaryArgs& a = na.r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned t0 = blockIdx.x << deal.tok_shift;
  const int nt = static_cast<int>(min(1u << deal.tok_shift, deal.rows - t0));
  const int half = a.inv_freq ? a.rot >> 1 : 0;
  const int heads = a.Hq + a.Hk + (APPEND ? a.Hk : 0);
  const Part<D> p(deal);
  const int t = p.t, e1 = first_of<M>(p.item, half), e2 = second_of<M>(p.item, half);
  const bool live = t < nt;
  const unsigned row = t0 + (live ? t : 0), b = APPEND ? 0 : deal.length(row);
  const unsigned n = APPEND ? row : row - b * deal.length.d;
  auto at = [&](const Strides& st) { return (APPEND ? 0 : b * st.b) + n * st.n; };
  const int hk = a.Hq, hv = APPEND ? a.Hq + a.Hk : INT_MAX;
  const bool spread = M == kHalves && 2 * half == D;
  auto ask = [&](int h, int s) {
    if (live && h < heads) {
      const T* src;
      if (h < hk) src = static_cast<const T*>(a.q) + at(a.sq) + h * a.sq.h;
      else if (h < hv) src = static_cast<const T*>(a.k) + at(a.sk) + (h - hk) * a.sk.h;
      else src = static_cast<const T*>(a.v) + at(a.sv) + (h - hv) * a.sv.h;
      feed.ask(s, 0, src + e1, src + e2, spread);
    }
    feed.asked();
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) ask(p.hl + i * p.HL, i);
  read_frequencies<D>(a, half, angles);
  read_gains<D, M>(na, half, gains);
  if (warp < nt) {
    const Token k = find_token<APPEND>(a, deal, t0 + warp, lane);
    if (lane == 0) tk[warp] = k;
  }
  __syncthreads();
  norm_angles<D, M>(a, half, nt, tk, angles);
  __syncthreads();
  if (!live) return;
  const int flags = APPEND ? tk[t].flags : 3;
  int s = 0;
  for (int h = p.hl; h < heads; h += p.HL) {
    Item<V> x;
    feed.wait();
    feed.read(s, 0, x);
    if (h < hv) {
      float2 x1[W], x2[W], w[W], sum = make_float2(0.f, 0.f);
      unpack_item<T>(x, x1, x2);
#pragma unroll
      for (int i = 0; i < W; ++i) sum = ffma2(x1[i], x1[i], ffma2(x2[i], x2[i], sum));
      float size = fmaf(head_sum<NormCfg<D>::S>(sum.x + sum.y, p.mask), 1.f / D, na.eps), scale;
      if (far_from_one<T>(size)) size = scale_far<D>(x1, x2, na.eps, p.mask, &scale);
      const float r = rsqrtf(size);
      const float(*g)[D / 2] = gains.g[h < hk ? 0 : 1];
      pairs_load<D>(g[0], p.item, w);
#pragma unroll
      for (int i = 0; i < W; ++i) x1[i] = fmul2(x1[i], w[i]);
      pairs_load<D>(g[1], p.item, w);
#pragma unroll
      for (int i = 0; i < W; ++i) x2[i] = fmul2(x2[i], w[i]);
      turn<D, M>(angles, t, rows.x + p.row * RowTable<D, M>::STRIDE, p.item, half, p.mask, x1, x2);
      const float2 rr = make_float2(r, r);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 y1 = fmul2(x1[i], rr), y2 = fmul2(x2[i], rr);
        x.p1.w[i] = Elem<T>::pack(y1.x, y1.y);
        x.p2.w[i] = Elem<T>::pack(y2.x, y2.y);
      }
    }
    T* dst;
    if (h < hk) dst = static_cast<T*>(a.q_out) + at(a.sqo) + h * a.sqo.h;
    else if (!APPEND) dst = static_cast<T*>(a.k_out) + at(a.sko) + (h - hk) * a.sko.h;
    else if (h < hv) dst = static_cast<T*>(a.k_out) + tk[t].k + (h - hk) * a.sko.h;
    else dst = static_cast<T*>(a.v_out) + tk[t].v + (h - hv) * a.svo.h;
    if (flags & (h < hk ? 1 : 2)) {
      *reinterpret_cast<Vector*>(dst + e1) = x.p1.v;
      *reinterpret_cast<Vector*>(dst + e2) = x.p2.v;
    }
    ask(h + DEPTH * p.HL, s);
    s = s + 1 == DEPTH ? 0 : s + 1;
  }
}

// The gradient.  A block takes the token groups blockIdx.x, + gridDim.x, ...; a thread sums
// h e of its places over its heads of Q, then of K, in registers, and over the token groups
// in shared memory.
template <typename T, int D, Turn M>
__global__ void __launch_bounds__(kRotaryThreads, kNormGradBlocks) norm_rotary_grad_kernel(const __grid_constant__ NormArgs na,
                                                                                          const __grid_constant__ Deal deal) {
  using C = NormCfg<D>;
  constexpr int DEPTH = kNormGradDepth;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  NormGradShared<D, M>& sm = *reinterpret_cast<NormGradShared<D, M>*>(smem_raw);
  const RotaryArgs& a = na.r;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int half = a.rot >> 1, heads = a.Hq + a.Hk, hk = a.Hq;
  const Part<D> p(deal);
  const int t = p.t, e1 = first_of<M>(p.item, half), e2 = second_of<M>(p.item, half);
  const bool spread = M == kHalves && 2 * half == D;
  // A group's tokens are looked up while the group before is worked on.
  auto look_up = [&](unsigned t0) {
    const unsigned tok = t0 + warp;
    return tok < deal.rows && warp < 1 << deal.tok_shift ? find_token<false>(a, deal, tok, lane) : Token{};
  };
  Token next = look_up(blockIdx.x << deal.tok_shift);
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) (&sm.sums[0][0][0][0])[i * kRotaryThreads + tid] = 0.f;
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
        sm.feed.ask(s, 0, xs + e1, xs + e2, spread);
        sm.feed.ask(s, 1, gs + e1, gs + e2, spread);
      }
      sm.feed.asked();
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) ask(p.hl + i * p.HL, i);
    if (first) {
      read_frequencies<D>(a, half, sm.angles);
      read_gains<D, M>(na, half, sm.gains);
      first = false;
    } else {
      __syncthreads();  // the last group's angles are used up
    }
    if (warp < nt && lane == 0) sm.tk[warp] = next;
    __syncthreads();
    next = look_up(t0 + (gridDim.x << deal.tok_shift));
    norm_angles<D, M>(a, half, nt, sm.tk, sm.angles);
    __syncthreads();
    if (!live) continue;
    float2 s1[W], s2[W];  // this thread's sums of h e for one tensor
    int which = p.hl < hk ? 0 : 1, s = 0;
    auto clear = [&]() {
#pragma unroll
      for (int i = 0; i < W; ++i) s1[i] = s2[i] = make_float2(0.f, 0.f);
    };
    auto flush = [&]() {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sm.sums[which][0][i][tid] += i & 1 ? s1[i / 2].y : s1[i / 2].x;
        sm.sums[which][1][i][tid] += i & 1 ? s2[i / 2].y : s2[i / 2].x;
      }
    };
    clear();
    for (int h = p.hl; h < heads; h += p.HL) {
      if (which == 0 && h >= hk) {
        flush();
        clear();
        which = 1;
      }
      Item<V> x, g;
      sm.feed.wait();
      sm.feed.read(s, 0, x);
      sm.feed.read(s, 1, g);
      float2 x1[W], x2[W], h1[W], h2[W], w[W], sq = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
      const float(*gain)[D / 2] = sm.gains.g[which];
      unpack_item<T>(x, x1, x2);
      unpack_item<T>(g, h1, h2);
      turn<D, M>(sm.angles, t, sm.rows.x + p.row * RowTable<D, M>::STRIDE, p.item, half, p.mask, h1, h2);
      pairs_load<D>(gain[0], p.item, w);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        sq = ffma2(x1[i], x1[i], sq);
        dot = ffma2(fmul2(h1[i], w[i]), x1[i], dot);
      }
      pairs_load<D>(gain[1], p.item, w);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        sq = ffma2(x2[i], x2[i], sq);
        dot = ffma2(fmul2(h2[i], w[i]), x2[i], dot);
      }
      float size = fmaf(head_sum<C::S>(sq.x + sq.y, p.mask), 1.f / D, na.eps);
      float product = head_sum<C::S>(dot.x + dot.y, p.mask), scale;
      const bool far = far_from_one<T>(size);
      if (far) {
        size = scale_far<D>(x1, x2, na.eps, p.mask, &scale);
        dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < W; ++i) dot = ffma2(fmul2(h2[i], w[i]), x2[i], dot);
        pairs_load<D>(gain[0], p.item, w);
#pragma unroll
        for (int i = 0; i < W; ++i) dot = ffma2(fmul2(h1[i], w[i]), x1[i], dot);
        product = head_sum<C::S>(dot.x + dot.y, p.mask);
      }
      const float r = rsqrtf(size);
      const float mean = product * r * (1.f / D);  // of g h e
      const float2 rr = make_float2(r, r), mm = make_float2(-mean, -mean);
      pairs_load<D>(gain[0], p.item, w);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 e = fmul2(x1[i], rr);
        s1[i] = ffma2(h1[i], e, s1[i]);
        h1[i] = fmul2(ffma2(e, mm, fmul2(h1[i], w[i])), rr);  // dx from here on
      }
      pairs_load<D>(gain[1], p.item, w);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 e = fmul2(x2[i], rr);
        s2[i] = ffma2(h2[i], e, s2[i]);
        h2[i] = fmul2(ffma2(e, mm, fmul2(h2[i], w[i])), rr);
      }
      if (far) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          h1[i] = fmul2(h1[i], make_float2(scale, scale));
          h2[i] = fmul2(h2[i], make_float2(scale, scale));
        }
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        x.p1.w[i] = Elem<T>::pack(h1[i].x, h1[i].y);
        x.p2.w[i] = Elem<T>::pack(h2[i].x, h2[i].y);
      }
      T* dst = h < hk ? static_cast<T*>(a.q_out) + at(a.sqo) + h * a.sqo.h
                      : static_cast<T*>(a.k_out) + at(a.sko) + (h - hk) * a.sko.h;
      *reinterpret_cast<Vector*>(dst + e1) = x.p1.v;
      *reinterpret_cast<Vector*>(dst + e2) = x.p2.v;
      ask(h + DEPTH * p.HL, s);
      s = s + 1 == DEPTH ? 0 : s + 1;
    }
    flush();
  }
  __syncthreads();
  // The block's sums, a value a thread, its rows in order.
  for (int i = tid; i < 2 * D; i += kRotaryThreads) {
    const int which = i / D, part = i / (D / 2) & 1, j = i % (D / 2) / C::S, item = i % C::S;
    const float* from = sm.sums[which][part][j] + item;
    float sum = 0.f;
#pragma unroll 8
    for (int r = 0; r < C::ROWS; ++r) sum += from[r * C::S];
    const int e = (part ? second_of<M>(item, half) : first_of<M>(item, half)) + j;
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

template <typename T, int D, Turn M>
cudaError_t launch_t(const NormArgs& na, cudaStream_t stream) {
  const RotaryArgs& a = na.r;
  using C = NormCfg<D>;
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
    auto kern = a.append ? norm_rotary_kernel<T, D, M, true> : norm_rotary_kernel<T, D, M, false>;
    return launch_dependent("norm kernel launch", kern, groups, kRotaryThreads, 0, stream, na, deal);
  }
  NormArgs g = na;
  g.parts = static_cast<int>(std::min<unsigned>(groups, kNormParts));
  auto grad = norm_rotary_grad_kernel<T, D, M>;
  constexpr int smem = sizeof(NormGradShared<D, M>);
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(grad), smem, na.device);
  if (e != cudaSuccess) return e;
  e = launch_dependent("norm gradient kernel launch", grad, g.parts, kRotaryThreads, smem, stream, g, deal);
  if (e != cudaSuccess || (!g.q_dgain && !g.k_dgain)) return e;
  return launch_dependent("gains' gradient kernel launch", norm_gains_kernel<D>, 2 * D / 32, 1024, 0, stream, g);
}

template <typename T, int D>
cudaError_t launch_d(const NormArgs& a, cudaStream_t stream) {
  if (!a.r.inv_freq) return launch_t<T, D, kHalves>(a, stream);  // nothing is turned
  if (a.r.interleaved) return launch_t<T, D, kPairs>(a, stream);
  return a.r.rot % 16 == 0 ? launch_t<T, D, kHalves>(a, stream) : launch_t<T, D, kAnywhere>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rotary(const NormArgs& a, cudaStream_t stream) {
  if (a.r.dtype == kF16) return a.r.d == 64 ? launch_d<__half, 64>(a, stream) : launch_d<__half, 128>(a, stream);
  return a.r.d == 64 ? launch_d<__nv_bfloat16, 64>(a, stream) : launch_d<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
