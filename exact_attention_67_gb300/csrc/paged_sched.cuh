// paged_sched.cuh -- how the paged attention kernels share their work.
//
// A unit is a run of new tokens of one sequence with one key head: rows of
// queries that stream the same keys.  Laid end to end (sequence, head, run),
// with a unit weighing its 128-key tiles plus a fixed cost for its start and
// end, the units form one line of W weights, which the CTAs cut into equal
// chunks: CTA g takes [g chunk, (g + 1) chunk).  Whatever the lengths in a batch,
// every CTA streams the same number of keys, in one wave.  A unit cut by a chunk's
// end leaves pieces: each CTA has at most one piece that continues a unit and
// one that is continued, so two slots of partial results a CTA hold them all,
// and the merge joins them.  The lengths stay on the device; every CTA derives the
// line from them by itself.
#pragma once
#include "paged.cuh"
#include "ptx.cuh"

namespace exattn {

constexpr int kKeyTile = 128;

struct PagedSeq {
  int row0, n;  // first packed row, new tokens
  int len;      // keys
  int off;      // position of new token 0
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int b) {
  PagedSeq s;
  int n;
  if (a.nt.cu_seqlens) {
    const int c0 = min(max(a.nt.cu_seqlens[b], 0), a.nt.total);
    n = min(max(a.nt.cu_seqlens[b + 1], c0), a.nt.total) - c0;
    s.row0 = c0;
  } else {
    n = a.nt.each;
    s.row0 = b * n;
  }
  const int len = min(max(a.nt.seqlens[b], 0), 1 << 30);
  s.n = min(n, a.max_q);
  s.len = min(len, a.max_k);
  s.off = len - n;
  return s;
}

// Keys that some of the tokens [t0, t1) of a sequence see: [lo, hi).
__device__ __forceinline__ void paged_keys(const PagedArgs& a, const PagedSeq& s, int t0, int t1, int* lo, int* hi) {
  *lo = a.window > 0 ? max(0, s.off + t0 - a.window + 1) : 0;
  int e = s.len;
  if (a.causal) e = min(e, s.off + t1);
  else if (a.window > 0) e = min(e, s.off + t1 - 1 + a.window);
  *hi = max(e, *lo);
}

// One piece of a unit: its key tiles [t_lo, t_hi) of the unit's [k_lo, k_hi).
struct PagedPiece {
  PagedSeq s;
  int b, h;
  int tok0, ntok;   // tokens of the unit
  int key_hi;       // keys end
  int t_lo, t_hi, k_lo, k_hi;
  __device__ bool whole() const { return t_lo == k_lo && t_hi == k_hi; }
  __device__ int slot() const { return t_lo == k_lo ? 1 : 0; }
};

// A place in the line and the way through it.  UT: tokens a unit.
struct PagedCursor {
  int b, h, t;
  int pos;          // weights of unit t already passed
  long long left;   // weights left of this CTA's chunk

  // The next piece with anything to do (an empty unit has its zeros to
  // write); false at the chunk's end.
  __device__ __forceinline__ bool next(const PagedArgs& a, int UT, PagedSeq& s, PagedPiece* p) {
    while (left > 0) {
      while (t * UT >= s.n) {
        t = 0;
        if (++h >= a.Hkv || s.n <= 0) {
          h = 0;
          if (++b >= a.nt.B) {
            left = 0;
            return false;
          }
          s = paged_seq(a, b);
        }
      }
      const int t0 = t * UT, t1 = min(s.n, t0 + UT);
      int lo, hi;
      paged_keys(a, s, t0, t1, &lo, &hi);
      const int k0 = lo / kKeyTile, k1 = hi > lo ? (hi + kKeyTile - 1) / kKeyTile : k0;
      const int w = k1 - k0 + a.unit_cost;
      const int take = static_cast<int>(min(left, static_cast<long long>(w - pos)));
      p->s = s;
      p->b = b;
      p->h = h;
      p->tok0 = t0;
      p->ntok = t1 - t0;
      p->key_hi = hi;
      p->k_lo = k0;
      p->k_hi = k1;
      p->t_lo = k0 + max(0, pos - a.unit_cost);
      p->t_hi = k0 + max(0, pos + take - a.unit_cost);
      const bool first = pos == 0;
      left -= take;
      pos += take;
      if (pos == w) {
        pos = 0;
        ++t;
      }
      if (p->t_hi > p->t_lo || (first && k1 == k0)) return true;
    }
    return false;
  }
};

// Weight of sequence b's units with one key head.
__device__ __forceinline__ long long paged_weight(const PagedArgs& a, const PagedSeq& s, int UT) {
  long long w = 0;
  for (int t0 = 0; t0 < s.n; t0 += UT) {
    int lo, hi;
    paged_keys(a, s, t0, min(s.n, t0 + UT), &lo, &hi);
    const int k0 = lo / kKeyTile, k1 = hi > lo ? (hi + kKeyTile - 1) / kKeyTile : k0;
    w += k1 - k0 + a.unit_cost;
  }
  return w;
}

// Start of CTA `cta`'s chunk, found by one warp; the same in every lane.  W and
// chunk come back for the merge.
__device__ __forceinline__ PagedCursor paged_start(const PagedArgs& a, int UT, int cta, int lane, long long* chunk_out) {
  const int B = a.nt.B;
  auto weight = [&](int b) {
    return b < B ? paged_weight(a, paged_seq(a, b), UT) * a.Hkv : 0ll;
  };
  auto warp_sum = [](long long x) {
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
  const long long w0 = weight(lane);  // kept: most batches have at most 32 sequences
  long long W = warp_sum(w0);
  for (int b0 = 32; b0 < B; b0 += 32) W += warp_sum(weight(b0 + lane));
  long long chunk = (W + a.ctas - 1) / a.ctas;
  if (chunk < a.min_chunk) chunk = a.min_chunk;
  *chunk_out = chunk;
  PagedCursor c;
  const long long lo = cta * chunk;
  c.left = min(chunk, W - lo);
  c.b = c.h = c.t = c.pos = 0;
  if (c.left <= 0) {
    c.left = 0;
    return c;
  }
  long long before = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const long long w = b0 == 0 ? w0 : weight(b0 + lane);
    long long inc = w;  // inclusive prefix over the lanes
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + inc > lo);
    if (past) {
      const int l = __ffs(past) - 1;
      c.b = b0 + l;
      const long long start = before + __shfl_sync(0xffffffffu, inc - w, l);
      const long long per_head = __shfl_sync(0xffffffffu, w, l) / a.Hkv;
      long long r = lo - start;
      c.h = static_cast<int>(r / per_head);
      r -= c.h * per_head;
      const PagedSeq s = paged_seq(a, c.b);
      for (;;) {
        int klo, khi;
        paged_keys(a, s, c.t * UT, min(s.n, (c.t + 1) * UT), &klo, &khi);
        const int k0 = klo / kKeyTile, k1 = khi > klo ? (khi + kKeyTile - 1) / kKeyTile : k0;
        const int u = k1 - k0 + a.unit_cost;
        if (r < u) break;
        r -= u;
        ++c.t;
      }
      c.pos = static_cast<int>(r);
      return c;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  c.left = 0;
  return c;
}

// What CTA `cta` found, for the merge.
__device__ __forceinline__ void paged_note(const PagedArgs& a, const PagedCursor& c, long long chunk, int cta) {
  int* p = a.plan + cta * 8;
  p[0] = c.left > 0 ? 1 : 0;
  p[1] = c.b;
  p[2] = c.h;
  p[3] = c.t;
  p[4] = c.pos;
  p[5] = static_cast<int>(chunk & 0x7fffffff);
  p[6] = static_cast<int>(chunk >> 31);
}

}  // namespace exattn
