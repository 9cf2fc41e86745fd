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
// line from them by itself.  Where the largest length allows only short units, none
// is cut, and no merge runs.
#pragma once
#include "paged.cuh"
#include "ptx.cuh"

#include <limits.h>

namespace exattn {

constexpr int kKeyTile = 128;

// 1 / x and log2 x of a sum of weights, to 2^-22: it is at least 1 (the weight that
// set the reference) or NaN.  The full functions are a subroutine each at a unit's
// end: one next token at 777 keys 9.3 us with them, 9.1 without.
__device__ __forceinline__ float sum_inverse(float x) { return __fdividef(1.f, x); }
__device__ __forceinline__ float sum_log2(float x) { return __log2f(x); }

// Weights are f16 operands of the second product, and f16 drops what is below 2^-25.
// A row's weights are 1 at its reference and, the reference being moved once the
// maximum is 2^kRescale above it, at most 2^kRescale; taken 2^kLift times as large
// they still stay below f16's 65,504, and a key is dropped only 2^-32 below the row's
// largest weight instead of 2^-25 (one key 17.5 above 131,071 others: the others' 3 in
// 1,000 of the mass).  Sums and O are scaled alike, the logsumexp takes it out.
constexpr float kRescale = 8.f, kLift = 7.f;  // log2

// V enters the second product in f16.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  return pack_f16x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

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
struct alignas(16) PagedPiece {  // 64 bytes
  PagedSeq s;
  int b, h;
  int tok0, ntok;   // tokens of the unit
  int key_lo, key_hi;  // keys that some token sees
  int t_lo, t_hi, k_lo, k_hi;
  int n[2];         // forward kernel: key tiles from t_lo on that each query tile takes part in
  __device__ bool whole() const { return t_lo == k_lo && t_hi == k_hi; }
  __device__ int slot() const { return t_lo == k_lo ? 1 : 0; }
};

// The pieces of a CTA's chunk in order, from the warp that walks the line to the
// other warps: they keep no state of the walk, and hold a slot as long as they
// read it.  A piece with ntok = 0 ends the chunk.
constexpr int kRing = 4;
struct PagedRing {
  uint64_t full[kRing], empty[kRing];
  PagedPiece piece[kRing];

  __device__ void init(int readers) {  // reading warps
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], readers);
    }
  }
  // By one warp: piece i, or with p = nullptr the end.
  __device__ bool put(int i, const PagedPiece* p, int lane, const WaitCtl& wc) {
    const int s = i % kRing;
    if (i >= kRing && !mbar_wait_warp(&empty[s], (i / kRing - 1) & 1, wc)) return false;
    if (lane == 0) {
      if (p) piece[s] = *p;
      else piece[s].ntok = 0;
      mbar_arrive(&full[s]);
    }
    __syncwarp();
    return true;
  }
  // By each reading warp: piece i, or nullptr at the end (and when a wait gave up).
  __device__ const PagedPiece* get(int i, const WaitCtl& wc) {
    const int s = i % kRing;
    if (!mbar_wait_warp(&full[s], (i / kRing) & 1, wc)) return nullptr;
    return piece[s].ntok > 0 ? &piece[s] : nullptr;
  }
  __device__ void release(int i) { mbar_arrive_warp(&empty[i % kRing]); }
};

// A place in the line and the way through it.  UT: tokens a unit.
struct PagedCursor {
  int b, h, t;
  int pos;    // weights of unit t already passed
  int cost;   // fixed weight of a unit
  int left;   // weights left of this CTA's chunk

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
      const int w = k1 - k0 + cost;
      const int take = a.whole ? w : min(left, w - pos);
      p->s = s;
      p->b = b;
      p->h = h;
      p->tok0 = t0;
      p->ntok = t1 - t0;
      p->key_lo = lo;
      p->key_hi = hi;
      p->k_lo = k0;
      p->k_hi = k1;
      p->t_lo = k0 + max(0, pos - cost);
      p->t_hi = k0 + max(0, pos + take - cost);
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

// Key tiles of the unit of tokens [t0, t0 + UT).
__device__ __forceinline__ int paged_tiles(const PagedArgs& a, const PagedSeq& s, int t0, int UT) {
  int lo, hi;
  paged_keys(a, s, t0, min(s.n, t0 + UT), &lo, &hi);
  return hi > lo ? (hi + kKeyTile - 1) / kKeyTile - lo / kKeyTile : 0;
}

// Weight of a sequence's units with one key head.
__device__ __forceinline__ int paged_weight(const PagedArgs& a, const PagedSeq& s, int UT) {
  int w = 0;
  for (int t0 = 0; t0 < s.n; t0 += UT) w += paged_tiles(a, s, t0, UT) + a.unit_cost;
  return w;
}

// What the merge needs of the boundary before a CTA's chunk.
struct PagedPlan {
  int pos;           // weights of the unit before the boundary (0: it starts there)
  int chunk;
  int tiles;         // key tiles of the unit
  int cost;          // its fixed weight
  int row, ntok, h;  // its first packed row, tokens, key head
  int pad;           // 32 bytes
};

// x / y for x >= 0, y > 0, without the division's subroutine: it and the loads are
// the start of every call.
__device__ __forceinline__ int paged_div(int x, int y) {
  int q = static_cast<int>(__fdividef(static_cast<float>(x), static_cast<float>(y)));
  while (static_cast<long long>(q) * y > x) --q;
  while ((q + 1ll) * y <= x) ++q;
  return q;
}

// Reads the call's constants before griddepcontrol.wait: they need not wait for
// anything, and the first read of each line of them takes a few hundred clocks.
__device__ __forceinline__ void paged_touch(const PagedArgs& a) {
  asm volatile("" ::"l"(a.nt.cu_seqlens), "l"(a.nt.seqlens), "r"(a.nt.B), "r"(a.nt.total), "l"(a.pv.table),
               "r"(a.pv.page_size), "r"(a.pv.k_page_step), "r"(a.Hkv), "r"(a.max_q), "r"(a.window), "r"(a.ctas),
               "l"(a.plan), "l"(a.err));
}

// Start of this CTA's chunk, found by one warp; the same in every lane.  Leaves
// the merge its PagedPlan.  The line's weights fit 31 bits (checked on the host
// against the largest that the sizes allow).
__device__ __forceinline__ PagedCursor paged_start(const PagedArgs& a, int UT, int lane, PagedSeq* seq) {
  const int B = a.nt.B, cta = static_cast<int>(blockIdx.x);
  auto read = [&](int b) { return b < B ? paged_seq(a, b) : PagedSeq{0, 0, 0, 0}; };
  const PagedSeq s0 = read(lane);
  const int w0 = paged_weight(a, s0, UT);  // kept: most batches have at most 32 sequences
  int sum = w0, most = w0, least = w0 > 0 ? w0 : INT_MAX, count = w0 > 0;
  for (int b = 32 + lane; b < B; b += 32) {
    const int w = paged_weight(a, paged_seq(a, b), UT);
    sum += w;
    most = max(most, w);
    least = min(least, w > 0 ? w : INT_MAX);
    count += w > 0;
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  const int units = __reduce_add_sync(0xffffffffu, count) * a.Hkv, tiles_each = most - a.unit_cost;
  int W = sum * a.Hkv, cost = a.unit_cost;
  int chunk = max(paged_div(W + a.ctas - 1, a.ctas), a.min_chunk);
  // The decode kernel, where a unit is a (sequence, key head), and all weigh the same.
  if (a.cols > 0 && most == least && tiles_each > 0 && units <= a.ctas) {
    // As many pieces a unit as CTAs, of two tiles at least; none of four or fewer
    // (joining pieces takes some 2 us, a tile 0.6).  Unless this leaves over a
    // quarter of the SMs out of long work.
    const int most_pieces = paged_div(a.ctas, units);
    const int each = tiles_each <= 4 || a.whole ? tiles_each : max(paged_div(tiles_each + most_pieces - 1, most_pieces), 2);
    const int k = paged_div(tiles_each + each - 1, each);
    if (4 * units * k >= 3 * a.ctas || each <= 4 || a.whole) {
      chunk = each;
      cost = k * chunk - tiles_each;  // less than a chunk: the first piece's tiles are fewer by it
      W = units * k * chunk;
    }
  }
  const long long lo64 = static_cast<long long>(cta) * chunk;
  const int pad = cost - a.unit_cost;  // of every unit's weight
  PagedCursor c{0, 0, 0, 0, cost, 0};
  PagedPlan plan{0, chunk, 0, cost, 0, 0, 0, 0};
  *seq = PagedSeq{0, 0, 0, 0};
  int before = 0;
  for (int b0 = 0; b0 < B && lo64 < W; b0 += 32) {
    const int lo = static_cast<int>(lo64);
    const PagedSeq sl = b0 == 0 ? s0 : read(b0 + lane);
    int w = b0 == 0 ? w0 : paged_weight(a, sl, UT);
    if (w > 0) w += pad;  // not 0 only where a sequence has one unit a key head
    const int per_head = w;
    w *= a.Hkv;
    int inc = w;  // inclusive prefix over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + inc > lo);
    if (past) {
      const int l = __ffs(past) - 1;
      PagedSeq s;
      s.row0 = __shfl_sync(0xffffffffu, sl.row0, l);
      s.n = __shfl_sync(0xffffffffu, sl.n, l);
      s.len = __shfl_sync(0xffffffffu, sl.len, l);
      s.off = __shfl_sync(0xffffffffu, sl.off, l);
      const int each_head = __shfl_sync(0xffffffffu, per_head, l);
      int r = lo - before - __shfl_sync(0xffffffffu, inc - w, l);
      c.left = min(chunk, W - lo);
      c.b = b0 + l;
      c.h = paged_div(r, each_head);
      r -= c.h * each_head;
      int tiles;
      for (;;) {
        tiles = paged_tiles(a, s, c.t * UT, UT);
        if (r < tiles + cost) break;
        r -= tiles + cost;
        ++c.t;
      }
      c.pos = r;
      *seq = s;
      if (a.whole && r > 0) {  // the CTA before has it
        c.left -= tiles + cost - r;
        c.pos = 0;
        ++c.t;
      }
      plan = PagedPlan{r, chunk, tiles, cost, s.row0 + c.t * UT, min(UT, s.n - c.t * UT), c.h, 0};
      break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) a.plan[cta] = plan;
  return c;
}

// The page numbers of a piece's tiles, read 32 boxes at a time and as many ahead (one
// read a tile, a tile ahead: a producer took 1,300 clocks a tile, now 1,000).
struct PageNumbers {
  int shift;         // log2 of the boxes a tile
  int t0;            // first tile of `now`
  int now, ahead;    // a lane's box: tile t0 + (lane >> shift), box lane & (2^shift - 1) of it

  // Boxes of tile t that hold a key that some query sees.
  __device__ int boxes(const PagedPiece& p, int t) const {
    const int rows = kKeyTile >> shift;
    return min(1 << shift, (p.key_hi - t * kKeyTile + rows - 1) >> (7 - shift));
  }
  __device__ int read(const PagedArgs& a, const PagedPiece& p, int from, int lane) const {
    const int t = from + (lane >> shift), box = lane & ((1 << shift) - 1);
    return t < p.t_hi && box < boxes(p, t) ? a.pv.table[p.b * a.pv.table_stride + (t * kKeyTile >> a.pv.page_shift) + box]
                                           : 0;
  }
  __device__ void start(const PagedArgs& a, const PagedPiece& p, int lane) {
    t0 = p.t_lo;
    now = read(a, p, t0, lane);
    ahead = read(a, p, t0 + (32 >> shift), lane);
  }
  // The page of box `lane` of tile t; tiles in order.
  __device__ int take(const PagedArgs& a, const PagedPiece& p, int t, int lane) {
    if (t - t0 == 32 >> shift) {
      t0 = t;
      now = ahead;
      ahead = read(a, p, t0 + (32 >> shift), lane);
    }
    return __shfl_sync(0xffffffffu, now, ((t - t0) << shift) + lane);
  }
};

// One page's (at most 128) rows of a K or V tile: a box of the 5-D map
// (64 elements, 8 rows, d / 64, groups of 8 rows, places), which lands as groups
// of 8 rows, each with its 64-element atoms side by side.  A place is a (page,
// key head), so K and V of any strides take one box a page whatever d is.  A
// page outside the pool loads zeros (a place before the map's first).
__device__ __forceinline__ void load_page(const CUtensorMap* m, uint64_t* bar, void* dst, const PageView& pv, int group,
                                          int page, int head, bool is_k, uint64_t cache_hint) {
  const int place = page >= 0 && page < pv.num_pages
                        ? page * (is_k ? pv.k_page_step : pv.v_page_step) + head * (is_k ? pv.k_head_step : pv.v_head_step)
                        : -1;
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %3, %3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(0), "r"(group), "r"(place), "l"(cache_hint)
      : "memory");
}

}  // namespace exattn
