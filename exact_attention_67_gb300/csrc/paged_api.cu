// paged_api.cu -- the C ABI of the operators around a paged key/value cache
// (declared in include/exattn.h): argument validation, plans, tensor maps and
// launches.  No device memory is allocated and nothing synchronises.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <numeric>

#include "exattn.h"
#include "paged.cuh"

using namespace exattn;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

Strides to_strides(const exattn_strides& s) { return Strides{s.b_stride, s.h_stride, s.n_stride}; }

// As for the attention calls: non-negative multiples of 8 elements below
// 2^36, positive along every axis of extent > 1.
int check_strides(const exattn_strides& s, long long B, long long H, long long N) {
  const long long v[3] = {s.b_stride, s.h_stride, s.n_stride}, ext[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (v[i] < 0 || v[i] >= (1ll << 36) || (v[i] & 7) != 0) return EXATTN_ERR_ALIGN;
    if (ext[i] > 1 && v[i] == 0) return EXATTN_ERR_SHAPE;
  }
  return EXATTN_OK;
}

bool known_dtype(int dtype) { return dtype == EXATTN_DTYPE_BF16 || dtype == EXATTN_DTYPE_F16; }

// The turned part of a head: even, within it, with finite positive factor.
int check_rotary(const double* inv_freq, int rot_dim, int d, float factor) {
  if (rot_dim < 2 || rot_dim > d || (rot_dim & 1)) return EXATTN_ERR_UNSUPPORTED;
  if (!aligned(inv_freq, 8)) return EXATTN_ERR_ALIGN;
  if (!std::isfinite(factor) || !(factor > 0.f)) return EXATTN_ERR_VALUE;
  return EXATTN_OK;
}

// Gains [d] of the norms (each may be missing), of a 16-bit type or fp32.
int check_gains(const void* q_gain, const void* k_gain, int gain_dtype, float eps) {
  if (!known_dtype(gain_dtype) && gain_dtype != EXATTN_DTYPE_F32) return EXATTN_ERR_UNSUPPORTED;
  const uintptr_t size = gain_dtype == EXATTN_DTYPE_F32 ? 4 : 2;
  if (!aligned(q_gain, size) || !aligned(k_gain, size)) return EXATTN_ERR_ALIGN;
  if (!std::isfinite(eps) || eps < 0.f) return EXATTN_ERR_VALUE;
  return EXATTN_OK;
}

int element_type(int dtype) { return dtype == EXATTN_DTYPE_F32 ? kF32 : dtype == EXATTN_DTYPE_F16 ? kF16 : kBF16; }

// Shared checks of a cache and its page table; fills the view.
int check_pages(PageView* pv, const int* page_table, long long table_stride, int max_pages, int num_pages,
                int page_size, int B, int Hkv, const exattn_strides& sk, const exattn_strides& sv) {
  if (!aligned(page_table, 4)) return EXATTN_ERR_ALIGN;
  if (num_pages < 1 || max_pages < 1 || Hkv < 1 || B < 1) return EXATTN_ERR_SHAPE;
  if (table_stride < 0 || (B > 1 && table_stride < max_pages)) return EXATTN_ERR_SHAPE;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1))) return EXATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size >= (1ll << 31)) return EXATTN_ERR_SHAPE;
  int rc;
  if ((rc = check_strides(sk, num_pages, Hkv, page_size)) != EXATTN_OK ||
      (rc = check_strides(sv, num_pages, Hkv, page_size)) != EXATTN_OK)
    return rc;
  pv->table = page_table;
  pv->table_stride = table_stride;
  pv->max_pages = max_pages;
  pv->num_pages = num_pages;
  pv->page_size = page_size;
  pv->page_shift = 0;
  while ((1 << pv->page_shift) < page_size) ++pv->page_shift;
  return EXATTN_OK;
}

// The new tokens of B sequences in `total` packed rows.
int check_tokens(NewTokens* nt, const int* cu_seqlens, const int* seqlens, int B, int total) {
  if (B < 1 || total < 1) return EXATTN_ERR_SHAPE;
  if (!aligned(seqlens, 4) || !aligned(cu_seqlens, 4)) return EXATTN_ERR_ALIGN;
  if (!cu_seqlens && total % B != 0) return EXATTN_ERR_SHAPE;
  *nt = NewTokens{cu_seqlens, seqlens, B, total, cu_seqlens ? 0 : total / B};
  return EXATTN_OK;
}

}  // namespace

namespace {

// Checks of a call that turns [B, H, N, d] views, and its kernel's arguments.
int rotary_args(RotaryArgs* out, int dtype, const void* q, exattn_strides sq, void* q_out, exattn_strides sqo, int Hq,
                const void* k, exattn_strides sk, void* k_out, exattn_strides sko, int Hk, const int* positions,
                long long pos_stride, const double* inv_freq, int rot_dim, int interleaved, int inverse, float factor, int B,
                int N, int d) {
  if (!q || !q_out || !positions || !inv_freq || (Hk > 0 && (!k || !k_out))) return EXATTN_ERR_NULL;
  if (!known_dtype(dtype) || (d != 64 && d != 128)) return EXATTN_ERR_UNSUPPORTED;
  if (B < 1 || N < 1 || Hq < 1 || Hk < 0 || Hq > 65536 || Hk > 65536) return EXATTN_ERR_SHAPE;
  if (static_cast<long long>(B) * N >= (1ll << 31) || pos_stride < 0) return EXATTN_ERR_SHAPE;
  int rc = check_rotary(inv_freq, rot_dim, d, factor);
  if (rc != EXATTN_OK) return rc;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16) || !aligned(positions, 4))
    return EXATTN_ERR_ALIGN;
  if ((rc = check_strides(sq, B, Hq, N)) != EXATTN_OK || (rc = check_strides(sqo, B, Hq, N)) != EXATTN_OK) return rc;
  if (Hk > 0 &&
      ((rc = check_strides(sk, B, Hk, N)) != EXATTN_OK || (rc = check_strides(sko, B, Hk, N)) != EXATTN_OK))
    return rc;
  RotaryArgs& a = *out;
  a.q = q;
  a.sq = to_strides(sq);
  a.q_out = q_out;
  a.sqo = to_strides(sqo);
  a.k = k;
  a.sk = to_strides(sk);
  a.k_out = k_out;
  a.sko = to_strides(sko);
  a.Hq = Hq;
  a.Hk = Hk;
  a.B = B;
  a.N = N;
  a.d = d;
  a.dtype = element_type(dtype);
  a.positions = positions;
  a.pos_stride = pos_stride;
  a.inv_freq = inv_freq;
  a.rot = rot_dim;
  a.interleaved = interleaved ? 1 : 0;
  a.inverse = inverse ? 1 : 0;
  a.factor = factor;
  return EXATTN_OK;
}

// The same of a call that appends to a cache; `normed`: q needs no frequencies.
int append_args(RotaryArgs* out, bool normed, int dtype, const void* q, exattn_strides sq, void* q_out, exattn_strides sqo,
                int Hq, const void* k, exattn_strides sk, const void* v, exattn_strides sv, void* k_cache, exattn_strides skc,
                void* v_cache, exattn_strides svc, int Hkv, int num_pages, int page_size, const int* page_table,
                long long table_stride, int max_pages, const int* seqlens, const int* cu_seqlens, int B, int total, int d,
                const double* inv_freq, int rot_dim, int interleaved, float factor) {
  if (!k || !v || !k_cache || !v_cache || !page_table || !seqlens) return EXATTN_ERR_NULL;
  if (Hq > 0 && (!q || !q_out || (!inv_freq && !normed))) return EXATTN_ERR_NULL;
  if (!known_dtype(dtype) || (d != 64 && d != 128)) return EXATTN_ERR_UNSUPPORTED;
  if (Hq < 0 || Hq > 65536 || Hkv < 1 || Hkv > 65536) return EXATTN_ERR_SHAPE;
  RotaryArgs& a = *out;
  int rc = check_tokens(&a.nt, cu_seqlens, seqlens, B, total);
  if (rc != EXATTN_OK) return rc;
  if ((rc = check_pages(&a.pv, page_table, table_stride, max_pages, num_pages, page_size, B, Hkv, skc, svc)) !=
      EXATTN_OK)
    return rc;
  if (inv_freq && (rc = check_rotary(inv_freq, rot_dim, d, factor)) != EXATTN_OK) return rc;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16))
    return EXATTN_ERR_ALIGN;
  if (Hq > 0 && ((rc = check_strides(sq, 1, Hq, total)) != EXATTN_OK ||
                 (rc = check_strides(sqo, 1, Hq, total)) != EXATTN_OK))
    return rc;
  if ((rc = check_strides(sk, 1, Hkv, total)) != EXATTN_OK || (rc = check_strides(sv, 1, Hkv, total)) != EXATTN_OK)
    return rc;
  a.q = q;
  a.sq = to_strides(sq);
  a.q_out = q_out;
  a.sqo = to_strides(sqo);
  a.k = k;
  a.sk = to_strides(sk);
  a.k_out = k_cache;
  a.sko = to_strides(skc);
  a.v = v;
  a.sv = to_strides(sv);
  a.v_out = v_cache;
  a.svo = to_strides(svc);
  a.Hq = Hq;
  a.Hk = Hkv;
  a.d = d;
  a.dtype = element_type(dtype);
  a.inv_freq = inv_freq;
  a.rot = rot_dim;
  a.interleaved = interleaved ? 1 : 0;
  a.factor = factor;
  a.append = true;
  return EXATTN_OK;
}

// The current device's set-up; calls that do not use its watchdog word.
int device_ready(int* dev = nullptr) {
  int own = 0;
  unsigned* err = nullptr;
  return setup_device(dev ? dev : &own, &err);
}

int status_of(cudaError_t e) { return e == cudaSuccess ? EXATTN_OK : EXATTN_ERR_CUDA; }

}  // namespace

extern "C" int attn_rotary(int dtype, const void* q, exattn_strides sq, void* q_out, exattn_strides sqo, int Hq,
                           const void* k, exattn_strides sk, void* k_out, exattn_strides sko, int Hk,
                           const int* positions, long long pos_stride, const double* inv_freq, int rot_dim,
                           int interleaved, int inverse, float factor, int B, int N, int d, void* stream) {
  RotaryArgs a{};
  int rc = rotary_args(&a, dtype, q, sq, q_out, sqo, Hq, k, sk, k_out, sko, Hk, positions, pos_stride, inv_freq, rot_dim,
                       interleaved, inverse, factor, B, N, d);
  if (rc != EXATTN_OK || (rc = device_ready()) != EXATTN_OK) return rc;
  return status_of(launch_rotary(a, static_cast<cudaStream_t>(stream)));
}

extern "C" int attn_norm_rotary(int dtype, const void* q, exattn_strides sq, void* q_out, exattn_strides sqo, int Hq,
                                const void* k, exattn_strides sk, void* k_out, exattn_strides sko, int Hk,
                                const int* positions, long long pos_stride, const double* inv_freq, int rot_dim,
                                int interleaved, float factor, const void* q_gain, const void* k_gain, int gain_dtype,
                                float eps, int B, int N, int d, void* stream) {
  NormArgs a{};
  int rc = rotary_args(&a.r, dtype, q, sq, q_out, sqo, Hq, k, sk, k_out, sko, Hk, positions, pos_stride, inv_freq, rot_dim,
                       interleaved, 0, factor, B, N, d);
  if (rc != EXATTN_OK || (rc = check_gains(q_gain, k_gain, gain_dtype, eps)) != EXATTN_OK) return rc;
  if ((rc = device_ready()) != EXATTN_OK) return rc;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.gain_dtype = element_type(gain_dtype);
  a.eps = eps;
  return status_of(launch_norm_rotary(a, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t attn_norm_rotary_backward_workspace_size(int B, int N, int d) {
  if (B < 1 || N < 1 || static_cast<long long>(B) * N >= (1ll << 31) || (d != 64 && d != 128)) return 0;
  return std::min<size_t>(static_cast<size_t>(B) * N, kNormParts) * 2 * d * sizeof(float);
}

extern "C" int attn_norm_rotary_backward(int dtype, const void* dq, exattn_strides sdq, const void* q, exattn_strides sq,
                                         void* dq_out, exattn_strides sqo, int Hq, const void* dk, exattn_strides sdk,
                                         const void* k, exattn_strides sk, void* dk_out, exattn_strides sko, int Hk,
                                         const int* positions, long long pos_stride, const double* inv_freq, int rot_dim,
                                         int interleaved, float factor, const void* q_gain, const void* k_gain,
                                         int gain_dtype, float eps, void* dq_gain, void* dk_gain, int B, int N, int d,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!dq || (Hk > 0 && !dk)) return EXATTN_ERR_NULL;
  NormArgs a{};
  int rc = rotary_args(&a.r, dtype, q, sq, dq_out, sqo, Hq, k, sk, dk_out, sko, Hk, positions, pos_stride, inv_freq, rot_dim,
                       interleaved, 1, factor, B, N, d);
  if (rc != EXATTN_OK || (rc = check_gains(q_gain, k_gain, gain_dtype, eps)) != EXATTN_OK ||
      (rc = check_gains(dq_gain, dk_gain, gain_dtype, eps)) != EXATTN_OK)
    return rc;
  if (!aligned(dq, 16) || !aligned(dk, 16)) return EXATTN_ERR_ALIGN;
  if ((rc = check_strides(sdq, B, Hq, N)) != EXATTN_OK || (Hk > 0 && (rc = check_strides(sdk, B, Hk, N)) != EXATTN_OK))
    return rc;
  if (!workspace || workspace_bytes < attn_norm_rotary_backward_workspace_size(B, N, d)) return EXATTN_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return EXATTN_ERR_ALIGN;
  if ((rc = device_ready(&a.device)) != EXATTN_OK) return rc;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.gain_dtype = element_type(gain_dtype);
  a.eps = eps;
  a.dq = dq;
  a.sdq = to_strides(sdq);
  a.dk = dk;
  a.sdk = to_strides(sdk);
  a.q_dgain = dq_gain;
  a.k_dgain = dk_gain;
  a.partial = static_cast<float*>(workspace);
  return status_of(launch_norm_rotary(a, static_cast<cudaStream_t>(stream)));
}

extern "C" int attn_cache_append(int dtype, const void* q, exattn_strides sq, void* q_out, exattn_strides sqo, int Hq,
                                 const void* k, exattn_strides sk, const void* v, exattn_strides sv, void* k_cache,
                                 exattn_strides skc, void* v_cache, exattn_strides svc, int Hkv, int num_pages,
                                 int page_size, const int* page_table, long long table_stride, int max_pages,
                                 const int* seqlens, const int* cu_seqlens, int B, int total, int d,
                                 const double* inv_freq, int rot_dim, int interleaved, float factor, void* stream) {
  RotaryArgs a{};
  int rc = append_args(&a, false, dtype, q, sq, q_out, sqo, Hq, k, sk, v, sv, k_cache, skc, v_cache, svc, Hkv, num_pages,
                       page_size, page_table, table_stride, max_pages, seqlens, cu_seqlens, B, total, d, inv_freq, rot_dim,
                       interleaved, factor);
  if (rc != EXATTN_OK || (rc = device_ready()) != EXATTN_OK) return rc;
  return status_of(launch_rotary(a, static_cast<cudaStream_t>(stream)));
}

extern "C" int attn_cache_append_norm(int dtype, const void* q, exattn_strides sq, void* q_out, exattn_strides sqo, int Hq,
                                      const void* k, exattn_strides sk, const void* v, exattn_strides sv, void* k_cache,
                                      exattn_strides skc, void* v_cache, exattn_strides svc, int Hkv, int num_pages,
                                      int page_size, const int* page_table, long long table_stride, int max_pages,
                                      const int* seqlens, const int* cu_seqlens, int B, int total, int d,
                                      const double* inv_freq, int rot_dim, int interleaved, float factor,
                                      const void* q_gain, const void* k_gain, int gain_dtype, float eps, void* stream) {
  NormArgs a{};
  int rc = append_args(&a.r, true, dtype, q, sq, q_out, sqo, Hq, k, sk, v, sv, k_cache, skc, v_cache, svc, Hkv, num_pages,
                       page_size, page_table, table_stride, max_pages, seqlens, cu_seqlens, B, total, d, inv_freq, rot_dim,
                       interleaved, factor);
  if (rc != EXATTN_OK || (rc = check_gains(q_gain, k_gain, gain_dtype, eps)) != EXATTN_OK) return rc;
  if ((rc = device_ready()) != EXATTN_OK) return rc;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.gain_dtype = element_type(gain_dtype);
  a.eps = eps;
  return status_of(launch_norm_rotary(a, static_cast<cudaStream_t>(stream)));
}

extern "C" int attn_cache_copy(void* pool, long long slab_stride, long long page_stride, long long page_bytes,
                               int slabs, int num_pages, const int* src, const int* dst, int n, void* stream) {
  if (n < 0) return EXATTN_ERR_SHAPE;
  if (!pool || (n > 0 && (!src || !dst))) return EXATTN_ERR_NULL;
  if (slabs < 1 || slabs > 65535 || num_pages < 1 || page_bytes < 16 || page_bytes > (1ll << 30))
    return EXATTN_ERR_SHAPE;
  if (slabs == 1) slab_stride = 0;  // never used
  if (num_pages == 1) page_stride = 0;
  if (!aligned(pool, 16) || ((slab_stride | page_stride | page_bytes) & 15)) return EXATTN_ERR_ALIGN;
  // Pages of a slab, and slabs, must not overlap (either may be the outer one).
  if ((num_pages > 1 && page_stride < page_bytes) || (slabs > 1 && slab_stride < page_bytes)) return EXATTN_ERR_SHAPE;
  if (page_stride >= (1ll << 40) || slab_stride >= (1ll << 44)) return EXATTN_ERR_SHAPE;
  if (page_stride > (1ll << 61) / num_pages) return EXATTN_ERR_SHAPE;  // a slab's extent below 2^62
  if (num_pages > 1 && slabs > 1 && slab_stride < page_stride * (num_pages - 1) + page_bytes &&
      page_stride < slab_stride * (slabs - 1) + page_bytes)
    return EXATTN_ERR_SHAPE;
  if (n == 0) return EXATTN_OK;
  // One bit a page for the destinations, so that every pair is independent:
  // none named twice, none read.
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= num_pages || dst[i] < 0 || dst[i] >= num_pages) return EXATTN_ERR_VALUE;
  bool clash = false;
  if (n <= 32) {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < n; ++j) clash |= dst[i] == src[j] || (i < j && dst[i] == dst[j]);
  } else {
    uint64_t* written = static_cast<uint64_t*>(std::calloc((static_cast<size_t>(num_pages) + 63) / 64, 8));
    if (!written) return EXATTN_ERR_WORKSPACE;
    for (int i = 0; i < n; ++i) {
      uint64_t& w = written[dst[i] >> 6];
      const uint64_t bit = 1ull << (dst[i] & 63);
      clash |= (w & bit) != 0;
      w |= bit;
    }
    for (int i = 0; i < n; ++i) clash |= (written[src[i] >> 6] >> (src[i] & 63)) & 1;
    std::free(written);
  }
  if (clash) return EXATTN_ERR_VALUE;
  int dev = 0;
  unsigned* err = nullptr;
  const int rc = setup_device(&dev, &err);
  if (rc != EXATTN_OK) return rc;
  const CopyArgs a{static_cast<char*>(pool), slab_stride, page_stride, page_bytes, slabs, src, dst, n};
  return launch_page_copy(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? EXATTN_OK : EXATTN_ERR_CUDA;
}

namespace {

constexpr int kSMs = 152;
// Key tiles of a unit that is not cut: of few units, of half the SMs' count on.
constexpr int kWholeFew = 4, kWholeMany = 8;

// How a paged attention is laid out on the GPU, from sizes alone.
struct AttendPlan {
  int cols;  // of the decode kernel, 0: the forward kernel
  int tile_tokens, ctas, rows, unit_cost, min_chunk;
  size_t plan_bytes, sum_bytes, total_bytes;
  double units, weights;  // of the line, at most
};

// shared: the line over shared rows, whose decode kernel has 8, 16 or 32 columns.
AttendPlan paged_plan(int B, int Hq, int Hkv, int total, int max_q, int max_k, int d, bool shared = false) {
  AttendPlan p{};
  const int G = Hq / Hkv;
  max_q = std::min(max_q, total);
  const long long need = static_cast<long long>(max_q) * G;
  p.cols = shared && need <= kPagedDecodeCols ? (need <= 8 ? 8 : need <= 16 ? 16 : 32) : need <= 4 ? 4 : need <= 8 ? 8 : need <= 16 ? 16 : need <= kPagedDecodeCols ? 32 : 0;
  p.rows = p.cols ? std::max(p.cols, 16) : kPagedRows;
  p.tile_tokens = (p.cols ? p.cols : 128) / G;
  // A unit's fixed cost in key tiles, and the least worth a CTA.  Chunks of 3, 6 and
  // 9 weights: one sequence of 777 keys, 8 key heads 10.9, 13.3, 12.1 us; of 2,000
  // 11.0, 13.4, 15.6; unit costs of 2 to 8 change long chunks by 3 % at most.
  p.unit_cost = 2;
  p.min_chunk = 3;
  const int ut = p.cols ? p.tile_tokens : 2 * p.tile_tokens;
  // At most so many weights (paged_sched.cuh): units of full length.
  p.units = static_cast<double>(Hkv) * std::min<double>(static_cast<double>(B) * ((max_q + ut - 1) / ut),
                                                        static_cast<double>(total) / ut + B);
  p.weights = p.units * ((static_cast<double>(max_k) + 127) / 128 + p.unit_cost);
  p.ctas = static_cast<int>(std::min<double>(kSMs, std::max(1.0, std::ceil(p.weights / 2))));
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t slots = static_cast<size_t>(p.ctas) * 2 * p.rows;
  p.plan_bytes = up(static_cast<size_t>(p.ctas) * 32);  // a PagedPlan each
  p.sum_bytes = up(slots * sizeof(float2));
  p.total_bytes = p.plan_bytes + p.sum_bytes + up(slots * d * sizeof(float));
  return p;
}

int check_paged(int B, int Hq, int Hkv, int total, int max_q, int max_k, int d) {
  if (B < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || total < 1 || max_q < 1 || max_k < 1) return EXATTN_ERR_SHAPE;
  if (Hq > 65536 || static_cast<long long>(Hq) * total >= (1ll << 31) || total >= (1 << 30) || max_k >= (1 << 30) ||
      B >= (1 << 24))
    return EXATTN_ERR_SHAPE;
  if ((d != 64 && d != 128) || Hq / Hkv > 128) return EXATTN_ERR_UNSUPPORTED;
  return EXATTN_OK;
}

}  // namespace

extern "C" size_t attn_fwd_paged_workspace_size(int B, int Hq, int Hkv, int total, int max_seqlen_q, int max_seqlen_k,
                                                int d) {
  if (check_paged(B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d) != EXATTN_OK) return 0;
  const AttendPlan p = paged_plan(B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d);
  return p.weights < 2e9 ? p.total_bytes : 0;
}

namespace {

// The tensor map of packed queries, tiles of `tokens` tokens of one key head.
bool query_map(CUtensorMap* m, int dt, const void* q, const exattn_strides& sq, int Hkv, int G, int total, int d, int tokens) {
  // A stride along an axis of extent 1 is never used; the encoder gets a legal one.
  auto bytes = [&](int extent, long long stride) { return static_cast<cuuint64_t>(extent > 1 ? stride : d) * 2; };
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(G), static_cast<cuuint64_t>(Hkv),
                              static_cast<cuuint64_t>(total)};
  const cuuint64_t str[3] = {bytes(G, sq.h_stride), bytes(Hkv, G * sq.h_stride), bytes(total, sq.n_stride)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), 1, static_cast<cuuint32_t>(tokens)};
  return encode_map(m, dt, 4, q, dims, str, box);
}

// The maps of a cache's K (i = 0) or V, and its steps in the view.
int cache_map(CUtensorMap* m, PageView* pv, int i, int dt, const void* base, const exattn_strides& s, int num_pages, int Hkv,
              int page_size, int d) {
  // Pages and heads as one axis: places a common divisor of both strides apart.
  const long long sb = num_pages > 1 ? s.b_stride : 0, sh = Hkv > 1 ? s.h_stride : 0;
  const long long step = std::max(std::gcd(sb, sh), 8ll);
  const long long page_step = sb / step, head_step = sh / step;
  if (page_step >= (1ll << 31) || head_step >= (1ll << 31)) return EXATTN_ERR_SHAPE;  // the sums below: 2^62 each
  const long long places = (num_pages - 1) * page_step + (Hkv - 1) * head_step + 1;
  if (places >= (1ll << 31)) return EXATTN_ERR_SHAPE;
  (i == 0 ? pv->k_page_step : pv->v_page_step) = static_cast<int>(page_step);
  (i == 0 ? pv->k_head_step : pv->v_head_step) = static_cast<int>(head_step);
  const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(d / 64), static_cast<cuuint64_t>(page_size / 8),
                              static_cast<cuuint64_t>(places)};
  const cuuint64_t str[4] = {static_cast<cuuint64_t>(s.n_stride) * 2, 128, static_cast<cuuint64_t>(s.n_stride) * 16,
                             static_cast<cuuint64_t>(step) * 2};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(d / 64), static_cast<cuuint32_t>(std::min(page_size, 128) / 8), 1};
  return encode_map(m, dt, 5, base, dims, str, box) ? EXATTN_OK : EXATTN_ERR_CUDA;
}

// What a launch of an attention over pages has from its plan and its place in the
// workspace.
void plan_args(PagedArgs* a, const AttendPlan& plan, char* ws) {
  a->tile_tokens = plan.tile_tokens;
  a->cols = plan.cols;
  a->rows = plan.rows;
  a->ctas = plan.ctas;
  a->unit_cost = plan.unit_cost;
  a->min_chunk = plan.min_chunk;
  a->plan = reinterpret_cast<exattn::PagedPlan*>(ws);
  a->part_sum = reinterpret_cast<float2*>(ws + plan.plan_bytes);
  a->part_o = reinterpret_cast<float*>(ws + plan.plan_bytes + plan.sum_bytes);
}

// Checks of an attention over pages that hold whatever its masks, and what its launches
// have in common.
int attend_args(PagedArgs* out, int dtype, const void* q, const exattn_strides& sq, const void* k_cache,
                const exattn_strides& skc, const void* v_cache, const exattn_strides& svc, void* o, const exattn_strides& so,
                float* lse, int num_pages, int page_size, const int* page_table, long long table_stride, int max_pages,
                const int* seqlens, const int* cu_seqlens, int B, int Hq, int Hkv, int total, int max_seqlen_q,
                int max_seqlen_k, int d, int causal, int window, float scale) {
  if (!q || !k_cache || !v_cache || !o || !lse || !page_table || !seqlens) return EXATTN_ERR_NULL;
  if (!known_dtype(dtype)) return EXATTN_ERR_UNSUPPORTED;
  int rc = check_paged(B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d);
  if (rc != EXATTN_OK) return rc;
  PagedArgs& a = *out;
  if ((rc = check_tokens(&a.nt, cu_seqlens, seqlens, B, total)) != EXATTN_OK) return rc;
  if ((rc = check_pages(&a.pv, page_table, table_stride, max_pages, num_pages, page_size, B, Hkv, skc, svc)) !=
      EXATTN_OK)
    return rc;
  if (window < 0 || !std::isfinite(scale) || !(scale > 0.f)) return EXATTN_ERR_VALUE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return EXATTN_ERR_ALIGN;
  if ((rc = check_strides(sq, 1, Hq, total)) != EXATTN_OK || (rc = check_strides(so, 1, Hq, total)) != EXATTN_OK)
    return rc;
  a.o = o;
  a.so = to_strides(so);
  a.lse = lse;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.d = d;
  a.dtype = element_type(dtype);
  a.max_q = max_seqlen_q;
  a.max_k = static_cast<int>(std::min<long long>(max_seqlen_k, static_cast<long long>(max_pages) * page_size));
  a.causal = causal ? 1 : 0;
  a.window = std::min(window, 1 << 30);
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  return EXATTN_OK;
}

}  // namespace

extern "C" int attn_fwd_paged(int dtype, const void* q, exattn_strides sq, const void* k_cache, exattn_strides skc,
                              const void* v_cache, exattn_strides svc, void* o, exattn_strides so, float* lse,
                              int num_pages, int page_size, const int* page_table, long long table_stride,
                              int max_pages, const int* seqlens, const int* cu_seqlens, int B, int Hq, int Hkv,
                              int total, int max_seqlen_q, int max_seqlen_k, int d, int causal, int window,
                              float scale, void* workspace, size_t workspace_bytes, void* stream) {
  PagedArgs a{};
  int rc = attend_args(&a, dtype, q, sq, k_cache, skc, v_cache, svc, o, so, lse, num_pages, page_size, page_table, table_stride,
                       max_pages, seqlens, cu_seqlens, B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d, causal, window, scale);
  if (rc != EXATTN_OK) return rc;
  const AttendPlan plan = paged_plan(B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d);
  if (plan.weights >= 2e9) return EXATTN_ERR_SHAPE;
  if (!workspace || workspace_bytes < plan.total_bytes) return EXATTN_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return EXATTN_ERR_ALIGN;
  if ((rc = setup_device(&a.device, &a.err)) != EXATTN_OK) return rc;
  CUtensorMap mq, mk, mv;
  if (!query_map(&mq, a.dtype, q, sq, Hkv, a.G, total, d, plan.tile_tokens)) return EXATTN_ERR_CUDA;
  if ((rc = cache_map(&mk, &a.pv, 0, a.dtype, k_cache, skc, num_pages, Hkv, page_size, d)) != EXATTN_OK ||
      (rc = cache_map(&mv, &a.pv, 1, a.dtype, v_cache, svc, num_pages, Hkv, page_size, d)) != EXATTN_OK)
    return rc;
  a.tm_q = &mq;
  a.tm_k = &mk;
  a.tm_v = &mv;
  plan_args(&a, plan, static_cast<char*>(workspace));
  {
    // A unit's key tiles at most.  Short units are not cut: the merge takes some 3 us, a
    // tile 0.3 (decode) to 2.  Cut and whole: one next token at 500 keys, 8 key heads
    // (4 tiles) 8.9 and 8.2 us, at 777 keys (7) 9.3 and 10.3; 16 sequences of 5 tokens
    // at 1,000 keys, 128 units of 8 tiles, 15.3 and 13.0, of 12 17.9 and 16.6; prompts
    // of 512 tokens, 32 heads on 8, 21.2 and 17.1, of 1,024 29.1 and 25.5, of 1,500 (12
    // tiles) 40.4 and 42.3; 6 chunks under a window of 1,024 (10) 33.3 and 39.3.
    const long long span = a.window == 0 ? a.max_k : (a.causal ? 1ll : 2ll) * a.window + 2 * plan.tile_tokens;
    const long long tiles = std::min((a.max_k + 127ll) / 128, span / 128 + 2);
    a.whole = tiles <= (2 * plan.units >= kSMs ? kWholeMany : kWholeFew);
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((plan.cols ? launch_paged_decode(a, st) : launch_paged_fwd(a, st)) != cudaSuccess) return EXATTN_ERR_CUDA;
  return a.whole || launch_paged_merge(a, st) == cudaSuccess ? EXATTN_OK : EXATTN_ERR_CUDA;
}

namespace {

// How an attention behind shared rows is laid out: each line's plan, and its part of the
// workspace (what attn_fwd_paged's has, then the row buffer and the records).
struct SharedPlan {
  AttendPlan line[2];
  size_t at[2], rec_at[2], total_bytes;
  bool fits;  // the lines' weights in 31 bits
};

constexpr int kRowsUnitCost = 4;

SharedPlan shared_plan(int B, int groups, int Hq, int Hkv, int total, int max_q, int max_k, int max_group_q, int d) {
  SharedPlan p{};
  // A group has as many new tokens as its sequences, whatever the hint says.
  p.line[0] = paged_plan(groups, Hq, Hkv, total, std::max(max_group_q, max_q), max_k, d, true);
  p.line[1] = paged_plan(B, Hq, Hkv, total, max_q, max_k, d);
  // max_group_q chooses the kernel and sizes the grid; a larger group is only slower.
  const int ut = (p.line[0].cols ? 1 : 2) * p.line[0].tile_tokens;
  const double most = Hkv * (static_cast<double>(total) / ut + groups) *
                      ((static_cast<double>(max_k) + 127) / 128 + kRowsUnitCost);
  p.fits = most < 2e9 && 2 * p.line[1].weights < 2e9;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t rows = static_cast<size_t>(total) * Hq;
  for (int i = 0; i < 2; ++i) {
    p.at[i] = p.total_bytes;
    p.rec_at[i] = p.at[i] + p.line[i].total_bytes + up(rows * d * sizeof(float));
    p.total_bytes = p.rec_at[i] + up(rows * sizeof(PagedRecord));
  }
  return p;
}

// Whether sharing can pay, were max_k rows shared: else the call runs as attn_fwd_paged,
// which reads shared pages again mostly from L2.  (The shared rows are known on the device only:
// few of them before many of their own, or under a wide max_k, are shared at a loss.  Behind 512 rows
// with 200 of their own, shared and not, five tokens of 4 groups of 32, 8 key heads of 128, 81.9 and
// 63.7 us, one with 32 key heads 190.6 and 157.2; one of 4 groups of 8 with 2,000 of their own behind
// 512 and 1,024 60.0 and 51.1, 63.7 and 54.9; one of 16 with one key head behind 16,384 22.7 and 20.0:
// of 120 sizes the largest losses, and three more of 5 %.)
bool worth_sharing(int B, int groups, int Hq, int Hkv, int total, int max_q, int max_k, int d) {
  const int G = Hq / Hkv;
  const double tiles = max_k / 128;  // only whole tiles are shared
  if (tiles < 1 || B <= groups) return false;
  if (static_cast<long long>(std::min(max_q, total)) * G <= kPagedDecodeCols) {
    // Saved reads, mostly of L2, against the second line's units and the join.  Shared and
    // not: one token of 2 sequences behind 512 rows, 8 key heads of 128, 11.6 and 9.3 us (2 MB),
    // of 16 behind 2,048 21.5 and 19.6 (126 MB), behind 4,096 21.5 and 30.6; heads of 64, 63 MB
    // 20.2 and 17.0, 126 MB 19.4 and 25.4.  Five tokens of 16 behind 4,096, heads of 64, 126 MB
    // 38.2 and 34.9, 252 MB 53.5 and 57.5; of 32 in 4 groups behind 2,048, heads of 128, 235 MB 46.6
    // and 46.7, 470 MB 62.8 and 78.9.
    const double bytes = (B - static_cast<double>(groups)) * tiles * 128 * Hkv * d * 4;
    return bytes >= (max_q == 1 ? 96e6 : 256e6);
  }
  // Chunks are bound by their products: units of 256 query rows (of up to 128 four fifths of the
  // time) that fewer sequences fill better, 1.4 us a key tile and SM, against the join, 0.4 us
  // for 1,000 rows and heads.  Ten tokens of 2 sequences behind 4,096 rows, 32 heads on 8 of 128, 17.3
  // and 20.3 us (too few units to count so: not shared), of 24 44.2 and 80.3; 30 of 8 behind 1,024 25.3 and 23.1, behind 16,384 73.3 and 98.7;
  // 64 (256 rows each) of 24 behind 16,384 329.9 and 305.6; 150 of 8 behind 4,096 97.5 and 97.0,
  // behind 16,384 266 and 300.
  auto units = [](double rows) {
    const double full = std::floor(rows / kPagedRows), rest = rows - full * kPagedRows;
    return full + (rest <= 0 ? 0. : rest <= kPagedRows / 2 ? 0.8 : 1.);
  };
  const double rows = static_cast<double>(total) * G;
  const double saved = (B * units(rows / B) - groups * units(rows / groups)) * tiles * Hkv;
  return saved * 1.4 / kSMs >= 5 + 0.4e-3 * total * Hq;
}

int check_shared(int groups, int max_group_q) {
  return groups < 1 || groups >= (1 << 24) || max_group_q < 1 ? EXATTN_ERR_SHAPE : EXATTN_OK;
}

}  // namespace

extern "C" size_t attn_fwd_paged_shared_workspace_size(int B, int groups, int Hq, int Hkv, int total, int max_seqlen_q,
                                                       int max_seqlen_k, int max_group_q, int d) {
  if (check_paged(B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d) != EXATTN_OK ||
      check_shared(groups, max_group_q) != EXATTN_OK)
    return 0;
  if (!worth_sharing(B, groups, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d))
    return attn_fwd_paged_workspace_size(B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d);
  const SharedPlan p = shared_plan(B, groups, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, max_group_q, d);
  return p.fits ? p.total_bytes : 0;
}

extern "C" int attn_fwd_paged_shared(int dtype, const void* q, exattn_strides sq, const void* k_cache, exattn_strides skc,
                                     const void* v_cache, exattn_strides svc, void* o, exattn_strides so, float* lse,
                                     int num_pages, int page_size, const int* page_table, long long table_stride,
                                     int max_pages, const int* seqlens, const int* cu_seqlens, const int* cu_groups,
                                     const int* prefix_lens, int B, int groups, int Hq, int Hkv, int total,
                                     int max_seqlen_q, int max_seqlen_k, int max_group_q, int d, int causal, float scale,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  if (!cu_groups || !prefix_lens) return EXATTN_ERR_NULL;
  PagedArgs a{};
  int rc = attend_args(&a, dtype, q, sq, k_cache, skc, v_cache, svc, o, so, lse, num_pages, page_size, page_table, table_stride,
                       max_pages, seqlens, cu_seqlens, B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d, causal, 0, scale);
  if (rc != EXATTN_OK || (rc = check_shared(groups, max_group_q)) != EXATTN_OK) return rc;
  if (!aligned(cu_groups, 4) || !aligned(prefix_lens, 4)) return EXATTN_ERR_ALIGN;
  if (!worth_sharing(B, groups, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d))
    return attn_fwd_paged(dtype, q, sq, k_cache, skc, v_cache, svc, o, so, lse, num_pages, page_size, page_table, table_stride,
                          max_pages, seqlens, cu_seqlens, B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d, causal, 0, scale,
                          workspace, workspace_bytes, stream);
  const SharedPlan plan = shared_plan(B, groups, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, max_group_q, d);
  if (!plan.fits) return EXATTN_ERR_SHAPE;
  if (!workspace || workspace_bytes < plan.total_bytes) return EXATTN_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return EXATTN_ERR_ALIGN;
  if ((rc = setup_device(&a.device, &a.err)) != EXATTN_OK) return rc;
  CUtensorMap mq[2], mk, mv;
  for (int i = 0; i < 2; ++i)
    if (!query_map(&mq[i], a.dtype, q, sq, Hkv, a.G, total, d, plan.line[i].tile_tokens)) return EXATTN_ERR_CUDA;
  if ((rc = cache_map(&mk, &a.pv, 0, a.dtype, k_cache, skc, num_pages, Hkv, page_size, d)) != EXATTN_OK ||
      (rc = cache_map(&mv, &a.pv, 1, a.dtype, v_cache, svc, num_pages, Hkv, page_size, d)) != EXATTN_OK)
    return rc;
  a.tm_k = &mk;
  a.tm_v = &mv;
  PagedShare& s = a.share;
  s.cu_groups = cu_groups;
  s.prefix = prefix_lens;
  s.groups = groups;
  s.sms = std::min(kSMs, std::max(2, plan.line[0].ctas + plan.line[1].ctas));
  for (int i = 0; i < 2; ++i) {
    const AttendPlan& l = plan.line[i];
    s.ctas[i] = l.ctas;
    s.unit_tokens[i] = (l.cols ? 1 : 2) * l.tile_tokens;
  }
  // A key tile of the forward kernel beside decode CTAs, which have more loads in flight,
  // takes two (one query tile) to three times theirs: 4 groups of 8 to 256 rows behind
  // 16,384 86.7 us at 3, 93 at 2.5, 90 at 4; 32 of 5 tokens (d = 64) 45.8 at 2, 49.5 at 1.5.
  const bool two = std::min(total, max_group_q) > plan.line[0].tile_tokens;
  s.tile_time[0] = plan.line[0].cols || !plan.line[1].cols ? 2 : two ? 6 : 4;
  s.tile_time[1] = 2;
  PagedLines both{{a, a}};
  for (int i = 0; i < 2; ++i) {
    PagedArgs& l = both.line[i];
    const AttendPlan& p = plan.line[i];
    char* ws = static_cast<char*>(workspace) + plan.at[i];
    plan_args(&l, p, ws);
    l.tm_q = &mq[i];
    l.share.line = i == 0 ? kSharedLine : kOwnLine;
    l.share.rec = reinterpret_cast<PagedRecord*>(static_cast<char*>(workspace) + plan.rec_at[i]);
    l.share.rows_at = static_cast<long long>((p.total_bytes - p.plan_bytes - p.sum_bytes) / sizeof(float));
    if (i == 0) l.causal = 0;  // all of a group's tokens stand behind its shared rows
    // A unit of the forward kernel that ends in the row buffer, mostly of a few masked
    // tiles: six of some 320 tokens behind a document 9.2 us a unit, a tile 1.6.
    if (!p.cols) l.unit_cost = kRowsUnitCost;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto launch = a.dtype == kF16 ? (d == 64 ? launch_paged_shared_f16_64 : launch_paged_shared_f16_128)
                                : (d == 64 ? launch_paged_shared_bf16_64 : launch_paged_shared_bf16_128);
  if (launch(both, st) != cudaSuccess) return EXATTN_ERR_CUDA;
  return status_of(launch_paged_join(both.line[0], both.line[1], st));
}
