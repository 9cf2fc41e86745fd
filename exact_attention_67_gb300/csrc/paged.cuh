// paged.cuh -- launch interfaces of the operators around a paged key/value
// cache (rotary.cu, pages.cu, paged_decode.cu, paged_fwd.cu, paged_merge.cu) and the
// set-up that paged_api.cu shares with api.cu.
#pragma once
#include "kernels.cuh"

namespace exattn {

// api.cu: the current device's set-up (architecture check, watchdog word) and
// the driver's tensor-map encoder.
int setup_device(int* dev, unsigned** err);
bool encode_map(CUtensorMap* m, int dtype, int rank, const void* base, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box);

// Launches a kernel that may start before the stream's last kernel has ended (a
// programmatic dependent launch): it sets itself up meanwhile and executes
// griddepcontrol.wait before it reads or writes global memory, which holds it
// until everything before it in the stream is done and visible.
template <typename... Args, typename... Given>
cudaError_t launch_dependent(const char* what, void (*kern)(Args...), dim3 grid, dim3 block, int smem,
                             cudaStream_t stream, const Given&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  const cudaError_t last = cudaGetLastError();  // also clears a launch error e reported
  return note_cuda(e != cudaSuccess ? e : last, what);
}

// Pages of a cache: K and V are [num_pages, Hkv, page_size, d] views (Strides:
// b = page, h = head, n = row), and row b of the table lists the pages of
// sequence b in order.
struct PageView {
  const int* table;        // device [B, max_pages], row stride table_stride
  long long table_stride;
  int max_pages;
  int num_pages;
  int page_size;           // a power of two
  int page_shift;          // log2(page_size)
  // Attention: steps of a page and a key head in the places of the tensor maps.
  int k_page_step, k_head_step, v_page_step, v_head_step;
};

// Which rows of a packed tensor are the new tokens of sequence b: rows
// [cu_seqlens[b], cu_seqlens[b + 1]), or, without a table, `each` rows a
// sequence.  seqlens[b] is the sequence's length with its new tokens.
struct NewTokens {
  const int* cu_seqlens;
  const int* seqlens;
  int B, total, each;
};

struct RotaryArgs {
  const void* q;  // [B, Hq, N, d] (append: [total, Hq, d], n = token) or nullptr
  Strides sq;
  void* q_out;
  Strides sqo;
  const void* k;
  Strides sk;
  void* k_out;    // append: the K cache
  Strides sko;
  const void* v;  // append only
  Strides sv;
  void* v_out;    // append: the V cache
  Strides svo;
  int Hq, Hk;
  int B, N, d, dtype;
  const int* positions;    // [B, N], row stride pos_stride; append: unused
  long long pos_stride;
  const double* inv_freq;  // [rot / 2] radians a token, or nullptr (append: no rotation)
  int rot, interleaved, inverse;
  float factor;
  bool append;
  NewTokens nt;
  PageView pv;
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t stream);

// Attention of new tokens over a paged cache.  The query heads of a key head
// (G of them) and consecutive new tokens share the rows (forward kernel) or
// columns (decode kernel) of a unit: unit row r is token r / G, head r % G.
struct PagedArgs {
  const CUtensorMap* tm_q;  // (d, G, Hkv, total), box 64 x G x 1 x tokens of a query tile
  const CUtensorMap* tm_k;  // (64, 8, d / 64, page_size / 8, places): load_page in paged_sched.cuh
  const CUtensorMap* tm_v;
  void* o;                  // [total, Hq, d], strides h and n
  Strides so;
  float* lse;               // fp32 [Hq, total]
  NewTokens nt;
  PageView pv;
  int Hkv, G, d, dtype;
  int max_q, max_k;         // bounds of the new tokens and lengths of a sequence
  int causal, window;
  float scale_log2;
  int tile_tokens;          // tokens of a query tile: 128 / G (forward), cols / G (decode)
  int cols;                 // decode kernel: query columns, 4, 8, 16 or 32
  int rows;                 // rows of a piece's partial results
  int ctas;                 // grid; the work's split follows from it (paged_sched.cuh)
  int unit_cost, min_chunk;
  int whole;                // no unit is cut: a CTA takes the units that begin in its chunk
  float* part_o;            // [ctas][2][rows][d]
  float2* part_sum;         // [ctas][2][rows]: reference (log2 units) and sum of weights, mass = y 2^x
  struct PagedPlan* plan;   // [ctas]
  unsigned* err;
  int device;
};
constexpr int kPagedDecodeCols = 32;  // query columns of the decode kernel at most
constexpr int kPagedRows = 256;       // unit rows of the forward kernel: two query tiles
cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t stream);
cudaError_t launch_paged_fwd(const PagedArgs& a, cudaStream_t stream);
// Joins the pieces of the units that ended up on several CTAs.
cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t stream);

struct CopyArgs {
  char* pool;
  long long slab_stride, page_stride, page_bytes;  // bytes
  int slabs;
  const int* src;  // host
  const int* dst;  // host
  int n;
};
cudaError_t launch_page_copy(const CopyArgs& a, cudaStream_t stream);

}  // namespace exattn
