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

// Norms of the heads with the turn (norm_rotary.cu).  r.q, r.k are the rows x; the
// gradient (partial not null) turns dq, dk back (r.inverse) and writes r.q_out, r.k_out.
struct NormArgs {
  RotaryArgs r;
  const void* q_gain;  // [d] or nullptr (all 1)
  const void* k_gain;
  int gain_dtype;      // kBF16, kF16 or kF32
  float eps;
  const void* dq;
  Strides sdq;
  const void* dk;
  Strides sdk;
  void* q_dgain;       // [d] or nullptr
  void* k_dgain;
  float* partial;      // [parts][2][d]: the blocks' sums for the gains of Q and K
  int parts;
  int device;
};
constexpr int kNormParts = 152 * 2;  // blocks of the gradient at most
cudaError_t launch_norm_rotary(const NormArgs& a, cudaStream_t stream);

// Attention over rows that several sequences share (attn_fwd_paged_shared): two lines of
// units, one over the groups' shared rows, one over the sequences' own, side by side on
// the GPU's SMs in one launch; then a join of every row's parts.
enum : int { kNoLine = 0, kSharedLine = 1, kOwnLine = 2 };

// Where a row's part of one line is.
struct alignas(16) PagedRecord {
  float ref, mass;  // rest = 0: of the result in the row buffer
  int part;         // rest > 0: slot of its first piece; the next CTAs' follow
  int rest;         // key tiles after the first piece
};

struct PagedShare {
  int line;                // of these arguments
  const int* cu_groups;    // device [groups + 1]: sequences [cu_groups[g], cu_groups[g + 1]) share rows
  const int* prefix;       // device [B]: rows that a sequence shares with its group
  int groups;
  int sms;                 // that the two lines divide between them
  int ctas[2];             // that each has room for at most
  int unit_tokens[2];
  int tile_time[2];        // relative time of a key tile in a line's kernel
  PagedRecord* rec;        // this line's [total, Hq]
  long long rows_at;       // this line's row buffer [total, Hq, d], floats from part_o on
};

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
  PagedShare share;         // share.line = kNoLine: attn_fwd_paged
};
constexpr int kPagedDecodeCols = 32;  // query columns of the decode kernel at most
constexpr int kPagedRows = 256;       // unit rows of the forward kernel: two query tiles
cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t stream);
cudaError_t launch_paged_fwd(const PagedArgs& a, cudaStream_t stream);
// Joins the pieces of the units that ended up on several CTAs.
cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t stream);
// The two lines behind shared rows (paged_shared.cuh), arguments by line, then the join of
// every row's parts (paged_join.cu).
struct PagedLines {
  PagedArgs line[2];
};
cudaError_t launch_paged_shared_bf16_64(const PagedLines& a, cudaStream_t stream);
cudaError_t launch_paged_shared_bf16_128(const PagedLines& a, cudaStream_t stream);
cudaError_t launch_paged_shared_f16_64(const PagedLines& a, cudaStream_t stream);
cudaError_t launch_paged_shared_f16_128(const PagedLines& a, cudaStream_t stream);
cudaError_t launch_paged_join(const PagedArgs& shared, const PagedArgs& own, cudaStream_t stream);

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
