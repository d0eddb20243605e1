// Paged key/value cache: parameter blocks and addressing shared by the append,
// gather and attention kernels.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace fm {

// Device view of flashmask_pages.  Rows (one token of one head) are numbered
// page-major: row = (page * Hkv + head) * page_size + slot.
struct Pages {
  uint8_t *k, *v;             // rows of row_bytes
  uint32_t *k_scales, *v_scales;  // bits 4: (scale, minimum) of each row as two bf16; else null
  const int32_t* table;
  int64_t table_stride;
  int B, table_width, num_pages, page_shift, Hkv, d, bits;
  int row_bytes;              // 2 d, or d / 2 with 4 bits
  int* status;
};

struct AppendParams {
  Pages pg;
  const __nv_bfloat16 *q, *k, *v;
  int64_t qs[3], ks[3], vs[3];  // {batch, token, head} strides in elements
  __nv_bfloat16* q_out;
  const int32_t *start, *counts, *positions;
  const float *cos, *sin;
  int N, Hq, rot, table_len, interleaved;
};

struct GatherParams {
  Pages pg;
  const int32_t* lens;
  int N;
  __nv_bfloat16 *k, *v;
  int wide;  // k and v are 32-byte aligned
};

// Division of numbers below 2^31 by a constant of the call: x / d = (x * m) >> 32 >> s with m = ceil(2^(32 + s) / d),
// exact for x < 2^31 when 2^s < d <= 2^(s+1) (the error x (m d - 2^(32+s)) / (d 2^(32+s)) stays below 1 / d).
struct FastDiv {
  uint32_t m, s;
  __device__ __forceinline__ int operator()(int x) const { return m ? (int)(__umulhi((uint32_t)x, m) >> s) : x; }
};
inline FastDiv fast_div(int d) {
  FastDiv f{0, 0};
  if (d <= 1) return f;
  while ((2ull << f.s) < (uint64_t)d) ++f.s;
  f.m = (uint32_t)(((1ull << (32 + f.s)) + d - 1) / d);
  return f;
}

// How the work is divided: equal runs of tiles per warp (items may be cut), whole items per warp, or one
// CTA per item.
enum PagedMode { kPagedSplit = 0, kPagedWhole = 1, kPagedCoop = 2 };

// Warps of an attention CTA (one per SM).  Registers allow 8 at 255 a thread and 12 at 168; the rings of
// tiles in shared memory allow 12 tiles of 16 KiB (two for each of 6 warps, three for 4 with their rows of Q), 24 of
// 8.5 KiB.  Blocks of 32 rows are for bf16 alone.
__host__ __device__ constexpr int paged_warps(int d, int bits, int rows) {
  return bits == 16 ? (rows == 32 ? 4 : 6) : (rows == 16 ? 8 : 12);
}

struct PagedAttnParams {
  Pages pg;
  const __nv_bfloat16* q;
  int64_t qs[3];
  const int32_t *lens, *start;
  const int32_t *lts, *lte, *uts, *ute;
  int Nq, Hq, Hm, Nm, G, causal;
  float scale_log2;  // scale * log2(e)
  __nv_bfloat16* o;
  float* lse;
  // work: groups (a sequence, or a sequence and KV head with per-head masks) of `mult` items of `rows` rows
  int per_head, n_groups, mult, n_rb, rows, tile_keys;
  FastDiv div_g, div_hkv, div_rb, div_mult;  // by G, Hkv, n_rb, mult
  uint32_t q_bytes, table_bytes;  // to prefetch (0: not in one piece)
  int mode;                 // kPaged*: how the work is divided
  // plan (with mask vectors): visible tiles of each group, row-visibility words of each key
  const int* counts;        // [n_groups]
  const int* list;          // [n_groups, list_stride]: tile << 1 | some pair hidden
  int list_stride;
  const uint32_t* words;    // [n_groups, n_words, words_stride]: bit i = row 32 w + i of the KV head sees the key
  int n_words;
  int64_t words_stride;
  // partial sums of cut items: two slots per run (worker: a warp)
  float* part;              // [2 workers, rows, d]
  float2* stat;             // [2 workers, rows]: running maximum, sum
  int* meta;                // [workers, 8]: the item that begins in a run and goes on in the next
  uint64_t wait_limit_ns;
};

// What the plan kernels write: counts, list and words as above, and the class of every tile
// (0 no pair visible, 1 some pair hidden, 2 all visible), [n_groups, list_stride].
struct PlanOut {
  int *counts, *list;
  uint32_t* words;
  uint8_t* flags;
};

constexpr int kPagedMaxCtas = 160;

static __device__ __noinline__ void record_bounds(int* status) { atomicCAS(status, 0, kDevErrBounds); }

// Page of position j of sequence b; -1 (recorded) for an entry out of range.
// j must lie in [0, table_width * page_size).
__device__ __forceinline__ int page_of(const Pages& pg, int b, int j) {
  const int id = pg.table[b * pg.table_stride + (j >> pg.page_shift)];
  if ((unsigned)id < (unsigned)pg.num_pages) return id;
  record_bounds(pg.status);
  return -1;
}

__device__ __forceinline__ int64_t row_of(const Pages& pg, int page, int head, int j) {
  return (((int64_t)page * pg.Hkv + head) << pg.page_shift) + (j & ((1 << pg.page_shift) - 1));
}

// Cached keys of sequence b: a length beyond the table is recorded and cut.
__device__ __forceinline__ int checked_len(const Pages& pg, const int32_t* lens, int b) {
  const int n = lens[b];
  const int64_t cap = (int64_t)pg.table_width << pg.page_shift;
  if (n < 0 || n > cap) record_bounds(pg.status);
  return n < 0 ? 0 : n > cap ? (int)cap : n;
}

cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t st);
cudaError_t launch_paged_gather(const GatherParams& p, cudaStream_t st);
int paged_tile_keys(int d, int bits);
// Plan (when p.list is set), attention and merge.
cudaError_t launch_paged_attention(const PagedAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                                   const PlanOut& plan, cudaStream_t st);

}  // namespace fm
