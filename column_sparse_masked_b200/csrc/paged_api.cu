// Host side of the paged-cache entry points: argument checks and launches.
#include <climits>
#include <cmath>

#include "api_internal.h"
#include "common.cuh"
#include "launchers.h"
#include "paged.cuh"

namespace fm {
namespace {

int check_pages(const flashmask_pages* pg) {
  if (!pg) return FLASHMASK_ERR_INVALID_ARG;
  if (pg->B < 0 || pg->table_width < 0 || pg->num_pages < 0 || pg->Hkv <= 0 || pg->table_stride < 0)
    return FLASHMASK_ERR_INVALID_ARG;
  if (pg->bits != 16 && pg->bits != 4) return FLASHMASK_ERR_UNSUPPORTED;
  if (pg->d != 64 && pg->d != 128) return FLASHMASK_ERR_UNSUPPORTED;
  const int ps = pg->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0) return FLASHMASK_ERR_UNSUPPORTED;
  // positions, and row numbers of the whole cache, are 32-bit
  if ((int64_t)pg->table_width * ps > (1 << 30)) return FLASHMASK_ERR_UNSUPPORTED;
  if ((int64_t)pg->num_pages * pg->Hkv > (int64_t)INT_MAX / ps) return FLASHMASK_ERR_UNSUPPORTED;
  if (pg->num_pages > 0 && (!pg->k || !pg->v)) return FLASHMASK_ERR_INVALID_ARG;
  if (pg->bits == 4 && pg->num_pages > 0 && (!pg->k_scales || !pg->v_scales)) return FLASHMASK_ERR_INVALID_ARG;
  if (pg->B > 0 && pg->table_width > 0 && !pg->table) return FLASHMASK_ERR_INVALID_ARG;
  if (!aligned16(pg->k) || !aligned16(pg->v) || !aligned16(pg->k_scales) || !aligned16(pg->v_scales))
    return FLASHMASK_ERR_ALIGN;
  return FLASHMASK_OK;
}

// Strided rows: pointer and strides keep every 16-byte load of a row aligned.
int check_rows(const void* p, const int64_t* strides) {
  if (!p) return FLASHMASK_ERR_INVALID_ARG;
  if (!aligned16(p)) return FLASHMASK_ERR_ALIGN;
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0) return FLASHMASK_ERR_INVALID_ARG;
    if (strides[i] % 8 != 0) return FLASHMASK_ERR_ALIGN;
  }
  return FLASHMASK_OK;
}

Pages device_pages(const flashmask_pages& pg, const DeviceInfo& di) {
  Pages p{};
  p.k = static_cast<uint8_t*>(pg.k);
  p.v = static_cast<uint8_t*>(pg.v);
  p.k_scales = static_cast<uint32_t*>(pg.k_scales);
  p.v_scales = static_cast<uint32_t*>(pg.v_scales);
  p.table = pg.table;
  p.table_stride = pg.table_stride;
  p.B = pg.B;
  p.table_width = pg.table_width;
  p.num_pages = pg.num_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < pg.page_size) ++p.page_shift;
  p.Hkv = pg.Hkv;
  p.d = pg.d;
  p.bits = pg.bits;
  p.row_bytes = pg.bits == 4 ? pg.d / 2 : 2 * pg.d;
  p.status = di.status;
  return p;
}

int check_paged_rows(const flashmask_pages* pg, const flashmask_paged_rows* r) {
  FM_TRY(check_pages(pg));
  if (!r) return FLASHMASK_ERR_INVALID_ARG;
  if (r->Nq < 0 || r->Hq <= 0 || r->Hq % pg->Hkv != 0) return FLASHMASK_ERR_INVALID_ARG;
  if (r->causal != 0 && r->causal != 1) return FLASHMASK_ERR_INVALID_ARG;
  FM_TRY(check_masks(r->lts, r->lte, r->uts, r->ute));
  if (r->lts || r->uts) {
    if (r->Nm < 0 || (r->Hm != 1 && r->Hm != r->Hq)) return FLASHMASK_ERR_INVALID_ARG;
  }
  // work items are numbered in 32 bits (by division: the products may pass 64)
  if ((int64_t)pg->B * r->Nq > INT_MAX / 4 / r->Hq) return FLASHMASK_ERR_UNSUPPORTED;
  const int64_t units = ((int64_t)pg->table_width * pg->page_size + 31) / 32 + 2;
  const int64_t blocks = ((int64_t)r->Nq * (r->Hq / pg->Hkv) + 7) / 8;
  if (blocks * pg->Hkv * pg->B > INT_MAX / 2 / units) return FLASHMASK_ERR_UNSUPPORTED;
  return FLASHMASK_OK;
}

// Work split and workspace of an attention call.
struct PagedLayout {
  int plan, per_head, n_groups, mult, n_rb, rows, tile_keys, n_words, mode;
  int64_t keys;  // capacity of the table, in whole tiles
  size_t part, stat, meta, counts, list, words, flags, bytes;
};

constexpr int kSms = 148;  // of a B200: workspace sizes must not depend on the current device

PagedLayout paged_layout(const flashmask_pages& pg, const flashmask_paged_rows& r) {
  PagedLayout L{};
  const int64_t R = (int64_t)r.Nq * (r.Hq / pg.Hkv);
  L.tile_keys = paged_tile_keys(pg.d, pg.bits);
  L.n_words = (int)((R + 31) / 32);
  const int64_t cap = (int64_t)pg.table_width * pg.page_size;
  L.keys = (cap + L.tile_keys - 1) / L.tile_keys * L.tile_keys;
  const int64_t tiles = L.keys / L.tile_keys;
  const bool masked = r.lts || r.uts;
  auto blocks = [&](int rows) { return (R + rows - 1) / rows; };
  // Rows of a block.  A block reads its keys once, so the fewest blocks read least; but blocks of 32 rows run
  // with 4 warps an SM, whose 128 accumulators a thread leave no room in 255 registers (156 bytes of stores and 144 of
  // loads are spilled at d = 128), and a long way through cold instructions.  bf16, 32 rows over 32 sequences of 4K keys: blocks
  // of 32 take 145 us, of 16 188, of 8 331; over 8 sequences 59, 48 and 61; with masks that hide three
  // quarters 70, 61 and 76 over 32, 34, 30 and 30 over 8.  In 4 bits the codes' conversion counts and not the bytes: 32
  // rows over 32 sequences take 125 us in blocks of 16, 153 in blocks of 8 and 167 in blocks of 32.
  const bool wide = pg.bits == 16 && !masked && blocks(32) * pg.B * pg.Hkv * tiles >= 24 * 4 * kSms;  // 24 tiles a warp
  L.rows = R <= 8 ? 8 : R <= 16 || !wide ? 16 : 32;
  // Whole items where cutting has nothing to give, and no second kernel.  One per CTA if the table bounds them to
  // four tiles a warp and the device takes them all at once, in the smallest blocks of rows for which it does (4
  // sequences of 103 keys and 32 rows: 10.7 us in blocks of 32, 6.8 in blocks of 8); masks are then read with the
  // tiles, without a plan, and hidden tiles with them.  8 KV heads of 4 sequences of 700 keys: 9.3 us, cut 10.8, with
  // masks 12.0 and 14.1.  In 4 bits a round of tiles takes 3.4 us at d = 128, and an item that leaves SMs idle for
  // more than 1.25 rounds (2 with masks, whose plan counts too) is better cut: 32 items of 3000 keys 20 us, cut 14,
  // but 144 of 2000 keys 16.1 and 18.1.  One after another per warp if the table bounds them to eight tiles (20
  // sequences of 110 keys: 10 us, 16 with four waves of CTAs).  Else cut, unless two waves of CTAs take items of some twelve tiles (29 sequences
  // of 619 keys with masks in 4 bits: 17.2 us, cut 19.6; 36 of 1300 keys 24 and 20).
  L.mode = tiles <= 8 ? kPagedWhole : kPagedSplit;
  for (int waves = 1; waves <= (tiles <= 8 ? 1 : 2) && L.mode != kPagedCoop; ++waves)
    for (int rows = 8; rows <= (pg.bits == 16 ? 32 : 16) && L.mode != kPagedCoop; rows *= 2) {
      const int warps = paged_warps(pg.d, pg.bits, rows);
      const int64_t items = blocks(rows) * pg.B * pg.Hkv;
      const int64_t most = waves == 1 ? 4 * warps : pg.bits == 16 ? 2 * warps : warps;
      if (items > waves * kSms || tiles > most) continue;
      if (waves == 1 && pg.bits == 4 && 4 * (kSms - items) * tiles * pg.d > (masked ? 8 : 5) * 128 * kSms * warps) continue;
      L.mode = kPagedCoop;
      L.rows = rows;
    }
  L.n_rb = (int)blocks(L.rows);
  const int warps = paged_warps(pg.d, pg.bits, L.rows);
  L.plan = masked && tiles > 0 && L.mode != kPagedCoop;
  L.per_head = L.plan && r.Hm > 1;
  L.n_groups = L.per_head ? pg.B * pg.Hkv : pg.B;
  L.mult = L.per_head ? L.n_rb : pg.Hkv * L.n_rb;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t o = off; off = ws_align(off + bytes); return o; };
  if (L.mode == kPagedSplit) {
    const size_t slots = (size_t)2 * kPagedMaxCtas * warps;
    L.part = take(slots * L.rows * pg.d * 4);
    L.stat = take(slots * L.rows * 8);
    L.meta = take(slots / 2 * 8 * 4);
  }
  if (L.plan) {
    L.counts = take((size_t)L.n_groups * 4);
    L.list = take((size_t)L.n_groups * tiles * 4);
    L.words = take((size_t)L.n_groups * L.n_words * L.keys * 4);
    L.flags = take((size_t)L.n_groups * tiles);
  }
  L.bytes = off > 0 ? off : 256;
  return L;
}

// Map over the rows of all pages as {64 values, row, 64-value part}: a box holds box_rows whole
// rows, part by part, with 128-byte swizzle.
int make_rows_map(CUtensorMap* m, const void* ptr, int64_t rows, int d, int box_rows) {
  auto enc = encode_fn();
  if (!enc) return FLASHMASK_ERR_CUDA;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(d / 64)};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)(d / 64)};
  cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FLASHMASK_OK : cuda_status(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" {

int flashmask_paged_append(const flashmask_pages* pages, const flashmask_append* tokens, void* stream) {
  NvtxRange nvtx("flashmask_paged_append");
  FM_TRY(check_pages(pages));
  if (!tokens) return FLASHMASK_ERR_INVALID_ARG;
  const flashmask_append& t = *tokens;
  if (t.N < 0 || t.table_len < 0 || (t.interleaved != 0 && t.interleaved != 1)) return FLASHMASK_ERR_INVALID_ARG;
  if (t.q && t.Hq <= 0) return FLASHMASK_ERR_INVALID_ARG;
  if (t.rot < 0 || t.rot > pages->d || t.rot % 16 != 0) return FLASHMASK_ERR_UNSUPPORTED;
  // rows are numbered in 32 bits (by division: the product may pass 64)
  if ((int64_t)pages->B * t.N > INT_MAX / ((t.q ? t.Hq : 0) + 2 * (int64_t)pages->Hkv)) return FLASHMASK_ERR_UNSUPPORTED;
  if ((int64_t)pages->B * t.N == 0) return FLASHMASK_OK;
  if (!t.start) return FLASHMASK_ERR_INVALID_ARG;
  if (t.rot > 0 && (!t.cos || !t.sin)) return FLASHMASK_ERR_INVALID_ARG;
  if (!aligned16(t.cos) || !aligned16(t.sin)) return FLASHMASK_ERR_ALIGN;
  FM_TRY(check_rows(t.k, t.k_strides));
  FM_TRY(check_rows(t.v, t.v_strides));
  if (t.q) {
    FM_TRY(check_rows(t.q, t.q_strides));
    if (!t.q_out) return FLASHMASK_ERR_INVALID_ARG;
    if (!aligned16(t.q_out)) return FLASHMASK_ERR_ALIGN;
  }
  DeviceInfo di;
  FM_TRY(current_device(&di));
  AppendParams p{};
  p.pg = device_pages(*pages, di);
  p.q = static_cast<const __nv_bfloat16*>(t.q);
  p.k = static_cast<const __nv_bfloat16*>(t.k);
  p.v = static_cast<const __nv_bfloat16*>(t.v);
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = t.q_strides[i];
    p.ks[i] = t.k_strides[i];
    p.vs[i] = t.v_strides[i];
  }
  p.q_out = static_cast<__nv_bfloat16*>(t.q_out);
  p.start = t.start;
  p.counts = t.counts;
  p.positions = t.positions;
  p.cos = t.cos;
  p.sin = t.sin;
  p.N = t.N;
  p.Hq = t.Hq;
  p.rot = t.rot;
  p.table_len = t.table_len;
  p.interleaved = t.interleaved;
  FM_CUDA(launch_paged_append(p, static_cast<cudaStream_t>(stream)));
  return FLASHMASK_OK;
}

size_t flashmask_paged_attention_workspace_size(const flashmask_pages* pages, const flashmask_paged_rows* rows) {
  if (check_paged_rows(pages, rows) != FLASHMASK_OK) return 0;
  return paged_layout(*pages, *rows).bytes;
}

int flashmask_paged_attention(const flashmask_pages* pages, const flashmask_paged_rows* rows, void* workspace,
                              size_t workspace_bytes, void* stream) {
  NvtxRange nvtx("flashmask_paged_attention");
  FM_TRY(check_paged_rows(pages, rows));
  const flashmask_paged_rows& r = *rows;
  if ((int64_t)pages->B * r.Nq == 0) return FLASHMASK_OK;
  if (!r.lens || !r.o || !r.lse) return FLASHMASK_ERR_INVALID_ARG;
  FM_TRY(check_rows(r.q, r.q_strides));
  if (!aligned16(r.o) || !aligned16(r.lse)) return FLASHMASK_ERR_ALIGN;
  const PagedLayout L = paged_layout(*pages, r);
  FM_TRY(check_ws(workspace, workspace_bytes, L.bytes));
  DeviceInfo di;
  FM_TRY(current_device(&di));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PagedAttnParams p{};
  p.pg = device_pages(*pages, di);
  p.q = static_cast<const __nv_bfloat16*>(r.q);
  for (int i = 0; i < 3; ++i) p.qs[i] = r.q_strides[i];
  p.lens = r.lens;
  p.start = r.start;
  p.lts = r.lts;
  p.lte = r.lte;
  p.uts = r.uts;
  p.ute = r.ute;
  const bool masked = r.lts || r.uts;
  p.Nq = r.Nq;
  p.Hq = r.Hq;
  p.Hm = masked ? r.Hm : 1;
  p.Nm = masked ? r.Nm : 0;
  p.G = r.Hq / pages->Hkv;
  p.causal = r.causal;
  const float scale = r.scale > 0.f ? r.scale : 1.0f / std::sqrt((float)pages->d);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.o = static_cast<__nv_bfloat16*>(r.o);
  p.lse = r.lse;
  p.per_head = L.per_head;
  p.n_groups = L.n_groups;
  p.mult = L.mult;
  p.n_rb = L.n_rb;
  p.rows = L.rows;
  p.tile_keys = L.tile_keys;
  p.div_g = fast_div(p.G);
  p.div_hkv = fast_div(pages->Hkv);
  p.div_rb = fast_div(L.n_rb);
  p.div_mult = fast_div(L.mult);
  {
    const int64_t row = (int64_t)r.Hq * pages->d, batch = row * r.Nq, all = batch * pages->B * 2;
    const bool dense = (r.Hq == 1 || r.q_strides[2] == pages->d) && (r.Nq == 1 || r.q_strides[1] == row) &&
                       (pages->B == 1 || r.q_strides[0] == batch);
    p.q_bytes = dense && all < (1 << 20) ? (uint32_t)all : 0;
    const int64_t table = (int64_t)pages->B * pages->table_width * 4;
    const bool whole = pages->B == 1 || pages->table_stride == pages->table_width;
    p.table_bytes = whole && table < (1 << 20) ? (uint32_t)table : 0;
  }
  p.mode = L.mode;
  p.part = reinterpret_cast<float*>(ws + L.part);
  p.stat = reinterpret_cast<float2*>(ws + L.stat);
  p.meta = reinterpret_cast<int*>(ws + L.meta);
  PlanOut plan{};
  if (L.plan) {
    p.counts = plan.counts = reinterpret_cast<int*>(ws + L.counts);
    p.list = plan.list = reinterpret_cast<int*>(ws + L.list);
    p.words = plan.words = reinterpret_cast<uint32_t*>(ws + L.words);
    plan.flags = ws + L.flags;
    p.list_stride = (int)(L.keys / L.tile_keys);
    p.n_words = L.n_words;
    p.words_stride = L.keys;
  }
  p.wait_limit_ns = wait_limit_ns();
  CUtensorMap tk{}, tv{};
  if (pages->bits == 16 && pages->num_pages > 0) {
    const int box = pages->page_size < L.tile_keys ? pages->page_size : L.tile_keys;
    const int64_t rows = (int64_t)pages->num_pages * pages->Hkv * pages->page_size;
    FM_TRY(make_rows_map(&tk, pages->k, rows, pages->d, box));
    FM_TRY(make_rows_map(&tv, pages->v, rows, pages->d, box));
  }
  const int grid = L.mode == kPagedCoop ? L.n_groups * L.mult : persistent_grid(kPagedMaxCtas, di.sm_count);
  FM_CUDA(launch_paged_attention(p, tk, tv, grid, plan, static_cast<cudaStream_t>(stream)));
  return FLASHMASK_OK;
}

int flashmask_paged_gather(const flashmask_pages* pages, const int32_t* lens, int32_t N, void* k, void* v,
                           void* stream) {
  NvtxRange nvtx("flashmask_paged_gather");
  FM_TRY(check_pages(pages));
  if (N < 0) return FLASHMASK_ERR_INVALID_ARG;
  if ((int64_t)pages->B * N > INT_MAX / pages->Hkv) return FLASHMASK_ERR_UNSUPPORTED;
  if ((int64_t)pages->B * N == 0) return FLASHMASK_OK;
  if (!lens || !k || !v) return FLASHMASK_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return FLASHMASK_ERR_ALIGN;
  DeviceInfo di;
  FM_TRY(current_device(&di));
  GatherParams p{};
  p.pg = device_pages(*pages, di);
  p.lens = lens;
  p.N = N;
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  p.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  FM_CUDA(launch_paged_gather(p, static_cast<cudaStream_t>(stream)));
  return FLASHMASK_OK;
}

}  // extern "C"
