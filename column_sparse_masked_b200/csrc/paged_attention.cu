// Attention of a few rows per sequence over a paged key/value cache.
//
// The rows of one KV head (new tokens x the q-heads that share it) read every
// visible key and value once and do 4 d FLOP with each: bytes bound it as long
// as a block holds at most some 32 rows, so the design is about keeping the
// memory system full and the work even.
//
//  - Work.  An item is (sequence, KV head, block of 8, 16 or 32 rows); its
//    units are its tiles of 32 or 64 keys.  All units are laid end to end and
//    every CTA (one per SM) takes an equal run of them, whatever the lengths
//    of the sequences: a run may end one item, hold several and begin another.
//    An item inside one run is finished there; one that is cut leaves fp32
//    partial sums, which a second kernel joins in a fixed order (no atomics:
//    equal calls give equal bits).  Lengths are device data and the grid does
//    not depend on them, so a captured graph serves growing sequences.
//  - Masks.  With mask vectors a plan kernel runs first: it turns each key's
//    four boundaries into one bit per row, and lists the tiles that some row
//    sees, so hidden tiles are neither read nor counted as work.
//  - Loads.  One warp looks pages up and fills a ring of tiles in shared
//    memory by TMA (swizzled boxes for bf16, plain bulk copies for 4 bits);
//    the ring spans items, so the loads never pause at an item's end.
//  - Products.  Tensor cores with the keys as the M side (mma m16n8k16): S^T =
//    K Q^T and O^T = V^T P^T need only 8 row columns, where the usual
//    orientation pads the rows to 16.  mma.sync and not tcgen05: rows are
//    few, P never leaves registers, and the tensor pipe is far from the bound.
//    Each warp keeps its own running maximum and sums over its tiles; warps
//    meet once per item.
//  - 4 bits.  A row's codes enter the products as the integers code - 8 (exact
//    in bf16); scale and minimum are applied to sums in fp32:
//      q.k = s (q.(c - 8)) + (m + 8 s) sum(q)
//      o   = sum (p s)(c - 8) + sum p (m + 8 s)
//    The contraction may run over the head's values in any order as long as
//    both sides agree, so each thread takes whole 16-byte pieces of code rows.
#include <cuda_bf16.h>

#include "launchers.h"
#include "paged.cuh"
#include "sm100_primitives.cuh"

namespace fm {
namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr int kMetaInts = 8;

// ---------------------------------------------------------------------------
// work: groups of items with the same number of tiles, and a CTA's run of units
// ---------------------------------------------------------------------------
__device__ __forceinline__ int group_batch(const PagedAttnParams& p, int g) { return p.per_head ? g / p.pg.Hkv : g; }

// Keys of sequence b that its rows can see at all, and its first row's position.
__device__ __forceinline__ int key_bound(const PagedAttnParams& p, int b, int* len_out, int64_t* first) {
  const int len = checked_len(p.pg, p.lens, b);
  const int64_t st = p.start ? (int64_t)p.start[b] : (int64_t)len - p.Nq;
  *len_out = len;
  *first = st;
  const int64_t hi = p.causal ? min((int64_t)len, st + p.Nq) : (int64_t)len;
  return hi > 0 ? (int)hi : 0;
}

__device__ __forceinline__ int tiles_of(const PagedAttnParams& p, int g) {
  if (p.counts) return p.counts[g];
  int len;
  int64_t st;
  return (key_bound(p, group_batch(p, g), &len, &st) + p.tile_keys - 1) / p.tile_keys;
}

// A run of units, walked segment by segment (a segment: tiles [t, t + n) of
// one item).  Every warp of the CTA walks it the same way.
struct Walk {
  int g, in, t, T;  // group, item in the group, first tile, tiles of the group's items
  int left;         // units left in the run
  int n;            // tiles of this segment
  __device__ __forceinline__ bool next(const PagedAttnParams& p) {
    left -= n;
    if (left <= 0) return false;
    t = 0;
    if (++in == p.mult) {
      in = 0;
      do {
        ++g;
        T = tiles_of(p, g);
      } while (T == 0);
    }
    n = min(T, left);
    return true;
  }
};

struct Item {
  int b, kvh, row0;
};
__device__ __forceinline__ Item item_of(const PagedAttnParams& p, int g, int in, int rows_per_item) {
  Item it;
  it.b = group_batch(p, g);
  const int rb = in % p.n_rb;
  it.kvh = p.per_head ? g % p.pg.Hkv : in / p.n_rb;
  it.row0 = rb * rows_per_item;
  return it;
}

// ---------------------------------------------------------------------------
// tiles and shared memory
// ---------------------------------------------------------------------------
template <int D, int BITS, int NT>
struct Cfg {
  static constexpr int kKT = BITS == 16 && D == 128 ? 32 : 64;  // keys of a tile
  static constexpr int kRows = 8 * NT;
  static constexpr int kWarps = BITS == 16 ? (NT == 4 ? 4 : NT == 2 ? 5 : 6) : (NT == 4 ? 4 : NT == 2 ? 7 : 8);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr bool kQShared = NT == 4;                     // Q fragments in shared memory
  static constexpr int kRowBytes = BITS == 16 ? 2 * D : D / 2;
  static constexpr int kHalf = kKT * kRowBytes;                 // K or V part of a stage
  static constexpr int kScales = BITS == 4 ? kKT * 4 : 0;
  static constexpr int kStage = 2 * kHalf + 2 * kScales;
  static constexpr int kStride = D + 4;                         // floats between rows of the merge buffer
  static constexpr int kMerge = kWarps * kRows * kStride * 4;
  static constexpr int kQBytes = kQShared ? (D / 16) * NT * 32 * 8 : 0;
  static constexpr int kPerStage = kStage + 16 + 8;             // + header, barrier
  static constexpr int kFixed = kMerge + kQBytes + 3 * kWarps * kRows * 4 + kRows * 4 + 1024 + 256;
  // Every warp has a ring of its own, which it fills and empties itself: a stage is refilled by the warp
  // that has just read it, so nothing waits for another warp between the ends of items.
  static constexpr int kFit = (225 * 1024 - kFixed) / kPerStage / kWarps;
  static constexpr int kDepth = kFit > 4 ? 4 : kFit;
  static constexpr int kStages = kWarps * kDepth;
  static constexpr int kSmem = kFixed + kStages * kPerStage;
  static constexpr int kBoxes = kKT / 16;                       // copies of a tile's rows at most
  static_assert(kDepth >= 2, "ring too short");
};

template <int D, int BITS, int NT>
struct Smem {
  using C = Cfg<D, BITS, NT>;
  uint8_t* stage;      // kStages x kStage, 1024-byte aligned for the swizzle
  int4* hdr;           // kStages: first key, some pair hidden, valid boxes
  uint64_t* full;      // kStages
  float* merge;        // kWarps x kRows x kStride
  uint2* q;            // Q fragments (kQShared)
  float *m, *l, *c;    // kWarps x kRows
  float* qsum;         // kRows
  int* abort;
  __device__ __forceinline__ explicit Smem(uint8_t* raw) {
    const uint32_t a = smem_addr(raw);
    uint8_t* x = raw + ((1024u - (a & 1023u)) & 1023u);
    stage = x; x += C::kStages * C::kStage;
    merge = reinterpret_cast<float*>(x); x += C::kMerge;
    q = reinterpret_cast<uint2*>(x); x += C::kQBytes;
    hdr = reinterpret_cast<int4*>(x); x += C::kStages * 16;
    full = reinterpret_cast<uint64_t*>(x); x += C::kStages * 8;
    m = reinterpret_cast<float*>(x); x += C::kWarps * C::kRows * 4;
    l = reinterpret_cast<float*>(x); x += C::kWarps * C::kRows * 4;
    c = reinterpret_cast<float*>(x); x += C::kWarps * C::kRows * 4;
    qsum = reinterpret_cast<float*>(x); x += C::kRows * 4;
    abort = reinterpret_cast<int*>(x);
  }
};

// ---------------------------------------------------------------------------
// warp-level building blocks
// ---------------------------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Box of rows of one head in one page: [D/64][rows][64 values] in shared memory.
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %3}], [%2];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(row)
      : "memory");
}

// Codes at nibbles i and i + 4 of each half of x as the bf16 pair (code - 8):
// 0x4300 + code is 128 + code, and 128 + code - 136 is exact.
__device__ __forceinline__ uint32_t centred(uint32_t x, int i) {
  uint32_t y;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(y) : "r"(x >> (4 * i)));  // (x & a) | b
  asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(0x43084308u));
  return y;
}

// Key of slot s (0..7) of an 8-key block in the 4-bit layout: a thread's four
// keys of V must be spread so that code rows (64 or 32 bytes) meet in few
// banks, and the rows of K next to one another in a load must have opposite
// parity.  Any permutation gives the same sums.
__device__ __forceinline__ int slot_key(int s) { return (s & 1) ? 4 + ((s >> 1) ^ 1) : s >> 1; }

// Largest value over the 8 lanes that share lane % 4.
__device__ __forceinline__ float max8(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum8(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Fills one warp's ring: the tiles of the CTA's run that are the warp's, in
// order, across segments.  Pages are looked up for 32 of them at a time, one
// by each lane.
template <int D, int BITS, int NT>
struct Issuer {
  using C = Cfg<D, BITS, NT>;
  Walk w;
  int k;        // the warp's next tile that is not in the batch, in the segment
  int x, nb;    // next tile of the batch, and its size
  int issued;
  bool more;
  int kvh;
  int j0, flags, page[C::kBoxes];  // a lane's tile: first key, masked | valid boxes << 1, pages

  __device__ __forceinline__ void batch(const PagedAttnParams& p) {
    constexpr int KT = C::kKT;
    const int lane = threadIdx.x & 31, box_shift = min(p.pg.page_shift, KT == 32 ? 5 : 6);
    const int boxes = KT >> box_shift;
    const Item it = item_of(p, w.g, w.in, C::kRows);
    kvh = it.kvh;
    int len;
    int64_t first;
    const int hi = key_bound(p, it.b, &len, &first);
    nb = min(32, (w.n - k + C::kWarps - 1) / C::kWarps);
    x = 0;
    j0 = 0;
    int masked = 0, valid = 0;
#pragma unroll
    for (int i = 0; i < C::kBoxes; ++i) page[i] = 0;
    if (lane < nb) {
      const int t = w.t + k + lane * C::kWarps;
      if (p.list) {
        const int e = p.list[(int64_t)w.g * p.list_stride + t];
        j0 = (e >> 1) * KT;
        masked = e & 1;
      } else {
        j0 = t * KT;
        // keys that every row of the item sees
        const int64_t all = p.causal ? min((int64_t)len, first + it.row0 / p.G + 1) : (int64_t)len;
        masked = (int64_t)j0 + KT > all;
      }
#pragma unroll
      for (int i = 0; i < C::kBoxes; ++i) {
        const int j = j0 + (i << box_shift);
        if (i < boxes && j < hi) {
          page[i] = page_of(p.pg, it.b, j);
          if (page[i] >= 0) valid |= 1 << i;
        }
      }
      if (valid != (1 << boxes) - 1) masked = 1;
    }
    flags = masked | (valid << 1);
    k += nb * C::kWarps;
  }

  __device__ __forceinline__ void start(const PagedAttnParams& p, const Walk& wk, int warp) {
    w = wk;
    k = warp;
    issued = 0;
    x = nb = 0;
    more = true;
  }

  __device__ __forceinline__ void issue(const PagedAttnParams& p, const CUtensorMap* tk, const CUtensorMap* tv,
                                        const Smem<D, BITS, NT>& sm, int warp) {
    if (x == nb) {
      if (!more) return;
      while (k >= w.n) {
        k -= w.n;
        if (!w.next(p)) {
          more = false;
          x = nb = 0;
          return;
        }
      }
      batch(p);
    }
    constexpr int KT = C::kKT;
    const int lane = threadIdx.x & 31, box_shift = min(p.pg.page_shift, KT == 32 ? 5 : 6);
    const int tj = __shfl_sync(0xffffffffu, j0, x), f = __shfl_sync(0xffffffffu, flags, x);
    const int bx = BITS == 16 ? lane >> 1 : lane >> 2;  // a copy per lane
    int pid = 0;
#pragma unroll
    for (int i = 0; i < C::kBoxes; ++i) {
      const int v = __shfl_sync(0xffffffffu, page[i], x);
      if (i == bx) pid = v;
    }
    ++x;
    const int stage = warp * C::kDepth + issued % C::kDepth;
    ++issued;
    uint64_t* bar = &sm.full[stage];
    if (lane == 0) {
      sm.hdr[stage] = make_int4(tj, f & 1, f >> 1, 0);
      mbar_arrive_expect_tx(bar, (uint32_t)(__popc(f >> 1) << box_shift) * (2 * C::kRowBytes + (BITS == 4 ? 8 : 0)));
    }
    __syncwarp();
    if (bx < C::kBoxes && ((f >> (1 + bx)) & 1)) {
      const int64_t row = row_of(p.pg, pid, kvh, tj + (bx << box_shift));
      uint8_t* st = sm.stage + stage * C::kStage;
      if (BITS == 16) {
        tma_load_rows(st + (lane & 1) * C::kHalf + (bx << box_shift) * C::kRowBytes, (lane & 1) ? tv : tk, bar,
                      (int)row);
      } else {
        const int part = lane & 3;  // K codes, V codes, K scales, V scales
        const uint8_t* src = part == 0 ? p.pg.k : part == 1 ? p.pg.v
                             : reinterpret_cast<const uint8_t*>(part == 2 ? p.pg.k_scales : p.pg.v_scales);
        const int rb = part < 2 ? C::kRowBytes : 4;
        const int at = (part & 1) * (part < 2 ? C::kHalf : C::kScales) + (part < 2 ? 0 : 2 * C::kHalf);
        bulk_load(st + at + (bx << box_shift) * rb, src + row * rb, (uint32_t)rb << box_shift, bar);
      }
    }
  }
};

template <int D, int BITS, int NT>
__device__ __forceinline__ void attend(const PagedAttnParams& p, const CUtensorMap* tk, const CUtensorMap* tv,
                                       const Smem<D, BITS, NT>& sm, Walk wk, const WaitCtx& wc) {
  using C = Cfg<D, BITS, NT>;
  constexpr int KT = C::kKT, MT = D / 16, KS = D / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, q4 = lane & 3;  // the fragment's row in a block of 8, and its column pair
  const int box_shift = min(p.pg.page_shift, KT == 32 ? 5 : 6);
  const uint32_t box_rows = 1u << box_shift;
  Issuer<D, BITS, NT> is;
  is.start(p, wk, warp);
#pragma unroll 1
  for (int i = 0; i < C::kDepth; ++i) is.issue(p, tk, tv, sm, warp);
  int k = warp, taken = 0;  // the warp's next tile in the segment, and the tiles it has taken
  bool alive = true, first_seg = true;
  do {
    const Item it = item_of(p, wk.g, wk.in, C::kRows);
    int len;
    int64_t first;
    key_bound(p, it.b, &len, &first);
    const int R = p.Nq * p.G - it.row0;  // real rows of the block (may exceed kRows)
    const __nv_bfloat16* qb = p.q + it.b * p.qs[0];

    // ---- Q fragments (B operand of S^T: k = values of the head, n = rows) ----
    uint2 qf[C::kQShared ? 1 : KS][C::kQShared ? 1 : NT];
    float qsum[2 * NT];
    auto load_q = [&](int ks, int nt) {
      const int r = nt * 8 + g8;
      if (r >= R) return make_uint2(0u, 0u);
      const int row = it.row0 + r, i = row / p.G, h = it.kvh * p.G + row % p.G;
      const __nv_bfloat16* src = qb + i * p.qs[1] + h * p.qs[2];
      if (BITS == 16) {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(src + ks * 16 + 2 * q4);
        return make_uint2(s[0], s[4]);
      } else {
        // values base + {0, 4} and base + {1, 5}: the nibble pairs that centred() gives
        const uint32_t* s = reinterpret_cast<const uint32_t*>(src + (D / 4) * q4 + 8 * (ks >> 1) + 2 * (ks & 1));
        const uint32_t lo = s[0], hi = s[2];
        return make_uint2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
      }
    };
    if (!C::kQShared) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) qf[C::kQShared ? 0 : ks][C::kQShared ? 0 : nt] = load_q(ks, nt);
      if (BITS == 4) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float s = 0.f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint2 u = qf[C::kQShared ? 0 : ks][C::kQShared ? 0 : nt];
            s += (__uint_as_float(u.x << 16) + __uint_as_float(u.x & 0xffff0000u)) +
                 (__uint_as_float(u.y << 16) + __uint_as_float(u.y & 0xffff0000u));
          }
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);  // lanes of row g8 hold its sum
          qsum[2 * nt] = __shfl_sync(0xffffffffu, s, 8 * q4);
          qsum[2 * nt + 1] = __shfl_sync(0xffffffffu, s, 8 * q4 + 4);
        }
      }
    } else {
      for (int x = warp; x < KS * NT; x += C::kWarps) sm.q[x * 32 + lane] = load_q(x / NT, x % NT);
      if (BITS == 4 && warp == 0) {
        float s = 0.f;
        if (lane < C::kRows && lane < R) {
          const int row = it.row0 + lane, i = row / p.G, h = it.kvh * p.G + row % p.G;
          const __nv_bfloat16* src = qb + i * p.qs[1] + h * p.qs[2];
          for (int x = 0; x < D; ++x) s += __bfloat162float(src[x]);
        }
        if (lane < C::kRows) sm.qsum[lane] = s;
      }
      __syncthreads();
      if (BITS == 4) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          qsum[2 * nt] = sm.qsum[nt * 8 + 2 * q4];
          qsum[2 * nt + 1] = sm.qsum[nt * 8 + 2 * q4 + 1];
        }
      }
    }

    float acc[MT][NT][4], mx[2 * NT], sum[2 * NT], cor[2 * NT];
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      mx[x] = -INFINITY;
      sum[x] = 0.f;
      cor[x] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;

    for (; k < wk.n; k += C::kWarps) {
      const int stage = warp * C::kDepth + taken % C::kDepth;
      if (alive) alive = mbar_wait(&sm.full[stage], (taken / C::kDepth) & 1u, wc);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) continue;  // keeps walking: the barriers at the ends of segments are still met
      ++taken;
      const int4 hd = sm.hdr[stage];
      uint8_t* st = sm.stage + stage * C::kStage;
      const uint32_t kaddr = smem_addr(st), vaddr = kaddr + C::kHalf;
      bool wrote = false;
      // bf16 rows lie [box][64-value part][row of the box]: bytes to the 16 rows from `key` on
      auto block16 = [&](int key) {
        return (uint32_t)((key >> box_shift) << box_shift) * C::kRowBytes + (key & (box_rows - 1)) * 128u;
      };
      auto chunk_at = [&](int key, int ch) {  // 16-byte chunk ch of a row
        return block16(key & ~15) + (ch >> 3) * (box_rows * 128) + (key & 15) * 128 + (((ch & 7) ^ (key & 7)) << 4);
      };
#pragma unroll 1
      for (int sb = 0; sb < KT; sb += 32) {
        // ---- S^T: 32 keys x rows ----
        float s[2][NT][4];
#pragma unroll
        for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[m2][nt][e] = 0.f;
        if (BITS == 16) {
          const uint32_t lrow = ((lane & 7) + ((lane >> 3) & 1) * 8) * 128, hi = lane >> 4;
#pragma unroll
          for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const uint32_t ch = ks * 2 + hi;
              uint32_t a[4];
              ldsm4(a, kaddr + block16(sb + m2 * 16) + (ks >> 2) * (box_rows * 128) + lrow + (((ch & 7) ^ (lane & 7)) << 4));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint2 b = C::kQShared ? sm.q[(ks * NT + nt) * 32 + lane] : qf[C::kQShared ? 0 : ks][C::kQShared ? 0 : nt];
                mma16816(s[m2][nt], a, b.x, b.y);
              }
            }
        } else {
#pragma unroll
          for (int m2 = 0; m2 < 2; ++m2) {
            uint32_t r0[D / 32], r1[D / 32];  // the thread's piece of two code rows
            const uint8_t* row = st + (sb + m2 * 16 + slot_key(g8)) * C::kRowBytes + q4 * (D / 8);
            if (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(row), y = *reinterpret_cast<const uint4*>(row + 8 * C::kRowBytes);
              r0[0] = x.x; r0[1] = x.y; r0[D / 32 - 2] = x.z; r0[D / 32 - 1] = x.w;
              r1[0] = y.x; r1[1] = y.y; r1[D / 32 - 2] = y.z; r1[D / 32 - 1] = y.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(row), y = *reinterpret_cast<const uint2*>(row + 8 * C::kRowBytes);
              r0[0] = x.x; r0[1] = x.y;
              r1[0] = y.x; r1[1] = y.y;
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const int i = 2 * (ks & 1);
              const uint32_t a[4] = {centred(r0[ks >> 1], i), centred(r1[ks >> 1], i), centred(r0[ks >> 1], i + 1),
                                     centred(r1[ks >> 1], i + 1)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint2 b = C::kQShared ? sm.q[(ks * NT + nt) * 32 + lane] : qf[C::kQShared ? 0 : ks][C::kQShared ? 0 : nt];
                mma16816(s[m2][nt], a, b.x, b.y);
              }
            }
          }
        }
        // keys of the thread's four fragment rows
        auto key_of = [&](int m2, int hf) { return sb + m2 * 16 + hf * 8 + (BITS == 4 ? slot_key(g8) : g8); };
        float vs[2][2], vm[2][2];
        if (BITS == 4) {
          const uint32_t* ksc = reinterpret_cast<const uint32_t*>(st + 2 * C::kHalf);
          const uint32_t* vsc = ksc + KT;
#pragma unroll
          for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int key = key_of(m2, hf);
              const uint32_t a = ksc[key], b = vsc[key];
              const float ks_ = __uint_as_float(a << 16), km = fmaf(8.f, ks_, __uint_as_float(a & 0xffff0000u));
              vs[m2][hf] = __uint_as_float(b << 16);
              vm[m2][hf] = fmaf(8.f, vs[m2][hf], __uint_as_float(b & 0xffff0000u));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  s[m2][nt][2 * hf + e] = fmaf(ks_, s[m2][nt][2 * hf + e], km * qsum[2 * nt + e]);
            }
        }
        // ---- hidden pairs ----
        const bool masked = hd.y != 0;
        uint32_t hid = 0;  // bit (m2 * 2 + hf) * 2 NT + nt * 2 + e
        if (masked) {
#pragma unroll
          for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int key = key_of(m2, hf), j = hd.x + key;
              const bool there = (hd.z >> (key >> box_shift)) & 1;
              const uint32_t w = p.words_shared && there ? p.words[(int64_t)it.b * p.words_stride + j] : 0u;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int row = it.row0 + nt * 8 + 2 * q4 + e, i = row / p.G;
                  bool see;
                  if (p.words_shared) {
                    see = (w >> (i & 31)) & 1u;
                  } else if (p.words) {
                    see = false;
                    if (i < p.Nq && there) {
                      const int hm = p.Hm == 1 ? 0 : it.kvh * p.G + row % p.G;
                      const int64_t at = ((int64_t)(it.b * p.Hm + hm) * p.n_words + (i >> 5)) * p.words_stride + j;
                      see = (p.words[at] >> (i & 31)) & 1u;
                    }
                  } else {
                    see = j < len && (!p.causal || j <= first + i);
                  }
                  if (!(see && there)) {
                    hid |= 1u << ((m2 * 2 + hf) * 2 * NT + nt * 2 + e);
                    s[m2][nt][2 * hf + e] = -INFINITY;
                  }
                }
            }
        }
        // ---- running maximum ----
        float mn[2 * NT];
        bool grew = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = fmaxf(fmaxf(s[0][nt][e], s[0][nt][2 + e]), fmaxf(s[1][nt][e], s[1][nt][2 + e]));
            mn[2 * nt + e] = fmaxf(mx[2 * nt + e], max8(x));
            grew |= mn[2 * nt + e] > mx[2 * nt + e];
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int x = 0; x < 2 * NT; ++x) {
            const float f = mx[x] == -INFINITY ? 0.f : fast_exp2((mx[x] - mn[x]) * p.scale_log2);
            mx[x] = mn[x];
            sum[x] *= f;
            cor[x] *= f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              acc[mt][x >> 1][x & 1] *= f;
              acc[mt][x >> 1][2 + (x & 1)] *= f;
            }
          }
        }
        // ---- P^T, its sums, and its transpose as the B operand of O^T ----
        float off[2 * NT];
#pragma unroll
        for (int x = 0; x < 2 * NT; ++x) off[x] = mx[x] == -INFINITY ? 0.f : mx[x] * p.scale_log2;
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float w[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int x = 2 * nt + e;
                const float pr = fast_exp2(fmaf(s[m2][nt][2 * hf + e], p.scale_log2, -off[x]));
                sum[x] += pr;
                w[e] = pr;
                if (BITS == 4) {
                  // a hidden key's scale may be anything, NaN included
                  const bool hidden = (hid >> ((m2 * 2 + hf) * 2 * NT + x)) & 1u;
                  w[e] = hidden ? 0.f : pr * vs[m2][hf];
                  cor[x] = hidden ? cor[x] : fmaf(pr, vm[m2][hf], cor[x]);
                } else {
                  s[m2][nt][2 * hf + e] = pr;
                }
              }
              pb[m2][nt][hf] = transpose8x8(pack_bf16x2(w[0], w[1]));
            }
        // ---- values that are not finite, in a tile that some row does not see whole ----
        // 0 * NaN must not reach a row that the key is hidden from: such keys leave the product and are
        // added by rows that see them, one by one.
        if (BITS == 16 && masked) {
          const int kk = sb + lane;
          __nv_bfloat162 z = __float2bfloat162_rn(0.f);
          const __nv_bfloat162 zero = z;
#pragma unroll
          for (int ch = 0; ch < D / 8; ++ch) {
            const uint4 u = *reinterpret_cast<const uint4*>(st + C::kHalf + chunk_at(kk, ch));
            const uint32_t ww[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&ww[y]), zero, z);
          }
          const float2 zf = __bfloat1622float2(z);
          uint32_t bad = __ballot_sync(0xffffffffu, !(zf.x == 0.f && zf.y == 0.f));
          while (bad) {
            const int k5 = __ffs(bad) - 1;  // key in the 32
            bad &= bad - 1;
            const int src = (k5 & 7) * 4 + q4, sel = k5 >> 3;  // sel = m2 * 2 + hf
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float c0 = sel & 2 ? s[1][nt][e] : s[0][nt][e], c1 = sel & 2 ? s[1][nt][2 + e] : s[0][nt][2 + e];
                const float pr = __shfl_sync(0xffffffffu, sel & 1 ? c1 : c0, src);
                const uint32_t hb = __shfl_sync(0xffffffffu, hid, src);
                if (!((hb >> (sel * 2 * NT + nt * 2 + e)) & 1u)) {
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                      const int x = mt * 16 + u * 8 + g8;
                      const __nv_bfloat16 v = *reinterpret_cast<const __nv_bfloat16*>(
                          st + C::kHalf + chunk_at(sb + k5, x >> 3) + (x & 7) * 2);
                      acc[mt][nt][2 * u + e] = fmaf(pr, __bfloat162float(v), acc[mt][nt][2 * u + e]);
                    }
                }
              }
            __syncwarp();
            if (lane < D / 8)
              *reinterpret_cast<uint4*>(st + C::kHalf + chunk_at(sb + k5, lane)) = make_uint4(0u, 0u, 0u, 0u);
            wrote = true;
          }
          __syncwarp();
        }
        // ---- O^T += V^T P^T ----
        if (BITS == 16) {
          const uint32_t lrow = ((lane & 7) + (lane >> 4) * 8) * 128, hi = (lane >> 3) & 1;
#pragma unroll
          for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint32_t ch = mt * 2 + hi;
              uint32_t a[4];
              ldsm4_t(a, vaddr + block16(sb + m2 * 16) + (mt >> 2) * (box_rows * 128) + lrow + (((ch & 7) ^ (lane & 7)) << 4));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(acc[mt][nt], a, pb[m2][nt][0], pb[m2][nt][1]);
            }
        } else {
#pragma unroll
          for (int m2 = 0; m2 < 2; ++m2) {
            // slots 2 q4, 2 q4 + 1 and the same + 8; the thread takes values [g8 D/8, (g8 + 1) D/8) of each
            uint32_t r[4][D / 64];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int key = sb + m2 * 16 + (y >> 1) * 8 + slot_key(2 * q4 + (y & 1));
              const uint8_t* src = st + C::kHalf + key * C::kRowBytes + g8 * (D / 16);
              if (D == 128) {
                const uint2 x = *reinterpret_cast<const uint2*>(src);
                r[y][0] = x.x;
                r[y][D / 64 - 1] = x.y;
              } else {
                r[y][0] = *reinterpret_cast<const uint32_t*>(src);
              }
            }
#pragma unroll
            for (int w = 0; w < D / 64; ++w)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {  // low and high 16 bits: four values each
                const uint32_t lo = __byte_perm(r[0][w], r[1][w], hh ? 0x7632 : 0x5410);
                const uint32_t up = __byte_perm(r[2][w], r[3][w], hh ? 0x7632 : 0x5410);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const int mt = w * 4 + hh * 2 + z;
                  const uint32_t a[4] = {centred(lo, 2 * z), centred(lo, 2 * z + 1), centred(up, 2 * z),
                                         centred(up, 2 * z + 1)};
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma16816(acc[mt][nt], a, pb[m2][nt][0], pb[m2][nt][1]);
                }
              }
          }
        }
      }
      if (wrote) fence_async_smem();
      __syncwarp();
      is.issue(p, tk, tv, sm, warp);
    }
    k -= wk.n;

    // ---- the warps' sums together ----
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      sum[x] = sum8(sum[x]);
      if (BITS == 4) cor[x] = sum8(cor[x]);
    }
    if (g8 == 0) {
#pragma unroll
      for (int x = 0; x < 2 * NT; ++x) {
        const int r = warp * C::kRows + (x >> 1) * 8 + 2 * q4 + (x & 1);
        sm.m[r] = mx[x];
        sm.l[r] = sum[x];
        if (BITS == 4) sm.c[r] = cor[x];
      }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      const int r = (x >> 1) * 8 + 2 * q4 + (x & 1);
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) top = fmaxf(top, sm.m[w * C::kRows + r]);
      const float f = mx[x] == -INFINITY ? 0.f : fast_exp2((mx[x] - top) * p.scale_log2);
      float* dst = sm.merge + (warp * C::kRows + r) * C::kStride;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (BITS == 16) {
          dst[mt * 16 + g8] = acc[mt][x >> 1][x & 1] * f;
          dst[mt * 16 + 8 + g8] = acc[mt][x >> 1][2 + (x & 1)] * f;
        } else {
          *reinterpret_cast<float2*>(dst + g8 * (D / 8) + 2 * mt) =
              make_float2(acc[mt][x >> 1][x & 1] * f, acc[mt][x >> 1][2 + (x & 1)] * f);
        }
      }
    }
    __syncthreads();
    const bool whole = wk.n == wk.T;
    const int slot = 2 * blockIdx.x + (first_seg ? 0 : 1);
    for (int x = threadIdx.x; x < C::kRows * (D / 4); x += 32 * C::kWarps) {
      const int r = x / (D / 4), d4 = x % (D / 4);
      if (r >= R) continue;
      float top = -INFINITY, L = 0.f, cc = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) top = fmaxf(top, sm.m[w * C::kRows + r]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float m = sm.m[w * C::kRows + r];
        const float f = m == -INFINITY ? 0.f : fast_exp2((m - top) * p.scale_log2);
        L = fmaf(sm.l[w * C::kRows + r], f, L);
        if (BITS == 4) cc = fmaf(sm.c[w * C::kRows + r], f, cc);
        const float4 v = *reinterpret_cast<const float4*>(sm.merge + (w * C::kRows + r) * C::kStride + 4 * d4);
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
      if (BITS == 4) {
        o.x += cc;
        o.y += cc;
        o.z += cc;
        o.w += cc;
      }
      if (whole) {
        const int row = it.row0 + r, i = row / p.G, h = it.kvh * p.G + row % p.G;
        const float inv = top == -INFINITY ? 0.f : 1.f / L;
        const int64_t at = (((int64_t)it.b * p.Nq + i) * p.Hq + h) * D + 4 * d4;
        *reinterpret_cast<uint2*>(p.o + at) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (d4 == 0)
          p.lse[((int64_t)it.b * p.Hq + h) * p.Nq + i] =
              top == -INFINITY ? -INFINITY : fmaf(top, p.scale_log2, log2f(L)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(p.part + (slot * C::kRows + r) * D + 4 * d4) = o;
        if (d4 == 0) p.stat[slot * C::kRows + r] = make_float2(top, L);
      }
    }
    __syncthreads();
    first_seg = false;
  } while (wk.next(p));
  if (!alive && lane == 0) {  // gave up: let the copies in flight land before the CTA ends
    WaitCtx w2 = wc;
    int zero = 0;
    w2.abort = &zero;
    for (int i = taken; i < is.issued; ++i)
      mbar_wait(&sm.full[warp * C::kDepth + i % C::kDepth], (i / C::kDepth) & 1u, w2);
  }
}

// Rows of a group (items in0 <= item < in1 of it) whose keys are all hidden or missing.
template <int D>
__device__ void write_empty(const PagedAttnParams& p, int g, int in0, int in1, int threads) {
  const int b = group_batch(p, g), R = p.Nq * p.G;
  for (int in = in0; in < in1; ++in) {
    const Item it = item_of(p, g, in, p.rows);
    const int n = min(p.rows, R - it.row0);
    for (int x = threadIdx.x; x < n * (D / 8); x += threads) {
      const int row = it.row0 + x / (D / 8), c = x % (D / 8), i = row / p.G, h = it.kvh * p.G + row % p.G;
      *reinterpret_cast<uint4*>(p.o + (((int64_t)b * p.Nq + i) * p.Hq + h) * D + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
      if (c == 0) p.lse[((int64_t)b * p.Hq + h) * p.Nq + i] = -INFINITY;
    }
  }
}

template <int D, int BITS, int NT>
__global__ void __launch_bounds__(Cfg<D, BITS, NT>::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                           const __grid_constant__ PagedAttnParams p) {
  using C = Cfg<D, BITS, NT>;
  extern __shared__ uint8_t raw[];
  Smem<D, BITS, NT> sm(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (lane == 0) {
    for (int i = 0; i < C::kDepth; ++i) mbar_init(&sm.full[warp * C::kDepth + i], 1);
    if (warp == 0) *sm.abort = 0;
    fence_mbar_init();
  }
  WaitCtx wc;
  wc.abort = sm.abort;
  wc.status = p.pg.status;
  wc.limit_ns = p.wait_limit_ns;
  wc.smem_base = smem_addr(raw);
  wc.kernel = 5;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  if (p.uncut) {  // one item per CTA
    Walk wk;
    wk.g = blockIdx.x / p.mult;
    wk.in = blockIdx.x % p.mult;
    wk.t = 0;
    wk.T = wk.n = wk.left = tiles_of(p, wk.g);
    if (wk.T == 0) write_empty<D>(p, wk.g, wk.in, wk.in + 1, C::kThreads);
    else attend<D, BITS, NT>(p, &tk, &tv, sm, wk, wc);
    return;
  }

  // ---- this CTA's run of units: every warp sums the groups' tiles and finds the group it begins in ----
  const int per = (p.n_groups + 31) / 32, ga = min(lane * per, p.n_groups), gb = min(ga + per, p.n_groups);
  int mine = 0;
#pragma unroll 4
  for (int g = ga; g < gb; ++g) mine += tiles_of(p, g);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31) * p.mult;
  // units of a run: total / ctas, one more for the first total % ctas
  const int ctas = min((int)gridDim.x, max(1, total / p.min_tiles)), q = total / ctas, rem = total - q * ctas;
  const int c = blockIdx.x;
  const int u0 = c * q + min(c, rem), n_units = c < ctas ? q + (c < rem ? 1 : 0) : 0;
  if (n_units > 0) {
    const unsigned has = __ballot_sync(0xffffffffu, u0 < incl * p.mult);
    const int src = __ffs(has) - 1;
    Walk wk;
    int at = (incl - mine) * p.mult;
    wk.g = ga;
    wk.T = 0;
    if (lane == src) {
      wk.T = tiles_of(p, wk.g);
      while (u0 >= at + wk.T * p.mult) {
        at += wk.T * p.mult;
        wk.T = tiles_of(p, ++wk.g);
      }
    }
    wk.g = __shfl_sync(0xffffffffu, wk.g, src);
    wk.T = __shfl_sync(0xffffffffu, wk.T, src);
    const int off = u0 - __shfl_sync(0xffffffffu, at, src);
    wk.in = off / wk.T;
    wk.t = off - wk.in * wk.T;
    wk.left = n_units;
    wk.n = min(wk.T - wk.t, n_units);
    attend<D, BITS, NT>(p, &tk, &tv, sm, wk, wc);

    // an item that begins in this run and goes on in the next ones: where its parts are
    if (tid == 0) {
      int* meta = p.meta + c * kMetaInts;
      bool first = true;
      int u = u0;
      while (u + wk.n < u0 + n_units) {
        u += wk.n;
        first = false;
        wk.next(p);
      }
      meta[0] = -1;
      if (wk.t == 0 && wk.n < wk.T) {
        const Item it = item_of(p, wk.g, wk.in, C::kRows);
        const int last = u + wk.T - 1, big = rem * (q + 1);  // the CTA that ends it holds unit `last`
        meta[0] = it.b;
        meta[1] = it.kvh;
        meta[2] = it.row0;
        meta[3] = last < big ? last / (q + 1) : rem + (last - big) / q;
        meta[4] = first ? 0 : 1;
      }
    }
  } else if (tid == 0) {
    p.meta[c * kMetaInts] = -1;
  }
  for (int g = c; g < p.n_groups; g += gridDim.x)
    if (tiles_of(p, g) == 0) write_empty<D>(p, g, 0, p.mult, C::kThreads);
}

// ---------------------------------------------------------------------------
// joining the parts of cut items: one CTA per (run, row)
// ---------------------------------------------------------------------------
template <int D, int ROWS>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int LG = D / 4, NGR = 256 / LG;
  __shared__ float w[256], red[8];
  __shared__ float4 buf[NGR][LG];
  griddep_wait();
  const int* meta = p.meta + blockIdx.x * kMetaInts;
  const int b = meta[0];
  if (b < 0) return;
  const int r = blockIdx.y, row = meta[2] + r;
  if (row >= p.Nq * p.G) return;
  const int kvh = meta[1], parts = meta[3] - (int)blockIdx.x + 1, tid = threadIdx.x;
  auto slot = [&](int k) { return 2 * ((int64_t)blockIdx.x + k) + (k == 0 ? meta[4] : 0); };
  // weights of the parts (at most 160)
  float2 ml = make_float2(-INFINITY, 0.f);
  if (tid < parts) ml = p.stat[slot(tid) * ROWS + r];
  float top = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, red[i]);
  const float f = ml.x == -INFINITY ? 0.f : fast_exp2((ml.x - top) * p.scale_log2);
  w[tid] = f;
  float L = ml.y * f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  __syncthreads();
  if ((tid & 31) == 0) red[tid >> 5] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) L += red[i];
  const int grp = tid / LG, d4 = tid % LG;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = grp; k < parts; k += NGR) {
    const float4 v = *reinterpret_cast<const float4*>(p.part + (slot(k) * ROWS + r) * D + 4 * d4);
    const float wk = w[k];
    if (wk == 0.f) continue;  // a part that saw nothing
    o.x = fmaf(wk, v.x, o.x);
    o.y = fmaf(wk, v.y, o.y);
    o.z = fmaf(wk, v.z, o.z);
    o.w = fmaf(wk, v.w, o.w);
  }
  buf[grp][d4] = o;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int k = 1; k < NGR; ++k) {
    const float4 v = buf[k][d4];
    o.x += v.x;
    o.y += v.y;
    o.z += v.z;
    o.w += v.w;
  }
  const int i = row / p.G, h = kvh * p.G + row % p.G;
  const float inv = top == -INFINITY ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(p.o + (((int64_t)b * p.Nq + i) * p.Hq + h) * D + 4 * d4) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (d4 == 0)
    p.lse[((int64_t)b * p.Hq + h) * p.Nq + i] =
        top == -INFINITY ? -INFINITY : fmaf(top, p.scale_log2, log2f(L)) * kLn2;
}

// ---------------------------------------------------------------------------
// plan: row-visibility words and tile flags (one warp per tile), then the list
// of visible tiles (one CTA per group)
// ---------------------------------------------------------------------------
constexpr int kPlanTiles = 64;  // tiles of one CTA (8 warps)

// Rows [p0, p0 + 32) with [lo, hi) cut out, as a word.
__device__ __forceinline__ uint32_t rows_in(int64_t lo, int64_t hi, int64_t p0) {
  const int a = (int)min(max(lo - p0, (int64_t)0), (int64_t)32), b = (int)min(max(hi - p0, (int64_t)0), (int64_t)32);
  return bit_range(a, b);
}

template <int KT>
__global__ void __launch_bounds__(256) paged_plan_kernel(const __grid_constant__ PagedAttnParams p, PlanOut out) {
  griddep_wait();
  griddep_launch_dependents();
  const int g = blockIdx.x / out.chunks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = group_batch(p, g);
  const int hm0 = p.per_head ? (g % p.pg.Hkv) * p.G : 0, nh = p.per_head ? p.G : 1;
  int len;
  int64_t first;
  const int hi = key_bound(p, b, &len, &first);
  const int tiles = (hi + KT - 1) / KT;
#pragma unroll 2
  for (int x = warp; x < kPlanTiles; x += 8) {
    const int t = (blockIdx.x % out.chunks) * kPlanTiles + x;
    if (t >= tiles) break;
    bool any = false, all = true;
#pragma unroll
    for (int jj = 0; jj < KT; jj += 32) {
      const int j = t * KT + jj + lane;
      for (int h = 0; h < nh; ++h) {
        const int64_t at = ((int64_t)b * p.Hm + hm0 + h);
        int lts = 0, lte = 0, uts = 0, ute = 0;
        if (j < p.Nm && j < hi) {
          const int64_t m = at * p.Nm + j;
          if (p.lts) {
            lts = p.lts[m];
            lte = p.lte[m];
          }
          if (p.uts) {
            uts = p.uts[m];
            ute = p.ute[m];
          }
        }
        for (int w = 0; w < p.n_words; ++w) {
          const int64_t p0 = first + 32 * w;
          const uint32_t rows = bit_range(0, min(32, p.Nq - 32 * w));
          uint32_t see = 0;
          if (j < hi) {
            uint32_t hid = rows_in(lts, lte, p0) | rows_in(uts, ute, p0);
            if (p.causal) hid |= rows_in(p0, j, p0);
            see = rows & ~hid;
          }
          out.words[(at * p.n_words + w) * p.words_stride + j] = see;
          any |= see != 0;
          all &= see == rows;
        }
      }
    }
    any = __any_sync(0xffffffffu, any);
    all = __all_sync(0xffffffffu, all);
    if (lane == 0) out.flags[(int64_t)g * p.list_stride + t] = any ? (all ? 2 : 1) : 0;
  }
}

__global__ void __launch_bounds__(1024) paged_list_kernel(const __grid_constant__ PagedAttnParams p, PlanOut out) {
  __shared__ int wsum[32];
  griddep_wait();
  griddep_launch_dependents();
  const int g = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len;
  int64_t first;
  const int hi = key_bound(p, group_batch(p, g), &len, &first);
  const int tiles = (hi + p.tile_keys - 1) / p.tile_keys;
  const uint8_t* flags = out.flags + (int64_t)g * p.list_stride;
  int* list = out.list + (int64_t)g * p.list_stride;
  int done = 0;
  for (int t0 = 0; t0 < tiles; t0 += 4096) {  // four tiles a thread at a time
    int f[4], mine = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int t = t0 + 4 * tid + x;
      f[x] = t < tiles ? flags[t] : 0;
      mine += f[x] != 0;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int at = done + incl - mine;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) at += wsum[i];
      done += wsum[i];
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (f[x]) list[at++] = ((t0 + 4 * tid + x) << 1) | (f[x] == 1);
    __syncthreads();
  }
  if (tid == 0) out.counts[g] = done;
}

}  // namespace

template <int D, int BITS, int NT>
static cudaError_t launch_variant(const PagedAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                                  cudaStream_t st) {
  using C = Cfg<D, BITS, NT>;
  auto* k = paged_attention_kernel<D, BITS, NT>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(k), C::kSmem);
  if (e != cudaSuccess) return e;
  if (p.list) {
    e = launch_after(k, dim3(grid), dim3(C::kThreads), C::kSmem, st, tk, tv, p);
  } else {
    note_launch();
    k<<<grid, C::kThreads, C::kSmem, st>>>(tk, tv, p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || p.uncut) return e;
  return launch_after(paged_merge_kernel<D, C::kRows>, dim3(grid, C::kRows), dim3(256), 0, st, p);
}

int paged_tile_keys(int d, int bits) { return bits == 16 && d == 128 ? 32 : 64; }

cudaError_t launch_paged_attention(const PagedAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                                   PlanOut plan, cudaStream_t st) {
  if (p.list) {
    plan.chunks = (p.list_stride + kPlanTiles - 1) / kPlanTiles;
    if (plan.chunks > 0) {
      const unsigned blocks = (unsigned)plan.chunks * p.n_groups;
      note_launch();
      if (p.tile_keys == 32) paged_plan_kernel<32><<<blocks, 256, 0, st>>>(p, plan);
      else paged_plan_kernel<64><<<blocks, 256, 0, st>>>(p, plan);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch_after(paged_list_kernel, dim3(p.n_groups), dim3(1024), 0, st, p, plan);
    if (e != cudaSuccess) return e;
  }
#define FM_PAGED(D, BITS)                                                              \
  if (p.pg.d == D && p.pg.bits == BITS) {                                              \
    if (p.rows == 8) return launch_variant<D, BITS, 1>(p, tk, tv, grid, st);           \
    if (p.rows == 16) return launch_variant<D, BITS, 2>(p, tk, tv, grid, st);          \
    return launch_variant<D, BITS, 4>(p, tk, tv, grid, st);                            \
  }
  FM_PAGED(64, 16)
  FM_PAGED(128, 16)
  FM_PAGED(64, 4)
  FM_PAGED(128, 4)
#undef FM_PAGED
  return cudaErrorInvalidValue;
}

}  // namespace fm
