// Attention of a few rows per sequence over a paged key/value cache.
//
// The rows of one KV head (new tokens x the q-heads that share it) read every
// visible key and value once and do 4 d FLOP with each: bytes bound it as long
// as a block holds at most some 32 rows, so the design is about keeping the
// memory system full and the work even.
//
//  - Work.  An item is (sequence, KV head, block of 8, 16 or 32 rows); its
//    units are its tiles of 32 or 64 keys.  All units are laid end to end and
//    every warp of the device takes an equal run of them, whatever the lengths
//    of the sequences: a run may end one item, hold several and begin another.
//    An item inside one run is finished there; one that is cut leaves fp32
//    partial sums, which a second kernel joins in a fixed order (no atomics:
//    equal calls give equal bits).  Lengths are device data and the grid does
//    not depend on them, so a captured graph serves growing sequences.  Runs
//    handed out as warps become free (fixed chunks, joined in order) were no
//    better: 103 us against 99 for 64 sequences of 256 to 8192 keys.
//  - Warps work alone: each looks its pages up, fills a ring of tiles of its
//    own in shared memory (bf16: TMA, swizzled boxes; 4 bits: cp.async, whole
//    code rows) and keeps its own running maximum and sums; the ring runs on
//    into the next item, so the loads never pause at an item's end.  (A ring
//    shared by the warps needs two waits on one phase and a warp that fills
//    it; it took 133 us.)
//  - Few short items take one CTA each instead, whose warps share the tiles
//    and join their sums in shared memory; many of a few tiles go whole to a
//    warp.  Neither needs the second kernel.
//  - Masks.  With mask vectors a plan kernel runs first: it turns each key's
//    boundaries into one bit per row, and a second one lists the tiles that
//    some row sees, so hidden tiles are neither read nor counted as work.
//    Items of one CTA turn the boundaries into bits themselves.
//  - Products.  Tensor cores with the keys as the M side (mma m16n8k16): S^T =
//    K Q^T and O^T = V^T P^T need only 8 row columns, where the usual
//    orientation pads the rows to 16.  mma.sync and not tcgen05: rows are
//    few, P never leaves registers, and the tensor pipe is far from the bound
//    (10 % busy in bf16, 18 % in 4 bits).
//  - 4 bits.  A row's codes enter the products as integers, exact in bf16 (K:
//    16 + code, which costs no subtraction, with -24 sum(q) as the sum's first
//    value; V: code - 8); scale and minimum are applied to sums in fp32:
//      q.k = s (q.(c - 8)) + (m + 8 s) sum(q)
//      o   = sum (p s)(c - 8) + sum p (m + 8 s)
//    The contraction may run over the head's values in any order as long as
//    both sides agree, so each thread takes whole 16-byte pieces of code rows.
//    Codes as e4m3 bytes, which would need no conversion, lose: m16n8k32 in
//    e4m3 issues every 21 clocks, m16n8k16 in bf16 every 8.5.
//
// Measured, heads of 128, 8 KV heads of 4 q-heads, one new token for each of 64 sequences of 256 to 8192 keys (262
// thousand in all): bf16 99 us, 89 % of the measured copy bandwidth over the bytes that it cannot do
// without; the rest is the chain lengths - pages - rows - tiles at the start, the merge, and SMs whose
// bandwidth differs by 11 %.  In 4 bits 48.6 us, 45 %, with no unit used up (issue slots and ALU pipe 50 %, memory
// 38 %): 1400 instructions for 64 keys, most of them the codes' conversion, in one chain from conversion to scores
// to softmax to values, and three warps a scheduler to overlap it, which is as many as 168 registers allow.  A call of one tile takes 5.8 us: launch, the same chain, and code that is not in the
// instruction cache.
#include <cuda_bf16.h>

#include <algorithm>

#include "launchers.h"
#include "paged.cuh"
#include "sm100_primitives.cuh"

namespace fm {
namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr int kMetaInts = 8;
// Units that a run holds at least (kItemCost of them may stand for an item).  A long sequence with few visible
// tiles wants short runs on every SM: 20 us with 2 for the window of two sequences of 64K keys, 26 with 6; 1 and
// 2 are alike.
constexpr int kMinUnits = 2;

// ---------------------------------------------------------------------------
// work: groups of items with the same number of tiles, and a CTA's run of units
// ---------------------------------------------------------------------------
__device__ __forceinline__ int group_batch(const PagedAttnParams& p, int g) { return p.per_head ? p.div_hkv(g) : g; }

// A sequence as the kernels use it: cached keys, and its first row's position.
// Positions beyond +-2^30 see what those see (keys are fewer), so sums with row
// numbers stay in 32 bits.
struct Seq {
  int len, first;
};
__device__ __forceinline__ Seq load_seq(const PagedAttnParams& p, int b) {
  Seq q;
  q.len = checked_len(p.pg, p.lens, b);
  q.first = p.start ? min(max(p.start[b], -(1 << 30)), 1 << 30) : q.len - p.Nq;
  return q;
}
// Keys that the sequence's rows can see at all.
__device__ __forceinline__ int key_bound(const PagedAttnParams& p, const Seq& q) {
  return p.causal ? max(min(q.len, q.first + p.Nq), 0) : q.len;
}

__device__ __forceinline__ int load_tiles(const PagedAttnParams& p, int g) {
  return p.counts ? p.counts[g] : (key_bound(p, load_seq(p, group_batch(p, g))) + p.tile_keys - 1) / p.tile_keys;
}

// The CTA's copy of the sequences and of the groups' tile counts: once the
// rings are filled a load from memory waits behind them.
constexpr int kSeqCache = 512;
struct Seqs {
  const Seq* seq;    // shared memory: the sequences (held: B <= kSeqCache)
  const int* tiles_; // shared memory: tiles of the groups' items (held: n_groups <= kSeqCache)
  bool has_seq, has_tiles;
  __device__ __forceinline__ Seq get(const PagedAttnParams& p, int b) const { return has_seq ? seq[b] : load_seq(p, b); }
  __device__ __forceinline__ int tiles(const PagedAttnParams& p, int g) const {
    return has_tiles ? tiles_[g] : load_tiles(p, g);
  }
};

// A run, walked segment by segment (a segment: tiles [t, t + n) of one item).
// Runs are made of units, or of whole items.  An item has a unit for each of
// its tiles and kItemCost units before them, which stand for what an item
// costs besides (rows of Q, pages, output): a run of many short items would
// end late without them.  With 0, 2 and 4: 64 sequences of up to 8K keys 100.9, 98.9 and 99.3 us, in 4 bits 52.0, 50.1
// and 52.4, 41 sequences of up to 6.7K keys 32.5, 30.6 and 30.8.
constexpr int kItemCost = 2;
struct Walk {
  int g, in, T;   // group, item in the group, tiles of the group's items
  int pos, left;  // unit of the item that the segment begins at; units (items) left in the run
  int base;       // number of the item's first unit
  int t, n;       // first tile and tiles of the segment
  __device__ __forceinline__ void cut(const PagedAttnParams& p) {
    if (p.mode != kPagedSplit) {
      t = 0;
      n = T;
    } else {
      t = max(pos - kItemCost, 0);
      n = max(min(T + kItemCost, pos + left) - kItemCost, 0) - t;
    }
  }
  // The next segment that has tiles (of whole items: the next item); false at the run's end.
  __device__ __forceinline__ bool next(const PagedAttnParams& p, const Seqs& sq) {
    do {
      left -= p.mode == kPagedSplit ? T + kItemCost - pos : 1;
      if (left <= 0) return false;
      base += T + kItemCost;
      pos = 0;
      if (++in == p.mult) {
        in = 0;
        do {
          ++g;
          T = sq.tiles(p, g);
        } while (T == 0 && p.mode == kPagedSplit);
      }
      cut(p);
    } while (n <= 0 && p.mode == kPagedSplit);
    return true;
  }
  __device__ __forceinline__ bool first(const PagedAttnParams& p, const Seqs& sq) {
    cut(p);
    return n > 0 || p.mode != kPagedSplit || next(p, sq);
  }
};

// A warp's run: one of runs of q units, one more for the first rem.
struct Run {
  int worker, q, rem;
};

struct Item {
  int b, kvh, row0;
};
__device__ __forceinline__ Item item_of(const PagedAttnParams& p, int g, int in, int rows_per_item) {
  Item it;
  const int kv = p.div_rb(in);
  it.b = group_batch(p, g);
  it.kvh = p.per_head ? g - it.b * p.pg.Hkv : kv;
  it.row0 = (in - kv * p.n_rb) * rows_per_item;
  return it;
}

// ---------------------------------------------------------------------------
// masks
// ---------------------------------------------------------------------------
// Which of the ROWS rows of a KV head from r0 on see key j (j < hi), from the mask vectors, as a word.  Rows are
// numbered position by position, the heads of one position together: an interval of positions is an
// interval of rows, of which a mask head of its own has every G-th.
template <int ROWS>
__device__ __forceinline__ uint32_t seen_by(const PagedAttnParams& p, int b, int kvh, const Seq& seq, int j, int r0) {
  const int first = p.start ? p.start[b] : seq.first;  // as given: masks are applied literally
  // the word's first row at or after position `pos` (saturated: boundaries and starts are any 32-bit numbers)
  auto row_at = [&](int pos) {
    int i;
    asm("sub.sat.s32 %0, %1, %2;" : "=r"(i) : "r"(pos), "r"(first));
    return min(max(min(max(i, 0), p.Nq) * p.G - r0, 0), ROWS);
  };
  uint32_t hid = p.causal ? bit_range(0, row_at(j)) : 0u;
  if (j < p.Nm) {
    if (p.Hm == 1) {
      const int64_t m = (int64_t)b * p.Nm + j;
      const int a0 = p.lts ? p.lts[m] : 0, a1 = p.lts ? p.lte[m] : 0, a2 = p.uts ? p.uts[m] : 0, a3 = p.uts ? p.ute[m] : 0;
      hid |= bit_range(row_at(a0), row_at(a1)) | bit_range(row_at(a2), row_at(a3));
    } else {
      const int heads = min(p.G, ROWS), h0 = r0 - p.div_g(r0) * p.G;  // heads of rows r0, r0 + 1, ...
      const int64_t base = ((int64_t)b * p.Hm + kvh * p.G) * p.Nm + j;
      for (int x0 = 0; x0 < heads; x0 += 4) {  // the vectors of four heads are asked for together
        int v[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int h = h0 + x0 + x;
          const int64_t m = base + (int64_t)(h < p.G ? h : h - p.G) * p.Nm;
          const bool in = x0 + x < heads;
          v[x][0] = in && p.lts ? p.lts[m] : 0;
          v[x][1] = in && p.lts ? p.lte[m] : 0;
          v[x][2] = in && p.uts ? p.uts[m] : 0;
          v[x][3] = in && p.uts ? p.ute[m] : 0;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (x0 + x >= heads) break;
          uint32_t mine = 0u;  // rows of the head
          for (int r = x0 + x; r < ROWS; r += p.G) mine |= 1u << r;
          hid |= (bit_range(row_at(v[x][0]), row_at(v[x][1])) | bit_range(row_at(v[x][2]), row_at(v[x][3]))) & mine;
        }
      }
    }
  }
  return bit_range(0, min(ROWS, p.Nq * p.G - r0)) & ~hid;
}

// ---------------------------------------------------------------------------
// tiles and shared memory
// ---------------------------------------------------------------------------
template <int D, int BITS, int NT>
struct Cfg {
  static constexpr int kKT = BITS == 16 && D == 128 ? 32 : 64;  // keys of a tile
  static constexpr int kRows = 8 * NT;
  static constexpr int kWarps = paged_warps(D, BITS, kRows);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr bool kQShared = NT == 4;                     // Q fragments in shared memory
  static constexpr int kRowBytes = BITS == 16 ? 2 * D : D / 2;
  static constexpr int kHalf = kKT * kRowBytes;                 // K or V part of a stage
  static constexpr int kScales = BITS == 4 ? kKT * 4 : 0;
  static constexpr int kStage = 2 * kHalf + 2 * kScales;
  static constexpr int kStride = D + 4;                         // floats between rows of the merge buffer
  static constexpr int kMerge = kWarps * kRows * kStride * 4;   // on top of the rings
  static constexpr int kQBytes = kQShared ? (D / 16) * NT * 32 * 8 : 0;  // per warp
  static constexpr int kPerStage = kStage + 16 + 8;             // + header, barrier
  static constexpr int kFixed = kWarps * (kQBytes + 3 * kRows * 4) + kSeqCache * 12 + 1024 + 256;
  // Every warp has a ring of its own, which it fills and empties itself: a stage is refilled by the warp
  // that has just read it, so nothing waits for another warp.
  static constexpr int kFit = (225 * 1024 - kFixed) / kPerStage / kWarps;
  static constexpr int kDepth = kFit > 4 ? 4 : kFit;
  static constexpr int kStages = kWarps * kDepth;
  static constexpr int kSmem = kFixed + kStages * kPerStage;
  static constexpr int kBoxes = kKT / 16;                       // copies of a tile's rows at most
  static_assert(kDepth >= 2, "ring too short");
  static_assert(kMerge <= kStages * kStage, "the merge buffer lies on the rings");
};

template <int D, int BITS, int NT>
struct Smem {
  using C = Cfg<D, BITS, NT>;
  uint8_t* stage;      // kStages x kStage, 1024-byte aligned for the swizzle; kDepth in a row per warp
  int4* hdr;           // kStages: first key, some pair hidden, valid boxes
  uint64_t* full;      // kStages
  uint2* q;            // Q fragments of each warp (kQShared)
  float *m, *l, *c;    // kWarps x kRows (one item per CTA)
  Seq* seq;            // kSeqCache
  int* counts;         // kSeqCache
  int* abort;
  __device__ __forceinline__ explicit Smem(uint8_t* raw) {
    const uint32_t a = smem_addr(raw);
    uint8_t* x = raw + ((1024u - (a & 1023u)) & 1023u);
    stage = x; x += C::kStages * C::kStage;
    q = reinterpret_cast<uint2*>(x); x += C::kWarps * C::kQBytes;
    hdr = reinterpret_cast<int4*>(x); x += C::kStages * 16;
    full = reinterpret_cast<uint64_t*>(x); x += C::kStages * 8;
    m = reinterpret_cast<float*>(x); x += C::kWarps * C::kRows * 4;
    l = reinterpret_cast<float*>(x); x += C::kWarps * C::kRows * 4;
    c = reinterpret_cast<float*>(x); x += C::kWarps * C::kRows * 4;
    seq = reinterpret_cast<Seq*>(x); x += kSeqCache * 8;
    counts = reinterpret_cast<int*>(x); x += kSeqCache * 4;
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

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// 16 bytes per lane, global to shared memory; a group of them is one tile.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

// The code at nibble i of each half of x as the bf16 pair 16 + code: the four
// bits become the upper mantissa bits of 16.0.
__device__ __forceinline__ uint32_t raised(uint32_t x, int i) {
  uint32_t y;
  const uint32_t v = i == 0 ? x << 3 : x >> (4 * i - 3);
  asm("lop3.b32 %0, %1, 0x00780078, 0x41804180, 0xea;" : "=r"(y) : "r"(v));  // (v & a) | b
  return y;
}

// The code at nibble i of each half of x as the bf16 pair code - 8:
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

// The larger value, NaN if either is: a row with a score of NaN keeps a maximum of NaN, and is not taken for one
// that saw nothing.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Largest value over the 8 lanes that share lane % 4.
__device__ __forceinline__ float max8(float x) {
  x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return max_nan(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum8(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Fills one warp's ring with the warp's tiles of the run, in order, across
// segments: every STEP-th tile from the first one on.  Pages are looked up
// for 32 of them at a time, one by each lane.
template <int D, int BITS, int NT, int STEP>
struct Issuer {
  using C = Cfg<D, BITS, NT>;
  Walk w;
  int k;        // the warp's next tile that is not in the batch, in the segment
  int x, nb;    // next tile of the batch, and its size
  int issued;
  bool more;
  int kvh;
  int j0, flags, page[C::kBoxes];  // a lane's tile: first key, masked | valid boxes << 1, pages

  __device__ __forceinline__ void batch(const PagedAttnParams& p, const Seqs& sq, int box_shift) {
    constexpr int KT = C::kKT;
    const int lane = threadIdx.x & 31, boxes = KT >> box_shift;
    const Item it = item_of(p, w.g, w.in, C::kRows);
    kvh = it.kvh;
    const Seq seq = sq.get(p, it.b);
    const int hi = key_bound(p, seq);
    nb = min(32, (w.n - k + STEP - 1) / STEP);
    x = 0;
    j0 = 0;
    int masked = 0, valid = 0;
#pragma unroll
    for (int i = 0; i < C::kBoxes; ++i) page[i] = 0;
    if (lane < nb) {
      const int t = w.t + k + lane * STEP;
      if (p.list) {
        const int e = p.list[(int64_t)w.g * p.list_stride + t];
        j0 = (e >> 1) * KT;
        masked = e & 1;
      } else {
        j0 = t * KT;
        // keys that every row of the item sees
        masked = j0 + KT > (p.causal ? min(seq.len, seq.first + p.div_g(it.row0) + 1) : seq.len);
      }
#pragma unroll
      for (int i = 0; i < C::kBoxes; ++i) {
        const int j = j0 + (i << box_shift);
        if (i < boxes && j < hi) {
          page[i] = page_of(p.pg, it.b, j);
          if (page[i] >= 0) valid |= 1 << i;
        }
      }
      if (valid != (1 << boxes) - 1 || (STEP > 1 && (p.lts || p.uts))) masked = 1;
    }
    flags = masked | (valid << 1);
    k += nb * STEP;
  }

  __device__ __forceinline__ void start(const Walk& wk, int first_tile) {
    w = wk;
    k = first_tile;
    issued = 0;
    x = nb = 0;
    more = true;
  }

  // The next batch, if the run has more tiles.
  __device__ __forceinline__ void look_up(const PagedAttnParams& p, const Seqs& sq, int box_shift) {
    x = nb = 0;
    while (more && k >= w.n) {
      k -= w.n;
      more = w.next(p, sq);
    }
    if (more) batch(p, sq, box_shift);
  }

  __device__ __forceinline__ void issue(const PagedAttnParams& p, const CUtensorMap* tk, const CUtensorMap* tv,
                                        const Smem<D, BITS, NT>& sm, int warp, int box_shift) {
    const int lane = threadIdx.x & 31;
    const int tj = __shfl_sync(0xffffffffu, j0, x), f = __shfl_sync(0xffffffffu, flags, x);
    const int stage = warp * C::kDepth + issued % C::kDepth;
    uint64_t* bar = &sm.full[stage];
    uint8_t* st = sm.stage + stage * C::kStage;
    if (lane == 0) {
      sm.hdr[stage] = make_int4(tj, f & 1, f >> 1, 0);
      if (BITS == 16)
        mbar_arrive_expect_tx(bar, (uint32_t)(__popc(f >> 1) << box_shift) * (2 * C::kRowBytes));
    }
#pragma unroll
    for (int i = 0; i < C::kBoxes; ++i) {
      if (i >= (C::kKT >> box_shift)) break;
      const int pid = __shfl_sync(0xffffffffu, page[i], x);
      if (!((f >> (1 + i)) & 1)) continue;
      const int64_t row = row_of(p.pg, pid, kvh, tj + (i << box_shift));
      if (BITS == 16) {
        if (lane == 0) {
          uint8_t* dst = st + (i << box_shift) * C::kRowBytes;
          tma_load_rows(dst, tk, bar, (int)row);
          tma_load_rows(dst + C::kHalf, tv, bar, (int)row);
        }
      } else {
        // Every lane copies 16-byte pieces: four bulk copies a tile kept the copy engine, which takes some
        // 60 ns for each whatever its size, busier than the memory.
        const uint32_t dst = smem_addr(st) + (i << box_shift) * C::kRowBytes + lane * 16;
        const uint8_t* sk = p.pg.k + row * C::kRowBytes + lane * 16;
        const uint8_t* sv = p.pg.v + row * C::kRowBytes + lane * 16;
#pragma unroll 2
        for (int c = 0; c < (C::kRowBytes << box_shift); c += 512) {
          copy16(dst + c, sk + c);
          copy16(dst + C::kHalf + c, sv + c);
        }
        if ((lane & 15) < (1 << box_shift) / 4)  // scales and minima: K by the lower half of the warp, V by the upper
          copy16(smem_addr(st) + 2 * C::kHalf + (lane >> 4) * C::kScales + (i << box_shift) * 4 + (lane & 15) * 16,
                 (lane < 16 ? p.pg.k_scales : p.pg.v_scales) + row + (lane & 15) * 4);
      }
    }
    ++x;
    ++issued;
  }
};

// One warp's run (COOP: its share of the CTA's item): scores, softmax and
// values of every tile, and the item's rows or its partial sums at the end of
// each segment.
template <int D, int BITS, int NT, bool COOP>
__device__ __forceinline__ void attend(const PagedAttnParams& p, const CUtensorMap* tk, const CUtensorMap* tv,
                                       const Smem<D, BITS, NT>& sm, const Seqs& sq, Walk wk, const WaitCtx& wc,
                                       const Run& run) {
  using C = Cfg<D, BITS, NT>;
  constexpr int KT = C::kKT, MT = D / 16, KS = D / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, q4 = lane & 3;  // the fragment's row in a block of 8, and its column pair
  const int box_shift = min(p.pg.page_shift, KT == 32 ? 5 : 6);
  const uint32_t box_rows = 1u << box_shift;
  constexpr int STEP = COOP ? C::kWarps : 1;
  const bool masks = p.lts || p.uts;

  // ---- Q fragments (B operand of S^T: k = values of the head, n = rows) ----
  // A lane's pieces of its row of each 8: for 4 bits values base + {0, 1} and base + {4, 5}, which
  // turn_q() pairs as centred() pairs the codes.
  uint2 qf[C::kQShared ? 1 : KS][C::kQShared ? 1 : NT];
  float qsum[2 * NT];
  uint2* qw = sm.q + warp * (C::kQBytes / 8);
  auto row_ptr = [&](const Item& it, int r) {
    const int row = it.row0 + r, i = p.div_g(row);
    return p.q + it.b * p.qs[0] + i * p.qs[1] + (it.kvh * p.G + row - i * p.G) * p.qs[2];
  };
  auto load_q = [&](const Item& it) {
    const int R = p.Nq * p.G - it.row0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g8;
      const __nv_bfloat16* src = row_ptr(it, min(r, R - 1));
      uint2 v[KS];  // all of them asked for before the first is stored
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint32_t* a = reinterpret_cast<const uint32_t*>(
            BITS == 16 ? src + ks * 16 + 2 * q4 : src + (D / 4) * q4 + 8 * (ks >> 1) + 2 * (ks & 1));
        v[ks] = make_uint2(a[0], a[BITS == 16 ? 4 : 2]);
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if constexpr (C::kQShared) qw[(ks * NT + nt) * 32 + lane] = r < R ? v[ks] : make_uint2(0u, 0u);
        else qf[ks][nt] = v[ks];
      }
    }
  };
  auto turn_q = [&](const Item& it) {
    if constexpr (C::kQShared) {
      __syncwarp();
    } else {
      const int R = p.Nq * p.G - it.row0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float s = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint2& u = qf[ks][nt];
          if (nt * 8 + g8 >= R) u = make_uint2(0u, 0u);
          if (BITS == 4) {
            u = make_uint2(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.x, u.y, 0x7632));
            s += (__uint_as_float(u.x << 16) + __uint_as_float(u.x & 0xffff0000u)) +
                 (__uint_as_float(u.y << 16) + __uint_as_float(u.y & 0xffff0000u));
          }
        }
        if (BITS == 4) {
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);  // lanes of row g8 hold its sum
          qsum[2 * nt] = __shfl_sync(0xffffffffu, s, 8 * q4);
          qsum[2 * nt + 1] = __shfl_sync(0xffffffffu, s, 8 * q4 + 4);
        }
      }
    }
  };

  Issuer<D, BITS, NT, STEP> is;
  is.start(wk, COOP ? warp : 0);
  Item it{};
  Seq seq{};
  int R = 0;                          // real rows of the block (may exceed kRows)
  int k = COOP ? warp : 0;            // the warp's next tile in the segment
  int ahead = 0, taken = 0;           // tiles in the ring, and tiles taken out of it
  bool alive = true, fresh = true, first_seg = true;
  float acc[MT][NT][4], mx[2 * NT], sum[2 * NT], cor[2 * NT];
  // One loop for all tiles of the run, with one place each that loads rows, looks pages up, fills the
  // ring and works on a tile: the instruction cache is cold at every launch.
  for (;;) {
    if (fresh) {
      it = item_of(p, wk.g, wk.in, C::kRows);
      load_q(it);
    }
    if (is.x == is.nb) is.look_up(p, sq, box_shift);
    if (fresh) {
      turn_q(it);
      seq = sq.get(p, it.b);
      R = p.Nq * p.G - it.row0;
      fresh = false;
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
    }
    const int stage = warp * C::kDepth + taken % C::kDepth;
    // row-visibility words of the thread's keys, asked for before the tile is waited for
    uint32_t seen[KT / 32 * 4];
    if (COOP && masks && ahead > 0 && k < wk.n) {
      const int j0 = sm.hdr[stage].x;
#pragma unroll
      for (int y = 0; y < KT / 32; ++y) {
        const int j = j0 + y * 32 + lane;
        const uint32_t w = j < key_bound(p, seq) ? seen_by<C::kRows>(p, it.b, it.kvh, seq, j, it.row0) : 0u;
#pragma unroll
        for (int x = 0; x < 4; ++x) seen[y * 4 + x] = __shfl_sync(0xffffffffu, w, x * 8 + (BITS == 4 ? slot_key(g8) : g8));
      }
    }
    if (!COOP && masks && ahead > 0 && k < wk.n && sm.hdr[stage].y) {
      const uint32_t* w = p.words + ((int64_t)wk.g * p.n_words + (it.row0 >> 5)) * p.words_stride + sm.hdr[stage].x;
#pragma unroll
      for (int y = 0; y < KT / 32 * 4; ++y) seen[y] = w[(y >> 2) * 32 + (y & 3) * 8 + (BITS == 4 ? slot_key(g8) : g8)] >> (it.row0 & 31);
    }
    if (BITS == 16 && ahead > 0 && k < wk.n) {
      if (alive) alive = mbar_wait(&sm.full[stage], (taken / C::kDepth) & 1u, wc);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive)  // gave up: walks to the run's end
        while (k < wk.n) k += STEP;
    }
    if (ahead > 0 && k < wk.n) {
      if (BITS == 4) {
        if (ahead == C::kDepth) copy_wait<C::kDepth - 1>();
        else copy_wait<0>();
        __syncwarp();
      }
      ++taken;
      --ahead;
      k += STEP;
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
            for (int e = 0; e < 4; ++e) s[m2][nt][e] = BITS == 4 ? -24.f * qsum[2 * nt + (e & 1)] : 0.f;  // 16 + code -> code - 8
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
                const uint2 b = C::kQShared ? qw[(ks * NT + nt) * 32 + lane] : qf[C::kQShared ? 0 : ks][C::kQShared ? 0 : nt];
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
              const uint32_t a[4] = {raised(r0[ks >> 1], i), raised(r1[ks >> 1], i), raised(r0[ks >> 1], i + 1),
                                     raised(r1[ks >> 1], i + 1)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint2 b = C::kQShared ? qw[(ks * NT + nt) * 32 + lane] : qf[C::kQShared ? 0 : ks][C::kQShared ? 0 : nt];
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
              const uint32_t w = sb == 0 ? seen[m2 * 2 + hf] : seen[(KT / 32 - 1) * 4 + m2 * 2 + hf];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int r = nt * 8 + 2 * q4 + e;
                  const bool see = masks ? (w >> r) & 1u
                                           : j < seq.len && (!p.causal || j <= seq.first + p.div_g(it.row0 + r));
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
            const float x = max_nan(max_nan(s[0][nt][e], s[0][nt][2 + e]), max_nan(s[1][nt][e], s[1][nt][2 + e]));
            mn[2 * nt + e] = max_nan(mx[2 * nt + e], max8(x));
            grew |= !(mn[2 * nt + e] <= mx[2 * nt + e]);
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
                  w[e] = pr * vs[m2][hf];
                  if (!masked) {
                    cor[x] = fmaf(pr, vm[m2][hf], cor[x]);
                  } else {  // a hidden key's scale may be anything, NaN included
                    const bool hidden = (hid >> ((m2 * 2 + hf) * 2 * NT + x)) & 1u;
                    w[e] = hidden ? 0.f : w[e];
                    cor[x] = hidden ? cor[x] : fmaf(pr, vm[m2][hf], cor[x]);
                  }
                } else {
                  s[m2][nt][2 * hf + e] = pr;
                }
              }
              // Weights (4 bits: times the value's scale) are rounded to bf16, the type that the tensor cores take next to
              // bf16 values, as in the dense forward; their sum takes them unrounded.  O is off by at most 2^-8
              // sum w |v| so; against 64 bits 0.0019 to 0.0024 of its size, of which rounding O is 0.0016.
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
      if (BITS == 16 && wrote) fence_async_smem();
      __syncwarp();
    }
    while (ahead < C::kDepth && is.x < is.nb && alive) {
      is.issue(p, tk, tv, sm, warp, box_shift);
      if (BITS == 4) copy_commit();
      ++ahead;
    }
    __syncwarp();  // the headers of the tiles just asked for
    if (k < wk.n) continue;
    k -= wk.n;

    // ---- the segment's end ----
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      sum[x] = sum8(sum[x]);
      if (BITS == 4) cor[x] = sum8(cor[x]);
    }
    if (COOP) {
      // ---- the warps' sums together; the rings are empty and hold them ----
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
      float* merge = reinterpret_cast<float*>(sm.stage);
#pragma unroll
      for (int x = 0; x < 2 * NT; ++x) {
        const int r = (x >> 1) * 8 + 2 * q4 + (x & 1);
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) top = max_nan(top, sm.m[w * C::kRows + r]);
        const float f = mx[x] == -INFINITY ? 0.f : fast_exp2((mx[x] - top) * p.scale_log2);
        float* dst = merge + (warp * C::kRows + r) * C::kStride;
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
      for (int x = threadIdx.x; x < min(C::kRows, R) * (D / 4); x += 32 * C::kWarps) {
        const int r = x / (D / 4), d4 = x % (D / 4);
        float top = -INFINITY, L = 0.f, cc = 0.f;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) top = max_nan(top, sm.m[w * C::kRows + r]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
          const float m = sm.m[w * C::kRows + r];
          const float f = m == -INFINITY ? 0.f : fast_exp2((m - top) * p.scale_log2);
          L = fmaf(sm.l[w * C::kRows + r], f, L);
          if (BITS == 4) cc = fmaf(sm.c[w * C::kRows + r], f, cc);
          const float4 v = *reinterpret_cast<const float4*>(merge + (w * C::kRows + r) * C::kStride + 4 * d4);
          o.x += v.x;
          o.y += v.y;
          o.z += v.z;
          o.w += v.w;
        }
        const int row = it.row0 + r, i = p.div_g(row), h = it.kvh * p.G + row - i * p.G;
        const float inv = top == -INFINITY ? 0.f : 1.f / L;
        *reinterpret_cast<uint2*>(p.o + (((int64_t)it.b * p.Nq + i) * p.Hq + h) * D + 4 * d4) =
            make_uint2(pack_bf16x2((o.x + cc) * inv, (o.y + cc) * inv), pack_bf16x2((o.z + cc) * inv, (o.w + cc) * inv));
        if (d4 == 0)
          p.lse[((int64_t)it.b * p.Hq + h) * p.Nq + i] =
              top == -INFINITY ? -INFINITY : fmaf(top, p.scale_log2, log2f(L)) * kLn2;
      }
    } else if (wk.n == wk.T) {
      // ---- the whole item: its rows ----
#pragma unroll
      for (int x = 0; x < 2 * NT; ++x) {
        const float inv = mx[x] == -INFINITY ? 0.f : 1.f / sum[x];
        const int r = (x >> 1) * 8 + 2 * q4 + (x & 1), row = it.row0 + r, i = p.div_g(row);
        if (g8 == 0 && r < R)
          p.lse[((int64_t)it.b * p.Hq + it.kvh * p.G + row - i * p.G) * p.Nq + i] =
              mx[x] == -INFINITY ? -INFINITY : fmaf(mx[x], p.scale_log2, log2f(sum[x])) * kLn2;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          acc[mt][x >> 1][x & 1] = (acc[mt][x >> 1][x & 1] + cor[x]) * inv;
          acc[mt][x >> 1][2 + (x & 1)] = (acc[mt][x >> 1][2 + (x & 1)] + cor[x]) * inv;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (BITS == 16) {  // 8 x 8 blocks turned, so that a lane has neighbouring values of one row
          const int r = nt * 8 + g8, row = it.row0 + r, i = p.div_g(row);
          __nv_bfloat16* dst = p.o + (((int64_t)it.b * p.Nq + i) * p.Hq + it.kvh * p.G + row - i * p.G) * D + 2 * q4;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t v = transpose8x8(pack_bf16x2(acc[mt][nt][2 * u], acc[mt][nt][2 * u + 1]));
              if (r < R) *reinterpret_cast<uint32_t*>(dst + mt * 16 + u * 8) = v;
            }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = nt * 8 + 2 * q4 + e, row = it.row0 + r, i = p.div_g(row);
            if (r >= R) continue;
            __nv_bfloat16* dst = p.o + (((int64_t)it.b * p.Nq + i) * p.Hq + it.kvh * p.G + row - i * p.G) * D + g8 * (D / 8);
#pragma unroll
            for (int mt = 0; mt < MT; mt += 4)
              *reinterpret_cast<uint4*>(dst + 2 * mt) =
                  make_uint4(pack_bf16x2(acc[mt][nt][e], acc[mt][nt][2 + e]),
                             pack_bf16x2(acc[mt + 1][nt][e], acc[mt + 1][nt][2 + e]),
                             pack_bf16x2(acc[mt + 2][nt][e], acc[mt + 2][nt][2 + e]),
                             pack_bf16x2(acc[mt + 3][nt][e], acc[mt + 3][nt][2 + e]));
          }
        }
      }
    } else {
      // ---- part of an item: sums and running maximum ----
      const int slot = 2 * run.worker + (first_seg ? 0 : 1);
      if (wk.t == 0 && lane == 0) {  // it begins here and goes on in the next runs: where its parts are
        const int last = wk.base + wk.T + kItemCost - 1, big = run.rem * (run.q + 1);  // the run that ends it holds unit `last`
        int* meta = p.meta + run.worker * kMetaInts;
        meta[0] = it.b;
        meta[1] = it.kvh;
        meta[2] = it.row0;
        meta[3] = last < big ? last / (run.q + 1) : run.rem + (last - big) / run.q;
        meta[4] = first_seg ? 0 : 1;
      }
#pragma unroll
      for (int x = 0; x < 2 * NT; ++x) {
        const int r = (x >> 1) * 8 + 2 * q4 + (x & 1);
        if (r >= R) continue;
        if (g8 == 0) p.stat[slot * C::kRows + r] = make_float2(mx[x], sum[x]);
        float* dst = p.part + ((int64_t)slot * C::kRows + r) * D;
        if (BITS == 16) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            dst[mt * 16 + g8] = acc[mt][x >> 1][x & 1];
            dst[mt * 16 + 8 + g8] = acc[mt][x >> 1][2 + (x & 1)];
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; mt += 2)
            *reinterpret_cast<float4*>(dst + g8 * (D / 8) + 2 * mt) =
                make_float4(acc[mt][x >> 1][x & 1] + cor[x], acc[mt][x >> 1][2 + (x & 1)] + cor[x],
                            acc[mt + 1][x >> 1][x & 1] + cor[x], acc[mt + 1][x >> 1][2 + (x & 1)] + cor[x]);
        }
      }
    }
    first_seg = false;
    if (!wk.next(p, sq)) break;
    fresh = true;
  }
  if (BITS == 16 && !alive && lane == 0) {  // gave up: let the copies in flight land before the CTA ends
    WaitCtx w2 = wc;
    int zero = 0;
    w2.abort = &zero;
    w2.limit_ns = max(wc.limit_ns, (uint64_t)1000000000);
    for (int i = taken; i < is.issued; ++i)
      mbar_wait(&sm.full[warp * C::kDepth + i % C::kDepth], (i / C::kDepth) & 1u, w2);
  }
}

// Rows of a group whose keys are all hidden or missing.
template <int D>
__device__ void write_empty(const PagedAttnParams& p, int g, int threads) {
  const int b = group_batch(p, g), heads = p.per_head ? p.G : p.Hq, h0 = p.per_head ? (g % p.pg.Hkv) * p.G : 0;
  for (int64_t x = threadIdx.x; x < (int64_t)p.Nq * heads * (D / 8); x += threads) {
    const int c = (int)(x % (D / 8)), h = h0 + (int)(x / (D / 8) % heads), i = (int)(x / (D / 8) / heads);
    *reinterpret_cast<uint4*>(p.o + (((int64_t)b * p.Nq + i) * p.Hq + h) * D + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
    if (c == 0) p.lse[((int64_t)b * p.Hq + h) * p.Nq + i] = -INFINITY;
  }
}

template <int D, int BITS, int NT, bool COOP>
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
  // Rows of Q and the page table towards the L2: a batch's keys have evicted them since the last call, and
  // a run's chain of lengths, pages, rows and tiles would wait for each in turn.  (No value is read.)
  {
    const uint32_t at = (blockIdx.x * C::kThreads + tid) * 128;
    if (at < p.q_bytes) prefetch_l2(reinterpret_cast<const char*>(p.q) + at);
    if (at < p.table_bytes) prefetch_l2(reinterpret_cast<const char*>(p.pg.table) + at);
  }
  const Seqs sq{sm.seq, sm.counts, p.pg.B <= kSeqCache, p.n_groups <= kSeqCache};
  if (sq.has_seq)
    for (int b = tid; b < p.pg.B; b += C::kThreads) {
      const Seq q = load_seq(p, b);
      sm.seq[b] = q;
      if (!p.counts && sq.has_tiles && !p.per_head) sm.counts[b] = (key_bound(p, q) + C::kKT - 1) / C::kKT;
    }
  griddep_wait();  // the plan; what is read above are the call's inputs, which were there before the plan began
  griddep_launch_dependents();
  if (p.counts && sq.has_tiles)
    for (int g = tid; g < p.n_groups; g += C::kThreads) sm.counts[g] = p.counts[g];
  __syncthreads();

  Walk wk;
  Run run{};
  bool works = true;
  // neighbouring runs go to different SMs: a small problem's few runs are spread over the device
  const int worker = warp * gridDim.x + blockIdx.x, all_workers = C::kWarps * gridDim.x;
  if (COOP || p.mode == kPagedWhole) {  // whole items: one per CTA, or an equal share of them per warp
    int first = blockIdx.x;
    wk.left = 1;
    if (!COOP) {
      const int items = p.n_groups * p.mult, q = items / all_workers, rem = items - q * all_workers;
      first = worker * q + min(worker, rem);
      wk.left = q + (worker < rem ? 1 : 0);
      works = wk.left > 0;
    }
    wk.g = works ? p.div_mult(first) : 0;
    wk.in = first - wk.g * p.mult;
    wk.T = sq.tiles(p, wk.g);
    wk.pos = wk.base = 0;
  } else {
    // every warp sums the groups' units and finds the group that its run begins in
    const int per = (p.n_groups + 31) / 32, ga = min(lane * per, p.n_groups), gb = min(ga + per, p.n_groups);
    auto units = [&](int g) {
      const int T = sq.tiles(p, g);
      return T > 0 ? (T + kItemCost) * p.mult : 0;
    };
    int mine = 0;
    for (int g = ga; g < gb; ++g) mine += units(g);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    // units of a run: total / workers, one more for the first total % workers
    const int workers = min(all_workers, max(1, total / kMinUnits));
    run.worker = worker;
    run.q = total / workers;
    run.rem = total - run.q * workers;
    const int u0 = worker * run.q + min(worker, run.rem);
    wk.left = worker < workers ? run.q + (worker < run.rem ? 1 : 0) : 0;
    works = wk.left > 0;
    if (lane == 0) p.meta[worker * kMetaInts] = -1;
    if (works) {
      const int src = __ffs(__ballot_sync(0xffffffffu, u0 < incl)) - 1;
      int at = incl - mine, g = ga;
      if (lane == src)
        for (int n = units(g); u0 >= at + n; n = units(g)) {
          at += n;
          ++g;
        }
      wk.g = __shfl_sync(0xffffffffu, g, src);
      wk.T = sq.tiles(p, wk.g);
      const int off = u0 - __shfl_sync(0xffffffffu, at, src);
      wk.in = off / (wk.T + kItemCost);
      wk.pos = off - wk.in * (wk.T + kItemCost);
      wk.base = u0 - wk.pos;
      works = wk.first(p, sq);
    }
  }
  if (COOP || p.mode == kPagedWhole) wk.cut(p);
  if (works) attend<D, BITS, NT, COOP>(p, &tk, &tv, sm, sq, wk, wc, run);
  if (COOP || p.mode == kPagedWhole) return;
  if constexpr (!COOP)
    for (int g = blockIdx.x; g < p.n_groups; g += gridDim.x)
      if (sq.tiles(p, g) == 0) write_empty<D>(p, g, C::kThreads);
}

// ---------------------------------------------------------------------------
// joining the parts of cut items, in the order of their runs: a warp per item
// and row where the parts are few, the CTA's 8 warps together where they are
// many.  Latency is all it costs: the parts' values are asked for before their
// weights are known, and of the items that begin in a CTA's runs each warp takes
// its own without a barrier (with one warp for each run and barriers, 9 sequences
// of 32 rows took 26.6 us, now 20.9).
// ---------------------------------------------------------------------------
struct Joined {
  float m, l;
  float4 o;
};

// Parts k0, k0 + step, ... of an item's row (a warp's lanes hold 4 values each, D/4 of them a part).
template <int D, int ROWS>
__device__ __forceinline__ Joined join(const PagedAttnParams& p, int run, int first_slot, int parts, int k0, int step,
                                       int r) {
  constexpr int LG = D / 4, PP = 32 / LG;  // lanes of a part, parts that a warp reads at a time
  const int lane = threadIdx.x & 31, d4 = lane % LG, sub = lane / LG;
  auto slot = [&](int k) { return 2 * (run + k) + (k == 0 ? first_slot : 0); };
  Joined j{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int base = k0; base < parts; base += 32 * step) {
    const int mine = base + lane * step, n = min(32, (parts - base + step - 1) / step);
    const float2 ml = mine < parts ? p.stat[slot(mine) * ROWS + r] : make_float2(-INFINITY, 0.f);
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = max_nan(top, j.m);
    const float f = j.m == -INFINITY ? 0.f : fast_exp2((j.m - top) * p.scale_log2);
    const float w = ml.x == -INFINITY ? 0.f : fast_exp2((ml.x - top) * p.scale_log2);
    float l = ml.y * w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    j.m = top;
    j.l = fmaf(j.l, f, l);
    j.o.x *= f;
    j.o.y *= f;
    j.o.z *= f;
    j.o.w *= f;
    for (int i0 = 0; i0 < n; i0 += 8 * PP) {
      float4 v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int i = i0 + x * PP + sub;
        v[x] = i < n ? *reinterpret_cast<const float4*>(p.part + ((int64_t)slot(base + i * step) * ROWS + r) * D + 4 * d4)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float wx = __shfl_sync(0xffffffffu, w, (i0 + x * PP + sub) & 31);
        if (i0 + x * PP + sub < n && wx != 0.f) {  // 0: a part that saw nothing
          j.o.x = fmaf(wx, v[x].x, j.o.x);
          j.o.y = fmaf(wx, v[x].y, j.o.y);
          j.o.z = fmaf(wx, v[x].z, j.o.z);
          j.o.w = fmaf(wx, v[x].w, j.o.w);
        }
      }
    }
  }
  if (PP == 2) {
    j.o.x += __shfl_xor_sync(0xffffffffu, j.o.x, 16);
    j.o.y += __shfl_xor_sync(0xffffffffu, j.o.y, 16);
    j.o.z += __shfl_xor_sync(0xffffffffu, j.o.z, 16);
    j.o.w += __shfl_xor_sync(0xffffffffu, j.o.w, 16);
  }
  return j;
}

template <int D, int ROWS>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PagedAttnParams p, int workers,
                                                          int runs) {
  __shared__ float ms[8], ls[8];
  __shared__ float4 os[8][32];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y, v0 = blockIdx.x * runs;
  // every warp reads what begins in the CTA's runs, a lane per run
  int4 it = make_int4(-1, 0, 0, 0);  // sequence, KV head, first row, last run
  int slot = 0;
  if (lane < runs && v0 + lane < workers) {
    const int* meta = p.meta + (v0 + lane) * kMetaInts;
    it = *reinterpret_cast<const int4*>(meta);
    slot = meta[4];
  }
  const int mine = it.x < 0 || it.z + r >= p.Nq * p.G ? 0 : it.w - (v0 + lane) + 1;  // parts of the lane's item
  auto store = [&](int x, const Joined& j) {
    const int b = __shfl_sync(0xffffffffu, it.x, x), kvh = __shfl_sync(0xffffffffu, it.y, x);
    const int row = __shfl_sync(0xffffffffu, it.z, x) + r, i = p.div_g(row), h = kvh * p.G + row - i * p.G;
    const int d4 = lane % (D / 4);
    const float inv = j.m == -INFINITY ? 0.f : 1.f / j.l;
    if (lane >= D / 4) return;
    *reinterpret_cast<uint2*>(p.o + (((int64_t)b * p.Nq + i) * p.Hq + h) * D + 4 * d4) =
        make_uint2(pack_bf16x2(j.o.x * inv, j.o.y * inv), pack_bf16x2(j.o.z * inv, j.o.w * inv));
    if (d4 == 0)
      p.lse[((int64_t)b * p.Hq + h) * p.Nq + i] = j.m == -INFINITY ? -INFINITY : fmaf(j.m, p.scale_log2, log2f(j.l)) * kLn2;
  };
  auto joined = [&](int x, int k0, int step) {
    return join<D, ROWS>(p, v0 + x, __shfl_sync(0xffffffffu, slot, x), __shfl_sync(0xffffffffu, mine, x), k0, step, r);
  };
  int at = 0;
  for (uint32_t few = __ballot_sync(0xffffffffu, mine > 0 && mine <= 16); few; few &= few - 1)
    if ((at++ & 7) == warp) {
      const int x = __ffs(few) - 1;
      store(x, joined(x, 0, 1));
    }
  for (uint32_t many = __ballot_sync(0xffffffffu, mine > 16); many; many &= many - 1) {
    const int x = __ffs(many) - 1;
    const Joined j = joined(x, warp, 8);
    __syncthreads();
    if (lane == 0) {
      ms[warp] = j.m;
      ls[warp] = j.l;
    }
    os[warp][lane] = j.o;
    __syncthreads();
    if (warp != 0) continue;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max_nan(top, ms[i]);
    Joined all{top, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = ms[i] == -INFINITY ? 0.f : fast_exp2((ms[i] - top) * p.scale_log2);
      const float4 o = os[i][lane];
      if (f == 0.f) continue;
      all.l = fmaf(ls[i], f, all.l);
      all.o.x = fmaf(o.x, f, all.o.x);
      all.o.y = fmaf(o.y, f, all.o.y);
      all.o.z = fmaf(o.z, f, all.o.z);
      all.o.w = fmaf(o.w, f, all.o.w);
    }
    store(x, all);
  }
}

// ---------------------------------------------------------------------------
// plan: row-visibility words and the class of every tile (one warp per tile),
// then the list of visible tiles (one CTA per group); 3 us each.  A cluster of 8
// CTAs per group that does both in one launch took 30 us for one sequence of
// 128K keys: 8 SMs do not have enough loads in flight for 2 MB of vectors.
// Lists made by every attention CTA for itself save 1 us with few groups, but
// cost 2 where one group has 4096 tiles and 19 with 400 groups of one tile.
// ---------------------------------------------------------------------------
template <int KT>
__global__ void __launch_bounds__(256) paged_plan_kernel(const __grid_constant__ PagedAttnParams p, PlanOut out) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, x = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int g = x / p.list_stride, t = x - g * p.list_stride;
  if (g >= p.n_groups) return;
  const int b = group_batch(p, g);
  const Seq seq = load_seq(p, b);
  const int hi = key_bound(p, seq);
  if (t * KT >= hi) return;
  bool any = false, all = true;
#pragma unroll 1
  for (int w = 0; w < p.n_words; ++w) {
    const uint32_t rows = bit_range(0, min(32, p.Nq * p.G - 32 * w));
#pragma unroll
    for (int y = 0; y < KT / 32; ++y) {
      const int j = t * KT + y * 32 + lane;
      const uint32_t see = j < hi ? seen_by<32>(p, b, p.per_head ? g - b * p.pg.Hkv : 0, seq, j, 32 * w) : 0u;
      out.words[((int64_t)g * p.n_words + w) * p.words_stride + j] = see;
      any |= see != 0;
      all &= see == rows;
    }
  }
  any = __any_sync(0xffffffffu, any);
  all = __all_sync(0xffffffffu, all);
  if (lane == 0) out.flags[x] = any ? (all ? 2 : 1) : 0;
}

__global__ void __launch_bounds__(1024) paged_list_kernel(const __grid_constant__ PagedAttnParams p, PlanOut out) {
  __shared__ int wsum[32];
  const int g = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hi = key_bound(p, load_seq(p, group_batch(p, g)));  // the call's inputs, not the plan's
  const int tiles = (hi + p.tile_keys - 1) / p.tile_keys;
  griddep_wait();
  griddep_launch_dependents();
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
    int v = wsum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    int at = done + incl - mine + (warp > 0 ? __shfl_sync(0xffffffffu, v, (warp - 1) & 31) : 0);
    done += __shfl_sync(0xffffffffu, v, 31);
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (f[x]) list[at++] = ((t0 + 4 * tid + x) << 1) | (f[x] == 1);
    __syncthreads();
  }
  if (tid == 0) out.counts[g] = done;
}

}  // namespace

template <int D, int BITS, int NT, bool COOP>
static cudaError_t launch_variant(const PagedAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                                  cudaStream_t st) {
  using C = Cfg<D, BITS, NT>;
  auto* k = paged_attention_kernel<D, BITS, NT, COOP>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(k), C::kSmem);
  if (e != cudaSuccess) return e;
  if (p.list) {
    e = launch_after(k, dim3(grid), dim3(C::kThreads), C::kSmem, st, tk, tv, p);
  } else {
    note_launch();
    k<<<grid, C::kThreads, C::kSmem, st>>>(tk, tv, p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || p.mode != kPagedSplit) return e;
  // Runs of a CTA: 8 while all CTAs fit on the device at once (three an SM), else 16.  64 sequences of 4 rows: 98.4 us
  // with 8, 100.0 with 16 (101.4 and 103.0 in a slower process); 9 sequences of 32 rows 22.5 and 20.9.
  const int workers = grid * C::kWarps, rows = std::min(C::kRows, p.Nq * p.G);
  const int runs = (workers + 7) / 8 * rows <= 3 * 148 ? 8 : 16;
  return launch_after(paged_merge_kernel<D, C::kRows>, dim3((workers + runs - 1) / runs, rows), dim3(256), 0, st, p, workers,
                      runs);
}

template <int D, int BITS>
static cudaError_t launch_rows(const PagedAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                               cudaStream_t st) {
  const bool coop = p.mode == kPagedCoop;
  if (p.rows == 8)
    return coop ? launch_variant<D, BITS, 1, true>(p, tk, tv, grid, st) : launch_variant<D, BITS, 1, false>(p, tk, tv, grid, st);
  if constexpr (BITS == 16)  // (4 bits: blocks of at most 16 rows)
    if (p.rows == 32)
      return coop ? launch_variant<D, BITS, 4, true>(p, tk, tv, grid, st) : launch_variant<D, BITS, 4, false>(p, tk, tv, grid, st);
  return coop ? launch_variant<D, BITS, 2, true>(p, tk, tv, grid, st) : launch_variant<D, BITS, 2, false>(p, tk, tv, grid, st);
}

int paged_tile_keys(int d, int bits) { return bits == 16 && d == 128 ? 32 : 64; }

cudaError_t launch_paged_attention(const PagedAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                                   const PlanOut& plan, cudaStream_t st) {
  if (p.list && p.list_stride > 0) {
    const unsigned blocks = (unsigned)(((int64_t)p.n_groups * p.list_stride + 7) / 8);
    note_launch();
    if (p.tile_keys == 32) paged_plan_kernel<32><<<blocks, 256, 0, st>>>(p, plan);
    else paged_plan_kernel<64><<<blocks, 256, 0, st>>>(p, plan);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_after(paged_list_kernel, dim3(p.n_groups), dim3(1024), 0, st, p, plan);
    if (e != cudaSuccess) return e;
  }
  if (p.pg.d == 128) return p.pg.bits == 16 ? launch_rows<128, 16>(p, tk, tv, grid, st) : launch_rows<128, 4>(p, tk, tv, grid, st);
  return p.pg.bits == 16 ? launch_rows<64, 16>(p, tk, tv, grid, st) : launch_rows<64, 4>(p, tk, tv, grid, st);
}

}  // namespace fm
