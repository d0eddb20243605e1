// Appending to a paged key/value cache (rotation and 4-bit storage on the way)
// and gathering pages into dense tensors.  Both move bytes: a row (one token
// of one head) is read once and written once, and the arithmetic in between
// has to stay below the time that takes.
#include <cuda_bf16.h>

#include "launchers.h"
#include "paged.cuh"
#include "sm100_primitives.cuh"

namespace fm {
namespace {

// 16 values of one row as fp32, from two 16-byte chunks at offsets a and b.
__device__ __forceinline__ void load_chunks(const __nv_bfloat16* row, int a, int b, float (&x)[16]) {
  const uint4 u = *reinterpret_cast<const uint4*>(row + a), w = *reinterpret_cast<const uint4*>(row + b);
  const uint32_t r[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(r[i] << 16);
    x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void pack_chunks(const float (&x)[16], uint32_t (&r)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
}

__device__ __forceinline__ void store_chunks(__nv_bfloat16* row, int a, int b, const uint32_t (&r)[8]) {
  *reinterpret_cast<uint4*>(row + a) = make_uint4(r[0], r[1], r[2], r[3]);
  *reinterpret_cast<uint4*>(row + b) = make_uint4(r[4], r[5], r[6], r[7]);
}

// a c - b s rounded to fp32 once (to within 2^-47 of the exact value before
// that): products and their difference carried with their rounding errors
// (Dekker and Knuth's error-free product and sum).  Rows stored in 4 bits need
// it: where a rotated value lands next to the middle of two bf16 values, and
// so of two codes, the rounding of the products must not decide.
__device__ __forceinline__ float cross_exact(float a, float c, float b, float s) {
  const float p = a * c, ep = fmaf(a, c, -p);
  const float r = -(b * s), er = fmaf(-b, s, -r);
  const float t = p + r, z = t - p;
  const float et = (p - (t - z)) + (r - z);
  return t + ((ep + er) + et);
}

template <bool EXACT>
__device__ __forceinline__ void rotate_pair(float& x, float& y, float c, float s) {
  const float x1 = x, x2 = y;
  if (EXACT) {
    x = cross_exact(x1, c, x2, s);
    y = cross_exact(x2, c, -x1, s);
  } else {
    x = fmaf(x1, c, -(x2 * s));
    y = fmaf(x2, c, x1 * s);
  }
}

// Chunk a holds pairs' first values and chunk b their second (halves), or each
// holds four whole pairs (neighbours).
template <bool EXACT>
__device__ __forceinline__ void rotate(float (&x)[16], const float (&c)[8], const float (&s)[8], bool interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (interleaved)
      rotate_pair<EXACT>(x[2 * i], x[2 * i + 1], c[i], s[i]);
    else
      rotate_pair<EXACT>(x[i], x[i + 8], c[i], s[i]);
  }
}

// The code of x in a row with minimum lo, as a float: the integer nearest to
// (x - lo) / scale, ties to even.  The quotient in fp32 only proposes an integer
// k; the decision is whether |x - lo - k scale| exceeds half the scale.  x - lo is
// diff + err without error (Knuth's sum), r = diff - k scale is exact (k scale has
// 12 bits), and so is |r| - half wherever err, at most 2^-20 of the scale, can decide.
// err is added to that last, small difference: fp32 addition rounds no sum across
// zero, whereas r + err can round onto the middle of two codes.  Ties are
// common, since values and scales lie on the same few binary places: one value in
// some 300 of normal data.
__device__ __forceinline__ float code_of(float x, float lo, float scale, float inv, float half) {
  const float diff = x - lo, z = diff - x, err = (x - (diff - z)) + (-lo - z);
  const float m = fmaf(diff, inv, 12582912.f), k = m - 12582912.f;  // to an integer, which is in m's low bits
  const float r = fmaf(-k, scale, diff);
  const float over = (fabsf(r) - half) + __uint_as_float(__float_as_uint(err) ^ (__float_as_uint(r) & 0x80000000u));
  // an odd code gives way at the middle too: there over is +0, whose bits and the code's last make 1
  return __float_as_int(over) + (__float_as_int(m) & 1) > 0 ? k + copysignf(1.f, r) : k;
}

// Lower of two bf16 pairs, NaN if either is.
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// One thread takes 16 values of a row (two 16-byte chunks that hold whole
// pairs), D/16 neighbouring lanes a row, and goes through rows of one token
// `gpt` apart with that token's cosines and sines in registers.
// Bound by memory for bf16 (8192 tokens of 48 rows: 36.6 us, 86 % of the measured copy bandwidth).
// 4 bits are bound by issue and latency together (60 % of the issue slots busy): 64 registers, for 32 warps an
// SM, take 41.6 us with the gather of 9 ragged prompts, 72 registers 43.8, 56 with a few spilled 41.9, 48 44.4 (40.7 with 64
// since the codes are decided as they are now).
template <int D, int BITS>
__global__ void __launch_bounds__(128, BITS == 4 ? 8 : 1) paged_append_kernel(AppendParams p, int gpt_log2) {
  constexpr int L = D / 16;
  const int lane = threadIdx.x & 31, e = lane & (L - 1);
  const unsigned gmask = ((1u << L) - 1u) << (lane & ~(L - 1));
  const int64_t group = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) / L;
  const int64_t token = group >> gpt_log2;
  const int g0 = (int)(group & ((1 << gpt_log2) - 1));
  if (token >= (int64_t)p.pg.B * p.N) return;
  const int b = (int)(token / p.N), i = (int)(token % p.N);

  int count = p.N;
  if (p.counts) {
    count = p.counts[b];
    if (count < 0 || count > p.N) {
      if (i == 0 && g0 == 0 && e == 0) record_bounds(p.pg.status);
      count = min(max(count, 0), p.N);
    }
  }
  const bool real = i < count;
  // where the token goes, and by which angles it turns
  const int64_t pos = (int64_t)p.start[b] + i;
  bool turn_ok = real, store_ok = real;
  int page = -1;
  float c[8], s[8];
  const bool turns = e < p.rot / 16;
  if (real) {
    if (pos < 0 || pos >= (int64_t)p.pg.table_width << p.pg.page_shift) {
      record_bounds(p.pg.status);
      store_ok = false;
    } else {
      page = page_of(p.pg, b, (int)pos);
      store_ok = page >= 0;
    }
    if (p.rot > 0) {
      const int64_t r = p.positions ? (int64_t)p.positions[token] : pos;
      if (r < 0 || r >= p.table_len) {
        record_bounds(p.pg.status);
        turn_ok = store_ok = false;
      } else if (turns) {
        const float4* cp = reinterpret_cast<const float4*>(p.cos + r * (p.rot / 2) + 8 * e);
        const float4* sp = reinterpret_cast<const float4*>(p.sin + r * (p.rot / 2) + 8 * e);
        const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
        c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
        s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
      }
    }
  }
  // offsets of the two chunks
  int a = 16 * e, bo = 16 * e + 8;
  if (turns && !p.interleaved) {
    a = 8 * e;
    bo = p.rot / 2 + 8 * e;
  }
  const int Hq = p.q ? p.Hq : 0, Hkv = p.pg.Hkv, step = 1 << gpt_log2;
  int r = g0;
  {
    const __nv_bfloat16* qb = p.q + b * p.qs[0] + i * p.qs[1];
    __nv_bfloat16* ob = p.q_out + token * Hq * D;
    for (; r < Hq; r += step) {
      uint32_t w[8] = {};
      if (turn_ok) {
        float x[16];
        load_chunks(qb + r * p.qs[2], a, bo, x);
        if (turns) rotate<false>(x, c, s, p.interleaved);
        pack_chunks(x, w);
      }
      store_chunks(ob + (int64_t)r * D, a, bo, w);
    }
  }
  if (!store_ok) return;
  const __nv_bfloat16 *kb = p.k + b * p.ks[0] + i * p.ks[1], *vb = p.v + b * p.vs[0] + i * p.vs[1];
  for (r -= Hq; r < 2 * Hkv; r += step) {
    float x[16];
    uint32_t w[8];
    const bool is_k = r < Hkv;
    const int h = is_k ? r : r - Hkv;
    load_chunks(is_k ? kb + h * p.ks[2] : vb + h * p.vs[2], a, bo, x);
    if (is_k && turns) rotate<BITS == 4>(x, c, s, p.interleaved);
    pack_chunks(x, w);
    const int64_t row = row_of(p.pg, page, h, (int)pos);
    uint8_t* dst = (is_k ? p.pg.k : p.pg.v) + row * (BITS == 4 ? D / 2 : 2 * D);
    if (BITS == 16) {
      store_chunks(reinterpret_cast<__nv_bfloat16*>(dst), a, bo, w);
      continue;
    }
    // Minimum and negated maximum of the row, side by side in one bf16 pair (NaN stays NaN).
    uint32_t ends;
    {
      uint32_t mn = w[0], mx = w[0] ^ 0x80008000u;
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        mn = min2(mn, w[j]);
        mx = min2(mx, w[j] ^ 0x80008000u);
      }
      ends = min2(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) ends = min2(ends, __shfl_xor_sync(gmask, ends, o));
    float lo = __uint_as_float(ends << 16);
    const float spread = -__uint_as_float(ends & 0xffff0000u) - lo;
    const uint32_t sm = spread < INFINITY ? pack_bf16x2(__fdiv_rn(spread, 15.f), lo) : 0x7fff7fffu;  // else NaN
    float scale = __uint_as_float(sm << 16);
    uint32_t w0 = 0u, w1 = 0u;
    if (scale > 0.f) {  // false for a row of equal values and for NaN
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
      const bool tiny = scale < 0x1p-100f;
      if (tiny) {  // no reciprocal: the row is scaled by a power of two
        scale *= 0x1p64f;
        lo *= 0x1p64f;
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= 0x1p64f;
      }
      const float inv = 1.f / scale, half = 0.5f * scale;
      // codes are put together four at a time as a sum of code * 16^j, exact in fp32
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float k = code_of(x[j], lo, scale, inv, half);
        if (tiny) k = fminf(k, 15.f);  // the scale of so small a spread may be rounded down by a half
        part[j >> 2] = fmaf(k, (float)(1 << (4 * (j & 3))), part[j >> 2]);
      }
      w0 = (uint32_t)part[0] | (uint32_t)part[1] << 16;
      w1 = (uint32_t)part[2] | (uint32_t)part[3] << 16;
    }
    *reinterpret_cast<uint32_t*>(dst + a / 2) = w0;
    *reinterpret_cast<uint32_t*>(dst + bo / 2) = w1;
    if (e == 0) (is_k ? p.pg.k_scales : p.pg.v_scales)[row] = sm;
  }
}

// Eight values minimum + scale * code (codes: nibbles of x, in order) as four
// bf16 pairs.  A fused bf16 multiply-add rounds the exact value once; the
// same comes of rounding it to fp32 and then to bf16, since the sum has at most
// 24 bits wherever it lies near the middle of two bf16 values (a code times a
// scale has 12, and more than 12 binary places below the minimum's last it
// cannot reach that middle).
__device__ __forceinline__ void values8(uint32_t x, __nv_bfloat162 scale, __nv_bfloat162 lo, uint32_t* out) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // codes i and i + 4
    uint32_t y;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(y) : "r"(x >> (4 * i)));  // 128 + code
    asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(0x43004300u));
    const __nv_bfloat162 r = __hfma2(scale, *reinterpret_cast<__nv_bfloat162*>(&y), lo);
    v[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  out[0] = __byte_perm(v[0], v[1], 0x5410);
  out[1] = __byte_perm(v[2], v[3], 0x5410);
  out[2] = __byte_perm(v[0], v[1], 0x7632);
  out[3] = __byte_perm(v[2], v[3], 0x7632);
}

// One thread writes 16 values of k and of v (32-byte stores where the outputs allow, whole rows by
// D/16 lanes): neighbouring lanes take neighbouring heads of one token, as the
// output has them.
template <int D, int BITS>
__global__ void __launch_bounds__(256) paged_gather_kernel(GatherParams p, int64_t total) {
  constexpr int L = D / 16;
  const int64_t t = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (t >= total) return;
  const int e = (int)(t % L);
  const int64_t out_row = t / L;  // (b, j, h)
  const int h = (int)(out_row % p.pg.Hkv);
  const int64_t bj = out_row / p.pg.Hkv;
  const int b = (int)(bj / p.N), j = (int)(bj % p.N);
  uint32_t wk[8] = {}, wv[8] = {};
  if (j < checked_len(p.pg, p.lens, b)) {
    const int page = page_of(p.pg, b, j);
    if (page >= 0) {
      const int64_t row = row_of(p.pg, page, h, j);
      if (BITS == 16) {
        const uint4* sk = reinterpret_cast<const uint4*>(p.pg.k + row * (2 * D) + 32 * e);
        const uint4* sv = reinterpret_cast<const uint4*>(p.pg.v + row * (2 * D) + 32 * e);
        const uint4 k0 = sk[0], k1 = sk[1], v0 = sv[0], v1 = sv[1];
        wk[0] = k0.x; wk[1] = k0.y; wk[2] = k0.z; wk[3] = k0.w; wk[4] = k1.x; wk[5] = k1.y; wk[6] = k1.z; wk[7] = k1.w;
        wv[0] = v0.x; wv[1] = v0.y; wv[2] = v0.z; wv[3] = v0.w; wv[4] = v1.x; wv[5] = v1.y; wv[6] = v1.z; wv[7] = v1.w;
      } else {
        const uint2 ck = *reinterpret_cast<const uint2*>(p.pg.k + row * (D / 2) + 8 * e);
        const uint2 cv = *reinterpret_cast<const uint2*>(p.pg.v + row * (D / 2) + 8 * e);
        const uint32_t ks = p.pg.k_scales[row], vs = p.pg.v_scales[row];
        const __nv_bfloat162 km = *reinterpret_cast<const __nv_bfloat162*>(&ks);
        const __nv_bfloat162 vm = *reinterpret_cast<const __nv_bfloat162*>(&vs);
        values8(ck.x, __low2bfloat162(km), __high2bfloat162(km), wk);
        values8(ck.y, __low2bfloat162(km), __high2bfloat162(km), wk + 4);
        values8(cv.x, __low2bfloat162(vm), __high2bfloat162(vm), wv);
        values8(cv.y, __low2bfloat162(vm), __high2bfloat162(vm), wv + 4);
      }
    }
  }
  __nv_bfloat16 *ok = p.k + out_row * D + 16 * e, *ov = p.v + out_row * D + 16 * e;
  if (p.wide) {
    st_global_v8_na(ok, wk);
    st_global_v8_na(ov, wv);
  } else {  // outputs inside a buffer, 16-byte aligned as everything else
    st_global_v4_na(ok, wk[0], wk[1], wk[2], wk[3]);
    st_global_v4_na(ok + 8, wk[4], wk[5], wk[6], wk[7]);
    st_global_v4_na(ov, wv[0], wv[1], wv[2], wv[3]);
    st_global_v4_na(ov + 8, wv[4], wv[5], wv[6], wv[7]);
  }
}

}  // namespace

cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t st) {
  const int64_t tokens = (int64_t)p.pg.B * p.N;
  if (tokens == 0) return cudaSuccess;
  const int L = p.pg.d / 16, rows = (p.q ? p.Hq : 0) + 2 * p.pg.Hkv;
  // Lane groups per token (log2).  Few groups share a token's place and angles among many rows (8192 tokens of
  // 48 bf16 rows: 4 groups 36.6 us, 8 groups 37.4, 16 groups 38.7; rows stored in 4 bits take longer each, and
  // 8 groups are best: 40.7 us with the gather; at 72 registers 43.4 against 47.7 with 4 and 43.6 with 16); a
  // small call spreads over the device, at most one group a row.
  int gl = 0;
  while ((1 << gl) < rows && (1 << gl) < 128 / L && (gl < (p.pg.bits == 4 ? 3 : 2) || (tokens << gl) * L / 32 < 148 * 32)) ++gl;
  const int64_t threads = (tokens << gl) * L;
  const unsigned blocks = (unsigned)((threads + 127) / 128);
  note_launch();
  if (p.pg.d == 128) {
    if (p.pg.bits == 4) paged_append_kernel<128, 4><<<blocks, 128, 0, st>>>(p, gl);
    else paged_append_kernel<128, 16><<<blocks, 128, 0, st>>>(p, gl);
  } else {
    if (p.pg.bits == 4) paged_append_kernel<64, 4><<<blocks, 128, 0, st>>>(p, gl);
    else paged_append_kernel<64, 16><<<blocks, 128, 0, st>>>(p, gl);
  }
  return cudaGetLastError();
}

cudaError_t launch_paged_gather(const GatherParams& p, cudaStream_t st) {
  const int64_t total = (int64_t)p.pg.B * p.N * p.pg.Hkv * (p.pg.d / 16);
  if (total == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)((total + 255) / 256);
  note_launch();
  if (p.pg.d == 128) {
    if (p.pg.bits == 4) paged_gather_kernel<128, 4><<<blocks, 256, 0, st>>>(p, total);
    else paged_gather_kernel<128, 16><<<blocks, 256, 0, st>>>(p, total);
  } else {
    if (p.pg.bits == 4) paged_gather_kernel<64, 4><<<blocks, 256, 0, st>>>(p, total);
    else paged_gather_kernel<64, 16><<<blocks, 256, 0, st>>>(p, total);
  }
  return cudaGetLastError();
}

}  // namespace fm
