// Attention over a paged key/value cache: one warp per row.
#include <cuda_bf16.h>

#include "launchers.h"
#include "paged.cuh"
#include "sm100_primitives.cuh"

namespace fm {
namespace {

template <int D, int BITS>
__global__ void __launch_bounds__(128) paged_attention_kernel(PagedAttnParams p) {
  constexpr int E = D / 32;  // values of a row per lane
  const int lane = threadIdx.x & 31;
  const int64_t w = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  if (w >= (int64_t)p.pg.B * p.Nq * p.Hq) return;
  const int h = (int)(w % p.Hq);
  const int64_t bi = w / p.Hq;
  const int i = (int)(bi % p.Nq), b = (int)(bi / p.Nq);
  const int len = checked_len(p.pg, p.lens, b);
  const int64_t pos = (p.start ? (int64_t)p.start[b] : (int64_t)len - p.Nq) + i;
  const int kvh = h / p.G, hm = p.Hm == 1 ? 0 : h;
  float q[E], acc[E];
  const __nv_bfloat16* qp = p.q + b * p.qs[0] + i * p.qs[1] + h * p.qs[2];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qp[lane * E + e]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int64_t end = p.causal ? min((int64_t)len, pos + 1) : len;
  for (int j = 0; j < end; ++j) {
    if (j < p.Nm) {
      const int64_t at = ((int64_t)b * p.Hm + hm) * p.Nm + j;
      if (p.lts && p.lts[at] <= pos && pos < p.lte[at]) continue;
      if (p.uts && p.uts[at] <= pos && pos < p.ute[at]) continue;
    }
    const int page = page_of(p.pg, b, j);
    if (page < 0) continue;
    const int64_t row = row_of(p.pg, page, kvh, j);
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int x = lane * E + e;
      if (BITS == 16) {
        k[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.pg.k)[row * D + x]);
        v[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.pg.v)[row * D + x]);
      } else {
        const uint32_t ks = p.pg.k_scales[row], vs = p.pg.v_scales[row];
        const int ck = (p.pg.k[row * (D / 2) + x / 2] >> (4 * (x & 1))) & 15;
        const int cv = (p.pg.v[row * (D / 2) + x / 2] >> (4 * (x & 1))) & 15;
        k[e] = fmaf(__uint_as_float(ks << 16), (float)ck, __uint_as_float(ks & 0xffff0000u));
        v[e] = fmaf(__uint_as_float(vs << 16), (float)cv, __uint_as_float(vs & 0xffff0000u));
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), keep = m == -INFINITY ? 0.f : exp2f(m - mn), pr = exp2f(s - mn);
    l = l * keep + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(pr, v[e], acc[e] * keep);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) p.o[w * D + lane * E + e] = __float2bfloat16(acc[e] * inv);
  if (lane == 0)
    p.lse[((int64_t)b * p.Hq + h) * p.Nq + i] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnParams& p, cudaStream_t st) {
  const int64_t warps = (int64_t)p.pg.B * p.Nq * p.Hq;
  if (warps == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)((warps + 3) / 4);
  note_launch();
  if (p.pg.d == 128) {
    if (p.pg.bits == 4) paged_attention_kernel<128, 4><<<blocks, 128, 0, st>>>(p);
    else paged_attention_kernel<128, 16><<<blocks, 128, 0, st>>>(p);
  } else {
    if (p.pg.bits == 4) paged_attention_kernel<64, 4><<<blocks, 128, 0, st>>>(p);
    else paged_attention_kernel<64, 16><<<blocks, 128, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fm
