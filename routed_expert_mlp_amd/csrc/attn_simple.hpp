// Attention of one query row by one wavefront: scores with a lane per key,
// then the weighted sum of values with a lane per dim.  Right for every case,
// and slow: each query head reads its keys and values by itself.
#pragma once

#include "attn.hpp"

namespace moe {

template <int D>
__global__ __launch_bounds__(64) void k_attn_row(AttnArgs a) {
  const int h = blockIdx.x % a.heads, i = (blockIdx.x / a.heads) % a.n_q, b = blockIdx.x / a.heads / a.n_q;
  const int lane = threadIdx.x;
  const AttnSeq s = attn_seq(a, b);
  if (i >= s.n) return;
  const int kvh = h / a.group;
  const int p = s.len - s.n + i;
  const int lo = attn_window_lo(a, p);
  const int64_t qo = ((s.row0 + i) * a.heads + h) * D;
  __shared__ float lq[D], lp[64];
  for (int d = lane; d < D; d += 64) lq[d] = bf16_to_f32(a.q[qo + d]) * a.scale_log2;
  __syncthreads();
  constexpr int ND = D / 64;
  float m = -INFINITY, l = 0.0f, o[ND] = {};
  const int ps = 1 << a.page_shift;
  const int64_t page_elems = static_cast<int64_t>(a.kv_heads) * D << a.page_shift;
  const int64_t head_elems = static_cast<int64_t>(D) << a.page_shift;
  for (int k0 = 0; k0 <= p; k0 += 64) {
    if (k0 >= a.sinks && k0 + 64 <= lo) continue;
    const int key = k0 + lane;
    const bool seen = attn_visible(key, p, lo, a.sinks);
    float x = -INFINITY;
    if (seen) {
      const int id = min(max(a.page_table[b * a.max_pages + (key >> a.page_shift)], 0), a.n_pages - 1);
      const uint16_t* kp = a.k + id * page_elems + kvh * head_elems + (key & (ps - 1)) * 8;
      x = 0.0f;
      for (int c = 0; c < D / 8; ++c)
        for (int j = 0; j < 8; ++j) x += lq[8 * c + j] * bf16_to_f32(kp[static_cast<int64_t>(c) * ps * 8 + j]);
    }
    float mx = x;
    for (int w = 32; w; w >>= 1) mx = fmaxf(mx, __shfl_xor(mx, w));
    if (mx == -INFINITY) continue;
    const float mn = fmaxf(m, mx), r = exp2f(m - mn);
    const float e = seen ? exp2f(x - mn) : 0.0f;
    m = mn;
    l = l * r + e;
    lp[lane] = e;
    __syncthreads();
    for (int n = 0; n < ND; ++n) o[n] *= r;
    for (int j = 0; j < 64; ++j) {
      const float pj = lp[j];
      if (pj == 0.0f) continue;
      const int kk = k0 + j;
      const int id = min(max(a.page_table[b * a.max_pages + (kk >> a.page_shift)], 0), a.n_pages - 1);
      const int at = kk & (ps - 1);
      const uint16_t* vp = a.v + id * page_elems + kvh * head_elems + static_cast<int64_t>(at >> 3) * D * 8 + (at & 7);
      for (int n = 0; n < ND; ++n) o[n] += pj * bf16_to_f32(vp[(n * 64 + lane) * 8]);
    }
    __syncthreads();
  }
  for (int w = 32; w; w >>= 1) l += __shfl_xor(l, w);
  for (int n = 0; n < ND; ++n) a.out[qo + n * 64 + lane] = f32_to_bf16(l > 0.0f ? o[n] / l : 0.0f);
}

}  // namespace moe
