// Head norms, rotation and cache append of new tokens.
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (a, b) -> (a c - b s, b c + a s)
//
// A lane holds 8 neighbouring dims (16 bytes) of one head row, D / 8 lanes a
// row, so the mean square is a reduction over D / 8 lanes and the other half
// of a rotated pair is in the same lane (neighbouring pairs) or rotary / 16
// lanes away (halves).  Everything is fp32 between the load and one rounding.
#pragma once

#include "attn.hpp"

namespace moe {

struct PrepArgs {
  const uint16_t* qkv;
  uint16_t* k;
  uint16_t* v;
  uint16_t* q_out;
  const float* qw;
  const float* kw;
  const float* cos_sin;
  const int32_t* positions;
  const int64_t* slots;
  int64_t stride, T, n_positions, n_slots;
  int32_t heads, kv_heads, page_shift, rotary, interleaved;
  float eps;
};

// blockIdx.x: block of 2048 / D tokens (256 threads of 8 dims); blockIdx.y:
// head row of qkv (query heads, key heads, value heads).
template <int D>
__global__ __launch_bounds__(256) void k_attn_prepare(PrepArgs a) {
  constexpr int LR = D / 8, TB = 256 / LR;
  const int tid = threadIdx.x, c = tid % LR, tt = tid / LR;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TB + tt;
  const int h = blockIdx.y;
  const bool live = t < a.T;
  const int64_t tl = live ? t : a.T - 1;
  const uint4 raw = *reinterpret_cast<const uint4*>(a.qkv + tl * a.stride + static_cast<int64_t>(h) * D + 8 * c);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const int64_t slot = live && h >= a.heads ? a.slots[t] : -1;
  const bool store = slot >= 0 && slot < a.n_slots;
  const int ps = 1 << a.page_shift;
  const int64_t page = slot >> a.page_shift;
  const int at = static_cast<int>(slot & (ps - 1));
  if (h >= a.heads + a.kv_heads) {
    if (!store) return;
    const int64_t o = (page * a.kv_heads + (h - a.heads - a.kv_heads)) * (static_cast<int64_t>(D) << a.page_shift) +
                      (static_cast<int64_t>(at >> 3) * D + 8 * c) * 8 + (at & 7);
#pragma unroll
    for (int j = 0; j < 8; ++j) a.v[o + 8 * j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    return;
  }
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = bf16_to_f32(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
  const bool isq = h < a.heads;
  const float* nw = isq ? a.qw : a.kw;
  if (nw) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
#pragma unroll
    for (int m = 1; m < LR; m <<= 1) s += __shfl_xor(s, m);
    const float r = 1.0f / sqrtf(s * (1.0f / D) + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * r * nw[8 * c + j];
  }
  if (a.rotary) {
    const int64_t pos = min(max(static_cast<int64_t>(a.positions[tl]), int64_t(0)), a.n_positions - 1);
    const float* cs = a.cos_sin + pos * a.rotary;
    const int half = a.rotary >> 1;
    if (a.interleaved) {
      if (8 * c < a.rotary) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float co = cs[4 * c + j], si = cs[half + 4 * c + j];
          const float p = x[2 * j], q = x[2 * j + 1];
          x[2 * j] = p * co - q * si;
          x[2 * j + 1] = q * co + p * si;
        }
      }
    } else {
      const int hl = half >> 3;                 // lanes of half a rotation
      const int lane = tid & 63;
      const int other = c < hl ? lane + hl : c < 2 * hl ? lane - hl : lane;
      const int i0 = 8 * (c < hl ? c : c - hl);
      const float sg = c < hl ? -1.0f : 1.0f;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __shfl(x[j], other);
      if (c < 2 * hl) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * cs[i0 + j] + sg * y[j] * cs[half + i0 + j];
      }
    }
  }
  const uint4 res = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7])};
  if (isq) {
    if (live) *reinterpret_cast<uint4*>(a.q_out + (t * a.heads + h) * D + 8 * c) = res;
  } else if (store) {
    const int64_t o = (page * a.kv_heads + (h - a.heads)) * (static_cast<int64_t>(D) << a.page_shift) +
                      (static_cast<int64_t>(c) * ps + at) * 8;
    *reinterpret_cast<uint4*>(a.k + o) = res;
  }
}

}  // namespace moe
