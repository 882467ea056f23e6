// The residual's addition, the RMS norm of the row and its E4M3 form, in one pass.
//
//   h = x + r;  y = h rsqrt(mean(h^2) + eps) w;  per 128 columns s = max|y| / 448, q = e4m3(y / s)
//
// What bounds it: every value is read and written once, for a dozen operations;
// with few rows, the launch (4096 columns, all outputs: 4096 rows 27.4 us, 5.5 TB/s, a
// copy's rate; one row 2.5 us).  So a row is read into registers, WPR wavefronts of
// NV pieces of 8 values a lane, its squares are summed (over the wavefronts in
// LDS), and everything that is asked for goes out from there.  16 neighbouring
// lanes hold the 128 columns of a scale.
//
// The sum, the norm and the scales are in fp32; h and y are each rounded once to
// bf16, the type of the layer's rows, and q once to E4M3, from y before any
// rounding.
#pragma once

#include "common.hpp"

namespace moe {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* r;
  const float* w;
  uint16_t* h;
  uint16_t* y;
  uint8_t* q;
  float* s;
  int64_t x_stride, T;
  int32_t hidden, blocks;    // columns; scales of a row
  float eps, per;            // per: 1 / hidden
};

__device__ __forceinline__ float dpp_max(float v, int o) { return fmaxf(v, __int_as_float(o)); }

// Largest of the 16 lanes of a row.
__device__ __forceinline__ float row_max(float v) {
  v = dpp_max(v, dpp_mov<DPP_QUAD_1032>(__float_as_int(v)));
  v = dpp_max(v, dpp_mov<DPP_QUAD_2301>(__float_as_int(v)));
  v = dpp_max(v, dpp_mov<DPP_ROW_HALF_MIRROR>(__float_as_int(v)));
  return dpp_max(v, dpp_mov<DPP_ROW_MIRROR>(__float_as_int(v)));
}

// Rows that are read once go around the caches (4096 rows of 2048 columns 16.6 us
// with ordinary loads and 15.7 with these, of 4096 30.4 and 30.3, of 16384 115.7 and
// 114.1; 300 of 7168 7.7 and 8.1).
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return uint4{v.x, v.y, v.z, v.w};
}

// Four values to E4M3 bytes, nearest even; |v| < 464, or NaN.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

__device__ __forceinline__ void bf16x8_to_f32(uint4 v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&f)[8]) {
  return uint4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// Eight columns of a block of 128 (16 lanes) on their way to E4M3.
//
// y / scale = h w 448 / max |h w|: the root of the mean is in both.  Near the border
// of two codes every rounding on the way may choose the wrong one, 2^-3 of the value,
// so the products and the quotient are kept with what their rounding left over, and
// what is left of the last one tips a value that lies on a border.
struct E4m3Block {
  float p[8], e[8];          // |h w| = |p + e|
  float top, rest;           // the largest of the block, and what is left over of it
  __device__ __forceinline__ void products(const float (&h)[8], const float (&w)[8]) {
#pragma clang fp contract(off)
    top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = h[j] * w[j];
      e[j] = fmaf(h[j], w[j], -p[j]);
      top = fmaxf(top, fabsf(p[j]));
    }
    top = row_max(top);
    rest = -top;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (fabsf(p[j]) == top) rest = fmaxf(rest, p[j] < 0.0f ? -e[j] : e[j]);
    rest = row_max(rest);
  }
  // s: the scale.
  __device__ __forceinline__ uint2 codes(float inv, float s) const {
#pragma clang fp contract(off)       // the products below are rounded where it says so
    float z[8];
    if (top >= 0x1p-60f && top <= 0x1p100f && s > 1.17549435e-38f) {
      const float one = __builtin_amdgcn_rcpf(top), r = 448.0f * one;
      const float left = (fmaf(-r, top, 448.0f) - r * rest) * one;           // 448 / (top + rest) = r + left
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = p[j] * r, more = fmaf(p[j], r, -m) + fmaf(p[j], left, e[j] * r);
        const float sum = m + more, over = more - (sum - m);
        // borders have 5 bits; one step to the side that the rest is on
        const uint32_t bits = __float_as_uint(sum);
        const bool border = (bits & 0xFFFFu) == 0 && over != 0.0f && sum != 0.0f;
        z[j] = __uint_as_float(bits + (border ? ((over > 0.0f) == (sum > 0.0f) ? 1u : ~0u) : 0u));
      }
    } else {                 // the least scale, values that are not finite
      const float to = 1.0f / s;
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = p[j] * inv * to;
    }
    return uint2{pack_e4m3x4(z[0], z[1], z[2], z[3]), pack_e4m3x4(z[4], z[5], z[6], z[7])};
  }
};

// WPR wavefronts a row (1: four rows a block), NV pieces of 8 values a lane.
template <int WPR, int NV>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * 64) void k_proj_norm(NormArgs a) {
  constexpr int RPB = WPR == 1 ? 4 : 1, LANES = WPR * 64;
  const int lane = threadIdx.x % LANES;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / LANES;
  if (RPB > 1 && t >= a.T) return;
  const int pieces = a.hidden / 8;
  const uint4* const x = reinterpret_cast<const uint4*>(a.x + t * a.x_stride);
  const int64_t row = t * pieces;
  float v[NV][8], weight[NV][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = lane + LANES * i;
    const bool in = p < pieces;
    uint4 raw = {}, res = {};
    if (in) raw = load_once(x + p);
    if (in && a.r) res = load_once(reinterpret_cast<const uint4*>(a.r) + row + p);
    f32x4 w0{1.0f, 1.0f, 1.0f, 1.0f}, w1 = w0;   // on their way before the sum is there (4096 rows 28.8 us behind it)
    if (in && a.w) {
      w0 = reinterpret_cast<const f32x4*>(a.w)[2 * p];
      w1 = reinterpret_cast<const f32x4*>(a.w)[2 * p + 1];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      weight[i][j] = w0[j];
      weight[i][4 + j] = w1[j];
    }
    bf16x8_to_f32(raw, v[i]);
    if (a.r) {
      float f[8];
      bf16x8_to_f32(res, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += f[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
  }
  sum = wave_sum(sum);
  if constexpr (WPR > 1) {
    __shared__ float part[WPR];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = part[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) sum += part[i];
  }
  // the instruction takes numbers below 2^-126 for 0; a factor of 2^96, whose root is exact, keeps them out of its way
  const float mean = fmaf(sum, a.per, a.eps);
  const float inv = mean < 0x1p-96f ? __builtin_amdgcn_rsqf(mean * 0x1p96f) * 0x1p48f : __builtin_amdgcn_rsqf(mean);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = lane + LANES * i;
    const bool in = p < pieces;
    if (in && a.h) reinterpret_cast<uint4*>(a.h)[row + p] = f32_to_bf16x8(v[i]);
    if (in && a.y) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = v[i][j] * (inv * weight[i][j]);
      reinterpret_cast<uint4*>(a.y)[row + p] = f32_to_bf16x8(y);
    }
    if (a.q) {
      E4m3Block q;
      q.products(v[i], weight[i]);            // lanes past the row's end have zeros
      const float s = fmaxf(q.top * inv * (1.0f / 448.0f), 1.17549435e-38f);
      if (in) {
        reinterpret_cast<uint2*>(a.q)[row + p] = q.codes(inv, s);
        if ((lane & 15) == 0) a.s[t * a.blocks + p / 16] = s;
      }
    }
  }
}

}  // namespace moe
