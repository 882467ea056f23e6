// Head norms, rotation and cache append of new tokens.
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (a, b) -> (a c - b s, b c + a s)
//
// What bounds it: the rows are read once and written once, a few operations a
// value; with one token, the launch.  So:
//   * a lane holds 8 dims of one row, D / 8 lanes a row, in two pieces of 4: the
//     two halves of 4 rotated pairs, or 8 neighbouring dims.  Either way the
//     rotation stays in the lane and takes the table's entries 4 c .. 4 c + 3,
//     and the mean square is a sum over D / 8 lanes; everything is fp32 between
//     the load and one rounding;
//   * a block keeps its 2048 / D tokens and goes through several heads, so that
//     a token's cosines and sines, as long as two of its rows, are read once
//     for all of them and the next row is on its way while one is worked on;
//   * the cache's order of keys (16 bytes of a token, then the next token's) and
//     of values (8 tokens of a dim) is made in LDS, so that the stores are runs
//     of a block's tokens.  Eight tokens whose slots are not one aligned run of
//     8 store their values one by one.
//
// Measured, 32 query and 8 key/value heads of 128 dims: 4096 tokens 21.5 us, 4.8
// TB/s, the rate of a large copy; one token 2.7 us in a graph, a launch; 2056
// tokens of 128/8 heads of 256 dims 64-69 us, 4.4-4.8 TB/s, and 85-92 us if each
// is of another sequence: its keys and values then go out in pieces of 16 and 2
// bytes.  7 wavefronts a SIMD are the best number (8, with 64 registers: 69-86 us;
// 6: 66-70 us).
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
  int32_t rows_per_block;    // heads that a block goes through
  float eps;
};

// blockIdx.x: block of 2048 / D tokens (256 threads of 8 dims); blockIdx.y:
// rows_per_block rows of qkv (query heads, key heads, value heads).
template <int D>
__global__ __launch_bounds__(256) void k_attn_prepare(PrepArgs a) {
  constexpr int LR = D / 8, TB = 256 / LR;
  const int tid = threadIdx.x, c = tid % LR, tt = tid / LR;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TB;
  const int64_t t = min(t0 + tt, a.T - 1);         // past the end: the last token again, not stored
  const bool live = t0 + tt < a.T;
  const int rows = a.heads + 2 * a.kv_heads;
  const int r0 = blockIdx.y * a.rows_per_block, r1 = min(r0 + a.rows_per_block, rows);
  // this lane's dims: d0 .. d0 + 3 and d1 .. d1 + 3
  const int half = a.rotary >> 1;
  const bool turned = 8 * c < a.rotary;
  const bool apart = turned && !a.interleaved;
  const int d0 = apart ? 4 * c : 8 * c, d1 = apart ? half + 4 * c : 8 * c + 4;
  // one piece of 16 bytes where no lane has two halves (2056 tokens of 128/8 heads
  // of 256 dims, interleaved pairs: 64 us, and 79 us in two pieces)
  const bool joined = a.interleaved || !a.rotary;
  const uint16_t* const x0 = a.qkv + t * a.stride;
  auto load_row = [&](int h, uint2& lo, uint2& hi) {
    const uint16_t* const x = x0 + static_cast<int64_t>(h) * D;
    if (joined) {
      const uint4 v = load_stream(reinterpret_cast<const uint4*>(x + d0));
      lo = uint2{v.x, v.y};
      hi = uint2{v.z, v.w};
    } else {
      lo = load_stream(reinterpret_cast<const uint2*>(x + d0));
      hi = load_stream(reinterpret_cast<const uint2*>(x + d1));
    }
  };
  uint2 raw0, raw1;
  load_row(r0, raw0, raw1);

  __shared__ int64_t lslot[TB];
  __shared__ __align__(16) uint16_t tile[2048];
  const int ps = 1 << a.page_shift;
  if (r1 > a.heads) {
    if (tid < TB) lslot[tid] = t0 + tid < a.T ? a.slots[t0 + tid] : -1;
  }
  f32x4 co = {}, si = {};
  if (turned && r0 < a.heads + a.kv_heads) {
    const int64_t pos = min(max(static_cast<int64_t>(a.positions[t]), int64_t(0)), a.n_positions - 1);
    const float* cs = a.cos_sin + pos * a.rotary + 4 * c;
    co = *reinterpret_cast<const f32x4*>(cs);
    si = *reinterpret_cast<const f32x4*>(cs + half);
  }
  f32x4 n0 = {}, n1 = {};
  if (r1 > a.heads) __syncthreads();

  for (int h = r0; h < r1; ++h) {
    const uint2 now0 = raw0, now1 = raw1;
    if (h + 1 < r1) load_row(h + 1, raw0, raw1);
    const bool isq = h < a.heads;
    if (h >= a.heads + a.kv_heads) {
      // values: thread (g, d) stores dim d of tokens 8 g .. 8 g + 7
      __syncthreads();
      *reinterpret_cast<uint2*>(tile + tt * D + d0) = now0;
      *reinterpret_cast<uint2*>(tile + tt * D + d1) = now1;
      __syncthreads();
      const int d = tid % D, g = tid / D;
      const uint16_t* col = tile + 8 * g * D + d;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = col[2 * j * D] | static_cast<uint32_t>(col[(2 * j + 1) * D]) << 16;
      const int64_t s0 = lslot[8 * g];
      bool run = s0 >= 0 && s0 < a.n_slots && (s0 & 7) == 0;
#pragma unroll
      for (int j = 1; j < 8; ++j) run = run && lslot[8 * g + j] == s0 + j;
      auto place = [&](int64_t slot) {
        return ((slot >> a.page_shift) * a.kv_heads + (h - a.heads - a.kv_heads)) *
                   (static_cast<int64_t>(D) << a.page_shift) +
               (((slot & (ps - 1)) >> 3) * D + d) * 8 + (slot & 7);
      };
      if (run) {
        *reinterpret_cast<uint4*>(a.v + place(s0)) = uint4{w[0], w[1], w[2], w[3]};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t slot = lslot[8 * g + j];
          if (slot >= 0 && slot < a.n_slots) a.v[place(slot)] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
        }
      }
      continue;
    }
    const uint32_t w[4] = {now0.x, now0.y, now1.x, now1.y};
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = bf16_to_f32(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
    const float* norm = isq ? a.qw : a.kw;
    if (norm) {
      if (h == r0 || h == a.heads) {
        n0 = *reinterpret_cast<const f32x4*>(norm + d0);
        n1 = *reinterpret_cast<const f32x4*>(norm + d1);
      }
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
      s = dpp_add<DPP_QUAD_1032>(s);
      s = dpp_add<DPP_QUAD_2301>(s);
      s = dpp_add<DPP_ROW_HALF_MIRROR>(s);
      if (LR > 8) s = dpp_add<DPP_ROW_MIRROR>(s);
      if (LR > 16) s += __shfl_xor(s, 16);
      const float r = 1.0f / sqrtf(s * (1.0f / D) + a.eps);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = x[j] * r * n0[j];
        x[4 + j] = x[4 + j] * r * n1[j];
      }
    }
    if (turned) {      // not a turn by 0: next to an infinity or a NaN that would give a NaN
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // pair j: dims (2 j, 2 j + 1) of the lane's 8, or (j, 4 + j)
        const float p = a.interleaved ? x[2 * j] : x[j], q = a.interleaved ? x[2 * j + 1] : x[4 + j];
        const float u = p * co[j] - q * si[j], v = q * co[j] + p * si[j];
        (a.interleaved ? x[2 * j] : x[j]) = u;
        (a.interleaved ? x[2 * j + 1] : x[4 + j]) = v;
      }
    }
    const uint2 res0 = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    const uint2 res1 = {pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    if (isq) {
      if (live) {
        uint16_t* o = a.q_out + (t * a.heads + h) * D;
        if (joined) {
          *reinterpret_cast<uint4*>(o + d0) = uint4{res0.x, res0.y, res1.x, res1.y};
        } else {
          *reinterpret_cast<uint2*>(o + d0) = res0;
          *reinterpret_cast<uint2*>(o + d1) = res1;
        }
      }
    } else {
      // keys: thread (chunk, token) stores 16 bytes
      __syncthreads();
      *reinterpret_cast<uint2*>(tile + ((d0 >> 3) * TB + tt) * 8 + (d0 & 7)) = res0;
      *reinterpret_cast<uint2*>(tile + ((d1 >> 3) * TB + tt) * 8 + (d1 & 7)) = res1;
      __syncthreads();
      const int ch = tid / TB;
      const int64_t slot = lslot[tid % TB];
      if (slot >= 0 && slot < a.n_slots)
        *reinterpret_cast<uint4*>(a.k + ((slot >> a.page_shift) * a.kv_heads + (h - a.heads)) *
                                            (static_cast<int64_t>(D) << a.page_shift) +
                                  ((static_cast<int64_t>(ch) << a.page_shift) + (slot & (ps - 1))) * 8) =
            *reinterpret_cast<const uint4*>(tile + 8 * tid);
    }
  }
}

}  // namespace moe
