// Decode of a batch whose sequences begin with the same tokens: the keys and
// values of that prefix are in pages of their own, once, and are read once for
// the new tokens of all sequences.
//
//   out = sum_k p_k v_k / sum_k p_k  over the prefix and the own keys of a sequence
//
// in parts, each with its maximum m, its sum l and its sums o of weighted values,
// as decode does for long sequences:
//   * the prefix: the new tokens of the whole batch are the columns of one product
//     per key/value head (attn_decode.hpp's blocks of 32 columns where they are
//     few, attn_prefill.hpp's of 128 or 256 where they are many), each column at
//     its own position;
//   * the own keys of each sequence: k_attn_decode from the end of the prefix on;
//   * k_attn_shared_join adds them up: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
//
// The prefix may end inside a page, and inside a tile: the rest of its last tile is
// masked there, and the keys before its end in the first own tile.
#pragma once

#include "attn.hpp"
#include "attn_decode.hpp"
#include "attn_prefill.hpp"

namespace moe {

// RW wavefronts a row; lane i of each has part i's maximum and sum (64 at a time):
// the prefix's p_splits parts first, then the sequence's own.  A part whose sum is
// 0 has no values to read.
template <int D, int RW>
__global__ __launch_bounds__(256) void k_attn_shared_join(AttnArgs a) {
  constexpr int ND = D / 64, UNROLL = 4;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int cols = a.n_q * a.group;
  const int row = blockIdx.x * (4 / RW) + w / RW;
  const int col = row % cols, kvh = (row / cols) % a.kv_heads, b = row / cols / a.kv_heads;
  if (RW == 1 && b >= a.B) return;
  const int64_t item = ((static_cast<int64_t>(b) * a.kv_heads + kvh) * cols + col) * a.splits;
  const int64_t p_item = (static_cast<int64_t>(kvh) * (a.B * cols) + b * cols + col) * a.p_splits;
  const float2* const ml = reinterpret_cast<const float2*>(a.ml) + item;
  const float2* const pml = reinterpret_cast<const float2*>(a.pml) + p_item;
  const float* const sums = a.ws + item * D + lane * ND;
  const float* const p_sums = a.pws + p_item * D + lane * ND;
  const AttnSeq s = attn_seq(a, b);
  const AttnTiles tl = attn_tiles_between<32>(a, a.shared, attn_window_lo(a, s.first), s.len);
  const int lead = a.p_splits, parts = lead + (tl.n + a.tiles_per_split - 1) / a.tiles_per_split;
  float M = ATTN_NO_MAX, L = 0.0f, o[ND] = {};
  for (int p0 = 0; p0 < parts; p0 += 64) {
    const int here = min(parts - p0, 64), mine = p0 + min(lane, here - 1);
    const float2 p = mine < lead ? pml[mine] : ml[mine - lead];
    const bool live = lane < here && p.y != 0.0f;
    const float m = live ? p.x : ATTN_NO_MAX;
    float mn = fmaxf(M, m);
#pragma unroll
    for (int x = 32; x; x >>= 1) mn = fmaxf(mn, __shfl_xor(mn, x));
    const float f = live ? exp2_fast(m - mn) : 0.0f, old = exp2_fast(M - mn);
    M = mn;
    L = L * old + wave_sum(live ? p.y * f : 0.0f);
#pragma unroll
    for (int n = 0; n < ND; ++n) o[n] *= old;
    for (int i0 = w % RW; i0 < here; i0 += RW * UNROLL) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int i = min(i0 + RW * u, here - 1);
        const float g = i0 + RW * u < here ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), i)) : 0.0f;
        const int part = p0 + i;
        const float* src = part < lead ? p_sums + static_cast<int64_t>(part) * D
                                       : sums + static_cast<int64_t>(part - lead) * D;
#pragma unroll
        for (int n = 0; n < ND; ++n) o[n] += g != 0.0f ? src[n] * g : 0.0f;
      }
    }
  }
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
  uint16_t* out = a.out + attn_row(a, s.row0, kvh, col) * D;
  if constexpr (RW == 1) {
    if constexpr (ND == 1) {
      out[lane] = f32_to_bf16(o[0] * inv);
    } else {
#pragma unroll
      for (int n = 0; n < ND; n += 2)
        *reinterpret_cast<uint32_t*>(out + lane * ND + n) = pack_bf16x2(o[n] * inv, o[n + 1] * inv);
    }
  } else {
    __shared__ float lo_[4][D];
#pragma unroll
    for (int n = 0; n < ND; ++n) lo_[w][lane * ND + n] = o[n];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 256)
      out[d] = f32_to_bf16(((lo_[0][d] + lo_[1][d]) + (lo_[2][d] + lo_[3][d])) * inv);
  }
}

}  // namespace moe
