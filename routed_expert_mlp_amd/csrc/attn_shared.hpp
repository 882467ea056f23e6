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
//
// Sequences may see different keys of the prefix (they end inside it, or have
// windows), and 0 * inf is NaN: a part of a column that comes out as NaN where that
// may be so is computed again with the column's own keys alone (attn_part_alone, by
// one wavefront on the vector units).  Such batches take 64 additions a part to know
// it, others nothing.  64 sequences of 1 to 33000 keys behind 32768, 32/8 heads of 128
// dims: 58 us, and 186 us with a page of infinities in the middle.
//
// What bounds it: few rows behind a short prefix, two launches (4 sequences behind
// 1024 keys, 32/8 heads of 128 dims: 10.4 us); many behind a long one, the prefix's
// products and bytes, then the own keys' bytes, then the parts' sums, one after the
// other (64 sequences behind 32768 keys with up to 1024 of their own: 46, 33 and 10
// us; with up to 256 of their own 62 us in all, and 498 us by moe_attn_decode).
#pragma once

#include "attn.hpp"
#include "attn_decode.hpp"
#include "attn_prefill.hpp"

namespace moe {

// A row has RW wavefronts; lane i of each has part i's maximum and sum (64 at a
// time): the prefix's p_splits parts first, then the sequence's own.  A lane takes 4
// dims, so that a wavefront has 256 / D parts' sums in each load, UNROLL loads in
// flight; the wavefronts' shares are added up in LDS.  A part whose sum is 0 has no
// values to read.  Few rows have 4 wavefronts each, 1024 or more one (2048 rows of
// 33 to 36 parts of 128 dims 10.4 us, and 9.5 us with four, 2304 of 25 of 64 dims
// 5.5 and 7.3 us; 2 dims a lane and one part a load: 20.7 and 10.4 us).
template <int D, int RW>
__global__ __launch_bounds__(256) void k_attn_shared_join(AttnArgs a) {
  constexpr int LR = D / 4, PW = 64 / LR, UNROLL = 4;        // lanes of a part, parts of a load
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int cols = a.n_q * a.group;
  const int row = blockIdx.x * (4 / RW) + w / RW;
  const int col = row % cols, kvh = (row / cols) % a.kv_heads, b = row / cols / a.kv_heads;
  __shared__ f32x4 share[4][64];
  const int64_t item = ((static_cast<int64_t>(b) * a.kv_heads + kvh) * cols + col) * a.splits;
  const int64_t p_item = (static_cast<int64_t>(kvh) * (a.B * cols) + b * cols + col) * a.p_splits;
  const float2* const ml = reinterpret_cast<const float2*>(a.ml) + item;
  const float2* const pml = reinterpret_cast<const float2*>(a.pml) + p_item;
  const int at = 4 * (lane % LR), sub = lane / LR;
  const float* const sums = a.ws + item * D + at;
  const float* const p_sums = a.pws + p_item * D + at;
  float L = 0.0f;
  f32x4 o = {};
  AttnSeq s{};
  if (RW == 4 || b < a.B) {
    s = attn_seq(a, b);
    const AttnTiles tl = attn_tiles_between<32>(a, a.shared, attn_window_lo(a, s.first), s.len);
    const int lead = a.p_splits, parts = lead + (tl.n + a.tiles_per_split - 1) / a.tiles_per_split;
    float M = ATTN_NO_MAX;
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
      o *= old;
      for (int i0 = PW * (w % RW); i0 < here; i0 += PW * RW * UNROLL) {
        f32x4 v[UNROLL];
        float g[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          const int i = i0 + PW * RW * u + sub, in = min(i, here - 1), part = p0 + in;
          const float* src = part < lead ? p_sums + static_cast<int64_t>(part) * D
                                         : sums + static_cast<int64_t>(part - lead) * D;
          v[u] = *reinterpret_cast<const f32x4*>(src);
          g[u] = __shfl(f, in);
          if (i >= here) g[u] = 0.0f;
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] += g[u] != 0.0f ? v[u][j] * g[u] : 0.0f;
      }
    }
  }
  share[w][lane] = o;
  __syncthreads();
  if ((RW == 4 ? w != 0 : b >= a.B) || sub) return;
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int j = 0; j < PW; ++j)
      if (i || j) o += share[w + i][j * LR + lane];
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
  uint16_t* out = a.out + attn_row(a, s.row0, kvh, col) * D + at;
  *reinterpret_cast<uint2*>(out) = uint2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
}

}  // namespace moe
