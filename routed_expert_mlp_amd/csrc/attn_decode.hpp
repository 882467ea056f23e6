// Attention of a few new tokens of each sequence over the paged cache, split
// over the cache's length and joined.
//
//   out = sum_k p_k v_k / sum_k p_k,  p_k = exp2(c q.k - m),  c = scale log2(e)
//
// with the running maximum m per query, in one pass over the keys.
//
// What bounds it: every key and value row is read once for all query heads of
// its group and all new tokens (4 D bytes for 4 D flops per column), so the
// stream from HBM is the floor; the matrix instructions, which carry the
// group's heads as columns of one operand, take a few percent of that time
// even with most columns empty.  So:
//   * K and V go from HBM straight into the operand registers of the matrix
//     instructions, 16 bytes a lane and whole lines an instruction, with no
//     LDS and no transposition: that is what the cache's layout is for;
//   * one block is 4 wavefronts that take tiles of 32 keys in turn, each with
//     its next tile's keys and values in flight while it works on the present
//     one; they join their parts in LDS.  Two blocks share a CU (at 128 dims),
//     so that one streams while the other starts or joins (one block of 8: 106 us
//     where this took 100);
//   * the visible tiles of a sequence are cut into parts of tiles_per_split,
//     a block each; a sequence with one part is done by then, the others'
//     parts (unnormalised sums, maximum and sum, in fp32) are joined by
//     k_attn_join.
//
// Measured, 32 query and 8 key/value heads of 128 dims: one token over 131071 keys
// 87 us, 6.2 TB/s (a large copy reaches 4.8 TB/s, reads and writes together); 64
// sequences of 1..8192 keys 179 us, 6.0 TB/s; 777 keys 8.4-9.5 us, which is two
// launches that wait for one load after the other.
//
// The weights meet the values in bf16, the type that the matrix instruction takes
// them in beside bf16 values; their sum is of the weights before that rounding.
// Against 64 bits the result is off by 1.9e-3 of its size, where rounding it alone
// makes 1.6e-3.
#pragma once

#include "attn.hpp"

namespace moe {

constexpr int ATTN_MAX_TPS = 64;      // most 32-key tiles of a part
constexpr int ATTN_NW = 4;            // wavefronts of a block

// Blocks that a CU holds at once, by the registers of a wavefront's sums and
// operands (at most 256 and 512).  At 64 dims 4 would fit; 2, with longer parts, are
// faster (16 sequences of 4 new tokens, window 4096: 18.4 us, and 19.9 us with 3 or 4).
constexpr int attn_blocks_per_cu(int D) { return D <= 128 ? 2 : 1; }

// Column col of a sequence and key/value head: new token col / group, head col % group.
__device__ __forceinline__ int64_t attn_row(const AttnArgs& a, int64_t row0, int kvh, int col) {
  const int t = col / a.group;
  return (row0 + t) * a.heads + kvh * a.group + (col - t * a.group);
}

// More rows of a head than 32 (heads of the group x new tokens) take several
// blocks, which read the same keys (AGAIN): through the caches then, around them
// otherwise (64 sequences of up to 4096 keys, 32/8 heads of 128 dims, one token: 136
// us around, 156 us through).  Blocks of 64 rows, which read the keys once, have
// half as many blocks, and wavefronts, a CU: 8 sequences of 8 new tokens of 64/2
// heads 44 us, and 35 us in blocks of 32; 64 of 4 tokens of 64/4 heads 100 and
// 107 us, the only case of many where they were faster.
template <int D, bool AGAIN>
__global__ __launch_bounds__(ATTN_NW * 64, attn_blocks_per_cu(D)) void k_attn_decode(AttnArgs a) {
  constexpr int NW = ATTN_NW, KS = D / 16, DT = D / 32, COLS = 32, LD = D + 4;
  const int cols = a.n_q * a.group;
  const int col_blocks = (cols + COLS - 1) / COLS;
  // the parts of a sequence run slowest: with parts next to each other, the
  // later ones, which shorter sequences lack, would all fall to the same XCDs
  // (64 sequences of 1..8192 keys: 209 us that way, 180 us this way)
  // the column blocks that read the same keys are 8 blocks apart, on one XCD at
  // about the same time, so that its L2 has the keys for the second (64 sequences
  // of 4 new tokens, 64/4 heads of 256 dims, up to 4096 keys: 305 us next to each
  // other and around the caches, 237 us this way, 211 us through the caches too)
  const int cb = static_cast<int>(blockIdx.x / 8) % col_blocks;
  int bi = static_cast<int>(blockIdx.x / (8 * col_blocks)) * 8 + blockIdx.x % 8;
  const int kvh = bi % a.kv_heads;
  bi /= a.kv_heads;
  const int b = bi % a.B, split = bi / a.B;
  if (split >= a.splits) return;
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, half = lane >> 5;
  const int w = uniform(tid >> 6);
  // the queries are on their way before the sequence's length is known
  bf16x8 qf[KS];
  const int col = min(cb * COLS + r, cols - 1);
  const int tok = col / a.group;                   // new token of this lane's column
  const uint16_t* qp = a.q + attn_row(a, static_cast<int64_t>(b) * a.n_q, kvh, col) * D + 8 * half;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) qf[ks] = *reinterpret_cast<const bf16x8*>(qp + 16 * ks);
  const AttnSeq s = attn_seq(a, b);
  const int first = s.first;
  AttnTiles tl = attn_tiles<32>(a, first, s.len - 1);
  const bool whole = tl.n <= a.tiles_per_split;
  if (!tl.keep_part(split, a.tiles_per_split)) return;

  __shared__ int ids[2 * ATTN_MAX_TPS];
  __shared__ float lm[NW][COLS], ll[NW][COLS];
  __shared__ float lo_[NW / 2][COLS * LD];

  // page of each 16 keys of this part
  for (int i = tid; i < 2 * tl.n; i += NW * 64) {
    const int key = min(32 * tl.tile(i >> 1) + 16 * (i & 1), s.len - 1);
    ids[i] = min(max(a.page_table[b * a.max_pages + (key >> a.page_shift)], 0), a.n_pages - 1);
  }

  const int pos = first + tok;
  __syncthreads();

  const int ps = 1 << a.page_shift;
  const int64_t head_elems = static_cast<int64_t>(D) << a.page_shift;
  auto load = [](const uint16_t* p) {
    return AGAIN ? *reinterpret_cast<const uint4*>(p) : load_stream(reinterpret_cast<const uint4*>(p));
  };
  auto load_k = [&](int v, uint4 (&kf)[KS]) {
    const int key = 32 * tl.tile(v) + swap23(r);
    const int64_t base = (static_cast<int64_t>(ids[2 * v + (r >> 4)]) * a.kv_heads + kvh) * head_elems +
                         ((half << a.page_shift) + (key & (ps - 1))) * 8;
    const uint16_t* p = a.k + base;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) kf[ks] = load(p + ((2 * ks * 8) << a.page_shift));
  };
  auto load_v = [&](int v, uint4 (&vf)[2][DT]) {
    const int key0 = 32 * tl.tile(v);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int at = ((key0 + 16 * g) & (ps - 1)) + 8 * half;
      const uint16_t* p = a.v + (static_cast<int64_t>(ids[2 * v + g]) * a.kv_heads + kvh) * head_elems +
                          at * D + r * 8;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) vf[g][dt] = load(p + 32 * 8 * dt);
    }
  };

  f32x16 acc[DT];
  float m = ATTN_NO_MAX, l = 0.0f;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[dt][e] = 0.0f;
  uint4 kf[KS], vf[2][DT];
  int v = w;
  if (v < tl.n) {
    load_k(v, kf);
    load_v(v, vf);
  }
  for (; v < tl.n; v += NW) {
    f32x16 sc;
#pragma unroll
    for (int e = 0; e < 16; ++e) sc[e] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf[ks]), qf[ks], sc, 0, 0, 0);
    const int vn = v + NW;
    if (vn < tl.n) load_k(vn, kf);
    const int key0 = 32 * tl.tile(v);
    // a tile that some column sees only in part: scores of invisible keys go to
    // -inf, and the values of keys that nobody sees, whatever the slots hold, to 0
    if (key0 + 31 > first || (a.window && key0 < max(0, s.len - a.window) && key0 + 31 >= tl.sinks)) {
      const uint32_t see = static_cast<uint32_t>(
          visible_bits(key0 + 8 * half, pos, attn_window_lo(a, pos), tl.sinks));
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[e] = keep_if(see, 16 * (e >> 3) + (e & 7), sc[e]);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint4 mk = value_mask(static_cast<uint32_t>(
            visible_bits(key0 + 16 * g + 8 * half, tl.hi - 1, tl.lo, tl.sinks)));
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) vf[g][dt] = and4(vf[g][dt], mk);
      }
    }
    float mx = sc[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) mx = fmaxf(mx, sc[e]);
    const float mn = fmaxf(m, max_halves(mx) * a.scale_log2);
    if (__any(mn > m)) {
      const float f = exp2_fast(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[dt][e] *= f;
    }
    uint32_t pk[8];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float p0 = exp2_fast(fmaf(sc[e], a.scale_log2, -m));
      const float p1 = exp2_fast(fmaf(sc[e + 1], a.scale_log2, -m));
      l += p0 + p1;
      pk[e >> 1] = pack_bf16x2(p0, p1);
    }
    const uint4 pf[2] = {{pk[0], pk[1], pk[2], pk[3]}, {pk[4], pk[5], pk[6], pk[7]}};
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
        acc[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf[g][dt]),
                                                          __builtin_bit_cast(bf16x8, pf[g]), acc[dt], 0, 0, 0);
    if (vn < tl.n) load_v(vn, vf);
  }

  // join the wavefronts: common maximum, then the sums in a tree
  const int live = min(cols - cb * COLS, COLS);
  const float lt = sum_halves(l);
  if (half == 0) {
    lm[w][r] = m;
    ll[w][r] = lt;
  }
  __syncthreads();
  float M = lm[0][r], L = 0.0f;
#pragma unroll
  for (int i = 1; i < NW; ++i) M = fmaxf(M, lm[i][r]);
#pragma unroll
  for (int i = 0; i < NW; ++i) L += ll[i][r] * exp2_fast(lm[i][r] - M);
  const float f = exp2_fast(m - M);
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[dt][e] *= f;
#pragma unroll
  for (int step = NW / 2; step; step >>= 1) {
    __syncthreads();
    if (r < live && w >= step && w < 2 * step) {
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4*>(&lo_[w - step][r * LD + 32 * dt + 8 * i + 4 * half]) =
              f32x4{acc[dt][4 * i], acc[dt][4 * i + 1], acc[dt][4 * i + 2], acc[dt][4 * i + 3]};
    }
    __syncthreads();
    if (r < live && w < step) {
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 o = *reinterpret_cast<const f32x4*>(&lo_[w][r * LD + 32 * dt + 8 * i + 4 * half]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[dt][4 * i + j] += o[j];
        }
    }
  }
  if (w != 0 || r >= live) return;
  if (whole) {
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    uint16_t* o = a.out + attn_row(a, s.row0, kvh, col) * D + 4 * half;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 p = {pack_bf16x2(acc[dt][4 * i] * inv, acc[dt][4 * i + 1] * inv),
                         pack_bf16x2(acc[dt][4 * i + 2] * inv, acc[dt][4 * i + 3] * inv)};
        *reinterpret_cast<uint2*>(o + 32 * dt + 8 * i) = p;
      }
  } else {
    const int64_t item = ((static_cast<int64_t>(b) * a.kv_heads + kvh) * cols + col) * a.splits + split;
    const int64_t items = static_cast<int64_t>(a.B) * a.kv_heads * cols * a.splits;
    if (half == 0) *reinterpret_cast<float2*>(a.ws + items * D + item * 2) = float2{M, L};
    float* o = a.ws + item * D + 4 * half;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(o + 32 * dt + 8 * i) =
            f32x4{acc[dt][4 * i], acc[dt][4 * i + 1], acc[dt][4 * i + 2], acc[dt][4 * i + 3]};
  }
}

// Joins the parts of an output row: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// Lane i of every wavefront has part i's maximum and sum (64 parts at a time),
// so that M and the factors are known after one load; then the RW wavefronts of
// a row add up every RW'th part, D / 64 dims a lane, with several loads in
// flight.  Few rows have 4 wavefronts each, which join in LDS (one token over
// 131071 keys, 32 rows of 64 parts: 86.9 us in all, and 89.5 us with one); 1024
// rows or more have one each, in a quarter of the blocks (2048 rows of at most 7
// parts of 64 dims: 19.6 us in all, and 21.1 us with 4).
template <int D, int RW>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int ND = D / 64, UNROLL = 4;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int cols = a.n_q * a.group;
  const int row = blockIdx.x * (4 / RW) + w / RW;
  const int col = row % cols, kvh = (row / cols) % a.kv_heads, b = row / cols / a.kv_heads;
  if (RW == 1 && b >= a.B) return;
  const int64_t item = ((static_cast<int64_t>(b) * a.kv_heads + kvh) * cols + col) * a.splits;
  const int64_t items = static_cast<int64_t>(a.B) * a.kv_heads * cols * a.splits;
  const float2* ml = reinterpret_cast<const float2*>(a.ws + items * D) + item;
  const float* const sums = a.ws + item * D + lane * ND;
  // asked for before the sequence's length is known: whether it has that part or not
  const float2 first_ml = ml[min(lane, a.splits - 1)];
  const AttnSeq s = attn_seq(a, b);
  const AttnTiles tl = attn_tiles<32>(a, s.first, s.len - 1);
  if (tl.n <= a.tiles_per_split) return;
  const int parts = (tl.n + a.tiles_per_split - 1) / a.tiles_per_split;
  float M = ATTN_NO_MAX, L = 0.0f, o[ND] = {};
  for (int p0 = 0; p0 < parts; p0 += 64) {
    const int here = min(parts - p0, 64);
    const float2 p = p0 ? ml[p0 + min(lane, here - 1)] : first_ml;
    const float m = lane < here ? p.x : ATTN_NO_MAX;
    float mn = fmaxf(M, m);
#pragma unroll
    for (int x = 32; x; x >>= 1) mn = fmaxf(mn, __shfl_xor(mn, x));
    const float f = lane < here ? exp2_fast(m - mn) : 0.0f, old = exp2_fast(M - mn);
    M = mn;
    L = L * old + wave_sum(lane < here ? p.y * f : 0.0f);
#pragma unroll
    for (int n = 0; n < ND; ++n) o[n] *= old;
    for (int i0 = w % RW; i0 < here; i0 += RW * UNROLL) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int i = min(i0 + RW * u, here - 1);
        const float g = i0 + RW * u < here ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), i)) : 0.0f;
        const float* src = sums + static_cast<int64_t>(p0 + i) * D;
#pragma unroll
        for (int n = 0; n < ND; ++n) o[n] += src[n] * g;
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
