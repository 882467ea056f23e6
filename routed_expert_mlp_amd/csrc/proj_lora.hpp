// Low-rank adapters of many requests beside a shared projection.
//
//   v[t] = x[t] A_a^T;  out[t] = base[t] + s_a v[t] B_a^T,   a = adapter[t]
//
// The tokens of an adapter are gathered into the rows of a matrix product, 64 at a
// time (a tile), in whatever order they come, so that an adapter is read once for
// them.  Up to 64 tokens each block finds its adapter's tokens itself: every
// wavefront reads the adapter numbers, one a lane, and lanes of one adapter find each
// other with a ballot for each bit of its number.  With more, k_lora_group sorts the tokens by adapter first (4096
// tokens of 50 adapters in any order: 466 us in windows of 64 tokens, each of which
// reads most adapters again).
//
// v is a sum over thousands of columns, cut into parts for the blocks; k_lora_up
// adds up the parts (fp32, in order), and gives v to the matrix unit as the sum of
// two bf16 values, beside the bf16 weights: 16 bits of it, at the price of half a
// matrix instruction more, where the time is that of the memory.
#pragma once

#include "common.hpp"

#include <type_traits>

namespace moe {

struct LoraArgs {
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* ranks;
  const float* scales;
  const uint16_t* x;
  const int32_t* adapter;
  const uint16_t* base;
  uint16_t* out;
  float* v;                  // [parts][T][vr]
  int32_t* order;            // grouped: tokens by adapter, those without one last
  int4* tiles;               // grouped: adapter (-1: none), first place in order, tokens, rank
  int32_t* n_tiles;
  int64_t x_stride, base_stride, out_stride, T, n_adapters;
  int32_t R, K, N;           // R: max_rank
  int32_t vr;                // columns of v: R up to a multiple of 16
  int32_t parts, part_chunks;     // of K: parts, and chunks of 64 columns of one
  int32_t slots;             // not grouped: blocks that share a window's tiles
  int32_t bits;              // of n_adapters
};

constexpr int LORA_RT = 4;        // 16-rank tiles of a block of k_lora_down
constexpr int LORA_DOWN = 8;      // wavefronts of a block of k_lora_down
constexpr int LORA_UP = 4;        // wavefronts of a block of k_lora_up
constexpr int LORA_BINS = 512;    // k_lora_group: adapters, and the tokens without one
constexpr int LORA_GROUP = 16;    // wavefronts of k_lora_group

// Place (0..63) of set bit number n of a word that has more than n.
__device__ __forceinline__ int nth_bit(uint64_t word, int n) {
  int at = 0;
#pragma unroll
  for (int step = 32; step; step >>= 1) {
    const int here = __popcll((word >> at) & ((uint64_t(1) << step) - 1));
    if (n >= here) {
      n -= here;
      at += step;
    }
  }
  return at;
}

// Tokens of one adapter; all lanes the same.
struct LoraGroupedTile {
  int adapter, first, rows, rank;
  __device__ __forceinline__ int64_t token(const LoraArgs& a, int n) const { return a.order[first + min(n, rows - 1)]; }
};

struct LoraWindowTile {
  int adapter, first, rows, rank;
  uint64_t mine;             // places of the adapter's tokens in the window, of which the tile has some from `first` on
  int64_t t0;
  __device__ __forceinline__ int64_t token(const LoraArgs&, int n) const {
    return t0 + nth_bit(mine, first + min(n, rows - 1));
  }
};

__device__ __forceinline__ int lora_rank(const LoraArgs& a, int id) {
  return a.ranks ? min(max(a.ranks[id], 0), a.R) : a.R;
}

// Calls f(tile) for the tiles of this block: grouped, tile blockIdx.x, of up to 64 tokens; otherwise, of window
// blockIdx.x / slots, every slots'th tile of up to 16 tokens from blockIdx.x % slots on, and the tokens without an
// adapter (-1) with the first.  (Tiles of 64 tokens there need twice the registers, for calls that mostly have one
// or two tokens of an adapter: 64 tokens of 32 adapters 24 us.)
template <bool GROUPED, typename F>
__device__ __forceinline__ void lora_tiles(const LoraArgs& a, F&& f) {
  if constexpr (GROUPED) {
    const int4 t = a.tiles[blockIdx.x];          // as far as blocks go there is room in the table
    if (static_cast<int>(blockIdx.x) >= *a.n_tiles) return;
    f(LoraGroupedTile{__builtin_amdgcn_readfirstlane(t.x), __builtin_amdgcn_readfirstlane(t.y),
                      __builtin_amdgcn_readfirstlane(t.z), __builtin_amdgcn_readfirstlane(t.w)});
  } else {
    const int slot = blockIdx.x % a.slots;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / a.slots) * 64, t = t0 + (threadIdx.x & 63);
    int id = t < a.T ? a.adapter[t] : -2;
    if (t < a.T && (id < 0 || id >= a.n_adapters)) id = -1;
    const int rank_of = lora_rank(a, max(id, 0));        // ahead of the search
    const uint64_t none = __ballot(id == -1);
    if (slot == 0 && none) f(LoraWindowTile{-1, 0, static_cast<int>(__popcll(none)), 0, none, t0});
    // lanes of this lane's adapter, and this lane's number among them; every sixteenth begins a tile
    uint64_t alike = __ballot(id >= 0);
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t ones = __ballot(id >> b & 1);
      alike &= id >> b & 1 ? ones : ~ones;
    }
    const int number = static_cast<int>(__popcll(alike & ((uint64_t(1) << (threadIdx.x & 63)) - 1)));
    const uint64_t leads = __ballot(id >= 0 && (number & 15) == 0);
    for (int i = slot, n = static_cast<int>(__popcll(leads)); i < n; i += a.slots) {
      const int lead = __builtin_amdgcn_readfirstlane(nth_bit(leads, i));
      const uint64_t mine = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(alike), lead)) |
                            static_cast<uint64_t>(static_cast<uint32_t>(
                                __builtin_amdgcn_readlane(static_cast<int>(alike >> 32), lead))) << 32;
      const int first = __builtin_amdgcn_readlane(number, lead);
      f(LoraWindowTile{__builtin_amdgcn_readlane(id, lead), first, min(static_cast<int>(__popcll(mine)) - first, 16),
                       __builtin_amdgcn_readlane(rank_of, lead), mine, t0});
    }
  }
}

// Tokens in the order of their adapters (stable), and the table of tiles; one block.  Each wavefront has a run of the
// tokens: it counts them by adapter, the counts are added up over wavefronts and adapters, and it puts its tokens in
// their places.  Lanes of one adapter find each other as above; the first of them
// counts for all, so that nothing is added up by two lanes at once.
__global__ __launch_bounds__(64 * LORA_GROUP) void k_lora_group(LoraArgs a) {
  __shared__ int count[LORA_GROUP][LORA_BINS];
  __shared__ int place[2][LORA_BINS], tile[2][LORA_BINS];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int bins = static_cast<int>(a.n_adapters) + 1;
  const int run = static_cast<int>((a.T + 64 * LORA_GROUP - 1) / (64 * LORA_GROUP)) * 64;
  const int64_t t0 = static_cast<int64_t>(run) * w, t1 = t0 + run < a.T ? t0 + run : a.T;
  for (int i = tid; i < LORA_GROUP * LORA_BINS; i += 64 * LORA_GROUP) count[i / LORA_BINS][i % LORA_BINS] = 0;
  __syncthreads();
  auto bin_of = [&](int64_t t) __attribute__((always_inline)) {
    const int id = t < t1 ? a.adapter[t] : -1;
    return id >= 0 && id < bins - 1 ? id : bins - 1;
  };
  auto alike = [&](int bin, bool in) __attribute__((always_inline)) {
    uint64_t m = __ballot(in);
    for (int b = 0; b < a.bits; ++b) {
      const bool one = bin >> b & 1;
      const uint64_t ones = __ballot(one);
      m &= one ? ones : ~ones;
    }
    return m;
  };
  volatile int* const mine = count[w];
  constexpr int AHEAD = 8;                       // loads in flight
  for (int64_t t8 = t0; t8 < t1; t8 += 64 * AHEAD) {
    int next[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) next[i] = bin_of(t8 + 64 * i + lane);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const bool in = t8 + 64 * i + lane < t1;
      const uint64_t m = alike(next[i], in);
      if (in && __builtin_ctzll(m) == lane) mine[next[i]] = mine[next[i]] + __popcll(m);
    }
  }
  __syncthreads();
  // of each bin: where the wavefronts' tokens go within it, its tokens and tiles in all
  int total = 0;
  if (tid < LORA_BINS) {
    for (int i = 0; i < LORA_GROUP; ++i) {
      const int n = count[i][tid];
      count[i][tid] = total;
      total += n;
    }
    place[0][tid] = total;
    tile[0][tid] = (total + 63) >> 6;
  }
  __syncthreads();
  int from = 0;
  for (int step = 1; step < bins; step <<= 1, from ^= 1) {
    if (tid < LORA_BINS) {
      place[from ^ 1][tid] = place[from][tid] + (tid >= step ? place[from][tid - step] : 0);
      tile[from ^ 1][tid] = tile[from][tid] + (tid >= step ? tile[from][tid - step] : 0);
    }
    __syncthreads();
  }
  if (tid < bins) {
    const int first = place[from][tid] - total, tiles = (total + 63) >> 6;
    const int rank = tid < bins - 1 ? lora_rank(a, tid) : 0;
    for (int i = 0; i < tiles; ++i)
      a.tiles[tile[from][tid] - tiles + i] =
          int4{tid == bins - 1 ? -1 : tid, first + 64 * i, min(total - 64 * i, 64), rank};
    for (int i = 0; i < LORA_GROUP; ++i) count[i][tid] += first;
    if (tid == bins - 1) *a.n_tiles = tile[from][tid];
  }
  __syncthreads();
  for (int64_t t8 = t0; t8 < t1; t8 += 64 * AHEAD) {
    int next[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) next[i] = bin_of(t8 + 64 * i + lane);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const bool in = t8 + 64 * i + lane < t1;
      const uint64_t m = alike(next[i], in);
      if (in) {
        const int at = mine[next[i]];
        a.order[at + __popcll(m & ((uint64_t(1) << lane) - 1))] = static_cast<int32_t>(t8 + 64 * i + lane);
        if (__builtin_ctzll(m) == lane) mine[next[i]] = at + __popcll(m);
      }
    }
  }
}

// Sums of a wavefront over its chunks: MT tiles of 16 gathered tokens, RT tiles of 16 ranks.  Lanes of rows or ranks
// past the last one have the last one's again; nobody reads what comes of it.
template <int MT, int RT, typename Tile>
__device__ __forceinline__ void lora_rows(const LoraArgs& a, const Tile& tile, int rank, int r0, int c0, int c1,
                                          f32x4 (*acc)[LORA_RT]) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int pieces = a.K >> 3;                   // of 8 columns
  const uint4* xp[MT];
  const uint4* ap[RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xp[m] = reinterpret_cast<const uint4*>(a.x + tile.token(a, 16 * m + c) * a.x_stride) + g;
#pragma unroll
  for (int n = 0; n < RT; ++n)
    ap[n] = reinterpret_cast<const uint4*>(
                a.a + (static_cast<int64_t>(tile.adapter) * a.R + min(r0 + 16 * n + c, rank - 1)) * a.K) + g;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < RT; ++n) acc[m][n] = f32x4{};
  // a chunk is 64 columns: pieces g and 4 + g of 8
  auto chunk = [&](int k, auto whole) __attribute__((always_inline)) {
    bf16x8 xf[2][MT], af[2][RT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int p = 8 * k + 4 * h;
      const bool in = decltype(whole)::value || p + g < pieces;
      if (!in) p = -g;
#pragma unroll
      for (int n = 0; n < RT; ++n) {
        uint4 v = ap[n][p];
        if (!in) v = uint4{};
        af[h][n] = __builtin_bit_cast(bf16x8, v);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint4 v = xp[m][p];
        if (!in) v = uint4{};
        xf[h][m] = __builtin_bit_cast(bf16x8, v);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < RT; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[h][n], xf[h][m], acc[m][n], 0, 0, 0);
  };
  const int full = min(c1, pieces >> 3);
  int k = c0 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (; k < full; k += LORA_DOWN) chunk(k, std::true_type{});
  for (; k < c1; k += LORA_DOWN) chunk(k, std::false_type{});
}

// v of a tile's tokens: .y = part of K, .z = group of 64 ranks.  The wavefronts take the part's chunks of 64 columns
// in turn and join in LDS, pair by pair.
template <bool GROUPED>
__global__ __launch_bounds__(64 * LORA_DOWN, 2) void k_lora_down(LoraArgs a) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = blockIdx.y, r0 = blockIdx.z * (16 * LORA_RT);
  const int c0 = part * a.part_chunks, c1 = min(c0 + a.part_chunks, (a.K + 63) >> 6);
  constexpr int MT = GROUPED ? 4 : 1;
  __shared__ f32x4 join[LORA_DOWN / 2][MT][LORA_RT][64];
  lora_tiles<GROUPED>(a, [&](const auto& tile) __attribute__((always_inline)) {
    if (tile.adapter < 0) return;
    const int rank = tile.rank;
    const int tiles = min((rank - r0 + 15) >> 4, LORA_RT), mt = (tile.rows + 15) >> 4;
    if (tiles <= 0) return;
    f32x4 acc[MT][LORA_RT];
    if (!GROUPED || mt == 1) {
      if (tiles == 1) lora_rows<1, 1>(a, tile, rank, r0, c0, c1, acc);
      else if (tiles == 2) lora_rows<1, 2>(a, tile, rank, r0, c0, c1, acc);
      else lora_rows<1, 4>(a, tile, rank, r0, c0, c1, acc);
    } else if constexpr (GROUPED) {
      if (tiles == 1) lora_rows<4, 1>(a, tile, rank, r0, c0, c1, acc);
      else if (tiles == 2) lora_rows<4, 2>(a, tile, rank, r0, c0, c1, acc);
      else lora_rows<4, 4>(a, tile, rank, r0, c0, c1, acc);
    }
#pragma unroll
    for (int step = LORA_DOWN / 2; step; step >>= 1) {
      __syncthreads();
      if (w >= step && w < 2 * step) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < LORA_RT; ++n)
            if (m < mt && n < tiles) join[w - step][m][n][lane] = acc[m][n];
      }
      __syncthreads();
      if (w < step) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < LORA_RT; ++n)
            if (m < mt && n < tiles) acc[m][n] += join[w][m][n][lane];
      }
    }
    // lane: token c of a tile of 16, ranks 4 g .. +3
    if (w == 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (16 * m + c >= tile.rows) continue;
        float* v = a.v + (static_cast<int64_t>(part) * a.T + tile.token(a, 16 * m + c)) * a.vr + r0 + 4 * g;
#pragma unroll
        for (int n = 0; n < LORA_RT; ++n)
          if (n < tiles) *reinterpret_cast<f32x4*>(v + 16 * n) = acc[m][n];
      }
    }
  });
}

// The columns n0 .. n0 + 63 of a tile's tokens, MT tiles of 16 of them, by one wavefront of a block that has called
// it with its others.  v goes to LDS in two bf16 values, upper halves and what is left of them; the weights come
// straight from memory, and are on their way with the base rows before v is there.  16 ranks an instruction: lanes
// of g = 0, 1 have the upper halves, g = 2, 3 the rest, of the same weights.  Lane: token c of a tile of 16, columns
// 16 g .. +15 (row 4 g + i of matrix tile j is column 16 g + 4 j + i).
template <int MT, typename Tile>
__device__ __forceinline__ void lora_columns(const LoraArgs& a, const Tile& tile, int n0, uint4* vl) {
  constexpr int RG = 2;            // steps of 16 ranks whose weights are read at once
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int rank = tile.rank, rows = tile.rows;
  const float scale = a.scales ? a.scales[tile.adapter] : 1.0f;
  const int pitch = a.vr / 8 + 1;                // of half a row, in pieces of 8; odd: rows fall to different banks
  const uint16_t* const bt = a.b + (static_cast<int64_t>(tile.adapter) * a.N) * a.R;
  const uint16_t* bp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    bp[j] = bt + static_cast<int64_t>(min(n0 + 16 * (c >> 2) + 4 * j + (c & 3), a.N - 1)) * a.R;
  uint4 bq[RG][4];
  auto read_b = [&](int r0) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < RG; ++s) {
      if (r0 + 16 * s >= rank) continue;
      const int rr = r0 + 16 * s + 8 * (g & 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) bq[s][j] = *reinterpret_cast<const uint4*>(bp[j] + (rr < rank ? rr : 0));
    }
  };
  read_b(0);
  int t[MT];
  uint4 old[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    t[m] = static_cast<int>(tile.token(a, 16 * m + c));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      old[m][h] = *reinterpret_cast<const uint4*>(a.base + t[m] * a.base_stride + min(n0 + 16 * g + 8 * h, a.N - 8));
  }
  // v: 2^sh pieces of a row, of which (rank + 7) / 8 are there
  const int per = (rank + 7) >> 3, sh = per > 1 ? 32 - __builtin_clz(per - 1) : 0;
  __syncthreads();                               // the previous tile's rows have been read
  for (int e = threadIdx.x; e < rows << sh; e += 64 * LORA_UP) {
    const int row = e >> sh, piece = e & ((1 << sh) - 1);
    if (piece >= per) continue;
    const float* v = a.v + tile.token(a, row) * a.vr + 8 * piece;
    f32x4 s0 = {}, s1 = {};
#pragma unroll 4
    for (int p = 0; p < a.parts; ++p, v += a.T * a.vr) {
      s0 += *reinterpret_cast<const f32x4*>(v);
      s1 += *reinterpret_cast<const f32x4*>(v + 4);
    }
    bf16x8 hi, lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = 8 * piece + j < rank ? (j < 4 ? s0[j & 3] : s1[j & 3]) : 0.0f;
      hi[j] = static_cast<__bf16>(f);
      lo[j] = static_cast<__bf16>(f - static_cast<float>(hi[j]));
    }
    vl[(2 * row) * pitch + piece] = __builtin_bit_cast(uint4, hi);
    vl[(2 * row + 1) * pitch + piece] = __builtin_bit_cast(uint4, lo);
  }
  __syncthreads();
  if (n0 >= a.N) return;
  f32x4 acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = f32x4{};
  for (int r0 = 0; r0 < rank; r0 += 16 * RG) {
    if (r0) read_b(r0);
#pragma unroll
    for (int s = 0; s < RG; ++s) {
      if (r0 + 16 * s >= rank) continue;
      const int rr = r0 + 16 * s + 8 * (g & 1);
      const int left = rank - rr;                // what the weights hold past the rank does not matter
      if (r0 + 16 * s + 16 > rank) {
        auto keep = [&](int e) { return (left > e ? 0xFFFFu : 0u) | (left > e + 1 ? 0xFFFF0000u : 0u); };
        const uint32_t k0 = keep(0), k1 = keep(2), k2 = keep(4), k3 = keep(6);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bq[s][j].x &= k0;
          bq[s][j].y &= k1;
          bq[s][j].z &= k2;
          bq[s][j].w &= k3;
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint4 v = vl[(2 * min(16 * m + c, rows - 1) + (g >> 1)) * pitch + (rr < rank ? rr >> 3 : 0)];
        if (rr >= rank) v = uint4{};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, bq[s][j]),
                                                              __builtin_bit_cast(bf16x8, v), acc[m][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (16 * m + c >= rows) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + 16 * g + 8 * h;
      if (n >= a.N) continue;
      const uint32_t u[4] = {old[m][h].x, old[m][h].y, old[m][h].z, old[m][h].w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x4& s = acc[m][2 * h + (e >> 1)];
        o[e] = pack_bf16x2(fmaf(scale, s[2 * (e & 1)], __uint_as_float(u[e] << 16)),
                           fmaf(scale, s[2 * (e & 1) + 1], __uint_as_float(u[e] & 0xFFFF0000u)));
      }
      *reinterpret_cast<uint4*>(a.out + t[m] * a.out_stride + n) = uint4{o[0], o[1], o[2], o[3]};
    }
  }
}

// Rows of the output: .y = 256 columns, 64 a wavefront.
template <bool GROUPED>
__global__ __launch_bounds__(64 * LORA_UP, GROUPED ? 3 : 4) void k_lora_up(LoraArgs a) {
  extern __shared__ uint4 vl[];                  // [tokens of a tile: 64 grouped, else 16][2 halves][pitch] pieces of 8 values
  const int n0 = blockIdx.y * (64 * LORA_UP) + 64 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  lora_tiles<GROUPED>(a, [&](const auto& tile) __attribute__((always_inline)) {
    if (tile.adapter < 0) {                      // base as it is, 8 tokens at a time
      const int lane = threadIdx.x & 63, n = n0 + 8 * (lane & 7);
      if (a.out == a.base || n >= a.N) return;
      for (int i = lane >> 3; i < tile.rows; i += 8) {
        const int64_t t = tile.token(a, i);
        *reinterpret_cast<uint4*>(a.out + t * a.out_stride + n) =
            *reinterpret_cast<const uint4*>(a.base + t * a.base_stride + n);
      }
    } else if (!GROUPED || tile.rows <= 16) {
      lora_columns<1>(a, tile, n0, vl);
    } else if constexpr (GROUPED) {
      lora_columns<4>(a, tile, n0, vl);
    }
  });
}

}  // namespace moe
