// Low-rank adapters of many requests beside a shared projection.
//
//   v[t] = x[t] A_a^T;  out[t] = base[t] + s_a v[t] B_a^T,   a = adapter[t]
//
// The tokens of an adapter are gathered into the rows of a matrix product, 64 at a
// time (a tile), in whatever order they come, so that an adapter is read once for
// them.  In windows of 64 tokens each block finds its adapter's tokens itself: every
// wavefront reads the adapter numbers, one a lane, and lanes of one adapter find each
// other with a ballot for each bit of its number.  Where windows would read the
// adapters too often, k_lora_group sorts the tokens by adapter first (4096 columns to
// 4096, 4096 tokens of 50 adapters of rank 32 in any order: 252 us in windows of 64
// tokens, each of which reads most adapters again, and 49 us sorted).
//
// v is a sum over thousands of columns, cut into parts for the blocks; k_lora_up
// adds up the parts (fp32, in order), and gives v to the matrix unit as the sum of
// two bf16 values, beside the bf16 weights: 16 bits of it, at the price of half a
// matrix instruction more, where the time is that of the memory.
//
// What bounds it: with few tokens two launches, each with a chain of reads behind it
// (adapter numbers, weights, parts); with many the rows, x once and base in and out
// once, at two thirds of a copy's rate, and the sort.  4096 columns: one token of
// rank 16 to 6144 10 us (5.0 and 5.6 in the kernels), 64 tokens of 32 adapters of
// rank 64 to 6144 17 us (7.5 and 9.3), 4096 tokens of 5 adapters of rank 32
// to 4096 38 us (sort 7.0, 12.2 for 34 MB and 19.5 for 67 MB).
#pragma once

#include "common.hpp"

#include <type_traits>

namespace moe {

typedef int lora_piece __attribute__((ext_vector_type(4)));       // 16 bytes: 8 values

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
  constexpr int AHEAD = 8;                       // loads in flight
  int bin[AHEAD];
  uint64_t same[AHEAD];                          // lanes of this lane's bin
  auto read = [&](int64_t t8) __attribute__((always_inline)) {
    int id[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int64_t t = t8 + 64 * i + lane;
      id[i] = t < t1 ? a.adapter[t] : -1;
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      bin[i] = id[i] >= 0 && id[i] < bins - 1 ? id[i] : bins - 1;
      same[i] = 0;
      if (t8 + 64 * i >= t1) continue;
      same[i] = __ballot(t8 + 64 * i + lane < t1);
      for (int b = 0; b < a.bits; ++b) {
        const bool one = bin[i] >> b & 1;
        const uint64_t ones = __ballot(one);
        same[i] &= one ? ones : ~ones;
      }
    }
  };
  read(t0);
  const int rank = tid < bins - 1 ? lora_rank(a, tid) : 0;
  volatile int* const mine = count[w];
  for (int i = lane; i < bins; i += 64) mine[i] = 0;
  for (int64_t t8 = t0; t8 < t1; t8 += 64 * AHEAD) {
    if (t8 > t0) read(t8);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (t8 + 64 * i >= t1) continue;
      if (t8 + 64 * i + lane < t1 && __builtin_ctzll(same[i]) == lane) mine[bin[i]] = mine[bin[i]] + __popcll(same[i]);
    }
  }
  __syncthreads();
  // of each bin: where the wavefronts' tokens go within it, its tokens and tiles in all
  int total = 0;
  if (tid < bins) {
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
    if (tid < bins) {
      place[from ^ 1][tid] = place[from][tid] + (tid >= step ? place[from][tid - step] : 0);
      tile[from ^ 1][tid] = tile[from][tid] + (tid >= step ? tile[from][tid - step] : 0);
    }
    __syncthreads();
  }
  if (tid < bins) {
    const int first = place[from][tid] - total, tiles = (total + 63) >> 6;
    for (int i = 0; i < LORA_GROUP; ++i) count[i][tid] += first;
    for (int i = 0; i < tiles; ++i)
      a.tiles[tile[from][tid] - tiles + i] =
          int4{tid == bins - 1 ? -1 : tid, first + 64 * i, min(total - 64 * i, 64), rank};
    if (tid == bins - 1) *a.n_tiles = tile[from][tid];
  }
  __syncthreads();
  for (int64_t t8 = t0; t8 < t1; t8 += 64 * AHEAD) {
    if (run > 64 * AHEAD) read(t8);              // otherwise they are here still
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (t8 + 64 * i + lane >= t1) continue;
      const int at = mine[bin[i]];
      a.order[at + __popcll(same[i] & ((uint64_t(1) << lane) - 1))] = static_cast<int32_t>(t8 + 64 * i + lane);
      if (__builtin_ctzll(same[i]) == lane) mine[bin[i]] = at + __popcll(same[i]);
    }
  }
}

// Writes of a wavefront to LDS, and its reads behind them: done in order, if the compiler keeps it.
__device__ __forceinline__ void lora_in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Sums of a wavefront over its chunks of 64 columns: MT tiles of 16 gathered tokens, RT tiles of 16 ranks.  Eight lanes
// read the 128 bytes of a row, which become operands (16 rows in neighbouring lanes) in LDS of the wavefront's own;
// piece p of row r is at p ^ (r & 7), so that the rows of an operand fall to different banks.  Lanes of rows or ranks
// past the last one have the last one's again; nobody reads what comes of it.  (LINES false: loads straight into
// operands, with 16 rows an instruction: 64 tokens of 64 adapters of rank 16 6.2 and 8.7 us, where LDS is one more wait;
// 32 adapters of rank 64 9.3 and 7.6 us, 4096 tokens 13.9 and 12.1 us.)
template <int MT, int RT, bool LINES, typename Tile>
__device__ __forceinline__ void lora_rows(const LoraArgs& a, const Tile& tile, int rank, int r0, int c0, int c1,
                                          f32x4 (*acc)[LORA_RT], uint4* mine) {
  constexpr int X = 2 * MT, L = 2 * (MT + RT);
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15, lr = lane >> 3, lp = lane & 7;
  const int pieces = a.K >> 3;                   // of 8 columns
  // row and piece of load i
  auto row_of = [&](int i) __attribute__((always_inline)) { return LINES ? 8 * i + lr : 16 * (i >> 1) + c; };
  auto piece_of = [&](int i) __attribute__((always_inline)) { return LINES ? lp : 4 * (i & 1) + g; };
  const uint16_t* row[X];
#pragma unroll
  for (int i = 0; i < X; ++i) row[i] = a.x + tile.token(a, row_of(i)) * a.x_stride;
  const uint16_t* const at = a.a + static_cast<int64_t>(tile.adapter) * a.R * a.K;
  uint32_t off[L - X];                           // of rows of the adapter: at most 256 of less than 2^20 columns
#pragma unroll
  for (int i = 0; i < L - X; ++i) off[i] = static_cast<uint32_t>(min(r0 + row_of(i), rank - 1)) * a.K;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < RT; ++n) acc[m][n] = f32x4{};
  lora_piece raw[L];
  auto read = [&](int k) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int p = 8 * k + piece_of(i);
      const bool in = p < pieces;
      const uint32_t k8 = 8 * (in ? p : 0);
      raw[i] = *reinterpret_cast<const lora_piece*>(i < X ? row[i] + k8 : at + (off[i - X] + k8));
      if (!in) raw[i] = lora_piece{};
    }
  };
  const int put = 8 * lr + (lp ^ lr);
  int k = c0 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (k < c1) read(k);
  for (; k < c1; k += LORA_DOWN) {
    if constexpr (!LINES) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < RT; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, raw[X + 2 * n + h]),
                                                                __builtin_bit_cast(bf16x8, raw[2 * m + h]), acc[m][n],
                                                                0, 0, 0);
      if (k + LORA_DOWN < c1) read(k + LORA_DOWN);
      continue;
    }
#pragma unroll
    for (int i = 0; i < L; ++i) *reinterpret_cast<lora_piece*>(mine + 64 * i + put) = raw[i];
    lora_in_order();
    if (k + LORA_DOWN < c1) read(k + LORA_DOWN);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4* const from = mine + 8 * c + ((4 * h + g) ^ (c & 7));
      bf16x8 af[RT];
#pragma unroll
      for (int n = 0; n < RT; ++n) af[n] = *reinterpret_cast<const bf16x8*>(from + 64 * X + 128 * n);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bf16x8 xf = *reinterpret_cast<const bf16x8*>(from + 128 * m);
#pragma unroll
        for (int n = 0; n < RT; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[n], xf, acc[m][n], 0, 0, 0);
      }
    }
    lora_in_order();
  }
}

// v of a tile's tokens: .y = part of K, .z = group of 64 ranks.  The wavefronts take the part's chunks of 64 columns
// in turn and join in LDS, pair by pair.
template <bool GROUPED>
__global__ __launch_bounds__(64 * LORA_DOWN, GROUPED ? 2 : 4) void k_lora_down(LoraArgs a) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = blockIdx.y, r0 = blockIdx.z * (16 * LORA_RT);
  const int c0 = part * a.part_chunks, c1 = min(c0 + a.part_chunks, (a.K + 63) >> 6);
  constexpr int MT = GROUPED ? 4 : 1;
  __shared__ uint4 lines[LORA_DOWN][(MT + LORA_RT) * 128];
  uint4* const mine = lines[w];
  // the sums of half of the wavefronts, where the lines were
  static_assert(sizeof(lines) >= sizeof(f32x4) * (LORA_DOWN / 2) * MT * LORA_RT * 64, "room for the sums");
  f32x4 (*const join)[MT][LORA_RT][64] = reinterpret_cast<f32x4 (*)[MT][LORA_RT][64]>(&lines[0][0]);
  lora_tiles<GROUPED>(a, [&](const auto& tile) __attribute__((always_inline)) {
    if (tile.adapter < 0) return;
    const int rank = tile.rank;
    const int tiles = min((rank - r0 + 15) >> 4, LORA_RT), mt = (tile.rows + 15) >> 4;
    if (tiles <= 0) return;
    __syncthreads();                             // the sums of the block's last tile have been read
    f32x4 acc[MT][LORA_RT];
    if (!GROUPED || mt == 1) {
      if (tiles == 1) lora_rows<1, 1, GROUPED>(a, tile, rank, r0, c0, c1, acc, mine);
      else if (tiles == 2) lora_rows<1, 2, true>(a, tile, rank, r0, c0, c1, acc, mine);
      else lora_rows<1, 4, true>(a, tile, rank, r0, c0, c1, acc, mine);
    } else if constexpr (GROUPED) {
      if (tiles == 1) lora_rows<4, 1, true>(a, tile, rank, r0, c0, c1, acc, mine);
      else if (tiles == 2) lora_rows<4, 2, true>(a, tile, rank, r0, c0, c1, acc, mine);
      else lora_rows<4, 4, true>(a, tile, rank, r0, c0, c1, acc, mine);
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

// The sums v B of 8 columns of a token again, from v as it is: an infinity in v or in B has none in two halves (the rest
// of one is inf - inf, and a rest of 0 times one in B is NaN), nor has a v that bf16 rounds up to one.
__device__ __forceinline__ void lora_whole(const LoraArgs& a, int adapter, int rank, int64_t token, int n, f32x4& s0,
                                           f32x4& s1) {
  const uint16_t* const b = a.b + (static_cast<int64_t>(adapter) * a.N + n) * a.R;
  s0 = s1 = f32x4{};
#pragma unroll 1
  for (int r = 0; r < rank; ++r) {
    const float* at = a.v + token * a.vr + r;
    float v = 0.0f;
    for (int p = 0; p < a.parts; ++p, at += a.T * a.vr) v += *at;
    bool number = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f32x4& s = e < 4 ? s0 : s1;
      s[e & 3] = fmaf(v, __uint_as_float(static_cast<uint32_t>(b[static_cast<int64_t>(e) * a.R + r]) << 16), s[e & 3]);
      number |= s[e & 3] == s[e & 3];
    }
    if (!number) return;
  }
}

// The columns n0 .. n0 + 63 of a tile's tokens from m0 on, MT tiles of 16 of them, by one wavefront of a block that
// has called it with all of its NW.  v goes to LDS in two bf16 values, upper halves and what is left of them.  The weights of 32
// ranks at a time, and at the end the sums of 16 tokens, go through LDS of the wavefront's own (`mine`, 4 KB): memory
// is read and written in runs of 64 and 128 bytes, the matrix unit wants 16 rows in neighbouring lanes (with its
// order in memory too 4096 tokens took 24 us).  16 ranks an instruction: lanes of g = 0, 1 have the upper halves,
// g = 2, 3 the rest, of the same weights.  The many rows of a sorted call go around the caches, which the tokens' v
// and x then stay in (8000 tokens of 2048 columns to 2048, rank 64: both products 46.3 and 42.4 us).
template <int MT, int NW, typename Tile>
__device__ __forceinline__ void lora_columns(const LoraArgs& a, const Tile& tile, int n0, int m0, uint4* vl,
                                             uint4* mine) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15, lr = lane >> 3, lp = lane & 7;
  const int rank = tile.rank, rows = tile.rows;
  const float scale = a.scales ? a.scales[tile.adapter] : 1.0f;
  const int pitch = a.vr / 8 + 1;                // of half a row, in pieces of 8; odd: rows fall to different banks
  // weights: lane / 4 of 16 rows, piece lane % 4 of 8 ranks; what they hold past the rank does not matter
  const uint16_t* const bt = a.b + static_cast<int64_t>(tile.adapter) * a.N * a.R;
  lora_piece raw[4];
  auto read_b = [&](int r0) __attribute__((always_inline)) {
    const int rr = r0 + 8 * (lane & 3), left = rank - rr;
    auto keep = [&](int e) { return static_cast<int>((left > e ? 0xFFFFu : 0u) | (left > e + 1 ? 0xFFFF0000u : 0u)); };
    const lora_piece kept{keep(0), keep(2), keep(4), keep(6)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = min(n0 + 16 * j + (lane >> 2), a.N - 1);
      raw[j] = *reinterpret_cast<const lora_piece*>(bt + n * a.R + (left > 0 ? rr : 0)) & kept;
    }
  };
  if (rank) read_b(0);
  // rows of base and out: 8 at a time, 8 lanes each
  int t[MT][2];
  lora_piece old[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      t[m][h] = static_cast<int>(tile.token(a, m0 + 16 * m + 8 * h + lr));
      const auto* const p =
          reinterpret_cast<const lora_piece*>(a.base + t[m][h] * a.base_stride + min(n0 + 8 * lp, a.N - 8));
      old[m][h] = MT > 1 ? __builtin_nontemporal_load(p) : *p;
    }
  // v: 2^sh pieces of a row, of which (rank + 7) / 8 are there
  const int per = (rank + 7) >> 3, sh = per > 1 ? 32 - __builtin_clz(per - 1) : 0;
  __syncthreads();                               // the previous tile's rows have been read
  for (int e = threadIdx.x; e < rows << sh; e += 64 * NW) {
    const int row = e >> sh, piece = e & ((1 << sh) - 1);
    if (piece >= per) continue;
    const float* v = a.v + tile.token(a, row) * a.vr + 8 * piece;
    f32x4 s0 = {}, s1 = {};
#pragma unroll 2
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
  if (n0 >= a.N || m0 >= rows) return;
  f32x4 acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = f32x4{};
  // rows of 4 pieces; piece p of row r at p ^ (r / 2 & 3): 8 rows of an operand fall to different banks
  const int put = lane ^ (lane >> 3 & 3);
  for (int r0 = 0; r0 < rank; r0 += 32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<lora_piece*>(mine + 64 * j + put) = raw[j];
    lora_in_order();
    if (r0 + 32 < rank) read_b(r0 + 32);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (r0 + 16 * s >= rank) continue;
      const int rr = r0 + 16 * s + 8 * (g & 1);
      bf16x8 bf[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        bf[j] = *reinterpret_cast<const bf16x8*>(mine + 64 * j + 4 * c + ((2 * s + (g & 1)) ^ (c >> 1 & 3)));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint4 v = vl[(2 * min(m0 + 16 * m + c, rows - 1) + (g >> 1)) * pitch + (rr < rank ? rr >> 3 : 0)];
        if (rr >= rank) v = uint4{};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], __builtin_bit_cast(bf16x8, v), acc[m][j], 0, 0, 0);
      }
    }
    lora_in_order();
  }
  // lane: columns 16 j + 4 g .. +3 of token c, which is piece 4 j + g of row c, at that ^ c
  const int n = n0 + 8 * lp;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4*>(mine + 16 * c + ((4 * j + g) ^ c)) = acc[m][j];
    lora_in_order();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 8 * h + lr;
      f32x4 s0 = *reinterpret_cast<const f32x4*>(mine + 16 * r + ((2 * lp) ^ r));
      f32x4 s1 = *reinterpret_cast<const f32x4*>(mine + 16 * r + ((2 * lp + 1) ^ r));
      const f32x4 all = s0 + s1;
      const float one = (all[0] + all[1]) + (all[2] + all[3]);
      if (__builtin_expect(one != one, 0)) lora_whole(a, tile.adapter, rank, t[m][h], min(n, a.N - 8), s0, s1);
      lora_piece o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x4& s = e < 2 ? s0 : s1;
        const uint32_t u = static_cast<uint32_t>(old[m][h][e]);
        o[e] = static_cast<int>(pack_bf16x2(fmaf(scale, s[2 * (e & 1)], __uint_as_float(u << 16)),
                                            fmaf(scale, s[2 * (e & 1) + 1], __uint_as_float(u & 0xFFFF0000u))));
      }
      if (m0 + 16 * m + r < rows && n < a.N) {
        auto* const p = reinterpret_cast<lora_piece*>(a.out + t[m][h] * a.out_stride + n);
        if (MT > 1) __builtin_nontemporal_store(o, p);
        else *p = o;
      }
    }
    lora_in_order();
  }
}

// Rows of the output: .y = 256 columns, 64 a wavefront; grouped, the second four wavefronts have the tokens from 32 on
// (4096 tokens of 4096 columns, rank 32: 21.0 us, and 23.3 with all 64 in each of four wavefronts, of which a CU then
// has 12 in place of 16; several strips of columns in turn, the next one's base on its way: 29 us).
template <bool GROUPED>
__global__ __launch_bounds__(64 * LORA_UP * (GROUPED ? 2 : 1), 4) void k_lora_up(LoraArgs a) {
  constexpr int NW = LORA_UP * (GROUPED ? 2 : 1);
  __shared__ uint4 turn[NW][256];
  extern __shared__ uint4 vl[];                  // [tokens of a tile: 64 grouped, else 16][2 halves][pitch] pieces of 8 values
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint4* const mine = turn[w];
  const int n0 = blockIdx.y * (64 * LORA_UP) + 64 * (w % LORA_UP), m0 = w / LORA_UP * 32;
  lora_tiles<GROUPED>(a, [&](const auto& tile) __attribute__((always_inline)) {
    if (tile.adapter < 0) {                      // base as it is, 8 tokens at a time
      const int lane = threadIdx.x & 63, n = n0 + 8 * (lane & 7);
      if (a.out == a.base || n >= a.N) return;
      for (int i = m0 + (lane >> 3); i < min(tile.rows, GROUPED ? m0 + 32 : 64); i += 8) {
        const int64_t t = tile.token(a, i);
        *reinterpret_cast<uint4*>(a.out + t * a.out_stride + n) =
            *reinterpret_cast<const uint4*>(a.base + t * a.base_stride + n);
      }
    } else if constexpr (GROUPED) {
      lora_columns<2, NW>(a, tile, n0, m0, vl, mine);
    } else {
      lora_columns<1, NW>(a, tile, n0, m0, vl, mine);
    }
  });
}

}  // namespace moe
