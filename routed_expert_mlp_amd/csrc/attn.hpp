// What the attention kernels share: arguments, a sequence's lengths, the
// visible keys of a query, and addresses inside the paged cache.
//
// Cache layout (include/moe_attn.h): K [page][head][dim / 8][token][8] and
// V [page][head][token / 8][dim][8], 16 bytes = 8 values along the reduction
// of the product that reads them.
#pragma once

#include "common.hpp"

namespace moe {

typedef float f32x16 __attribute__((ext_vector_type(16)));

struct AttnArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  const int32_t* seq_lens;
  const int32_t* page_table;
  const int32_t* cu_q;        // NULL: n_q tokens of every sequence
  float* ws;
  int64_t T;                  // rows of q
  int64_t max_pages;
  int32_t n_pages;
  int32_t B, n_q, max_len;    // n_q: new tokens per sequence (cu_q given: the most)
  int32_t heads, kv_heads, group;
  int32_t page_shift;
  int32_t window, sinks;      // window 0: none
  int32_t splits, tiles_per_split;   // parts of the visible tiles (at most), and their size
  int32_t col_blocks;         // prefill: column blocks of all sequences (at most)
  int32_t ws_cols;            // prefill: columns that a block has in the workspace
  float scale_log2;           // scale * log2(e): the softmax runs on exp2
};

// New tokens of a sequence that are computed (rows row0 .. row0 + n - 1 of q),
// its length, and the position of row0.
struct AttnSeq {
  int64_t row0;
  int n, len, first;
};

// The same for every lane; said so, because values out of vector loads would
// otherwise be kept, and worked on, in vector registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b) {
  AttnSeq s;
  s.len = uniform(min(max(a.seq_lens[b], 0), a.max_len));
  if (a.cu_q) {
    const int T = static_cast<int>(a.T);
    const int r0 = uniform(min(max(a.cu_q[b], 0), T));
    const int r1 = uniform(min(max(a.cu_q[b + 1], r0), T));
    s.row0 = r0;
    s.n = min(r1 - r0, a.n_q);
    s.first = s.len - (r1 - r0);       // of all its new tokens, also those past n_q
  } else {
    s.row0 = static_cast<int64_t>(b) * a.n_q;
    s.n = a.n_q;
    s.first = s.len - s.n;
  }
  return s;
}

// First key of the window of position p (0 without a window).
__device__ __forceinline__ int attn_window_lo(const AttnArgs& a, int p) {
  return a.window ? max(0, p - a.window + 1) : 0;
}

// The tiles of TS keys that hold a key visible to any of the positions
// first .. last (consecutive, so their windows join up): tiles 0 .. na-1 hold
// the sinks, tiles b0 .. the window up to key `last`; n in all.
struct AttnTiles {
  int na, b0, n;
  int lo, hi, sinks;        // visible to some position: key < hi and (key >= lo or key < sinks)
  int skip;                 // tiles before the part that n counts
  __device__ __forceinline__ int tile(int v) const {
    v += skip;
    return v < na ? v : v - na + b0;
  }
  // Keeps part `split` of parts of `size` tiles; false if there is none, except for an empty first one.
  __device__ __forceinline__ bool keep_part(int split, int size) {
    skip = split * size;
    n = min(n - skip, size);
    if (n > 0) return true;
    n = 0;
    return split == 0;
  }
};

template <int TS>
__device__ __forceinline__ AttnTiles attn_tiles(const AttnArgs& a, int first, int last) {
  AttnTiles t;
  t.hi = uniform(max(last + 1, 0));
  t.lo = uniform(attn_window_lo(a, first));
  t.sinks = a.window ? a.sinks : 0;
  t.b0 = t.lo / TS;
  t.na = (min(t.sinks, t.hi) + TS - 1) / TS;
  if (t.na >= t.b0) t.na = t.b0 = 0;
  t.n = uniform(t.hi ? t.na + (t.hi + TS - 1) / TS - t.b0 : 0);
  t.na = uniform(t.na);
  t.b0 = uniform(t.b0);
  t.skip = 0;
  return t;
}

// 32x32x16 MFMA, C = A B: lane l holds column l % 32 and rows
// 8 (e / 4) + 4 (l / 32) + e % 4 (e = 0..15) of C, and 8 reduction elements
// 8 (l / 32) .. +7 of row (column) l % 32 of A (B).
//
// Scores are computed transposed, keys x queries, so that a lane's 16 values
// belong to one query: its softmax needs one exchange between lanes l and
// l + 32, and the values go back in as the B operand of V^T P^T without any
// other exchange, provided the keys sit in the tile's rows in the right order:
// with key swap23(r) in row r (bits 2 and 3 swapped) value e of lane l is key
// 16 (e / 8) + 8 (l / 32) + e % 8, which is element e % 8 of that operand.
__device__ __forceinline__ int swap23(int r) { return (r & ~12) | ((r & 4) << 1) | ((r & 8) >> 1); }

// Bits 0 .. n-1.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1;
}

// Bit j: key key0 + j is visible to position p with window start lo:
// key <= p and (key >= lo or key < sinks).
__device__ __forceinline__ uint64_t visible_bits(int key0, int p, int lo, int sinks) {
  return low_bits(p + 1 - key0) & (~low_bits(lo - key0) | low_bits(sinks - key0));
}

// x where bit `bit` of the mask is set, else -inf.
__device__ __forceinline__ float keep_if(uint32_t mask, int bit, float x) {
  const uint32_t t = static_cast<uint32_t>(static_cast<int32_t>(mask << (31 - bit)) >> 31);
  return __uint_as_float((__float_as_uint(x) & t) | (0xFF800000u & ~t));
}

// The same mask for the 8 values of 8 keys (4 words of 2): bits 0..7.
__device__ __forceinline__ uint4 value_mask(uint32_t bits) {
  auto w = [&](int j) { return (bits >> j & 1 ? 0xFFFFu : 0u) | (bits >> (j + 1) & 1 ? 0xFFFF0000u : 0u); };
  return uint4{w(0), w(2), w(4), w(6)};
}

__device__ __forceinline__ uint4 and4(uint4 a, uint4 b) { return uint4{a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w}; }

// v of lane l and of lane l ^ 32, larger of the two.
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Rows that are read or written once and not soon again go around the caches
// (decode of 64 sequences of up to 4096 keys: 156 us with ordinary loads, 136 us
// with these; 4096 tokens prepared: 22.7 us and 21.5 us).
__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return uint4{v.x, v.y, v.z, v.w};
}

__device__ __forceinline__ uint2 load_stream(const uint2* p) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
  return uint2{v.x, v.y};
}

// Below every score, and finite: the running maximum of a row that has seen nothing.
constexpr float ATTN_NO_MAX = -1e30f;

}  // namespace moe
