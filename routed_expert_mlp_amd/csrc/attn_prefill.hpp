// Causal attention of prompts over the paged cache.
//
//   out = sum_k p_k v_k / sum_k p_k,  p_k = exp2(c q.k - m),  c = scale log2(e)
//
// with the running maximum m per query, in one pass over the keys.
//
// What bounds it: 4 D flops per query head and visible key on the matrix
// cores.  The softmax's exponentials, conversions and sums take the vector
// units nearly as long, so the two have to run at once; and the operands of
// every matrix instruction come from LDS at about the rate that it has.
//   * A wavefront owns 32 columns (query rows of one key/value head: new
//     token x head of the group, the head running faster, so that a key tile
//     serves the whole group) and a block NW of them.  64 columns a wavefront
//     would halve the reads of LDS, but their sums and weights do not fit its
//     registers (4096 tokens 271 us, copying them to and fro).
//   * Tiles of keys go from the cache to LDS by DMA, in rings of 2 slots for K
//     and 4 for V, in the cache's own order: operand fragments are then
//     consecutive 16 bytes a lane, free of bank conflicts, and nothing is
//     transposed.  (Rings of 4 and 4: 1-3% slower.)
//   * Scores are computed transposed (attn.hpp), so the weights go from the
//     softmax back into the matrix unit without leaving the lane.
//   * One iteration computes the scores of tile t + 1 while the vector units
//     turn those of tile t into weights (phase A), then adds tile t's
//     weighted values while they finish that and look for tile t + 1's maximum
//     (phase B); the sums are rescaled only when a maximum rises by more than
//     2^8.  There is one barrier a tile.
//   * Fragments are read four matrix instructions ahead of their use, across
//     the barrier.  The transfers are buffer loads: behind global ones the
//     compiler waits for all reads of LDS at every fragment.
//   * With few columns and a long cache (a piece of a prompt far into its
//     sequence) the key tiles are cut into parts, a block each, which
//     k_attn_prefill_join adds up.
//
// Measured, 32 query and 8 key/value heads of 128 dims: 4096 tokens 130 us,
// 1.06 PFLOP/s, where a large library matrix product reaches 1.2-1.4; the
// chip is at its power limit then (2.1 of 2.4 GHz).  Left out one after the
// other, the exponentials take 7% of that, the maximum 2%, the transfers 3% and
// the reads of LDS 17%; the rest is the products.  Window of 1024 and 4 sinks on
// 8192 tokens: 151-154 us, 840 TFLOP/s of visible pairs; a block then visits 35 tiles
// for the 32 that a query sees, and starts and ends too often to hide that.  Prompts
// of 1024 and 2048 tokens: 23 us (3.5 times what a large product would take) and 48
// us (1.8 times), where the longest block's tiles, one after the other, are the time.
//
// The weights meet the values in bf16, the type that the matrix instruction takes
// them in beside bf16 values; their sum is of the weights before that rounding.
// Against 64 bits the result is off by 1.8e-3 (37 tokens, 128 dims) to 2.3e-3
// (pieces, 64 dims) of its size, where rounding it alone makes 1.6e-3.
#pragma once

#include "attn.hpp"

#include <type_traits>

namespace moe {

constexpr int PF_RING = 4;           // slots for values
constexpr int PF_KRING = 2;          // slots for keys
constexpr int PF_AHEAD = 4;          // matrix instructions between a fragment's read and its use
constexpr int PF_IDS = 64;           // tiles whose page ids are in LDS, in two halves

template <int D, int NW_>
struct PrefillShape {
  static constexpr int NW = NW_;                                          // wavefronts of a block
  static constexpr int TS = D == 256 || (D == 128 && NW == 4) ? 32 : 64;  // keys of a tile
  static constexpr int COLS = 32 * NW;
  static constexpr int PER_CU = D == 256 || NW == 8 ? 1 : 2;              // blocks that a CU holds at once
};

// Column block r of all sequences' column blocks in a row: its sequence and its
// number there, counted from the last one (the longest); false past the end.
// Every wavefront looks it up for itself, 64 sequences at a time.  (With a grid
// of sequences x the most column blocks instead, most blocks of a ragged batch
// are empty, and the busy ones fall to the same shader engines: 8 pieces behind
// prefixes 105 us where this way took 70.)
template <int COLS>
__device__ __forceinline__ bool prefill_block(const AttnArgs& a, int r, int& b, int& cb) {
  if (a.B == 1) {
    b = 0;
    cb = (attn_seq(a, 0).n * a.group + COLS - 1) / COLS - 1 - r;
    return cb >= 0;
  }
  const int lane = threadIdx.x & 63, T = static_cast<int>(a.T);
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int n = 0;
    if (b0 + lane < a.B) {
      const int r0 = min(max(a.cu_q[b0 + lane], 0), T), r1 = min(max(a.cu_q[b0 + lane + 1], r0), T);
      n = (min(r1 - r0, a.n_q) * a.group + COLS - 1) / COLS;
    }
    int sum = n;                       // column blocks up to and with this lane's sequence
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
      const int y = __shfl_up(sum, x);
      sum += lane >= x ? y : 0;
    }
    const uint64_t past = __ballot(sum > r);
    if (past) {
      const int l = __builtin_ctzll(past);
      b = b0 + l;
      cb = __builtin_amdgcn_readlane(sum, l) - 1 - r;
      return true;
    }
    r -= __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

// The same for every lane, and kept in a scalar register: computed again in a
// branch that not all lanes take, it would come out of it in a vector register.
__device__ __forceinline__ int scalar(int v) {
  v = uniform(v);
  asm volatile("" : "+s"(v));
  return v;
}

// Where a column of a block (column block `block` of all, as prefill_block counts
// them) has its parts in the workspace: their sums, and behind all sums their
// maxima and totals.  By blocks and not by rows of q, so that the room that parts
// need follows the places of the GPU and not T.
__device__ __forceinline__ int64_t prefill_item(const AttnArgs& a, int block, int kvh, int col) {
  return ((static_cast<int64_t>(block) * a.kv_heads + kvh) * a.ws_cols + col) * a.splits;
}

__device__ __forceinline__ int64_t prefill_items(const AttnArgs& a) { return prefill_item(a, a.col_blocks, 0, 0); }

// Weights may exceed the running maximum by this many powers of two before
// the sums are rescaled (fp32 sums and bf16 weights have the range).
constexpr float PF_SLACK = 8.0f;

// LEAD: not the prompts of sequences, but the new tokens of a whole batch over the
// prefix that its sequences share (attn_shared.hpp), each at its own position, in
// parts that are left to k_attn_shared_join.
template <int D, int NW, bool LEAD = false>
__global__ __launch_bounds__(NW * 64, D == 256 ? 1 : 2) void k_attn_prefill(AttnArgs a) {
  constexpr int TS = PrefillShape<D, NW>::TS, COLS = PrefillShape<D, NW>::COLS;
  constexpr int RING = PF_RING, KRING = PF_KRING, KS = D / 16, DT = D / 32, SUB = TS / 32;
  constexpr int AHEAD = PF_AHEAD;
  constexpr int NP = 8 * SUB;                                    // pairs of scores of a lane
  constexpr int NSA = SUB * KS, NSB = 2 * SUB * DT;              // steps (matrix instructions) of the two phases
  static_assert(NSA % AHEAD == 0 && NSB % AHEAD == 0, "fragment i has register i % AHEAD");
  // Pairs that phase A turns into weights; phase B does the rest before step
  // LB, where the last 16 keys' values begin, and looks for the maximum before
  // step MB.  With more dims the matrix instructions of both phases hide the
  // softmax better than those of one (4096 tokens: 132 and 129.5 us); with 64
  // the values wait for the weights instead (8 pieces: 66.2 us this way, 67.0).
  constexpr int QA = D == 64 ? NP : NP * 5 / 8, LB = NSB - NSB / (2 * SUB), MB = NSB * 3 / 4;
  // key/value heads run fastest over the blocks: with a multiple of 8 of them
  // the blocks of one stay on one XCD, whose L2 then holds its keys
  const int kvh = blockIdx.x % a.kv_heads, bi = blockIdx.x / a.kv_heads, split = bi / a.col_blocks;
  int b, cb;
  AttnSeq s;
  if constexpr (LEAD) {
    b = 0;
    cb = bi - split * a.col_blocks;
    s = AttnSeq{0, a.B * a.n_q, a.shared, 0};
  } else {
    if (!prefill_block<COLS>(a, bi - split * a.col_blocks, b, cb)) return;
    s = attn_seq(a, b);
  }
  const int cols = s.n * a.group;
  const int c0 = cb * COLS;
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, half = lane >> 5;
  const int w = uniform(tid >> 6);
  const int first = s.first;
  int p_first, p_last;
  AttnTiles tl;
  AttnSpan span{};
  bool whole = false;
  if constexpr (LEAD) {
    span = attn_span(a, min(c0 + 32 * w + r, cols - 1), c0, min(c0 + COLS, cols));
    p_first = min(span.first, a.shared - 1);
    p_last = span.last;
    tl = attn_tiles_between<TS>(a, 0, attn_window_lo(a, span.first), min(a.shared, p_last + 1));
    if (!tl.keep_part(split, a.p_tiles_per_split)) tl.n = 0;
  } else {
    p_first = uniform(first + c0 / a.group), p_last = uniform(first + (min(c0 + COLS, cols) - 1) / a.group);
    tl = attn_tiles<TS>(a, p_first, p_last);
    whole = tl.n <= a.tiles_per_split;
    if (!tl.keep_part(split, a.tiles_per_split)) return;
  }
  const int last = scalar(tl.n - 1), skip = scalar(tl.skip), na = scalar(tl.na), jump = scalar(tl.b0 - tl.na);
  // first key of tile v of this part; past its end, of the last one
  auto key_of = [&](int v) __attribute__((always_inline)) {
    v = min(v, last) + skip;
    return TS * (v < na ? v : v + jump);
  };

  // slots are arrays of their own, so that the compiler knows which reads a
  // transfer in flight cannot touch
  __shared__ uint4 k0[TS * D / 8], k1[TS * D / 8];
  __shared__ uint4 v0[TS * D / 8], v1[TS * D / 8], v2[TS * D / 8], v3[TS * D / 8];
  __shared__ int ids[TS / 16 * PF_IDS];          // pages of 16 keys each
  uint4* const kslot[KRING] = {k0, k1};
  uint4* const vslot[RING] = {v0, v1, v2, v3};

  // this lane's column
  const int col = min(c0 + 32 * w + r, cols - 1);
  auto row_of = [&]() __attribute__((always_inline)) {
    const int tok = col / a.group;
    return (s.row0 + tok) * a.heads + kvh * a.group + (col - tok * a.group);
  };
  bf16x8 qf[KS];
  {
    const uint16_t* qp = a.q + row_of() * D + 8 * half;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) qf[ks] = *reinterpret_cast<const bf16x8*>(qp + 16 * ks);
  }
  // of this wavefront's columns, the first position and the last window start
  const int wp_first = LEAD ? p_first : uniform(first + min(c0 + 32 * w, cols - 1) / a.group);
  const int wlo_last =
      attn_window_lo(a, LEAD ? p_last : uniform(first + min(c0 + 32 * w + 31, cols - 1) / a.group));

  const int ps = 1 << a.page_shift;
  const uint32_t head_bytes = static_cast<uint32_t>(2 * D) << a.page_shift;
  const uint32_t page_bytes = head_bytes * a.kv_heads;
  // Pages of tiles v0 .. v0 + n - 1 to their places of `ids`.
  auto load_ids = [&](int first_tile, int n) __attribute__((always_inline)) {
    for (int i = tid; i < TS / 16 * n; i += NW * 64) {
      const int v = first_tile + i / (TS / 16), part = i % (TS / 16);
      const int key = min(key_of(v) + 16 * part, s.len - 1);
      const int32_t page = LEAD ? a.shared_pages[key >> a.page_shift]
                                : a.page_table[b * a.max_pages + (key >> a.page_shift)];
      ids[TS / 16 * (v & (PF_IDS - 1)) + part] = min(max(page, 0), a.n_pages - 1);
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);          // the writes have been done (lgkmcnt 0)
  };
  // Transfers: 64 pieces of 16 bytes to consecutive places of a slot, out of one
  // page, whose address is the same for all lanes.
  using lds_t = void __attribute__((address_space(3)));
  constexpr int NI = TS * D / 8 / 64 / NW;       // transfers of a wavefront for a tile's keys, and for its values
  auto bring = [&](const uint16_t* base, int id, int at, int lane_at, int step, uint4* dst) __attribute__((always_inline)) {
    const uint64_t src = reinterpret_cast<uint64_t>(base) + static_cast<uint64_t>(static_cast<uint32_t>(id)) * page_bytes +
                         static_cast<uint64_t>(kvh) * head_bytes + static_cast<uint32_t>(at);
    const uint64_t one = static_cast<uint32_t>(uniform(static_cast<uint32_t>(src))) |
                         static_cast<uint64_t>(static_cast<uint32_t>(uniform(static_cast<uint32_t>(src >> 32)))) << 32;
    const auto page = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(one), 0, head_bytes, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(page, (lds_t*)dst, 16, lane_at, step, 0, 0);
  };
  // K slot: [TS / 16][D / 8][16 keys][16 bytes], row j of 16 keys is key
  // swap23(j); a transfer brings 4 chunks of 8 dims of 16 keys, a wavefront's
  // are of the same keys
  constexpr int PER16 = D / 32;                  // transfers for 16 keys
  static_assert(PER16 % NI == 0, "one page a wavefront");
  const int kgroup = w * NI / PER16, kchunk = 4 * (w * NI % PER16);
  const int klane = (((kchunk + (lane >> 4)) << a.page_shift) + swap23(lane & 15)) * 16;
  auto key_page = [&](int v) __attribute__((always_inline)) {
    return ids[TS / 16 * (min(v, last) & (PF_IDS - 1)) + kgroup];
  };
  auto issue_k = [&](int v, int id, uint4* slot, int i) __attribute__((always_inline)) {
    bring(a.k, id, ((key_of(v) + 16 * kgroup) & (ps - 1)) * 16, klane, (64 * i) << a.page_shift,
          slot + (NI * w + i) * 64);
  };
  // V slot: [TS / 8][D][16 bytes]; wavefront w brings keys TS / NW * w and on, all of one page
  constexpr int WK = TS / NW;
  auto value_page = [&](int v) __attribute__((always_inline)) {
    return ids[TS / 16 * (min(v, last) & (PF_IDS - 1)) + (WK * w >> 4)];
  };
  auto issue_v = [&](int v, int id, uint4* slot, int i) __attribute__((always_inline)) {
    bring(a.v, id, ((key_of(v) + WK * w) & (ps - 1)) * (2 * D), lane * 16, 1024 * i,
          slot + (NI * w + i) * 64);
  };
  auto all_k = [&](int v) __attribute__((always_inline)) {
    const int id = uniform(key_page(v));
#pragma unroll
    for (int i = 0; i < NI; ++i) issue_k(v, id, kslot[v % KRING], i);
  };
  auto all_v = [&](int v) __attribute__((always_inline)) {
    const int id = uniform(value_page(v));
#pragma unroll
    for (int i = 0; i < NI; ++i) issue_v(v, id, vslot[v], i);
  };
  // Waits for this wavefront's transfers but the VM latest, then for the other
  // wavefronts to be here too.
  auto arrive = [&](auto vm) __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(decltype(vm)::value));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  f32x16 acc[DT], sa[SUB], sb[SUB];
  float m = ATTN_NO_MAX, l = 0.0f;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[dt][e] = 0.0f;

  // scores of invisible keys to -inf, where the tile has some for this wavefront
  auto mask = [&](int v, f32x16 (&x)[SUB]) __attribute__((always_inline)) {
    const int key0 = key_of(v);
    if (key0 + TS - 1 <= wp_first && (key0 >= wlo_last || key0 + TS <= tl.sinks)) return;
    const int pos = LEAD ? span.pos : first + col / a.group;
    const uint64_t see =
        visible_bits(key0 + 8 * half, LEAD ? min(pos, a.shared - 1) : pos, attn_window_lo(a, pos), tl.sinks);
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        x[sub][e] = keep_if(static_cast<uint32_t>(see >> (32 * sub)), 16 * (e >> 3) + (e & 7), x[sub][e]);
  };
  // new maximum (mt: the largest score of the tile), and the sums rescaled if it rose enough
  auto rescale = [&](float mt) __attribute__((always_inline)) {
    if (__builtin_expect(!__any(mt > m + PF_SLACK), 1)) return;
    const float mn = fmaxf(m, mt);
    const float f = exp2_fast(m - mn);
    m = mn;
    l *= f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[dt][e] *= f;
  };
  // values of keys that no column sees, whatever their slots hold, to 0 (all wavefronts)
  auto clear_holes = [&](int v, uint4* slot) __attribute__((always_inline)) {
    const int key0 = key_of(v);
    if constexpr (LEAD) {
      // windows of sequences that end inside the prefix may leave gaps between tl.lo and tl.hi
      if (a.window && p_first < a.shared - 1) {
        uint64_t any = 0;
        for (int t = c0 / a.group + lane; t <= (min(c0 + COLS, cols) - 1) / a.group; t += 64) {
          const int p = attn_position(a, t);
          any |= visible_bits(key0, min(p, a.shared - 1), attn_window_lo(a, p), tl.sinks);
        }
#pragma unroll
        for (int x = 32; x; x >>= 1) any |= __shfl_xor(any, x);
        for (int i = tid; i < TS * D / 8; i += NW * 64)
          slot[i] = and4(slot[i], value_mask(static_cast<uint32_t>(any >> (8 * (i / D)))));
        __syncthreads();
        return;
      }
    }
    if (key0 + TS <= tl.hi && (key0 >= tl.lo || key0 + TS <= tl.sinks)) return;
    for (int i = tid; i < TS * D / 8; i += NW * 64)
      slot[i] = and4(slot[i], value_mask(static_cast<uint32_t>(visible_bits(key0 + 8 * (i / D), tl.hi - 1, tl.lo, tl.sinks))));
    __syncthreads();
  };
  // Fragment i of a K slot (32 keys, then 16 dims on) or V slot (16 keys, then 32 dims on).
  bf16x8 fr[AHEAD];
  auto key_at = [&](int i) __attribute__((always_inline)) {
    return (r >> 4) * (2 * D) + 16 * half + (r & 15) + i / KS * (4 * D) + 32 * (i % KS);
  };
  auto read_k = [&](const uint4* slot, int i) __attribute__((always_inline)) {
    fr[i % AHEAD] = __builtin_bit_cast(bf16x8, slot[key_at(i)]);
  };
  auto read_v = [&](const uint4* slot, int i) __attribute__((always_inline)) {
    fr[i % AHEAD] = __builtin_bit_cast(bf16x8, slot[(2 * (i / DT) + half) * D + 32 * (i % DT) + r]);
  };
  int kid = 0, vid = 0;          // pages of the keys and values to bring next
  // Pair p of the scores to weights, their sum to l.
  uint32_t pk[2 * SUB][4];
  auto weigh = [&](int p, const f32x16 (&x)[SUB]) __attribute__((always_inline)) {
    const int su = p >> 3, e = 2 * (p & 7);
    const float p0 = exp2_fast(fmaf(x[su][e], a.scale_log2, -m));
    const float p1 = exp2_fast(fmaf(x[su][e + 1], a.scale_log2, -m));
    uint32_t pp = pack_bf16x2(p0, p1);
    l += p0 + p1;
    asm volatile("" : "+v"(pp), "+v"(l));        // here, beside the matrix instructions, and not where it is used
    pk[2 * su + (e >> 3)][(e & 7) >> 1] = pp;
  };
  auto weights = [&](int kk) __attribute__((always_inline)) {
    return __builtin_bit_cast(bf16x8, uint4{pk[kk][0], pk[kk][1], pk[kk][2], pk[kk][3]});
  };
  // Phases A and B of tile t; x: its scores, y: those of tile t + 1.  Between
  // the two, everyone is past its reads of the keys of tile t + 1 and the
  // values of tile t - 1, whose slots take the keys of t + 3 and the values of
  // t + 3 (past the end the last tile again, which nobody reads); the keys of
  // tile t + 2 and the values of t + 1 have come.
  // tiles inner0 .. inner1 - 1 are visible as a whole to every column
  const int inner0 = uniform(max(0, (attn_window_lo(a, p_last) + TS - 1) / TS - tl.b0) + tl.na - tl.skip);
  const int inner1 = uniform(p_first < 0 ? 0 : (p_first + 1) / TS - tl.b0 + tl.na - tl.skip);
  auto iteration = [&](auto jc, int t, f32x16 (&x)[SUB], f32x16 (&y)[SUB]) __attribute__((always_inline)) {
    constexpr int J = decltype(jc)::value;       // t % RING
    constexpr int GAP = NSB / (2 * NI) < 3 ? NSB / (2 * NI) : 3;   // steps between transfers
#pragma unroll
    for (int i = 0; i < NSA; ++i) {
      const int sub = i / KS;
      f32x16 z = {};
      y[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[i % AHEAD], qf[i % KS], i % KS ? y[sub] : z, 0, 0, 0);
      if (i + AHEAD < NSA) read_k(kslot[(J + 1) % KRING], i + AHEAD);
      else read_v(vslot[J], i + AHEAD - NSA);
#pragma unroll
      for (int p = i * QA / NSA; p < (i + 1) * QA / NSA; ++p) weigh(p, x);
      __builtin_amdgcn_sched_barrier(0);
    }
    arrive(std::integral_constant<int, NI>{});
    if (__builtin_expect(t + 1 < inner0 || t + 1 >= inner1, 0)) {
      clear_holes(t + 1, vslot[(J + 1) % RING]);
      mask(t + 1, y);
    }
    float mx = y[0][0];
    const int kpage = uniform(kid), vpage = uniform(vid);
#pragma unroll
    for (int i = 0; i < NSB; ++i) {
      acc[i % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[i % AHEAD], weights(i / DT), acc[i % DT], 0, 0, 0);
      if (i + AHEAD < NSB) read_v(vslot[J], i + AHEAD);
      else read_k(kslot[J % KRING], i + AHEAD - NSB);
      if (i % GAP == GAP - 1 && i / GAP < NI) issue_k(t + 3, kpage, kslot[(J + 1) % KRING], i / GAP);
      if (i % GAP == GAP - 1 && i / GAP >= NI && i / GAP < 2 * NI) issue_v(t + 3, vpage, vslot[(J + 3) % RING], i / GAP - NI);
      if (i == NSB - 1) {
        kid = key_page(t + 4);
        vid = value_page(t + 4);
      }
#pragma unroll
      for (int p = QA + min(i, LB) * (NP - QA) / LB; p < QA + min(i + 1, LB) * (NP - QA) / LB; ++p) weigh(p, x);
#pragma unroll
      for (int p = min(i, MB) * NP / MB; p < min(i + 1, MB) * NP / MB; ++p) {
        const int su = p >> 3, e = 2 * (p & 7);
        mx = fmaxf(fmaxf(mx, y[su][e]), y[su][e + 1]);
        asm volatile("" : "+v"(mx));
      }
      if (i == MB) mx = max_halves(mx) * a.scale_log2;
      __builtin_amdgcn_sched_barrier(0);
    }
    rescale(mx);
  };

  if (last >= 0) {
    load_ids(0, PF_IDS);
    __syncthreads();
    all_k(0);
    all_k(1);
    all_v(0);
    all_v(1);
    kid = key_page(3);
    vid = value_page(3);
    arrive(std::integral_constant<int, 3 * NI>{});
#pragma unroll
    for (int i = 0; i < NSA; ++i) {
      f32x16 z = {};
      const bf16x8 f = __builtin_bit_cast(bf16x8, k0[key_at(i)]);
      sa[i / KS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, qf[i % KS], i % KS ? sa[i / KS] : z, 0, 0, 0);
    }
    mask(0, sa);
    float mx = sa[0][0];
#pragma unroll
    for (int su = 0; su < SUB; ++su)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, sa[su][e]);
    rescale(max_halves(mx) * a.scale_log2);
    arrive(std::integral_constant<int, NI>{});   // and everyone is past its reads of the keys of tile 0
    all_k(2);
    all_v(2);
    clear_holes(0, v0);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      read_k(k1, i);
      __builtin_amdgcn_sched_barrier(0);         // in this order, which the waits in the loop count on
    }
    for (int t = 0; t < last; t += RING) {
      if (__builtin_expect(t % (PF_IDS / 2) == 0 && t, 0)) load_ids(t + PF_IDS / 2, PF_IDS / 2);
      iteration(std::integral_constant<int, 0>{}, t, sa, sb);
      if (t + 1 >= last) break;
      iteration(std::integral_constant<int, 1>{}, t + 1, sb, sa);
      if (t + 2 >= last) break;
      iteration(std::integral_constant<int, 2>{}, t + 2, sa, sb);
      if (t + 3 >= last) break;
      iteration(std::integral_constant<int, 3>{}, t + 3, sb, sa);
    }
    // the last tile's weights and values; transfers end before the block gives up its LDS
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    if (last & 1) {
#pragma unroll
      for (int su = 0; su < SUB; ++su) sa[su] = sb[su];
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) weigh(p, sa);
    const int j = last % RING;
    const uint4* vl = j == 0 ? v0 : j == 1 ? v1 : j == 2 ? v2 : v3;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) read_v(vl, i);
#pragma unroll
    for (int i = 0; i < NSB; ++i) {
      acc[i % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[i % AHEAD], weights(i / DT), acc[i % DT], 0, 0, 0);
      if (i + AHEAD < NSB) read_v(vl, i + AHEAD);
    }
  }

  float lt = sum_halves(l);
  if (LEAD && span.pos < 0) lt = 0.0f;           // tiles that the other columns see as a whole are not masked for it
  if (!LEAD && c0 + 32 * w + r >= cols) return;
  const int64_t row = row_of();
  if (!whole) {
    int64_t item;
    float *sums, *ml;
    if constexpr (LEAD) {
      item = (static_cast<int64_t>(kvh) * cols + col) * a.p_splits + split;
      sums = a.pws;
      ml = a.pml;
    } else {
      item = prefill_item(a, bi - split * a.col_blocks, kvh, 32 * w + r) + split;
      sums = a.ws;
      ml = a.ws + prefill_items(a) * D;
    }
    if constexpr (LEAD) {
      const bool mine = c0 + 32 * w + r < cols;
      uint32_t alone = 0;                        // columns whose sums attn_part_alone has
      if (a.window || p_first < a.shared - 1) {  // where columns may see different keys
        float sum = 0.0f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int e = 0; e < 16; ++e) sum += acc[dt][e];
        const uint64_t nan = __ballot(mine && lt != 0.0f && sum != sum);
        alone = static_cast<uint32_t>(nan | nan >> 32);
        for (uint32_t left = alone; left; left &= left - 1) {
          const int i = __builtin_ctz(left);
          attn_part_alone<D, TS>(a, tl, kvh, c0 + 32 * w + i, __shfl(span.pos, i), __shfl(m, i),
                                 sums + __shfl(item, i) * D);
        }
      }
      if (!mine) return;
      if (half == 0) *reinterpret_cast<float2*>(ml + 2 * item) = float2{m, lt};
      // a part without keys has a sum of 0, and its values are not read
      if (last < 0 || (alone >> r & 1)) return;
    } else if (half == 0) {
      *reinterpret_cast<float2*>(ml + 2 * item) = float2{m, lt};
    }
    float* o = sums + item * D + 4 * half;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(o + 32 * dt + 8 * i) =
            f32x4{acc[dt][4 * i], acc[dt][4 * i + 1], acc[dt][4 * i + 2], acc[dt][4 * i + 3]};
    return;
  }
  const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
  uint16_t* o = a.out + row * D + 4 * half;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 p = {pack_bf16x2(acc[dt][4 * i] * inv, acc[dt][4 * i + 1] * inv),
                       pack_bf16x2(acc[dt][4 * i + 2] * inv, acc[dt][4 * i + 3] * inv)};
      *reinterpret_cast<uint2*>(o + 32 * dt + 8 * i) = p;
    }
}

// Joins the parts of the columns that k_attn_prefill left in parts: a block
// takes 4 NC of a column block's columns, a wavefront NC of them side by side,
// D / 64 dims a lane, in one pass over the parts with a running maximum.  Up to
// 6400 rows a wavefront has one, and more parts in flight (50 tokens of 16/1 heads
// of 256 dims behind 6000: 26 us in all, and 39 us with four; 400 of 16 heads,
// 6400 rows, 46 and 49 us, of 128 dims 34.8 and 34.0 us), above that four (8 pieces
// of 50 of 32/8 heads of 128 dims 39 us, and 43 us with one).
template <int D, int NW, int NC>
__global__ __launch_bounds__(256) void k_attn_prefill_join(AttnArgs a) {
  constexpr int TS = PrefillShape<D, NW>::TS, COLS = PrefillShape<D, NW>::COLS, ND = D / 64;
  constexpr int PER = COLS / (4 * NC), AT_ONCE = NC == 1 ? 8 : 4;
  const int kvh = blockIdx.x % a.kv_heads, bi = blockIdx.x / a.kv_heads;
  int b, cb;
  if (!prefill_block<COLS>(a, bi / PER, b, cb)) return;
  const AttnSeq s = attn_seq(a, b);
  const int cols = s.n * a.group, c0 = cb * COLS, first = s.first;
  const AttnTiles tl = attn_tiles<TS>(a, uniform(first + c0 / a.group),
                                      uniform(first + (min(c0 + COLS, cols) - 1) / a.group));
  if (tl.n <= a.tiles_per_split) return;
  const int parts = (tl.n + a.tiles_per_split - 1) / a.tiles_per_split;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const float2* const ml = reinterpret_cast<const float2*>(a.ws + prefill_items(a) * D);
  const int col0 = c0 + 4 * NC * (bi % PER) + NC * w;
  int64_t row[NC], first_item[NC];
  float M[NC], L[NC], o[NC][ND];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int col = min(col0 + i, cols - 1), t = col / a.group;
    row[i] = (s.row0 + t) * a.heads + kvh * a.group + (col - t * a.group);
    first_item[i] = prefill_item(a, bi / PER, kvh, col - c0);
    M[i] = ATTN_NO_MAX;
    L[i] = 0.0f;
#pragma unroll
    for (int n = 0; n < ND; ++n) o[i][n] = 0.0f;
  }
#pragma unroll AT_ONCE
  for (int j = 0; j < parts; ++j) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t item = first_item[i] + j;
      const float2 p = ml[item];
      const float* src = a.ws + item * D + lane * ND;
      const float mn = fmaxf(M[i], p.x);
      const float f = exp2_fast(M[i] - mn), g = exp2_fast(p.x - mn);
      M[i] = mn;
      L[i] = L[i] * f + p.y * g;
#pragma unroll
      for (int n = 0; n < ND; ++n) o[i][n] = o[i][n] * f + src[n] * g;
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (col0 + i >= cols) return;
    const float inv = L[i] > 0.0f ? 1.0f / L[i] : 0.0f;
    uint16_t* out = a.out + row[i] * D + lane * ND;
    if constexpr (ND == 1) {
      out[0] = f32_to_bf16(o[i][0] * inv);
    } else {
#pragma unroll
      for (int n = 0; n < ND; n += 2)
        *reinterpret_cast<uint32_t*>(out + n) = pack_bf16x2(o[i][n] * inv, o[i][n + 1] * inv);
    }
  }
}

}  // namespace moe
