// Causal attention of prompts over the paged cache.
//
// What bounds it: 4 D flops per query head and visible key on the matrix
// cores; the softmax's exponentials, conversions and sums on the vector units
// take a little less time than that, so the two have to run at once.
//   * A block is 4 wavefronts, one per SIMD with up to 512 registers, and 4 x
//     32 CT columns (CT = 2, and 1 at 256 dims): the query rows of one
//     key/value head, (new token, head of the group) with the head running
//     faster, so that a key tile serves the whole group.  64 columns a
//     wavefront halve the LDS reads per matrix instruction against 32: each
//     operand fragment of K or V feeds two of them.
//   * Tiles of 64 keys go from the cache to LDS by DMA, two slots for K and
//     two for V, in the cache's own order: fragments are then consecutive 16
//     bytes a lane, free of bank conflicts, and nothing is transposed.
//   * Scores are computed transposed (attn.hpp), so the weights go from the
//     softmax back into the matrix unit without leaving the lane.
//   * One iteration computes the scores of tile t + 1 while the vector units
//     turn those of tile t into weights, then adds tile t's weighted values
//     while they look for tile t + 1's maximum; the sums are rescaled only
//     when a maximum rises by more than 2^8.
#pragma once

#include "attn.hpp"

namespace moe {

constexpr int PF_TS = 64;            // keys of a tile

template <int D>
struct PrefillShape {
  static constexpr int CT = 1;
  static constexpr int NW = D == 256 ? 4 : 8;
  static constexpr int COLS = NW * 32 * CT;
};

// Weights may exceed the running maximum by this many powers of two before
// the sums are rescaled (fp32 sums and bf16 weights have the range).
constexpr float PF_SLACK = 8.0f;

template <int D>
__global__ __launch_bounds__(PrefillShape<D>::NW * 64, 1) void k_attn_prefill(AttnArgs a) {
  constexpr int NW = PrefillShape<D>::NW, CT = PrefillShape<D>::CT, COLS = PrefillShape<D>::COLS, KS = D / 16, DT = D / 32;
  constexpr int NSA = 2 * KS, NSB = 4 * DT;     // steps (of CT matrix instructions) of the two phases
  constexpr int NP = 16 * CT;                   // pairs of scores of a lane
  // pairs a step, and steps a pair
  constexpr int PA = NP > NSA ? NP / NSA : 1, SA = NP > NSA ? 1 : NSA / NP;
  constexpr int PB = NP > NSB ? NP / NSB : 1, SB = NP > NSB ? 1 : NSB / NP;
  // key/value heads run fastest over the blocks: with a multiple of 8 of them
  // the blocks of one stay on one XCD, whose L2 then holds its keys; the
  // longest column blocks start first
  const int groups = a.B * a.kv_heads;
  const int gi = blockIdx.x % groups;
  const int cb = static_cast<int>(gridDim.x) / groups - 1 - static_cast<int>(blockIdx.x) / groups;
  const int kvh = gi % a.kv_heads, b = gi / a.kv_heads;
  const AttnSeq s = attn_seq(a, b);
  const int cols = s.n * a.group;
  const int c0 = cb * COLS;
  if (c0 >= cols) return;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, r = lane & 31, half = lane >> 5;
  const int first = s.len - s.n;
  const int p_first = first + c0 / a.group, p_last = first + (min(c0 + COLS, cols) - 1) / a.group;
  const AttnTiles tl = attn_tiles<PF_TS>(a, p_first, p_last);

  __shared__ uint4 k0[D * 8], k1[D * 8], v0[D * 8], v1[D * 8];

  // this lane's columns
  int pos[CT], wlo[CT];
  int64_t row[CT];
  bf16x8 qf[CT][KS];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int col = min(c0 + 32 * (CT * w + ct) + r, cols - 1);
    const int t = col / a.group;
    pos[ct] = first + t;
    wlo[ct] = attn_window_lo(a, pos[ct]);
    row[ct] = (s.row0 + t) * a.heads + kvh * a.group + (col - t * a.group);
    const uint16_t* qp = a.q + row[ct] * D + 8 * half;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) qf[ct][ks] = *reinterpret_cast<const bf16x8*>(qp + 16 * ks);
  }
  // of this wavefront's columns, the first and last position and the last window start
  const int wp_first = first + min(c0 + 32 * CT * w, cols - 1) / a.group;
  const int wp_last = first + min(c0 + 32 * CT * (w + 1) - 1, cols - 1) / a.group;
  const int wlo_last = attn_window_lo(a, wp_last);

  const int ps = 1 << a.page_shift;
  const int64_t head_elems = static_cast<int64_t>(D) << a.page_shift;
  // Key of the tile that this lane loads (row l of the K slot holds key
  // swap23(l % 32) of its half), and its page.
  const int lkey = 32 * half + swap23(r);
  auto page_of = [&](int v) __attribute__((always_inline)) {
    const int key = min(PF_TS * tl.tile(min(v, tl.n - 1)) + lkey, s.len - 1);
    return min(max(a.page_table[b * a.max_pages + (key >> a.page_shift)], 0), a.n_pages - 1);
  };
  using lds_t = void __attribute__((address_space(3)));
  // K slot: [D / 8][64 keys][16 bytes]; wavefront w brings every fourth row
  auto issue_k = [&](int v, int id, uint4* slot) __attribute__((always_inline)) {
    const int at = (PF_TS * tl.tile(v) + lkey) & (ps - 1);
    const uint16_t* p = a.k + (static_cast<int64_t>(id) * a.kv_heads + kvh) * head_elems +
                        ((static_cast<int64_t>(w) << a.page_shift) + at) * 8;
#pragma unroll
    for (int i = 0; i < D / 8 / NW; ++i)
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(p + ((NW * i * 8) << a.page_shift)),
                                       (lds_t*)(slot + (NW * i + w) * 64), 16, 0, 0);
  };
  // V slot: [8 groups of 8 keys][D][16 bytes]; wavefront w brings keys 16 w .. +15
  // (one page), whose page is that of the key that lane 16 w loads
  auto issue_v = [&](int v, int id, uint4* slot) __attribute__((always_inline)) {
    constexpr int WK = PF_TS / NW;                // keys a wavefront brings
    const int at = (PF_TS * tl.tile(v) + WK * w) & (ps - 1);
    const int vid = __builtin_amdgcn_readlane(id, swap23(WK * w));
    const uint16_t* p = a.v + (static_cast<int64_t>(vid) * a.kv_heads + kvh) * head_elems + at * D + lane * 8;
#pragma unroll
    for (int i = 0; i < D / 8 / NW; ++i)
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(p + 512 * i), (lds_t*)(slot + D * 8 / NW * w + 64 * i),
                                       16, 0, 0);
  };
  auto arrive = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  f32x16 acc[CT][DT], sa[2][CT], sb[2][CT];
  float m[CT], l[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    m[ct] = ATTN_NO_MAX;
    l[ct] = 0.0f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[ct][dt][e] = 0.0f;
  }

  // scores of invisible keys to -inf, where the tile has some for this wavefront
  auto mask = [&](int v, f32x16 (&x)[2][CT]) __attribute__((always_inline)) {
    const int key0 = PF_TS * tl.tile(v);
    if (key0 + PF_TS - 1 <= wp_first && (key0 >= wlo_last || key0 + PF_TS <= tl.sinks)) return;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const uint64_t see = visible_bits(key0 + 8 * half, pos[ct], wlo[ct], tl.sinks);
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          x[sub][ct][e] = keep_if(static_cast<uint32_t>(see >> (32 * sub)), 16 * (e >> 3) + (e & 7), x[sub][ct][e]);
    }
  };
  // new maxima (mx: this lane's largest scores), and the sums rescaled if one rose enough
  auto rescale = [&](const float (&mx)[CT]) __attribute__((always_inline)) {
    float mt[CT];
    bool up = false;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      mt[ct] = max_halves(mx[ct]) * a.scale_log2;
      up |= mt[ct] > m[ct] + PF_SLACK;
    }
    if (!__any(up)) return;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const float mn = fmaxf(m[ct], mt[ct]);
      const float f = exp2_fast(m[ct] - mn);
      m[ct] = mn;
      l[ct] *= f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[ct][dt][e] *= f;
    }
  };
  // values of keys that no column sees, whatever their slots hold, to 0 (all wavefronts)
  auto clear_holes = [&](int v, uint4* slot) __attribute__((always_inline)) {
    const int key0 = PF_TS * tl.tile(v);
    if (key0 + PF_TS <= tl.hi && (key0 >= tl.lo || key0 + PF_TS <= tl.sinks)) return;
    for (int i = tid; i < D * 8; i += NW * 64) {
      const int ka = key0 + 8 * (i / D);
      slot[i] = and4(slot[i], value_mask(static_cast<uint32_t>(visible_bits(ka, tl.hi - 1, tl.lo, tl.sinks))));
    }
    __syncthreads();
  };
  auto kfrag = [&](const uint4* slot, int step) __attribute__((always_inline)) {          // step = sub * KS + ks
    return __builtin_bit_cast(bf16x8, slot[(2 * (step % KS) + half) * 64 + 32 * (step / KS) + r]);
  };
  auto vfrag = [&](const uint4* slot, int step) __attribute__((always_inline)) {          // step = 16 keys * DT + dt
    return __builtin_bit_cast(bf16x8, slot[(2 * (step / DT) + half) * D + 32 * (step % DT) + r]);
  };

  // One iteration: weights and values of tile v, scores of tile v + 1.
  // kn: slot of tile v + 1's keys; kf: slot for tile v + 2's; vc: slot of
  // tile v's values; vf: slot for tile v + 1's.  id1, id2: pages of tiles
  // v + 1 and v + 2.
  auto iteration = [&](int v, f32x16 (&sc)[2][CT], f32x16 (&sn)[2][CT], const uint4* kn, uint4* kf, uint4* vc, uint4* vf, int id1, int id2) __attribute__((always_inline)) {
    arrive();
    if (v + 2 < tl.n) issue_k(v + 2, id2, kf);
    if (v + 1 < tl.n) issue_v(v + 1, id1, vf);
    clear_holes(v, vc);
    uint32_t pk[CT][4][4];
    constexpr int AHEAD = 3;
    bf16x8 fr[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fr[i] = kfrag(kn, i);
#pragma unroll
    for (int i = 0; i < NSA; ++i) {
      const int sub = i / KS, ks = i % KS;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x16 z = {};
        sn[sub][ct] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[i % AHEAD], qf[ct][ks], ks == 0 ? z : sn[sub][ct], 0, 0, 0);
      }
      if (i + AHEAD < NSA) fr[i % AHEAD] = kfrag(kn, i + AHEAD);
#pragma unroll
      for (int j = 0; j < PA; ++j) {
        if (i % SA) break;
        const int p = i / SA * PA + j;
        const int ct = p % CT, q = p / CT, su = q >> 3, e = 2 * (q & 7);   // pair of tile v's scores
        const float p0 = exp2_fast(fmaf(sc[su][ct][e], a.scale_log2, -m[ct]));
        const float p1 = exp2_fast(fmaf(sc[su][ct][e + 1], a.scale_log2, -m[ct]));
        l[ct] += p0 + p1;
        pk[ct][2 * su + (e >> 3)][(e & 7) >> 1] = pack_bf16x2(p0, p1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (v + 1 < tl.n) mask(v + 1, sn);
    float mx[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) mx[ct] = sn[0][ct][0];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fr[i] = vfrag(vc, i);
#pragma unroll
    for (int i = 0; i < NSB; ++i) {
      const int kk = i / DT, dt = i % DT;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const uint4 pf = {pk[ct][kk][0], pk[ct][kk][1], pk[ct][kk][2], pk[ct][kk][3]};
        acc[ct][dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[i % AHEAD], __builtin_bit_cast(bf16x8, pf), acc[ct][dt], 0, 0, 0);
      }
      if (i + AHEAD < NSB) fr[i % AHEAD] = vfrag(vc, i + AHEAD);
#pragma unroll
      for (int j = 0; j < PB; ++j) {
        if (i % SB) break;
        const int p = i / SB * PB + j;
        const int ct = p % CT, q = p / CT, su = q >> 3, e = 2 * (q & 7);
        mx[ct] = fmaxf(fmaxf(mx[ct], sn[su][ct][e]), sn[su][ct][e + 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (v + 1 < tl.n) rescale(mx);
  };

  if (tl.n > 0) {
    int ida = page_of(0), idb = page_of(1);
    issue_k(0, ida, k0);
    issue_v(0, ida, v0);
    if (tl.n > 1) issue_k(1, idb, k1);
    arrive();
#pragma unroll
    for (int i = 0; i < NSA; ++i) {
      const int sub = i / KS, ks = i % KS;
      const bf16x8 f = kfrag(k0, i);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x16 z = {};
        sa[sub][ct] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, qf[ct][ks], ks == 0 ? z : sa[sub][ct], 0, 0, 0);
      }
    }
    mask(0, sa);
    float mx[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      mx[ct] = sa[0][ct][0];
#pragma unroll
      for (int su = 0; su < 2; ++su)
#pragma unroll
        for (int e = 0; e < 16; ++e) mx[ct] = fmaxf(mx[ct], sa[su][ct][e]);
    }
    rescale(mx);
    for (int v = 0; v < tl.n; v += 2) {
      // page of tile v + 2 was asked for two tiles ago, in the shadow of the work since
      const int idc = page_of(v + 2);
      iteration(v, sa, sb, k1, k0, v0, v1, idb, idc);
      ida = idc;
      if (v + 1 >= tl.n) break;
      idb = page_of(v + 3);
      iteration(v + 1, sb, sa, k0, k1, v1, v0, ida, idb);
    }
  }

#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const float lt = sum_halves(l[ct]);
    const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
    if (c0 + 32 * (CT * w + ct) + r >= cols) continue;
    uint16_t* o = a.out + row[ct] * D + 4 * half;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 p = {pack_bf16x2(acc[ct][dt][4 * i] * inv, acc[ct][dt][4 * i + 1] * inv),
                         pack_bf16x2(acc[ct][dt][4 * i + 2] * inv, acc[ct][dt][4 * i + 3] * inv)};
        *reinterpret_cast<uint2*>(o + 32 * dt + 8 * i) = p;
      }
  }
}

}  // namespace moe
