// Low-rank adapters of many requests beside a shared projection.
//
//   v[t] = x[t] A_a^T;  out[t] = base[t] + s_a v[t] B_a^T,   a = adapter[t]
//
// Two kernels.  Both take the tokens in windows of 64, as many as a wavefront has
// lanes: each wavefront reads the window's adapter numbers, one a lane, finds the
// adapters that occur with ballots, and gathers the tokens of one of them, in
// whatever order they come, into the rows of a matrix product.  An adapter is read
// once for the tokens that a window has of it, and nothing has to be sorted.
//
// v is a sum over thousands of columns, cut into parts for the blocks; the second
// kernel adds up the parts (fp32, in order), and gives v to the matrix unit as the
// sum of two bf16 values, beside the bf16 weights: 16 bits of it, at the price of
// half a matrix instruction more, where the time is that of the memory.
#pragma once

#include "common.hpp"

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
  float* v;                  // [parts][T][R]
  int64_t x_stride, base_stride, out_stride, T, n_adapters;
  int32_t R, K, N;           // R: max_rank, up to a multiple of 16 in v
  int32_t vr;                // columns of v
  int32_t parts, part_chunks;     // of K: parts, and chunks of 64 columns of one
  int32_t slots;             // blocks that share a window's adapters
};

constexpr int LORA_WINDOW = 64;   // tokens of a window
constexpr int LORA_RT = 4;        // 16-rank tiles of a block of the first kernel

// The adapters of a window, one after the other; all lanes the same.
struct LoraWindow {
  uint64_t rest, mine;       // lanes not yet seen; lanes of the present adapter
  int id;                    // this lane's adapter, -1: none
  int now;                   // the present adapter
  __device__ __forceinline__ bool next() {
    if (!rest) return false;
    now = __builtin_amdgcn_readlane(id, __builtin_ctzll(rest));
    mine = __ballot(id == now);
    rest &= ~mine;
    return true;
  }
  __device__ __forceinline__ int tokens() const { return __popcll(mine); }
};

__device__ __forceinline__ LoraWindow lora_window(const LoraArgs& a, int64_t t0) {
  const int lane = threadIdx.x & 63;
  LoraWindow w;
  w.id = -1;
  if (t0 + lane < a.T) {
    const int id = a.adapter[t0 + lane];
    if (id >= 0 && id < a.n_adapters) w.id = id;
  }
  w.rest = __ballot(w.id >= 0);
  w.mine = 0;
  w.now = 0;
  return w;
}

__device__ __forceinline__ int lora_rank(const LoraArgs& a, int id) {
  return __builtin_amdgcn_readfirstlane(a.ranks ? min(max(a.ranks[id], 0), a.R) : a.R);
}

// Place (0..63) in the window of token number n among the lanes of `mine`; the last one past its end.
__device__ __forceinline__ int lora_place(uint64_t mine, int n) {
  n = min(n, __popcll(mine) - 1);
  int at = 0;
#pragma unroll
  for (int step = 32; step; step >>= 1) {
    const uint64_t low = step == 32 ? 0xFFFFFFFFull : ((uint64_t(1) << step) - 1);
    const int here = __popcll((mine >> at) & low);
    if (n >= here) {
      n -= here;
      at += step;
    }
  }
  return at;
}

// v of the tokens of a window: blockIdx.x = window * slots + slot, .y = part of K, .z = group of 64 ranks.
// The four wavefronts take the part's chunks of 64 columns in turn and join in LDS.
__global__ __launch_bounds__(256) void k_lora_down(LoraArgs a) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot = blockIdx.x % a.slots, part = blockIdx.y, r0 = blockIdx.z * (16 * LORA_RT);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / a.slots) * LORA_WINDOW;
  const int pieces = a.K >> 3;                   // of 8 columns
  const int c0 = part * a.part_chunks, c1 = min(c0 + a.part_chunks, (pieces + 7) >> 3);
  __shared__ f32x4 join[3][4][LORA_RT][64];
  LoraWindow win = lora_window(a, t0);
  for (int i = 0; win.next(); ++i) {
    if (i % a.slots != slot) continue;
    const int rank = lora_rank(a, win.now);
    const int tiles = min((rank - r0 + 15) >> 4, LORA_RT), rows = win.tokens(), mt = (rows + 15) >> 4;
    if (tiles <= 0) continue;
    const uint4* xp[4];
    const uint4* ap[LORA_RT];
#pragma unroll
    for (int m = 0; m < 4; ++m)
      xp[m] = reinterpret_cast<const uint4*>(a.x + (t0 + lora_place(win.mine, 16 * m + c)) * a.x_stride);
#pragma unroll
    for (int n = 0; n < LORA_RT; ++n)
      ap[n] = reinterpret_cast<const uint4*>(a.a + (static_cast<int64_t>(win.now) * a.R + min(r0 + 16 * n + c, a.R - 1)) * a.K);
    f32x4 acc[4][LORA_RT];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int n = 0; n < LORA_RT; ++n) acc[m][n] = f32x4{};
    for (int k = c0 + w; k < c1; k += 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p = 8 * k + 4 * h + g;
        const bool in = p < pieces;
        bf16x8 xf[4], af[LORA_RT];
#pragma unroll
        for (int n = 0; n < LORA_RT; ++n) {
          uint4 v = {};
          if (n < tiles && in && r0 + 16 * n + c < rank) v = ap[n][p];
          af[n] = __builtin_bit_cast(bf16x8, v);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          uint4 v = {};
          if (m < mt && in) v = xp[m][p];
          xf[m] = __builtin_bit_cast(bf16x8, v);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int n = 0; n < LORA_RT; ++n)
            if (m < mt && n < tiles) acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[n], xf[m], acc[m][n], 0, 0, 0);
      }
    }
    // wavefront 0 adds up the four; lane: token c of a tile, ranks 4 g .. +3
    __syncthreads();
    if (w) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < LORA_RT; ++n)
          if (m < mt && n < tiles) join[w - 1][m][n][lane] = acc[m][n];
    }
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m >= mt || 16 * m + c >= rows) continue;
        float* v = a.v + (static_cast<int64_t>(part) * a.T + t0 + lora_place(win.mine, 16 * m + c)) * a.vr + r0 + 4 * g;
#pragma unroll
        for (int n = 0; n < LORA_RT; ++n)
          if (n < tiles)
            *reinterpret_cast<f32x4*>(v + 16 * n) =
                (acc[m][n] + join[0][m][n][lane]) + (join[1][m][n][lane] + join[2][m][n][lane]);
      }
    }
  }
}

// Rows of the output: blockIdx.x = window * slots + slot, .y = 256 columns, 64 a wavefront.  Lane: token c of a
// tile, columns 16 g .. +15 of the wavefront's 64 (row 4 g + i of matrix tile j is column 16 g + 4 j + i).
__global__ __launch_bounds__(256) void k_lora_up(LoraArgs a) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot = blockIdx.x % a.slots;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / a.slots) * LORA_WINDOW;
  const int n0 = blockIdx.y * 256 + 64 * w;
  if (n0 >= a.N) return;
  LoraWindow win = lora_window(a, t0);
  // tokens without an adapter: the first slot's
  if (slot == 0 && a.out != a.base) {
    uint64_t none = ~win.rest & (a.T - t0 >= 64 ? ~uint64_t(0) : (uint64_t(1) << (a.T - t0)) - 1);
    while (none) {
      const int at = __builtin_ctzll(none);
      none &= none - 1;
      if (lane < 8 && n0 + 8 * lane < a.N)
        reinterpret_cast<uint4*>(a.out + (t0 + at) * a.out_stride + n0)[lane] =
            reinterpret_cast<const uint4*>(a.base + (t0 + at) * a.base_stride + n0)[lane];
    }
  }
  for (int i = 0; win.next(); ++i) {
    if (i % a.slots != slot) continue;
    const int rank = lora_rank(a, win.now), rows = win.tokens(), mt = (rows + 15) >> 4;
    const float scale = a.scales ? a.scales[win.now] : 1.0f;
    const uint16_t* bp[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = min(n0 + 16 * (c >> 2) + 4 * j + (c & 3), a.N - 1);
      bp[j] = a.b + (static_cast<int64_t>(win.now) * a.N + n) * a.R;
    }
    for (int m = 0; m < mt; ++m) {
      const bool live = 16 * m + c < rows;
      const int64_t t = t0 + lora_place(win.mine, 16 * m + c);
      const float* vp = a.v + t * a.vr;
      f32x4 acc[4] = {};
      // 16 ranks an instruction: lanes of g = 0, 1 have their upper halves, g = 2, 3 what is left of them
      for (int r = 0; r < rank; r += 16) {
        const int rr = r + 8 * (g & 1);
        float f[8] = {};
        if (rr < rank) {
          for (int p = 0; p < a.parts; ++p) {
            const f32x4* s = reinterpret_cast<const f32x4*>(vp + static_cast<int64_t>(p) * a.T * a.vr + rr);
            const f32x4 s0 = s[0], s1 = s[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] += s0[e];
              f[4 + e] += s1[e];
            }
          }
        }
        bf16x8 vf;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __bf16 hi = static_cast<__bf16>(f[e]);
          const __bf16 lo = static_cast<__bf16>(f[e] - static_cast<float>(hi));
          vf[e] = rr + e < rank ? (g < 2 ? hi : lo) : static_cast<__bf16>(0.0f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 q = {};
          if (rr < rank) q = *reinterpret_cast<const uint4*>(bp[j] + rr);
          bf16x8 bf = __builtin_bit_cast(bf16x8, q);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (rr + e >= rank) bf[e] = static_cast<__bf16>(0.0f);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf, vf, acc[j], 0, 0, 0);
        }
      }
      if (live) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = n0 + 16 * g + 8 * h;
          if (n >= a.N) continue;
          const uint4 old = *reinterpret_cast<const uint4*>(a.base + t * a.base_stride + n);
          const uint32_t u[4] = {old.x, old.y, old.z, old.w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f32x4& s = acc[2 * h + (e >> 1)];
            o[e] = pack_bf16x2(fmaf(scale, s[2 * (e & 1)], __uint_as_float(u[e] << 16)),
                               fmaf(scale, s[2 * (e & 1) + 1], __uint_as_float(u[e] & 0xFFFF0000u)));
          }
          *reinterpret_cast<uint4*>(a.out + t * a.out_stride + n) = uint4{o[0], o[1], o[2], o[3]};
        }
      }
    }
  }
}

}  // namespace moe
