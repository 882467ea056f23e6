// C ABI of the operators around the halves of the layer (declarations and
// contract in include/moe_proj.h).  Host code: argument validation before
// anything is enqueued, and the launches.  Nothing here allocates, synchronises
// or keeps state.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_proj.h"
#include "proj_fp8.hpp"
#include "proj_lora.hpp"
#include "proj_norm.hpp"

namespace {

using namespace moe;

constexpr int64_t kInt32End = int64_t(1) << 31;
constexpr int64_t kMaxTokens = int64_t(1) << 22;   // rows of one call: with 1024 threads each, 2^32 in all

bool aligned(const void* p, uintptr_t n = 16) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// hipLaunchKernel says whether this launch failed; an error that an earlier
// call of the process left behind is not taken for it.
template <typename A>
int launch(void (*kernel)(A), dim3 grid, dim3 block, hipStream_t s, A args, size_t lds = 0) {
  void* p[] = {&args};
  if (hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, p, lds, s) == hipSuccess)
    return MOE_MLP_OK;
  (void)hipGetLastError();
  return MOE_MLP_ERR_HIP;
}

bool features_ok(int64_t n, int64_t multiple) { return n >= multiple && n < MOE_PROJ_MAX_FEATURES && n % multiple == 0; }

bool stride_ok(int64_t stride, int64_t row) { return stride >= row && stride < kInt32End && stride % 8 == 0; }

// One piece of 8 values a lane as far as 16 wavefronts a row go: the pieces' reductions for the scales follow one
// another.  All outputs, wavefronts of one piece and half as many of two: 4096 columns, one row 2.8 and 3.5 us, 4096
// rows 30.3 and 31.5 us; 8192 columns, one row 3.7 and 4.1 (and 5.7 of four), 300 rows of 7168 8.1 and 8.6, but 4096
// rows 61.8 and 58.9.
template <int WPR, int NV>
int norm(const NormArgs& a, hipStream_t s) {
  return launch(k_proj_norm<WPR, NV>, dim3(static_cast<unsigned>(WPR == 1 ? cdiv(a.T, 4) : a.T)),
                dim3(WPR == 1 ? 256 : WPR * 64), s, a);
}

template <int NT, int MT, int U>
int fp8_few(const Fp8Args& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(cdiv(a.N, 16 * NT) * cdiv(a.T, 16 * MT)));
  return launch(k_proj_fp8_few<NT, MT, 8, U>, grid, dim3(512), s, a);
}

template <int WN, int WT, int TT, int SLOTS>
int fp8_tile(const Fp8Args& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(cdiv(cdiv(a.N, 64 * WN) * cdiv(a.T, 16 * TT * WT), 8) * 8));
  return launch(k_proj_fp8_tile<WN, WT, 4, TT, SLOTS>, grid, dim3(64 * WN * WT), s, a);
}

// The smallest blocks that the 256 CUs take at once, one each: a block's time is that of
// its chain of reads (4096 columns; blocks of 16 x 16, 32 x 16, 32 x 32, 64 x 32, 64 x 64
// outputs x tokens, tiles of 128 x 128; us, those not shown are slower):
//   1 token to 1024: 3.8, 4.5; 64 to 2048: 5.9, 5.7, 6.5; 32 to 6144: 9.5, 9.3, 8.4, 9.3;
//   64 to 6144: -, 12.3, 11.1, 9.9, 12.9; 128 to 6144: -, 19.4, 15.5, 16.3, 13.1, 22.
// Up to 16 tokens the weights' stream is all there is, and small blocks may share a CU
// (to 6144: 7.1, 7.4; to 12288: 10.7, 11.9; 2048 to 16384: 10.0, 7.8).  Past one block of
// 64 x 64 a CU, up to five of 32 x 32 (700 to 1536: -, -, 19.5, 22.3, 23.1, 21.9; 300 to
// 4096: -, -, 22.0, 23.7, 23.3, 21.8; 384 to 6144, nine of them: -, -, 38.4, 37.5, 34.3,
// 22.8), then tiles of 128 x 128, with four slots while each has a CU to itself (512 to
// 6144: 23.4 us, 25.9 with two slots) and two while two a CU have places at once (2048
// to 4096: 49 and 38 us), and of 256 x 256 after that (2048 to 4096 48, 4096 to 6144 104
// and 107 us).
int fp8(const Fp8Args& a, hipStream_t s) {
  auto blocks = [&](int n, int t) { return cdiv(a.N, n) * cdiv(a.T, t); };
  if (blocks(16, 16) <= (a.T <= 16 ? 768 : 256)) return fp8_few<1, 1, 4>(a, s);
  if (a.T <= 16 || blocks(32, 16) <= 256) return fp8_few<2, 1, 2>(a, s);
  if (blocks(32, 32) <= 256) return fp8_few<2, 2, 2>(a, s);
  if (blocks(64, 32) <= 256) return fp8_few<4, 2, 1>(a, s);
  if (blocks(64, 64) <= 256) return fp8_few<4, 4, 1>(a, s);
  if (blocks(32, 32) <= 5 * 256) return fp8_few<2, 2, 2>(a, s);
  if (blocks(128, 128) <= 256) return fp8_tile<2, 2, 4, 4>(a, s);
  if (blocks(128, 128) <= 512) return fp8_tile<2, 2, 4, 2>(a, s);
  return fp8_tile<4, 2, 8, 2>(a, s);
}

// How the adapters' products are cut.
struct LoraPlan {
  bool grouped;                      // by k_lora_group
  int64_t parts, part_chunks, down_x, up_x;
  int slots_down, slots_up, groups, col_blocks;
  size_t tiles_at, count_at, order_at, ws_bytes;     // in the workspace, behind v
};

// Every tile of a window reads its adapter again, and the sort is a launch more, of 4 to 10 us: as many tiles are read
// in less (4096 columns to 4096, windows and sorted: 512 tokens of 3 adapters of rank 16 or 64, 56 tiles, 12.6 and 17.7,
// 15.9 and 22.1 us; 1024 of them, 112 tiles, 20.9 and 19.9, 27.2 and 27.6; 128 tokens of 32, 72 tiles, 14.2 and 16.0,
// 20.5 and 20.3; 192 of them, 108 tiles, 19.6 and 15.8, 30.2 and 20.1).  The rule is that of those sizes: a tile costs
// by its rank and columns, a sort hardly, so that narrow calls would rather keep their windows (512 columns to 512, rank
// 8, 2048 tokens of 3 adapters 9.6 and 17.9 us) and wide ones leave them earlier (8192 to 8192, rank 128, 512 tokens of
// 3 45.0 and 33.9 us).  With LORA_BINS adapters or more, however many of them a call uses, windows are all there is:
// 4096 tokens of 50 of 511 adapters of rank 32 55 us, of 512 234 us.
constexpr int64_t LORA_WINDOW_TILES = 80;
// Blocks of k_lora_down: of a sorted call one a CU, 128 KB of LDS, its unfilled tiles counted too (as many parts as fill
// 256 with full tiles alone, and this way: 4096 tokens of 50 adapters of rank 32 51 and 46 us, 2000 of 4 of rank 128 43
// and 36 us, 200 of 60 of rank 32 27 and 23 us).
constexpr int64_t LORA_BLOCKS = 256;

LoraPlan lora_plan(const moe_proj_adapters* d, int64_t T) {
  LoraPlan p{};
  const int64_t chunks = cdiv(d->in_features, 64), vr = cdiv(d->max_rank, 16) * 16;
  p.groups = static_cast<int>(cdiv(d->max_rank, 16 * LORA_RT));
  p.col_blocks = static_cast<int>(cdiv(d->out_features, 64 * LORA_UP));
  // windows of 64 tokens, and the most tiles of up to 16 tokens of an adapter in one
  const int64_t windows = cdiv(T, 64), in = std::min<int64_t>(64, T), most = std::min(in, d->n_adapters + in / 16);
  p.grouped = windows * most > LORA_WINDOW_TILES && d->n_adapters < LORA_BINS;
  // sorted, every adapter, and the tokens without one, leave at most one tile unfilled
  const int64_t tiles = T / 64 + std::min(T, d->n_adapters + 1);
  // parts of the sum over the input; none shorter than 8 chunks of 64 columns
  const int64_t most_parts = cdiv(chunks, 8);
  const int64_t parts = LORA_BLOCKS / (p.grouped ? tiles * p.groups : windows);
  p.part_chunks = cdiv(chunks, std::max<int64_t>(1, std::min(most_parts, parts)));
  p.parts = cdiv(chunks, p.part_chunks);
  if (p.grouped) {
    p.down_x = p.up_x = tiles;
  } else {
    auto slots = [&](int64_t blocks) { return static_cast<int>(std::max<int64_t>(1, std::min(most, blocks))); };
    p.slots_down = slots(2048 / (windows * p.parts));
    p.slots_up = slots(4096 / (windows * p.col_blocks));
    p.down_x = windows * p.slots_down;
    p.up_x = windows * p.slots_up;
  }
  // of T tokens or fewer: more than one part only while parts x full tiles of 64 tokens are at most LORA_BLOCKS
  const int64_t rows = std::min(T * most_parts, std::max<int64_t>(T, LORA_BLOCKS * 64));
  p.tiles_at = size_t(rows) * vr * 4;
  p.count_at = p.tiles_at + size_t(tiles) * 16;
  p.order_at = p.count_at + 16;
  p.ws_bytes = p.order_at + size_t(T) * 4;
  return p;
}

int validate_adapters(const moe_proj_adapters* d, int64_t T) {
  if (!d) return MOE_MLP_ERR_NULL_ARG;
  if (T < 0 || T >= kMaxTokens) return MOE_MLP_ERR_BAD_SHAPE;
  if (d->n_adapters < 1 || d->n_adapters > (int64_t(1) << 20)) return MOE_MLP_ERR_BAD_SHAPE;
  if (d->max_rank < 8 || d->max_rank > MOE_PROJ_LORA_MAX_RANK || d->max_rank % 8 != 0) return MOE_MLP_ERR_BAD_SHAPE;
  if (!features_ok(d->in_features, 8) || !features_ok(d->out_features, 8)) return MOE_MLP_ERR_BAD_SHAPE;
  return MOE_MLP_OK;
}

}  // namespace

extern "C" {

int moe_proj_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual, const float* weight, float eps,
                  int64_t T, int64_t hidden, uint16_t* h_out, uint16_t* y_out, uint8_t* q_out, float* q_scale,
                  void* stream) {
  if (T < 0 || T >= kMaxTokens || hidden < 8 || hidden % 8 != 0 || hidden > MOE_PROJ_NORM_MAX_HIDDEN ||
      !stride_ok(x_stride, hidden))
    return MOE_MLP_ERR_BAD_SHAPE;
  if (!std::isfinite(eps) || eps < 0.0f) return MOE_MLP_ERR_BAD_VALUE;
  if (T == 0) return MOE_MLP_OK;
  if (!x || (!y_out && !q_out) || !q_out != !q_scale) return MOE_MLP_ERR_NULL_ARG;
  if (!aligned(x) || !aligned(residual) || !aligned(weight) || !aligned(h_out) || !aligned(y_out) || !aligned(q_out) ||
      !aligned(q_scale))
    return MOE_MLP_ERR_MISALIGNED;
  // an output row written into x has to be that row
  if ((h_out == x || y_out == x) && x_stride != hidden) return MOE_MLP_ERR_BAD_VALUE;
  if (h_out && h_out == y_out) return MOE_MLP_ERR_BAD_VALUE;
  NormArgs a{};
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.h = h_out;
  a.y = y_out;
  a.q = q_out;
  a.s = q_scale;
  a.x_stride = x_stride;
  a.T = T;
  a.hidden = static_cast<int32_t>(hidden);
  a.blocks = static_cast<int32_t>(cdiv(hidden, 128));
  a.eps = eps;
  a.per = 1.0f / static_cast<float>(hidden);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (hidden <= 512) return norm<1, 1>(a, s);
  if (hidden <= 1024) return norm<2, 1>(a, s);
  if (hidden <= 2048) return norm<4, 1>(a, s);
  if (hidden <= 4096) return norm<8, 1>(a, s);
  return hidden <= 8192 ? norm<16, 1>(a, s) : norm<16, 2>(a, s);
}

int moe_proj_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale, int64_t T, int64_t N,
                 int64_t K, uint16_t* y, void* stream) {
  if (T < 0 || T >= kMaxTokens || !features_ok(N, 16) || !features_ok(K, 128) || T * N >= int64_t(1) << 32)
    return MOE_MLP_ERR_BAD_SHAPE;
  if (T == 0) return MOE_MLP_OK;
  if (!x || !x_scale || !w || !w_scale || !y) return MOE_MLP_ERR_NULL_ARG;
  if (!aligned(x) || !aligned(x_scale) || !aligned(w) || !aligned(w_scale) || !aligned(y)) return MOE_MLP_ERR_MISALIGNED;
  Fp8Args a{};
  a.x = x;
  a.xs = x_scale;
  a.w = w;
  a.ws = w_scale;
  a.y = y;
  a.T = T;
  a.N = static_cast<int32_t>(N);
  a.K = static_cast<int32_t>(K);
  return fp8(a, static_cast<hipStream_t>(stream));
}

int moe_proj_lora_workspace_size(const moe_proj_adapters* adapters, int64_t T, size_t* bytes) {
  const int st = validate_adapters(adapters, T);
  if (st) return st;
  if (!bytes) return MOE_MLP_ERR_NULL_ARG;
  *bytes = T ? lora_plan(adapters, T).ws_bytes : 0;
  return MOE_MLP_OK;
}

int moe_proj_lora(const moe_proj_adapters* adapters, const uint16_t* x, int64_t x_stride, int64_t T,
                  const int32_t* adapter, const uint16_t* base, int64_t base_stride, uint16_t* out,
                  int64_t out_stride, void* workspace, size_t ws_bytes, void* stream) {
  const moe_proj_adapters* d = adapters;
  const int st = validate_adapters(d, T);
  if (st) return st;
  if (!stride_ok(x_stride, d->in_features) || !stride_ok(base_stride, d->out_features) ||
      !stride_ok(out_stride, d->out_features))
    return MOE_MLP_ERR_BAD_SHAPE;
  if (T == 0) return MOE_MLP_OK;
  if (!d->a || !d->b || !x || !adapter || !base || !out || !workspace) return MOE_MLP_ERR_NULL_ARG;
  if (!aligned(d->a) || !aligned(d->b) || !aligned(d->ranks, 4) || !aligned(d->scales, 4) || !aligned(x) ||
      !aligned(adapter, 4) || !aligned(base) || !aligned(out) || !aligned(workspace))
    return MOE_MLP_ERR_MISALIGNED;
  if (out == base && out_stride != base_stride) return MOE_MLP_ERR_BAD_VALUE;
  const LoraPlan p = lora_plan(d, T);
  if (ws_bytes < p.ws_bytes) return MOE_MLP_ERR_WORKSPACE_TOO_SMALL;
  LoraArgs a{};
  a.a = d->a;
  a.b = d->b;
  a.ranks = d->ranks;
  a.scales = d->scales;
  a.x = x;
  a.adapter = adapter;
  a.base = base;
  a.out = out;
  a.v = static_cast<float*>(workspace);
  a.x_stride = x_stride;
  a.base_stride = base_stride;
  a.out_stride = out_stride;
  a.T = T;
  a.n_adapters = d->n_adapters;
  a.R = d->max_rank;
  a.K = d->in_features;
  a.N = d->out_features;
  a.vr = static_cast<int32_t>(cdiv(d->max_rank, 16) * 16);
  a.bits = 64 - __builtin_clzll(static_cast<unsigned long long>(d->n_adapters));
  a.parts = static_cast<int32_t>(p.parts);
  a.part_chunks = static_cast<int32_t>(p.part_chunks);
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* const ws = static_cast<char*>(workspace);
  a.tiles = reinterpret_cast<int4*>(ws + p.tiles_at);
  a.n_tiles = reinterpret_cast<int32_t*>(ws + p.count_at);
  a.order = reinterpret_cast<int32_t*>(ws + p.order_at);
  if (p.grouped) {
    const int sg = launch(k_lora_group, dim3(1), dim3(64 * LORA_GROUP), s, a);
    if (sg) return sg;
  }
  a.slots = p.slots_down;
  const dim3 down(static_cast<unsigned>(p.down_x), static_cast<unsigned>(p.parts), static_cast<unsigned>(p.groups));
  const int sd = launch(p.grouped ? k_lora_down<true> : k_lora_down<false>, down, dim3(64 * LORA_DOWN), s, a);
  if (sd) return sd;
  a.slots = p.slots_up;
  return launch(p.grouped ? k_lora_up<true> : k_lora_up<false>,
                dim3(static_cast<unsigned>(p.up_x), static_cast<unsigned>(p.col_blocks)),
                dim3(64 * LORA_UP * (p.grouped ? 2 : 1)), s, a,
                size_t(2 * (p.grouped ? 64 : 16)) * (a.vr / 8 + 1) * 16);
}

}  // extern "C"
