// C ABI of the attention operators (declarations and contract in
// include/moe_attn.h).  Host code: argument validation before anything is
// enqueued, and the launches.  Nothing here allocates, synchronises or keeps
// state.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/moe_attn.h"
#include "attn.hpp"
#include "attn_decode.hpp"
#include "attn_prefill.hpp"
#include "attn_prepare.hpp"

namespace {

using namespace moe;

constexpr int64_t kInt32End = int64_t(1) << 31;
constexpr int64_t kMaxTokens = int64_t(1) << 26;   // rows of one call
constexpr int64_t kMaxColumns = int64_t(1) << 30;  // prefill: heads of a sequence's rows, which the kernels count in 32 bits
constexpr int64_t kMaxRagged = int64_t(1) << 16;   // prefill: sequences that each wavefront goes through to find its own
constexpr int64_t kMaxKeys = int64_t(1) << 30;     // no sequence is as long: as good as no limit
constexpr int64_t kMaxThreads = int64_t(1) << 32;  // of a launch, along one side; a grid takes fewer

bool aligned(const void* p, uintptr_t n = 16) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int page_shift_of(int32_t page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

int validate_cfg(const moe_attn_config* c) {
  if (!c) return MOE_MLP_ERR_NULL_ARG;
  if (c->n_heads < 1 || c->n_heads > MOE_ATTN_MAX_HEADS || c->n_kv_heads < 1 || c->n_heads % c->n_kv_heads != 0)
    return MOE_MLP_ERR_BAD_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_MLP_ERR_BAD_SHAPE;
  if (page_shift_of(c->page_size) < 0) return MOE_MLP_ERR_BAD_SHAPE;
  if (c->rotary_dim < 0 || c->rotary_dim > c->head_dim || c->rotary_dim % 16 != 0) return MOE_MLP_ERR_BAD_SHAPE;
  if (c->rope_style != MOE_ATTN_ROPE_HALF && c->rope_style != MOE_ATTN_ROPE_INTERLEAVED)
    return MOE_MLP_ERR_BAD_VALUE;
  if (c->window < 0 || c->n_sinks < 0) return MOE_MLP_ERR_BAD_VALUE;
  if (!std::isfinite(c->norm_eps) || c->norm_eps < 0.0f) return MOE_MLP_ERR_BAD_VALUE;
  if (!std::isfinite(c->scale) || !(c->scale > 0.0f)) return MOE_MLP_ERR_BAD_VALUE;
  return MOE_MLP_OK;
}

int validate_cache(const moe_attn_config* c, const moe_attn_cache* cache) {
  if (!cache || !cache->k || !cache->v) return MOE_MLP_ERR_NULL_ARG;
  if (cache->n_pages < 1 || cache->n_pages >= kInt32End / c->page_size) return MOE_MLP_ERR_BAD_SHAPE;
  if (!aligned(cache->k) || !aligned(cache->v)) return MOE_MLP_ERR_MISALIGNED;
  return MOE_MLP_OK;
}

// Blocks of moe_attn_prepare that fill the GPU (925 tokens of 128/8 heads of 128
// dims: 17.9 us, with 1024 blocks 19.4, with 2048 21.0).
constexpr int64_t PREP_BLOCKS = 1536;

// hipLaunchKernel says whether this launch failed; an error that an earlier
// call of the process left behind is not taken for it.
template <typename A>
int launch(void (*kernel)(A), dim3 grid, dim3 block, hipStream_t s, A args) {
  void* p[] = {&args};
  if (hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, p, 0, s) == hipSuccess)
    return MOE_MLP_OK;
  (void)hipGetLastError();
  return MOE_MLP_ERR_HIP;
}

// Calls f(std::integral_constant<int, head_dim>).
template <typename F>
int with_dim(int head_dim, F&& f) {
  switch (head_dim) {
    case 64: return f(std::integral_constant<int, 64>{});
    case 128: return f(std::integral_constant<int, 128>{});
    default: return f(std::integral_constant<int, 256>{});
  }
}

// Sizes that both forms of attention check: B sequences, at most max_q new
// tokens and max_len tokens of each.
int validate_sizes(const moe_attn_config* c, int64_t T, int64_t B, int64_t max_q, int64_t max_len, int prefill) {
  const int st = validate_cfg(c);
  if (st) return st;
  if (T < 0 || T >= kMaxTokens) return MOE_MLP_ERR_BAD_SHAPE;
  if (B < 0 || max_q < 0 || max_len < 0 || B >= kInt32End || max_q >= kInt32End || max_len >= kMaxKeys)
    return MOE_MLP_ERR_BAD_SHAPE;
  if (!prefill && (max_q < 1 || max_q > MOE_ATTN_DECODE_MAX_Q)) return MOE_MLP_ERR_BAD_SHAPE;
  if (B && max_q * c->n_heads >= kMaxTokens / B && (!prefill || B >= kMaxRagged)) return MOE_MLP_ERR_BAD_SHAPE;
  if (B && prefill && std::min(max_q, T) * c->n_heads >= kMaxColumns) return MOE_MLP_ERR_BAD_SHAPE;
  return MOE_MLP_OK;
}

// How a decode call is cut: columns (new tokens x query heads of a key/value
// head) in blocks of 32, the visible tiles of 32 keys in parts.
struct DecodePlan {
  int col_blocks, splits, tiles_per_split;
  int join_waves;                    // of an output row of the join
  int64_t blocks, join_blocks;
  size_t ws_bytes;
};

// The most 32-key tiles that the new tokens of a sequence see.
int64_t decode_tiles(const moe_attn_config* c, int64_t n_q, int64_t max_len) {
  const int64_t tiles = cdiv(max_len, 32);
  if (!c->window) return tiles;
  return std::min(tiles, cdiv(int64_t(c->window) + n_q, 32) + 1 + cdiv(c->n_sinks, 32));
}

DecodePlan decode_plan(const moe_attn_config* c, int64_t B, int64_t n_q, int64_t max_len) {
  DecodePlan p{};
  const int64_t cols = n_q * (c->n_heads / c->n_kv_heads);
  const int64_t tiles = decode_tiles(c, n_q, max_len);
  p.col_blocks = static_cast<int>(cdiv(cols, 32));
  // parts that together fill the places of the GPU's 256 CUs once, if all
  // sequences were as long as the longest may be; no smaller than a tile per
  // wavefront, and no larger than ATTN_MAX_TPS, since the others should not
  // wait for one long sequence
  const int64_t places = 256 * attn_blocks_per_cu(c->head_dim);
  int64_t tps = cdiv(cdiv(B * c->n_kv_heads * p.col_blocks * tiles, places), ATTN_NW) * ATTN_NW;
  tps = tps < ATTN_NW ? ATTN_NW : tps > ATTN_MAX_TPS ? ATTN_MAX_TPS : tps;
  p.tiles_per_split = static_cast<int>(tps);
  p.splits = tiles ? static_cast<int>(cdiv(tiles, tps)) : 1;
  p.blocks = B * c->n_kv_heads * p.splits;
  if (p.col_blocks > 1) p.blocks = cdiv(p.blocks, 8) * 8 * p.col_blocks;
  const int64_t rows = B * n_q * c->n_heads;
  p.join_waves = rows < 1024 ? 4 : 1;            // measured at k_attn_join
  p.join_blocks = p.splits > 1 ? cdiv(rows, 4 / p.join_waves) : 0;
  if (p.splits > 1) p.ws_bytes = size_t(B) * c->n_kv_heads * cols * p.splits * (c->head_dim + 2) * 4;
  return p;
}

// The most workspace of a decode call with no larger sizes.  Items (a column's
// sums of a part) are rows x parts.  Parts shorter than ATTN_MAX_TPS are at most
// places / blocks + 1 of each sequence, and a block has at most min(cols, 32)
// columns; the others are as many as the longest sequence has.
size_t decode_bound(const moe_attn_config* c, int64_t B, int64_t n_q, int64_t max_len) {
  const int64_t tiles = decode_tiles(c, n_q, max_len);
  if (tiles <= ATTN_NW) return 0;
  const int64_t cols = n_q * (c->n_heads / c->n_kv_heads), rows = B * c->n_kv_heads * cols;
  int64_t items = std::min(rows * cdiv(tiles, ATTN_NW),
                           std::min<int64_t>(cols, 32) * 256 * attn_blocks_per_cu(c->head_dim) + rows);
  if (tiles > ATTN_MAX_TPS) items = std::max(items, rows * cdiv(tiles, ATTN_MAX_TPS));
  return size_t(items) * (c->head_dim + 2) * 4;
}

// How a prefill call is cut: column blocks of all sequences, and the visible tiles of a
// block in parts where there are too few blocks to fill the GPU.
struct PrefillPlan {
  int64_t col_blocks, tiles;         // tiles: the most that a column block can see
  int splits, tiles_per_split;
  int ws_cols;                       // columns of a block that can be there
  int join_rows;                     // of a wavefront of the join
  int64_t blocks, join_blocks;
  size_t ws_bytes, ws_bound;
};

constexpr int64_t PF_LEAST = 8;      // tiles of a part, but for a last one

template <int D, int NW>
PrefillPlan prefill_plan(const moe_attn_config* c, int64_t T, int64_t B, int64_t max_q, int64_t max_len) {
  using S = PrefillShape<D, NW>;
  PrefillPlan p{};
  max_q = std::min(max_q, T);
  const int64_t group = c->n_heads / c->n_kv_heads;
  // every sequence leaves at most one column block unfilled
  p.col_blocks = std::min(B * cdiv(max_q * group, S::COLS), T * group / S::COLS + B);
  const int64_t busy = p.col_blocks * c->n_kv_heads;
  int64_t tiles = cdiv(max_len, S::TS);
  if (c->window)
    tiles = std::min(tiles, cdiv(int64_t(c->window) + cdiv(S::COLS, group), S::TS) + 1 + cdiv(c->n_sinks, S::TS));
  // Parts where the longest block's tiles take longer than its parts' and the
  // join: about TILE_NS a tile, 1.6 times that with two blocks on a CU, and for
  // the join 4 us and the partial sums' way out and back.  Parts of one size that
  // have places at once, or as many as there are places if all blocks were as
  // long as the longest may be; none shorter than PF_LEAST tiles.  32/8 heads: 512
  // tokens behind 65024 cached ones 466 us, and 1248 us whole; 64 behind 7168
  // 23 and 123 us, behind 1024 14.3 and 23 us; 8 pieces of 8/2 heads of 256 dims
  // behind prefixes 71 and 108 us; but 1024 tokens of a prompt 23.3 us whole, and
  // 28.8 us in two parts.
  constexpr int64_t TILE_NS = D == 64 ? 600 : D == 256 ? 780 : NW == 8 ? 1900 : 550;
  const int64_t places = 256 * S::PER_CU, rows = std::min(T, B * max_q) * c->n_heads;
  int64_t size = tiles, best = tiles * TILE_NS * (busy > 256 ? 8 : 5) / 5;
  auto consider = [&](int64_t tps) {
    const int64_t ns = tps * TILE_NS * (busy * tiles > 256 * tps ? 8 : 5) / 5 + 4000 +
                       rows * cdiv(tiles, tps) * D * 8 / (D == 64 ? 4000 : 6000);
    if (ns < best) best = ns, size = tps;
  };
  for (int64_t n = 2; busy * n <= places && tiles >= PF_LEAST * n; n += n / 4 + 1) consider(cdiv(tiles, n));
  if (busy <= places) consider(std::max(cdiv(busy * tiles, places), PF_LEAST));
  p.tiles = tiles;
  p.tiles_per_split = static_cast<int>(std::max<int64_t>(size, 1));
  p.splits = tiles ? static_cast<int>(cdiv(tiles, size)) : 1;
  p.blocks = busy * p.splits;
  p.join_rows = rows <= 6400 ? 1 : 4;                 // measured at k_attn_prefill_join
  p.join_blocks = p.splits > 1 ? busy * (S::COLS / (4 * p.join_rows)) : 0;
  p.ws_cols = static_cast<int>(std::min<int64_t>(max_q * group, S::COLS));
  if (p.splits > 1) p.ws_bytes = size_t(p.blocks) * p.ws_cols * (D + 2) * 4;
  // The most that a call with no larger sizes takes: parts come only where the
  // column blocks have places at once, at most ceil(places / blocks) of each, none
  // shorter than PF_LEAST tiles.
  if (tiles > PF_LEAST)
    p.ws_bound = size_t(std::min(busy * cdiv(tiles, PF_LEAST), places + std::min(busy, places))) * p.ws_cols * (D + 2) * 4;
  return p;
}

// Calls f(head_dim, wavefronts of a block) with both as integral constants.  At
// 128 dims a block has 8 wavefronts, which share a tile's transfers, or 4 with
// tiles of 32 keys, two blocks a CU, of which one starts or ends while the other
// computes.  Long blocks that fill the GPU for 16 tiles want the former (32/8
// heads: 4096 tokens 130 us, and 144 us with 4; 512 tokens behind 65024 466 and
// 533 us, behind 3072 41.4 and 44.5 us), short or few ones the latter (2048 tokens
// 48 us, and 51 us with 8; a window of 1024 on 8192 tokens 151 and 159 us; 256
// tokens behind 3072 27.3 and 29.5 us; 16 behind 8176 16.3 and 19.5 us).  Other widths
// have one form.
template <typename F>
int with_prefill_shape(const moe_attn_config* c, int64_t T, int64_t B, int64_t max_q, int64_t max_len, F&& f) {
  using four = std::integral_constant<int, 4>;
  using eight = std::integral_constant<int, 8>;
  return with_dim(c->head_dim, [&](auto dc) {
    if constexpr (decltype(dc)::value == 128) {
      const PrefillPlan p = prefill_plan<128, 4>(c, T, B, max_q, max_len);
      if (p.tiles > 64 && p.col_blocks * c->n_kv_heads * p.tiles > 16 * 512) return f(dc, eight{});
    }
    return f(dc, four{});
  });
}

template <int D>
int decode(const AttnArgs& a, const DecodePlan& p, hipStream_t s) {
  const int st = launch(p.col_blocks > 1 ? k_attn_decode<D, true> : k_attn_decode<D, false>,
                        dim3(static_cast<unsigned>(p.blocks)), dim3(ATTN_NW * 64), s, a);
  if (st || p.splits == 1) return st;
  const dim3 grid(static_cast<unsigned>(p.join_blocks));
  return p.join_waves == 1 ? launch(k_attn_join<D, 1>, grid, dim3(256), s, a)
                           : launch(k_attn_join<D, 4>, grid, dim3(256), s, a);
}

int attention(const moe_attn_config* c, const moe_attn_cache* cache, const uint16_t* q, int64_t T, const int32_t* cu_q,
              int64_t B, int64_t max_q, const int32_t* seq_lens, const int32_t* page_table, int64_t max_pages,
              int64_t max_len, uint16_t* out, void* workspace, size_t ws_bytes, void* stream, int prefill) {
  size_t need = 0;
  int st = moe_attn_workspace_size(c, T, B, max_q, max_len, prefill, &need);
  if (st) return st;
  if (max_pages < 0 || max_pages >= kInt32End || max_len > max_pages * c->page_size) return MOE_MLP_ERR_BAD_SHAPE;
  if (!prefill) T = B * max_q;
  if (B == 0 || T == 0 || max_q == 0) return MOE_MLP_OK;
  st = validate_cache(c, cache);
  if (st) return st;
  if (!q || !out || !seq_lens || (prefill && !cu_q) || (max_len > 0 && !page_table)) return MOE_MLP_ERR_NULL_ARG;
  if (need && !workspace) return MOE_MLP_ERR_NULL_ARG;
  if (!aligned(q) || !aligned(out) || !aligned(workspace) || !aligned(seq_lens, 4) || !aligned(page_table, 4) ||
      !aligned(cu_q, 4))
    return MOE_MLP_ERR_MISALIGNED;
  if (ws_bytes < need) return MOE_MLP_ERR_WORKSPACE_TOO_SMALL;
  AttnArgs a{};
  a.q = q;
  a.k = cache->k;
  a.v = cache->v;
  a.out = out;
  a.seq_lens = seq_lens;
  a.page_table = page_table;
  a.cu_q = prefill ? cu_q : nullptr;
  a.ws = static_cast<float*>(workspace);
  a.T = T;
  a.max_pages = max_pages;
  a.n_pages = static_cast<int32_t>(cache->n_pages);
  a.B = static_cast<int32_t>(B);
  a.n_q = static_cast<int32_t>(max_q);
  a.max_len = static_cast<int32_t>(max_len);
  a.heads = c->n_heads;
  a.kv_heads = c->n_kv_heads;
  a.group = c->n_heads / c->n_kv_heads;
  a.page_shift = page_shift_of(c->page_size);
  a.window = static_cast<int32_t>(std::min<int64_t>(c->window, kMaxKeys));
  a.sinks = static_cast<int32_t>(std::min<int64_t>(c->n_sinks, kMaxKeys));
  a.scale_log2 = c->scale * 1.44269504088896340736f;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!prefill) {
    const DecodePlan p = decode_plan(c, B, max_q, max_len);
    a.splits = p.splits;
    a.tiles_per_split = p.tiles_per_split;
    return with_dim(c->head_dim, [&](auto dc) { return decode<decltype(dc)::value>(a, p, s); });
  }
  return with_prefill_shape(c, T, B, max_q, max_len, [&](auto dc, auto nc) {
    constexpr int D = decltype(dc)::value, NW = decltype(nc)::value;
    const PrefillPlan p = prefill_plan<D, NW>(c, T, B, max_q, max_len);
    a.splits = p.splits;
    a.tiles_per_split = p.tiles_per_split;
    a.col_blocks = static_cast<int32_t>(p.col_blocks);
    a.ws_cols = p.ws_cols;
    const int st = launch(k_attn_prefill<D, NW>, dim3(static_cast<unsigned>(p.blocks)), dim3(NW * 64), s, a);
    if (st || p.splits == 1) return st;
    const dim3 grid(static_cast<unsigned>(p.join_blocks));
    return p.join_rows == 1 ? launch(k_attn_prefill_join<D, NW, 1>, grid, dim3(256), s, a)
                            : launch(k_attn_prefill_join<D, NW, 4>, grid, dim3(256), s, a);
  });
}

}  // namespace

extern "C" {

int moe_attn_prepare(const moe_attn_config* cfg, const moe_attn_cache* cache, const uint16_t* qkv,
                     int64_t qkv_stride, int64_t T, const float* q_norm_w, const float* k_norm_w,
                     const float* cos_sin, int64_t n_positions, const int32_t* positions, const int64_t* slots,
                     uint16_t* q_out, void* stream) {
  int st = validate_cfg(cfg);
  if (st) return st;
  const int64_t rows = cfg->n_heads + 2 * int64_t(cfg->n_kv_heads);
  if (T < 0 || T >= kMaxTokens || qkv_stride < rows * cfg->head_dim || qkv_stride % 8 != 0 ||
      qkv_stride >= kInt32End)
    return MOE_MLP_ERR_BAD_SHAPE;
  if (cfg->rotary_dim && n_positions < 1) return MOE_MLP_ERR_BAD_SHAPE;
  if (T == 0) return MOE_MLP_OK;
  st = validate_cache(cfg, cache);
  if (st) return st;
  if (!qkv || !slots || !q_out || (cfg->rotary_dim && (!cos_sin || !positions))) return MOE_MLP_ERR_NULL_ARG;
  if (!aligned(qkv) || !aligned(q_out) || !aligned(q_norm_w) || !aligned(k_norm_w) || !aligned(cos_sin) ||
      !aligned(positions, 4) || !aligned(slots, 8))
    return MOE_MLP_ERR_MISALIGNED;
  PrepArgs a{};
  a.qkv = qkv;
  a.k = cache->k;
  a.v = cache->v;
  a.q_out = q_out;
  a.qw = q_norm_w;
  a.kw = k_norm_w;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.slots = slots;
  a.stride = qkv_stride;
  a.T = T;
  a.n_positions = n_positions;
  a.n_slots = cache->n_pages * cfg->page_size;
  a.heads = cfg->n_heads;
  a.kv_heads = cfg->n_kv_heads;
  a.page_shift = page_shift_of(cfg->page_size);
  a.rotary = cfg->rotary_dim;
  a.interleaved = cfg->rope_style == MOE_ATTN_ROPE_INTERLEAVED;
  a.eps = cfg->norm_eps;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return with_dim(cfg->head_dim, [&](auto dc) {
    constexpr int D = decltype(dc)::value;
    const int64_t token_blocks = cdiv(T, 2048 / D);
    // one head a block while the blocks are few, up to 8 with thousands of them
    // (4096 tokens of 32/8 heads of 128 dims: 21.7 us, and 26.9 us with one always;
    // 64 tokens of 64/8 heads: 3.6 us, and 8.1 us with 8 always)
    const int64_t per = rows * token_blocks / PREP_BLOCKS;
    a.rows_per_block = static_cast<int32_t>(per < 1 ? 1 : per > 8 ? 8 : per);
    return launch(k_attn_prepare<D>, dim3(static_cast<unsigned>(token_blocks),
                                          static_cast<unsigned>(cdiv(rows, a.rows_per_block))), dim3(256), s, a);
  });
}

int moe_attn_workspace_size(const moe_attn_config* cfg, int64_t T, int64_t B, int64_t max_q, int64_t max_len,
                            int prefill, size_t* bytes) {
  const int st = validate_sizes(cfg, T, B, max_q, max_len, prefill);
  if (st) return st;
  if (!bytes) return MOE_MLP_ERR_NULL_ARG;
  *bytes = 0;
  if (B == 0 || (prefill && (T == 0 || max_q == 0))) return MOE_MLP_OK;   // nothing to do
  if (!prefill) {
    const DecodePlan p = decode_plan(cfg, B, max_q, max_len);
    if (p.blocks >= kMaxThreads / (ATTN_NW * 64) || p.join_blocks >= kMaxThreads / 256)
      return MOE_MLP_ERR_BAD_SHAPE;
    *bytes = p.ws_bytes;
    return MOE_MLP_OK;
  }
  return with_prefill_shape(cfg, T, B, max_q, max_len, [&](auto dc, auto nc) -> int {
    constexpr int NW = decltype(nc)::value;
    const PrefillPlan p = prefill_plan<decltype(dc)::value, NW>(cfg, T, B, max_q, max_len);
    if (p.col_blocks >= kInt32End || p.blocks >= kMaxThreads / (NW * 64) || p.join_blocks >= kMaxThreads / 256)
      return MOE_MLP_ERR_BAD_SHAPE;
    *bytes = p.ws_bytes;
    return MOE_MLP_OK;
  });
}

int moe_attn_workspace_bound(const moe_attn_config* cfg, int64_t T, int64_t B, int64_t max_q, int64_t max_len,
                             int prefill, size_t* bytes) {
  size_t need = 0;
  const int st = moe_attn_workspace_size(cfg, T, B, max_q, max_len, prefill, &need);
  if (st) return st;
  if (!bytes) return MOE_MLP_ERR_NULL_ARG;
  *bytes = 0;
  if (B == 0 || (prefill && (T == 0 || max_q == 0))) return MOE_MLP_OK;
  if (!prefill) {
    *bytes = decode_bound(cfg, B, max_q, max_len);
    return MOE_MLP_OK;
  }
  // smaller calls may take either number of wavefronts
  return with_dim(cfg->head_dim, [&](auto dc) -> int {
    constexpr int D = decltype(dc)::value;
    *bytes = prefill_plan<D, 4>(cfg, T, B, max_q, max_len).ws_bound;
    if constexpr (D == 128) *bytes = std::max(*bytes, prefill_plan<D, 8>(cfg, T, B, max_q, max_len).ws_bound);
    return MOE_MLP_OK;
  });
}

int moe_attn_decode(const moe_attn_config* cfg, const moe_attn_cache* cache, const uint16_t* q, int64_t B,
                    int64_t n_q, const int32_t* seq_lens, const int32_t* page_table, int64_t max_pages,
                    int64_t max_len, uint16_t* out, void* workspace, size_t ws_bytes, void* stream) {
  return attention(cfg, cache, q, 0, nullptr, B, n_q, seq_lens, page_table, max_pages, max_len, out, workspace,
                   ws_bytes, stream, 0);
}

int moe_attn_prefill(const moe_attn_config* cfg, const moe_attn_cache* cache, const uint16_t* q, int64_t T,
                     const int32_t* cu_q, int64_t B, int64_t max_q, const int32_t* seq_lens,
                     const int32_t* page_table, int64_t max_pages, int64_t max_len, uint16_t* out, void* workspace,
                     size_t ws_bytes, void* stream) {
  return attention(cfg, cache, q, T, cu_q, B, max_q, seq_lens, page_table, max_pages, max_len, out, workspace,
                   ws_bytes, stream, 1);
}

}  // extern "C"
