// What the attention kernels share: arguments, a sequence's lengths, the
// visible keys of a query, and addresses inside the paged cache.
//
// Cache layout (include/moe_attn.h): K [page][head][dim / 8][token][8] and
// V [page][head][token / 8][dim][8], 16 bytes = 8 values along the reduction
// of the product that reads them.
#pragma once

#include "common.hpp"

namespace moe {

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
  float scale_log2;           // scale * log2(e): the softmax runs on exp2
};

// New tokens of a sequence (rows row0 .. row0 + n of q) and its length.
struct AttnSeq {
  int64_t row0;
  int n, len;
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b) {
  AttnSeq s;
  s.len = min(max(a.seq_lens[b], 0), a.max_len);
  if (a.cu_q) {
    const int64_t r0 = min(max(static_cast<int64_t>(a.cu_q[b]), int64_t(0)), a.T);
    const int64_t r1 = min(max(static_cast<int64_t>(a.cu_q[b + 1]), r0), a.T);
    s.row0 = r0;
    s.n = static_cast<int>(min(r1 - r0, static_cast<int64_t>(a.n_q)));
  } else {
    s.row0 = static_cast<int64_t>(b) * a.n_q;
    s.n = a.n_q;
  }
  return s;
}

// First key of the window of position p (0 without a window).
__device__ __forceinline__ int attn_window_lo(const AttnArgs& a, int p) {
  return a.window ? max(0, p - a.window + 1) : 0;
}

__device__ __forceinline__ bool attn_visible(int key, int p, int lo, int sinks) {
  return key <= p && (key >= lo || key < sinks);
}

}  // namespace moe
