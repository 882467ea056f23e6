/*
 * moe_proj.h -- C ABI of what stands around the two halves of the decoder layer
 * (moe_attn.h, moe_mlp.h) in a server of many requests: the residual's addition
 * and the RMS norm before a half, the FP8 projection that takes the normed
 * rows, and the requests' own low-rank adapters beside such a projection.
 * Same library, same conventions as moe_mlp.h:
 *   - every pointer argument except `stream` is a DEVICE pointer; the adapter
 *     descriptor is HOST memory;
 *   - tensors are row-major, and contiguous unless a stride is an argument
 *     (strides count elements); bf16, fp32 and E4M3 tensors are 16-byte
 *     aligned, int32 arrays 4-byte aligned; bf16 values travel as uint16_t bit
 *     patterns, E4M3 ("fn": no infinities, 0x7F and 0xFF are NaN) as bytes;
 *   - the caller owns every buffer, the workspace too, whose contents need no
 *     initialisation and are garbage after a call; the library allocates,
 *     frees and synchronises nothing, and keeps no pointer;
 *   - arguments are validated on the host before anything is enqueued; on an
 *     error nothing is enqueued.  Work goes to `stream` (a hipStream_t, NULL =
 *     the default stream) of the current device and the call returns without
 *     waiting; calls can be captured into a HIP graph;
 *   - results are deterministic: no atomics, fixed summation orders.
 * Status codes are those of moe_mlp.h.  A call has T < 2^22 tokens; T == 0 is
 * a no-op returning MOE_MLP_OK.
 */
#ifndef MOE_PROJ_H
#define MOE_PROJ_H

#include <stddef.h>
#include <stdint.h>

#include "moe_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_PROJ_NORM_MAX_HIDDEN 16384  /* columns of moe_proj_norm */
#define MOE_PROJ_LORA_MAX_RANK   256    /* max_rank of moe_proj_adapters */
#define MOE_PROJ_MAX_FEATURES    (1 << 20)  /* columns of the projections, below this */

/*
 * The row between two halves of a layer:
 *   h = x + residual                                  (x alone without a residual)
 *   y = h * rsqrt(mean(h^2) + eps) * weight           (weight NULL: ones)
 * in fp32, the mean and the norm of the sum as it is before its own rounding.
 * Outputs, each of them optional (NULL) but at least one of y_out and q_out:
 *   h_out   [T, hidden] bf16: h, rounded once (nearest even);
 *   y_out   [T, hidden] bf16: y, rounded once;
 *   q_out, q_scale (both or neither): y in E4M3, q_out [T, hidden], with one
 *     scale per row and MOE_MLP_FP8_BLOCK columns, q_scale
 *     [T, ceil(hidden / 128)] fp32:
 *       scale = max(max |y| / 448, 2^-126),  q = e4m3(y / scale)  (nearest even).
 *   x       [T, hidden] bf16, rows x_stride >= hidden elements apart (a multiple of 8);
 *   residual [T, hidden] bf16 or NULL;  weight [hidden] fp32 or NULL.
 *   hidden  a multiple of 8, at most MOE_PROJ_NORM_MAX_HIDDEN.
 *   eps     finite, >= 0 (with 0, a row of zeros is 0 / 0: NaN).
 * h_out and y_out may be the buffer of x (of stride hidden) or of residual, as a
 * whole, and not each other; no other overlap of an output with another tensor is
 * allowed.  A row with a NaN is NaN in y_out and q_out; one with an infinity is NaN
 * there and 0 elsewhere (x / inf); their scales are finite.  Finite |h| up to 2^56,
 * so that the sum of their squares is finite; with eps below 2^-100 that sum has to be
 * 2^-100 at least, or the row one of zeros.
 */
int moe_proj_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual, const float* weight, float eps,
                  int64_t T, int64_t hidden, uint16_t* h_out, uint16_t* y_out, uint8_t* q_out, float* q_scale,
                  void* stream);

/*
 * Projection of E4M3 rows by E4M3 weights, one fp32 scale per row and 128
 * columns of x (moe_proj_norm) and per 128 x 128 block of w (the format of the
 * FP8 experts of moe_mlp.h):
 *   y[t][n] = sum_k x[t][k] x_scale[t][k / 128] w[n][k] w_scale[n / 128][k / 128]
 * in fp32 and one rounding to bf16, on the matrix unit's E4M3 products: it adds
 * them in groups of 8 columns, each cut to 13 bits below the largest of its group
 * (7 * 2^-13 of that largest product at most, for a group), and everything after
 * that in fp32.
 *   x       [T, K] E4M3;  x_scale [T, K / 128] fp32;
 *   w       [N, K] E4M3;  w_scale [ceil(N / 128), K / 128] fp32;
 *   y       [T, N] bf16.
 *   K a multiple of 128, N of 16, both below MOE_PROJ_MAX_FEATURES;  T * N < 2^32.
 * A product of two scales that meet has to be a normal fp32 number, or 0.
 */
int moe_proj_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale, int64_t T, int64_t N,
                 int64_t K, uint16_t* y, void* stream);

/* Low-rank adapters of one projection of in_features to out_features. */
typedef struct moe_proj_adapters {
  const uint16_t* a;       /* [n_adapters, max_rank, in_features] bf16 */
  const uint16_t* b;       /* [n_adapters, out_features, max_rank] bf16 */
  const int32_t*  ranks;   /* [n_adapters] int32, clamped to 0 .. max_rank: what a and b hold past it does
                              not matter (NaN too); NULL: max_rank, all of them */
  const float*    scales;  /* [n_adapters] fp32; NULL: ones */
  int64_t n_adapters;      /* 1 .. 2^20; with 512 or more, however many a call uses, long calls in mixed order read
                              adapters again for every 64 tokens: 4096 tokens of 50 adapters of rank 32, 4096 columns
                              to 4096, 55 us with 511 adapters here and 234 us with 512 (in runs 76 us) */
  int32_t max_rank;        /* a multiple of 8 up to MOE_PROJ_LORA_MAX_RANK */
  int32_t in_features;     /* a multiple of 8 below MOE_PROJ_MAX_FEATURES */
  int32_t out_features;    /* a multiple of 8 below MOE_PROJ_MAX_FEATURES */
} moe_proj_adapters;

/* Workspace bytes of moe_proj_lora for T tokens, or fewer.  `bytes` is a HOST pointer. */
int moe_proj_lora_workspace_size(const moe_proj_adapters* adapters, int64_t T, size_t* bytes);

/*
 * Each token's own adapter beside the shared projection that gave `base`:
 *   out[t] = base[t] + scales[a] * (x[t] A_a^T) B_a^T,   a = adapter[t]
 *   out[t] = base[t]                                      where adapter[t] is not in 0 .. n_adapters - 1
 * with fp32 sums, the inner row x A^T kept to 16 bits of mantissa, and one
 * rounding to bf16; what is not finite is as in fp32.
 *   x       [T, in_features] bf16, rows x_stride apart;
 *   adapter [T] int32;
 *   base    [T, out_features] bf16, rows base_stride apart;
 *   out     [T, out_features] bf16, rows out_stride apart: may be base (the same
 *           buffer and stride); no other overlap.  Rows of base and out may be
 *           columns of a wider tensor (the queries' part of a fused projection).
 *   Strides: multiples of 8, at least the row's length, below 2^31.
 * Tokens may come in any order; those of a request one after the other are the
 * fastest.  x of a token without an adapter is not read.
 */
int moe_proj_lora(const moe_proj_adapters* adapters, const uint16_t* x, int64_t x_stride, int64_t T,
                  const int32_t* adapter, const uint16_t* base, int64_t base_stride, uint16_t* out,
                  int64_t out_stride, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_PROJ_H */
