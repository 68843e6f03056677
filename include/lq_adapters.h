/*
 * lq_adapters.h -- many low-rank adapters over one frozen quantized
 * projection, and the clipping of their gradients. Companion of lq.h, whose
 * conventions (device pointers owned by the caller, caller workspaces, status
 * codes, validation before any launch, asynchronous on `stream`) hold for
 * every entry point here.
 *
 * The layer equation is the QLoRA page's (introduction) with an adapter per
 * token: with W' the bfloat16 dequantized weight and a = ids[m],
 *     t[m] = A_a X[m]
 *     H[m] = W' X[m] + s_a B_a t[m],   s_a = alpha_a / r_a,
 * and H[m] = W' X[m] for a token without an adapter (an id outside [0, n)).
 * Only the adapters get gradients.
 */
#ifndef LQ_ADAPTERS_H
#define LQ_ADAPTERS_H

#include "lq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LQ_ADAPTERS_MAX 1000 /* adapters in one set */

/* One adapter: A [r, K], B [N, r] bfloat16, row-major, 16-byte aligned device
 * pointers; r in 1..128; scale = alpha / r. row and row8 are the sums of the
 * ranks, and of the ranks rounded up to a multiple of 8, of the adapters
 * before it in its set. */
typedef struct lq_adapter {
  const uint16_t* A;
  const uint16_t* B;
  int32_t r;
  float scale;
  int32_t row;
  int32_t row8;
} lq_adapter;

/* A set of n adapters of one [N, K] projection: the same entries in a host
 * array (read by the calls for validation and sizes) and in device memory
 * (read by the kernels, 8-byte aligned). r_max is the largest rank. The
 * device copy's equality with the host array is the caller's. */
typedef struct lq_adapter_set {
  const lq_adapter* host;
  const lq_adapter* dev;
  int32_t n;
  int32_t r_max;
} lq_adapter_set;

/*
 * Host check of a set against an [N, K] weight. LQ_ERR_ARG: a null or
 * misaligned pointer, r_max not the largest rank, row / row8 not the running
 * sums; LQ_ERR_SHAPE: n outside [1, LQ_ADAPTERS_MAX], a rank outside [1, 128],
 * N or K <= 0. Pure host function; the calls below make the same check.
 */
int lq_check_adapters(const lq_adapter_set* set, int64_t N, int64_t K);

/* Bytes of the route of M tokens over n adapters (0 for an invalid size). */
size_t lq_adapter_route_bytes(int64_t M, int32_t n);

/*
 * Sorts the tokens by adapter, stably (equal ids stay in token order; tokens
 * without an adapter come last). A route depends on ids alone, so one serves
 * every projection of a step whose sets have n adapters.
 *   ids    [M] int32, read: the adapter of each token; outside [0, n) = none
 *   route  lq_adapter_route_bytes(M, n) bytes, 16-byte aligned, written (int32):
 *          off [n + 2] first sorted position of each adapter, then of the
 *          tokens without one, then M; perm [M] token of each sorted position;
 *          sid [M] adapter of each sorted position (n = none)
 * Errors: LQ_ERR_ARG, LQ_ERR_SHAPE (M outside [1, 2^31), n outside
 * [1, LQ_ADAPTERS_MAX]), LQ_ERR_WORKSPACE (bytes too few), LQ_ERR_LAUNCH.
 */
int lq_adapter_route(const int32_t* ids, int64_t M, int32_t n, int32_t* route, size_t bytes, void* stream);

/* Workspace bytes of lq_adapters_forward (0 for an invalid argument): up to 64
 * tokens of an NF4 weight with K <= 49152 about the size of X and t; otherwise
 * above all the weight in bfloat16, 2 N K bytes. */
size_t lq_adapters_forward_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set);

/*
 * Forward of M tokens, each with its own adapter.
 *   X      [M, K] bf16;  ids [M] int32 (4-byte aligned)
 *   route  lq_adapter_route's output for these ids (so this M) and set->n, or
 *          NULL: built in the workspace when the call needs it. Its contents
 *          are not checked: one of another M or n sends the kernels out of range
 *   H      [M, N] of h_dtype (LQ_BF16 or LQ_F32), written
 *   t_save [M, r_max] float32, written if not NULL: t in its token's first r_a
 *          columns, 0 in the others and for tokens without an adapter
 * An adapter's values and its scale reach only its own tokens' outputs, also
 * where they are infinite or NaN. An infinite t gives infinities by the
 * equation; t's products with an infinite B are formed in parts, and give an
 * infinity or NaN (likewise in the backward: an infinite u, and the infinities
 * of A in grad_X, of X in dA, of G in dB). Errors: as lq_qlora_forward and lq_check_adapters.
 */
int lq_adapters_forward(const lq_qweight* w, const uint16_t* X, int64_t M, const lq_adapter_set* set,
                        const int32_t* ids, const int32_t* route, void* H, int32_t h_dtype, float* t_save,
                        void* workspace, size_t ws_bytes, void* stream);

/* Workspace bytes of lq_adapters_backward (0 for an invalid argument): above all
 * the transposed weight in bfloat16, 2 N K bytes, twice that for a codebook
 * weight. */
size_t lq_adapters_backward_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set);

/*
 * Backward: with G = dL/dH, a = ids[m] and u[m] = B_a^T G[m],
 *     grad_X[m] = W'^T G[m] + s_a A_a^T u[m]      (no second term without an adapter)
 *     dA_a = s_a sum over a's tokens of u[m] X[m]^T
 *     dB_a = s_a sum over a's tokens of G[m] t[m]^T
 *   X [M, K] bf16 (read for dA, and for t when t_saved is NULL and dB is wanted);
 *   G [M, N] bf16; t_saved [M, r_max] float32 as the forward writes it, or NULL
 *   grad_X [M, K] bf16; dA [sum of ranks, K] float32, adapter a's rows from
 *   row_a; dB float32, adapter a's [N, r_a] block from element N * row_a.
 *   Each of grad_X, dA and dB may be NULL to skip it. An adapter without
 *   tokens gets zero gradients.
 * Needs N % 8 == 0 (LQ_ERR_SHAPE). Sums are formed in a fixed order, so
 * results repeat exactly. Errors: as lq_qlora_backward and lq_check_adapters.
 */
int lq_adapters_backward(const lq_qweight* w, const uint16_t* X, const uint16_t* G, int64_t M,
                         const lq_adapter_set* set, const int32_t* ids, const int32_t* route, const float* t_saved,
                         uint16_t* grad_X, float* dA, float* dB, void* workspace, size_t ws_bytes, void* stream);

/* ---- gradient norms and clipping ------------------------------------------- */

/* One gradient tensor: `numel` contiguous elements of `dtype` (LQ_F32,
 * LQ_BF16, LQ_F16) at `data` (aligned to the element), counted in the norm of
 * `group` (0 .. n_groups - 1: for instance one group per fine-tuning job). */
typedef struct lq_grad_tensor {
  void* data;
  int64_t numel;
  int32_t dtype;
  int32_t group;
} lq_grad_tensor;

/* A list of gradient tensors prepared for the kernels. `dev` is the device
 * copy of the table that lq_grad_list_build wrote (16-byte aligned); `digest`
 * stands for the tensors' sizes, types and groups. */
typedef struct lq_grad_list {
  const void* dev;
  int64_t n_pieces;
  int32_t n_slots;
  int32_t n_groups;
  uint64_t digest;
} lq_grad_list;

/* Bytes of the table of a list (0 for an invalid argument). Host function. */
size_t lq_grad_list_bytes(const lq_grad_tensor* tensors, int64_t n, int32_t n_groups);

/*
 * Writes the table into host memory and fills *list except list->dev: the
 * caller copies the table to the device and sets dev. Tensors may be in any
 * order of groups; empty tensors and groups without tensors are allowed (norm
 * 0). Host function. Errors: LQ_ERR_ARG (null or misaligned data of a
 * non-empty tensor, bad dtype or group), LQ_ERR_SHAPE (n < 0, numel < 0,
 * n_groups outside 1 .. 65535, too many elements), LQ_ERR_WORKSPACE.
 */
int lq_grad_list_build(const lq_grad_tensor* tensors, int64_t n, int32_t n_groups, void* table, size_t bytes,
                       lq_grad_list* list);

/* Workspace bytes of lq_grad_norm and lq_clip_grad_norm. */
size_t lq_grad_norm_workspace(const lq_grad_list* list);

/*
 * norms[g] = sqrt(sum of x^2 over the tensors of group g): squares and sums in
 * float64 in a fixed order, rounded to float32 once. A NaN gives NaN, else an
 * infinity gives infinity.
 *   norms [n_groups] float32, written
 */
int lq_grad_norm(const lq_grad_list* list, float* norms, void* workspace, size_t ws_bytes, void* stream);

/*
 * The norms, and out = x * min(1, max_norm / (norm_g + eps)) for every element
 * (the factor in float32; the product rounded once to the tensor's type). A
 * NaN norm gives a NaN factor; an infinite one the factor 0. `out` has the
 * sizes, types and groups of `in` (equal digests, else LQ_ERR_ARG); it may be
 * `in` itself, but must not overlap it otherwise.
 *   max_norm >= 0, eps > 0, both finite (LQ_ERR_ARG)
 * Errors: LQ_ERR_ARG, LQ_ERR_WORKSPACE, LQ_ERR_LAUNCH.
 */
int lq_clip_grad_norm(const lq_grad_list* in, const lq_grad_list* out, float max_norm, float eps, float* norms,
                      void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LQ_ADAPTERS_H */
