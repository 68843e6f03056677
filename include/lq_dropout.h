/*
 * lq_dropout.h -- dropout whose mask is a function of a counter and stored
 * nowhere: applied to a tensor, and inside the many-adapter forward and
 * backward (dropout of the adapters' input). Companion of lq.h and
 * lq_adapters.h, whose conventions hold for every entry point here.
 *
 * The random bits come from Philox 4x32 with ten rounds (Salmon, Moraes, Dror,
 * Shaw: "Parallel random numbers: as easy as 1, 2, 3", SC 2011). Elements
 * 8 i .. 8 i + 7 of a row-major tensor share the block with the counter words
 *     low 32 bits of i;  site * 4096 + the bits of i above;  step, low word;  step, high word
 * and the key (low word of seed, high word of seed). Element 8 i + j takes the
 * 16 bits of half j % 2 (0: low) of output word j / 2 and is dropped where they
 * are below T = round(65536 p) (ties to even, at most 65535); a kept element is multiplied
 * by 65536 / (65536 - T). So p counts in steps of 2^-16, and the mean of a kept
 * or dropped element is the element itself.
 */
#ifndef LQ_DROPOUT_H
#define LQ_DROPOUT_H

#include "lq_adapters.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LQ_DROPOUT_SITES (1 << 20)

/* key: two uint64 in device memory (8-byte aligned), seed and step, read when
 * the kernels run: a captured graph whose step is advanced between replays
 * draws a new mask each time. A forward and its backward must find the same
 * two values there. site (0 .. LQ_DROPOUT_SITES - 1) tells the places of a
 * model apart that share a key. p in [0, 1). */
typedef struct lq_dropout {
  const uint64_t* key;
  double p;
  uint32_t site;
} lq_dropout;

/*
 * out = dropout(x), elements of dtype (LQ_F32, LQ_BF16, LQ_F16; pointers
 * aligned to the element); a dropped element is +0 whatever it was, a kept one
 * is multiplied in float32 and rounded once. The gradient of x is the same call
 * on the gradient of out. out may be x itself, but must not overlap it
 * otherwise. numel 0 .. 2^47 - 1; nothing is launched for 0.
 * Errors: LQ_ERR_ARG (null or misaligned pointer, p outside [0, 1), a site too
 * large, bad dtype), LQ_ERR_SHAPE (numel), LQ_ERR_LAUNCH.
 */
int lq_dropout_apply(const lq_dropout* d, const void* x, int64_t numel, int32_t dtype, void* out, void* stream);

/*
 * lq_adapters_forward with dropout before the adapters:
 *     D = dropout(X) (element m K + k of X),  t[m] = A_a D[m],  H[m] = W' X[m] + s_a B_a t[m]
 * D is not rounded: kept elements of X enter the products as they are and the
 * factor multiplies their float32 sum. t_save holds t with its factor. With
 * p = 0 (also: p below 2^-17) t is lq_adapters_forward's for sizes that run
 * alike. M K below 2^47 (LQ_ERR_SHAPE). Other arguments and errors as there.
 */
size_t lq_adapters_forward_dropout_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set);
int lq_adapters_forward_dropout(const lq_qweight* w, const uint16_t* X, int64_t M, const lq_adapter_set* set,
                                const int32_t* ids, const int32_t* route, const lq_dropout* d, void* H,
                                int32_t h_dtype, float* t_save, void* workspace, size_t ws_bytes, void* stream);

/*
 * lq_adapters_backward of that forward:
 *     grad_X[m] = W'^T G[m] + dropout(s_a A_a^T u[m]),
 *     dA_a = s_a sum u[m] D[m]^T,  dB_a = s_a sum G[m] t[m]^T
 * t_saved: the forward's t, its factor included, or NULL. The mask of grad_X
 * leaves exact zeros of the adapter's part, also where that is infinite or NaN.
 */
size_t lq_adapters_backward_dropout_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set);
int lq_adapters_backward_dropout(const lq_qweight* w, const uint16_t* X, const uint16_t* G, int64_t M,
                                 const lq_adapter_set* set, const int32_t* ids, const int32_t* route,
                                 const lq_dropout* d, const float* t_saved, uint16_t* grad_X, float* dA, float* dB,
                                 void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LQ_DROPOUT_H */
