/*
 * lq_gated.h -- a gated pair of quantized projections (the first half of a
 * transformer's MLP), with adapters: h = act(g) * u with g and u two
 * projections of the same X, their activation and their product in one pass.
 * Companion of lq.h, lq_adapters.h and lq_dropout.h, whose conventions hold for
 * every entry point here.
 *
 * With W'_g, W'_u the bfloat16 dequantized weights [N, K] and a = ids[m]:
 *     g[m] = W'_g X[m] + s_a B_a t_g[m],  t_g[m] = A_a D_g[m]     (gate's set, its dropout)
 *     u[m] = W'_u X[m] + s_a B_a t_u[m],  t_u[m] = A_a D_u[m]     (up's set, its dropout)
 *     H[m] = act(g[m]) u[m]
 */
#ifndef LQ_GATED_H
#define LQ_GATED_H

#include "lq_dropout.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  LQ_SILU = 0,     /* x / (1 + e^-x) */
  LQ_GELU = 1,     /* x Phi(x), Phi the normal distribution function */
  LQ_GELU_TANH = 2 /* x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2 */
};

/* A pair of [N, K] weights, of either format each, and their adapters: two
 * sets with the same number of adapters (ranks may differ), or both NULL for
 * the weights alone. The calls read the structures on the host. */
typedef struct lq_gated {
  const lq_qweight* gate;
  const lq_qweight* up;
  const lq_adapter_set* gate_set;
  const lq_adapter_set* up_set;
  int32_t act;
} lq_gated;

/* Host check of a pair: LQ_ERR_ARG (a null weight, one set without the other,
 * bad act, and as lq_check_adapters), LQ_ERR_SHAPE (weights of different sizes,
 * sets of different n), and the weights' own errors. The calls make it too. */
int lq_check_gated(const lq_gated* p);

/* Workspace bytes of lq_gated_forward (0 for an invalid argument); drops: 1 if
 * a dropout is given. Up to 64 tokens of two NF4 weights with constants of one
 * kind (both double-quantized or neither), K <= 49152, without dropout, about
 * the size of X and t, as far as both sides' t and a workgroup's constants fit
 * the chip's shared memory: where 2 K + 6 T (r + r') <= 130560, with T the
 * tokens rounded up to 16, 32 or 64 and r, r' the sets' r_max rounded up to
 * multiples of 8 (64 tokens: any ranks up to K = 16128). Otherwise above all both
 * weights in bfloat16, 4 N K bytes. */
size_t lq_gated_forward_workspace(const lq_gated* p, int64_t M, int32_t drops);

/*
 *   X [M, K] bf16; ids [M] int32; route lq_adapter_route's of ids and the sets'
 *   n, or NULL. Without sets ids and route are NULL.
 *   drop_gate, drop_up: dropout of the adapters' input (lq_dropout.h; their
 *   element m K + k), each NULL for none; without sets both are NULL.
 *   H [M, N] of h_dtype (LQ_BF16 or LQ_F32), written: act and product are taken
 *   of the float32 g and u and rounded once.
 *   For the backward, each written if not NULL: g, u [M, N] bf16 (rounded);
 *   t_gate, t_up [M, r_max of the set] float32 as lq_adapters_forward's t_save.
 * What lq_adapters_forward says of infinite values holds for g and u. silu and
 * the gelus of an infinity or NaN are what their formulas give (silu(-inf): NaN).
 * Errors: as lq_check_gated, lq_adapters_forward, lq_adapters_forward_dropout.
 */
int lq_gated_forward(const lq_gated* p, const uint16_t* X, int64_t M, const int32_t* ids, const int32_t* route,
                     const lq_dropout* drop_gate, const lq_dropout* drop_up, void* H, int32_t h_dtype, uint16_t* g,
                     uint16_t* u, float* t_gate, float* t_up, void* workspace, size_t ws_bytes, void* stream);

/* Workspace bytes of lq_gated_backward (0 for an invalid argument): above all
 * both transposed weights (4 N K bytes, twice that for codebook weights) and
 * the gradients of g and u (4 M N). */
size_t lq_gated_backward_workspace(const lq_gated* p, int64_t M);

/*
 * Backward: with G = dL/dH and g, u of the forward,
 *     dg = G u act'(g),  du = G act(g)
 * and, with those as the gradients of the two projections, what
 * lq_adapters_backward (with dropout: lq_adapters_backward_dropout) gives for
 * each; grad_X is the sum of both.
 *   X, G, g, u bf16; t_gate, t_up as the forward writes them, or NULL: formed
 *   again from X (and the dropout). X may be NULL where nothing needs it.
 *   grad_X [M, K] bf16; dA_gate, dA_up, dB_gate, dB_up float32, laid out as
 *   lq_adapters_backward's; each may be NULL to skip it (without sets they are).
 * dg and du are formed in float32, G u first (an infinity where it passes
 * float32's range); the adapters' products take all their bits (as three
 * bfloat16 terms), grad_X's large product their bfloat16 rounding, which raises
 * the relative error of grad_X from 0.0017, its own rounding, to 0.0023.
 * Needs N % 8 == 0 (LQ_ERR_SHAPE). Sums are formed in a fixed order. Errors: as
 * lq_check_gated and lq_adapters_backward_dropout.
 */
int lq_gated_backward(const lq_gated* p, const uint16_t* X, const uint16_t* G, int64_t M, const int32_t* ids,
                      const int32_t* route, const lq_dropout* drop_gate, const lq_dropout* drop_up, const uint16_t* g,
                      const uint16_t* u, const float* t_gate, const float* t_up, uint16_t* grad_X, float* dA_gate,
                      float* dB_gate, float* dA_up, float* dB_up, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LQ_GATED_H */
