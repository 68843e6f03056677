// The dropout generator (include/lq_dropout.h) as the kernels and the host use it.
#pragma once

#include "../../include/lq_dropout.h"
#include "lq_device.h"
#include "lq_internal.h"

namespace lq {

// What a kernel gets. T == 0: nothing is dropped (key may be null).
struct DropView {
  const uint64_t* key;
  uint32_t T;
  uint32_t site;
};

// Checks d (null: no dropout) and fills the view and the kept elements' factor.
inline int drop_view(const lq_dropout* d, DropView* v, float* factor) {
  *v = DropView{nullptr, 0, 0};
  *factor = 1.0f;
  if (!d) return LQ_OK;
  if (!d->key || ((uintptr_t)d->key & 7) || !(d->p >= 0.0) || !(d->p < 1.0) || d->site >= LQ_DROPOUT_SITES)
    return LQ_ERR_ARG;
  const uint32_t T = (uint32_t)__builtin_rint(d->p * 65536.0);
  v->key = d->key;
  v->T = T < 65535u ? T : 65535u;
  v->site = d->site;
  *factor = (float)(65536.0 / (65536.0 - v->T));
  return LQ_OK;
}

hipError_t launch_dropout(const DropView& d, float factor, const void* x, int64_t numel, int dtype, void* out,
                          hipStream_t s);

// The generator's words that every block shares, in scalar registers.
struct DropGen {
  uint32_t k0, k1, step0, step1, site;
};
__device__ __forceinline__ uint32_t drop_uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ __forceinline__ DropGen drop_gen(const DropView& d) {
  const uint64_t seed = d.key[0], step = d.key[1];
  return DropGen{drop_uniform((uint32_t)seed), drop_uniform((uint32_t)(seed >> 32)), drop_uniform((uint32_t)step),
                 drop_uniform((uint32_t)(step >> 32)), d.site * 4096u};
}

// The eight 16-bit fields of block i. A round is two 32 x 32 -> 64 bit products
// (quarter rate) and two three-way exclusive ors; the round keys are uniform.
__device__ __forceinline__ u32x4_t drop_bits(const DropGen& g, uint64_t i) {
  uint32_t c0 = (uint32_t)i, c1 = (uint32_t)(i >> 32) + g.site, c2 = g.step0, c3 = g.step1;
  uint32_t k0 = g.k0, k1 = g.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = __builtin_amdgcn_bitop3_b32((uint32_t)(b >> 32), c1, k0, 0x96);   // 0x96: the exclusive or of three
    c1 = (uint32_t)b;
    c2 = __builtin_amdgcn_bitop3_b32((uint32_t)(a >> 32), c3, k1, 0x96);
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{c0, c1, c2, c3};
}

// Eight 16-bit elements with the dropped ones zeroed (T >= 1): the field less
// T - 1, saturated at 0 and 1, is 1 where the element stays, and the bit
// pattern times 0 or 1 a selection: three packed operations for two elements.
__device__ __forceinline__ u32x4_t drop_16bit(u32x4_t x, u32x4_t bits, uint32_t T) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  const uint16_t below = (uint16_t)(T - 1);
  const u16x2_t b = {below, below}, one = {1, 1};
  u32x4_t o;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t bw = bits[w], xw = x[w];   // (a bit cast of a vector's element itself takes the first one's bits)
    const u16x2_t kept = __builtin_elementwise_min(__builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2_t, bw), b), one);
    const u16x2_t left = __builtin_bit_cast(u16x2_t, xw) * kept;
    o[w] = __builtin_bit_cast(uint32_t, left);
  }
  return o;
}
// Whether element j of the block stays.
__device__ __forceinline__ bool drop_keeps(u32x4_t bits, int j, uint32_t T) {
  return ((bits[j >> 1] >> (16 * (j & 1))) & 0xFFFFu) >= T;
}

}  // namespace lq
