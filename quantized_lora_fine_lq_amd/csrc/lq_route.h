// Device helpers of the kernels that work on routed tokens: loads, the runs of one
// adapter's tokens, fragments read transposed from LDS, a barrier.
#pragma once

#include "lq_device.h"

namespace lq {

__device__ __forceinline__ u32x4_t ld16(const void* p) { return *reinterpret_cast<const u32x4_t*>(p); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
// Memory to LDS, 16 bytes a lane: lane i's 16 bytes land at dst + 16 i.
__device__ __forceinline__ void load_lds16(const uint16_t* src, uint16_t* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// Item b of the segments [off[a], off[a + 1]), a < nseg, cut into pieces of
// `rows` sorted positions: its segment, first position and row count. With
// slot: the index of the piece among those of segments with more than one, or
// -1. Every wave finds the item for itself (uniform results); false past the
// last item.
struct Item {
  int seg, start, count, slot;
};
__device__ __forceinline__ bool find_item(const int32_t* __restrict__ off, int nseg, int rows, int b, Item& it) {
  const int lane = threadIdx.x & 63;
  int base = 0, sbase = 0;
  for (int a0 = 0; a0 < nseg; a0 += 64) {
    const int a = a0 + lane;
    int lo = 0, len = 0;
    if (a < nseg) {
      lo = off[a];
      len = off[a + 1] - lo;
    }
    const int c = (len + rows - 1) / rows, cs = c > 1 ? c : 0;
    int inc = c, incs = cs;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(inc, d), os = __shfl_up(incs, d);
      if (lane >= d) {
        inc += o;
        incs += os;
      }
    }
    const int first = base + inc - c;
    const uint64_t hit = __ballot(b >= first && b < first + c);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int k = b - __shfl(first, l);
      const int s = __shfl(lo, l) + k * rows;
      const int e = __shfl(lo + len, l);
      const int sl = __shfl(cs > 0 ? sbase + incs - cs : -1, l);
      it.seg = uniform(a0 + l);
      it.start = uniform(s);
      it.count = uniform(min(rows, e - s));
      it.slot = uniform(sl < 0 ? -1 : sl + k);
      return true;
    }
    base += uniform(__shfl(inc, 63));
    sbase += uniform(__shfl(incs, 63));
  }
  return false;
}

// lane's 8 values k = 8 lg + [0, 8) of column li, from rows of `pitch` elements
__device__ __forceinline__ u32x4_t tr_frag(const uint16_t* base, int pitch, int li, int lg) {
  typedef __bf16 v4b __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) v4b* lds_p;
  const uint16_t* p = base + (8 * lg + (li >> 2)) * pitch + 4 * (li & 3);
  const u32x2_t lo = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_p)p));
  const u32x2_t hi = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_p)(p + 4 * pitch)));
  return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

// LDS written before it is there for everyone after it; loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

}  // namespace lq
