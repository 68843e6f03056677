// Dropout of a tensor, its mask formed from a counter (include/lq_dropout.h):
//   out = kept(seed, step, site, element) ? x * 65536 / (65536 - T) : 0
//
// A thread owns whole generator blocks (8 elements), DROP_U of them in flight,
// the loads asked for before the rounds of the generator, which run while they
// travel. Bound by memory for large tensors: 4096 x 11008 bfloat16, 37 us, that is
// 4.9 TB/s, where a copy of 1 GiB reaches 5.05. Small ones are bound by the launch:
// 300 x 1021 float16, 3 us.
#include "lq_dropout.h"
#include "lq_route.h"

namespace lq {
namespace {

constexpr int DROP_THREADS = 256, DROP_U = 2;

template <int DT>
struct Elem;
template <>
struct Elem<LQ_F32> {
  typedef float type;
  static __device__ __forceinline__ float mul(float x, float f) { return x * f; }
};
template <>
struct Elem<LQ_BF16> {
  typedef uint16_t type;
  static __device__ __forceinline__ uint16_t mul(uint16_t x, float f) {
    return (uint16_t)(pack_bf16x2(bf16_to_f32(x) * f, 0.0f) & 0xFFFFu);
  }
};
template <>
struct Elem<LQ_F16> {
  typedef _Float16 type;
  static __device__ __forceinline__ _Float16 mul(_Float16 x, float f) { return (_Float16)((float)x * f); }
};

// VEC: x and out are 16-byte aligned; otherwise element by element. A kept
// element is multiplied in float32 and rounded once to its type.
template <int DT, bool VEC>
__global__ __launch_bounds__(DROP_THREADS) void k_dropout(DropView d, float factor, const void* x_, int64_t numel, void* out_) {
  typedef typename Elem<DT>::type T;
  typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
  constexpr int V = 16 / sizeof(T), P = 8 / V;   // elements a vector, vectors a block
  const T* x = reinterpret_cast<const T*>(x_);
  T* out = reinterpret_cast<T*>(out_);
  const DropGen g = drop_gen(d);
  const int64_t whole = numel / 8, blocks = (numel + 7) / 8;
  for (int64_t i0 = (int64_t)blockIdx.x * (DROP_THREADS * DROP_U) + threadIdx.x; i0 < blocks;
       i0 += (int64_t)gridDim.x * (DROP_THREADS * DROP_U)) {
    if constexpr (VEC) {
      u32x4_t v[DROP_U][P];
#pragma unroll
      for (int u = 0; u < DROP_U; ++u) {
        const int64_t i = i0 + u * DROP_THREADS;
        if (i < whole)
#pragma unroll
          for (int p = 0; p < P; ++p) v[u][p] = ld16(x + 8 * i + V * p);
      }
#pragma unroll
      for (int u = 0; u < DROP_U; ++u) {
        const int64_t i = i0 + u * DROP_THREADS;
        if (i >= whole) continue;
        const u32x4_t bits = drop_bits(g, (uint64_t)i);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          vec e = __builtin_bit_cast(vec, v[u][p]);
#pragma unroll
          for (int k = 0; k < V; ++k) e[k] = drop_keeps(bits, V * p + k, d.T) ? Elem<DT>::mul(e[k], factor) : T(0);
          *reinterpret_cast<u32x4_t*>(out + 8 * i + V * p) = __builtin_bit_cast(u32x4_t, e);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < DROP_U; ++u) {   // what the vectors leave: nothing but the last, partial block where VEC
      const int64_t i = i0 + u * DROP_THREADS;
      if (i >= blocks || (VEC && i < whole)) continue;
      const u32x4_t bits = drop_bits(g, (uint64_t)i);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (8 * i + k < numel) out[8 * i + k] = drop_keeps(bits, k, d.T) ? Elem<DT>::mul(x[8 * i + k], factor) : T(0);
    }
  }
}

template <int DT>
void launch(const DropView& d, float factor, const void* x, int64_t numel, void* out, bool vec, dim3 grid, hipStream_t s) {
  if (vec) hipLaunchKernelGGL((k_dropout<DT, true>), grid, dim3(DROP_THREADS), 0, s, d, factor, x, numel, out);
  else hipLaunchKernelGGL((k_dropout<DT, false>), grid, dim3(DROP_THREADS), 0, s, d, factor, x, numel, out);
}

}  // namespace

hipError_t launch_dropout(const DropView& d, float factor, const void* x, int64_t numel, int dtype, void* out,
                          hipStream_t s) {
  const int64_t per = 8 * DROP_THREADS * DROP_U, most = 1 << 20;   // past 2^32 elements a workgroup takes several shares
  const int64_t grid = (numel + per - 1) / per < most ? (numel + per - 1) / per : most;
  const bool vec = (((uintptr_t)x | (uintptr_t)out) & 15) == 0;
  const dim3 g((unsigned)grid);
  if (dtype == LQ_F32) launch<LQ_F32>(d, factor, x, numel, out, vec, g, s);
  else if (dtype == LQ_BF16) launch<LQ_BF16>(d, factor, x, numel, out, vec, g, s);
  else launch<LQ_F16>(d, factor, x, numel, out, vec, g, s);
  return hipGetLastError();
}

}  // namespace lq
