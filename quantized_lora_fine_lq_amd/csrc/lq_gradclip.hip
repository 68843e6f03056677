// Gradient norms over many tensors and the clipping of the gradients.
//
//   norm_g = sqrt(sum x^2 over group g),  out = x * min(1, max_norm / (norm_g + eps))
//
// The host cuts every tensor into pieces (one wave's work) and packs
// consecutive pieces of one group into slots (one workgroup's), see
// lq_grad_list_build. Squares are summed in float64: a float32 square over- or
// underflows for |x| outside about 1e-19 .. 1e19, and float64 has room for any
// float32 gradient; the additions are few against the memory traffic that
// bounds both passes. All sums run in a fixed order.
//
// The squares of a group must all be known before its first product, so large
// gradients are read twice: two launches, the second from the last slot to the
// first, which finds some of what the first read last in the 256 MB cache.
// Every workgroup of the second adds its group's slot sums itself (a third
// launch would cost about as much as they do). 16-byte vectors, eight in flight
// per lane. Measured, float32 from one list to another: 640 MB (1792 tensors in
// 4 groups) 141 + 246 us, 4.6 and 5.2 TB/s; 5 MB 4.1 + 6.4 us, latency; 19.6 MB
// of bfloat16 at odd addresses, alike in both lists, 6 to 8 + 9 to 10 us. Tensors
// that lie differently to 16 bytes in the two lists go element by element, one
// load a lane in flight: a call over the 640 MB takes 549 us for 386, over
// 19.6 MB of bfloat16 30 for 15.
#include "lq_adapters.h"
#include "lq_device.h"

namespace lq {
namespace {

constexpr int GW = kGradThreads / 64;

// Element types: load and store of one element and of a 16-byte vector of V.
struct ElemF32 {
  typedef float type;
  static constexpr int V = 4;
  static __device__ __forceinline__ float get(type v) { return v; }
  static __device__ __forceinline__ type put(float v) { return v; }
  static __device__ __forceinline__ void unpack(u32x4_t w, float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]);
  }
  static __device__ __forceinline__ u32x4_t pack(const float (&x)[4]) {
    return u32x4_t{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
  }
};
struct ElemBF16 {
  typedef uint16_t type;
  static constexpr int V = 8;
  static __device__ __forceinline__ float get(type v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ type put(float v) { return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu); }
  static __device__ __forceinline__ void unpack(u32x4_t w, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = bf16lo_to_f32(w[e]);
      x[2 * e + 1] = bf16hi_to_f32(w[e]);
    }
  }
  static __device__ __forceinline__ u32x4_t pack(const float (&x)[8]) {
    return u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  }
};
struct ElemF16 {
  typedef _Float16 type;
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  static constexpr int V = 8;
  static __device__ __forceinline__ float get(type v) { return (float)v; }
  static __device__ __forceinline__ type put(float v) { return (_Float16)v; }
  static __device__ __forceinline__ void unpack(u32x4_t w, float (&x)[8]) {
    const v8 h = __builtin_bit_cast(v8, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)h[e];
  }
  static __device__ __forceinline__ u32x4_t pack(const float (&x)[8]) {
    v8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (_Float16)x[e];
    return __builtin_bit_cast(u32x4_t, h);
  }
};

// A piece is read in 16-byte vectors from its first aligned element on; the
// few elements before and after go one by one. UN vectors of a lane are in
// flight together (a lane past the end reads the last vector again).
constexpr int UN = 8;

template <class E>
__device__ __forceinline__ int head_elems(const void* p, int count) {
  return min(count, (int)(((16 - ((uintptr_t)p & 15)) & 15) / sizeof(typename E::type)));
}

template <class E>
__device__ __forceinline__ double piece_squares(const GradPiece& pc, int lane) {
  const typename E::type* p = reinterpret_cast<const typename E::type*>(pc.data);
  const int head = head_elems<E>(p, pc.count), nv = (pc.count - head) / E::V, tail = head + nv * E::V;
  double acc = 0.0;
  auto one = [&](int i) {
    const double x = (double)E::get(p[i]);
    acc = __builtin_fma(x, x, acc);
  };
  if (lane < head) one(lane);
  if (tail + lane < pc.count) one(tail + lane);   // fewer than V elements
  const u32x4_t* v = reinterpret_cast<const u32x4_t*>(p + head);
  double accs[2] = {0.0, 0.0};                    // two chains of dependent additions
  for (int i = 0; i < nv; i += 64 * UN) {
    u32x4_t w[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) w[u] = v[min(i + 64 * u + lane, nv - 1)];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      float x[E::V];
      E::unpack(w[u], x);
      if (i + 64 * u + lane < nv) {
#pragma unroll
        for (int e = 0; e < E::V; ++e) {
          const double d = (double)x[e];
          accs[e & 1] = __builtin_fma(d, d, accs[e & 1]);
        }
      }
    }
  }
  return acc + (accs[0] + accs[1]);
}

template <class E>
__device__ __forceinline__ void piece_scale(const GradPiece& pi, const GradPiece& po, float coef, int lane) {
  typedef typename E::type T;
  const T* p = reinterpret_cast<const T*>(pi.data);
  T* o = reinterpret_cast<T*>(po.data);
  const int n = min(pi.count, po.count);
  if (((uintptr_t)p ^ (uintptr_t)o) & 15) {   // no common 16-byte boundary
    for (int i = lane; i < n; i += 64) o[i] = E::put(E::get(p[i]) * coef);
    return;
  }
  const int head = head_elems<E>(p, n), nv = (n - head) / E::V, tail = head + nv * E::V;
  if (lane < head) o[lane] = E::put(E::get(p[lane]) * coef);
  if (tail + lane < n) o[tail + lane] = E::put(E::get(p[tail + lane]) * coef);
  const u32x4_t* v = reinterpret_cast<const u32x4_t*>(p + head);
  u32x4_t* ov = reinterpret_cast<u32x4_t*>(o + head);
  for (int i = 0; i < nv; i += 64 * UN) {
    u32x4_t w[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) w[u] = v[min(i + 64 * u + lane, nv - 1)];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      float x[E::V];
      E::unpack(w[u], x);
#pragma unroll
      for (int e = 0; e < E::V; ++e) x[e] *= coef;
      if (i + 64 * u + lane < nv) ov[i + 64 * u + lane] = E::pack(x);
    }
  }
}

// Sum over the workgroup in a fixed order (thread 0 returns it).
__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < GW; ++w) s += sh[w];
  return s;
}

__global__ __launch_bounds__(kGradThreads) void k_grad_squares(const GradSlot* __restrict__ slots,
                                                               const GradPiece* __restrict__ pieces,
                                                               double* __restrict__ part) {
  __shared__ double sh[GW];
  const GradSlot sl = slots[blockIdx.x];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  double acc = 0.0;
  for (int k = wave; k < sl.count; k += GW) {
    const GradPiece pc = pieces[sl.first + k];
    if (pc.dtype == LQ_F32) acc += piece_squares<ElemF32>(pc, lane);
    else if (pc.dtype == LQ_BF16) acc += piece_squares<ElemBF16>(pc, lane);
    else acc += piece_squares<ElemF16>(pc, lane);
  }
  const double s = block_sum(acc, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm of the slot's group from the slots' sums, the same in every thread.
__device__ __forceinline__ float group_norm(const GradSlot& sl, const double* __restrict__ part, double* sh) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < sl.group_count; i += kGradThreads) acc += part[sl.group_first + i];
  return (float)__builtin_sqrt(block_sum(acc, sh));
}

__global__ __launch_bounds__(kGradThreads) void k_grad_norms(const GradSlot* __restrict__ slots,
                                                             const double* __restrict__ part,
                                                             float* __restrict__ norms) {
  __shared__ double sh[GW];
  const GradSlot sl = slots[blockIdx.x];
  if ((int)blockIdx.x != sl.group_first) return;
  const float norm = group_norm(sl, part, sh);
  if (threadIdx.x == 0) norms[sl.group] = norm;
}

__global__ __launch_bounds__(kGradThreads) void k_grad_clip(const GradSlot* __restrict__ slots,
                                                            const GradPiece* __restrict__ in,
                                                            const GradPiece* __restrict__ out,
                                                            const double* __restrict__ part, float max_norm, float eps,
                                                            float* __restrict__ norms) {
  __shared__ double sh[GW];
  // last slot first: what the first pass read last is still in the cache
  const int slot = (int)(gridDim.x - 1 - blockIdx.x);
  const GradSlot sl = slots[slot];
  const float norm = group_norm(sl, part, sh);
  if (slot == sl.group_first && threadIdx.x == 0) norms[sl.group] = norm;
  const float q = max_norm / (norm + eps);
  const float coef = q > 1.0f ? 1.0f : q;   // a NaN stays one
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int k = wave; k < sl.count; k += GW) {
    const GradPiece pi = in[sl.first + k], po = out[sl.first + k];
    if (coef == 1.0f && pi.data == po.data) continue;   // in place and within the limit: nothing changes
    if (pi.dtype == LQ_F32) piece_scale<ElemF32>(pi, po, coef, lane);
    else if (pi.dtype == LQ_BF16) piece_scale<ElemBF16>(pi, po, coef, lane);
    else piece_scale<ElemF16>(pi, po, coef, lane);
  }
}

}  // namespace

hipError_t launch_grad_squares(const GradSlot* slots, const GradPiece* pieces, int32_t n_slots, double* part,
                               hipStream_t s) {
  hipLaunchKernelGGL(k_grad_squares, dim3((unsigned)n_slots), dim3(kGradThreads), 0, s, slots, pieces, part);
  return hipGetLastError();
}

hipError_t launch_grad_norms(const GradSlot* slots, int32_t n_slots, const double* part, float* norms, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_norms, dim3((unsigned)n_slots), dim3(kGradThreads), 0, s, slots, part, norms);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradSlot* slots, const GradPiece* in, const GradPiece* out, int32_t n_slots,
                            const double* part, float max_norm, float eps, float* norms, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_clip, dim3((unsigned)n_slots), dim3(kGradThreads), 0, s, slots, in, out, part, max_norm,
                     eps, norms);
  return hipGetLastError();
}

}  // namespace lq
