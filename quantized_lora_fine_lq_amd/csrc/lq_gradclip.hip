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
#include "lq_adapters.h"
#include "lq_device.h"

namespace lq {
namespace {

constexpr int GW = kGradThreads / 64;

__device__ __forceinline__ float load_f32(const void* p, int dtype, int64_t i) {
  if (dtype == LQ_F32) return reinterpret_cast<const float*>(p)[i];
  if (dtype == LQ_BF16) return bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
  return (float)reinterpret_cast<const _Float16*>(p)[i];
}
__device__ __forceinline__ void store_f32(void* p, int dtype, int64_t i, float v) {
  if (dtype == LQ_F32) reinterpret_cast<float*>(p)[i] = v;
  else if (dtype == LQ_BF16) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
  else reinterpret_cast<_Float16*>(p)[i] = (_Float16)v;
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
    for (int i = lane; i < pc.count; i += 64) {
      const double x = (double)load_f32(pc.data, pc.dtype, i);
      acc = __builtin_fma(x, x, acc);
    }
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
  const GradSlot sl = slots[blockIdx.x];
  const float norm = group_norm(sl, part, sh);
  if ((int)blockIdx.x == sl.group_first && threadIdx.x == 0) norms[sl.group] = norm;
  const float q = max_norm / (norm + eps);
  const float coef = q > 1.0f ? 1.0f : q;   // a NaN stays one
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int k = wave; k < sl.count; k += GW) {
    const GradPiece pi = in[sl.first + k], po = out[sl.first + k];
    const int n = min(pi.count, po.count);
    for (int i = lane; i < n; i += 64) store_f32(po.data, po.dtype, i, load_f32(pi.data, pi.dtype, i) * coef);
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
