// The many-adapter GEMM: out[token] = A[token] Bt^T + s_a L[token] Lb_a^T over
// the tokens in sorted order (equal adapters side by side), Bt the bfloat16
// dequantized weight (forward) or its transpose (backward, grad_X).
//
// QLoRA (Heng's Blog), introduction: h = dequant(W0_NF4) x + (alpha/r) B A x.
#include <algorithm>

#include "lq_adapters.h"
#include "lq_device.h"

namespace lq {
namespace {

__device__ __forceinline__ u32x4_t ld16(const void* p) { return *reinterpret_cast<const u32x4_t*>(p); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

constexpr int GM = 256, GK = 64, G_THREADS = 512;

// Memory to LDS, 16 bytes a lane: lane i's 16 bytes land at dst + 16 i.
__device__ __forceinline__ void load_lds16(const uint16_t* src, uint16_t* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}


// Term `t` of v = hi + mid (+ lo): bfloat16 values, each the rounding of what
// the ones before leave.
__device__ __forceinline__ float term_of(float v, int t) {
  const float hi = bf16lo_to_f32(pack_bf16x2(v, 0.0f));
  if (t == 0) return hi;
  const float mid = bf16lo_to_f32(pack_bf16x2(v - hi, 0.0f));
  return t == 1 ? mid : v - hi - mid;
}

// Lane (li, lg)'s operands of one step of 32 contraction columns of adapter
// ad's term: runs of 8 columns, TERMS copies of the r columns rounded up to
// whole runs. Weight side: row c of Lb (8 values of a run); token side: term of
// s * L[token] at the same run.
template <bool BWD>
__device__ __forceinline__ u32x4_t lora_weight(const AdapterGemm& p, const lq_adapter& ad, int64_t c, int j0,
                                               bool live) {
  const int64_t cc = min(c, p.Ncols - 1);
  u32x4_t o;
  if (BWD) {
    const int r8 = (ad.r + 7) & ~7;
    o = ld16(p.lt + p.Ncols * ad.row8 + cc * r8 + j0);
  } else if (ad.r % 8 == 0) {
    o = ld16(ad.B + cc * ad.r + j0);
  } else {
    const uint16_t* b = ad.B + cc * ad.r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + 2 * e;
      const uint32_t x = b[min(j, ad.r - 1)], y = b[min(j + 1, ad.r - 1)];
      o[e] = (j < ad.r ? x : 0u) | ((j + 1 < ad.r ? y : 0u) << 16);
    }
  }
  if (!live) o = u32x4_t{0u, 0u, 0u, 0u};
  return o;
}
__device__ __forceinline__ u32x4_t lora_token(const AdapterGemm& p, float s, int64_t token, int j0, int term,
                                              bool live) {
  const float* l = p.L + token * p.v.rs + j0;
  const f32x4_t x = *reinterpret_cast<const f32x4_t*>(l), y = *reinterpret_cast<const f32x4_t*>(l + 4);
  u32x4_t o;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    o[e] = pack_bf16x2(term_of(s * x[2 * e], term), term_of(s * x[2 * e + 1], term));
    o[2 + e] = pack_bf16x2(term_of(s * y[2 * e], term), term_of(s * y[2 * e + 1], term));
  }
  if (!live) o = u32x4_t{0u, 0u, 0u, 0u};
  return o;
}

// The adapters' part of a wave's CT x RT tiles of 16 x 16 (weight rows c0 ..,
// sorted positions p0 ..), before the main loop. A tile whose 16 tokens share
// an adapter accumulates into acc; in a tile with several, each adapter's
// product is formed apart and added to its own tokens' columns alone, so that
// one adapter's infinities and NaN cannot reach another's tokens.
template <int CT, int RT, int TERMS, bool BWD>
__device__ __forceinline__ void lora_init(const AdapterGemm& p, int64_t p0, int64_t c0, f32x4_t (&acc)[CT][RT]) {
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int64_t pend = min(p0 + 16 * RT, p.M);
  int64_t pos = p0;
  while (pos < pend) {
    const int a = uniform(p.rt.sid[pos]);
    if (a >= p.v.n) break;   // sorted: the rest has none
    const int64_t send = min((int64_t)uniform(p.rt.off[a + 1]), pend);
    const lq_adapter ad = p.v.tab[a];
    const int runs = (ad.r + 7) >> 3, total = TERMS * runs;
    for (int q0 = 0; q0 < total; q0 += 4) {
      const int run = q0 + lg;
      const bool live = run < total;
      const int term = live ? run / runs : 0, j0 = live ? 8 * (run - term * runs) : 0;
      u32x4_t w[CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) w[ct] = lora_weight<BWD>(p, ad, c0 + 16 * ct + li, j0, live);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int64_t t0 = p0 + 16 * rt, t1 = min(t0 + 16, pend);
        if (t0 < send && t1 > pos) {
          const u32x4_t x = lora_token(p, ad.scale, p.rt.perm[min(t0 + li, p.M - 1)], j0, term, live);
          const bool whole = pos <= t0 && send >= t1;
          const bool mine = t0 + li >= pos && t0 + li < send;
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            if (whole) {
              acc[ct][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w[ct]), as_bf16x8(x), acc[ct][rt], 0, 0, 0);
            } else {
              const f32x4_t d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w[ct]), as_bf16x8(x),
                                                                        f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[ct][rt][e] += mine ? d[e] : 0.0f;
            }
          }
        }
      }
    }
    pos = send;
  }
}

// Tile 256 positions x BN weight rows, 8 waves; 64-wide steps, two LDS buffers
// filled by memory-to-LDS loads one step ahead. Row r of a tile keeps its
// 16-byte chunk c at slot c ^ (r % 8), so fragment reads of 8 rows hit distinct
// banks. The matrix product is taken with weights as rows and tokens as
// columns: a lane then holds 4 consecutive outputs of one token.
template <int BN, bool OUT_F32, bool BWD>
__global__ __launch_bounds__(G_THREADS) void k_adapter_gemm(AdapterGemm p) {
  constexpr int WN = BN == 256 ? 4 : 2, WM = 8 / WN;       // waves over weight rows, tokens
  constexpr int CT = BN / WN / 16, RT = GM / WM / 16;      // 16 x 16 tiles per wave
  constexpr int QA = GM / 64, QB = BN / 64;                // 16-byte loads per thread and tile
  struct __attribute__((aligned(16))) Lds {
    uint16_t a[2][GM * GK];
    uint16_t b[2][BN * GK];
  };
  __shared__ Lds lds;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;
  const int64_t tiles_m = (p.M + GM - 1) / GM, tiles_n = (p.Ncols + BN - 1) / BN;
  const int64_t total = tiles_m * tiles_n;
  // XCD x (workgroups x, x + 8, ...) takes a contiguous range of tiles, the
  // token tiles inner
  const int64_t x = blockIdx.x % 8, per = total / 8, rem = total % 8;
  const int64_t t = x * per + min(x, rem) + blockIdx.x / 8;
  const int64_t m0 = t % tiles_m * GM, n0 = t / tiles_m * BN;

  const uint16_t *pa[QA], *pb[QB];
  const int sub = lane >> 3, ch = (lane & 7) ^ sub;        // row in the instruction's 8, chunk read
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int64_t pos = min(m0 + (wave * QA + q) * 8 + sub, p.M - 1);
    pa[q] = p.A + (int64_t)p.rt.perm[pos] * p.Kc;
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) pb[q] = p.Bt + min(n0 + (wave * QB + q) * 8 + sub, p.Ncols - 1) * p.ldb + 8 * ch;
  auto stage = [&](int buf, int64_t k0) {
    const bool ok = k0 + 8 * ch + 8 <= p.Kc;   // past the contraction: zeros (Bt is zero there, but 0 * NaN is not)
#pragma unroll
    for (int q = 0; q < QA; ++q)
      load_lds16(ok ? pa[q] + k0 + 8 * ch : p.zeros, lds.a[buf] + (wave * QA + q) * 8 * GK);
#pragma unroll
    for (int q = 0; q < QB; ++q) load_lds16(pb[q] + k0, lds.b[buf] + (wave * QB + q) * 8 * GK);
  };

  f32x4_t acc[CT][RT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  stage(0, 0);
  const int64_t pw = m0 + wm * 16 * RT, cw = n0 + wn * 16 * CT;
  lora_init<CT, RT, OUT_F32 ? 3 : 2, BWD>(p, pw, cw, acc);
  __syncthreads();
  const int nk = (int)((p.Kc + GK - 1) / GK);
  for (int it = 0; it < nk; ++it) {
    const int buf = it & 1;
    if (it + 1 < nk) stage(buf ^ 1, (int64_t)(it + 1) * GK);
    const uint16_t* sa = lds.a[buf] + (wm * 16 * RT + li) * GK;
    const uint16_t* sb = lds.b[buf] + (wn * 16 * CT + li) * GK;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int slot = 8 * ((4 * u + lg) ^ (li & 7));
      u32x4_t fa[RT], fb[CT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) fa[rt] = ld16(sa + 16 * rt * GK + slot);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) fb[ct] = ld16(sb + 16 * ct * GK + slot);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          acc[ct][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(fb[ct]), as_bf16x8(fa[rt]), acc[ct][rt], 0, 0, 0);
    }
    __syncthreads();
  }

  // lane: token position pw + 16 rt + li, outputs cw + 16 ct + 4 lg + [0, 4)
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int64_t pos = pw + 16 * rt + li;
    if (pos >= p.M) continue;
    const int64_t row = (int64_t)p.rt.perm[pos] * p.Ncols;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int64_t c = cw + 16 * ct + 4 * lg;
      const f32x4_t v = acc[ct][rt];
      if (p.Ncols % 4 == 0) {
        if (c >= p.Ncols) continue;
        if (OUT_F32) {
          float* o = reinterpret_cast<float*>(p.out) + row + c;
          o[0] = v[0]; o[1] = v[1]; o[2] = v[2]; o[3] = v[3];
        } else {
          uint2 o;
          o.x = pack_bf16x2(v[0], v[1]);
          o.y = pack_bf16x2(v[2], v[3]);
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + row + c) = o;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (c + e >= p.Ncols) break;
          if (OUT_F32) reinterpret_cast<float*>(p.out)[row + c + e] = v[e];
          else reinterpret_cast<uint16_t*>(p.out)[row + c + e] = (uint16_t)(pack_bf16x2(v[e], 0.f) & 0xFFFFu);
        }
      }
    }
  }
}

// 64 x 64 tiles through LDS; columns N .. ldb of the output are zero.
__global__ __launch_bounds__(256) void k_transpose_weight(const uint16_t* __restrict__ w, int64_t N, int64_t K,
                                                          int64_t ldb, uint16_t* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[64][72];   // [n][k]
  const int64_t n0 = (int64_t)blockIdx.x * 64, k0 = (int64_t)blockIdx.y * 64;   // K % 64 == 0
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = threadIdx.x + 256 * u, n = i >> 3, c = 8 * (i & 7);
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (n0 + n < N) v = ld16(w + (n0 + n) * K + k0 + c);
    *reinterpret_cast<u32x4_t*>(&tile[n][c]) = v;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = threadIdx.x + 256 * u, k = i >> 3, c = 8 * (i & 7);
    u32x4_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (uint32_t)tile[c + 2 * e][k] | ((uint32_t)tile[c + 2 * e + 1][k] << 16);
    *reinterpret_cast<u32x4_t*>(out + (k0 + k) * ldb + n0 + c) = v;   // ldb % 64 == 0 covers the tile
  }
}

__global__ void k_zero16(uint32_t* p) {
  if (threadIdx.x < 4) p[threadIdx.x] = 0u;
}

template <int BN>
hipError_t launch_tile(const AdapterGemm& g, hipStream_t s) {
  const int64_t tiles = ((g.M + GM - 1) / GM) * ((g.Ncols + BN - 1) / BN);
  LQ_DASSERT(tiles > 0 && tiles < (int64_t(1) << 31));
  const dim3 grid((unsigned)tiles), block(G_THREADS);
  if (g.lt) hipLaunchKernelGGL((k_adapter_gemm<BN, false, true>), grid, block, 0, s, g);
  else if (g.out_f32) hipLaunchKernelGGL((k_adapter_gemm<BN, true, false>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((k_adapter_gemm<BN, false, false>), grid, block, 0, s, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_gemm(const AdapterGemm& g, hipStream_t s) {
  LQ_DASSERT(g.M > 0 && g.Ncols > 0 && g.Kc > 0 && g.Kc % 8 == 0 && g.ldb % 64 == 0 && g.ldb >= g.Kc);
  const int64_t big = ((g.M + GM - 1) / GM) * ((g.Ncols + 255) / 256);
  return big >= 256 ? launch_tile<256>(g, s) : launch_tile<128>(g, s);
}

hipError_t launch_transpose_weight(const uint16_t* w, int64_t N, int64_t K, int64_t ldb, uint16_t* out,
                                   hipStream_t s) {
  LQ_DASSERT(K % 64 == 0 && ldb % 64 == 0 && ldb >= N && ldb < N + 64);
  hipLaunchKernelGGL(k_transpose_weight, dim3((unsigned)(ldb / 64), (unsigned)(K / 64)), dim3(256), 0, s, w, N, K, ldb,
                     out);
  return hipGetLastError();
}

hipError_t launch_zero16(uint16_t* p, hipStream_t s) {
  hipLaunchKernelGGL(k_zero16, dim3(1), dim3(64), 0, s, reinterpret_cast<uint32_t*>(p));
  return hipGetLastError();
}

}  // namespace lq
