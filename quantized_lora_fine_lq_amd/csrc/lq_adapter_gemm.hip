// The many-adapter GEMM: out[token] = A[token] Bt^T + s_a L[token] Lb_a^T over
// the tokens in sorted order (equal adapters side by side), Bt the bfloat16
// dequantized weight (forward) or its transpose (backward, grad_X).
//
// QLoRA (Heng's Blog), introduction: h = dequant(W0_NF4) x + (alpha/r) B A x.
#include <algorithm>
#include <type_traits>

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

// Wait until at most `n` of the wave's memory operations are outstanding.
template <int n>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }
// At most `n` loads outstanding and no reads of LDS, then the barrier: past it
// a buffer that everyone has read may be refilled.
template <int n>
__device__ __forceinline__ void ring_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(n) : "memory");
}

// The adapter of the sorted positions from pos on, inside a tile that ends at
// mend: its columns are steps of 64 (8 runs of 8) of TERMS copies of Lb.
struct Adapter {
  int64_t lo, hi;          // its positions inside the tile
  const uint16_t* base;    // Lb
  int stride, runs;        // of Lb: elements a row, runs of 8 columns
  int live, steps;         // runs of all terms, steps of 8 of them (0: no adapter)
};
template <int TERMS>
__device__ __forceinline__ Adapter adapter_at(const AdapterGemm& p, int64_t pos, int64_t mend) {
  Adapter s{pos, mend, nullptr, 8, 1, 0, 0};
  if (pos >= mend) return s;
  const int a = uniform(p.rt.sid[pos]);
  if (a >= p.v.n) return s;
  s.hi = min((int64_t)uniform(p.rt.off[a + 1]), mend);
  const lq_adapter ad = p.v.tab[a];
  const int r8 = (ad.r + 7) & ~7;
  s.base = !p.lt_all && ad.r % 8 == 0 ? ad.B : p.lt + p.Ncols * ad.row8;
  s.stride = r8;
  s.runs = r8 >> 3;
  s.live = TERMS * s.runs;
  s.steps = (s.live + 7) >> 3;
  return s;
}

// A lane's 4 consecutive outputs c .. c + 3 of one token.
template <bool OUT_F32>
__device__ __forceinline__ void store4(const AdapterGemm& p, int64_t row, int64_t c, const f32x4_t& v) {
  if (p.Ncols % 4 == 0) {
    if (c >= p.Ncols) return;
    if (OUT_F32) {
      float* o = reinterpret_cast<float*>(p.out) + row + c;   // 4-byte aligned
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

// Tile 256 positions x BN weight rows, 64-wide steps, 8 waves in two groups of
// four (one wave of each group per SIMD). The groups work one slot apart:
// while one group's waves multiply (16 MFMA each), the other's read their next
// fragments from LDS and issue memory-to-LDS loads, so matrix unit and LDS are
// busy at once; a barrier ends every slot. Row r of an LDS tile keeps its
// 16-byte chunk c at slot c ^ (r % 8): fragment reads of 8 rows hit distinct
// banks. The matrix product is taken with weights as rows and tokens as
// columns: a lane then holds 4 consecutive outputs of one token.
//
// BN = 256: waves 2 (tokens) x 4 (weight rows) of 128 x 64. A step is four
// quadrants, X0 Y0, X0 Y1, X1 Y1, X1 Y0, of 64 tokens x 32 weight rows; two
// buffers (128 KB), each refilled part by part as soon as both groups have
// read the part, which puts five to seven quadrants between a load and its
// use. BN = 128: waves 4 x 2 of 64 x 64, two halves a step, three buffers.
//
// Measured: 4096 tokens, 4096 -> 11008, rank 64: 325 to 394 us with the clock,
// 0.95 to 1.15 PFLOP/s; 1999 tokens, 4096 -> 4096: 71 us, 0.95 PFLOP/s;
// backward of 2048 tokens 70. The library's plain product reaches 0.87 PFLOP/s
// at the first size, 1.09 at 2048 tokens and 1.38 at 8192^3. Bound by the matrix cores'
// issue and the clock they leave; what the slots lose is the edges (a last
// round that is not full, the start of a tile) and, where a tile's tokens
// belong to several adapters, their steps at its end.
template <int BN, bool OUT_F32, bool BWD>
__global__ __launch_bounds__(G_THREADS) void k_adapter_gemm(AdapterGemm p) {
  constexpr bool BIG = BN == 256;
  constexpr int WN = BIG ? 4 : 2, WM = 8 / WN;         // waves over weight rows, tokens
  constexpr int CT = BN / WN / 16, RT = GM / WM / 16;  // 16 x 16 tiles per wave
  constexpr int RING = BIG ? 2 : 3;
  constexpr int XP = BIG ? 2 : 1;                      // parts of the token tile (each 64 rows of a wave's)
  constexpr int QX = GM / 64 / XP, QY = BN / 64 / 2;   // 16-byte loads per thread and part
  struct __attribute__((aligned(16))) Lds {
    uint16_t x[RING][GM * GK];
    uint16_t y[RING][BN * GK];
  };
  __shared__ Lds lds;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;
  const int64_t tiles_m = (p.M + GM - 1) / GM, tiles_n = (p.Ncols + BN - 1) / BN;
  const int64_t total = tiles_m * tiles_n;
  // XCD x (workgroups x, x + 8, ...) takes a contiguous range of tiles, the
  // token tiles inner
  const int64_t xcd = blockIdx.x % 8, per = total / 8, rem = total % 8;
  const int64_t t = xcd * per + min(xcd, rem) + blockIdx.x / 8;
  const int64_t m0 = t % tiles_m * GM, n0 = t / tiles_m * BN;

  // A load instruction of a wave fills 8 LDS rows (lane l: row l / 8, slot
  // l % 8). Part i of the token tile: rows 64 i .. of every wave's 128 (all
  // rows for BN = 128); part i of the weight tile: rows 16 CT / 2 i .. of every
  // wave's 16 CT.
  const int sub = lane >> 3, ch = (lane & 7) ^ sub;
  auto xrow = [&](int part, int q) {   // first tile row of the wave's q-th load
    const int k = wave * QX + q;       // 8-row groups 0 .. 8 QX - 1 of the part
    return BIG ? (k >> 3) * 128 + part * 64 + (k & 7) * 8 : k * 8;
  };
  auto yrow = [&](int part, int q) {
    const int k = wave * QY + q, per_wave = 16 * CT / 2 / 8;
    return (k / per_wave) * 16 * CT + part * 8 * CT + (k % per_wave) * 8;
  };
  const uint16_t *px[XP][QX], *py[2][QY];
#pragma unroll
  for (int i = 0; i < XP; ++i)
#pragma unroll
    for (int q = 0; q < QX; ++q) px[i][q] = p.A + (int64_t)p.rt.perm[min(m0 + xrow(i, q) + sub, p.M - 1)] * p.Kc + 8 * ch;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < QY; ++q) py[i][q] = p.Bt + min(n0 + yrow(i, q) + sub, p.Ncols - 1) * p.ldb + 8 * ch;
  const int nk = (int)((p.Kc + GK - 1) / GK);
  // Each XCD begins at an eighth of its own of the contraction (whole steps
  // only): in step, all eight would ask for the same columns, whose rows lie a
  // power of two apart, of the same memory channels. 2 to 4 % of the kernel's
  // time; a place of its own per tile costs the tiles of an XCD the weight rows
  // and tokens that they share in its L2 (2048 tokens: 72 -> 90 us).
  const int rot = p.Kc % GK ? 0 : (int)(xcd * nk / 8);
  auto column = [&](int it) {   // first column of step it
    const int at = it + rot;
    return (int64_t)(at < nk ? at : at - nk) * GK;
  };

  // The adapters' part: an adapter's [hi | mid (| lo)] columns of the terms
  // against as many copies of Lb, in steps of 64 (columns past the last are
  // zero on both sides). Of a tile whose tokens share one adapter it is simply
  // the end of the contraction, steps nk .. nk + nl - 1 of the main loop.
  constexpr int TERMS = OUT_F32 ? 3 : 2;
  const int64_t mend = min(m0 + GM, p.M);
  auto lora_x = [&](const Adapter& s, int kt, int i, int buf) {
    const int c = 8 * kt + ch;   // this lane's run of 8 columns
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int64_t pos = min(m0 + xrow(i, q) + sub, p.M - 1);
      load_lds16(c < s.live ? p.terms + pos * 3 * p.v.rs + 8 * c : p.zeros, lds.x[buf] + xrow(i, q) * GK);
    }
  };
  auto lora_y = [&](const Adapter& s, int kt, int i, int buf) {
    const int c = 8 * kt + ch;
#pragma unroll
    for (int q = 0; q < QY; ++q) {
      const int64_t n = min(n0 + yrow(i, q) + sub, p.Ncols - 1);
      load_lds16(c < s.live ? s.base + n * s.stride + 8 * (c % s.runs) : p.zeros, lds.y[buf] + yrow(i, q) * GK);
    }
  };

  // Part i of step it into its buffer; Plain: a whole step of the base
  // contraction. Past the last step zeros, into a buffer that nobody reads any
  // more: the count of outstanding loads, on which the waits rely, stays the
  // same.
  Adapter whole{0, 0, nullptr, 8, 1, 0, 0};   // the tile's one adapter, if it has one
  typedef std::integral_constant<bool, true> Plain;
  typedef std::integral_constant<bool, false> Any;
  auto load_x = [&](auto plain, int it, int i, int buf) {
    if (plain.value || it < nk) {
      const int64_t k0 = column(it);
      const bool ok = plain.value || !BWD || k0 + 8 * ch + 8 <= p.Kc;   // past the contraction: zeros (0 * NaN is not 0)
#pragma unroll
      for (int q = 0; q < QX; ++q) load_lds16(ok ? px[i][q] + k0 : p.zeros, lds.x[buf] + xrow(i, q) * GK);
    } else {
      lora_x(whole, it - nk, i, buf);
    }
  };
  auto load_y = [&](auto plain, int it, int i, int buf) {
    if (plain.value || it < nk) {
      const int64_t k0 = column(it);
#pragma unroll
      for (int q = 0; q < QY; ++q) load_lds16(py[i][q] + k0, lds.y[buf] + yrow(i, q) * GK);
    } else {
      lora_y(whole, it - nk, i, buf);
    }
  };

  f32x4_t acc[CT][RT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  u32x4_t fx[2][4], fy[2][2][CT / 2];   // [k half][tile], weight side [part][k half][tile]
  const int slot0 = 8 * (lg ^ (li & 7)), slot1 = 8 * ((4 + lg) ^ (li & 7));
  const int ox = (wm * 16 * RT + li) * GK, oy = (wn * 16 * CT + li) * GK;
  auto read_x = [&](int i, int buf) {
    const uint16_t* b = lds.x[buf] + ox + i * 64 * GK;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      fx[0][r] = ld16(b + 16 * r * GK + slot0);
      fx[1][r] = ld16(b + 16 * r * GK + slot1);
    }
  };
  auto read_y = [&](int i, int buf) {
    const uint16_t* b = lds.y[buf] + oy + i * 8 * CT * GK;
#pragma unroll
    for (int c = 0; c < CT / 2; ++c) {
      fy[i][0][c] = ld16(b + 16 * c * GK + slot0);
      fy[i][1][c] = ld16(b + 16 * c * GK + slot1);
    }
  };
  auto end_memory = [&]() {   // the fragments have arrived: a part may be refilled after the barrier
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](int xi, int yi) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < CT / 2; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[yi * (CT / 2) + c][xi * 4 + r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              as_bf16x8(fy[yi][u][c]), as_bf16x8(fx[u][r]), acc[yi * (CT / 2) + c][xi * 4 + r], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  const bool late = wave >= 4;   // the group that works one slot behind
  Adapter next = adapter_at<TERMS>(p, m0, mend);
  if (next.steps && next.hi == mend) whole = next;
  const int nsteps = nk + whole.steps;
  int it = 0, buf = 0;
  auto step = [&](auto plain) {
    if constexpr (BIG) {
      read_x(0, buf);
      read_y(0, buf);
      load_x(plain, it + 1, 1, buf ^ 1);
      wait_vm<10>();          // Y1 of this step
      end_memory();
      multiply(0, 0);
      read_y(1, buf);
      load_x(plain, it + 2, 0, buf);
      wait_vm<10>();          // X1 of this step
      end_memory();
      multiply(0, 1);
      read_x(1, buf);
      load_y(plain, it + 2, 0, buf);
      end_memory();
      multiply(1, 1);
      load_y(plain, it + 2, 1, buf);
      wait_vm<10>();          // X0 and Y0 of the next step
      end_memory();
      multiply(1, 0);
      buf ^= 1;
    } else {
      const int b2 = buf == 0 ? 2 : buf - 1;   // buffer of step it + 2
      read_x(0, buf);
      read_y(0, buf);
      load_x(plain, it + 2, 0, b2);
      end_memory();
      multiply(0, 0);
      read_y(1, buf);
      load_y(plain, it + 2, 0, b2);
      load_y(plain, it + 2, 1, b2);
      wait_vm<QX + 2 * QY>();   // the next step
      end_memory();
      multiply(0, 1);
      buf = buf == 2 ? 0 : buf + 1;
    }
    ++it;
  };
  if constexpr (BIG) {
    load_x(Any(), 0, 0, 0);
    load_y(Any(), 0, 0, 0);
    load_y(Any(), 0, 1, 0);
    load_x(Any(), 0, 1, 0);
    load_x(Any(), 1, 0, 1);
    load_y(Any(), 1, 0, 1);
    load_y(Any(), 1, 1, 1);
    ring_barrier<10>();
  } else {
    load_x(Any(), 0, 0, 0);
    load_y(Any(), 0, 0, 0);
    load_y(Any(), 0, 1, 0);
    load_x(Any(), 1, 0, 1);
    load_y(Any(), 1, 0, 1);
    load_y(Any(), 1, 1, 1);
    ring_barrier<QX + 2 * QY>();
  }
  if (late) barrier();
  const int nplain = nk - 3;   // steps that load whole steps of the contraction: without a branch
  while (it < nplain) step(Plain());
  while (it < nsteps) step(Any());
  if (!late) barrier();   // as many barriers as the other group
  wait_vm<0>();           // the loads past the last step, before the workgroup's LDS is given up

  const int64_t pw = m0 + wm * 16 * RT, cw = n0 + wn * 16 * CT;

  // A tile of several adapters: one after the other, each one's products formed
  // apart and added to its own tokens' columns alone, so that an adapter's
  // infinities and NaN stay with its tokens.
  if (!whole.steps && next.steps) {
    Adapter cur = next;
    int kt = 0;
    ring_barrier<0>();   // everyone has read the last step
    lora_x(cur, 0, 0, 0);
    if constexpr (XP == 2) lora_x(cur, 0, 1, 0);
    lora_y(cur, 0, 0, 0);
    lora_y(cur, 0, 1, 0);
    for (int b = 0; cur.steps; b ^= 1) {
      const int64_t lo = cur.lo, hi = cur.hi;
      if (++kt >= cur.steps) {
        cur = adapter_at<TERMS>(p, cur.hi, mend);
        kt = 0;
      }
      ring_barrier<0>();   // this step has landed, and the other buffer is read
      if (cur.steps) {
        lora_x(cur, kt, 0, b ^ 1);
        if constexpr (XP == 2) lora_x(cur, kt, 1, b ^ 1);
        lora_y(cur, kt, 0, b ^ 1);
        lora_y(cur, kt, 1, b ^ 1);
      }
      read_y(0, b);
      read_y(1, b);
#pragma unroll
      for (int xi = 0; xi < XP; ++xi) {
        read_x(xi, b);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t pos = pw + 16 * (xi * 4 + r) + li;
          const bool mine = pos >= lo && pos < hi;
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            f32x4_t d = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < 2; ++u)
              d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(fy[c / (CT / 2)][u][c % (CT / 2)]), as_bf16x8(fx[u][r]),
                                                          d, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][xi * 4 + r][e] += mine ? d[e] : 0.0f;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }

  // lane: token position pw + 16 rt + li, outputs cw + 16 ct + 4 lg + [0, 4)
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int64_t pos = pw + 16 * rt + li;
    if (pos >= p.M) continue;
    const int64_t row = (int64_t)p.rt.perm[pos] * p.Ncols;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      store4<OUT_F32>(p, row, cw + 16 * ct + 4 * lg, acc[ct][rt]);
    }
  }
}

// Few tokens or a small weight: tiles of 64 positions x 64 weight rows, four
// waves of 32 x 32, so that the tiles cover the chip. Steps pass through a ring
// of four LDS buffers (64 KB) with loads three ahead and one barrier a step. A
// step's chain (barrier, loads, fragment reads, eight MFMA) needs a second wave
// per SIMD beside it: past 256 tiles another workgroup's; up to 256 the
// workgroup has a second group of waves that takes every other step through a
// ring of its own, and the two sums meet at the end. (A ring of eight buffers
// instead did not shorten the chain.) Measured, N = K = 4096, 8 adapters of rank
// 16, bfloat16: 250 tokens 21 us (one group: 25), 500 tokens 31 (two groups:
// 38); 250 tokens of 20 adapters in float32 24.
//
// The adapters' steps follow the base contraction's in the same rings, from a
// table made at the start; the products of each go to its own tokens' columns
// alone.
constexpr int SM = 64, SN = 64, S_THREADS = 256, S_RING = 4;
constexpr int S_STEPS = SM * 6;   // an adapter per token, 3 terms of rank 128

struct SmallStep {
  const uint16_t* base;    // Lb
  int runs, live, first;   // of Lb: runs of 8 columns; of all terms; the step's first
  int lo, hi;              // its positions of the tile
};

template <int GROUPS, bool OUT_F32, bool BWD>
__global__ __launch_bounds__(S_THREADS * GROUPS, 2) void k_adapter_gemm_small(AdapterGemm p) {
  constexpr int TERMS = OUT_F32 ? 3 : 2;
  struct __attribute__((aligned(16))) Lds {
    uint16_t x[GROUPS][S_RING][SM * GK];
    uint16_t y[GROUPS][S_RING][SN * GK];
    SmallStep steps[S_STEPS];
    int total;
  };
  __shared__ Lds lds;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int group = wave >> 2, w4 = wave & 3;
  const int li = lane & 15, lg = lane >> 4;
  const int wn = w4 & 1, wm = w4 >> 1;
  const int64_t tiles_m = (p.M + SM - 1) / SM, tiles_n = (p.Ncols + SN - 1) / SN;
  const int64_t total = tiles_m * tiles_n;
  const int64_t xcd = blockIdx.x % 8, per = total / 8, rem = total % 8;
  const int64_t t = xcd * per + min(xcd, rem) + blockIdx.x / 8;
  const int64_t m0 = t % tiles_m * SM, n0 = t / tiles_m * SN, mend = min(m0 + SM, p.M);

  const int sub = lane >> 3, ch = (lane & 7) ^ sub;
  const uint16_t *px[2], *py[2], *pt[2];
  int64_t ny[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = (w4 * 2 + q) * 8 + sub;
    const int64_t pos = min(m0 + row, p.M - 1);
    px[q] = p.A + (int64_t)p.rt.perm[pos] * p.Kc + 8 * ch;
    pt[q] = p.terms + pos * 3 * p.v.rs;
    ny[q] = min(n0 + row, p.Ncols - 1);
    py[q] = p.Bt + ny[q] * p.ldb + 8 * ch;
  }
  const int nk = (int)((p.Kc + GK - 1) / GK);
  int steps = 0;   // of both parts, once the table is there
  uint16_t(*const rx)[SM * GK] = lds.x[group];
  uint16_t(*const ry)[SN * GK] = lds.y[group];
  // step it of the sequence into the group's buffer buf; past the end zeros
  auto load = [&](int it, int buf) {
    if (it < nk) {
      const int64_t k0 = (int64_t)it * GK;
      const bool ok = !BWD || k0 + 8 * ch + 8 <= p.Kc;   // past the contraction: zeros (0 * NaN is not 0)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        load_lds16(ok ? px[q] + k0 : p.zeros, rx[buf] + (w4 * 2 + q) * 8 * GK);
        load_lds16(py[q] + k0, ry[buf] + (w4 * 2 + q) * 8 * GK);
      }
      return;
    }
    SmallStep st{nullptr, 1, 0, 0, 0, 0};
    if (it < steps) st = lds.steps[it - nk];
    const int c = st.first + ch;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      load_lds16(c < st.live ? pt[q] + 8 * c : p.zeros, rx[buf] + (w4 * 2 + q) * 8 * GK);
      load_lds16(c < st.live ? st.base + (ny[q] * st.runs + c % st.runs) * 8 : p.zeros, ry[buf] + (w4 * 2 + q) * 8 * GK);
    }
  };
  auto prime = [&]() {
#pragma unroll
    for (int i = 0; i < S_RING - 1; ++i) load(GROUPS * i + group, i);
  };
  const bool early = nk >= GROUPS * (S_RING - 1);   // the first loads need no table
  if (early) prime();
  if (wave == 4 * GROUPS - 1) {
    // Lane l: position l of the tile. Equal adapters lie side by side; the
    // first position of each writes its steps, numbered by a sum over the
    // lanes below, bit by bit.
    const bool valid = m0 + lane < mend;
    const int a = valid ? p.rt.sid[m0 + lane] : -1, before = __shfl_up(a, 1);
    const uint64_t starts = __ballot(lane == 0 || a != before);
    const bool leads = valid && a < p.v.n && ((starts >> lane) & 1);
    const lq_adapter ad = p.v.tab[leads ? a : 0];
    const int runs = (ad.r + 7) >> 3, live = TERMS * runs, count = leads ? (live + 7) >> 3 : 0;
    int first = 0, sum = 0;
#pragma unroll
    for (int b = 0; b < 3; ++b) {
      const uint64_t one = __ballot((count >> b) & 1);
      first += (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(one >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)one, 0)) << b;
      sum += __popcll(one) << b;
    }
    const uint64_t above = lane < 63 ? starts >> (lane + 1) : 0;
    const int hi = above ? lane + __ffsll((unsigned long long)above) : SM;
    const uint16_t* base = !p.lt_all && ad.r % 8 == 0 ? ad.B : p.lt + p.Ncols * ad.row8;
    for (int k = 0; k < count; ++k) lds.steps[first + k] = SmallStep{base, runs, live, 8 * k, lane, hi};
    if (lane == 0) lds.total = sum;
  }
  __syncthreads();
  steps = nk + uniform(lds.total);
  if (!early) prime();

  f32x4_t acc[2][2];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int r = 0; r < 2; ++r) acc[c][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int slot[2] = {8 * (lg ^ (li & 7)), 8 * ((4 + lg) ^ (li & 7))};
  const int ox = (wm * 32 + li) * GK, oy = (wn * 32 + li) * GK;
  u32x4_t fx[2][2], fy[2][2];
  auto turn = [&](int i) {   // the group's step i is in LDS, and step i - 1 read by everyone
    ring_barrier<(S_RING - 2) * 4>();
    load(GROUPS * (i + S_RING - 1) + group, (i + S_RING - 1) % S_RING);
    const int buf = i % S_RING;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        fx[u][k] = ld16(rx[buf] + ox + 16 * k * GK + slot[u]);
        fy[u][k] = ld16(ry[buf] + oy + 16 * k * GK + slot[u]);
      }
  };
  auto multiply = [&]() {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          acc[c][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(fy[u][c]), as_bf16x8(fx[u][r]), acc[c][r], 0, 0, 0);
  };
  int i = 0;
  for (; GROUPS * (i + 1) <= nk; ++i) {
    turn(i);
    multiply();
  }
  for (; GROUPS * i < steps; ++i) {   // the same count for both groups
    turn(i);
    const int it = GROUPS * i + group;
    if (it < nk) {
      multiply();
    } else if (it < steps) {
      const int lo = lds.steps[it - nk].lo, hi = lds.steps[it - nk].hi;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int pos = wm * 32 + 16 * r + li;
        const bool mine = pos >= lo && pos < hi;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          f32x4_t d = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int u = 0; u < 2; ++u)
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(fy[u][c]), as_bf16x8(fx[u][r]), d, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[c][r][e] += mine ? d[e] : 0.0f;
        }
      }
    }
  }
  wait_vm<0>();   // the loads past the last step
  if constexpr (GROUPS == 2) {   // group g finishes the weight rows of c = g, group 0's sum first
    ring_barrier<0>();   // the tiles are read: the sums take their place
    f32x4_t* sum = reinterpret_cast<f32x4_t*>(lds.x) + 128 * w4 + lane;   // [group][w4][r][lane]
#pragma unroll
    for (int r = 0; r < 2; ++r) sum[512 * group + 64 * r] = group ? acc[0][r] : acc[1][r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const f32x4_t other = sum[512 * (1 - group) + 64 * r];
      if (group) acc[1][r] = other + acc[1][r];
      else acc[0][r] = acc[0][r] + other;
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t pos = m0 + wm * 32 + 16 * r + li;
    if (pos >= p.M) continue;
    const int64_t row = (int64_t)p.rt.perm[pos] * p.Ncols;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (GROUPS == 1 || c == group) store4<OUT_F32>(p, row, n0 + wn * 32 + 16 * c + 4 * lg, acc[c][r]);
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

template <int BN>
hipError_t launch_tile(const AdapterGemm& g, hipStream_t s) {
  const int64_t tiles = ((g.M + GM - 1) / GM) * ((g.Ncols + BN - 1) / BN);
  LQ_DASSERT(tiles > 0 && tiles < (int64_t(1) << 31));
  const dim3 grid((unsigned)tiles), block(G_THREADS);
  if (g.lt_all) hipLaunchKernelGGL((k_adapter_gemm<BN, false, true>), grid, block, 0, s, g);
  else if (g.out_f32) hipLaunchKernelGGL((k_adapter_gemm<BN, true, false>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((k_adapter_gemm<BN, false, false>), grid, block, 0, s, g);
  return hipGetLastError();
}

template <int GROUPS>
hipError_t launch_small(const AdapterGemm& g, int64_t tiles, hipStream_t s) {
  LQ_DASSERT(tiles > 0 && tiles < (int64_t(1) << 31));
  const dim3 grid((unsigned)tiles), block(S_THREADS * GROUPS);
  if (g.lt_all) hipLaunchKernelGGL((k_adapter_gemm_small<GROUPS, false, true>), grid, block, 0, s, g);
  else if (g.out_f32) hipLaunchKernelGGL((k_adapter_gemm_small<GROUPS, true, false>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((k_adapter_gemm_small<GROUPS, false, false>), grid, block, 0, s, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_gemm(const AdapterGemm& g, hipStream_t s) {
  LQ_DASSERT(g.M > 0 && g.Ncols > 0 && g.Kc > 0 && g.Kc % 8 == 0 && g.ldb % 64 == 0 && g.ldb >= g.Kc);
  // Rounds of a chip full of tiles times a tile's time per step, in us as
  // measured over K = 4096: 1.7 (256 x 256), 1.05 (256 x 128) and for 64 x 64,
  // two workgroups per CU, 0.3 where the tiles number more than the CUs. (Fewer
  // of them always win: 0.2.)
  auto tiles = [&](int64_t m, int64_t n) { return ((g.M + m - 1) / m) * ((g.Ncols + n - 1) / n); };
  auto cost = [&](int64_t count, int64_t slots, double us) { return (double)((count + slots - 1) / slots) * us; };
  const int64_t small = tiles(SM, SN);
  const double c256 = cost(tiles(256, 256), 256, 1.7), c128 = cost(tiles(256, 128), 256, 1.05), c64 = cost(small, 512, 0.3);
  if (small <= 256) return launch_small<2>(g, small, s);
  if (c64 < c128 && c64 < c256) return launch_small<1>(g, small, s);
  return c256 <= c128 ? launch_tile<256>(g, s) : launch_tile<128>(g, s);
}

hipError_t launch_transpose_weight(const uint16_t* w, int64_t N, int64_t K, int64_t ldb, uint16_t* out,
                                   hipStream_t s) {
  LQ_DASSERT(K % 64 == 0 && ldb % 64 == 0 && ldb >= N && ldb < N + 64);
  hipLaunchKernelGGL(k_transpose_weight, dim3((unsigned)(ldb / 64), (unsigned)(K / 64)), dim3(256), 0, s, w, N, K, ldb,
                     out);
  return hipGetLastError();
}

}  // namespace lq
