// The many-adapter GEMM: out[token] = A[token] Bt^T + s_a L[token] Lb_a^T over
// the tokens in sorted order (equal adapters side by side), Bt the bfloat16
// dequantized weight (forward) or its transpose (backward, grad_X).
//
// QLoRA (Heng's Blog), introduction: h = dequant(W0_NF4) x + (alpha/r) B A x.
#include <algorithm>
#include <type_traits>

#include "lq_act.h"
#include "lq_adapters.h"
#include "lq_device.h"
#include "lq_route.h"

namespace lq {
namespace {

constexpr int GM = 256, GK = 64, G_THREADS = 512;

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

// yes ? a : b as a selection: a is formed either way, or the compiler would
// branch around each address of a step.
__device__ __forceinline__ const uint16_t* chosen(bool yes, const uint16_t* a, const uint16_t* b) {
  asm("" : "+v"(a));
  return yes ? a : b;
}

// The adapter of the sorted positions from pos on, inside a tile that ends at
// mend: its columns are steps of 64 (8 runs of 8) of TERMS copies of Lb. Of a
// pair of sets, side 1's adapters follow side 0's, of the same positions from m0.
struct Adapter {
  int64_t lo, hi;          // its positions inside the tile
  const uint16_t* base;    // Lb
  int stride, runs;        // of Lb: elements a row, runs of 8 columns
  int live, steps;         // runs of all terms, steps of 8 of them (0: no adapter)
  int side;
  const uint16_t* terms;   // the side's
  int pitch;               // of its rows
};
template <int TERMS>
__device__ __forceinline__ Adapter adapter_at(const AdapterGemm& p, int side, int64_t pos, int64_t mend) {
  Adapter s{pos, mend, nullptr, 8, 1, 0, 0, side, side ? p.s[1].terms : p.s[0].terms, 3 * (side ? p.s[1].v.rs : p.s[0].v.rs)};
  if (pos >= mend) return s;
  const int a = uniform(p.rt.sid[pos]);
  if (a >= p.s[0].v.n) return s;
  s.hi = min((int64_t)uniform(p.rt.off[a + 1]), mend);
  const lq_adapter ad = (side ? p.s[1].v.tab : p.s[0].v.tab)[a];
  const int r8 = (ad.r + 7) & ~7;
  s.base = !p.lt_all && ad.r % 8 == 0 ? ad.B : (side ? p.s[1].lt : p.s[0].lt) + p.Ncols * ad.row8;
  s.stride = r8;
  s.runs = r8 >> 3;
  s.live = TERMS * s.runs;
  s.steps = (s.live + 7) >> 3;
  return s;
}

// Which of a lane's outputs dropout keeps: of the token at position pw + 16 rt +
// li, output cw + 16 ct + 4 lg + e, bit 8 ct + 4 (rt % 2) + e of word rt / 2. A
// generator block spans the 4 outputs of two lanes, 16 apart: for tokens rt and
// rt + 1 the even one runs the first's block, the odd one the second's, and they
// exchange halves. Past the last position: any bits. One block after the other:
// the accumulators leave few registers.
template <int RT>
struct Kept {
  uint32_t w[RT / 2];
};
template <int CT, int RT>
__device__ __forceinline__ Kept<RT> kept_outputs(const DropView& d, const int32_t* perm, int64_t M, int64_t ncols,
                                                 int64_t pw, int64_t cw) {
  static_assert(CT <= 4, "eight bits a tile of 16 outputs");
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const DropGen g = drop_gen(d);
  const bool odd = lg & 1;
  int32_t token[RT / 2];
#pragma unroll
  for (int k = 0; k < RT / 2; ++k) token[k] = perm[min(pw + 16 * (2 * k + odd) + li, M - 1)];
  Kept<RT> keep;
#pragma unroll
  for (int k = 0; k < RT / 2; ++k) {
    const int64_t first = token[k] * (ncols / 8) + (cw >> 3) + (lg >> 1);
    uint32_t word = 0;
#pragma unroll 1
    for (int ct = 0; ct < CT; ++ct) {
      const u32x4_t b = drop_bits(g, (uint64_t)(first + 2 * ct));
      const uint32_t o0 = __shfl_xor(odd ? b[0] : b[2], 16), o1 = __shfl_xor(odd ? b[1] : b[3], 16);
      const uint32_t w[4] = {odd ? o0 : b[0], odd ? o1 : b[1], odd ? b[2] : o0, odd ? b[3] : o1};
      uint32_t eight = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) eight |= (uint32_t)(((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) >= d.T) << e;
      word |= eight << (8 * ct);
    }
    keep.w[k] = word;
    __builtin_amdgcn_sched_barrier(0);
  }
  return keep;
}

// v where bit `at` of keep is set, else +0 (also of an infinity or NaN).
__device__ __forceinline__ float kept_value(float v, uint32_t keep, int at) {
  return __uint_as_float(__float_as_uint(v) & (uint32_t)__builtin_amdgcn_sbfe((int)keep, (uint32_t)at, 1u));
}

// A lane's 4 consecutive outputs c .. c + 3 of one token.
template <bool OUT_F32>
__device__ __forceinline__ void store4(const AdapterGemm& p, void* out, int64_t row, int64_t c, const f32x4_t& v) {
  if (p.Ncols % 4 == 0) {
    if (c >= p.Ncols) return;
    if (OUT_F32) {
      float* o = reinterpret_cast<float*>(out) + row + c;   // 4-byte aligned
      o[0] = v[0]; o[1] = v[1]; o[2] = v[2]; o[3] = v[3];
    } else {
      uint2 o;
      o.x = pack_bf16x2(v[0], v[1]);
      o.y = pack_bf16x2(v[2], v[3]);
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + row + c) = o;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c + e >= p.Ncols) break;
      if (OUT_F32) reinterpret_cast<float*>(out)[row + c + e] = v[e];
      else reinterpret_cast<uint16_t*>(out)[row + c + e] = (uint16_t)(pack_bf16x2(v[e], 0.f) & 0xFFFFu);
    }
  }
}

// The same lane's 4 outputs of a gated pair from g and u.
template <bool OUT_F32, int ACT>
__device__ __forceinline__ void store_gated4(const AdapterGemm& p, int64_t row, int64_t c, const f32x4_t& g, const f32x4_t& u) {
  f32x4_t h;
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = act_value<ACT>(g[e]) * u[e];
  store4<OUT_F32>(p, p.out, row, c, h);
  if (p.g_out) store4<false>(p, p.g_out, row, c, g);
  if (p.u_out) store4<false>(p, p.u_out, row, c, u);
}
// act as a constant, for code that unrolls over many outputs.
template <class F>
__device__ __forceinline__ void with_act(int act, const F& f) {
  if (act == LQ_SILU) f(std::integral_constant<int, LQ_SILU>());
  else if (act == LQ_GELU) f(std::integral_constant<int, LQ_GELU>());
  else f(std::integral_constant<int, LQ_GELU_TANH>());
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
//
// DROP (grad_X behind dropout): the adapters' part is always formed apart, after
// the main loop, and added where the generator keeps the output. The masks spill 12
// registers of the 256 x 256 tiles, a pair's 24, around the loop that adds; nothing else
// here spills.
//
// GATED: a wave's 64 weight rows are 32 of the gate (part 0) and the same 32 of
// up (part 1), so that a lane ends with g and u of the same outputs, whose
// activation and product are taken of the float32 sums; the tile is BN / 2
// outputs wide. TWO (grad_X of a pair): one contraction over both sides' columns,
// [D_g | D_u] against the two transposed weights side by side, so that grad_X is
// written once. In both, a tile whose tokens share one adapter runs on over its
// steps of side 0, then of side 1 (a gated step multiplies its own side's rows
// alone). Measured, both weights 4096 -> 11008: 4096 tokens of four adapters of
// rank 64, g and u kept, 693 to 782 us (0.94 to 1.07 PFLOP/s), without adapters and
// kept outputs 560; 1999 tokens of eight 331 to 368; grad_X 550 to 595. One library
// product of both weights' rows takes 626 at 4096 tokens, 407 at 1999.
template <int BN, bool OUT_F32, bool BWD, bool DROP, int MODE>
__global__ __launch_bounds__(G_THREADS) void k_adapter_gemm(AdapterGemm p) {
  constexpr bool BIG = BN == 256, GATED = MODE == GEMM_GATED, APART = DROP, PAIR = MODE != GEMM_ONE;
  constexpr int NT = GATED ? BN / 2 : BN;              // outputs per tile
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
  const int64_t tiles_m = (p.M + GM - 1) / GM, tiles_n = (p.Ncols + NT - 1) / NT;
  const int64_t total = tiles_m * tiles_n;
  // XCD x (workgroups x, x + 8, ...) takes a contiguous range of tiles, the
  // token tiles inner
  const int64_t xcd = blockIdx.x % 8, per = total / 8, rem = total % 8;
  const int64_t t = xcd * per + min(xcd, rem) + blockIdx.x / 8;
  const int64_t m0 = t % tiles_m * GM, n0 = t / tiles_m * NT;

  // A load instruction of a wave fills 8 LDS rows (lane l: row l / 8, slot
  // l % 8). Part i of the token tile: rows 64 i .. of every wave's 128 (all
  // rows for BN = 128); part i of the weight tile: rows 16 CT / 2 i .. of every
  // wave's 16 CT.
  const int sub = lane >> 3, ch = (lane & 7) ^ sub;
  auto xrow = [&](int part, int q) __attribute__((always_inline)) {   // first tile row of the wave's q-th load
    const int k = wave * QX + q;       // 8-row groups 0 .. 8 QX - 1 of the part
    return BIG ? (k >> 3) * 128 + part * 64 + (k & 7) * 8 : k * 8;
  };
  auto yrow = [&](int part, int q) __attribute__((always_inline)) {
    const int k = wave * QY + q, per_wave = 16 * CT / 2 / 8;
    return (k / per_wave) * 16 * CT + part * 8 * CT + (k % per_wave) * 8;
  };
  auto wrow = [&](int part, int q) __attribute__((always_inline)) {   // row of its weight that the lane loads there
    const int k = wave * QY + q, per_wave = 16 * CT / 2 / 8;
    return min(n0 + (GATED ? (k / per_wave) * 8 * CT + (k % per_wave) * 8 : yrow(part, q)) + sub, p.Ncols - 1);
  };
  const uint16_t *px[XP][QX], *py[2][QY];
#pragma unroll
  for (int i = 0; i < XP; ++i)
#pragma unroll
    for (int q = 0; q < QX; ++q) px[i][q] = p.A + (int64_t)p.rt.perm[min(m0 + xrow(i, q) + sub, p.M - 1)] * p.lda + 8 * ch;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < QY; ++q) py[i][q] = (GATED && i ? p.Bt2 : p.Bt) + wrow(i, q) * p.ldb + 8 * ch;
  const int nk = (int)((p.Kc + GK - 1) / GK);
  // Each XCD begins at an eighth of its own of the contraction (whole steps
  // only): in step, all eight would ask for the same columns, whose rows lie a
  // power of two apart, of the same memory channels. 2 to 4 % of the kernel's
  // time; a place of its own per tile costs the tiles of an XCD the weight rows
  // and tokens that they share in its L2 (2048 tokens: 72 -> 90 us).
  const int rot = p.Kc % GK ? 0 : (int)(xcd * nk / 8);
  auto column = [&](int it) __attribute__((always_inline)) {   // first column of step it
    const int at = it + rot;
    return (int64_t)(at < nk ? at : at - nk) * GK;
  };

  // The adapters' part: an adapter's [hi | mid (| lo)] columns of the terms
  // against as many copies of Lb, in steps of 64 (columns past the last are
  // zero on both sides). Of a tile whose tokens share one adapter it is simply
  // the end of the contraction, steps nk .. nk + nl - 1 of the main loop.
  constexpr int TERMS = OUT_F32 ? 3 : 2;
  const int64_t mend = min(m0 + GM, p.M);
  // (One set: the address stands inside the load's own call. Returned from here by
  // a function, as of a pair, it costs 7 registers too many.)
  auto lora_x = [&](const Adapter& s, int kt, int i, int buf) __attribute__((always_inline)) {
    const int c = 8 * kt + ch;   // this lane's run of 8 columns
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int64_t pos = min(m0 + xrow(i, q) + sub, p.M - 1);
      uint16_t* const dst = lds.x[buf] + xrow(i, q) * GK;
      if constexpr (PAIR) load_lds16(chosen(c < s.live, s.terms + pos * s.pitch + 8 * c, p.zeros), dst);
      else load_lds16(c < s.live ? p.s[0].terms + pos * 3 * p.s[0].v.rs + 8 * c : p.zeros, dst);
    }
  };
  auto lora_y = [&](const Adapter& s, int kt, int i, int buf) __attribute__((always_inline)) {
    const int c = 8 * kt + ch;
#pragma unroll
    for (int q = 0; q < QY; ++q) {
      const int64_t n = wrow(i, q);
      uint16_t* const dst = lds.y[buf] + yrow(i, q) * GK;
      if constexpr (PAIR) load_lds16(chosen(c < s.live, s.base + n * s.stride + 8 * (c % s.runs), p.zeros), dst);
      else load_lds16(c < s.live ? s.base + n * s.stride + 8 * (c % s.runs) : p.zeros, dst);
    }
  };

  // Part i of step it into its buffer; Plain: a whole step of the base
  // contraction. Past the last step zeros, into a buffer that nobody reads any
  // more: the count of outstanding loads, on which the waits rely, stays the
  // same.
  Adapter whole{0, 0, nullptr, 8, 1, 0, 0, 0, nullptr, 0};   // the tile's one adapter, if it has one
  Adapter whole1 = whole;                                    // PAIR: side 1's
  typedef std::integral_constant<bool, true> Plain;
  typedef std::integral_constant<bool, false> Any;
  // (The adapter's rows take the place of the base's pointers at its first step,
  // for each part when it gets there: a step then adds to them, and multiplies no
  // row by a pitch.)
  auto load_x = [&](auto plain, int it, int i, int buf) __attribute__((always_inline)) {
    const uint16_t* src[QX];
    if (plain.value || it < nk) {
      const int64_t k0 = column(it);
      const bool ok = plain.value || !BWD || k0 + 8 * ch + 8 <= p.Kc;   // past the contraction: zeros (0 * NaN is not 0)
#pragma unroll
      for (int q = 0; q < QX; ++q) src[q] = ok ? px[i][q] + k0 : p.zeros;
    } else if constexpr (APART) {
#pragma unroll
      for (int q = 0; q < QX; ++q) src[q] = p.zeros;
    } else if constexpr (!PAIR) {
      lora_x(whole, it - nk, i, buf);
      return;
    } else {
      const int from = PAIR && it >= nk + whole.steps ? nk + whole.steps : nk;
      const bool second = from != nk;
      if (it == from) {
        const uint16_t* const terms = PAIR && second ? whole1.terms : whole.terms;
        const int64_t pitch = PAIR && second ? whole1.pitch : whole.pitch;
#pragma unroll
        for (int q = 0; q < QX; ++q) px[i][q] = terms + min(m0 + xrow(i, q) + sub, p.M - 1) * pitch;
      }
      const int c = 8 * (it - from) + ch, live = PAIR && second ? whole1.live : whole.live;
#pragma unroll
      for (int q = 0; q < QX; ++q) src[q] = c < live ? px[i][q] + 8 * c : p.zeros;
    }
#pragma unroll
    for (int q = 0; q < QX; ++q) load_lds16(src[q], lds.x[buf] + xrow(i, q) * GK);
  };
  auto load_y = [&](auto plain, int it, int i, int buf) __attribute__((always_inline)) {
    const uint16_t* src[QY];
    if (plain.value || it < nk) {
      const int64_t k0 = column(it);
#pragma unroll
      for (int q = 0; q < QY; ++q) src[q] = py[i][q] + k0;
    } else if constexpr (APART) {
#pragma unroll
      for (int q = 0; q < QY; ++q) src[q] = p.zeros;
    } else if constexpr (!PAIR) {
      lora_y(whole, it - nk, i, buf);
      return;
    } else {
      const int from = PAIR && it >= nk + whole.steps ? nk + whole.steps : nk;
      const bool second = from != nk;
      if (it == from) {
        const uint16_t* const base = PAIR && second ? whole1.base : whole.base;
        const int64_t stride = PAIR && second ? whole1.stride : whole.stride;
#pragma unroll
        for (int q = 0; q < QY; ++q) py[i][q] = base + wrow(i, q) * stride;
      }
      const int c = 8 * (it - from) + ch, live = PAIR && second ? whole1.live : whole.live;
      const int run = c % (PAIR && second ? whole1.runs : whole.runs);
      const bool in = c < live && (!GATED || second == (i == 1));   // GATED: the side's own weight rows
#pragma unroll
      for (int q = 0; q < QY; ++q) src[q] = in ? py[i][q] + 8 * run : p.zeros;
    }
#pragma unroll
    for (int q = 0; q < QY; ++q) load_lds16(src[q], lds.y[buf] + yrow(i, q) * GK);
  };

  f32x4_t acc[CT][RT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  u32x4_t fx[2][4], fy[2][2][CT / 2];   // [k half][tile], weight side [part][k half][tile]
  const int slot0 = 8 * (lg ^ (li & 7)), slot1 = 8 * ((4 + lg) ^ (li & 7));
  const int ox = (wm * 16 * RT + li) * GK, oy = (wn * 16 * CT + li) * GK;
  auto read_x = [&](int i, int buf) __attribute__((always_inline)) {
    const uint16_t* b = lds.x[buf] + ox + i * 64 * GK;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      fx[0][r] = ld16(b + 16 * r * GK + slot0);
      fx[1][r] = ld16(b + 16 * r * GK + slot1);
    }
  };
  auto read_y = [&](int i, int buf) __attribute__((always_inline)) {
    const uint16_t* b = lds.y[buf] + oy + i * 8 * CT * GK;
#pragma unroll
    for (int c = 0; c < CT / 2; ++c) {
      fy[i][0][c] = ld16(b + 16 * c * GK + slot0);
      fy[i][1][c] = ld16(b + 16 * c * GK + slot1);
    }
  };
  auto end_memory = [&]() __attribute__((always_inline)) {   // the fragments have arrived: a part may be refilled after the barrier
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](int xi, int yi, bool on) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
    if (on)
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
  Adapter next = adapter_at<TERMS>(p, 0, m0, mend);
  if constexpr (!APART) {
    const bool one = next.steps && next.hi == mend;
    whole = next;
    whole.steps = one ? next.steps : 0;
    whole.live = one ? next.live : 0;
    if constexpr (PAIR) {
      whole1 = adapter_at<TERMS>(p, 1, m0, mend);
      whole1.steps = one ? whole1.steps : 0;
      whole1.live = one ? whole1.live : 0;
    }
  }
  const int nsteps = nk + whole.steps + (PAIR ? whole1.steps : 0);
  int it = 0, buf = 0;
  auto step = [&](auto plain) __attribute__((always_inline)) {
    // GATED, a side's adapter: its own weight rows alone (a zero against an infinite t is NaN)
    const bool gate = plain.value || !GATED || it < nk + whole.steps, up = plain.value || !GATED || it < nk || !gate;
    if constexpr (BIG) {
      read_x(0, buf);
      read_y(0, buf);
      load_x(plain, it + 1, 1, buf ^ 1);
      wait_vm<10>();          // Y1 of this step
      end_memory();
      multiply(0, 0, gate);
      read_y(1, buf);
      load_x(plain, it + 2, 0, buf);
      wait_vm<10>();          // X1 of this step
      end_memory();
      multiply(0, 1, up);
      read_x(1, buf);
      load_y(plain, it + 2, 0, buf);
      end_memory();
      multiply(1, 1, up);
      load_y(plain, it + 2, 1, buf);
      wait_vm<10>();          // X0 and Y0 of the next step
      end_memory();
      multiply(1, 0, gate);
      buf ^= 1;
    } else {
      const int b2 = buf == 0 ? 2 : buf - 1;   // buffer of step it + 2
      read_x(0, buf);
      read_y(0, buf);
      load_x(plain, it + 2, 0, b2);
      end_memory();
      multiply(0, 0, gate);
      read_y(1, buf);
      load_y(plain, it + 2, 0, b2);
      load_y(plain, it + 2, 1, b2);
      wait_vm<QX + 2 * QY>();   // the next step
      end_memory();
      multiply(0, 1, up);
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

  const int64_t pw = m0 + wm * 16 * RT, cw = n0 + wn * (GATED ? 8 : 16) * CT;

  // A tile of several adapters (APART: of any): one after the other, each one's
  // products formed apart and added to its own tokens' columns alone, so that an
  // adapter's infinities and NaN stay with its tokens (GATED: and with its own
  // side's weight rows). APART: without a branch around it, and in one loop for
  // both sides: the compiler would hold the sums twice.
  if (APART || (!whole.steps && next.steps)) {
    Kept<RT> keep0{}, keep1{};
    if constexpr (DROP) keep0 = kept_outputs<CT, RT>(p.s[0].drop, p.rt.perm, p.M, p.Ncols, pw, cw);
    if constexpr (DROP && MODE == GEMM_TWO) keep1 = kept_outputs<CT, RT>(p.s[1].drop, p.rt.perm, p.M, p.Ncols, pw, cw);
    Adapter cur = next;
    int kt = 0;
    auto load = [&](int b) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < XP; ++i) lora_x(cur, kt, i, b);
#pragma unroll
      for (int i = 0; i < 2; ++i) lora_y(cur, kt, i, b);
    };
    ring_barrier<0>();   // everyone has read the last step
    load(0);   // (APART: of a tile without adapters a step of zeros, no token's)
    int b = 0;
    do {
      const int64_t lo = cur.lo, hi = !APART || cur.steps ? cur.hi : cur.lo;
      const int side = cur.side;
      if (++kt >= cur.steps) {
        cur = adapter_at<TERMS>(p, side, cur.hi, mend);
        if (MODE != GEMM_ONE && !cur.steps && !side) cur = adapter_at<TERMS>(p, 1, m0, mend);
        kt = 0;
      }
      ring_barrier<0>();   // this step has landed, and the other buffer is read
      if (cur.steps) load(b ^ 1);
      read_y(0, b);
      read_y(1, b);
      Kept<RT> keep = keep0;
      if constexpr (DROP && MODE == GEMM_TWO)
#pragma unroll
        for (int i = 0; i < RT / 2; ++i) keep.w[i] = side ? keep1.w[i] : keep0.w[i];
      if constexpr (DROP)   // or each bit's mask would be formed before the loop and held
#pragma unroll
        for (uint32_t& w : keep.w) asm volatile("" : "+v"(w));
#pragma unroll
      for (int xi = 0; xi < XP; ++xi) {
        read_x(xi, b);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t first = pw + 16 * (xi * 4 + r), pos = first + li;
          const bool mine = pos >= lo && pos < hi;
          // A tile with none of these tokens: left out where the registers allow the
          // branch (elsewhere it costs 8 to 24 more of them spilled).
          if (MODE != GEMM_ONE && !DROP && (first >= hi || first + 16 <= lo)) continue;
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            if (GATED && side != c / (CT / 2)) continue;
            f32x4_t d = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < 2; ++u)
              d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(fy[c / (CT / 2)][u][c % (CT / 2)]), as_bf16x8(fx[u][r]),
                                                          d, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int rt = xi * 4 + r;
              const float add = DROP ? kept_value(d[e], keep.w[rt / 2], 8 * c + 4 * (rt % 2) + e) : d[e];
              acc[c][xi * 4 + r][e] += mine ? add : 0.0f;
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      b ^= 1;
    } while (cur.steps);
  }

  // lane: token position pw + 16 rt + li, outputs cw + 16 ct + 4 lg + [0, 4)
  if constexpr (GATED) {
    with_act(p.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int64_t pos = pw + 16 * rt + li;
        if (pos >= p.M) continue;
        const int64_t row = (int64_t)p.rt.perm[pos] * p.Ncols;
#pragma unroll
        for (int ct = 0; ct < CT / 2; ++ct)
          store_gated4<OUT_F32, decltype(act)::value>(p, row, cw + 16 * ct + 4 * lg, acc[ct][rt], acc[ct + CT / 2][rt]);
      }
    });
  } else {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int64_t pos = pw + 16 * rt + li;
      if (pos >= p.M) continue;
      const int64_t row = (int64_t)p.rt.perm[pos] * p.Ncols;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) store4<OUT_F32>(p, p.out, row, cw + 16 * ct + 4 * lg, acc[ct][rt]);
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
constexpr int S_STEPS = SM * 6;   // of a side: an adapter per token, 3 terms of rank 128

struct SmallStep {
  const uint16_t* base;           // Lb
  uint8_t runs, live, first;      // of Lb: runs of 8 columns; of all terms; the step's first
  uint8_t lo, hi;                 // its positions of the tile
  uint8_t side;
};

template <int GROUPS, bool OUT_F32, bool BWD, bool DROP, int MODE>
__global__ __launch_bounds__(S_THREADS * GROUPS, 2) void k_adapter_gemm_small(AdapterGemm p) {
  constexpr int TERMS = OUT_F32 ? 3 : 2, SIDES = MODE == GEMM_ONE ? 1 : 2;
  constexpr bool GATED = MODE == GEMM_GATED;   // c = 0: gate, c = 1: up
  constexpr int NT = GATED ? SN / 2 : SN;      // outputs per tile
  struct __attribute__((aligned(16))) Lds {
    uint16_t x[GROUPS][S_RING][SM * GK];
    uint16_t y[GROUPS][S_RING][SN * GK];
    SmallStep steps[SIDES * S_STEPS];
    int total;
  };
  __shared__ Lds lds;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int group = wave >> 2, w4 = wave & 3;
  const int li = lane & 15, lg = lane >> 4;
  const int wn = w4 & 1, wm = w4 >> 1;
  const int64_t tiles_m = (p.M + SM - 1) / SM, tiles_n = (p.Ncols + NT - 1) / NT;
  const int64_t total = tiles_m * tiles_n;
  const int64_t xcd = blockIdx.x % 8, per = total / 8, rem = total % 8;
  const int64_t t = xcd * per + min(xcd, rem) + blockIdx.x / 8;
  const int64_t m0 = t % tiles_m * SM, n0 = t / tiles_m * NT, mend = min(m0 + SM, p.M);

  const int sub = lane >> 3, ch = (lane & 7) ^ sub;
  const uint16_t *px[2], *py[2], *pt[SIDES][2];
  int64_t ny[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = (w4 * 2 + q) * 8 + sub;
    const int64_t pos = min(m0 + row, p.M - 1);
    px[q] = p.A + (int64_t)p.rt.perm[pos] * p.lda + 8 * ch;
#pragma unroll
    for (int sd = 0; sd < SIDES; ++sd) pt[sd][q] = p.s[sd].terms + pos * 3 * p.s[sd].v.rs;
    // GATED: row 32 wn + 16 c + i of the tile is row 16 wn + i of weight c
    ny[q] = min(n0 + (GATED ? (row >> 5) * 16 + (row & 15) : row), p.Ncols - 1);
    py[q] = (GATED && (w4 & 1) ? p.Bt2 : p.Bt) + ny[q] * p.ldb + 8 * ch;
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
    SmallStep st{nullptr, 1, 0, 0, 0, 0, 0};
    if (it < steps) st = lds.steps[it - nk];
    const int c = st.first + ch;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint16_t *const t0 = pt[0][q], *const t1 = pt[SIDES - 1][q];
      load_lds16(c < st.live ? (SIDES == 2 && st.side ? t1 : t0) + 8 * c : p.zeros,
                 rx[buf] + (w4 * 2 + q) * 8 * GK);
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
    const bool leads = valid && a < p.s[0].v.n && ((starts >> lane) & 1);
    const uint64_t above = lane < 63 ? starts >> (lane + 1) : 0;
    const int hi = above ? lane + __ffsll((unsigned long long)above) : SM;
    int total = 0;
    auto list = [&](const lq_adapter* tab, const uint16_t* lt, int side) {
      const lq_adapter ad = tab[leads ? a : 0];
      const int runs = (ad.r + 7) >> 3, live = TERMS * runs, count = leads ? (live + 7) >> 3 : 0;
      int first = total;
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        const uint64_t one = __ballot((count >> b) & 1);
        first += (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(one >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)one, 0)) << b;
        total += __popcll(one) << b;
      }
      const uint16_t* base = !p.lt_all && ad.r % 8 == 0 ? ad.B : lt + p.Ncols * ad.row8;
      for (int k = 0; k < count; ++k)
        lds.steps[first + k] = SmallStep{base, (uint8_t)runs, (uint8_t)live, (uint8_t)(8 * k), (uint8_t)lane, (uint8_t)hi, (uint8_t)side};
    };
    if (MODE == GEMM_ONE || p.s[0].v.n) list(p.s[0].v.tab, p.s[0].lt, 0);   // (a pair may be without sets)
    if (MODE != GEMM_ONE && p.s[0].v.n) list(p.s[1].v.tab, p.s[1].lt, 1);
    if (lane == 0) lds.total = total;
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
  uint32_t keep[SIDES];
#pragma unroll
  for (int sd = 0; sd < SIDES; ++sd) {
    keep[sd] = ~0u;
    if (DROP && steps > nk)
      keep[sd] = kept_outputs<2, 2>(p.s[sd].drop, p.rt.perm, p.M, p.Ncols, m0 + wm * 32, n0 + wn * 32).w[0];
  }
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
      const int side = SIDES == 2 ? uniform(lds.steps[it - nk].side) : 0;
      const uint32_t keep0 = keep[0], keep1 = keep[SIDES - 1], kept = SIDES == 2 && side ? keep1 : keep0;
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
          for (int e = 0; e < 4; ++e) {
            const float add = DROP ? kept_value(d[e], kept, 8 * c + 4 * r + e) : d[e];
            acc[c][r][e] += mine && (!GATED || side == c) ? add : 0.0f;
          }
        }
      }
    }
  }
  wait_vm<0>();   // the loads past the last step
  if constexpr (GROUPS == 2) {   // group g finishes the weight rows of c = g (GATED: the tokens of r = g), group 0's sum first
    ring_barrier<0>();   // the tiles are read: the sums take their place
    f32x4_t* sum = reinterpret_cast<f32x4_t*>(lds.x) + 128 * w4 + lane;   // [group][w4][k][lane]
#pragma unroll
    for (int k = 0; k < 2; ++k)
      sum[512 * group + 64 * k] = GATED ? (group ? acc[k][0] : acc[k][1]) : (group ? acc[0][k] : acc[1][k]);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const f32x4_t other = sum[512 * (1 - group) + 64 * k];
      if (GATED) {
        if (group) acc[k][1] = other + acc[k][1];
        else acc[k][0] = acc[k][0] + other;
      } else {
        if (group) acc[1][k] = other + acc[1][k];
        else acc[0][k] = acc[0][k] + other;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t pos = m0 + wm * 32 + 16 * r + li;
    if (pos >= p.M) continue;
    const int64_t row = (int64_t)p.rt.perm[pos] * p.Ncols;
    if constexpr (GATED) {
      if (GROUPS == 1 || r == group)
        with_act(p.act, [&](auto act) __attribute__((always_inline)) {
          store_gated4<OUT_F32, decltype(act)::value>(p, row, n0 + wn * 16 + 4 * lg, acc[0][r], acc[1][r]);
        });
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (GROUPS == 1 || c == group) store4<OUT_F32>(p, p.out, row, n0 + wn * 32 + 16 * c + 4 * lg, acc[c][r]);
    }
  }
}

// 64 x 64 tiles through LDS; columns past N, up to a multiple of 64, are zero.
__global__ __launch_bounds__(256) void k_transpose_weight(const uint16_t* w, int64_t N, int64_t K, int64_t ldb, uint16_t* out,
                                                          const uint16_t* w2, uint16_t* out2) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[64][72];   // [n][k]
  const int64_t n0 = (int64_t)blockIdx.x * 64, k0 = (int64_t)blockIdx.y * 64;   // K % 64 == 0
  if (blockIdx.z) {
    w = w2;
    out = out2;
  }
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
    *reinterpret_cast<u32x4_t*>(out + (k0 + k) * ldb + n0 + c) = v;   // the row stride covers the tile
  }
}

#define LQ_GEMM_MODES(KERNEL, SIZE)                                                                                \
  do {                                                                                                             \
    const bool drops = g.s[0].drop.T || g.s[1].drop.T;                                                             \
    if (g.mode == GEMM_GATED && g.out_f32) hipLaunchKernelGGL((KERNEL<SIZE, true, false, false, GEMM_GATED>), grid, block, 0, s, g); \
    else if (g.mode == GEMM_GATED) hipLaunchKernelGGL((KERNEL<SIZE, false, false, false, GEMM_GATED>), grid, block, 0, s, g); \
    else if (g.mode == GEMM_TWO && drops) hipLaunchKernelGGL((KERNEL<SIZE, false, true, true, GEMM_TWO>), grid, block, 0, s, g); \
    else if (g.mode == GEMM_TWO) hipLaunchKernelGGL((KERNEL<SIZE, false, true, false, GEMM_TWO>), grid, block, 0, s, g); \
    else if (g.lt_all && drops) hipLaunchKernelGGL((KERNEL<SIZE, false, true, true, GEMM_ONE>), grid, block, 0, s, g); \
    else if (g.lt_all) hipLaunchKernelGGL((KERNEL<SIZE, false, true, false, GEMM_ONE>), grid, block, 0, s, g);      \
    else if (g.out_f32) hipLaunchKernelGGL((KERNEL<SIZE, true, false, false, GEMM_ONE>), grid, block, 0, s, g);     \
    else hipLaunchKernelGGL((KERNEL<SIZE, false, false, false, GEMM_ONE>), grid, block, 0, s, g);                   \
  } while (0)

// Weight rows per output of a tile: a gated tile's are shared by two weights.
int64_t tile_cols(const AdapterGemm& g, int64_t bn) { return g.mode == GEMM_GATED ? bn / 2 : bn; }

template <int BN>
hipError_t launch_tile(const AdapterGemm& g, hipStream_t s) {
  const int64_t cols = tile_cols(g, BN), tiles = ((g.M + GM - 1) / GM) * ((g.Ncols + cols - 1) / cols);
  LQ_DASSERT(tiles > 0 && tiles < (int64_t(1) << 31));
  const dim3 grid((unsigned)tiles), block(G_THREADS);
  LQ_GEMM_MODES(k_adapter_gemm, BN);
  return hipGetLastError();
}

template <int GROUPS>
hipError_t launch_small(const AdapterGemm& g, int64_t tiles, hipStream_t s) {
  LQ_DASSERT(tiles > 0 && tiles < (int64_t(1) << 31));
  const dim3 grid((unsigned)tiles), block(S_THREADS * GROUPS);
  LQ_GEMM_MODES(k_adapter_gemm_small, GROUPS);
  return hipGetLastError();
}
#undef LQ_GEMM_MODES

}  // namespace

hipError_t launch_adapter_gemm(const AdapterGemm& g, hipStream_t s) {
  LQ_DASSERT(g.M > 0 && g.Ncols > 0 && g.Kc > 0 && g.Kc % 8 == 0 && g.ldb % 64 == 0 && g.ldb >= g.Kc && g.lda >= g.Kc);
  LQ_DASSERT(g.mode == GEMM_ONE || g.Kc % 64 == 0);
  // Rounds of a chip full of tiles times a tile's time per step, in us as
  // measured over K = 4096: 1.7 (256 x 256), 1.05 (256 x 128) and for 64 x 64,
  // two workgroups per CU, 0.3 where the tiles number more than the CUs. (Fewer
  // of them always win: 0.2.) Of a pair these are slower: 0.45 where g and u are formed,
  // whose tile has half the outputs (4096 -> 11008, calls of 64 x 64 / 256 x 128 / 256 x
  // 256: 200 tokens 146 / 123 / 152 us, 400 193 / 183 / 157, 700 277 / 238 / 245; 1024 ->
  // 2048, 1000 tokens 43 / 46 / 58, 1500 52 / 45 / 56), 0.7 in grad_X, whose contraction is long
  // (512 tokens 321 / 389 / 526, 1000 529 / 423 / 550).
  auto tiles = [&](int64_t m, int64_t n) {
    const int64_t cols = tile_cols(g, n);
    return ((g.M + m - 1) / m) * ((g.Ncols + cols - 1) / cols);
  };
  auto cost = [&](int64_t count, int64_t slots, double us) { return (double)((count + slots - 1) / slots) * us; };
  const int64_t small = tiles(SM, SN);
  const double c256 = cost(tiles(256, 256), 256, 1.7), c128 = cost(tiles(256, 128), 256, 1.05), c64 = cost(small, 512, g.mode == GEMM_GATED ? 0.45 : g.mode == GEMM_TWO ? 0.7 : 0.3);
  if (small <= 256) return launch_small<2>(g, small, s);
  if (c64 < c128 && c64 < c256) return launch_small<1>(g, small, s);
  return c256 <= c128 ? launch_tile<256>(g, s) : launch_tile<128>(g, s);
}

hipError_t launch_transpose_weight(const uint16_t* w, int64_t N, int64_t K, int64_t ldb, uint16_t* out, const uint16_t* w2,
                                   uint16_t* out2, hipStream_t s) {
  LQ_DASSERT(K % 64 == 0 && ldb % 64 == 0 && ldb >= N);
  hipLaunchKernelGGL(k_transpose_weight, dim3((unsigned)((N + 63) / 64), (unsigned)(K / 64), w2 ? 2u : 1u), dim3(256), 0, s, w, N,
                     K, ldb, out, w2, out2);
  return hipGetLastError();
}

}  // namespace lq
