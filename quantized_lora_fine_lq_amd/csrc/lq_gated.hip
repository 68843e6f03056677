// The gated pair's backward between its two ends: from G, g and u the gradients
//   dg = G u act'(g),  du = G act(g)
// and their skinny products with the adapters, u_g = B_g^T dg, u_u = B_u^T du,
// dB_g = s dg^T t_g, dB_u = s du^T t_u.
//
// dg and du are formed again where they are used, from the three bfloat16
// tensors: that is 6 bytes an element read against 12 if their three bfloat16
// terms were kept. They enter the adapters' products as those terms (all 24
// bits, since dA and dB are float32); grad_X's large product takes the first
// term alone, its bfloat16 rounding, as gradients in bfloat16 would enter it: the
// error of its rounded result, relative to 64 bits and over all elements, is 0.0023
// where 0.0017 is the rounding of the result itself. A second term would double the
// product, 580 of 945 us at 4096 tokens.
#include <algorithm>

#include "lq_act.h"
#include "lq_adapters.h"
#include "lq_device.h"
#include "lq_route.h"

namespace lq {
namespace {

// 8 elements' dg and du.
template <int ACT>
__device__ __forceinline__ void gate_grads(u32x4_t G, u32x4_t g, u32x4_t u, float (&dg)[8], float (&du)[8]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t Gw = G[w], gw = g[w], uw = u[w];
    const ActPair a0 = act_pair<ACT>(bf16lo_to_f32(gw)), a1 = act_pair<ACT>(bf16hi_to_f32(gw));
    const float G0 = bf16lo_to_f32(Gw), G1 = bf16hi_to_f32(Gw);
    dg[2 * w] = G0 * bf16lo_to_f32(uw) * a0.slope;
    dg[2 * w + 1] = G1 * bf16hi_to_f32(uw) * a1.slope;
    du[2 * w] = G0 * a0.value;
    du[2 * w + 1] = G1 * a1.value;
  }
}
// dg's and du's three bfloat16 terms. Below the largest bfloat16 the terms are
// the plain ones, hi = bf16(v), mid = bf16(v - hi), lo = bf16(v - hi - mid); a
// wave that holds a larger value (or an infinity) takes them as take_bf16_terms
// does. A NaN gives NaN either way.
__device__ __forceinline__ void split_grads(float (&d)[2][8], u32x4_t (&t)[2][3]) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(d[0][e]), fabsf(d[1][e])));
  if (__ballot(top >= 0x1.fep127f)) {   // 0x1.fep127: the largest bfloat16
#pragma unroll
    for (int sd = 0; sd < 2; ++sd)
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int w = 0; w < 4; ++w) t[sd][k][w] = take_bf16_terms(d[sd][2 * w], d[sd][2 * w + 1]);
    return;
  }
#pragma unroll
  for (int sd = 0; sd < 2; ++sd)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float a = d[sd][2 * w], b = d[sd][2 * w + 1];
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t x = pack_bf16x2(a, b);
        a -= bf16lo_to_f32(x);
        b -= bf16hi_to_f32(x);
        t[sd][k][w] = x;
      }
    }
}

// ===========================================================================
// Row form: 64 routed tokens of one adapter (or of none: D alone) per workgroup
// and share of the columns, 16 a wave, in steps of 64 columns. A lane forms dg
// and du of 8 columns of a token in registers, which is the matrix product's
// operand; as soon as a half step's G, g and u are used, the next step's are
// asked for into the same registers. B^T's rows pass through LDS, double
// buffered, loaded a step ahead.
//
// 4096 tokens, N = 11008, four adapters of rank 64: 139 us for 450 MB (270 read,
// 180 of D written), 3.2 TB/s; bound by the chain of a step (loads, activations,
// splits, products) at three waves a SIMD, its vector units 30 % busy. Loads two
// steps ahead in registers of their own left two waves a SIMD: 161 us; eight
// waves a workgroup spilled: 264.
// ===========================================================================
constexpr int GD_M = 64, GD_K = 64;

struct GatedDown {
  GatedGrad gr;
  AdapterView v[2];
  const uint16_t* bt[2];
  float* part[2];
  uint16_t* D;
  int64_t Np;
};

template <int JT, int ACT>
__global__ __launch_bounds__(256, JT <= 4 ? 3 : 2) void k_gated_down(GatedDown p, int64_t M, Route rt) {
  constexpr int ROWS = 16 * JT, PW = JT;                                  // 16-byte pieces of both sides' B^T per thread
  __shared__ __attribute__((aligned(16))) uint16_t sW[2][2][ROWS * GD_K];       // [buffer][side]
  Item it;
  if (!find_item(rt.off, p.v[0].n + 1, GD_M, (int)blockIdx.x, it)) return;
  const bool has = it.seg < p.v[0].n;
  const int64_t N = p.gr.N;
  int r[2] = {1, 1};
  const uint16_t* bt[2] = {nullptr, nullptr};
  if (has) {
#pragma unroll
    for (int sd = 0; sd < 2; ++sd) {
      const lq_adapter ad = p.v[sd].tab[it.seg];
      r[sd] = min(ad.r, ROWS);
      bt[sd] = p.bt[sd] + N * ad.row8;
    }
  }
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int all = (int)(p.Np / GD_K), per = (all + gridDim.y - 1) / gridDim.y;
  const int s0 = min(all, (int)blockIdx.y * per), s1 = min(all, s0 + per);
  const int row = 16 * wave + li;
  const bool live = row < it.count;
  const int64_t token = rt.perm[it.start + min(row, it.count - 1)];
  const uint16_t *pG = p.gr.G + token * N, *pg = p.gr.g + token * N, *pu = p.gr.u + token * N;
  u32x4_t qG[2], qg[2], qu[2], w[PW];
  auto load = [&](int s, int h) __attribute__((always_inline)) {
    const int64_t c = GD_K * (int64_t)s + 32 * h + 8 * lg, o = c < N ? c : 0;   // N % 8 == 0
    qG[h] = ld16(pG + o);
    qg[h] = ld16(pg + o);
    qu[h] = ld16(pu + o);
  };
  // piece i: side, row and chunk of 8 columns
  auto load_w = [&](int s) __attribute__((always_inline)) {
    if (!has) return;
#pragma unroll
    for (int k = 0; k < PW; ++k) {
      const int i = threadIdx.x + 256 * k, sd = i / (8 * ROWS), j = (i >> 3) % ROWS;
      const int64_t c = GD_K * (int64_t)s + 8 * (i & 7);
      w[k] = ld16((sd ? bt[1] : bt[0]) + min(j, (sd ? r[1] : r[0]) - 1) * N + (c < N ? c : 0));
    }
  };
  f32x4_t acc[2][JT];
#pragma unroll
  for (int sd = 0; sd < 2; ++sd)
#pragma unroll
    for (int c = 0; c < JT; ++c) acc[sd][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int slot[2] = {8 * (lg ^ (li & 7)), 8 * ((4 + lg) ^ (li & 7))};
  if (s0 < s1) {
    load(s0, 0);
    load(s0, 1);
    load_w(s0);
  }
  for (int s = s0; s < s1; ++s) {
    uint16_t(*buf)[ROWS * GD_K] = sW[(s - s0) & 1];
    const int next = min(s + 1, s1 - 1);
    // Past the last column both operands are zero: set here, not where they are
    // loaded, which would wait for the loads.
    const bool tail = GD_K * (int64_t)(s + 1) > N;
    const u32x4_t none = {0u, 0u, 0u, 0u};
    if (has) {
#pragma unroll
      for (int k = 0; k < PW; ++k) {
        const int i = threadIdx.x + 256 * k, sd = i / (8 * ROWS), j = (i >> 3) % ROWS;
        if (tail && GD_K * (int64_t)s + 8 * (i & 7) >= N) w[k] = none;
        *reinterpret_cast<u32x4_t*>(buf[sd] + j * GD_K + 8 * ((i & 7) ^ (j & 7))) = w[k];
      }
      // (one barrier a step: the buffer written at step s + 1 was read at s - 1, and
      // those reads are done before a wave reaches step s's barrier)
      lds_barrier();
    }
    load_w(next);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (tail && GD_K * (int64_t)s + 32 * h + 8 * lg >= N) qG[h] = qg[h] = qu[h] = none;
      float d[2][8];
      gate_grads<ACT>(qG[h], qg[h], qu[h], d[0], d[1]);
      load(next, h);
      u32x4_t t[2][3];
      split_grads(d, t);
      if (p.D && live) {
        uint16_t* o = p.D + token * 2 * p.Np + GD_K * (int64_t)s + 32 * h + 8 * lg;
        *reinterpret_cast<u32x4_t*>(o) = t[0][0];
        *reinterpret_cast<u32x4_t*>(o + p.Np) = t[1][0];
      }
      if (!has) continue;
#pragma unroll
      for (int sd = 0; sd < 2; ++sd) {
        u32x4_t b[JT];
#pragma unroll
        for (int c = 0; c < JT; ++c) b[c] = ld16(buf[sd] + (16 * c + li) * GD_K + slot[h]);
#pragma unroll
        for (int k = 0; k < 3; ++k)   // (the chains of one sum are JT products apart)
#pragma unroll
          for (int c = 0; c < JT; ++c)
            acc[sd][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(t[sd][k]), as_bf16x8(b[c]), acc[sd][c], 0, 0, 0);
      }
    }
  }
  if (!has) return;
  // lane: tokens 16 wave + 4 lg + e, row 16 c + li of the adapter
#pragma unroll
  for (int sd = 0; sd < 2; ++sd) {
    float* part = p.part[sd] + (int64_t)blockIdx.y * M * p.v[sd].rs;
#pragma unroll
    for (int c = 0; c < JT; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = 16 * wave + 4 * lg + e, j = 16 * c + li;
        if (m < it.count && j < r[sd]) part[(int64_t)(it.start + m) * p.v[sd].rs + j] = acc[sd][c][e];
      }
  }
}

// ===========================================================================
// Column form of both sides: one workgroup of eight waves per 128 columns and
// run of at most `rows` sorted positions, 32 tokens a step; waves 0 to 3 take dg
// with the gate's t, 4 to 7 du with up's, 32 columns each. The terms of dg and
// du lie in LDS with tokens as rows and are read transposed, as the terms of s t.
// Of the nine products of terms the six whose places add up to at most the third
// are formed: the others are below 2^-24 of the value.
//
// The size above: 127 us for 270 MB, 2.1 TB/s, at 49 % of the vector units, which
// form every dg and du again, once for both sides' products (eight waves, two
// workgroups a CU).
// ===========================================================================
constexpr int GC_COLS = 128, GC_THREADS = 512;

// lane's 8 values k = 8 lg + [0, 8) of column c0 + li (c0 a multiple of 16) of
// rows of 128 whose 16-byte chunks lie at chunk ^ 2 (row % 4): the four rows that
// a transposing read takes at once hit distinct banks.
__device__ __forceinline__ u32x4_t tr_frag_swizzled(const uint16_t* base, int c0, int li, int lg) {
  typedef __bf16 v4b __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) v4b* lds_p;
  const int row = 8 * lg + (li >> 2), chunk = (c0 >> 3) + ((li & 3) >> 1);
  const uint16_t* p = base + row * GC_COLS + 8 * (chunk ^ (2 * (li >> 2))) + 4 * (li & 1);   // row % 4 = li >> 2, also 4 rows on
  const u32x2_t lo = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_p)p));
  const u32x2_t hi = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_p)(p + 4 * GC_COLS)));
  return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

template <int JT, int ACT>
__global__ __launch_bounds__(GC_THREADS, JT <= 4 ? 4 : 2) void k_gated_col(GatedGrad gr, ColReq r0, ColReq r1, int rows, Route rt) {
  constexpr int PP = 16 * JT + 16;
  constexpr int PQ = (2 * 3 * 32 * 2 * JT + GC_THREADS - 1) / GC_THREADS;   // 16-byte pieces of both sides' t per thread
  __shared__ __attribute__((aligned(16))) uint16_t sQ[2][3][32 * GC_COLS];
  __shared__ __attribute__((aligned(16))) uint16_t sP[2][3 * 32 * PP];
  Item it;
  if (!find_item(rt.off, r0.v.n, rows, (int)blockIdx.y, it)) return;
  const lq_adapter ad0 = r0.v.tab[it.seg], ad1 = r1.v.tab[it.seg];
  const int r80 = (min(ad0.r, 16 * JT) + 7) & ~7, r81 = (min(ad1.r, 16 * JT) + 7) & ~7;
  const int64_t N = gr.N, c0 = (int64_t)blockIdx.x * GC_COLS;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int side = uniform(wave >> 2), quarter = wave & 3;
  const int qc = 8 * (threadIdx.x & 15), qr = threadIdx.x >> 4;   // 8 columns of token qr
  const bool qin = c0 + qc < N;                                   // N % 8 == 0
  u32x4_t xG, xg, xu, xp[PQ];
  int tok;
  auto tokens = [&](int mb) { tok = rt.perm[it.start + min(mb + qr, it.count - 1)]; };
  // piece k of t: (side and term) of a token row and 8 of its columns, at `from` in
  // the run's first 32 rows, to `to` in LDS (both sides' tiles in one array)
  const uint16_t* from[PQ];
  int prow[PQ], to[PQ];
  bool pin[PQ];
#pragma unroll
  for (int k = 0; k < PQ; ++k) {
    const int i = threadIdx.x + GC_THREADS * k, c8 = i % (2 * JT), t = min(i / (64 * JT), 5);
    const bool up = t >= 3;
    const int term = up ? t - 3 : t, r8 = up ? r81 : r80;
    prow[k] = (i / (2 * JT)) % 32;
    pin[k] = 8 * c8 < r8;
    from[k] = (up ? r1.terms : r0.terms) + (int64_t)(it.start + min(prow[k], it.count - 1)) * 3 * (up ? r1.v.rs : r0.v.rs) +
              (pin[k] ? term * r8 + 8 * c8 : 0);
    to[k] = i < 384 * JT ? (32 * t + prow[k]) * PP + 8 * c8 : -1;
  }
  auto load = [&](int mb) {
    const int64_t o = (int64_t)tok * N + (qin ? c0 + qc : 0);
    xG = ld16(gr.G + o);
    xg = ld16(gr.g + o);
    xu = ld16(gr.u + o);
#pragma unroll
    for (int k = 0; k < PQ; ++k) {   // (past the run its first rows again)
      const int64_t step = (int64_t)mb * 3 * ((threadIdx.x + GC_THREADS * k) / (192 * JT) ? r1.v.rs : r0.v.rs);
      xp[k] = ld16(from[k] + (mb + prow[k] < it.count ? step : 0));
    }
  };
  auto store = [&](int mb) {
    const u32x4_t none = {0u, 0u, 0u, 0u};
    const bool whole = mb + 32 <= it.count && c0 + GC_COLS <= N;   // others are zero past the run and the last column
    float d[2][8];
    gate_grads<ACT>(xG, xg, xu, d[0], d[1]);
    u32x4_t t3[2][3];
    split_grads(d, t3);
    if (!whole && !(qin && mb + qr < it.count))   // no neighbour's infinity enters
#pragma unroll
      for (int sd = 0; sd < 2; ++sd)
#pragma unroll
        for (int k = 0; k < 3; ++k) t3[sd][k] = none;
#pragma unroll
    for (int sd = 0; sd < 2; ++sd)
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x4_t*>(sQ[sd][k] + qr * GC_COLS + (qc ^ (16 * (qr & 3)))) = t3[sd][k];
#pragma unroll
    for (int k = 0; k < PQ; ++k) {
      if (!pin[k] || mb + prow[k] >= it.count) xp[k] = none;
      if (to[k] >= 0) *reinterpret_cast<u32x4_t*>(&sP[0][0] + to[k]) = xp[k];
    }
  };
  f32x4_t acc[JT][2];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt)
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) acc[jt][ct] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  tokens(0);
  load(0);
  tokens(32);
  for (int m = 0; m < it.count; m += 32) {
    store(m);
    lds_barrier();
    load(m + 32);
    tokens(m + 64);
    u32x4_t fq[3][2];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) fq[k][ct] = tr_frag_swizzled(sQ[side][k], 32 * quarter + 16 * ct, li, lg);
#pragma unroll
    for (int t = 0; t < 3; ++t)
#pragma unroll
      for (int jt = 0; jt < JT; ++jt) {
        const u32x4_t a = tr_frag(sP[side] + 32 * t * PP + 16 * jt, PP, li, lg);
#pragma unroll
        for (int k = 0; k < 3 - t; ++k)
#pragma unroll
          for (int ct = 0; ct < 2; ++ct)
            acc[jt][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(fq[k][ct]), acc[jt][ct], 0, 0, 0);
      }
    lds_barrier();   // read by everyone; the next step's loads stay in flight
  }
  // lane: column li of each tile, rows j = 4 lg + e
  const ColReq& rq = side ? r1 : r0;
  if (!rq.out) return;
  const lq_adapter ad = side ? ad1 : ad0;
  const int r = min(ad.r, 16 * JT);
  const bool vec = it.slot < 0 && r % 4 == 0 && (reinterpret_cast<uintptr_t>(rq.out) & 15) == 0;
#pragma unroll
  for (int jt = 0; jt < JT; ++jt)
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
      const int64_t c = c0 + 32 * quarter + 16 * ct + li;
      const int j0 = 16 * jt + 4 * lg;
      if (c >= N || j0 >= r) continue;
      if (vec) {   // N * row and c * r are multiples of 4
        *reinterpret_cast<f32x4_t*>(rq.out + N * ad.row + c * r + j0) = acc[jt][ct];
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + e;
        if (j >= r) break;
        if (it.slot >= 0) rq.part[((int64_t)it.slot * rq.v.rs + j) * N + c] = acc[jt][ct][e];
        else rq.out[N * ad.row + c * r + j] = acc[jt][ct][e];
      }
    }
}

// Runs of positions per workgroup: enough workgroups for the chip, runs of at
// least 256 so that the partial sums stay few.
int gated_col_rows(int64_t M, int64_t N) {
  const int64_t tiles = (N + GC_COLS - 1) / GC_COLS;
  return (int)std::max<int64_t>(256, std::min<int64_t>(M * tiles / 512 / 32 * 32, 4096));
}

}  // namespace

// Shares of the columns: what leaves the shortest queue of 64-column steps where
// three workgroups run on each CU, a share costing about two steps more. n: one
// more tile for each adapter's remainder.
int gated_down_shares(int64_t M, int64_t N, int32_t n) {
  const int64_t tiles = (M + GD_M - 1) / GD_M, steps = (N + GD_K - 1) / GD_K, items = tiles + std::min<int64_t>(n, tiles);
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int s = 1; s <= 16 && s <= steps; ++s) {
    const int64_t c = (items * s + 767) / 768 * ((steps + s - 1) / s + 2);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}
size_t gated_down_ws_floats(int64_t M, int64_t N, const AdapterView& v) { return (size_t)gated_down_shares(M, N, v.n) * M * v.rs; }

#define LQ_ACTS(CALL, JT)                      \
  do {                                         \
    if (act == LQ_SILU) CALL(JT, LQ_SILU);     \
    else if (act == LQ_GELU) CALL(JT, LQ_GELU); \
    else CALL(JT, LQ_GELU_TANH);               \
  } while (0)

hipError_t launch_gated_down(const GatedGrad& gr, int64_t M, const AdapterView (&v)[2], const uint16_t* const (&bt)[2],
                             float* const (&part)[2], uint16_t* D, const Route& rt, hipStream_t s) {
  LQ_DASSERT(gr.N % 8 == 0 && M > 0);
  const GatedDown p{gr, {v[0], v[1]}, {bt[0], bt[1]}, {part[0], part[1]}, D, (gr.N + 63) / 64 * 64};
  const int act = gr.act;
  const dim3 grid((unsigned)((M + GD_M - 1) / GD_M + std::min<int64_t>(v[0].n + 1, M)),
                  (unsigned)gated_down_shares(M, gr.N, v[0].n));
  const int32_t r = std::max(v[0].r_max, v[1].r_max);
#define LQ_GD(JT, ACT) hipLaunchKernelGGL((k_gated_down<JT, ACT>), grid, dim3(256), 0, s, p, M, rt)
  if (r <= 16) LQ_ACTS(LQ_GD, 1);
  else if (r <= 32) LQ_ACTS(LQ_GD, 2);
  else if (r <= 64) LQ_ACTS(LQ_GD, 4);
  else LQ_ACTS(LQ_GD, 8);
#undef LQ_GD
  return hipGetLastError();
}

hipError_t launch_gated_col(const GatedGrad& gr, const ColReq (&req)[2], int64_t M, const Route& rt, ColJoin* join,
                            hipStream_t s) {
  LQ_DASSERT(gr.N % 8 == 0 && M > 0 && req[0].v.n > 0);
  const int rows = gated_col_rows(M, gr.N), act = gr.act;
  const dim3 grid((unsigned)((gr.N + GC_COLS - 1) / GC_COLS), (unsigned)((M + rows - 1) / rows + std::min<int64_t>(req[0].v.n, M)));
  const int32_t r = std::max(req[0].v.r_max, req[1].v.r_max);
#define LQ_GC(JT, ACT) hipLaunchKernelGGL((k_gated_col<JT, ACT>), grid, dim3(GC_THREADS), 0, s, gr, req[0], req[1], rows, rt)
  if (r <= 16) LQ_ACTS(LQ_GC, 1);
  else if (r <= 32) LQ_ACTS(LQ_GC, 2);
  else if (r <= 64) LQ_ACTS(LQ_GC, 4);
  else LQ_ACTS(LQ_GC, 8);
#undef LQ_GC
  *join = ColJoin{{req[0], req[1]}, 0, rows, M <= rows};
  for (int i = 0; i < 2; ++i)
    if (req[i].out) join->q[join->n++] = req[i];
  return hipGetLastError();
}
#undef LQ_ACTS

}  // namespace lq
