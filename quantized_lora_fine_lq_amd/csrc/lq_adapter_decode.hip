// Many adapters at decode sizes (up to 64 tokens), NF4 weight:
//   t[m] = A_a x[m],  h[m] = W' x[m] + s_a B_a t[m],  a = ids[m],
// or of a gated pair act(g) u with g and u two such projections of one x,
// without sorting the tokens: a wave holds one id per lane, so the tokens of
// an adapter are one ballot. Bound by reading the packed weight once and, per
// code, by the lookup, product and rounding that make its bfloat16 weight.
//
// QLoRA (Heng's Blog), introduction: h = dequant(W0_NF4) x + (alpha/r) B A x.
#include <algorithm>

#include "lq_act.h"
#include "lq_adapters.h"
#include "lq_device.h"
#include "lq_route.h"

namespace lq {
namespace {

// set bits of m below the lane
__device__ __forceinline__ int bits_below(uint64_t m) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}
__device__ __forceinline__ f32x4_t zero4() { return f32x4_t{0.f, 0.f, 0.f, 0.f}; }

// The lane's token's adapter, or -1.
__device__ __forceinline__ int lane_key(const int32_t* ids, int M, int n) {
  const int lane = threadIdx.x & 63;
  const int id = lane < M ? ids[lane] : -1;
  return (uint32_t)id < (uint32_t)n ? id : -1;
}

// The tokens of the lane's adapter, one of n, from one ballot per bit.
__device__ __forceinline__ uint64_t same_key(int key, int n) {
  uint64_t peers = __ballot(key >= 0);
  for (int b = 0; (n - 1) >> b; ++b) {
    const uint64_t one = __ballot((key >> b) & 1);
    peers &= ((key >> b) & 1) ? one : ~one;
  }
  return peers;
}

// The adapters' part as steps of 32 contraction columns (4 runs of 8; TERMS
// copies of an adapter's runs), dealt to the waves in turn. Lane l holds the
// adapter of token l; the first token of each adapter in use leads it, and the
// leaders' step counts, summed over the lanes, number the steps. The launch
// that forms t writes the steps out for the projection (DcRecord), whose waves
// then start from one uniform load instead of a chain of them.
struct DcSteps {
  lq_adapter ad;     // the lane's token's adapter (leaders' entries are used)
  uint64_t same;     // its tokens
  int first, count;  // its steps (0 unless the lane leads)
  int total;
};
__device__ __forceinline__ DcSteps dc_steps(const lq_adapter& ad, int key, int n, int terms) {
  DcSteps st;
  st.ad = ad;
  const uint64_t peers = same_key(key, n);
  st.same = peers;
  const bool leads = key >= 0 && bits_below(peers) == 0;
  st.count = leads ? (terms * ((st.ad.r + 7) >> 3) + 3) >> 2 : 0;   // at most 12
  st.first = 0;
  st.total = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {   // the sum over the lanes below, bit by bit
    const uint64_t one = __ballot((st.count >> b) & 1);
    st.first += bits_below(one) << b;
    st.total += __popcll(one) << b;
  }
  return st;
}

struct DcRecord {
  uint64_t B, same;    // B_a, its tokens
  float scale;
  int32_t r;
  uint32_t runs;       // byte q, run q of the step: rank / 8, term << 4, 64 where it is one of the adapter's, 128 of side 1
  int32_t total;       // steps in all (every record)
};
constexpr int DC_PAD = 64;                        // no token's steps past the last: the projection asks for them too
constexpr int DC_RECORDS = 64 * 12 + DC_PAD;      // of a side

// ===========================================================================
// t = A_a x: one workgroup per 16 tokens of an adapter (workgroup b takes the
// b-th such tile, adapters in token order) and column part; the waves split
// the part's columns. (One workgroup for all of an adapter's tokens: 64 tokens of
// one adapter, K = 8192, 20 us more.) The parts' sums go to t [parts][M][rs]; the projection
// adds them. The workgroups past the adapters' lay X out for the projection's
// fragments (xp, see XPack): a load of 16 rows is then 1 KB in one piece, where
// the rows themselves are 64 pieces of 16 bytes in 32 cache lines. Bound by
// latency: one token 4.3 us, 16 tokens of 16 adapters 5.1 (K = 4096), 64 tokens
// of 32 adapters, K = 8192, 10.6.
//
// PAIR: the adapters of two sets, side 1's workgroups after side 0's, and its
// steps after side 0's. A pair may have no sets (n = 0): the steps past the last
// then point into the codes of a weight, whose rows are 32 bytes or more. Its
// workgroups are of eight waves: of sixteen, whose registers leave room for one
// on a CU, two sides' would not all run at once.
// ===========================================================================
// XPack: 16 bytes for (stage s, token tile tt, sub-step u, lane) at
// ((s TT + tt) 4 + u) 64 + lane: token 16 tt + lane % 16, columns 128 s + 32 (lane / 16) + 8 u
// of X, zero past K.
__device__ __forceinline__ int xp_units(int64_t K, int TT) { return (int)((K + 127) / 128) * TT * 256; }

// (The arguments of one set are as few as its kernels read: the size of both cost
// the one-token launches half a microsecond.)
template <bool PAIR>
struct DecodeDown {
  const uint16_t* X;
  int M;
  int64_t K;
  AdapterView v[PAIR ? 2 : 1];
  const int32_t* ids;
  float* t[PAIR ? 2 : 1];   // [parts][M][rs]
  u32x4_t* xp;
  int TT, wgs;         // token tiles; workgroups of a side's adapters
  DcRecord* records;
  int terms;
  const void* anywhere;
};

template <int JT, int W, bool PAIR>
__global__ __launch_bounds__(64 * W) void k_decode_down(DecodeDown<PAIR> p) {
  __shared__ f32x4_t part[W][JT][64];
  const uint16_t* __restrict__ X = p.X;
  const int32_t* __restrict__ ids = p.ids;
  const int M = p.M, TT = p.TT, wgs = p.wgs, all_wgs = PAIR ? 2 * wgs : wgs;
  const int64_t K = p.K;
  if ((int)blockIdx.x == all_wgs) {   // the steps, by the lanes that lead an adapter
    if (blockIdx.y || threadIdx.x >= 64) return;
    const int n = p.v[0].n, key = PAIR && !n ? -1 : lane_key(ids, M, n);
    int total = 0;
    lq_adapter any{};
    any.B = reinterpret_cast<const uint16_t*>(p.anywhere);
    any.r = 8;
    DcSteps st[PAIR ? 2 : 1];
    if (!PAIR || n) {
      any = p.v[0].tab[0];
#pragma unroll
      for (int sd = 0; sd < (PAIR ? 2 : 1); ++sd) {
        st[sd] = dc_steps(p.v[sd].tab[max(key, 0)], key, n, p.terms);
        st[sd].first += total;
        total += st[sd].total;
      }
#pragma unroll
      for (int sd = 0; sd < (PAIR ? 2 : 1); ++sd) {
        const DcSteps& at = st[sd];
        const int runs = (at.ad.r + 7) >> 3;
        for (int k = 0, term = 0, run = 0; k < at.count; ++k) {
          uint32_t packed = sd ? 0x80808080u : 0u;
          for (int q = 0; q < 4; ++q) {
            if (term < p.terms) packed |= (uint32_t)(run | term << 4 | 64) << (8 * q);
            if (++run == runs) run = 0, ++term;
          }
          p.records[at.first + k] = DcRecord{(uint64_t)reinterpret_cast<uintptr_t>(at.ad.B), at.same, at.ad.scale, at.ad.r, packed,
                                             total};
        }
      }
    }
    if (threadIdx.x < DC_PAD)
      p.records[total + threadIdx.x] = DcRecord{(uint64_t)reinterpret_cast<uintptr_t>(any.B), 0, 0.0f, any.r, 0, total};
    return;
  }
  if ((int)blockIdx.x > all_wgs) {
    const int workers = ((int)gridDim.x - all_wgs - 1) * (int)gridDim.y * 64 * W;
    int i = (((int)blockIdx.x - all_wgs - 1) * (int)gridDim.y + (int)blockIdx.y) * 64 * W + (int)threadIdx.x;
    for (; i < xp_units(K, TT); i += workers) {
      const int ln = i & 63, u = (i >> 6) & 3, tt = (i >> 8) % TT, s = (i >> 8) / TT;
      const int64_t k = 128 * (int64_t)s + 32 * (ln >> 4) + 8 * u;
      u32x4_t x = {0u, 0u, 0u, 0u};
      if (k < K) x = ld16(X + (int64_t)min(16 * tt + (ln & 15), M - 1) * K + k);
      p.xp[i] = x;
    }
    return;
  }
  const int side = PAIR && (int)blockIdx.x >= wgs ? 1 : 0, which = (int)blockIdx.x - side * wgs;
  const AdapterView v = side ? p.v[PAIR] : p.v[0];
  float* t = side ? p.t[PAIR] : p.t[0];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  // Few tokens: one adapter after the other, 0.07 us each. More: the lanes that lead
  // an adapter count its tiles and number them by a sum over the lanes below, 0.3 us
  // in all (64 tokens of 32 adapters: 10.6 us for 14.0 of this kernel).
  const int key = lane_key(ids, M, v.n);
  int a = -1, t0 = 0;
  uint64_t mine = 0;
  if (M <= 4) {
    uint64_t left = __ballot(key >= 0);
    for (int b = which; left; --b) {   // (at most 16 tokens: one tile each)
      a = __builtin_amdgcn_readlane(key, __ffsll((unsigned long long)left) - 1);
      mine = __ballot(key == a);
      if (b == 0) break;
      left &= ~mine;
      a = -1;
    }
    if (a < 0) return;
  } else {
    const uint64_t peers = same_key(key, v.n);
    const int tiles = key >= 0 && bits_below(peers) == 0 ? (__popcll(peers) + 15) >> 4 : 0;   // at most 4
    int before = 0;
#pragma unroll
    for (int b = 0; b < 3; ++b) before += bits_below(__ballot((tiles >> b) & 1)) << b;
    const uint64_t hit = __ballot(which >= before && which < before + tiles);
    if (!hit) return;
    const int leader = __ffsll((unsigned long long)hit) - 1;
    a = __builtin_amdgcn_readlane(key, leader);
    t0 = 16 * (which - __builtin_amdgcn_readlane(before, leader));
    mine = __ballot(key == a);
  }
  const lq_adapter ad = v.tab[a];
  const int r = min(ad.r, 16 * JT), count = __popcll(mine);
  const uint16_t* rr[JT];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) rr[jt] = ad.A + (int64_t)min(16 * jt + li, r - 1) * K;
  const int all = (int)(K / 64), per = (all + gridDim.y - 1) / gridDim.y;
  const int first = min(all, (int)blockIdx.y * per), blocks = min(all, first + per);   // this part's 64-column blocks
  t += (int64_t)blockIdx.y * M * v.rs;
  // token of row i of this 16: the (t0 + i)-th set bit of `mine`
  int tok = 0;
  {
    uint64_t m = mine;
    const int want = min(t0 + li, count - 1);
    for (int i = 0; i < want; ++i) m &= m - 1;
    tok = __ffsll((unsigned long long)m) - 1;
  }
  const uint16_t* q = X + (int64_t)tok * K;
  f32x4_t acc[JT];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) acc[jt] = zero4();
  constexpr int UB = JT <= 2 ? 4 : 1;   // blocks of 64 columns in flight
  for (int b = first + wave; b < blocks; b += W * UB) {
    u32x4_t x[UB][2], w[UB][2][JT];
#pragma unroll
    for (int u = 0; u < UB; ++u) {
      const int64_t c = 64 * (int64_t)min(b + W * u, blocks - 1) + 8 * lg;   // 64 bytes of each row a load
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[u][h] = ld16(q + c + 32 * h);
#pragma unroll
        for (int jt = 0; jt < JT; ++jt) w[u][h][jt] = ld16(rr[jt] + c + 32 * h);
      }
    }
#pragma unroll
    for (int u = 0; u < UB; ++u)
      if (b + W * u < blocks)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int jt = 0; jt < JT; ++jt)
            acc[jt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x[u][h]), as_bf16x8(w[u][h][jt]), acc[jt], 0, 0, 0);
  }
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) part[wave][jt][lane] = acc[jt];
  __syncthreads();
  for (int i = threadIdx.x; i < JT * 64 * 4; i += 64 * W) {
    const int e = i & 3, ln = (i >> 2) & 63, jt = i >> 8, j = 16 * jt + (ln & 15);
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += part[w][jt][ln][e];
    const int row = 4 * (ln >> 4) + e;
    if (t0 + row >= count) continue;
    uint64_t m = mine;
    for (int k = 0; k < t0 + row; ++k) m &= m - 1;
    const int token = __ffsll((unsigned long long)m) - 1;
    if (j < v.rs) t[token * v.rs + j] = j < r ? sum : 0.0f;
  }
}

// ===========================================================================
// The projection. A workgroup owns RG groups of 16 weight rows; its W waves
// take the 128-wide stages of the contraction in turn (the two stages of a
// 128-byte line of codes in the same iteration) and their partial sums meet in
// LDS at the end. Per stage and row group, lane (li, lg) loads 32 codes of row
// li, decodes them into the A operand of four MFMA 16x16x32, and multiplies TT
// tiles of 16 tokens; X comes from the L2.
//
// A code byte becomes two levels through an LDS table of level pairs in 16
// copies: entry e of copy s at 8 (16 e + s), and lane l reads copy l % 16. With
// one copy (2 KB) two thirds of the lookups' cycles were bank conflicts; with
// 32 none were, but the table (64 KB) left room for one workgroup per CU, which
// then started, waited and finished with nothing beside it.
//
// Four row groups run in workgroups of four waves, two of them per CU, fewer in
// workgroups of eight. Measured, 64 tokens, N = 28672, K = 8192, 32 adapters of
// rank 8 to 32: 71 us, that is 1.7 TB/s of codes, the launch before it 10.6. A
// workgroup's 60 us are 9 of start, 10 of the adapters' part (B is read from
// memory, 34 MB in all) and 38 of the stages, whose lookups and products wait
// for one another at two waves a SIMD: 64 tokens' sums and X take 128 registers.
// 16 tokens, N = K = 4096: 7.8 us after 5.1; one token: 7.0 after 4.3 (forming
// t in the projection instead took 14.0 in all).
//
// GATED: the first half of the row groups are the gate's, the second half the
// same rows of up, so that the join has g and u of an output side by side; the
// workgroup is RG / 2 groups of 16 outputs. Measured, N = 28672, K = 8192, 64
// tokens of 32 adapters of rank 8 to 32: 145 to 157 us, 121 without adapters; N =
// 11008, K = 4096: one token 18 to 20 us. Past the memory's 47 and 9 us it is bound as
// above.
// ===========================================================================
struct DecodeSide {
  QWeight w;
  AdapterView v;
  const float* t;      // [parts][M, rs]
  float* t_out;        // [M, r_max], or null
};
template <bool GATED>
struct DecodeParams {
  const u32x4_t* xp;   // X in fragment order
  const DcRecord* records;
  int M, parts;
  const int32_t* ids;
  void* out;
  DecodeSide s[GATED ? 2 : 1];
  Nf4Levels lv;
  int act;
  uint16_t *g_out, *u_out;
};

constexpr int DC_PAIRS = 256 * 16;   // f32x2_t, 32 KB
constexpr int DC_PARTS = 8;           // most column parts of t

constexpr int kXcds = 8;

template <int RG>
struct DcStage {
  u32x4_t code[RG];
  u32x4_t x[4];   // one token tile: its X ahead with the codes
  int bl;         // the lane's 64-block (the last one where that lies past the row)
};

// The constants' row stride. 16 rows' constants of one block have to hit distinct
// banks, and four blocks' to lie in one piece where rows hold whole fours of them: any
// odd stride, or an odd count of fours. Of four row groups a row of a multiple of 64
// (K of 4096) keeps its length and is turned by 4 (row % 16) places instead: 64 rows of
// K = 8192 and 64 tokens' t of rank 64 then leave two workgroups room.
__host__ __device__ constexpr bool dc_turns(int rg, int nb) { return rg == 4 && nb % 64 == 0; }
__host__ __device__ constexpr int dc_pitch(int rg, int nb) { return dc_turns(rg, nb) ? nb : nb % 4 == 0 ? nb | 4 : nb | 1; }
// floats of LDS after the pair table: constants, then the partial sums of one
// token tile
template <int RG, int W>
__host__ __device__ constexpr int dc_floats(int nb) {
  const int c = (16 * RG * dc_pitch(RG, nb) + 3) / 4 * 4, red = W * RG * 272;
  return c > red ? c : red;
}
size_t dc_lds_bytes(int rg, int tt, int w, int nb, int rs, int terms) {   // rs: of both sides of a pair
  const int c = (16 * rg * dc_pitch(rg, nb) + 3) / 4 * 4, red = w * rg * 272;
  return DC_PAIRS * sizeof(f32x2_t) +
         4 * (size_t)(c > red ? c : red) + 2 * (size_t)(16 * tt * rs * terms);
}

__device__ __forceinline__ DcRecord of_lane(const DcRecord& x, int l) {
  auto u = [&](uint32_t w) { return (uint32_t)__builtin_amdgcn_readlane((int)w, l); };
  return DcRecord{u((uint32_t)x.B) | (uint64_t)u((uint32_t)(x.B >> 32)) << 32,
                  u((uint32_t)x.same) | (uint64_t)u((uint32_t)(x.same >> 32)) << 32,
                  __uint_as_float(u(__float_as_uint(x.scale))), (int)u((uint32_t)x.r), u(x.runs), (int)u((uint32_t)x.total)};
}

// A step as every lane needs it, with the weight-side operand loaded.
template <int NG>
struct DcStep {
  u32x4_t w[NG];
  uint64_t same;
  float scale;
  int term, j0;
  bool live, side;
};
template <int NG, int RG>
__device__ __forceinline__ void dc_step(const DcRecord& rec, const int64_t (&row)[RG], DcStep<NG>& o) {
  const uint16_t* B = reinterpret_cast<const uint16_t*>(rec.B);
  const int r = rec.r;
  const uint32_t run = rec.runs >> (threadIdx.x >> 1 & 24);   // the lane's: byte lane / 16
  o.scale = rec.scale;
  o.same = rec.same;
  o.live = run & 64;
  o.side = rec.runs & 128;
  o.term = (run >> 4) & 3;
  o.j0 = 8 * (run & 15);
#pragma unroll
  for (int g = 0; g < NG; ++g) {   // (a pair's two halves are the same rows)
    const uint16_t* b = B + row[g] * r;
    if (NG == RG ? __builtin_expect(r % 8 == 0, 1) : r % 8 == 0) {   // (in line for one set; a pair's one group would spill)
      o.w[g] = ld16(b + o.j0);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = o.j0 + 2 * e;
        const uint32_t x = b[min(j, r - 1)], y = b[min(j + 1, r - 1)];
        o.w[g][e] = (j < r ? x : 0u) | ((j + 1 < r ? y : 0u) << 16);
      }
    }
    if (!o.live) o.w[g] = u32x4_t{0u, 0u, 0u, 0u};
  }
}
// Adds step o, of that side: each product goes to its own tokens' columns alone.
template <int SIDE, int NG, int RG, int TT, int TERMS>
__device__ __forceinline__ void dc_apply(const DcStep<NG>& o, const uint16_t* sT, int rs, int M, f32x4_t (&acc)[RG][TT]) {
  const int lane = threadIdx.x & 63, li = lane & 15;
  const u32x4_t none = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) {
    if (!((o.same >> (16 * tt)) & 0xFFFF)) continue;
    const int m = 16 * tt + li;
    const bool mine = (o.same >> m) & 1;
    u32x4_t tv = *reinterpret_cast<const u32x4_t*>(sT + (min(m, M - 1) * TERMS + o.term) * rs + o.j0);
    if (!o.live) tv = none;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const f32x4_t d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(o.w[g]), as_bf16x8(tv), zero4(), 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // selected last: a scale that is not finite makes NaN of 0, too
        f32x4_t& sum = acc[g + SIDE * NG][tt];
        const float with = __builtin_fmaf(o.scale, d[e], sum[e]);
        sum[e] = mine ? with : sum[e];
      }
    }
  }
}

// Outputs n .. n + 3 of a token, at element o.
template <bool OUT_F32>
__device__ __forceinline__ void dc_store(void* out, int64_t o, int64_t n, int64_t N, const f32x4_t& h) {
  if (N % 4 == 0) {
    if (OUT_F32) {
      float* f = reinterpret_cast<float*>(out) + o;   // 4-byte aligned
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = h[e];
    } else {
      uint2 v;
      v.x = pack_bf16x2(h[0], h[1]);
      v.y = pack_bf16x2(h[2], h[3]);
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + o) = v;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e >= N) break;
      if (OUT_F32) reinterpret_cast<float*>(out)[o + e] = h[e];
      else reinterpret_cast<uint16_t*>(out)[o + e] = (uint16_t)(pack_bf16x2(h[e], 0.f) & 0xFFFFu);
    }
  }
}

// (A pair's four waves over one group of outputs: three such workgroups share a CU, and
// registers for a fourth would spill.)
template <int RG, int TT, int W, bool DQ, bool OUT_F32, bool GATED>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(GATED && RG == 2 && W == 4 ? 3 : 2))) void k_decode_nf4(DecodeParams<GATED> p) {
  constexpr int NG = GATED ? RG / 2 : RG;   // groups of 16 outputs
  extern __shared__ __attribute__((aligned(16))) unsigned char dc_lds[];
  constexpr int TERMS = OUT_F32 ? 3 : 2;
  constexpr bool XA = TT == 1;   // X is loaded a stage ahead, with the codes
  f32x2_t* sPair = reinterpret_cast<f32x2_t*>(dc_lds);
  float* sC = reinterpret_cast<float*>(dc_lds + DC_PAIRS * sizeof(f32x2_t));
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int64_t N = p.s[0].w.N, K = p.s[0].w.K;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NG;
  const int rs0 = p.s[0].v.rs, rs1 = GATED ? p.s[GATED].v.rs : 0;
  const int nb = (int)(K / 64), pitch = dc_pitch(RG, nb), ns = (nb + 1) / 2;
  const int turn = dc_turns(RG, nb) ? 15 : 0;
  auto turned = [&](int r, int b) {   // place of block b's constant in row r
    if (RG < 4) return b;
    const int at = b + 4 * (r & turn);
    return at < nb ? at : at - nb;
  };
  uint16_t* sT = reinterpret_cast<uint16_t*>(sC + dc_floats<RG, W>(nb));   // t's bf16 terms [M][TERMS][rs], side 1's after side 0's

  const uint8_t* crow[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) crow[g] = (g < NG ? p.s[0].w : p.s[GATED].w).codes + min(n0 + 16 * (g % NG) + li, N - 1) * (K / 2) + 16 * (lg & 1);
  // The stages in an order rotated by workgroup: rows lie a power of two apart in
  // the common sizes, so workgroups in step would all read from the same few
  // channels of the L2.
  const int rot = (int)((blockIdx.x / kXcds * 4) % ns);
  auto place = [&](int s) {
    const int at = min(s, ns - 1) + rot;
    return at < ns ? at : at - ns;
  };
  auto load = [&](int s, DcStage<RG>& st) {
    const int ss = place(s);
    st.bl = min(2 * ss + (lg >> 1), nb - 1);
#pragma unroll
    for (int g = 0; g < RG; ++g) st.code[g] = ld16(crow[g] + (int64_t)st.bl * 32);
    if constexpr (XA)
#pragma unroll
      for (int u = 0; u < 4; ++u) st.x[u] = p.xp[((int64_t)ss * 4 + u) * 64 + lane];
  };
  // Several token tiles: each sub-step's X is refilled for the wave's next stage
  // as soon as it is used. Loads return in order, so X asked for when needed
  // would wait for the codes asked for before it, from memory.
  u32x4_t x[TT][4];
  auto load_x = [&](int s, int u) {
    const u32x4_t* xs = p.xp + (int64_t)place(s) * (TT * 256) + lane;
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) x[tt][u] = xs[(tt * 4 + u) * 64];
  };
  // Everything that the start waits for is asked for before any of it is used:
  // the first codes, and B of the wave's first DEEP steps (a step is a round
  // trip to memory).
  constexpr int DEEP = RG == 4 || TT == 4 ? 4 : 1;   // (16 tokens' steps are one or two a wave)
  static_assert(W * 2 * DEEP <= DC_PAD, "the steps asked for end within the padding");
  int64_t row[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) row[g] = min(n0 + 16 * (g % NG) + li, N - 1);
  DcStep<NG> steps[DEEP];
  DcStage<RG> s0, s1;
  load(wave, s0);
  if constexpr (XA) load(wave + W, s1);
  constexpr int kRecords = GATED ? 2 * DC_RECORDS : DC_RECORDS;
  // Lane l keeps the record of the wave's step 64 c + l.
  DcRecord rec;
  auto load_records = [&](int i) {
    const u32x4_t* at = reinterpret_cast<const u32x4_t*>(p.records + min(wave + W * (i + lane), kRecords - 1));
    const u32x4_t a = at[0], b = at[1];
    rec = DcRecord{a[0] | (uint64_t)a[1] << 32, a[2] | (uint64_t)a[3] << 32, __uint_as_float(b[0]), (int)b[1], b[2], (int)b[3]};
  };
  auto ask = [&](int i, DcStep<NG>& o) { dc_step<NG>(of_lane(rec, i & 63), row, o); };
  load_records(0);
#pragma unroll
  for (int d = 0; d < DEEP; ++d) ask(d, steps[d]);
  const int nsteps = of_lane(rec, 0).total;

  // The pair table: lane l of a wave writes slot l % 32 of entries e + l / 32
  const float level = p.lv.q[lane & 15], second = __shfl(level, 4 * (wave & 3) + (lane >> 4));
#pragma unroll
  for (int k = 0; k < 64 / W; ++k) {
    const int e = 4 * (wave + W * k);   // e .. e + 3: one first level
    sPair[16 * e + lane] = f32x2_t{__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(level), e >> 4)), second};
  }
  // the rows' constants, four a thread: thread t row t % (16 RG)
  float means[2] = {0.0f, 0.0f};
  if constexpr (DQ) {
    means[0] = *p.s[0].w.qc.dq_mean;
    if constexpr (GATED) means[1] = *p.s[GATED].w.qc.dq_mean;
  }
  if (nb % 4 == 0) {
    const int rr = threadIdx.x % (16 * RG);
    const bool up = GATED && rr >= 16 * NG;
    const QConst qc = up ? p.s[GATED].w.qc : p.s[0].w.qc;
    const float mean = up ? means[1] : means[0];
    const int64_t b0 = min(n0 + (up ? rr - 16 * NG : rr), N - 1) * nb;
#pragma unroll 4
    for (int c = 4 * (threadIdx.x / (16 * RG)); c < nb; c += 4 * (64 * W / (16 * RG))) {
      const int64_t blk = b0 + c;   // a multiple of 4: one second-level scale
      f32x4_t v;
      if constexpr (DQ) {
        const uint32_t q8 = *reinterpret_cast<const uint32_t*>(qc.absmax_q + blk);
        const float s2 = qc.dq_scale[blk >> 8];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(e4m3_decode((q8 >> (8 * e)) & 0xFFu), s2, mean);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = qc.absmax[blk + e];
      }
      *reinterpret_cast<f32x4_t*>(sC + rr * pitch + turned(rr, c)) = v;   // in one piece: stride and turn are whole fours
    }
  } else {
    for (int i = threadIdx.x; i < 16 * RG * nb; i += 64 * W) {
      const int rr = i / nb, bl = i - rr * nb;
      const bool up = GATED && rr >= 16 * NG;
      const QConst qc = up ? p.s[GATED].w.qc : p.s[0].w.qc;
      const int64_t blk = min(n0 + (up ? rr - 16 * NG : rr), N - 1) * nb + bl;
      sC[rr * pitch + bl] = DQ ? __builtin_fmaf(e4m3_decode(qc.absmax_q[blk]), qc.dq_scale[blk >> 8], up ? means[1] : means[0])
                               : qc.absmax[blk];
    }
  }
  // t: its parts added in order, and split into bf16 terms: two keep 16 bits
  // of it, 8 more than a bf16 H, three all 24 (rows of tokens without an
  // adapter hold anything: no step takes them). Token m's t is saved by workgroup m % grid.
#pragma unroll
  for (int sd = 0; sd < (GATED ? 2 : 1); ++sd) {
    const AdapterView& v = p.s[sd].v;
    const float* t = p.s[sd].t;
    uint16_t* to = sT + sd * p.M * TERMS * rs0;
    const int quads = v.rs / 4, nq = p.M * quads, nt = p.M * v.rs;
#pragma unroll 2
    for (int i = threadIdx.x; i < nq; i += 64 * W) {
      f32x4_t part[DC_PARTS];
#pragma unroll
      for (int k = 0; k < DC_PARTS; ++k)
        part[k] = *reinterpret_cast<const f32x4_t*>(t + (int64_t)min(k, p.parts - 1) * nt + 4 * i);
      f32x4_t sum = part[0];
#pragma unroll
      for (int k = 1; k < DC_PARTS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += k < p.parts ? part[k][e] : 0.0f;
      const int m = (uint32_t)i / (uint32_t)quads, j = 4 * (i - m * quads);
      if (p.s[sd].t_out && m % gridDim.x == blockIdx.x) {
        const bool has = (uint32_t)p.ids[m] < (uint32_t)v.n;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < v.r_max) p.s[sd].t_out[m * v.r_max + j + e] = has ? sum[e] : 0.0f;
      }
      float x[4] = {sum[0], sum[1], sum[2], sum[3]};
#pragma unroll
      for (int q = 0; q < TERMS; ++q) {
        const uint2 bits = {take_bf16_terms(x[0], x[1]), take_bf16_terms(x[2], x[3])};
        *reinterpret_cast<uint2*>(to + (m * TERMS + q) * v.rs + j) = bits;
      }
    }
  }
  __syncthreads();

  f32x4_t acc[RG][TT];
#pragma unroll
  for (int g = 0; g < RG; ++g)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) acc[g][tt] = zero4();
  for (int i = 0; wave + W * i < nsteps; i += DEEP) {
    if (((i + DEEP) & 63) == 0) load_records(i + DEEP);
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      if (GATED && steps[d].side) dc_apply<(GATED ? 1 : 0), NG, RG, TT, TERMS>(steps[d], sT + p.M * TERMS * rs0, rs1, p.M, acc);
      else dc_apply<0, NG, RG, TT, TERMS>(steps[d], sT, rs0, p.M, acc);
      ask(i + DEEP + d, steps[d]);
    }
  }
  if constexpr (!XA) {   // in the loop's order
#pragma unroll
    for (int u = 0; u < 4; ++u) load_x(wave, u);
    load(wave + W, s1);
  }
  const uint32_t slot = 8 * (lane & 15);
  constexpr int GB = RG < 2 ? RG : 2;   // row groups per batch of lookups
  auto stage = [&](int s, DcStage<RG>& st) {
    if constexpr (XA)
#pragma unroll
      for (int u = 0; u < 4; ++u) x[0][u] = st.x[u];
    // (K / 64 odd: the last stage's second block lies past the row, where
    // XPack holds zeros)
    float cp[RG];
#pragma unroll
    for (int g = 0; g < RG; ++g) cp[g] = sC[(16 * g + li) * pitch + turned(li, st.bl)];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int g0 = 0; g0 < RG; g0 += GB) {
        f32x2_t q[GB][4];
#pragma unroll
        for (int g = 0; g < GB; ++g)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            // (the table lies at LDS address 0: the kernel has no other static LDS)
            const uint32_t c = st.code[g0 + g][u];
            const uint32_t at = ((b ? c >> (8 * b - 7) : c << 7) & 0x7F80u) | slot;
            q[g][b] = *reinterpret_cast<const __attribute__((address_space(3))) f32x2_t*>(at);
          }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < GB; ++g) {
          u32x4_t wv;
#pragma unroll
          for (int b = 0; b < 4; ++b) wv[b] = pack_bf16x2(q[g][b].x * cp[g0 + g], q[g][b].y * cp[g0 + g]);
#pragma unroll
          for (int tt = 0; tt < TT; ++tt)
            acc[g0 + g][tt] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(wv), as_bf16x8(x[tt][u]), acc[g0 + g][tt], 0, 0, 0);
        }
      }
      if constexpr (!XA) load_x(s + W, u);
    }
    load(s + 2 * W, st);
  };
  // Pairs of stages without a way out between them: a path that skipped the
  // second would make every wait at the top one for all loads in flight.
  int s = wave;
  for (; s + W < ns; s += 2 * W) {
    stage(s, s0);
    stage(s + W, s1);
  }
  if (s < ns) stage(s, s0);
  // the waves' sums, one token tile at a time, over the constants' space. A lane
  // holds token li, rows 4 lg + [0, 4) of each row group; lane l of a group lies
  // at 16-byte slot l + l / 16 of 68, so that the readers (consecutive threads:
  // consecutive rows of one token) hit distinct banks.
  f32x4_t* sR = reinterpret_cast<f32x4_t*>(sC);   // [W][RG][68]
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) {
    __syncthreads();
#pragma unroll
    for (int g = 0; g < RG; ++g) sR[(wave * RG + g) * 68 + lane + lg] = acc[g][tt];
    __syncthreads();
    for (int i = threadIdx.x; i < NG * 64; i += 64 * W) {
      const int quad = i & 3, g = (i >> 2) % NG, m = i / (4 * NG);
      auto total = [&](int group) {
        f32x4_t h = sR[group * 68 + m + 17 * quad];
#pragma unroll
        for (int w = 1; w < W; ++w) h += sR[(w * RG + group) * 68 + m + 17 * quad];
        return h;
      };
      f32x4_t h = total(g);
      const int64_t n = n0 + 16 * g + 4 * quad;
      if (16 * tt + m >= p.M || n >= N) continue;
      const int64_t o = (int64_t)(16 * tt + m) * N + n;
      if constexpr (GATED) {
        const f32x4_t u = total(g + NG);
        if (p.g_out) dc_store<false>(p.g_out, o, n, N, h);
        if (p.u_out) dc_store<false>(p.u_out, o, n, N, u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = u[e] * (p.act == LQ_SILU ? act_value<LQ_SILU>(h[e]) : p.act == LQ_GELU ? act_value<LQ_GELU>(h[e])
                                                                                      : act_value<LQ_GELU_TANH>(h[e]));
      }
      dc_store<OUT_F32>(p.out, o, n, N, h);
    }
  }
}

template <int RG, int TT, int W, bool GATED>
hipError_t launch_rg(const DecodeParams<GATED>& p, bool f32, hipStream_t s) {
  constexpr int NG = GATED ? RG / 2 : RG;
  const dim3 grid((unsigned)((p.s[0].w.N + 16 * NG - 1) / (16 * NG))), block(64 * W);
  const size_t lds = dc_lds_bytes(RG, TT, W, (int)(p.s[0].w.K / 64), p.s[0].v.rs + (GATED ? p.s[GATED].v.rs : 0), f32 ? 3 : 2);
  const bool dq = p.s[0].w.qc.absmax == nullptr;
  if (dq && f32) hipLaunchKernelGGL((k_decode_nf4<RG, TT, W, true, true, GATED>), grid, block, lds, s, p);
  else if (dq) hipLaunchKernelGGL((k_decode_nf4<RG, TT, W, true, false, GATED>), grid, block, lds, s, p);
  else if (f32) hipLaunchKernelGGL((k_decode_nf4<RG, TT, W, false, true, GATED>), grid, block, lds, s, p);
  else hipLaunchKernelGGL((k_decode_nf4<RG, TT, W, false, false, GATED>), grid, block, lds, s, p);
  return hipGetLastError();
}

constexpr int kCus = 256;
constexpr size_t kLdsBytes = 160 * 1024;

// Row groups per workgroup: the shortest queue of the longest CU, a workgroup
// costing its row groups and about two more for its start and its X. Four need
// the LDS of two workgroups (K up to some 10000), but of a pair with more than 32
// tokens, where t takes much of it, of one with eight waves: two row groups a
// workgroup would ask the L2 for X twice as often (32 adapters of rank 64, N =
// 28672, K = 8192: 258 us for 309; N = 14336, K = 4096: 105 for 142; N = 11008:
// 103 for 102). Of a pair at least two; 0: none fits.
int decode_rg(int64_t N, int64_t K, int tt, int rs, int terms, bool pair) {
  const int64_t groups = (N + 15) / 16 * (pair ? 2 : 1);
  int best = pair ? 0 : 1;
  int64_t cost = INT64_MAX;
  for (int rg = pair ? 2 : 1; rg <= 4; rg *= 2) {
    const bool two = rg == 4 && !(pair && tt == 4);
    const size_t lds = two ? 2 * dc_lds_bytes(rg, tt, 4, (int)(K / 64), rs, terms)
                           : dc_lds_bytes(rg, tt, 8, (int)(K / 64), rs, terms);
    if (lds > kLdsBytes) break;
    const int64_t sets = (groups + rg - 1) / rg, c = (sets + kCus - 1) / kCus * (rg + 2);
    if (c <= cost) {
      cost = c;
      best = rg;
    }
  }
  return best;
}

// Token tiles of the projection; column parts of t: with few adapters the
// columns are shared by several workgroups, at least eight 64-column blocks each.
int token_tiles(int64_t M) { return M <= 16 ? 1 : (M <= 32 ? 2 : 4); }
int decode_parts(int64_t K, int64_t M, int32_t n, int sides) {
  const int64_t wgs = std::min<int64_t>(M, n) * sides;
  int parts = 1;
  while (parts < DC_PARTS && wgs * parts * 2 <= kCus && K / 64 / (parts * 2) >= 8) parts *= 2;
  return parts;
}
size_t t_bytes(int parts, int64_t M, const AdapterView& v) { return ((size_t)parts * M * v.rs * sizeof(float) + 255) / 256 * 256; }
size_t xp_bytes(int64_t K, int64_t M) { return (size_t)((K + 127) / 128) * token_tiles(M) * 256 * 16; }

// Workgroups that suffice for the adapters in use and their tokens, 16 each
// (none without adapters, where there are no ids either).
int down_items(int64_t M, int32_t n) {
  const int64_t used = std::min<int64_t>(M, n);
  return used ? (int)(used + (M - used) / 16) : 0;
}

template <bool PAIR>
hipError_t launch_decode_down(const DecodeDown<PAIR>& d, int parts, hipStream_t s) {
  const dim3 grid((unsigned)(d.wgs * (PAIR ? 2 : 1) + 1 + std::max(1, 16 * d.TT / parts)), (unsigned)parts);
  const int jt = (std::max(d.v[0].r_max, d.v[PAIR].r_max) + 15) / 16;
#define LQ_DD(JT, W) hipLaunchKernelGGL((k_decode_down<JT, W, PAIR>), grid, dim3(64 * W), 0, s, d)
  if (jt <= 1) LQ_DD(1, (PAIR ? 8 : 16));
  else if (jt <= 2) LQ_DD(2, (PAIR ? 8 : 16));
  else if (jt <= 4) LQ_DD(4, 8);
  else LQ_DD(8, 8);
#undef LQ_DD
  return hipGetLastError();
}

}  // namespace

// NF4, at most 64 tokens, and one row group's constants within the LDS that the
// table (32 KB) and t's terms (at most 48 KB) leave.
bool adapter_decode_supported(const QWeight& w, int64_t M) {
  return w.format == LQ_FMT_NF4 && M <= 64 && w.K <= 49152;
}
size_t adapter_decode_ws_bytes(const QWeight& w, int64_t M, const AdapterView& v) {
  return t_bytes(decode_parts(w.K, M, v.n, 1), M, v) + DC_RECORDS * sizeof(DcRecord) + xp_bytes(w.K, M);
}

hipError_t launch_adapter_decode(const QWeight& w, const uint16_t* X, int64_t M, const int32_t* ids,
                                 const AdapterView& v, void* ws, float* t_save, void* H, bool f32, hipStream_t s) {
  if (!adapter_decode_supported(w, M)) return hipErrorInvalidValue;
  const int parts = decode_parts(w.K, M, v.n, 1), tt = token_tiles(M), terms = f32 ? 3 : 2;
  float* t_ws = reinterpret_cast<float*>(ws);
  DcRecord* records = reinterpret_cast<DcRecord*>(reinterpret_cast<char*>(ws) + t_bytes(parts, M, v));
  u32x4_t* xp = reinterpret_cast<u32x4_t*>(records + DC_RECORDS);
  const DecodeDown<false> d{X, (int)M, w.K, {v}, ids, {t_ws}, xp, tt, down_items(M, v.n), records, terms, nullptr};
  const hipError_t e = launch_decode_down<false>(d, parts, s);
  if (e != hipSuccess) return e;
  const DecodeParams<false> p{xp, records, (int)M, parts, ids, H, {{w, v, t_ws, t_save}}, tables().lv, 0, nullptr, nullptr};
  const int rg = decode_rg(w.N, w.K, tt, v.rs, terms, false);
#define LQ_RG(TT)                                           \
  do {                                                      \
    if (rg == 4) return launch_rg<4, TT, 4, false>(p, f32, s); \
    if (rg == 2) return launch_rg<2, TT, 8, false>(p, f32, s); \
    return launch_rg<1, TT, 8, false>(p, f32, s);           \
  } while (0)
  if (tt == 1) LQ_RG(1);
  if (tt == 2) LQ_RG(2);
  LQ_RG(4);
#undef LQ_RG
}

// Both weights NF4 with constants of one kind, and two row groups' constants
// and both sides' t within the LDS (float32: three terms of t).
bool gated_decode_supported(const QWeight (&w)[2], int64_t M, const AdapterView (&v)[2]) {
  return w[0].format == LQ_FMT_NF4 && w[1].format == LQ_FMT_NF4 && (w[0].qc.absmax == nullptr) == (w[1].qc.absmax == nullptr) &&
         M <= 64 && w[0].K <= 49152 && decode_rg(w[0].N, w[0].K, token_tiles(M), v[0].rs + v[1].rs, 3, true) > 0;
}
size_t gated_decode_ws_bytes(const QWeight& w, int64_t M, const AdapterView (&v)[2]) {
  const int parts = decode_parts(w.K, M, v[0].n, 2);
  return t_bytes(parts, M, v[0]) + t_bytes(parts, M, v[1]) + 2 * DC_RECORDS * sizeof(DcRecord) + xp_bytes(w.K, M);
}

hipError_t launch_gated_decode(const QWeight (&w)[2], const uint16_t* X, int64_t M, const int32_t* ids,
                               const AdapterView (&v)[2], void* ws, int act, float* t_gate, float* t_up, uint16_t* g,
                               uint16_t* u, void* H, bool f32, hipStream_t s) {
  if (!gated_decode_supported(w, M, v)) return hipErrorInvalidValue;
  const int parts = decode_parts(w[0].K, M, v[0].n, 2), tt = token_tiles(M), terms = f32 ? 3 : 2;
  char* at = reinterpret_cast<char*>(ws);
  float* t0 = reinterpret_cast<float*>(at);
  float* t1 = reinterpret_cast<float*>(at += t_bytes(parts, M, v[0]));
  DcRecord* records = reinterpret_cast<DcRecord*>(at += t_bytes(parts, M, v[1]));
  u32x4_t* xp = reinterpret_cast<u32x4_t*>(records + 2 * DC_RECORDS);
  const DecodeDown<true> d{X, (int)M, w[0].K, {v[0], v[1]}, ids, {t0, t1}, xp, tt, down_items(M, v[0].n), records, terms,
                     w[0].codes};
  const hipError_t e = launch_decode_down<true>(d, parts, s);
  if (e != hipSuccess) return e;
  const DecodeParams<true> p{xp, records, (int)M, parts, ids, H, {{w[0], v[0], t0, t_gate}, {w[1], v[1], t1, t_up}},
                             tables().lv, act, g, u};
  const int rg = decode_rg(w[0].N, w[0].K, tt, v[0].rs + v[1].rs, terms, true);
  // More groups of 16 outputs than CUs, up to 32 tokens: workgroups of four waves over
  // one group, up to three on a CU, against those of rg. Where the latter hold four
  // groups of outputs on a CU (rg = 4), the smaller ones win as a single round, and up
  // to 16 tokens also in two rounds of either while the larger ones' second is mostly
  // empty; where rg = 2 (long rows, large ranks), if they take no more rounds. K = 4096,
  // 1 / 16 / 32 tokens, rank 16, smaller against larger, us: N = 5120 17.6 / 20.7 / 23.7
  // against 20.8 / 23.4 / 25.3; 12288 23.1 / 25.5 / 30.1 against 27.5 / 30.0 / 32.0; 14336
  // (two rounds against one) 29.6 / 33.8 / 39.2 against 27.6 / 30.1 / 32.7; 20480 (two
  // each) 34.2 / 38.9 / 44.8 against 41.3 / 44.4 / 48.4; 28672 (three against two) 45.6 /
  // 59.4 / 69.2 against 47.4 / 53.9 / 60.2; 4096 (no more groups than CUs) 15.6 / 18.3 /
  // 20.3 against 14.2 / 16.5 / 19.0. K = 8192: 20480 64.0 / 71.6 / 85.8 against 69.1 / 74.8 /
  // 81.0; 24576 77.9 / 81.8 / 101 against 74.3 / 77.2 / 85.5. Two of either on a CU: K =
  // 16384, N = 28672 159 / 166 / 203 against 171 / 181 / 206; K = 4096, rank 128, N =
  // 8192 21.0 / 37.9 / 46.6 against 24.4 / 39.4 / 53.4, N = 14336, 32 tokens 87 against 103.
  const int64_t groups = (w[0].N + 15) / 16;
  const int nb = (int)(w[0].K / 64), rs = v[0].rs + v[1].rs;
  auto rounds = [&](size_t lds, int64_t most) {   // of workgroups of one group
    const int64_t slots = kCus * std::min<int64_t>(most, (int64_t)(kLdsBytes / lds));
    return (groups + slots - 1) / slots;
  };
  bool flat = false;
  if (tt <= 2 && groups > kCus) {
    const size_t lds = dc_lds_bytes(2, tt, 4, nb, rs, terms);
    const int64_t mine = rounds(lds, 3);
    if (rg == 4) flat = mine == 1 || (tt == 1 && mine == 2 && groups > 4 * kCus && groups <= 5 * kCus);
    else flat = mine <= rounds(dc_lds_bytes(2, tt, 8, nb, rs, terms), 2);
  }
  if (flat && tt == 1) return launch_rg<2, 1, 4, true>(p, f32, s);
  if (flat) return launch_rg<2, 2, 4, true>(p, f32, s);
#define LQ_RG(TT)                                          \
  do {                                                     \
    if (rg == 4) return launch_rg<4, TT, 4, true>(p, f32, s); \
    return launch_rg<2, TT, 8, true>(p, f32, s);           \
  } while (0)
  if (tt == 1) LQ_RG(1);
  if (tt == 2) LQ_RG(2);
  if (rg == 4 && 2 * dc_lds_bytes(4, 4, 4, (int)(w[0].K / 64), v[0].rs + v[1].rs, terms) > kLdsBytes)
    return launch_rg<4, 4, 8, true>(p, f32, s);
  LQ_RG(4);
#undef LQ_RG
}

}  // namespace lq
