// Many adapters at decode sizes (up to 64 tokens), NF4 weight:
//   t[m] = A_a x[m],  h[m] = W' x[m] + s_a B_a t[m],  a = ids[m],
// without sorting the tokens: a wave holds one id per lane, so the tokens of
// an adapter are one ballot. Bound by reading the packed weight once and, per
// code, by the lookup, product and rounding that make its bfloat16 weight.
//
// QLoRA (Heng's Blog), introduction: h = dequant(W0_NF4) x + (alpha/r) B A x.
#include <algorithm>

#include "lq_adapters.h"
#include "lq_device.h"

namespace lq {
namespace {

__device__ __forceinline__ u32x4_t ld16(const void* p) { return *reinterpret_cast<const u32x4_t*>(p); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
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
__device__ __forceinline__ DcSteps dc_steps(const lq_adapter& ad, int key, int terms) {
  DcSteps st;
  st.ad = ad;
  // the tokens of the lane's adapter, from one ballot per bit of the key
  uint64_t peers = __ballot(key >= 0);
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    const uint64_t one = __ballot((key >> b) & 1);
    peers &= ((key >> b) & 1) ? one : ~one;
  }
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
  uint32_t runs;       // byte q, run q of the step: rank / 8, term << 4, 64 where it is one of the adapter's
  int32_t total;       // steps in all (every record)
};
constexpr int DC_PAD = 64;                        // no token's steps past the last: the projection asks for them too
constexpr int DC_RECORDS = 64 * 12 + DC_PAD;

// ===========================================================================
// t = A_a x: one workgroup per adapter in use (workgroup b takes the b-th in
// token order) and column part, 16 of its tokens at a time; the waves split
// the part's columns. The parts' sums go to t [parts][M][rs]; the projection
// adds them. The workgroups past the adapters' lay X out for the projection's
// fragments (xp, see XPack): a load of 16 rows is then 1 KB in one piece, where
// the rows themselves are 64 pieces of 16 bytes in 32 cache lines. Bound by
// latency: one token 4.4 us, 16 tokens of 16 adapters 5.6 (K = 4096), 64 tokens
// of 32 adapters, K = 8192, 13.
// ===========================================================================
// XPack: 16 bytes for (stage s, token tile tt, sub-step u, lane) at
// ((s TT + tt) 4 + u) 64 + lane: token 16 tt + lane % 16, columns 128 s + 32 (lane / 16) + 8 u
// of X, zero past K.
__device__ __forceinline__ int xp_units(int64_t K, int TT) { return (int)((K + 127) / 128) * TT * 256; }

template <int JT, int W>
__global__ __launch_bounds__(64 * W) void k_decode_down(const uint16_t* __restrict__ X, int M, int64_t K,
                                                        AdapterView v, const int32_t* __restrict__ ids,
                                                        float* __restrict__ t, u32x4_t* __restrict__ xp, int TT,
                                                        int wgs, DcRecord* __restrict__ records, int terms) {
  __shared__ f32x4_t part[W][JT][64];
  if ((int)blockIdx.x == wgs) {   // the steps, by the lanes that lead an adapter
    if (blockIdx.y || threadIdx.x >= 64) return;
    const int key = lane_key(ids, M, v.n);
    const DcSteps st = dc_steps(v.tab[max(key, 0)], key, terms);
    const int runs = (st.ad.r + 7) >> 3;
    for (int k = 0, term = 0, run = 0; k < st.count; ++k) {
      uint32_t packed = 0;
      for (int q = 0; q < 4; ++q) {
        if (term < terms) packed |= (uint32_t)(run | term << 4 | 64) << (8 * q);
        if (++run == runs) run = 0, ++term;
      }
      records[st.first + k] = DcRecord{(uint64_t)reinterpret_cast<uintptr_t>(st.ad.B), st.same, st.ad.scale, st.ad.r, packed,
                                       st.total};
    }
    const lq_adapter any = v.tab[0];
    if (threadIdx.x < DC_PAD)
      records[st.total + threadIdx.x] = DcRecord{(uint64_t)reinterpret_cast<uintptr_t>(any.B), 0, 0.0f, any.r, 0, st.total};
    return;
  }
  if ((int)blockIdx.x > wgs) {
    const int workers = ((int)gridDim.x - wgs - 1) * (int)gridDim.y * 64 * W;
    int i = (((int)blockIdx.x - wgs - 1) * (int)gridDim.y + (int)blockIdx.y) * 64 * W + (int)threadIdx.x;
    for (; i < xp_units(K, TT); i += workers) {
      const int ln = i & 63, u = (i >> 6) & 3, tt = (i >> 8) % TT, s = (i >> 8) / TT;
      const int64_t k = 128 * (int64_t)s + 32 * (ln >> 4) + 8 * u;
      u32x4_t x = {0u, 0u, 0u, 0u};
      if (k < K) x = ld16(X + (int64_t)min(16 * tt + (ln & 15), M - 1) * K + k);
      xp[i] = x;
    }
    return;
  }
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int key = lane_key(ids, M, v.n);
  uint64_t left = __ballot(key >= 0), mine = 0;
  int a = -1;
  for (int b = 0; left; ++b) {
    const int k = __shfl(key, __ffsll((unsigned long long)left) - 1);
    const uint64_t same = __ballot(key == k);
    if (b == (int)blockIdx.x) {
      a = uniform(k);
      mine = same;
      break;
    }
    left &= ~same;
  }
  if (a < 0) return;
  const lq_adapter ad = v.tab[a];
  const int r = min(ad.r, 16 * JT), count = __popcll(mine);
  const uint16_t* rr[JT];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) rr[jt] = ad.A + (int64_t)min(16 * jt + li, r - 1) * K;
  const int all = (int)(K / 64), per = (all + gridDim.y - 1) / gridDim.y;
  const int first = min(all, (int)blockIdx.y * per), blocks = min(all, first + per);   // this part's 64-column blocks
  t += (int64_t)blockIdx.y * M * v.rs;
  for (int t0 = 0; t0 < count; t0 += 16) {
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
    __syncthreads();
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
// rank 8 to 32: 71 us, that is 1.7 TB/s of codes, the launch before it 13. A
// workgroup's 60 us are 9 of start, 10 of the adapters' part (B is read from
// memory, 34 MB in all) and 38 of the stages, whose lookups and products wait
// for one another at two waves a SIMD: 64 tokens' sums and X take 128 registers.
// 16 tokens, N = K = 4096: 7.9 us after 5.6; one token: 7.5 after 4.4 (forming
// t in the projection instead took 14.0 in all).
// ===========================================================================
struct DecodeParams {
  const u32x4_t* xp;   // X in fragment order
  const DcRecord* records;
  int M;
  const int32_t* ids;
  AdapterView v;
  const float* t;      // [parts][M, rs]
  int parts;
  float* t_out;        // [M, r_max], or null
  void* out;
  QWeight w;
  Nf4Levels lv;
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

// floats of LDS after the pair table: constants, then the partial sums of one
// token tile
template <int RG, int W>
__host__ __device__ constexpr int dc_floats(int nb) {
  const int c = (16 * RG * (nb + 1) + 3) / 4 * 4, red = W * RG * 272;
  return c > red ? c : red;
}
size_t dc_lds_bytes(int rg, int tt, int w, int nb, int rs, int terms) {
  const int c = (16 * rg * (nb + 1) + 3) / 4 * 4, red = w * rg * 272;
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
template <int RG>
struct DcStep {
  u32x4_t w[RG];
  uint64_t same;
  float scale;
  int term, j0;
  bool live;
};
template <int RG>
__device__ __forceinline__ void dc_step(const DcRecord& rec, const int64_t (&row)[RG], DcStep<RG>& o) {
  const uint16_t* B = reinterpret_cast<const uint16_t*>(rec.B);
  const int r = rec.r;
  const uint32_t run = rec.runs >> (threadIdx.x >> 1 & 24);   // the lane's: byte lane / 16
  o.scale = rec.scale;
  o.same = rec.same;
  o.live = run & 64;
  o.term = (run >> 4) & 3;
  o.j0 = 8 * (run & 15);
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    const uint16_t* b = B + row[g] * r;
    if (r % 8 == 0) {
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
// Adds step o: each product goes to its own tokens' columns alone.
template <int RG, int TT, int TERMS>
__device__ __forceinline__ void dc_apply(const DcStep<RG>& o, const uint16_t* sT, int rs, int M, f32x4_t (&acc)[RG][TT]) {
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
    for (int g = 0; g < RG; ++g) {
      const f32x4_t d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(o.w[g]), as_bf16x8(tv), zero4(), 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // selected last: a scale that is not finite makes NaN of 0, too
        const float with = __builtin_fmaf(o.scale, d[e], acc[g][tt][e]);
        acc[g][tt][e] = mine ? with : acc[g][tt][e];
      }
    }
  }
}

template <int RG, int TT, int W, bool DQ, bool OUT_F32>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2))) void k_decode_nf4(DecodeParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char dc_lds[];
  constexpr int TERMS = OUT_F32 ? 3 : 2;
  constexpr bool XA = TT == 1;   // X is loaded a stage ahead, with the codes
  f32x2_t* sPair = reinterpret_cast<f32x2_t*>(dc_lds);
  float* sC = reinterpret_cast<float*>(dc_lds + DC_PAIRS * sizeof(f32x2_t));
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  const int64_t N = p.w.N, K = p.w.K;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * RG;
  const int nb = (int)(K / 64), pitch = nb + 1, ns = (nb + 1) / 2;
  uint16_t* sT = reinterpret_cast<uint16_t*>(sC + dc_floats<RG, W>(nb));   // t's bf16 terms [M][TERMS][rs]

  const uint8_t* crow[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) crow[g] = p.w.codes + min(n0 + 16 * g + li, N - 1) * (K / 2) + 16 * (lg & 1);
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
  constexpr int DEEP = RG == 4 ? 4 : 1;   // (few row groups: 16 tokens' steps are one or two a wave)
  static_assert(W * 2 * DEEP <= DC_PAD, "the steps asked for end within the padding");
  int64_t row[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) row[g] = min(n0 + 16 * g + li, N - 1);
  DcStep<RG> steps[DEEP];
  DcStage<RG> s0, s1;
  load(wave, s0);
  if constexpr (XA) load(wave + W, s1);
  // Lane l keeps the record of the wave's step 64 c + l.
  DcRecord rec;
  auto load_records = [&](int i) {
    const u32x4_t* at = reinterpret_cast<const u32x4_t*>(p.records + min(wave + W * (i + lane), DC_RECORDS - 1));
    const u32x4_t a = at[0], b = at[1];
    rec = DcRecord{a[0] | (uint64_t)a[1] << 32, a[2] | (uint64_t)a[3] << 32, __uint_as_float(b[0]), (int)b[1], b[2], (int)b[3]};
  };
  auto ask = [&](int i, DcStep<RG>& o) { dc_step<RG>(of_lane(rec, i & 63), row, o); };
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
  const float mean = DQ ? *p.w.qc.dq_mean : 0.0f;
  // the rows' constants, four a thread: thread t row t % (16 RG)
  if (nb % 4 == 0) {
    const int rr = threadIdx.x % (16 * RG);
    const int64_t b0 = min(n0 + rr, N - 1) * nb;
#pragma unroll 4
    for (int c = 4 * (threadIdx.x / (16 * RG)); c < nb; c += 4 * (64 * W / (16 * RG))) {
      const int64_t blk = b0 + c;   // a multiple of 4: one second-level scale
      f32x4_t v;
      if constexpr (DQ) {
        const uint32_t q8 = *reinterpret_cast<const uint32_t*>(p.w.qc.absmax_q + blk);
        const float s2 = p.w.qc.dq_scale[blk >> 8];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(e4m3_decode((q8 >> (8 * e)) & 0xFFu), s2, mean);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = p.w.qc.absmax[blk + e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sC[rr * pitch + c + e] = v[e];
    }
  } else {
    for (int i = threadIdx.x; i < 16 * RG * nb; i += 64 * W) {
      const int rr = i / nb, bl = i - rr * nb;
      const int64_t blk = min(n0 + rr, N - 1) * nb + bl;
      sC[rr * pitch + bl] = DQ ? __builtin_fmaf(e4m3_decode(p.w.qc.absmax_q[blk]), p.w.qc.dq_scale[blk >> 8], mean)
                               : p.w.qc.absmax[blk];
    }
  }
  {
    // t: its parts added in order, and split into bf16 terms: two keep 16 bits
    // of it, 8 more than a bf16 H, three all 24 (rows of tokens without an
    // adapter hold anything: no step takes them). Token m's t is saved by workgroup m % grid.
    const int quads = p.v.rs / 4, nq = p.M * quads, nt = p.M * p.v.rs;
#pragma unroll 2
    for (int i = threadIdx.x; i < nq; i += 64 * W) {
      f32x4_t part[DC_PARTS];
#pragma unroll
      for (int k = 0; k < DC_PARTS; ++k)
        part[k] = *reinterpret_cast<const f32x4_t*>(p.t + (int64_t)min(k, p.parts - 1) * nt + 4 * i);
      f32x4_t sum = part[0];
#pragma unroll
      for (int k = 1; k < DC_PARTS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += k < p.parts ? part[k][e] : 0.0f;
      const int m = (uint32_t)i / (uint32_t)quads, j = 4 * (i - m * quads);
      if (p.t_out && m % gridDim.x == blockIdx.x) {
        const bool has = (uint32_t)p.ids[m] < (uint32_t)p.v.n;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < p.v.r_max) p.t_out[m * p.v.r_max + j + e] = has ? sum[e] : 0.0f;
      }
      float v[4] = {sum[0], sum[1], sum[2], sum[3]};
#pragma unroll
      for (int q = 0; q < TERMS; ++q) {
        const uint2 bits = {take_bf16_terms(v[0], v[1]), take_bf16_terms(v[2], v[3])};
        *reinterpret_cast<uint2*>(sT + (m * TERMS + q) * p.v.rs + j) = bits;
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
      dc_apply<RG, TT, TERMS>(steps[d], sT, p.v.rs, p.M, acc);
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
    for (int g = 0; g < RG; ++g) cp[g] = sC[(16 * g + li) * pitch + st.bl];
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
    for (int i = threadIdx.x; i < RG * 64; i += 64 * W) {
      const int quad = i & 3, g = (i >> 2) % RG, m = i / (4 * RG);
      f32x4_t h = sR[g * 68 + m + 17 * quad];
#pragma unroll
      for (int w = 1; w < W; ++w) h += sR[(w * RG + g) * 68 + m + 17 * quad];
      const int64_t n = n0 + 16 * g + 4 * quad;
      if (16 * tt + m >= p.M || n >= N) continue;
      const int64_t o = (int64_t)(16 * tt + m) * N + n;
      if (N % 4 == 0) {
        if (OUT_F32) {
          float* f = reinterpret_cast<float*>(p.out) + o;   // 4-byte aligned
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = h[e];
        } else {
          uint2 v;
          v.x = pack_bf16x2(h[0], h[1]);
          v.y = pack_bf16x2(h[2], h[3]);
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + o) = v;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (n + e >= N) break;
          if (OUT_F32) reinterpret_cast<float*>(p.out)[o + e] = h[e];
          else reinterpret_cast<uint16_t*>(p.out)[o + e] = (uint16_t)(pack_bf16x2(h[e], 0.f) & 0xFFFFu);
        }
      }
    }
  }
}

template <int RG, int TT, int W>
hipError_t launch_rg(const DecodeParams& p, bool f32, hipStream_t s) {
  const dim3 grid((unsigned)((p.w.N + 16 * RG - 1) / (16 * RG))), block(64 * W);
  const size_t lds = dc_lds_bytes(RG, TT, W, (int)(p.w.K / 64), p.v.rs, f32 ? 3 : 2);
  const bool dq = p.w.qc.absmax == nullptr;
  if (dq && f32) hipLaunchKernelGGL((k_decode_nf4<RG, TT, W, true, true>), grid, block, lds, s, p);
  else if (dq) hipLaunchKernelGGL((k_decode_nf4<RG, TT, W, true, false>), grid, block, lds, s, p);
  else if (f32) hipLaunchKernelGGL((k_decode_nf4<RG, TT, W, false, true>), grid, block, lds, s, p);
  else hipLaunchKernelGGL((k_decode_nf4<RG, TT, W, false, false>), grid, block, lds, s, p);
  return hipGetLastError();
}

constexpr int kCus = 256;
constexpr size_t kLdsBytes = 160 * 1024;

// Row groups per workgroup: the shortest queue of the longest CU, a workgroup
// costing its row groups and about two more for its start and its X. Four need
// the LDS of two workgroups (K up to some 10000).
int decode_rg(int64_t N, int64_t K, int tt, int rs, int terms) {
  const int64_t groups = (N + 15) / 16;
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int rg = 1; rg <= 4; rg *= 2) {
    const size_t lds = rg == 4 ? 2 * dc_lds_bytes(rg, tt, 4, (int)(K / 64), rs, terms)
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

}  // namespace

// NF4, at most 64 tokens, and one row group's constants within the LDS that the
// table (32 KB) and t's terms (at most 48 KB) leave.
bool adapter_decode_supported(const QWeight& w, int64_t M) {
  return w.format == LQ_FMT_NF4 && M <= 64 && w.K <= 49152;
}
// Token tiles of the projection, and the workspace: t's parts, the steps, and
// X in fragment order.
static int token_tiles(int64_t M) { return M <= 16 ? 1 : (M <= 32 ? 2 : 4); }
static int adapter_decode_parts(const QWeight& w, int64_t M, const AdapterView& v);
static size_t t_bytes(const QWeight& w, int64_t M, const AdapterView& v) {
  return ((size_t)adapter_decode_parts(w, M, v) * M * v.rs * sizeof(float) + 255) / 256 * 256;
}
size_t adapter_decode_ws_bytes(const QWeight& w, int64_t M, const AdapterView& v) {
  return t_bytes(w, M, v) + DC_RECORDS * sizeof(DcRecord) + (size_t)((w.K + 127) / 128) * token_tiles(M) * 256 * 16;
}

// Column parts of t: with few adapters the columns are shared by several
// workgroups, at least eight 64-column blocks each.
static int adapter_decode_parts(const QWeight& w, int64_t M, const AdapterView& v) {
  const int64_t wgs = std::min<int64_t>(M, v.n);
  int parts = 1;
  while (parts < DC_PARTS && wgs * parts * 2 <= kCus && w.K / 64 / (parts * 2) >= 8) parts *= 2;
  return parts;
}

hipError_t launch_adapter_decode(const QWeight& w, const uint16_t* X, int64_t M, const int32_t* ids,
                                 const AdapterView& v, void* ws, float* t_save, void* H, bool f32, hipStream_t s) {
  if (!adapter_decode_supported(w, M)) return hipErrorInvalidValue;
  const int parts = adapter_decode_parts(w, M, v), tt = token_tiles(M);
  float* t_ws = reinterpret_cast<float*>(ws);
  DcRecord* records = reinterpret_cast<DcRecord*>(reinterpret_cast<char*>(ws) + t_bytes(w, M, v));
  u32x4_t* xp = reinterpret_cast<u32x4_t*>(records + DC_RECORDS);
  const int wgs = (int)std::min<int64_t>(M, v.n);
  const dim3 grid((unsigned)(wgs + 1 + std::max(1, 16 * tt / parts)), (unsigned)parts);
  const int jt = (v.r_max + 15) / 16;
#define LQ_DD(JT, W)                                                                                                 \
  hipLaunchKernelGGL((k_decode_down<JT, W>), grid, dim3(64 * W), 0, s, X, (int)M, w.K, v, ids, t_ws, xp, tt, wgs, records, \
                     f32 ? 3 : 2)
  if (jt <= 1) LQ_DD(1, 16);
  else if (jt <= 2) LQ_DD(2, 16);
  else if (jt <= 4) LQ_DD(4, 8);
  else LQ_DD(8, 8);
#undef LQ_DD
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const DecodeParams p{xp, records, (int)M, ids, v, t_ws, parts, t_save, H, w, tables().lv};
  const int rg = decode_rg(w.N, w.K, tt, v.rs, f32 ? 3 : 2);
#define LQ_RG(TT)                                    \
  do {                                               \
    if (rg == 4) return launch_rg<4, TT, 4>(p, f32, s); \
    if (rg == 2) return launch_rg<2, TT, 8>(p, f32, s); \
    return launch_rg<1, TT, 8>(p, f32, s);           \
  } while (0)
  if (tt == 1) LQ_RG(1);
  if (tt == 2) LQ_RG(2);
  LQ_RG(4);
#undef LQ_RG
}

}  // namespace lq
