// Many adapters over one projection: the route (tokens sorted by adapter) and
// the skinny products t = A_a x, u = B_a^T g, dA_a = s u^T X, dB_a = s G^T t.
//
// QLoRA (Heng's Blog), introduction: h = dequant(W0_NF4) x + (alpha/r) B A x,
// here with an adapter (A, B, alpha, r) per token.
#include <algorithm>

#include "lq_adapters.h"
#include "lq_device.h"
#include "lq_route.h"

namespace lq {
namespace {

// ===========================================================================
// Route: a stable counting sort of the tokens by adapter, by one workgroup.
// Wave w owns a contiguous run of tokens; pass 1 counts its tokens per adapter
// in LDS (integer additions: their order does not matter), the counts are
// scanned over adapters and waves, and pass 2 gives each token of a 64-token
// group its place among the group's equal ids from ballots (one per bit of
// the id). Bound by the latency of its few dependent passes; the first
// RT_KEEP groups of a wave keep their ids in registers between the passes.
// About 4 us at 250 tokens; in a call that decodes a weight too it runs beside
// that (k_adapter_prep) and costs nothing of its own.
// ===========================================================================
constexpr int RT_WAVES = 16, RT_KEEP = 4;

struct RouteJob {
  const int32_t* ids;   // null: no token has an adapter
  int64_t M;
  int32_t n;
  int32_t *off, *perm, *sid;
};
constexpr size_t route_lds_bytes(int n) { return (size_t)(RT_WAVES * (n + 1) + RT_WAVES) * sizeof(int32_t); }

__device__ __forceinline__ void route_tokens(const RouteJob& jb, int32_t* cnt) {
  const int n = jb.n, keys = n + 1;
  const int64_t M = jb.M;
  int32_t* wsum = cnt + RT_WAVES * keys;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t per = ((M + RT_WAVES - 1) / RT_WAVES + 63) / 64 * 64;
  const int64_t m0 = min(M, wave * per), m1 = min(M, m0 + per);
  // (one branch for all of them: a branch at each load would wait for the one before)
  int keep[RT_KEEP];
  if (jb.ids) {
#pragma unroll
    for (int g = 0; g < RT_KEEP; ++g) keep[g] = jb.ids[min(m0 + 64 * g + lane, M - 1)];
  } else {
#pragma unroll
    for (int g = 0; g < RT_KEEP; ++g) keep[g] = -1;
  }
  for (int i = threadIdx.x; i < RT_WAVES * keys; i += 64 * RT_WAVES) cnt[i] = 0;
  __syncthreads();
  auto key_of = [&](int id) { return (uint32_t)id < (uint32_t)n ? id : n; };
#pragma unroll
  for (int g = 0; g < RT_KEEP; ++g)
    if (m0 + 64 * g + lane < m1) atomicAdd(&cnt[wave * keys + key_of(keep[g])], 1);
  if (jb.ids)
    for (int64_t m = m0 + 64 * RT_KEEP + lane; m < m1; m += 64) atomicAdd(&cnt[wave * keys + key_of(jb.ids[m])], 1);
  else
    for (int64_t m = m0 + 64 * RT_KEEP + lane; m < m1; m += 64) atomicAdd(&cnt[wave * keys + n], 1);
  __syncthreads();
  // totals per key (thread k; keys <= 1024), waves' counts to exclusive sums
  const int k = threadIdx.x;
  int total = 0;
  if (k < keys) {
    int c[RT_WAVES];
#pragma unroll
    for (int w = 0; w < RT_WAVES; ++w) c[w] = cnt[w * keys + k];
#pragma unroll
    for (int w = 0; w < RT_WAVES; ++w) {
      const int x = c[w];
      c[w] = total;
      total += x;
    }
#pragma unroll
    for (int w = 0; w < RT_WAVES; ++w) cnt[w * keys + k] = c[w];
  }
  int inc = total;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int base = inc - total;
#pragma unroll
  for (int w = 0; w < RT_WAVES; ++w) base += w < wave ? wsum[w] : 0;
  if (k < keys) {
    jb.off[k] = base;
    if (k == n) jb.off[n + 1] = (int32_t)M;
#pragma unroll
    for (int w = 0; w < RT_WAVES; ++w) cnt[w * keys + k] += base;
  }
  __syncthreads();
  int bits = 0;
  while ((n >> bits) != 0) ++bits;
  auto place = [&](int64_t g, int id) {
    const int64_t m = g + lane;
    const bool live = m < m1;
    const int key = key_of(id);
    uint64_t peers = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t one = __ballot((key >> b) & 1);
      peers &= ((key >> b) & 1) ? one : ~one;
    }
    const int rank = __popcll(peers & ((uint64_t(1) << lane) - 1));
    volatile int32_t* c = &cnt[wave * keys + key];
    const int start = *c;                      // the wave's LDS operations run in order:
    __builtin_amdgcn_wave_barrier();           // every lane reads before the group's first lane of a key adds
    if (live && rank == 0) *c = start + __popcll(peers);
    __builtin_amdgcn_wave_barrier();
    if (live) {
      jb.perm[start + rank] = (int32_t)m;
      jb.sid[start + rank] = key;
    }
  };
#pragma unroll
  for (int g = 0; g < RT_KEEP; ++g)
    if (m0 + 64 * g < m1) place(m0 + 64 * g, keep[g]);
  for (int64_t g = m0 + 64 * RT_KEEP; g < m1; g += 64) place(g, g + lane < m1 && jb.ids ? jb.ids[g + lane] : -1);
}

// ===========================================================================
// Preparation, one launch: workgroup 0 builds the route, the others decode the
// weight (as it lies; NF4 transposed for the backward) and re-lay the
// adapters; none of it depends on the rest. Bound by writing the bfloat16
// weight: 4096 x 4096 10 us as it lies and 14 transposed (4.2 and 3.0 TB/s of
// codes and weight together), 11008 x 4096 25 and 43 us; the transposing form
// also writes the adapters' copies. Codebook 4096 x 4096: 16 us, of which about
// half is the chain from a row's width and offset to its first planes (a
// workgroup per row and a launch after the route's took 4 + 18).
// ===========================================================================
constexpr int PW_T = 128;                 // transposed: tiles of PW_T weight rows x PW_T columns
constexpr int PW_PITCH = PW_T + 16;       // bf16 per LDS row: the transposing reads of 4 rows hit distinct banks
constexpr int PW_FLAT = 4;                // as it lies: pieces of 16 codes per thread, all in flight together
constexpr int PC_ROWS = 8;                // codebook: rows per workgroup, two per 256 threads, their loads together
constexpr int RL_C = 128;                 // re-laid per workgroup: RL_C rows of A^T or B

struct PrepJob {
  RouteJob route;
  QWeight w;
  Nf4Levels lv;
  uint16_t* wd;          // W' [N, K], or transposed [K, ldb] (zero columns past N); null: not wanted
  int64_t ldb;           // 0: not transposed
  int64_t wcols;         // columns written of the transposed rows
  AdapterView v;
  uint16_t *at, *bt, *bp;
  uint16_t* zeros;       // 16 bytes, cleared
  unsigned route_wgs, weight_wgs, per_adapter, at_wgs, b_wgs;
};

// 16 codes (one 64-block's) and what makes their constant.
struct RawCodes {
  uint32_t code[2], q8;
  float c, s2;
};
template <bool DQ>
__device__ __forceinline__ RawCodes load_codes(const QWeight& w, int64_t e) {
  RawCodes r{};
  const uint32_t* src = reinterpret_cast<const uint32_t*>(w.codes + e / 2);
  r.code[0] = src[0];
  r.code[1] = src[1];
  const int64_t blk = e >> 6;
  if (DQ) {
    r.q8 = w.qc.absmax_q[blk];
    r.s2 = w.qc.dq_scale[blk >> 8];
  } else {
    r.c = w.qc.absmax[blk];
  }
  return r;
}
template <bool DQ>
__device__ __forceinline__ void decode16(const RawCodes& r, float mean, const f32x2_t* sPair, u32x4_t (&o)[2]) {
  const float c = DQ ? __builtin_fmaf(e4m3_decode(r.q8), r.s2, mean) : r.c;
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const f32x2_t q = sPair[(r.code[b >> 2] >> (8 * (b & 3))) & 0xFFu];
    o[b >> 2][b & 3] = pack_bf16x2(q.x * c, q.y * c);
  }
}

template <bool DQ>
__device__ __forceinline__ void prep_weight(const PrepJob& p, unsigned wg, unsigned char* lds) {
  f32x2_t* sPair = reinterpret_cast<f32x2_t*>(lds);
  uint16_t* sW = reinterpret_cast<uint16_t*>(lds + 256 * sizeof(f32x2_t));
  const int64_t N = p.w.N, K = p.w.K;
  const float mean = DQ ? *p.w.qc.dq_mean : 0.0f;
  if (!p.ldb) {
    const int64_t e0 = (int64_t)wg * (PW_FLAT * 1024 * 16) + threadIdx.x * 16, last = N * K - 16;
    RawCodes raw[PW_FLAT];
#pragma unroll
    for (int u = 0; u < PW_FLAT; ++u) raw[u] = load_codes<DQ>(p.w, min(e0 + u * 1024 * 16, last));
    if (threadIdx.x < 256) sPair[threadIdx.x] = f32x2_t{p.lv.q[threadIdx.x >> 4], p.lv.q[threadIdx.x & 15]};
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PW_FLAT; ++u) {
      const int64_t e = e0 + u * 1024 * 16;
      u32x4_t o[2];
      decode16<DQ>(raw[u], mean, sPair, o);
      if (e <= last) {
        u32x4_t* dst = reinterpret_cast<u32x4_t*>(p.wd + e);
        dst[0] = o[0];
        dst[1] = o[1];
      }
    }
    return;
  }
  // transposed: row tiles inner, so that neighbours write the same lines of W'^T
  const unsigned nt = (unsigned)((N + PW_T - 1) / PW_T);
  const int64_t n0 = PW_T * (int64_t)(wg % nt), k0 = PW_T * (int64_t)(wg / nt);
  const int row = threadIdx.x >> 3, piece = threadIdx.x & 7;
  const int64_t n = n0 + row, k = k0 + 16 * piece;
  const bool live = n < N && k < K;
  const RawCodes raw = load_codes<DQ>(p.w, live ? n * K + k : 0);
  if (threadIdx.x < 256) sPair[threadIdx.x] = f32x2_t{p.lv.q[threadIdx.x >> 4], p.lv.q[threadIdx.x & 15]};
  __syncthreads();
  u32x4_t o[2];
  decode16<DQ>(raw, mean, sPair, o);
  if (!live) o[0] = o[1] = u32x4_t{0u, 0u, 0u, 0u};
  u32x4_t* st = reinterpret_cast<u32x4_t*>(sW + row * PW_PITCH + 16 * piece);
  st[0] = o[0];
  st[1] = o[1];
  __syncthreads();
  // wave w: columns 16 (w % 8), rows 64 (w / 8) of the tile; lane (li, lg):
  // column li, rows 32 h + 8 lg + [0, 8)
  typedef __bf16 v4b __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) v4b* lds_p;
  const int wave = threadIdx.x >> 6, li = threadIdx.x & 15, lg = (threadIdx.x & 63) >> 4;
  const int64_t kk = k0 + 16 * (wave & 7) + li;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r0 = 64 * (wave >> 3) + 32 * h + 8 * lg;
    const uint16_t* src = sW + (r0 + (li >> 2)) * PW_PITCH + 16 * (wave & 7) + 4 * (li & 3);
    const u32x2_t a = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_p)src));
    const u32x2_t b = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_p)(src + 4 * PW_PITCH)));
    if (kk < K && n0 + r0 < p.wcols)   // N in whole runs of 64
      *reinterpret_cast<u32x4_t*>(p.wd + kk * p.ldb + n0 + r0) = u32x4_t{a[0], a[1], b[0], b[1]};
  }
}

// Codebook rows: 16 codes a thread, two bytes of each of the row's bit planes.
// The row's levels become a table of 256 pairs whose index interleaves the bits
// of two adjacent codes, so that a pair is one 2-bit field of each plane.
template <bool DQ>
__device__ __forceinline__ void prep_codebook(const PrepJob& p, unsigned wg, unsigned char* lds) {
  const int64_t N = p.w.N, K = p.w.K;
  const int part = threadIdx.x >> 8, th = threadIdx.x & 255;
  f32x2_t* sPair = reinterpret_cast<f32x2_t*>(lds) + 512 * part;   // of the part's two rows
  const float mean = DQ ? *p.w.qc.dq_mean : 0.0f;
  int64_t row[2];
  int bits[2];
  const uint8_t* src[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    row[u] = min((int64_t)wg * PC_ROWS + 2 * part + u, N - 1);   // past the last row: decoded, not stored
    bits[u] = min(max((int)p.w.row_bits[row[u]], 1), 4);
    src[u] = p.w.codes + p.w.row_offset[row[u]];
    uint32_t f = 0, g = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      f |= ((th >> (2 * b)) & 1u) << b;
      g |= ((th >> (2 * b + 1)) & 1u) << b;
    }
    sPair[256 * u + th] = f32x2_t{p.w.levels[row[u] * 16 + f], p.w.levels[row[u] * 16 + g]};
  }
  __syncthreads();
  for (int64_t i = th; i < K / 16; i += 256) {
    const int64_t blk = i >> 2;
    uint32_t plane[2][4], q8[2];
    float c[2], s2[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* at = src[u] + blk * 8 * bits[u] + 2 * (i & 3);
#pragma unroll
      for (int b = 0; b < 4; ++b) plane[u][b] = b < bits[u] ? at[8 * b] | (uint32_t)at[8 * b + 1] << 8 : 0u;
      const int64_t cb = row[u] * (K / 64) + blk;
      if (DQ) {
        q8[u] = p.w.qc.absmax_q[cb];
        s2[u] = p.w.qc.dq_scale[cb >> 8];
      } else {
        c[u] = p.w.qc.absmax[cb];
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float cp = DQ ? __builtin_fmaf(e4m3_decode(q8[u]), s2[u], mean) : c[u];
      u32x4_t o[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t idx = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) idx |= ((plane[u][b] >> (2 * e)) & 3u) << (2 * b);
        const f32x2_t q = sPair[256 * u + idx];
        o[e >> 2][e & 3] = pack_bf16x2(q.x * cp, q.y * cp);
      }
      if ((int64_t)wg * PC_ROWS + 2 * part + u < N) {
        u32x4_t* dst = reinterpret_cast<u32x4_t*>(p.wd + row[u] * K + 16 * i);
        dst[0] = o[0];
        dst[1] = o[1];
      }
    }
  }
}

// at[k][j] = A[j][k], bp[n][j] = B[n][j] (j < r8, zero past r), bt[j][n] = B[n][j],
// through an LDS tile of RL_C rows (k or n) x r8.
__device__ __forceinline__ void prep_adapter(const PrepJob& p, unsigned a, unsigned wg, unsigned char* lds) {
  uint16_t* s = reinterpret_cast<uint16_t*>(lds);
  const lq_adapter ad = p.v.tab[a];
  const int r = min(ad.r, 128), r8 = (r + 7) & ~7, pitch = r8 + 2;   // an odd count of 4-byte words
  const int64_t N = p.w.N, K = p.w.K;
  const bool of_a = wg < p.at_wgs;
  const int64_t x0 = RL_C * (int64_t)(of_a ? wg : wg - p.at_wgs), X = of_a ? K : N;
  if (x0 >= X) return;
  const int rows = (int)min((int64_t)RL_C, X - x0);
  if (of_a) {
    for (int i = threadIdx.x; i < r8 * RL_C; i += 1024) {
      const int j = i / RL_C, x = i % RL_C;
      s[x * pitch + j] = j < r && x < rows ? ad.A[j * K + x0 + x] : (uint16_t)0;
    }
    __syncthreads();
    uint16_t* out = p.at + K * ad.row8 + x0 * r8;
    for (int i = threadIdx.x; i < rows * r8 / 2; i += 1024) {
      const int x = i / (r8 / 2), j = 2 * (i % (r8 / 2));
      reinterpret_cast<uint32_t*>(out)[i] = *reinterpret_cast<const uint32_t*>(s + x * pitch + j);
    }
    return;
  }
  const uint16_t* B = ad.B + x0 * r;
  for (int i = threadIdx.x; i < rows * r; i += 1024) s[i / r * pitch + i % r] = B[i];
  __syncthreads();
  if (p.bt)
    for (int i = threadIdx.x; i < r * RL_C; i += 1024) {
      const int j = i / RL_C, x = i % RL_C;
      if (x < rows) p.bt[N * ad.row8 + j * N + x0 + x] = s[x * pitch + j];
    }
  if (p.bp && r % 8)
    for (int i = threadIdx.x; i < rows * r8; i += 1024) {
      const int x = i / r8, j = i % r8;
      p.bp[N * ad.row8 + (x0 + x) * r8 + j] = j < r ? s[x * pitch + j] : (uint16_t)0;
    }
}

// PAIR: two weights with their sets, the second's workgroups after the first's:
// both NF4 weights 4096 -> 11008 decoded 47 us (225 MB read and written, 4.8
// TB/s), transposed for the backward, with the adapters' layouts, 78.
template <bool PAIR>
struct PrepJobs {
  PrepJob j[PAIR ? 2 : 1];
  unsigned first;   // workgroups of the first
};

template <bool PAIR>
__global__ __launch_bounds__(1024) void k_adapter_prep(PrepJobs<PAIR> jobs) {
  extern __shared__ __attribute__((aligned(16))) unsigned char prep_lds[];
  const unsigned second = PAIR && blockIdx.x >= jobs.first ? 1 : 0;
  const PrepJob& p = jobs.j[second];
  unsigned wg = blockIdx.x - second * jobs.first;
  if (wg == 0 && threadIdx.x < 8 && p.zeros) p.zeros[threadIdx.x] = 0;
  if (wg < p.route_wgs) {
    route_tokens(p.route, reinterpret_cast<int32_t*>(prep_lds));
    return;
  }
  wg -= p.route_wgs;
  if (wg < p.weight_wgs) {
    if (p.w.format == LQ_FMT_CODEBOOK) {
      if (p.w.qc.absmax) prep_codebook<false>(p, wg, prep_lds);
      else prep_codebook<true>(p, wg, prep_lds);
    } else {
      if (p.w.qc.absmax) prep_weight<false>(p, wg, prep_lds);
      else prep_weight<true>(p, wg, prep_lds);
    }
    return;
  }
  wg -= p.weight_wgs;
  if (p.per_adapter) prep_adapter(p, wg / p.per_adapter, wg % p.per_adapter, prep_lds);
}

// The three bfloat16 terms of v.
__device__ __forceinline__ void split3(float v, uint16_t (&o)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    float none = 0.0f;
    o[k] = (uint16_t)take_bf16_terms(v, none);
  }
}

// t[row][j] = x of the token at sorted position pos: kept as given, and as the terms of s_a x.
__device__ __forceinline__ void put_t(const DownJob& jb, const AdapterView& v, const Route& rt, const lq_adapter& ad,
                                      int64_t pos, int j, float x) {
  const int r8 = (ad.r + 7) & ~7;
  if (jb.save && j < v.r_max) jb.save[(int64_t)rt.perm[pos] * v.r_max + j] = x;
  if (j < r8) {
    uint16_t o[3];
    split3(ad.scale * x, o);
    uint16_t* d = jb.terms + pos * 3 * v.rs + j;
#pragma unroll
    for (int k = 0; k < 3; ++k) d[k * r8] = o[k];
  }
}

// ===========================================================================
// Row form, few tokens: 16 routed tokens of one adapter per workgroup; its W waves take
// contiguous runs of 64-column blocks, MFMA 16x16x32 with tokens as rows and
// the adapter's rows as columns, both straight from memory into registers, a
// wave's next U blocks loading while the current ones are multiplied. The
// waves' partial sums meet in LDS and are added in wave order. Bound by the
// count of its 16-byte load instructions, which scattered rows make slow: 10 us
// at 250 to 2048 tokens of rank 16, K = 4096; 6 at 300 tokens, K = 1024.
// ===========================================================================
template <int JT, int W, int U, bool DROP>
__global__ __launch_bounds__(64 * W) void k_adapter_down(DownJobs jobs, int64_t M, Route rt) {
  __shared__ f32x4_t part[W][JT][64];
  const DownJob jb = jobs.j[blockIdx.y];
  const AdapterView& v = jb.v;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  Item it;
  if (!find_item(rt.off, v.n + 1, 16, (int)blockIdx.x, it)) return;
  if (it.seg == v.n) {   // tokens without an adapter
    if (jb.save)
      for (int i = threadIdx.x; i < it.count * v.r_max; i += 64 * W)
        jb.save[(int64_t)rt.perm[it.start + i / v.r_max] * v.r_max + i % v.r_max] = 0.0f;
    return;
  }
  const lq_adapter ad = v.tab[it.seg];
  const int r = min(ad.r, 16 * JT), r8 = (r + 7) & ~7;
  auto put = [&](int row, int j, float x) { put_t(jb, v, rt, ad, it.start + row, j, jb.post * x); };
  if (!jb.Q) {
    for (int i = threadIdx.x; i < it.count * r8; i += 64 * W) {
      const int row = i / r8, j = i - row * r8;
      put(row, j, j < r ? jb.given[(int64_t)rt.perm[it.start + row] * v.r_max + j] : 0.0f);
    }
    return;
  }
  const int64_t C = jb.C;
  const uint16_t* R = jb.rbase ? jb.rbase + C * ad.row8 : ad.A;
  const int64_t token = rt.perm[it.start + min(li, it.count - 1)];
  const uint16_t* q = jb.Q + token * C;
  const bool drops = DROP && jb.drop.T;
  DropGen gen{};
  if (drops) gen = drop_gen(jb.drop);
  const uint16_t* rr[JT];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) rr[jt] = R + (int64_t)min(16 * jt + li, r - 1) * C;
  f32x4_t acc[JT];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) acc[jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int blocks = (int)((C + 63) / 64), per = (blocks + W - 1) / W;
  const int b0 = min(blocks, wave * per), b1 = min(blocks, b0 + per);
  struct Set {
    u32x4_t a[U][2], w[U][2][JT];
  };
  auto load = [&](int b, Set& s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t c = 64 * (int64_t)(b + u) + 32 * h + 8 * lg;   // 64 bytes of each row a load
        const bool ok = b + u < b1 && c + 8 <= C;   // past the end: zeros in place of columns 0 .. 7
        const int64_t o = ok ? c : 0;
        s.a[u][h] = ld16(q + o);
#pragma unroll
        for (int jt = 0; jt < JT; ++jt) s.w[u][h][jt] = ld16(rr[jt] + o);
        if (!ok) {
          s.a[u][h] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
          for (int jt = 0; jt < JT; ++jt) s.w[u][h][jt] = u32x4_t{0u, 0u, 0u, 0u};
        }
      }
  };
  auto mul = [&](int b, const Set& s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4_t a = s.a[u][h];
        if (drops) a = drop_16bit(a, drop_bits(gen, (uint64_t)(token * (C / 8) + 8 * (int64_t)(b + u) + 4 * h + lg)), jb.drop.T);
#pragma unroll
        for (int jt = 0; jt < JT; ++jt)
          acc[jt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(s.w[u][h][jt]), acc[jt], 0, 0, 0);
      }
  };
  Set s0, s1;
  if (b0 < b1) load(b0, s0);
  for (int b = b0; b < b1; b += 2 * U) {
    if (b + U < b1) load(b + U, s1);
    mul(b, s0);
    if (b + U >= b1) break;
    if (b + 2 * U < b1) load(b + 2 * U, s0);
    mul(b + U, s1);
  }
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) part[wave][jt][lane] = acc[jt];
  __syncthreads();
  for (int i = threadIdx.x; i < JT * 256; i += 64 * W) {
    // consecutive threads: consecutive columns of one token
    const int row = i / (16 * JT), j = i % (16 * JT), jt = j >> 4;
    if (row >= it.count) continue;
    const int ln = 16 * (row >> 2) + (j & 15);
    float sum = part[0][jt][ln][row & 3];
#pragma unroll
    for (int w = 1; w < W; ++w) sum += part[w][jt][ln][row & 3];
    put(row, j, j < r ? sum : 0.0f);
  }
}

// ===========================================================================
// Row form, many tokens: 64 routed tokens of one adapter x BN of its rows per
// workgroup (a fourth of the reads of the adapter that 16 tokens cost), over a
// share of the columns; tiles through a ring of four LDS buffers filled by
// memory-to-LDS loads three 64-wide steps ahead. The shares' sums, float32 in
// sorted order [shares][M][rs], are joined by k_adapter_down_join, which also
// turns a given t into terms. 4096 tokens of rank 64, K = 4096: 19 + 6 us for
// 34 MB of X (7 us at the rate of a large copy); 1999 tokens of rank 8 to 64:
// 8.6 + 5.
//
// DROP: the generator's rounds (two blocks a lane and step) cost more issue than
// a step's products, so three buffers, whose three workgroups per CU fill each
// other's gaps, and shares of each job's own columns: 4096 tokens of rank 64, t
// over 11008 columns and u over 4096 in one launch, 45 us (four buffers and equal
// shares: 60).
// ===========================================================================
constexpr int DT_M = 64, DT_K = 64, DT_RING = 4;

template <int BN, bool DROP>
__global__ __launch_bounds__(256) void k_adapter_down_tiles(DownJobs jobs, int64_t M, Route rt, const uint16_t* zeros) {
  constexpr int CT = BN / 16, QW = BN >= 32 ? BN / 32 : 1, RING = DROP ? 3 : DT_RING;
  struct __attribute__((aligned(16))) Lds {
    uint16_t x[RING][DT_M * DT_K];
    uint16_t w[RING][(BN < 32 ? 32 : BN) * DT_K];
  };
  __shared__ Lds lds;
  const DownJob jb = jobs.j[blockIdx.z];
  const AdapterView& v = jb.v;
  const int shares = DROP ? jb.shares : (int)gridDim.y;
  if (!jb.Q || (DROP && (int)blockIdx.y >= shares)) return;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  Item it;
  if (!find_item(rt.off, v.n, DT_M, (int)blockIdx.x, it)) return;
  const lq_adapter ad = v.tab[it.seg];
  const int r = min(ad.r, BN);
  const int64_t C = jb.C;
  const uint16_t* R = jb.rbase ? jb.rbase + C * ad.row8 : ad.A;
  const int all = (int)((C + DT_K - 1) / DT_K), per = (all + shares - 1) / shares;
  const int s0 = min(all, (int)blockIdx.y * per), s1 = min(all, s0 + per);
  // a load instruction of a wave fills 8 rows of 128 bytes: lane l row l / 8,
  // slot l % 8 with chunk slot ^ (row % 8)
  const int sub = lane >> 3, ch = (lane & 7) ^ sub;
  const uint16_t *px[2], *pw[QW];
#pragma unroll
  for (int q = 0; q < 2; ++q)
    px[q] = jb.Q + (int64_t)rt.perm[it.start + min((wave * 2 + q) * 8 + sub, it.count - 1)] * C + 8 * ch;
#pragma unroll
  for (int q = 0; q < QW; ++q) pw[q] = R + (int64_t)min((wave * QW + q) * 8 + sub, r - 1) * C + 8 * ch;
  auto load = [&](int s) {   // step s into its buffer; past the end zeros (the count of outstanding loads stays)
    const int buf = (s - s0) % RING;
    const int64_t k0 = (int64_t)s * DT_K;
    const bool ok = s < s1 && k0 + 8 * ch + 8 <= C;
#pragma unroll
    for (int q = 0; q < 2; ++q) load_lds16(ok ? px[q] + k0 : zeros, lds.x[buf] + (wave * 2 + q) * 8 * DT_K);
#pragma unroll
    for (int q = 0; q < QW; ++q) load_lds16(ok ? pw[q] + k0 : zeros, lds.w[buf] + (wave * QW + q) * 8 * DT_K);
  };
  f32x4_t acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < RING - 1; ++k) load(s0 + k);
  const int slot[2] = {8 * (lg ^ (li & 7)), 8 * ((4 + lg) ^ (li & 7))};
  const bool drops = DROP && jb.drop.T;
  DropGen gen{};
  int64_t block = 0;   // of the generator: the lane's token and first column
  if (drops) {
    gen = drop_gen(jb.drop);
    block = rt.perm[it.start + min(16 * wave + li, it.count - 1)] * (C / 8) + lg;
  }
  for (int s = s0; s < s1; ++s) {
    u32x4_t bits[2];   // before the wait: the generator's rounds run while the tile travels
    if (drops)
#pragma unroll
      for (int u = 0; u < 2; ++u) bits[u] = drop_bits(gen, (uint64_t)(block + 8 * (int64_t)s + 4 * u));
    // this wave's share of step s is there and its reads of s - 1 are done; then everyone's
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((RING - 2) * (2 + QW)) : "memory");
    load(s + RING - 1);
    const int buf = (s - s0) % RING;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      u32x4_t a = ld16(lds.x[buf] + (16 * wave + li) * DT_K + slot[u]);
      if (drops) a = drop_16bit(a, bits[u], jb.drop.T);
#pragma unroll
      for (int c = 0; c < CT; ++c)
        acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(ld16(lds.w[buf] + (16 * c + li) * DT_K + slot[u])),
                                                         acc[c], 0, 0, 0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // before the workgroup's LDS is given up
  // lane: tokens 16 wave + 4 lg + e, row 16 c + li of the adapter
  float* part = jb.part + (int64_t)blockIdx.y * M * v.rs;
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 16 * wave + 4 * lg + e, j = 16 * c + li;
      if (row < it.count && j < r) part[(int64_t)(it.start + row) * v.rs + j] = acc[c][e];
    }
}

__global__ __launch_bounds__(256) void k_adapter_down_join(DownJobs jobs, int64_t M, Route rt) {
  const DownJob jb = jobs.j[blockIdx.y];
  const AdapterView& v = jb.v;
  const int64_t total = M * v.rs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t pos = i / v.rs;
    const int j = (int)(i - pos * v.rs), a = rt.sid[pos];
    if (a >= v.n) {   // a token without an adapter
      if (jb.save && j < v.r_max) jb.save[(int64_t)rt.perm[pos] * v.r_max + j] = 0.0f;
      continue;
    }
    const lq_adapter ad = v.tab[a];
    float x = 0.0f;
    if (j < ad.r) {
      if (jb.Q) {
        x = jb.part[i];
        for (int k = 1; k < jb.shares; ++k) x += jb.part[k * total + i];
        x *= jb.post;
      } else {
        x = jb.given[(int64_t)rt.perm[pos] * v.r_max + j];
      }
    }
    put_t(jb, v, rt, ad, pos, j, x);
  }
}

// The tiled form pays once the tokens fill it: at 2048 tokens of rank 16 the
// two took 10.5 us alike, at 4096 tokens of rank 64 45 against 23 us.
bool down_tiled(int64_t M, int32_t rs) { return M * rs >= 65536; }

// DROP: shares of each job's columns, of about `len` steps each, len chosen for the
// shortest queue where three workgroups run on a CU, a share costing about three
// steps more. At most 16, and 4096 tiles of sums in all, 1 MB per rank (65536 tokens:
// four shares instead of sixteen, 134 MB of rank 128 instead of 537), past which shares
// only even out the last of many rounds.
int64_t drop_shares_most(int64_t M) {
  return std::max<int64_t>(1, std::min<int64_t>(16, 4096 / ((M + DT_M - 1) / DT_M)));
}
void drop_shares(int64_t M, const int64_t* steps, int n, int* shares) {
  const int64_t tiles = (M + DT_M - 1) / DT_M, limit = drop_shares_most(M);
  int64_t most = 1, best = INT64_MAX;
  for (int i = 0; i < n; ++i) most = std::max(most, steps[i]);
  for (int64_t len = (most + limit - 1) / limit; len <= most; ++len) {
    int64_t all = 0;
    for (int i = 0; i < n; ++i) all += (steps[i] + len - 1) / len;
    const int64_t cost = (tiles * all + 767) / 768 * (len + 3);
    if (cost >= best) continue;
    best = cost;
    for (int i = 0; i < n; ++i) shares[i] = (int)std::max<int64_t>(1, (steps[i] + len - 1) / len);
  }
}

// Shares of the columns: two workgroups per CU, at least 8 steps each.
int down_shares(int64_t M, int64_t C) {
  const int64_t tiles = (M + DT_M - 1) / DT_M, steps = (C + DT_K - 1) / DT_K;
  int s = 1;
  while (s < 16 && tiles * s * 2 <= 512 && steps / (s * 2) >= 8) s *= 2;
  return s;
}

// ===========================================================================
// Column form: out_a[j][c] = sum_m (s_a P)[m][j] Q[m][c] over a's tokens. One
// workgroup per 256 columns (64 a wave) and run of at most `rows` sorted
// positions; 32 tokens per step. P comes as three bfloat16 terms, so the
// products carry float32 P on the bf16 matrix cores; all three go into the same
// accumulators. P and Q tiles lie in LDS with tokens as rows (the next step's
// loads are in flight while one is multiplied; two buffers up to rank 32, above
// it one and a second barrier, so that three workgroups fit a CU: rank 64 59 ->
// 55 us, rank 16 with one buffer 12.8 -> 13.4), and are read transposed
// (ds_read_b64_tr_b16: the 16 lanes of a group point at 4 rows of 16 elements,
// lane l gets column l of the 4 rows). Tokens past the segment are zero in
// both, so no neighbour's infinity or NaN enters. Bound by the chain of
// a step (stage, barrier, transposed reads) at three workgroups per CU:
// dA and dB of 2048 tokens of rank 16, N = K = 4096, 12.7 us for 34 MB; of 4096
// tokens of rank 64, N = 4096, K = 11008, 55 for 124 MB. Two steps in flight
// instead of one did not change that.
// ===========================================================================
constexpr int CQ_COLS = 256, CQ_PITCH = CQ_COLS + 16;

template <int JT, bool DROP>
__global__ __launch_bounds__(256, JT <= 4 ? 3 : 1) void k_adapter_col(ColReq q0, ColReq q1, unsigned tiles0, int rows, Route rt) {
  constexpr int PP = 16 * JT + 16;
  constexpr int BUFS = JT <= 2 ? 2 : 1;
  constexpr int PQ = (3 * 32 * 2 * JT + 255) / 256;   // 16-byte pieces of P per thread
  __shared__ __attribute__((aligned(16))) uint16_t sQ[BUFS][32 * CQ_PITCH];
  __shared__ __attribute__((aligned(16))) uint16_t sP[BUFS][3 * 32 * PP];
  const bool second = blockIdx.x >= tiles0;
  const ColReq rq = second ? q1 : q0;
  const AdapterView& v = rq.v;
  Item it;
  if (!find_item(rt.off, v.n, rows, (int)blockIdx.y, it)) return;
  const lq_adapter ad = v.tab[it.seg];
  const int r = min(ad.r, 16 * JT), r8 = (r + 7) & ~7;
  const int64_t C = rq.C, c0 = (int64_t)(second ? blockIdx.x - tiles0 : blockIdx.x) * CQ_COLS;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int li = lane & 15, lg = lane >> 4;
  // thread: columns 8 (t % 32) of tokens t / 32 + 8 u of Q; pieces of 8 columns
  // of (term, token) of P
  const int qc = 8 * (threadIdx.x & 31), qr = threadIdx.x >> 5;
  const bool qin = c0 + qc + 8 <= C;
  const bool drops = DROP && rq.drop.T;
  DropGen gen{};
  if (drops) gen = drop_gen(rq.drop);
  u32x4_t xq[4], xp[PQ];
  int tok[4], of[4];   // tokens to load next, and those in xq
  auto tokens = [&](int mb) {   // of the step's rows (a valid one past the end)
#pragma unroll
    for (int u = 0; u < 4; ++u) tok[u] = rt.perm[it.start + min(mb + qr + 8 * u, it.count - 1)];
  };
  auto load = [&](int mb) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      xq[u] = ld16(rq.Q + (int64_t)tok[u] * C + (qin ? c0 + qc : 0));
      of[u] = tok[u];
    }
#pragma unroll
    for (int k = 0; k < PQ; ++k) {
      const int i = threadIdx.x + 256 * k, c8 = i % (2 * JT), row = (i / (2 * JT)) % 32, term = min(i / (64 * JT), 2);
      xp[k] = ld16(rq.terms + (int64_t)(it.start + min(mb + row, it.count - 1)) * 3 * v.rs +
                   (8 * c8 < r8 ? term * r8 + 8 * c8 : 0));
    }
  };
  auto store = [&](int mb, int b) {
    const u32x4_t none = {0u, 0u, 0u, 0u};
    if (drops)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        xq[u] = drop_16bit(xq[u], drop_bits(gen, (uint64_t)(of[u] * (C / 8) + (c0 + qc) / 8)), rq.drop.T);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<u32x4_t*>(sQ[b] + (qr + 8 * u) * CQ_PITCH + qc) = qin && mb + qr + 8 * u < it.count ? xq[u] : none;
#pragma unroll
    for (int k = 0; k < PQ; ++k) {
      const int i = threadIdx.x + 256 * k, c8 = i % (2 * JT), row = (i / (2 * JT)) % 32, term = i / (64 * JT);
      if (term < 3)
        *reinterpret_cast<u32x4_t*>(sP[b] + (32 * term + row) * PP + 8 * c8) = mb + row < it.count && 8 * c8 < r8 ? xp[k] : none;
    }
  };
  f32x4_t acc[JT][4];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt)
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) acc[jt][ct] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  tokens(0);
  load(0);
  tokens(32);
  auto step = [&](int m, int b) {
    store(m, b);
    __syncthreads();
    load(m + 32);
    tokens(m + 64);
    u32x4_t fq[4];
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) fq[ct] = tr_frag(sQ[b] + 64 * wave + 16 * ct, CQ_PITCH, li, lg);
#pragma unroll
    for (int t = 0; t < 3; ++t)
#pragma unroll
      for (int jt = 0; jt < JT; ++jt) {
        const u32x4_t a = tr_frag(sP[b] + 32 * t * PP + 16 * jt, PP, li, lg);
#pragma unroll
        for (int ct = 0; ct < 4; ++ct)
          acc[jt][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(fq[ct]), acc[jt][ct], 0, 0, 0);
      }
  };
  for (int m = 0; m < it.count; m += 32 * BUFS) {
    step(m, 0);
    if constexpr (BUFS == 2) {
      if (m + 32 < it.count) step(m + 32, 1);
    } else {
      lds_barrier();   // read by everyone; the next step's loads stay in flight
    }
  }
  // lane: column li of each tile, rows j = 4 lg + e. Partial sums lie as
  // [slot][rs][C] (16 lanes 64 bytes in a row; [C][rs] measured slower).
  const bool vec = rq.transposed && it.slot < 0 && r % 4 == 0 && (reinterpret_cast<uintptr_t>(rq.out) & 15) == 0;
#pragma unroll
  for (int jt = 0; jt < JT; ++jt)
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      const int64_t c = c0 + 64 * wave + 16 * ct + li;
      const int j0 = 16 * jt + 4 * lg;
      if (c >= C || j0 >= r) continue;
      if (vec) {   // C * row and c * r are multiples of 4
        *reinterpret_cast<f32x4_t*>(rq.out + C * ad.row + c * r + j0) = acc[jt][ct];
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + e;
        if (j >= r) break;
        if (it.slot >= 0) rq.part[((int64_t)it.slot * v.rs + j) * C + c] = acc[jt][ct][e];
        else if (rq.transposed) rq.out[C * ad.row + c * r + j] = acc[jt][ct][e];
        else rq.out[(ad.row + (int64_t)j) * C + c] = acc[jt][ct][e];
      }
    }
}

// Joins the runs of adapters with more than one, in order, and writes the zero
// gradients of adapters without tokens. 6 us at 2048 tokens of rank 16, 13 at
// 4096 of rank 64 (four partial sums a thread at a time).
//
// A transposed output's rows (a column's r sums) are put together in LDS, 64
// columns and 32 of the r a workgroup: written from registers, 16 bytes here and
// there, they took twice as long. Zeros need no order and are written as they lie
// (61 adapters of rank 1, five tokens: 9.6 us through LDS, 3.2 so).
constexpr int CR_COLS = 64, CR_ROWS = 32;
struct ColJoins {
  ColJoin j[2];
};
__global__ __launch_bounds__(256) void k_adapter_col_reduce(ColJoins joins, Route rt) {
  __shared__ float tile[CR_COLS * (CR_ROWS + 1)];
  const ColJoin& jn = joins.j[blockIdx.z];
  const int rows = jn.rows;
  const int a = blockIdx.y, lane = threadIdx.x & 63;
  const int runs = (rt.off[a + 1] - rt.off[a] + rows - 1) / rows;
  if (runs == 1) return;
  const ColReq q0 = jn.q[0], q1 = jn.q[jn.n > 1 ? 1 : 0];
  const lq_adapter ad0 = q0.v.tab[a], ad1 = q1.v.tab[a];
  int before = 0;   // slots of the adapters before a, where there are runs to join
  if (runs) {
    for (int b = lane; b < a; b += 64) {
      const int c = (rt.off[b + 1] - rt.off[b] + rows - 1) / rows;
      before += c > 1 ? c : 0;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) before += __shfl_xor(before, d);
  }
  // workgroups' shares: of a transposed output as above, 1024 values of another and of zeros (C % 8 == 0)
  auto units = [&](const ColReq& q, int r) {
    return q.transposed && runs ? (q.C + CR_COLS - 1) / CR_COLS * ((r + CR_ROWS - 1) / CR_ROWS) : (r * q.C / 4 + 255) / 256;
  };
  const int64_t n0 = units(q0, ad0.r), n1 = jn.n > 1 ? units(q1, ad1.r) : 0;
  for (int64_t unit = blockIdx.x; unit < n0 + n1; unit += gridDim.x) {
    const bool second = unit >= n0;
    const int64_t t = second ? unit - n0 : unit, C = second ? q1.C : q0.C;
    const int r = second ? ad1.r : ad0.r, rs = second ? q1.v.rs : q0.v.rs;
    float* out = (second ? q1.out : q0.out) + C * (second ? ad1.row : ad0.row);   // 4-byte aligned
    const float* part = (second ? q1.part : q0.part) + (int64_t)before * rs * C;
    if (runs && (second ? q1.transposed : q0.transposed)) {
      const int64_t tiles = (C + CR_COLS - 1) / CR_COLS, c0 = t % tiles * CR_COLS;
      const int j0 = (int)(t / tiles) * CR_ROWS, n = min(CR_ROWS, r - j0), cols = (int)min((int64_t)CR_COLS, C - c0);
      for (int j = 4 * (threadIdx.x >> 6); j < n; j += 16) {   // four rows a thread (rs, a multiple of 8, are there)
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (lane < cols)
          for (int k = 0; k < runs; ++k) {
            const float* p = part + ((int64_t)k * rs + j0 + j) * C + c0 + lane;
#pragma unroll
            for (int u = 0; u < 4; ++u) sum[u] += p[u * C];
          }
#pragma unroll
        for (int u = 0; u < 4; ++u) tile[lane * (CR_ROWS + 1) + j + u] = sum[u];
      }
      __syncthreads();
      for (int i = threadIdx.x; i < cols * n; i += 256) out[(c0 + i / n) * r + j0 + i % n] = tile[i / n * (CR_ROWS + 1) + i % n];
      __syncthreads();
    } else {
      const int64_t i = t * 256 + threadIdx.x;
      if (i >= r * C / 4) continue;
      const int64_t j = 4 * i / C, c = 4 * i % C;
      f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int k = 0; k < runs; ++k) sum += *reinterpret_cast<const f32x4_t*>(part + ((int64_t)k * rs + j) * C + c);
#pragma unroll
      for (int u = 0; u < 4; ++u) out[4 * i + u] = sum[u];
    }
  }
}

// Sorted positions per workgroup of the column form: enough workgroups for
// the chip, but runs of at least 256 tokens so that the partial sums stay few.
int col_rows(int64_t M, int64_t cols) {
  const int64_t tiles = (cols + CQ_COLS - 1) / CQ_COLS;
  int64_t rows = M * tiles / 448 / 32 * 32;
  return (int)std::max<int64_t>(256, std::min<int64_t>(rows, 4096));
}

}  // namespace

namespace {

// Fills a job; returns its workgroups and raises lds to what they need.
int64_t prep_job(const Prep& a, int64_t M, const int32_t* ids, PrepJob* out, size_t* lds) {
  PrepJob p{};
  if (a.route) {
    const Route r = route_view(a.route, M, a.v.n);
    p.route = RouteJob{ids, M, a.v.n, const_cast<int32_t*>(r.off), const_cast<int32_t*>(r.perm), const_cast<int32_t*>(r.sid)};
    p.route_wgs = 1;
    *lds = std::max(*lds, route_lds_bytes(a.v.n));
  }
  p.w = a.w;
  p.lv = tables().lv;
  p.wd = a.wd;
  p.ldb = a.ldb;
  p.wcols = (a.w.N + 63) / 64 * 64;
  if (a.wd) {
    const int64_t flat = PW_FLAT * 1024 * 16;
    if (a.w.format == LQ_FMT_CODEBOOK) {
      p.weight_wgs = (unsigned)((a.w.N + PC_ROWS - 1) / PC_ROWS);
      *lds = std::max(*lds, (size_t)PC_ROWS * 256 * sizeof(f32x2_t));
    } else {
      p.weight_wgs = (unsigned)(a.ldb ? ((a.w.N + PW_T - 1) / PW_T) * ((a.w.K + PW_T - 1) / PW_T) : (a.w.N * a.w.K + flat - 1) / flat);
      *lds = std::max(*lds, 256 * sizeof(f32x2_t) + (a.ldb ? (size_t)PW_T * PW_PITCH * 2 : 0));
    }
  }
  p.v = a.v;
  p.at = a.at;
  p.bt = a.bt;
  p.bp = a.bp;
  p.zeros = a.zeros;
  p.at_wgs = a.at ? (unsigned)((a.w.K + RL_C - 1) / RL_C) : 0;
  p.b_wgs = a.bt || a.bp ? (unsigned)((a.w.N + RL_C - 1) / RL_C) : 0;
  p.per_adapter = p.at_wgs + p.b_wgs;
  if (p.per_adapter) *lds = std::max(*lds, (size_t)RL_C * (a.v.rs + 2) * 2);
  *out = p;
  return (int64_t)p.route_wgs + p.weight_wgs + (int64_t)a.v.n * p.per_adapter;
}

}  // namespace

hipError_t launch_adapter_prep(const int32_t* ids, int64_t M, const Prep* a, int n, hipStream_t s) {
  if (n < 1 || n > 2) return hipErrorInvalidValue;
  for (int i = 0; i < n; ++i) LQ_DASSERT(!a[i].wd || a[i].w.format == LQ_FMT_NF4 || !a[i].ldb);
  size_t lds = 0;
  if (n == 1) {
    PrepJobs<false> jobs{};
    const int64_t grid = std::max<int64_t>(1, prep_job(a[0], M, ids, &jobs.j[0], &lds));
    LQ_DASSERT(grid < (int64_t(1) << 31) && lds <= 65536);
    hipLaunchKernelGGL(k_adapter_prep<false>, dim3((unsigned)grid), dim3(1024), lds, s, jobs);
  } else {
    PrepJobs<true> jobs{};
    const int64_t first = std::max<int64_t>(1, prep_job(a[0], M, ids, &jobs.j[0], &lds));   // (one clears the zeros)
    const int64_t grid = first + prep_job(a[1], M, ids, &jobs.j[1], &lds);
    LQ_DASSERT(grid < (int64_t(1) << 31) && lds <= 65536);
    jobs.first = (unsigned)first;
    hipLaunchKernelGGL(k_adapter_prep<true>, dim3((unsigned)grid), dim3(1024), lds, s, jobs);
  }
  return hipGetLastError();
}

size_t adapter_down_ws_floats(int64_t M, int64_t C, int32_t rs, bool drops) {
  if (!down_tiled(M, rs)) return 0;
  const int64_t steps = (C + DT_K - 1) / DT_K, most = drops ? std::min(drop_shares_most(M), steps) : 1;
  return (size_t)std::max<int64_t>(down_shares(M, C), most) * M * rs;
}

hipError_t launch_adapter_join(const DownJob* jobs, int njobs, int64_t M, const Route& rt, hipStream_t s) {
  if (njobs < 1 || njobs > kDownJobs) return hipErrorInvalidValue;
  DownJobs all{};
  int32_t rs = 0;
  for (int i = 0; i < njobs; ++i) {
    all.j[i] = jobs[i];
    rs = std::max(rs, jobs[i].v.rs);
  }
  const unsigned gx = (unsigned)std::min<int64_t>((M * rs + 255) / 256, 8192);
  hipLaunchKernelGGL(k_adapter_down_join, dim3(gx, (unsigned)njobs), dim3(256), 0, s, all, M, rt);
  return hipGetLastError();
}

hipError_t launch_adapter_down(const DownJob* jobs, int njobs, int64_t M, const Route& rt, const uint16_t* zeros,
                               hipStream_t s) {
  if (njobs < 1 || njobs > kDownJobs) return hipErrorInvalidValue;
  DownJobs all{};
  bool drops = false, tiled = false;
  int32_t r_max = 0;
  const int32_t n = jobs[0].v.n;
  for (int i = 0; i < njobs; ++i) {
    all.j[i] = jobs[i];
    drops |= jobs[i].drop.T != 0;
    r_max = std::max(r_max, jobs[i].v.r_max);
    tiled |= down_tiled(M, jobs[i].v.rs);
  }
  // jobs of one form each: of sets whose ranks differ, some may be tiled
  if (tiled)
    for (int i = 0; i < njobs; ++i)
      if (!down_tiled(M, jobs[i].v.rs)) {
        if (njobs == 1) return hipErrorInvalidValue;
        DownJob a[kDownJobs], b[kDownJobs];
        int na = 0, nb = 0;
        for (int k = 0; k < njobs; ++k) (down_tiled(M, jobs[k].v.rs) ? a[na++] : b[nb++]) = jobs[k];
        const hipError_t e = launch_adapter_down(a, na, M, rt, zeros, s);
        return e != hipSuccess ? e : launch_adapter_down(b, nb, M, rt, zeros, s);
      }
  if (tiled) {
    int64_t C = 0;
    for (int i = 0; i < njobs; ++i)
      if (jobs[i].Q) C = C ? std::min(C, jobs[i].C) : jobs[i].C;   // all jobs' workspaces hold these shares
    int shares = C ? down_shares(M, C) : 1;
    for (int i = 0; i < njobs; ++i) all.j[i].shares = shares;
    if (C && drops) {
      int64_t steps[kDownJobs];
      int own[kDownJobs];
      for (int i = 0; i < njobs; ++i) steps[i] = jobs[i].Q ? (jobs[i].C + DT_K - 1) / DT_K : 0;
      drop_shares(M, steps, njobs, own);
      shares = 1;
      for (int i = 0; i < njobs; ++i) shares = std::max(shares, all.j[i].shares = own[i]);
    }
    if (C) {
      const dim3 grid((unsigned)((M + DT_M - 1) / DT_M + std::min<int64_t>(n, M)), (unsigned)shares, (unsigned)njobs);
#define LQ_AT(BN)                                                                                      \
  do {                                                                                                 \
    if (drops) hipLaunchKernelGGL((k_adapter_down_tiles<BN, true>), grid, dim3(256), 0, s, all, M, rt, zeros); \
    else hipLaunchKernelGGL((k_adapter_down_tiles<BN, false>), grid, dim3(256), 0, s, all, M, rt, zeros);      \
  } while (0)
      if (r_max <= 16) LQ_AT(16);
      else if (r_max <= 32) LQ_AT(32);
      else if (r_max <= 64) LQ_AT(64);
      else LQ_AT(128);
#undef LQ_AT
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return launch_adapter_join(all.j, njobs, M, rt, s);
  }
  // one item per 16 tokens, and one more per adapter (or none) for its remainder
  const dim3 grid((unsigned)((M + 15) / 16 + std::min<int64_t>(n + 1, M)), (unsigned)njobs);
#define LQ_AD(JT, W, U)                                                                              \
  do {                                                                                               \
    if (drops) hipLaunchKernelGGL((k_adapter_down<JT, W, U, true>), grid, dim3(64 * W), 0, s, all, M, rt); \
    else hipLaunchKernelGGL((k_adapter_down<JT, W, U, false>), grid, dim3(64 * W), 0, s, all, M, rt);      \
  } while (0)
  if (r_max <= 16) LQ_AD(1, 16, 2);
  else if (r_max <= 32) LQ_AD(2, 8, 2);
  else if (r_max <= 64) LQ_AD(4, 8, 1);
  else LQ_AD(8, 8, 1);
#undef LQ_AD
  return hipGetLastError();
}

// A segment of more than one run of `rows` has at most 2 len / rows of them.
size_t adapter_col_ws_floats(int64_t M, int64_t C, int32_t rs) {
  const int64_t rows = 256;
  return (size_t)(2 * ((M + rows - 1) / rows)) * rs * C;
}

hipError_t launch_adapter_col(const ColReq* reqs, int nreq, int64_t M, const Route& rt, ColJoin* join, hipStream_t s) {
  if (nreq < 1 || nreq > 2) return hipErrorInvalidValue;
  const ColReq q0 = reqs[0], q1 = reqs[nreq - 1];
  const bool drops = q0.drop.T || q1.drop.T;
  const int rows = col_rows(M, q0.C + (nreq > 1 ? q1.C : 0));
  const unsigned t0 = (unsigned)((q0.C + CQ_COLS - 1) / CQ_COLS);
  const unsigned t1 = nreq > 1 ? (unsigned)((q1.C + CQ_COLS - 1) / CQ_COLS) : 0u;
  const dim3 grid(t0 + t1, (unsigned)((M + rows - 1) / rows + std::min<int64_t>(q0.v.n, M)));
  switch ((std::max(q0.v.r_max, q1.v.r_max) + 15) / 16) {
#define LQ_AC(JT)                                                                                                  \
  case JT:                                                                                                         \
    if (drops) hipLaunchKernelGGL((k_adapter_col<JT, true>), grid, dim3(256), 0, s, q0, q1, t0, rows, rt);         \
    else hipLaunchKernelGGL((k_adapter_col<JT, false>), grid, dim3(256), 0, s, q0, q1, t0, rows, rt);              \
    break;
    LQ_AC(1) LQ_AC(2) LQ_AC(3) LQ_AC(4) LQ_AC(5) LQ_AC(6) LQ_AC(7) LQ_AC(8)
#undef LQ_AC
    default: return hipErrorInvalidValue;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  *join = ColJoin{{q0, q1}, nreq, rows, M <= rows};
  return hipSuccess;
}

hipError_t launch_adapter_col_reduce(const ColJoin* joins, int n, const Route& rt, hipStream_t s) {
  if (n < 1 || n > 2) return hipErrorInvalidValue;
  ColJoins all{};
  int64_t most = 0;
  for (int i = 0; i < n; ++i) {
    const ColJoin& j = all.j[i] = joins[i];
    int64_t units = 0;
    for (int k = 0; k < j.n; ++k) {
      const ColReq& q = j.q[k];
      units += q.transposed && !j.zeros ? (q.C + CR_COLS - 1) / CR_COLS * ((q.v.r_max + CR_ROWS - 1) / CR_ROWS)
                            : (q.v.r_max * q.C / 4 + 255) / 256;
    }
    most = std::max(most, units);
  }
  const int32_t sets = joins[0].q[0].v.n;
  const unsigned gx = (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, std::max(32, 4096 / sets)));
  hipLaunchKernelGGL(k_adapter_col_reduce, dim3(gx, (unsigned)sets, (unsigned)n), dim3(256), 0, s, all, rt);
  return hipGetLastError();
}

}  // namespace lq
