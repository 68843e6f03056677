// Internal declarations of the many-adapter path (include/lq_adapters.h).
#pragma once

#include "../../include/lq_adapters.h"
#include "lq_internal.h"

namespace lq {

// A route's arrays (lq_adapter_route): sorted positions by adapter.
struct Route {
  const int32_t* off;    // [n + 2]
  const int32_t* perm;   // [M] token of a sorted position
  const int32_t* sid;    // [M] adapter of a sorted position (n: none)
};
inline int64_t route_words(int64_t M, int32_t n) { return ((int64_t)n + 2 + 3) / 4 * 4 + 2 * ((M + 3) / 4 * 4); }
inline Route route_view(const int32_t* p, int64_t M, int32_t n) {
  const int64_t a = ((int64_t)n + 2 + 3) / 4 * 4, b = (M + 3) / 4 * 4;
  return Route{p, p + a, p + a + b};
}

// The set as the kernels see it. rs: r_max rounded up to a multiple of 8.
struct AdapterView {
  const lq_adapter* tab;   // device
  int32_t n;
  int32_t r_max;
  int32_t rs;
};

// s_a t and s_a u travel between the kernels as three bfloat16 terms, hi + mid
// + lo = the float32 value exactly (3 x 8 significand bits; short of it only
// where a term falls below bfloat16's range), an infinity or NaN as three
// copies of itself, in sorted order:
// row p holds the token of sorted position p, its hi terms in columns [0, r8),
// mid in [r8, 2 r8), lo in [2 r8, 3 r8) with r8 = r_a rounded up to a multiple
// of 8 (zero columns past r_a); row stride 3 rs. Rows of tokens without an
// adapter are not written. The matrix kernels take two terms for a bfloat16
// result and three for a float32 one.
inline size_t terms_elems(int64_t M, const AdapterView& v) { return (size_t)M * 3 * v.rs; }

// Row form over routed tokens: t[m][j] = sum_c Q[m][c] R_a[j][c], j < r_a, as
// terms of s_a t; or, with Q null, the terms of a given t.
struct DownJob {
  const uint16_t* Q;       // [M, C] bf16, or null
  int64_t C;               // C % 8 == 0
  const uint16_t* rbase;   // R_a at rbase + C * row8_a, or null: A_a of the table
  const float* given;      // Q null: t [M, r_max]
  uint16_t* terms;
  float* save;             // t [M, r_max] or null (zero past r_a and for tokens without an adapter)
  float* part;             // adapter_down_ws_floats(M, C, rs)
};
size_t adapter_down_ws_floats(int64_t M, int64_t C, int32_t rs);
hipError_t launch_adapter_down(const DownJob* jobs, int njobs, int64_t M, const AdapterView& v, const Route& rt,
                               const uint16_t* zeros, hipStream_t s);

// Preparation, one launch of independent parts, each left out where its
// pointer is null: 16 zero bytes (read by the other kernels in place of what
// lies past an end); the route of ids; the weight decoded to wd (W' [N, K], or,
// NF4 with ldb, W'^T [K, ldb], zero columns from N on); the adapters re-laid for the
// matrix kernels: at = A^T [K, r8] at K * row8_a, bt = B^T [r, N] at N *
// row8_a, bp = B [N, r8] at N * row8_a of the adapters whose rank is not a
// multiple of 8 (zero columns past r_a).
hipError_t launch_adapter_prep(const int32_t* ids, int64_t M, int32_t* route, const QWeight& w, uint16_t* wd,
                               int64_t ldb, const AdapterView& v, uint16_t* at, uint16_t* bt, uint16_t* bp,
                               uint16_t* zeros, hipStream_t s);

// Column form over routed tokens: out_a[j][c] = sum over a's tokens of
// (s_a P)[m][j] Q[m][c], written [r, C] at C * row_a, or transposed [C, r].
struct ColReq {
  const uint16_t* terms;   // of s_a P
  const uint16_t* Q;       // [M, C] bf16, C % 8 == 0
  int64_t C;
  float* out;
  int transposed;
  float* part;             // adapter_col_ws_floats
};
size_t adapter_col_ws_floats(int64_t M, int64_t C, int32_t rs);
hipError_t launch_adapter_col(const ColReq* reqs, int nreq, int64_t M, const AdapterView& v, const Route& rt,
                              hipStream_t s);

// out[token][c] = sum_k A[token][k] Bt[c][k] + sum_j (s_a L)[token][j] Lb_a(c, j)
// over the sorted positions; Lb_a(c, j): row c of lt + Ncols * row8_a
// [Ncols, r8]; of B_a itself where lt_all is 0 and r_a % 8 == 0.
struct AdapterGemm {
  const uint16_t* A;       // [M, Kc]
  int64_t M, Ncols, Kc;
  const uint16_t* Bt;      // [Ncols, ldb], ldb % 64 == 0, zero from Kc to ldb
  int64_t ldb;
  const uint16_t* terms;   // of s_a L
  AdapterView v;
  const uint16_t* lt;
  int lt_all;
  Route rt;
  void* out;               // [M, Ncols] bf16 or float32
  int out_f32;
  const uint16_t* zeros;   // 16 zero bytes
};
hipError_t launch_adapter_gemm(const AdapterGemm& g, hipStream_t s);
// [N, K] -> [K, ldb] bf16 (zero columns from N to ldb)
hipError_t launch_transpose_weight(const uint16_t* w, int64_t N, int64_t K, int64_t ldb, uint16_t* out, hipStream_t s);

// Decode sizes (NF4, M <= 64): the whole forward without a route, in two
// launches.
bool adapter_decode_supported(const QWeight& w, int64_t M);
size_t adapter_decode_ws_bytes(const QWeight& w, int64_t M, const AdapterView& v);
hipError_t launch_adapter_decode(const QWeight& w, const uint16_t* X, int64_t M, const int32_t* ids,
                                 const AdapterView& v, void* ws, float* t_save, void* H, bool f32, hipStream_t s);

// ---- gradient lists ----------------------------------------------------------
struct GradPiece {
  void* data;
  int32_t count;
  int32_t dtype;
};
struct GradSlot {
  int32_t first, count;        // pieces
  int32_t group;
  int32_t group_first;         // first slot of the group
  int32_t group_count;         // slots of the group
  int32_t pad[3];
};
constexpr int kGradThreads = 256;
hipError_t launch_grad_squares(const GradSlot* slots, const GradPiece* pieces, int32_t n_slots, double* part,
                               hipStream_t s);
hipError_t launch_grad_norms(const GradSlot* slots, int32_t n_slots, const double* part, float* norms, hipStream_t s);
hipError_t launch_grad_clip(const GradSlot* slots, const GradPiece* in, const GradPiece* out, int32_t n_slots,
                            const double* part, float max_norm, float eps, float* norms, hipStream_t s);

}  // namespace lq
