// Internal declarations of the many-adapter path (include/lq_adapters.h).
#pragma once

#include "../../include/lq_adapters.h"
#include "lq_dropout.h"
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

// Row form over routed tokens: t[m][j] = post * sum_c Q[m][c] R_a[j][c], j < r_a,
// Q's dropped elements left out, as terms of s_a t; or, with Q null, the terms
// of a given t.
struct DownJob {
  const uint16_t* Q;       // [M, C] bf16, or null
  int64_t C;               // C % 8 == 0
  const uint16_t* rbase;   // R_a at rbase + C * row8_a, or null: A_a of the table
  const float* given;      // Q null: t [M, r_max]
  uint16_t* terms;
  float* save;             // t [M, r_max] or null (zero past r_a and for tokens without an adapter)
  float* part;             // adapter_down_ws_floats(M, C, rs, drops)
  DropView drop;           // element m C + c of Q
  float post;              // 1 for a given t
  AdapterView v;           // sets of one n
  int shares;              // of the columns, joined in order (the launcher's)
};
constexpr int kDownJobs = 4;
struct DownJobs {
  DownJob j[kDownJobs];
};
size_t adapter_down_ws_floats(int64_t M, int64_t C, int32_t rs, bool drops);   // drops: of a call with dropout
hipError_t launch_adapter_down(const DownJob* jobs, int njobs, int64_t M, const Route& rt, const uint16_t* zeros,
                               hipStream_t s);
// The last part alone: `shares` partial sums of each job (or a given t) to terms.
hipError_t launch_adapter_join(const DownJob* jobs, int njobs, int64_t M, const Route& rt, hipStream_t s);

// Preparation, one launch of independent parts, each left out where its
// pointer is null: 16 zero bytes (read by the other kernels in place of what
// lies past an end); the route of ids (ids null with a route: all tokens without
// an adapter); the weight decoded to wd (W' [N, K], or, NF4 with ldb, W'^T [K, N
// rounded up to a multiple of 64] of row stride ldb, zero columns past N); the adapters re-laid for the
// matrix kernels: at = A^T [K, r8] at K * row8_a, bt = B^T [r, N] at N *
// row8_a, bp = B [N, r8] at N * row8_a of the adapters whose rank is not a
// multiple of 8 (zero columns past r_a).
struct Prep {
  int32_t* route;
  QWeight w;
  uint16_t* wd;
  int64_t ldb;
  AdapterView v;
  uint16_t *at, *bt, *bp, *zeros;
};
// Of one weight, or of two of one size (the route of the first's).
hipError_t launch_adapter_prep(const int32_t* ids, int64_t M, const Prep* a, int n, hipStream_t s);

// Column form over routed tokens: out_a[j][c] = sum over a's tokens of
// (s_a P)[m][j] Q[m][c], written [r, C] at C * row_a, or transposed [C, r].
struct ColReq {
  const uint16_t* terms;   // of s_a P
  const uint16_t* Q;       // [M, C] bf16, C % 8 == 0
  int64_t C;
  float* out;
  int transposed;
  float* part;             // adapter_col_ws_floats
  DropView drop;           // element m C + c of Q is left out
  AdapterView v;           // sets of one n
};
size_t adapter_col_ws_floats(int64_t M, int64_t C, int32_t rs);
// Two launches: the products, and the join of the runs of `rows` positions of
// adapters with more than one, which also writes the zeros of adapters without
// tokens (of one or two such products).
struct ColJoin {
  ColReq q[2];
  int n, rows;
  bool zeros;              // no adapter can have more than one run
};
hipError_t launch_adapter_col(const ColReq* reqs, int nreq, int64_t M, const Route& rt, ColJoin* join, hipStream_t s);
hipError_t launch_adapter_col_reduce(const ColJoin* joins, int n, const Route& rt, hipStream_t s);

// out[token][c] = sum_k A[token][k] Bt[c][k] + sum_j (s_a L)[token][j] Lb_a(c, j)
// over the sorted positions; Lb_a(c, j): row c of lt + Ncols * row8_a
// [Ncols, r8]; of B_a itself where lt_all is 0 and r_a % 8 == 0.
struct GemmSide {
  const uint16_t* terms;   // of s_a L
  AdapterView v;
  const uint16_t* lt;
  DropView drop;           // lt_all: element m Ncols + c of this side's part is left out
};
// GEMM_ONE: side 0. GEMM_TWO (lt_all): the parts of both sides. GEMM_GATED (not
// lt_all): two products of the same A, side 0 with Bt (g), side 1 with Bt2 (u);
// out = act(g) u, and g and u themselves in bf16 where wanted.
enum GemmMode { GEMM_ONE, GEMM_TWO, GEMM_GATED };
struct AdapterGemm {
  const uint16_t* A;       // [M, lda]
  int64_t M, Ncols, Kc;
  int64_t lda;
  const uint16_t* Bt;      // [Ncols, ldb], ldb % 64 == 0, zero from Kc to ldb
  int64_t ldb;
  GemmSide s[2];
  int lt_all;
  Route rt;
  void* out;               // [M, Ncols] bf16 or float32
  int out_f32;
  const uint16_t* zeros;   // 16 zero bytes
  int mode;
  const uint16_t* Bt2;
  int act;
  uint16_t *g_out, *u_out; // [M, Ncols] or null
};
hipError_t launch_adapter_gemm(const AdapterGemm& g, hipStream_t s);
// [N, K] -> [K, N rounded up to a multiple of 64] bf16 of row stride ldb (zero columns past N)
// (two of a size where w2 is given)
hipError_t launch_transpose_weight(const uint16_t* w, int64_t N, int64_t K, int64_t ldb, uint16_t* out, const uint16_t* w2,
                                   uint16_t* out2, hipStream_t s);

// Decode sizes (NF4, M <= 64): the whole forward without a route, in two
// launches.
bool adapter_decode_supported(const QWeight& w, int64_t M);
size_t adapter_decode_ws_bytes(const QWeight& w, int64_t M, const AdapterView& v);
hipError_t launch_adapter_decode(const QWeight& w, const uint16_t* X, int64_t M, const int32_t* ids,
                                 const AdapterView& v, void* ws, float* t_save, void* H, bool f32, hipStream_t s);

// ---- the gated pair ----------------------------------------------------------
// dg = G u act'(g), du = G act(g) of M tokens, formed from G, g, u [M, N] bf16.
struct GatedGrad {
  const uint16_t *G, *g, *u;
  int64_t N;               // N % 8 == 0
  int act;
};
// u_g = B_g^T dg and u_u = B_u^T du as partial sums [shares][M][rs] of each side
// (bt: B^T [r, N] at N * row8_a; v.n == 0: of neither), and dg, du in bfloat16 as
// D [M, 2 Np], Np = N rounded up to a multiple of 64, zero between (null: not wanted).
size_t gated_down_ws_floats(int64_t M, int64_t N, const AdapterView& v);
int gated_down_shares(int64_t M, int64_t N, int32_t n);
hipError_t launch_gated_down(const GatedGrad& gr, int64_t M, const AdapterView (&v)[2], const uint16_t* const (&bt)[2],
                             float* const (&part)[2], uint16_t* D, const Route& rt, hipStream_t s);
// dB of both sides: requests as launch_adapter_col's (transposed), Q in place of
// side 0's dg, side 1's du; a null out: not wanted (one is). The join is the caller's.
hipError_t launch_gated_col(const GatedGrad& gr, const ColReq (&req)[2], int64_t M, const Route& rt, ColJoin* join, hipStream_t s);

// Decode sizes of a pair: the whole forward, in two launches.
bool gated_decode_supported(const QWeight (&w)[2], int64_t M, const AdapterView (&v)[2]);
size_t gated_decode_ws_bytes(const QWeight& w, int64_t M, const AdapterView (&v)[2]);
hipError_t launch_gated_decode(const QWeight (&w)[2], const uint16_t* X, int64_t M, const int32_t* ids,
                               const AdapterView (&v)[2], void* ws, int act, float* t_gate, float* t_up, uint16_t* g,
                               uint16_t* u, void* H, bool f32, hipStream_t s);

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
