// The C ABI of include/lq_gated.h: argument validation, workspace carving and
// kernel dispatch.
#include <algorithm>

#include "../../include/lq_gated.h"
#include "lq_adapters.h"
#include "lq_adapters_host.h"

namespace {

using namespace lq;

struct Pair {
  QWeight q[2];
  AdapterView v[2];
  const lq_adapter_set* set[2];
  bool sets;
  int64_t N, K;
  int act;
};

int check_pair(const lq_gated* p, Pair* o) {
  if (!p || p->act < LQ_SILU || p->act > LQ_GELU_TANH || (p->gate_set == nullptr) != (p->up_set == nullptr)) return LQ_ERR_ARG;
  int st = check_qweight(p->gate, &o->q[0]);
  if (st != LQ_OK || (st = check_qweight(p->up, &o->q[1])) != LQ_OK) return st;
  o->N = o->q[0].N;
  o->K = o->q[0].K;
  if (o->q[1].N != o->N || o->q[1].K != o->K) return LQ_ERR_SHAPE;
  o->act = p->act;
  o->set[0] = p->gate_set;
  o->set[1] = p->up_set;
  o->sets = p->gate_set != nullptr;
  o->v[0] = o->v[1] = AdapterView{nullptr, 0, 0, 0};
  if (!o->sets) return LQ_OK;
  for (int i = 0; i < 2; ++i)
    if ((st = check_set(o->set[i], o->N, o->K, &o->v[i])) != LQ_OK) return st;
  return o->v[0].n == o->v[1].n ? LQ_OK : LQ_ERR_SHAPE;
}

// Both dropouts, of which either may be missing. A side without one keeps
// everything (T = 0); the kernels that drop at all read its key all the same.
int check_drops(const Pair& p, int64_t M, const lq_dropout* d0, const lq_dropout* d1, DropView (&drop)[2], float (&factor)[2]) {
  if (!p.sets && (d0 || d1)) return LQ_ERR_ARG;
  int st = drop_view(d0, &drop[0], &factor[0]);
  if (st != LQ_OK || (st = drop_view(d1, &drop[1], &factor[1])) != LQ_OK) return st;
  for (int i = 0; i < 2; ++i)
    if (!drop[i].key) drop[i].key = drop[1 - i].key;
  return (d0 || d1) && !drop_fits(M, p.K) ? LQ_ERR_SHAPE : LQ_OK;
}

// The pieces of a workspace; with a null base only their size counts.
struct Forward {
  int32_t* route;
  uint16_t *terms[2], *wd[2], *bp[2], *zeros;
  float* part[2];
  explicit Forward(Carver& cv, const Pair& p, int64_t M, bool drops) {
    route = cv.take<int32_t>(route_words(M, p.v[0].n));
    for (int i = 0; i < 2; ++i) {
      terms[i] = cv.take<uint16_t>(terms_elems(M, p.v[i]));
      wd[i] = cv.take<uint16_t>((size_t)p.N * p.K);
      part[i] = cv.take<float>(p.sets ? adapter_down_ws_floats(M, p.K, p.v[i].rs, drops) : 0);
      bp[i] = p.sets && any_odd_rank(p.set[i]) ? cv.take<uint16_t>((size_t)sum_r8(p.set[i]) * p.N) : nullptr;
    }
    zeros = cv.take<uint16_t>(8);
  }
};

struct Backward {
  int32_t* route;
  uint16_t *u[2], *t[2], *at[2], *bt[2], *wd[2], *wt, *D, *zeros;
  float *down_t[2], *down_u[2], *part_a[2], *part_b[2];
  explicit Backward(Carver& cv, const Pair& p, int64_t M, bool drops) {
    route = cv.take<int32_t>(route_words(M, p.v[0].n));
    for (int i = 0; i < 2; ++i) {
      const AdapterView& v = p.v[i];
      const size_t r8 = p.sets ? (size_t)sum_r8(p.set[i]) : 0;
      u[i] = cv.take<uint16_t>(terms_elems(M, v));
      t[i] = cv.take<uint16_t>(terms_elems(M, v));
      at[i] = cv.take<uint16_t>(r8 * p.K);
      bt[i] = cv.take<uint16_t>(r8 * p.N);
      wd[i] = p.q[i].format == LQ_FMT_NF4 ? nullptr : cv.take<uint16_t>((size_t)p.N * p.K);
      down_t[i] = cv.take<float>(p.sets ? adapter_down_ws_floats(M, p.K, v.rs, drops) : 0);
      down_u[i] = cv.take<float>(gated_down_ws_floats(M, p.N, v));
      part_a[i] = cv.take<float>(adapter_col_ws_floats(M, p.K, v.rs));
      part_b[i] = cv.take<float>(adapter_col_ws_floats(M, p.N, v.rs));
    }
    wt = cv.take<uint16_t>((size_t)p.K * 2 * ldb_of(p.N));
    D = cv.take<uint16_t>((size_t)M * 2 * ldb_of(p.N));
    zeros = cv.take<uint16_t>(8);
  }
};

// Whether the forward runs as at decode sizes.
bool decodes(const Pair& p, int64_t M, bool drops) { return !drops && gated_decode_supported(p.q, M, p.v); }

template <class W>
size_t ws_bytes_of(const Pair& p, int64_t M, bool drops) {
  Carver cv(nullptr, 0);
  W w(cv, p, M, drops);
  (void)w;
  return cv.used;
}

size_t forward_ws(const Pair& p, int64_t M, bool drops) {
  return decodes(p, M, drops) ? align_up(gated_decode_ws_bytes(p.q[0], M, p.v)) : ws_bytes_of<Forward>(p, M, drops);
}

}  // namespace

extern "C" {

int lq_check_gated(const lq_gated* p) {
  Pair o;
  return check_pair(p, &o);
}

size_t lq_gated_forward_workspace(const lq_gated* p, int64_t M, int32_t drops) {
  Pair o;
  if (check_pair(p, &o) != LQ_OK || !valid_M(M) || (drops && !drop_fits(M, o.K))) return 0;
  return forward_ws(o, M, drops);
}

int lq_gated_forward(const lq_gated* p, const uint16_t* X, int64_t M, const int32_t* ids, const int32_t* route,
                     const lq_dropout* drop_gate, const lq_dropout* drop_up, void* H, int32_t h_dtype, uint16_t* g,
                     uint16_t* u, float* t_gate, float* t_up, void* workspace, size_t ws_bytes, void* stream) {
  Pair o;
  DropView drop[2];
  float factor[2];
  int st = check_pair(p, &o);
  if (st != LQ_OK) return st;
  if (!X || !H || (ids == nullptr) != !o.sets || (!o.sets && (route || t_gate || t_up))) return LQ_ERR_ARG;
  if (!al(X, kVec) || !al(ids, 4) || !al(route, kVec) || !al(H, h_dtype == LQ_F32 ? 4 : kVec) || !al(g, kVec) ||
      !al(u, kVec) || !al(t_gate, 4) || !al(t_up, 4) || !al(workspace, kVec))
    return LQ_ERR_ARG;
  if (!valid_M(M)) return LQ_ERR_SHAPE;
  if ((st = check_drops(o, M, drop_gate, drop_up, drop, factor)) != LQ_OK) return st;
  if (h_dtype != LQ_BF16 && h_dtype != LQ_F32) return LQ_ERR_UNSUPPORTED;
  const bool drops = drop_gate || drop_up;
  if (!workspace || ws_bytes < forward_ws(o, M, drops)) return LQ_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  for (int i = 0; i < 2; ++i)
    if ((st = debug_check_weight(o.q[i], s)) != LQ_OK) return st;
  if (decodes(o, M, drops))
    return launch_status(launch_gated_decode(o.q, X, M, ids, o.v, workspace, o.act, t_gate, t_up, g, u, H, h_dtype == LQ_F32, s));
  Carver cv(workspace, ws_bytes);
  const Forward w(cv, o, M, drops);
  if (!cv.ok()) return LQ_ERR_WORKSPACE;

  Prep prep[2];
  for (int i = 0; i < 2; ++i)
    prep[i] = Prep{i == 0 && !route ? w.route : nullptr, o.q[i], w.wd[i], 0, o.v[i], nullptr, nullptr, w.bp[i],
                   i == 0 ? w.zeros : nullptr};
  if (launch_adapter_prep(ids, M, prep, 2, s) != hipSuccess) return LQ_ERR_LAUNCH;
  const Route rt = route_view(route ? route : w.route, M, o.v[0].n);
  if (o.sets) {
    float* const save[2] = {t_gate, t_up};
    DownJob jobs[2];
    for (int i = 0; i < 2; ++i)
      jobs[i] = DownJob{X, o.K, nullptr, nullptr, w.terms[i], save[i], w.part[i], drop[i], factor[i], o.v[i], 1};
    if (launch_adapter_down(jobs, 2, M, rt, w.zeros, s) != hipSuccess) return LQ_ERR_LAUNCH;
  }
  AdapterGemm gm{};
  gm.A = X;
  gm.M = M;
  gm.Ncols = o.N;
  gm.Kc = gm.lda = gm.ldb = o.K;
  gm.Bt = w.wd[0];
  gm.Bt2 = w.wd[1];
  for (int i = 0; i < 2; ++i) gm.s[i] = GemmSide{w.terms[i], o.v[i], w.bp[i], DropView{}};
  gm.rt = rt;
  gm.out = H;
  gm.out_f32 = h_dtype == LQ_F32;
  gm.zeros = w.zeros;
  gm.mode = GEMM_GATED;
  gm.act = o.act;
  gm.g_out = g;
  gm.u_out = u;
  return launch_status(launch_adapter_gemm(gm, s));
}

size_t lq_gated_backward_workspace(const lq_gated* p, int64_t M) {
  Pair o;
  if (check_pair(p, &o) != LQ_OK || !valid_M(M) || o.N % 8 != 0) return 0;
  return ws_bytes_of<Backward>(o, M, true);   // one size, with dropout or without
}

int lq_gated_backward(const lq_gated* p, const uint16_t* X, const uint16_t* G, int64_t M, const int32_t* ids,
                      const int32_t* route, const lq_dropout* drop_gate, const lq_dropout* drop_up, const uint16_t* g,
                      const uint16_t* u, const float* t_gate, const float* t_up, uint16_t* grad_X, float* dA_gate,
                      float* dB_gate, float* dA_up, float* dB_up, void* workspace, size_t ws_bytes, void* stream) {
  Pair o;
  DropView drop[2];
  float factor[2];
  int st = check_pair(p, &o);
  if (st != LQ_OK) return st;
  float *const dA[2] = {dA_gate, dA_up}, *const dB[2] = {dB_gate, dB_up};
  const float* const t_saved[2] = {t_gate, t_up};
  const bool any_dA = dA_gate || dA_up, any_dB = dB_gate || dB_up;
  const bool need_x = any_dA || (dB_gate && !t_gate) || (dB_up && !t_up);
  if (!G || !g || !u || (need_x && !X) || (ids == nullptr) != !o.sets) return LQ_ERR_ARG;
  if (!o.sets && (route || t_gate || t_up || any_dA || any_dB)) return LQ_ERR_ARG;
  if (!al(X, kVec) || !al(G, kVec) || !al(ids, 4) || !al(route, kVec) || !al(g, kVec) || !al(u, kVec) || !al(t_gate, 4) ||
      !al(t_up, 4) || !al(grad_X, kVec) || !al(dA_gate, 4) || !al(dB_gate, 4) || !al(dA_up, 4) || !al(dB_up, 4) ||
      !al(workspace, kVec))
    return LQ_ERR_ARG;
  if (!valid_M(M) || o.N % 8 != 0) return LQ_ERR_SHAPE;
  if ((st = check_drops(o, M, drop_gate, drop_up, drop, factor)) != LQ_OK) return st;
  if (!workspace || ws_bytes < ws_bytes_of<Backward>(o, M, true)) return LQ_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  for (int i = 0; i < 2; ++i)
    if ((st = debug_check_weight(o.q[i], s)) != LQ_OK) return st;
  Carver cv(workspace, ws_bytes);
  const Backward w(cv, o, M, true);
  if (!cv.ok()) return LQ_ERR_WORKSPACE;
  if (!grad_X && !any_dA && !any_dB) return LQ_OK;

  const int64_t Np = ldb_of(o.N), ldb = 2 * Np;
  const bool need_u = o.sets && (grad_X || any_dA);
  Prep prep[2];
  uint16_t* const wt[2] = {w.wt, w.wt + Np};
  const bool nf4[2] = {o.q[0].format == LQ_FMT_NF4, o.q[1].format == LQ_FMT_NF4};
  for (int i = 0; i < 2; ++i)
    prep[i] = Prep{i == 0 && !route ? w.route : nullptr, o.q[i], !grad_X ? nullptr : nf4[i] ? wt[i] : w.wd[i], nf4[i] ? ldb : 0,
                   o.v[i], o.sets && grad_X ? w.at[i] : nullptr, need_u ? w.bt[i] : nullptr, nullptr,
                   i == 0 ? w.zeros : nullptr};
  if (launch_adapter_prep(ids, M, prep, 2, s) != hipSuccess) return LQ_ERR_LAUNCH;
  if (grad_X && (!nf4[0] || !nf4[1])) {   // codebook weights: transposed from the decoded ones
    const int i = nf4[0] ? 1 : 0;
    const bool both = !nf4[0] && !nf4[1];
    if (launch_transpose_weight(w.wd[i], o.N, o.K, ldb, wt[i], both ? w.wd[1] : nullptr, wt[1], s) != hipSuccess)
      return LQ_ERR_LAUNCH;
  }
  const Route rt = route_view(route ? route : w.route, M, o.v[0].n);
  const GatedGrad gr{G, g, u, o.N, o.act};
  // t formed from X in launches of its own; given t and the partial sums of u become terms in one
  DownJob down[2], join[kDownJobs];
  int ndown = 0, njoin = 0;
  for (int i = 0; i < 2; ++i)
    if (dB[i]) {
      DownJob& job = t_saved[i] ? join[njoin++] : down[ndown++];
      job = DownJob{t_saved[i] ? nullptr : X, o.K, nullptr, t_saved[i], w.t[i], nullptr, w.down_t[i],
                    t_saved[i] ? DropView{} : drop[i], t_saved[i] ? 1.0f : factor[i], o.v[i], 1};
    }
  if (ndown && launch_adapter_down(down, ndown, M, rt, w.zeros, s) != hipSuccess) return LQ_ERR_LAUNCH;
  if (grad_X || need_u) {
    if (launch_gated_down(gr, M, o.v, {w.bt[0], w.bt[1]}, {w.down_u[0], w.down_u[1]}, grad_X ? w.D : nullptr, rt, s) !=
        hipSuccess)
      return LQ_ERR_LAUNCH;
  }
  if (need_u)
    for (int i = 0; i < 2; ++i)
      join[njoin++] = DownJob{G, o.N, nullptr, nullptr, w.u[i], nullptr, w.down_u[i], DropView{}, factor[i], o.v[i],
                              gated_down_shares(M, o.N, o.v[i].n)};
  if (njoin && launch_adapter_join(join, njoin, M, rt, s) != hipSuccess) return LQ_ERR_LAUNCH;
  ColJoin sums[2];
  int nsums = 0;
  if (any_dB) {
    const ColReq req[2] = {ColReq{w.t[0], nullptr, o.N, dB_gate, 1, w.part_b[0], DropView{}, o.v[0]},
                           ColReq{w.t[1], nullptr, o.N, dB_up, 1, w.part_b[1], DropView{}, o.v[1]}};
    if (launch_gated_col(gr, req, M, rt, &sums[nsums++], s) != hipSuccess) return LQ_ERR_LAUNCH;
  }
  if (any_dA) {
    ColReq req[2];
    int n = 0;
    for (int i = 0; i < 2; ++i)
      if (dA[i]) req[n++] = ColReq{w.u[i], X, o.K, dA[i], 0, w.part_a[i], drop[i], o.v[i]};
    if (launch_adapter_col(req, n, M, rt, &sums[nsums++], s) != hipSuccess) return LQ_ERR_LAUNCH;
  }
  if (nsums && launch_adapter_col_reduce(sums, nsums, rt, s) != hipSuccess) return LQ_ERR_LAUNCH;
  if (!grad_X) return LQ_OK;
  AdapterGemm gm{};
  gm.A = w.D;
  gm.M = M;
  gm.Ncols = o.K;
  gm.Kc = gm.lda = gm.ldb = ldb;
  gm.Bt = w.wt;
  for (int i = 0; i < 2; ++i) gm.s[i] = GemmSide{w.u[i], o.v[i], w.at[i], drop[i]};
  gm.lt_all = 1;
  gm.rt = rt;
  gm.out = grad_X;
  gm.zeros = w.zeros;
  gm.mode = GEMM_TWO;
  return launch_status(launch_adapter_gemm(gm, s));
}

}  // extern "C"
