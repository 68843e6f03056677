// The C ABI of include/lq_adapters.h: argument validation, workspace carving
// and kernel dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "lq_adapters.h"
#include "lq_host.h"

namespace {

using namespace lq;

int check_set(const lq_adapter_set* set, int64_t N, int64_t K, AdapterView* v) {
  if (!set || !set->host || !set->dev || !al(set->dev, 8)) return LQ_ERR_ARG;
  if (set->n < 1 || set->n > LQ_ADAPTERS_MAX || N <= 0 || K <= 0) return LQ_ERR_SHAPE;
  int32_t row = 0, row8 = 0, r_max = 0;
  for (int32_t a = 0; a < set->n; ++a) {
    const lq_adapter& ad = set->host[a];
    if (ad.r < 1 || ad.r > 128) return LQ_ERR_SHAPE;
    if (!ad.A || !ad.B || !al(ad.A, kVec) || !al(ad.B, kVec)) return LQ_ERR_ARG;
    if (ad.row != row || ad.row8 != row8) return LQ_ERR_ARG;
    row += ad.r;
    row8 += (ad.r + 7) / 8 * 8;
    r_max = std::max(r_max, ad.r);
  }
  if (set->r_max != r_max) return LQ_ERR_ARG;
  *v = AdapterView{set->dev, set->n, r_max, (r_max + 7) / 8 * 8};
  return LQ_OK;
}

int64_t sum_r8(const lq_adapter_set* set) {
  const lq_adapter& last = set->host[set->n - 1];
  return (int64_t)last.row8 + (last.r + 7) / 8 * 8;
}

bool valid_M(int64_t M) { return M >= 1 && M < (int64_t(1) << 31); }

size_t route_bytes(int64_t M, int32_t n) { return (size_t)route_words(M, n) * sizeof(int32_t); }

int64_t ldb_of(int64_t n) { return (n + 63) / 64 * 64; }

bool any_odd_rank(const lq_adapter_set* set) {
  for (int32_t a = 0; a < set->n; ++a)
    if (set->host[a].r % 8) return true;
  return false;
}

size_t bytes16(size_t elems) { return align_up(elems * sizeof(uint16_t)); }

// route, terms of t, W', zeros, B of ranks that are no multiple of 8; at
// decode sizes what that path keeps
size_t forward_ws(const QWeight& q, int64_t M, const AdapterView& v, const lq_adapter_set* set) {
  if (adapter_decode_supported(q, M)) return align_up(adapter_decode_ws_bytes(q, M, v));
  return align_up(route_bytes(M, v.n)) + bytes16(terms_elems(M, v)) + bytes16((size_t)q.N * q.K) + bytes16(8) +
         align_up(adapter_down_ws_floats(M, q.K, v.rs) * sizeof(float)) +
         (any_odd_rank(set) ? bytes16((size_t)sum_r8(set) * q.N) : 0);
}

// route, terms of u and t, A^T and B^T of the adapters, W'^T (and W' of a
// codebook weight, which is transposed from it), partial sums of dA and dB, zeros
size_t backward_ws(const QWeight& q, int64_t M, const AdapterView& v, int64_t r8) {
  return align_up(route_bytes(M, v.n)) + 2 * bytes16(terms_elems(M, v)) + bytes16((size_t)r8 * q.K) +
         bytes16((size_t)r8 * q.N) + (q.format == LQ_FMT_NF4 ? 0 : bytes16((size_t)q.N * q.K)) +
         bytes16((size_t)q.K * ldb_of(q.N)) +
         align_up(adapter_col_ws_floats(M, q.K, v.rs) * sizeof(float)) +
         align_up(adapter_col_ws_floats(M, q.N, v.rs) * sizeof(float)) + bytes16(8) +
         align_up(adapter_down_ws_floats(M, q.K, v.rs) * sizeof(float)) +
         align_up(adapter_down_ws_floats(M, q.N, v.rs) * sizeof(float));
}

}  // namespace

extern "C" {

int lq_check_adapters(const lq_adapter_set* set, int64_t N, int64_t K) {
  AdapterView v;
  return check_set(set, N, K, &v);
}

size_t lq_adapter_route_bytes(int64_t M, int32_t n) {
  if (!valid_M(M) || n < 1 || n > LQ_ADAPTERS_MAX) return 0;
  return route_bytes(M, n);
}

int lq_adapter_route(const int32_t* ids, int64_t M, int32_t n, int32_t* route, size_t bytes, void* stream) {
  if (!ids || !route || !al(ids, 4) || !al(route, kVec)) return LQ_ERR_ARG;
  if (!valid_M(M) || n < 1 || n > LQ_ADAPTERS_MAX) return LQ_ERR_SHAPE;
  if (bytes < route_bytes(M, n)) return LQ_ERR_WORKSPACE;
  QWeight none{};
  const AdapterView v{nullptr, n, 0, 0};
  return launch_status(launch_adapter_prep(ids, M, route, none, nullptr, 0, v, nullptr, nullptr, nullptr,
                                           nullptr, (hipStream_t)stream));
}

size_t lq_adapters_forward_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set) {
  QWeight q;
  AdapterView v;
  if (check_qweight(w, &q) != LQ_OK || !valid_M(M) || check_set(set, q.N, q.K, &v) != LQ_OK) return 0;
  return forward_ws(q, M, v, set);
}

int lq_adapters_forward(const lq_qweight* w, const uint16_t* X, int64_t M, const lq_adapter_set* set,
                        const int32_t* ids, const int32_t* route, void* H, int32_t h_dtype, float* t_save,
                        void* workspace, size_t ws_bytes, void* stream) {
  QWeight q;
  AdapterView v;
  int st = check_qweight(w, &q);
  if (st != LQ_OK) return st;
  if ((st = check_set(set, q.N, q.K, &v)) != LQ_OK) return st;
  if (!X || !ids || !H) return LQ_ERR_ARG;
  if (!al(X, kVec) || !al(ids, 4) || !al(route, kVec) || !al(H, h_dtype == LQ_F32 ? 4 : kVec) || !al(t_save, 4) ||
      !al(workspace, kVec))
    return LQ_ERR_ARG;
  if (!valid_M(M)) return LQ_ERR_SHAPE;
  if (h_dtype != LQ_BF16 && h_dtype != LQ_F32) return LQ_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < forward_ws(q, M, v, set)) return LQ_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  if ((st = debug_check_weight(q, s)) != LQ_OK) return st;
  Carver cv(workspace, ws_bytes);
  if (adapter_decode_supported(q, M))
    return launch_status(launch_adapter_decode(q, X, M, ids, v, workspace, t_save, H, h_dtype == LQ_F32, s));
  int32_t* rws = cv.take<int32_t>(route_words(M, v.n));
  uint16_t* terms = cv.take<uint16_t>(terms_elems(M, v));
  uint16_t* wd = cv.take<uint16_t>((size_t)q.N * q.K);
  uint16_t* zeros = cv.take<uint16_t>(8);
  float* part = cv.take<float>(adapter_down_ws_floats(M, q.K, v.rs));
  uint16_t* bp = any_odd_rank(set) ? cv.take<uint16_t>((size_t)sum_r8(set) * q.N) : nullptr;
  if (!cv.ok()) return LQ_ERR_WORKSPACE;

  hipError_t e = launch_adapter_prep(ids, M, route ? nullptr : rws, q, wd, 0, v, nullptr, nullptr, bp, zeros, s);
  if (e != hipSuccess) return LQ_ERR_LAUNCH;
  const Route rt = route_view(route ? route : rws, M, v.n);
  const DownJob job{X, q.K, nullptr, nullptr, terms, t_save, part};
  if ((e = launch_adapter_down(&job, 1, M, v, rt, zeros, s)) != hipSuccess) return LQ_ERR_LAUNCH;
  const AdapterGemm g{X, M, q.N, q.K, wd, q.K, terms, v, bp, 0, rt, H, h_dtype == LQ_F32 ? 1 : 0, zeros};
  return launch_status(launch_adapter_gemm(g, s));
}

size_t lq_adapters_backward_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set) {
  QWeight q;
  AdapterView v;
  if (check_qweight(w, &q) != LQ_OK || !valid_M(M) || check_set(set, q.N, q.K, &v) != LQ_OK || q.N % 8 != 0) return 0;
  return backward_ws(q, M, v, sum_r8(set));
}

int lq_adapters_backward(const lq_qweight* w, const uint16_t* X, const uint16_t* G, int64_t M,
                         const lq_adapter_set* set, const int32_t* ids, const int32_t* route, const float* t_saved,
                         uint16_t* grad_X, float* dA, float* dB, void* workspace, size_t ws_bytes, void* stream) {
  QWeight q;
  AdapterView v;
  int st = check_qweight(w, &q);
  if (st != LQ_OK) return st;
  if ((st = check_set(set, q.N, q.K, &v)) != LQ_OK) return st;
  const bool need_t = dB && !t_saved;
  if (!G || !ids || ((dA || need_t) && !X)) return LQ_ERR_ARG;
  if (!al(X, kVec) || !al(G, kVec) || !al(ids, 4) || !al(route, kVec) || !al(t_saved, 4) || !al(grad_X, kVec) ||
      !al(dA, 4) || !al(dB, 4) || !al(workspace, kVec))
    return LQ_ERR_ARG;
  if (!valid_M(M) || q.N % 8 != 0) return LQ_ERR_SHAPE;
  const int64_t r8 = sum_r8(set);
  if (!workspace || ws_bytes < backward_ws(q, M, v, r8)) return LQ_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  if ((st = debug_check_weight(q, s)) != LQ_OK) return st;
  Carver cv(workspace, ws_bytes);
  int32_t* rws = cv.take<int32_t>(route_words(M, v.n));
  uint16_t* u = cv.take<uint16_t>(terms_elems(M, v));
  uint16_t* t = cv.take<uint16_t>(terms_elems(M, v));
  uint16_t* at = cv.take<uint16_t>((size_t)r8 * q.K);
  uint16_t* bt = cv.take<uint16_t>((size_t)r8 * q.N);
  uint16_t* wd = q.format == LQ_FMT_NF4 ? nullptr : cv.take<uint16_t>((size_t)q.N * q.K);
  const int64_t ldb = ldb_of(q.N);
  uint16_t* wt = cv.take<uint16_t>((size_t)q.K * ldb);
  float* part_a = cv.take<float>(adapter_col_ws_floats(M, q.K, v.rs));
  float* part_b = cv.take<float>(adapter_col_ws_floats(M, q.N, v.rs));
  uint16_t* zeros = cv.take<uint16_t>(8);
  float* down_t = cv.take<float>(adapter_down_ws_floats(M, q.K, v.rs));
  float* down_u = cv.take<float>(adapter_down_ws_floats(M, q.N, v.rs));
  if (!cv.ok()) return LQ_ERR_WORKSPACE;
  if (!grad_X && !dA && !dB) return LQ_OK;

  const bool need_u = grad_X || dA, nf4 = q.format == LQ_FMT_NF4;
  hipError_t e = launch_adapter_prep(ids, M, route ? nullptr : rws, q, !grad_X ? nullptr : nf4 ? wt : wd, nf4 ? ldb : 0,
                                     v, grad_X ? at : nullptr, need_u ? bt : nullptr, nullptr, zeros, s);
  if (e != hipSuccess) return LQ_ERR_LAUNCH;
  const Route rt = route_view(route ? route : rws, M, v.n);
  DownJob jobs[2];
  int nj = 0;
  if (need_u) jobs[nj++] = DownJob{G, q.N, bt, nullptr, u, nullptr, down_u};
  if (dB) jobs[nj++] = DownJob{t_saved ? nullptr : X, q.K, nullptr, t_saved, t, nullptr, down_t};
  if (nj && (e = launch_adapter_down(jobs, nj, M, v, rt, zeros, s)) != hipSuccess) return LQ_ERR_LAUNCH;
  ColReq cols[2];
  int nc = 0;
  if (dB) cols[nc++] = ColReq{t, G, q.N, dB, 1, part_b};
  if (dA) cols[nc++] = ColReq{u, X, q.K, dA, 0, part_a};
  if (nc && (e = launch_adapter_col(cols, nc, M, v, rt, s)) != hipSuccess) return LQ_ERR_LAUNCH;
  if (!grad_X) return LQ_OK;
  if (!nf4 && (e = launch_transpose_weight(wd, q.N, q.K, ldb, wt, s)) != hipSuccess) return LQ_ERR_LAUNCH;
  const AdapterGemm g{G, M, q.K, q.N, wt, ldb, u, v, at, 1, rt, grad_X, 0, zeros};
  return launch_status(launch_adapter_gemm(g, s));
}

}  // extern "C"

// ---- gradient lists ------------------------------------------------------------
namespace {

// A piece is one wave's share of a tensor; slots hold whole pieces of one
// group. 2048 slots (8 workgroups of 4 waves per CU) fill the chip.
constexpr int64_t kPieceElems = 4096;
constexpr int64_t kSlotTarget = 2048;
constexpr int64_t kMaxPieces = int64_t(1) << 30;

int64_t pieces_of(int64_t numel) { return (numel + kPieceElems - 1) / kPieceElems; }

size_t elem_size(int32_t dtype) { return dtype == LQ_F32 ? 4 : 2; }

int check_tensors(const lq_grad_tensor* t, int64_t n, int32_t n_groups, int64_t* pieces) {
  if (n < 0 || n_groups < 1 || n_groups > 65535) return LQ_ERR_SHAPE;
  if (n > 0 && !t) return LQ_ERR_ARG;
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].dtype != LQ_F32 && t[i].dtype != LQ_BF16 && t[i].dtype != LQ_F16) return LQ_ERR_ARG;
    if (t[i].group < 0 || t[i].group >= n_groups) return LQ_ERR_ARG;
    if (t[i].numel < 0) return LQ_ERR_SHAPE;
    if (t[i].numel > 0 && (!t[i].data || !al(t[i].data, elem_size(t[i].dtype)))) return LQ_ERR_ARG;
    if (t[i].numel > kMaxPieces * kPieceElems) return LQ_ERR_SHAPE;
    total += pieces_of(t[i].numel);
    if (total > kMaxPieces) return LQ_ERR_SHAPE;
  }
  *pieces = total;
  return LQ_OK;
}

int64_t pieces_per_slot(int64_t pieces) {
  return std::max<int64_t>(kGradThreads / 64, (pieces + kSlotTarget - 1) / kSlotTarget);
}

size_t list_bytes(int64_t pieces, int32_t n_groups) {
  const int64_t slots = (pieces + pieces_per_slot(pieces) - 1) / pieces_per_slot(pieces) + n_groups;
  return align_up((size_t)slots * sizeof(GradSlot)) + align_up((size_t)pieces * sizeof(GradPiece));
}

int check_list(const lq_grad_list* l) {
  if (!l || !l->dev || !al(l->dev, kVec)) return LQ_ERR_ARG;
  if (l->n_slots < 1 || l->n_groups < 1 || l->n_groups > l->n_slots || l->n_pieces < 0) return LQ_ERR_ARG;
  return LQ_OK;
}

const GradSlot* slots_of(const lq_grad_list* l) { return reinterpret_cast<const GradSlot*>(l->dev); }
const GradPiece* pieces_at(const lq_grad_list* l) {
  return reinterpret_cast<const GradPiece*>((const char*)l->dev + align_up((size_t)l->n_slots * sizeof(GradSlot)));
}

}  // namespace

extern "C" {

size_t lq_grad_list_bytes(const lq_grad_tensor* tensors, int64_t n, int32_t n_groups) {
  int64_t pieces = 0;
  if (check_tensors(tensors, n, n_groups, &pieces) != LQ_OK) return 0;
  return list_bytes(pieces, n_groups);
}

int lq_grad_list_build(const lq_grad_tensor* tensors, int64_t n, int32_t n_groups, void* table, size_t bytes,
                       lq_grad_list* list) {
  int64_t pieces = 0;
  const int st = check_tensors(tensors, n, n_groups, &pieces);
  if (st != LQ_OK) return st;
  if (!table || !list || !al(table, 8)) return LQ_ERR_ARG;
  if (bytes < list_bytes(pieces, n_groups)) return LQ_ERR_WORKSPACE;
  try {
    // tensors in the order of their groups (stable), pieces per group
    std::vector<int64_t> order((size_t)n), first((size_t)n_groups + 1, 0), gp((size_t)n_groups, 0);
    for (int64_t i = 0; i < n; ++i) {
      first[(size_t)tensors[i].group + 1] += 1;
      gp[(size_t)tensors[i].group] += pieces_of(tensors[i].numel);
    }
    for (int32_t g = 0; g < n_groups; ++g) first[(size_t)g + 1] += first[(size_t)g];
    std::vector<int64_t> at(first.begin(), first.end() - 1);
    for (int64_t i = 0; i < n; ++i) order[(size_t)at[(size_t)tensors[i].group]++] = i;

    const int64_t per = pieces_per_slot(pieces);
    GradSlot* slots = reinterpret_cast<GradSlot*>(table);
    int64_t ns = 0, np = 0;
    for (int32_t g = 0; g < n_groups; ++g) {
      const int64_t count = std::max<int64_t>(1, (gp[(size_t)g] + per - 1) / per);
      for (int64_t k = 0; k < count; ++k) {
        GradSlot sl{};
        sl.first = (int32_t)(np + k * per);
        sl.count = (int32_t)std::max<int64_t>(0, std::min(per, gp[(size_t)g] - k * per));
        sl.group = g;
        sl.group_first = (int32_t)ns;
        sl.group_count = (int32_t)count;
        std::memcpy(&slots[ns + k], &sl, sizeof(sl));
      }
      ns += count;
      np += gp[(size_t)g];
    }
    GradPiece* out = reinterpret_cast<GradPiece*>((char*)table + align_up((size_t)ns * sizeof(GradSlot)));
    np = 0;
    for (int64_t i : order) {
      const lq_grad_tensor& t = tensors[i];
      for (int64_t e = 0; e < t.numel; e += kPieceElems) {
        const GradPiece pc{(char*)t.data + (size_t)e * elem_size(t.dtype),
                           (int32_t)std::min(kPieceElems, t.numel - e), t.dtype};
        std::memcpy(&out[np++], &pc, sizeof(pc));
      }
    }
    uint64_t h = 1469598103934665603ull;   // FNV-1a over sizes, types and groups
    auto mix = [&h](uint64_t v) {
      for (int b = 0; b < 8; ++b) h = (h ^ ((v >> (8 * b)) & 0xFF)) * 1099511628211ull;
    };
    mix((uint64_t)n_groups);
    for (int64_t i = 0; i < n; ++i) {
      mix((uint64_t)tensors[i].numel);
      mix(((uint64_t)(uint32_t)tensors[i].dtype << 32) | (uint32_t)tensors[i].group);
    }
    *list = lq_grad_list{nullptr, pieces, (int32_t)ns, n_groups, h};
  } catch (...) {
    return LQ_ERR_WORKSPACE;   // out of host memory
  }
  return LQ_OK;
}

size_t lq_grad_norm_workspace(const lq_grad_list* list) {
  if (!list || list->n_slots < 1) return 0;
  return align_up((size_t)list->n_slots * sizeof(double));
}

int lq_grad_norm(const lq_grad_list* list, float* norms, void* workspace, size_t ws_bytes, void* stream) {
  const int st = check_list(list);
  if (st != LQ_OK) return st;
  if (!norms || !al(norms, 4) || !al(workspace, kVec)) return LQ_ERR_ARG;
  if (!workspace || ws_bytes < lq_grad_norm_workspace(list)) return LQ_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  double* part = (double*)workspace;
  hipError_t e = launch_grad_squares(slots_of(list), pieces_at(list), list->n_slots, part, s);
  if (e != hipSuccess) return LQ_ERR_LAUNCH;
  return launch_status(launch_grad_norms(slots_of(list), list->n_slots, part, norms, s));
}

int lq_clip_grad_norm(const lq_grad_list* in, const lq_grad_list* out, float max_norm, float eps, float* norms,
                      void* workspace, size_t ws_bytes, void* stream) {
  int st = check_list(in);
  if (st != LQ_OK || (st = check_list(out)) != LQ_OK) return st;
  if (in->digest != out->digest || in->n_slots != out->n_slots || in->n_pieces != out->n_pieces) return LQ_ERR_ARG;
  if (!std::isfinite(max_norm) || max_norm < 0.0f || !std::isfinite(eps) || !(eps > 0.0f)) return LQ_ERR_ARG;
  if (!norms || !al(norms, 4) || !al(workspace, kVec)) return LQ_ERR_ARG;
  if (!workspace || ws_bytes < lq_grad_norm_workspace(in)) return LQ_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  double* part = (double*)workspace;
  hipError_t e = launch_grad_squares(slots_of(in), pieces_at(in), in->n_slots, part, s);
  if (e != hipSuccess) return LQ_ERR_LAUNCH;
  return launch_status(launch_grad_clip(slots_of(in), pieces_at(in), pieces_at(out), in->n_slots, part, max_norm, eps,
                                        norms, s));
}

}  // extern "C"
