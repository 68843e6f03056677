// The C ABI of include/lq_adapters.h: argument validation, workspace carving
// and kernel dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "lq_adapters.h"
#include "lq_adapters_host.h"

namespace lq {

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

}  // namespace lq

namespace {

using namespace lq;

// route, terms of t, W', zeros, B of ranks that are no multiple of 8; at
// decode sizes what that path keeps
size_t forward_ws(const QWeight& q, int64_t M, const AdapterView& v, const lq_adapter_set* set, bool drops) {
  if (!drops && adapter_decode_supported(q, M)) return align_up(adapter_decode_ws_bytes(q, M, v));
  return align_up(route_bytes(M, v.n)) + bytes16(terms_elems(M, v)) + bytes16((size_t)q.N * q.K) + bytes16(8) +
         align_up(adapter_down_ws_floats(M, q.K, v.rs, drops) * sizeof(float)) +
         (any_odd_rank(set) ? bytes16((size_t)sum_r8(set) * q.N) : 0);
}

// route, terms of u and t, A^T and B^T of the adapters, W'^T (and W' of a
// codebook weight, which is transposed from it), partial sums of dA and dB, zeros
size_t backward_ws(const QWeight& q, int64_t M, const AdapterView& v, int64_t r8, bool drops) {
  return align_up(route_bytes(M, v.n)) + 2 * bytes16(terms_elems(M, v)) + bytes16((size_t)r8 * q.K) +
         bytes16((size_t)r8 * q.N) + (q.format == LQ_FMT_NF4 ? 0 : bytes16((size_t)q.N * q.K)) +
         bytes16((size_t)q.K * ldb_of(q.N)) +
         align_up(adapter_col_ws_floats(M, q.K, v.rs) * sizeof(float)) +
         align_up(adapter_col_ws_floats(M, q.N, v.rs) * sizeof(float)) + bytes16(8) +
         align_up(adapter_down_ws_floats(M, q.K, v.rs, drops) * sizeof(float)) +
         align_up(adapter_down_ws_floats(M, q.N, v.rs, drops) * sizeof(float));
}

// The forward; d null: without dropout. Decode sizes with dropout run as larger ones.
int run_forward(const lq_qweight* w, const uint16_t* X, int64_t M, const lq_adapter_set* set, const int32_t* ids,
                const int32_t* route, const lq_dropout* d, void* H, int32_t h_dtype, float* t_save, void* workspace,
                size_t ws_bytes, void* stream) {
  QWeight q;
  AdapterView v;
  DropView drop;
  float factor;
  int st = check_qweight(w, &q);
  if (st != LQ_OK) return st;
  if ((st = check_set(set, q.N, q.K, &v)) != LQ_OK) return st;
  if ((st = drop_view(d, &drop, &factor)) != LQ_OK) return st;
  if (!X || !ids || !H) return LQ_ERR_ARG;
  if (!al(X, kVec) || !al(ids, 4) || !al(route, kVec) || !al(H, h_dtype == LQ_F32 ? 4 : kVec) || !al(t_save, 4) ||
      !al(workspace, kVec))
    return LQ_ERR_ARG;
  if (!valid_M(M) || (d && !drop_fits(M, q.K))) return LQ_ERR_SHAPE;
  if (h_dtype != LQ_BF16 && h_dtype != LQ_F32) return LQ_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < forward_ws(q, M, v, set, d != nullptr)) return LQ_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  if ((st = debug_check_weight(q, s)) != LQ_OK) return st;
  Carver cv(workspace, ws_bytes);
  if (!d && adapter_decode_supported(q, M))
    return launch_status(launch_adapter_decode(q, X, M, ids, v, workspace, t_save, H, h_dtype == LQ_F32, s));
  int32_t* rws = cv.take<int32_t>(route_words(M, v.n));
  uint16_t* terms = cv.take<uint16_t>(terms_elems(M, v));
  uint16_t* wd = cv.take<uint16_t>((size_t)q.N * q.K);
  uint16_t* zeros = cv.take<uint16_t>(8);
  float* part = cv.take<float>(adapter_down_ws_floats(M, q.K, v.rs, d != nullptr));
  uint16_t* bp = any_odd_rank(set) ? cv.take<uint16_t>((size_t)sum_r8(set) * q.N) : nullptr;
  if (!cv.ok()) return LQ_ERR_WORKSPACE;

  const Prep prep{route ? nullptr : rws, q, wd, 0, v, nullptr, nullptr, bp, zeros};
  hipError_t e = launch_adapter_prep(ids, M, &prep, 1, s);
  if (e != hipSuccess) return LQ_ERR_LAUNCH;
  const Route rt = route_view(route ? route : rws, M, v.n);
  const DownJob job{X, q.K, nullptr, nullptr, terms, t_save, part, drop, factor, v, 1};
  if ((e = launch_adapter_down(&job, 1, M, rt, zeros, s)) != hipSuccess) return LQ_ERR_LAUNCH;
  const AdapterGemm g{X,  M, q.N, q.K, q.K, wd, q.K, {{terms, v, bp, DropView{}}, {}}, 0, rt, H,
                      h_dtype == LQ_F32 ? 1 : 0, zeros, GEMM_ONE, nullptr, 0, nullptr, nullptr};
  return launch_status(launch_adapter_gemm(g, s));
}

int run_backward(const lq_qweight* w, const uint16_t* X, const uint16_t* G, int64_t M, const lq_adapter_set* set,
                 const int32_t* ids, const int32_t* route, const lq_dropout* d, const float* t_saved,
                 uint16_t* grad_X, float* dA, float* dB, void* workspace, size_t ws_bytes, void* stream) {
  QWeight q;
  AdapterView v;
  DropView drop;
  float factor;
  int st = check_qweight(w, &q);
  if (st != LQ_OK) return st;
  if ((st = check_set(set, q.N, q.K, &v)) != LQ_OK) return st;
  if ((st = drop_view(d, &drop, &factor)) != LQ_OK) return st;
  const bool need_t = dB && !t_saved;
  if (!G || !ids || ((dA || need_t) && !X)) return LQ_ERR_ARG;
  if (!al(X, kVec) || !al(G, kVec) || !al(ids, 4) || !al(route, kVec) || !al(t_saved, 4) || !al(grad_X, kVec) ||
      !al(dA, 4) || !al(dB, 4) || !al(workspace, kVec))
    return LQ_ERR_ARG;
  if (!valid_M(M) || q.N % 8 != 0 || (d && !drop_fits(M, q.K))) return LQ_ERR_SHAPE;
  const int64_t r8 = sum_r8(set);
  if (!workspace || ws_bytes < backward_ws(q, M, v, r8, d != nullptr)) return LQ_ERR_WORKSPACE;
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
  float* down_t = cv.take<float>(adapter_down_ws_floats(M, q.K, v.rs, d != nullptr));
  float* down_u = cv.take<float>(adapter_down_ws_floats(M, q.N, v.rs, d != nullptr));
  if (!cv.ok()) return LQ_ERR_WORKSPACE;
  if (!grad_X && !dA && !dB) return LQ_OK;

  const bool need_u = grad_X || dA, nf4 = q.format == LQ_FMT_NF4;
  const Prep prep{route ? nullptr : rws,   q, !grad_X ? nullptr : nf4 ? wt : wd, nf4 ? ldb : 0, v, grad_X ? at : nullptr,
                  need_u ? bt : nullptr, nullptr, zeros};
  hipError_t e = launch_adapter_prep(ids, M, &prep, 1, s);
  if (e != hipSuccess) return LQ_ERR_LAUNCH;
  const Route rt = route_view(route ? route : rws, M, v.n);
  DownJob jobs[2];
  int nj = 0;
  if (need_u) jobs[nj++] = DownJob{G, q.N, bt, nullptr, u, nullptr, down_u, DropView{}, factor, v, 1};
  if (dB) jobs[nj++] = DownJob{t_saved ? nullptr : X, q.K, nullptr, t_saved, t, nullptr, down_t,
                                t_saved ? DropView{} : drop, t_saved ? 1.0f : factor, v, 1};
  if (nj && (e = launch_adapter_down(jobs, nj, M, rt, zeros, s)) != hipSuccess) return LQ_ERR_LAUNCH;
  ColReq cols[2];
  int nc = 0;
  if (dB) cols[nc++] = ColReq{t, G, q.N, dB, 1, part_b, DropView{}, v};
  if (dA) cols[nc++] = ColReq{u, X, q.K, dA, 0, part_a, drop, v};
  ColJoin join;
  if (nc && ((e = launch_adapter_col(cols, nc, M, rt, &join, s)) != hipSuccess ||
             (e = launch_adapter_col_reduce(&join, 1, rt, s)) != hipSuccess))
    return LQ_ERR_LAUNCH;
  if (!grad_X) return LQ_OK;
  if (!nf4 && (e = launch_transpose_weight(wd, q.N, q.K, ldb, wt, nullptr, nullptr, s)) != hipSuccess) return LQ_ERR_LAUNCH;
  const AdapterGemm g{G,  M, q.K, q.N, q.N, wt, ldb, {{u, v, at, drop}, {}}, 1, rt, grad_X,
                      0,  zeros, GEMM_ONE, nullptr, 0, nullptr, nullptr};
  return launch_status(launch_adapter_gemm(g, s));
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
  const Prep prep{route, QWeight{}, nullptr, 0, AdapterView{nullptr, n, 0, 0}, nullptr, nullptr, nullptr, nullptr};
  return launch_status(launch_adapter_prep(ids, M, &prep, 1, (hipStream_t)stream));
}

size_t lq_adapters_forward_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set) {
  QWeight q;
  AdapterView v;
  if (check_qweight(w, &q) != LQ_OK || !valid_M(M) || check_set(set, q.N, q.K, &v) != LQ_OK) return 0;
  return forward_ws(q, M, v, set, false);
}

int lq_adapters_forward(const lq_qweight* w, const uint16_t* X, int64_t M, const lq_adapter_set* set,
                        const int32_t* ids, const int32_t* route, void* H, int32_t h_dtype, float* t_save,
                        void* workspace, size_t ws_bytes, void* stream) {
  return run_forward(w, X, M, set, ids, route, nullptr, H, h_dtype, t_save, workspace, ws_bytes, stream);
}

size_t lq_adapters_backward_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set) {
  QWeight q;
  AdapterView v;
  if (check_qweight(w, &q) != LQ_OK || !valid_M(M) || check_set(set, q.N, q.K, &v) != LQ_OK || q.N % 8 != 0) return 0;
  return backward_ws(q, M, v, sum_r8(set), false);
}

int lq_adapters_backward(const lq_qweight* w, const uint16_t* X, const uint16_t* G, int64_t M,
                         const lq_adapter_set* set, const int32_t* ids, const int32_t* route, const float* t_saved,
                         uint16_t* grad_X, float* dA, float* dB, void* workspace, size_t ws_bytes, void* stream) {
  return run_backward(w, X, G, M, set, ids, route, nullptr, t_saved, grad_X, dA, dB, workspace, ws_bytes, stream);
}

// ---- dropout --------------------------------------------------------------------
int lq_dropout_apply(const lq_dropout* d, const void* x, int64_t numel, int32_t dtype, void* out, void* stream) {
  DropView drop;
  float factor;
  if (!d) return LQ_ERR_ARG;
  const int st = drop_view(d, &drop, &factor);
  if (st != LQ_OK) return st;
  if (dtype != LQ_F32 && dtype != LQ_BF16 && dtype != LQ_F16) return LQ_ERR_ARG;
  if (numel < 0 || numel >= (int64_t(1) << 47)) return LQ_ERR_SHAPE;
  if (numel == 0) return LQ_OK;
  const uintptr_t size = dtype == LQ_F32 ? 4 : 2;
  if (!x || !out || !al(x, size) || !al(out, size)) return LQ_ERR_ARG;
  return launch_status(launch_dropout(drop, factor, x, numel, dtype, out, (hipStream_t)stream));
}

size_t lq_adapters_forward_dropout_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set) {
  QWeight q;
  AdapterView v;
  if (check_qweight(w, &q) != LQ_OK || !valid_M(M) || check_set(set, q.N, q.K, &v) != LQ_OK || !drop_fits(M, q.K)) return 0;
  return forward_ws(q, M, v, set, true);
}

int lq_adapters_forward_dropout(const lq_qweight* w, const uint16_t* X, int64_t M, const lq_adapter_set* set,
                                const int32_t* ids, const int32_t* route, const lq_dropout* d, void* H,
                                int32_t h_dtype, float* t_save, void* workspace, size_t ws_bytes, void* stream) {
  if (!d) return LQ_ERR_ARG;
  return run_forward(w, X, M, set, ids, route, d, H, h_dtype, t_save, workspace, ws_bytes, stream);
}

size_t lq_adapters_backward_dropout_workspace(const lq_qweight* w, int64_t M, const lq_adapter_set* set) {
  QWeight q;
  AdapterView v;
  if (check_qweight(w, &q) != LQ_OK || !valid_M(M) || check_set(set, q.N, q.K, &v) != LQ_OK || q.N % 8 != 0 ||
      !drop_fits(M, q.K))
    return 0;
  return backward_ws(q, M, v, sum_r8(set), true);
}

int lq_adapters_backward_dropout(const lq_qweight* w, const uint16_t* X, const uint16_t* G, int64_t M,
                                 const lq_adapter_set* set, const int32_t* ids, const int32_t* route,
                                 const lq_dropout* d, const float* t_saved, uint16_t* grad_X, float* dA, float* dB,
                                 void* workspace, size_t ws_bytes, void* stream) {
  if (!d) return LQ_ERR_ARG;
  return run_backward(w, X, G, M, set, ids, route, d, t_saved, grad_X, dA, dB, workspace, ws_bytes, stream);
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
