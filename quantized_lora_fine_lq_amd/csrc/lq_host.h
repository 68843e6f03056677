// Host-side helpers shared by the C-ABI files: alignment checks, workspace
// carving and the validation of weight descriptors.
#pragma once

#include "lq_internal.h"

namespace lq {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int launch_status(hipError_t e) { return e == hipSuccess ? LQ_OK : LQ_ERR_LAUNCH; }

// Alignment of a device pointer (a null pointer passes; nullness is checked
// separately). Bulk tensors are read and written with 16-byte vector
// accesses; per-element arrays need their natural alignment.
constexpr uintptr_t kVec = 16;
inline bool al(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Validate a weight descriptor and turn it into the kernels' view.
int check_qweight(const lq_qweight* w, QWeight* out);

// Debug build: the row layout of a codebook weight, checked on the host.
int debug_check_weight(const QWeight& q, hipStream_t s);

// Carves a caller workspace into aligned pieces; ok() is false if the pieces
// ran past its size (the entry points size the workspace first, so this is a
// bounds assert on that arithmetic).
struct Carver {
  char* base;
  size_t cap;
  size_t used = 0;
  Carver(void* p, size_t bytes) : base((char*)p), cap(bytes) {}
  template <class T> T* take(size_t count) {
    T* p = reinterpret_cast<T*>(base + used);
    used += align_up(count * sizeof(T));
    return p;
  }
  bool ok() const { return used <= cap; }
};

}  // namespace lq
