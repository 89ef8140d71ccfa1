// ss_host.h -- host-side checks of ss_tensor arguments and the workspace pool, shared by the C-ABI files.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <mutex>

#include "../../include/ss_scan.h"

namespace ss {
namespace host {

inline bool present(const ss_tensor* t) { return t != nullptr && t->data != nullptr; }

inline int64_t esize(int32_t dt) { return dt == SS_BF16 ? 2 : 4; }

// Byte extent [lo, hi) touched by a strided tensor (strides non-negative, checked first).
inline void extent(const ss_tensor* t, uintptr_t* lo, uintptr_t* hi) {
  int64_t last = 0;
  for (int i = 0; i < t->ndim; ++i) last += (t->shape[i] - 1) * t->stride[i];
  *lo = reinterpret_cast<uintptr_t>(t->data);
  *hi = *lo + (uintptr_t)((last + 1) * esize(t->dtype));
}

inline int64_t numel(const ss_tensor* t) {
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
  return n;
}

// passed by the caller: a descriptor with data, or one of no elements (whose data may be NULL)
inline bool given(const ss_tensor* t) {
  if (t == nullptr) return false;
  if (t->data != nullptr) return true;
  if (t->ndim < 1 || t->ndim > 4) return false;
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] == 0) return true;
  return false;
}

inline int check_basic(const ss_tensor* t, int ndim) {
  if (t->ndim != ndim) return SS_ERR_SHAPE;
  if (t->dtype != SS_F32 && t->dtype != SS_BF16) return SS_ERR_DTYPE;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] < 0) return SS_ERR_SHAPE;
    if (t->stride[i] < 0) return SS_ERR_STRIDE;
  }
  if (t->stride[ndim - 1] != 1 && t->shape[ndim - 1] > 1) return SS_ERR_STRIDE;
  return SS_OK;
}

inline bool aligned16(const ss_tensor* t) {
  if (reinterpret_cast<uintptr_t>(t->data) % 16) return false;
  const int64_t es = esize(t->dtype);
  for (int i = 0; i + 1 < t->ndim; ++i)
    if (t->shape[i] > 1 && (t->stride[i] * es) % 16) return false;
  return true;
}

// Stream-ordered workspace from a memory pool the library owns on each device.  The pool keeps
// freed blocks (its release threshold is "never"), so a call repeated on a stream reuses the
// same memory without a device allocation.  SS_FAULT=alloc in the environment makes the
// allocation fail, so that the failure path (SS_ERR_HIP, nothing enqueued, y untouched) can be
// exercised.
constexpr int kMaxDevices = 64;

inline hipError_t ws_pool(hipMemPool_t* pool) {
  static std::mutex mu;
  static hipMemPool_t pools[kMaxDevices] = {};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!pools[dev]) {
    hipMemPoolProps props = {};
    props.allocType = hipMemAllocationTypePinned;
    props.location.type = hipMemLocationTypeDevice;
    props.location.id = dev;
    hipMemPool_t p = nullptr;
    if ((e = hipMemPoolCreate(&p, &props)) != hipSuccess) return e;
    uint64_t keep = UINT64_MAX;
    if ((e = hipMemPoolSetAttribute(p, hipMemPoolAttrReleaseThreshold, &keep)) != hipSuccess) {
      (void)hipMemPoolDestroy(p);
      return e;
    }
    pools[dev] = p;
  }
  *pool = pools[dev];
  return hipSuccess;
}

inline hipError_t ws_alloc(void** ws, size_t bytes, hipStream_t s) {
  const char* fault = getenv("SS_FAULT");
  if (fault && strcmp(fault, "alloc") == 0) return hipErrorOutOfMemory;
  hipMemPool_t pool;
  hipError_t e = ws_pool(&pool);
  if (e != hipSuccess) return e;
  return hipMallocFromPoolAsync(ws, bytes, pool, s);
}

inline bool overlaps(const ss_tensor* a, const ss_tensor* b) {
  if (!present(a) || !present(b) || numel(a) == 0 || numel(b) == 0) return false;
  uintptr_t alo, ahi, blo, bhi;
  extent(a, &alo, &ahi);
  extent(b, &blo, &bhi);
  return alo < bhi && blo < ahi;
}

// Whether two views of the same rows lie in different parts of the row: the first `outer` dimensions
// of both are multiples of one common row stride, and the rest stays inside its own part of a row.
inline bool beside(const ss_tensor* a, const ss_tensor* b, int outer) {
  const int64_t ea = esize(a->dtype), eb = esize(b->dtype);
  int64_t row = 0;
  for (int i = 0; i < outer; ++i)
    if (a->shape[i] > 1 && (row == 0 || a->stride[i] * ea < row)) row = a->stride[i] * ea;
  if (row <= 0) return false;
  int64_t ia = ea, ib = eb;
  for (int i = 0; i < a->ndim; ++i) {
    if (i >= outer) ia += (a->shape[i] - 1) * a->stride[i] * ea;
    else if (a->shape[i] > 1 && (a->stride[i] * ea) % row) return false;
  }
  for (int i = 0; i < b->ndim; ++i) {
    if (i >= outer) ib += (b->shape[i] - 1) * b->stride[i] * eb;
    else if (b->shape[i] > 1 && (b->stride[i] * eb) % row) return false;
  }
  const int64_t from_a = (int64_t)(reinterpret_cast<uintptr_t>(b->data) - reinterpret_cast<uintptr_t>(a->data));
  const int64_t d = ((from_a % row) + row) % row;  // b's place in a's row
  return d >= ia && d + ib <= row;
}

// Like overlaps(), except that the slices of one fused buffer, whose byte ranges interleave without
// sharing an element, are told apart by their place in the row.
inline bool shares(const ss_tensor* a, const ss_tensor* b) {
  if (!overlaps(a, b)) return false;
  for (int outer = 1; outer < a->ndim && outer < b->ndim; ++outer)
    if (beside(a, b, outer)) return false;
  return true;
}

inline bool same_view(const ss_tensor* a, const ss_tensor* b) {
  if (!present(a) || !present(b)) return false;
  if (a->data != b->data || a->dtype != b->dtype || a->ndim != b->ndim) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i] || (a->shape[i] > 1 && a->stride[i] != b->stride[i])) return false;
  return true;
}

// whether two of a tensor's own elements may share an address (a tensor that is written must not)
inline bool folds(const ss_tensor* t) {
  int order[4], n = 0;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] == 0) return false;
    if (t->shape[i] > 1) order[n++] = i;
  }
  for (int i = 1; i < n; ++i)
    for (int j = i; j > 0 && t->stride[order[j]] < t->stride[order[j - 1]]; --j) {
      const int x = order[j];
      order[j] = order[j - 1];
      order[j - 1] = x;
    }
  int64_t reach = 0;
  for (int i = 0; i < n; ++i) {
    if (t->stride[order[i]] <= reach) return true;
    reach += (t->shape[order[i]] - 1) * t->stride[order[i]];
  }
  return false;
}

// ---- shared by the operators around and beside the scan ----

// an operand of float type: dimensions, strides, dtype
inline int check_in(const ss_tensor* t, int ndim, const int64_t* shape) {
  int rc;
  if ((rc = check_basic(t, ndim))) return rc;
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] != shape[i]) return SS_ERR_SHAPE;
  return SS_OK;
}

inline int check_out(const ss_tensor* t, int ndim, const int64_t* shape) {
  const int rc = check_in(t, ndim, shape);
  if (rc) return rc;
  return folds(t) ? SS_ERR_STRIDE : SS_OK;
}

// a 1-D f32 tensor of n values
inline int check_vector(const ss_tensor* t, int64_t n) {
  int rc;
  if ((rc = check_basic(t, 1))) return rc;
  if (t->dtype != SS_F32) return SS_ERR_DTYPE;
  return t->shape[0] == n ? SS_OK : SS_ERR_SHAPE;
}

// an i32 tensor of the given shape, any non-negative strides
inline int check_i32(const ss_tensor* t, int ndim, const int64_t* shape) {
  if (t->ndim != ndim) return SS_ERR_SHAPE;
  if (t->dtype != SS_I32) return SS_ERR_DTYPE;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] != shape[i]) return SS_ERR_SHAPE;
    if (t->stride[i] < 0) return SS_ERR_STRIDE;
  }
  return SS_OK;
}

// whether `out` shares an element with one of ts, of which ts[self] is out itself (a caller may pass one
// descriptor for two arguments, so its address does not tell)
inline bool any_shares(const ss_tensor* out, const ss_tensor* const* ts, int n, int self = -1) {
  for (int i = 0; i < n; ++i)
    if (i != self && shares(out, ts[i])) return true;
  return false;
}

// Workspace of `floats` floats: the caller's, or (absent) the pool's, freed on the stream by the
// destructor.  get() validates and allocates; nothing is enqueued before it succeeds.
class Workspace {
 public:
  Workspace(const ss_tensor* given, hipStream_t s) : given_(given), s_(s) {}
  ~Workspace() {
    if (pool_) (void)hipFreeAsync(pool_, s_);
  }
  int get(int64_t floats, float** out) {
    *out = nullptr;
    if (floats <= 0) return SS_OK;
    if (present(given_)) {
      if (given_->shape[0] < floats) return SS_ERR_SCRATCH;
      *out = static_cast<float*>(given_->data);
      return SS_OK;
    }
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(s_, &st) != hipSuccess) {
      (void)hipGetLastError();
      return SS_ERR_HIP;
    }
    if (st != hipStreamCaptureStatusNone) return SS_ERR_SCRATCH;
    if (ws_alloc(&pool_, (size_t)floats * sizeof(float), s_) != hipSuccess) {
      pool_ = nullptr;
      (void)hipGetLastError();
      return SS_ERR_HIP;
    }
    *out = static_cast<float*>(pool_);
    return SS_OK;
  }

 private:
  const ss_tensor* given_;
  hipStream_t s_;
  void* pool_ = nullptr;
};

// a given workspace: 1-D f32, dense, 16-byte aligned, sharing nothing with the call's tensors
inline int check_ws(const ss_tensor* ws, const ss_tensor* const* ts, int n) {
  if (!present(ws)) return SS_OK;
  int rc;
  if ((rc = check_basic(ws, 1))) return rc;
  if (ws->dtype != SS_F32) return SS_ERR_DTYPE;
  if (reinterpret_cast<uintptr_t>(ws->data) % 16) return SS_ERR_STRIDE;
  for (int i = 0; i < n; ++i)
    if (overlaps(ws, ts[i])) return SS_ERR_ALIAS;
  return SS_OK;
}

inline int done(hipError_t e) {
  if (e == hipSuccess) return SS_OK;
  (void)hipGetLastError();
  return SS_ERR_HIP;
}

}  // namespace host
}  // namespace ss
