// Host-side helpers shared by the API translation units: the thread's last error text, argument
// checks that return a status, and the tensor-map encoder of the driver.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <string>

#include "mlaprolog.h"

namespace mlap {

inline thread_local std::string g_last_error;   // mlap_last_error's text

inline mlap_status_t fail(mlap_status_t code, const std::string& msg) {
  g_last_error = msg;
  return code;
}

#define CHECK_STATUS(expr)              \
  do {                                  \
    mlap_status_t _s = (expr);          \
    if (_s != MLAP_OK) return _s;       \
  } while (0)

inline size_t dtype_bytes(int32_t dt) {
  switch (dt) {
    case MLAP_DTYPE_BF16:
    case MLAP_DTYPE_FP16: return 2;
    case MLAP_DTYPE_FP32: return 4;
    case MLAP_DTYPE_INT8: return 1;
    case MLAP_DTYPE_INT64: return 8;
    default: return 0;
  }
}

inline int64_t numel(const mlap_tensor_t& t) {
  int64_t n = 1;
  for (int i = 0; i < t.ndim; ++i) n *= t.shape[i];
  return n;
}

inline std::string shape_str(const mlap_tensor_t& t) {
  std::string s = "(";
  for (int i = 0; i < t.ndim; ++i) s += (i ? "," : "") + std::to_string(t.shape[i]);
  return s + ")";
}

inline bool present(const mlap_tensor_t& t) { return t.data != nullptr; }

// align: bytes that the kernels read or write of the tensor at a time.
inline mlap_status_t need(const mlap_tensor_t& t, const char* name, bool allow_empty, unsigned align = 16) {
  if (t.ndim < 0 || t.ndim > 4) return fail(MLAP_ERR_SHAPE, std::string(name) + ": ndim out of range");
  for (int i = 0; i < t.ndim; ++i)
    if (t.shape[i] < 0) return fail(MLAP_ERR_SHAPE, std::string(name) + ": negative dimension");
  if (t.data == nullptr && !(allow_empty && numel(t) == 0))
    return fail(MLAP_ERR_NULL, std::string(name) + " is NULL");
  if (t.data != nullptr && (reinterpret_cast<uintptr_t>(t.data) & (align - 1)) != 0)
    return fail(MLAP_ERR_UNSUPPORTED,
                std::string(name) + ": data pointer not " + std::to_string(align) + "-byte aligned");
  return MLAP_OK;
}

inline mlap_status_t want_dtype(const mlap_tensor_t& t, const char* name, int32_t dt) {
  if (t.dtype != dt) return fail(MLAP_ERR_DTYPE, std::string(name) + ": unexpected dtype");
  return MLAP_OK;
}

inline mlap_status_t want_shape(const mlap_tensor_t& t, const char* name, std::initializer_list<int64_t> s) {
  bool ok = t.ndim == static_cast<int32_t>(s.size());
  int i = 0;
  for (int64_t d : s) {
    if (!ok) break;
    ok = t.shape[i++] == d;
  }
  if (!ok) return fail(MLAP_ERR_SHAPE, std::string(name) + ": shape " + shape_str(t) + " does not match");
  return MLAP_OK;
}

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

inline mlap_status_t cuda_fail(cudaError_t e, const char* what) {
  return fail(MLAP_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

}  // namespace mlap
