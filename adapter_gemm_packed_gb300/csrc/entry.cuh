// What the C entry points of the operators around the packed projections share: error reporting,
// argument checks of head tensors, and the launch count.  (The layer's own entry points, in api.cu,
// keep their private helpers.)
#pragma once
#include <cstdint>
#include <cstdio>
#include <string>

#include <cudaTypedefs.h>

#include "common.cuh"
#include "mlora.h"

namespace mlora {

void set_last_error(const std::string& msg);
void count_launches(int n);
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

inline mlora_status op_fail(mlora_status s, const char* msg) {
  set_last_error(msg);
  return s;
}

inline mlora_status op_cuda_fail(cudaError_t e, const char* where) {
  set_last_error(std::string(where) + ": " + cudaGetErrorString(e));
  return MLORA_ERR_CUDA;
}

inline bool ptr_aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A head tensor [n_tokens, n_heads, head_dim] is usable when its base is 16-byte aligned, both strides
// are multiples of 16 bytes (so every head vector starts on a 16-byte boundary) and no two vectors
// overlap: token by token (the heads of a token together, as in a packed projection's output) or head
// by head (the tokens of a head together).
inline mlora_status check_heads(const mlora_heads* t, const char* name, int64_t n_tokens, int n_heads, int head_dim,
                                int esize) {
  char buf[200];
  if (!t || !t->data) {
    snprintf(buf, sizeof buf, "%s: null tensor argument", name);
    return op_fail(MLORA_ERR_INVALID, buf);
  }
  // (the stride of a dimension with one element is never used, and views carry anything there)
  const int64_t unit = 16 / esize, rs = n_tokens == 1 ? 0 : t->row_stride, hs = n_heads == 1 ? 0 : t->head_stride;
  if (!ptr_aligned(t->data, 16) || rs % unit || hs % unit) {
    snprintf(buf, sizeof buf, "%s: the base and both strides must be multiples of 16 bytes", name);
    return op_fail(MLORA_ERR_INVALID, buf);
  }
  constexpr int64_t FAR = int64_t(1) << 36;   // keeps every offset in bytes within 64 bits and a tensor map's limit
  if (rs < 0 || hs < 0 || rs > FAR || hs > FAR) {
    snprintf(buf, sizeof buf, "%s: stride out of range", name);
    return op_fail(MLORA_ERR_INVALID, buf);
  }
  const bool by_token = (n_heads == 1 || hs >= head_dim) && (n_tokens == 1 || rs >= (n_heads - 1) * hs + head_dim);
  const bool by_head = (n_tokens == 1 || rs >= head_dim) && (n_heads == 1 || hs >= (n_tokens - 1) * rs + head_dim);
  if (!by_token && !by_head) {
    snprintf(buf, sizeof buf, "%s: head vectors overlap (row stride %lld, head stride %lld)", name,
             static_cast<long long>(rs), static_cast<long long>(hs));
    return op_fail(MLORA_ERR_INVALID, buf);
  }
  return MLORA_OK;
}

inline cudaError_t device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) : e;
}

}  // namespace mlora
