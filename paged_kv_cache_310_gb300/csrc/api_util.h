// api_util.h -- what the translation units with extern "C" entry points share: error
// recording, descriptor checks, the device error flag (defined in api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pagedkv.h"

namespace pkv {

pkv_status fail(pkv_status st, const char* fmt, ...);
pkv_status cuda_fail(cudaError_t e, const char* what);
// Device address of the error flag on the current device (looked up once per device).
pkv_status device_flag(int** out);
// Checks a pool descriptor; PKV_KV4 pools only where `kv4` says the call takes them.
pkv_status check_cache(const pkv_cache_desc* c, bool kv4 = false);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t elem_bytes(int dtype) { return dtype == PKV_F32 ? 4 : 2; }
// Bytes of one token's row of one KV head, and of a whole block (all heads and rows).
inline int64_t row_bytes(const pkv_cache_desc* c) {
  return c->dtype == PKV_KV4 ? c->head_dim * 5 / 8 : static_cast<int64_t>(c->head_dim * elem_bytes(c->dtype));
}
inline int64_t block_bytes(const pkv_cache_desc* c) {
  return static_cast<int64_t>(c->num_kv_heads) * c->block_size * row_bytes(c);
}

}  // namespace pkv
