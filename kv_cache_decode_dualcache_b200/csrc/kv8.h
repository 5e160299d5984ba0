// What the 8-bit paged K/V cache's calls share on the host: argument checks
// and the cache's dense strides.  Not part of the public C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <initializer_list>
#include <string>

#include "../../include/fdllm.h"

namespace fd {

void set_thread_error(const std::string& msg);  // api.cu: fdllm_last_error(NULL)

namespace kv8 {

inline int fail(const char* call, int code, const std::string& msg) {
  set_thread_error(std::string(call) + ": " + msg);
  return code;
}

inline int elem_bytes(int dtype) {
  return dtype == FDLLM_DTYPE_F32 ? 4 : (dtype == FDLLM_DTYPE_BF16 || dtype == FDLLM_DTYPE_F16) ? 2 : 0;
}

inline bool aligned4(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 3) return false;
  return true;
}
// Whether arrays a of n and b of m int32 share a byte.
inline bool overlap(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return b && x < y + 4 * m && y < x + 4 * n;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Rows of `heads` vectors of hd elements that start on 16-byte boundaries.
inline bool rows_ok(const void* p, const int64_t* strides, int esz) {
  return aligned16(p) && (strides[0] * esz) % 16 == 0 && (strides[1] * esz) % 16 == 0;
}

#ifdef __CUDACC__
// Whether sequence i's rows [starts[i], starts[i + 1]) lie in [0, n_tokens).
__device__ __forceinline__ bool starts_ok(const int32_t* starts, int i, int n_tokens) {
  return 0 <= starts[i] && starts[i] <= starts[i + 1] && starts[i + 1] <= n_tokens;
}
#endif

// Device facts that do not change, asked once per device.
inline cudaError_t sm_count(int* n) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*n = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*n, std::memory_order_relaxed);
  return e;
}
// Raises a kernel's dynamic shared-memory limit, once per device (`ready`:
// one bit a device).
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Checks *c and copies it to *out with its strides filled in.
inline const char* check_cache(const fdllm_kv8* c, fdllm_kv8* out) {
  if (!c) return "cache is NULL";
  *out = *c;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->page_table)
    return "a cache pointer is NULL";
  if (!(c->head_dim == 32 || c->head_dim == 64 || c->head_dim == 128))
    return "head_dim must be 32, 64 or 128";
  if (c->n_kv_heads < 1 || c->n_kv_heads > 65535) return "n_kv_heads must be in [1, 65535]";
  if (c->n_seqs < 1 || c->n_seqs > 65535) return "n_seqs must be in [1, 65535]";
  if (c->n_pages < 1) return "n_pages must be >= 1";
  if (c->max_pages < 1 || c->max_pages > (1 << 24)) return "max_pages must be in [1, 2^24]";
  if (!aligned16(c->k) || !aligned16(c->v)) return "k and v must be 16-byte aligned";
  if (!aligned4({c->k_scale, c->v_scale, c->page_table}))
    return "scales and page_table must be 4-byte aligned";
  const int64_t page = (int64_t)c->n_kv_heads * FDLLM_KV8_PAGE * c->head_dim;
  const int64_t scales = (int64_t)c->n_kv_heads * (FDLLM_KV8_PAGE / FDLLM_KV8_BLOCK);
  if (!out->page_stride) out->page_stride = page;
  if (!out->scale_stride) out->scale_stride = scales;
  if (!out->table_stride) out->table_stride = c->max_pages;
  if (out->page_stride < page || out->page_stride % 16)
    return "page_stride must hold a page and be a multiple of 16";
  if (out->scale_stride < scales) return "scale_stride must hold a page's scales";
  if (out->table_stride < c->max_pages) return "table_stride must hold max_pages entries";
  return nullptr;
}

}  // namespace kv8
}  // namespace fd
