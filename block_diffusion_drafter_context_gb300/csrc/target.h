// Host-side checks shared by the target-side operators (append to the paged
// cache, attention over it).
#pragma once

#include <atomic>

#include "internal.h"

namespace dflash {

constexpr int PAGE = 64;             // tokens per cache page
constexpr int TARGET_MAX_NEW = 16;   // newest tokens per request of one attention call

// The arguments both calls share; `who` names the call in the message.
int check_target(const char *who, const dflash_heads *hs, const dflash_kv *kv, int layer, const void *rows,
                 long long row_stride, int row_elems, const int32_t *cu_new, int total_new, const int32_t *ctx_len,
                 int batch, const void *workspace, size_t workspace_bytes, size_t need);
int check_heads(const char *who, const dflash_heads *hs);
// The current device and its SM count, looked up once per device.
struct Device {
  int index = 0, sms = 0;
};
int current_device(Device *d);
// A kernel's dynamic shared memory limit, set once per device (`done`: a bit
// per device, one mask per kernel; devices past 63 are set on every call).
template <typename K>
int allow_smem(std::atomic<uint64_t> &done, const Device &d, K *kernel, int bytes) {
  const uint64_t bit = d.index < 64 ? 1ull << d.index : 0;
  if (done.load(std::memory_order_relaxed) & bit) return DFLASH_OK;
  if (int e = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes),
                         "dynamic shared memory"))
    return e;
  done.fetch_or(bit, std::memory_order_relaxed);
  return DFLASH_OK;
}
// the same for clusters of more than 8 CTAs
template <typename K>
int allow_wide_clusters(std::atomic<uint64_t> &done, const Device &d, K *kernel) {
  const uint64_t bit = d.index < 64 ? 1ull << d.index : 0;
  if (done.load(std::memory_order_relaxed) & bit) return DFLASH_OK;
  if (int e = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), "cluster size"))
    return e;
  done.fetch_or(bit, std::memory_order_relaxed);
  return DFLASH_OK;
}

// whether any of these pointers to 4-byte elements is misaligned
template <typename... P>
inline bool off_words(const P *...p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 3) != 0;
}
inline int elt_bytes(const dflash_heads &h) { return h.dtype == DFLASH_F32 ? 4 : 2; }
// first element of a layer's K (and V) pages
inline size_t layer_offset(const dflash_heads &h, const dflash_kv &kv, int layer) {
  return static_cast<size_t>(layer) * kv.num_pages * h.n_kv_heads * PAGE * h.head_dim;
}

}  // namespace dflash
