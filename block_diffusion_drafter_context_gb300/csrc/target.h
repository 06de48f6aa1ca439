// Host-side checks shared by the target-side operators (append to the paged
// cache, attention over it).
#pragma once

#include "internal.h"

namespace dflash {

constexpr int PAGE = 64;             // tokens per cache page
constexpr int TARGET_MAX_NEW = 16;   // newest tokens per request of one attention call

// The arguments both calls share; `who` names the call in the message.
int check_target(const char *who, const dflash_heads *hs, const dflash_kv *kv, int layer, const void *rows,
                 long long row_stride, int row_elems, const int32_t *cu_new, int total_new, const int32_t *ctx_len,
                 int batch, const void *workspace, size_t workspace_bytes, size_t need);
int check_heads(const char *who, const dflash_heads *hs);
// SM count of the current device, looked up once per device
int device_sms(int *sms);

inline int elt_bytes(const dflash_heads &h) { return h.dtype == DFLASH_F32 ? 4 : 2; }
// first element of a layer's K (and V) pages
inline size_t layer_offset(const dflash_heads &h, const dflash_kv &kv, int layer) {
  return static_cast<size_t>(layer) * kv.num_pages * h.n_kv_heads * PAGE * h.head_dim;
}

}  // namespace dflash
