// Appending keys and values to the paged cache: per-head q / k RMSNorm,
// rotation and the scatter into K and V^T pages, in one pass over a fused
// q | k | v projection (dflash_append_kv).
//
// For each token at position p and each q / k head x of d values:
//   y = g x / sqrt(mean(x^2) + eps),  (y_i, y_{i+d/2}) turned by p theta_i,
//   theta_i = base^(-2i/d);  V heads are copied.
// A value is read once and written once and takes some ten operations: with
// one token the launch is latency (three dependent loads: the token's
// request, its page, then the store), with prompts it is HBM.
#include "common.cuh"
#include "rope.cuh"
#include "target.h"

#include <mutex>

namespace dflash {
namespace {

constexpr int TT = 16;        // tokens per CTA
constexpr int THREADS = 256;

struct AppendArgs {
  const void *qkv;
  long long ld;               // elements
  const float *g_q, *g_k;     // null: no norm
  float eps;
  int rotate;
  const int32_t *cu_new, *ctx_len, *page_table;
  int B, total, max_pages, num_pages;
  int nq, nkv, g, hpc;        // hpc: kv heads (with their q heads) per CTA
  void *k, *v, *q_out;
  int *status;
};

// 8 consecutive values of a row
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The last b < B with cu[b] <= t, searched 32 ways by the whole warp: one
// dependent load for batches up to 32, two up to 1024.
__device__ __forceinline__ int request_of(const int32_t *cu, int B, int t, int lane) {
  int lo = 0, n = B;   // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, i < n && cu[lo + i] <= t);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// CTA (token tile, group of kv heads).  A row (one head of one token) is
// D / 8 lanes with 16 bytes of bf16 (or 32 of fp32) each, the pair
// (i, i + D/2) D/16 lanes apart.  The rotation of the tile's tokens is
// tabulated once per CTA and shared by its heads.  V rows pass through
// shared memory, so that a d-row's consecutive slots are written together.
template <typename T, int D>
__global__ void __launch_bounds__(THREADS) append_kernel(const AppendArgs a, const RopeArgs rp) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, HALF = D / 2, ROWS = (THREADS / 32) * RPW;
  __shared__ __align__(16) float2 cs[TT][HALF];
  __shared__ __align__(16) T vt[TT][D];
  __shared__ int s_page[TT], s_pos[TT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * TT, h0 = blockIdx.y * a.hpc, nh = min(a.hpc, a.nkv - h0);
  float th_hi[HALF / 32], th_lo[HALF / 32];
  lane_thetas(rp, lane, th_hi, th_lo);
  pdl_start();
  const int total = min(a.total, a.cu_new[a.B]);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && (a.cu_new[a.B] > a.total || a.cu_new[a.B] < 0))
    report(a.status, DFLASH_ERR_DEVICE);
  const int nt = min(TT, total - t0);
  if (nt <= 0) return;
  for (int j = warp; j < nt; j += THREADS / 32) {
    const int t = t0 + j, b = request_of(a.cu_new, a.B, t, lane);
    const int first = a.cu_new[b], c = a.ctx_len[b];
    const long long pos = static_cast<long long>(c) + t - first;
    const bool in = first >= 0 && first <= t && c >= 0 && pos < static_cast<long long>(a.max_pages) * PAGE;
    const int pg = in ? a.page_table[static_cast<size_t>(b) * a.max_pages + pos / PAGE] : -1;
    const bool ok = pg >= 0 && pg < a.num_pages;
    const int p = in ? static_cast<int>(pos) : 0;
    if (lane == 0) {
      if (!ok) report(a.status, DFLASH_ERR_DEVICE);
      s_page[j] = ok ? pg : -1;
      s_pos[j] = p;
    }
#pragma unroll
    for (int i = 0; i < HALF / 32; ++i) {
      float co = 1.f, si = 0.f;
      if (a.rotate) rope_cs(p, th_hi[i], th_lo[i], co, si);
      cs[j][lane + 32 * i] = make_float2(co, si);
    }
  }
  __syncthreads();
  const T *src = static_cast<const T *>(a.qkv) + static_cast<size_t>(t0) * a.ld;
  const int slot = threadIdx.x / LPR, l8 = (threadIdx.x % LPR) * 8;   // this thread's row of a pass, its 8 columns
  // ---- q heads of the group, then its k heads: rows (head, token)
  const int nqh = a.q_out ? nh * a.g : 0, items = (nqh + nh) * nt;
  float gq[8], gk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    gq[i] = a.g_q ? a.g_q[l8 + i] : 1.f;
    gk[i] = a.g_k ? a.g_k[l8 + i] : 1.f;
  }
  constexpr int U = 4;   // rows in flight per thread
  for (int it0 = slot; it0 - slot < items; it0 += ROWS * U) {
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = it0 + u * ROWS;
      if (it < items) {
        const int j = it % nt, hh = it / nt;
        const size_t col = static_cast<size_t>(hh < nqh ? h0 * a.g + hh : a.nq + h0 + hh - nqh) * D + l8;
        load8(src + j * a.ld + col, x[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = it0 + u * ROWS;
      const bool live = it < items;
      const int j = live ? it % nt : 0, hh = live ? it / nt : 0;
      const bool isq = hh < nqh;
      if (a.g_q) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[u][i], x[u][i], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss / D + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] *= r * (isq ? gq[i] : gk[i]);
      }
      const float4 *c4 = reinterpret_cast<const float4 *>(&cs[j][l8 % HALF]);
      const float sign = l8 < HALF ? -1.f : 1.f;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float4 c = c4[i / 2];
        const float o0 = __shfl_xor_sync(0xffffffffu, x[u][i], LPR / 2);
        const float o1 = __shfl_xor_sync(0xffffffffu, x[u][i + 1], LPR / 2);
        y[i] = fmaf(sign * c.y, o0, x[u][i] * c.x);
        y[i + 1] = fmaf(sign * c.w, o1, x[u][i + 1] * c.z);
      }
      if (live) {
        if (isq) {
          store8(static_cast<T *>(a.q_out) + (static_cast<size_t>(t0 + j) * a.nq + h0 * a.g + hh) * D + l8, y);
        } else if (s_page[j] >= 0) {
          store8(static_cast<T *>(a.k) +
                     ((static_cast<size_t>(s_page[j]) * a.nkv + h0 + hh - nqh) * PAGE + s_pos[j] % PAGE) * D + l8,
                 y);
        }
      }
    }
  }
  // ---- v heads, transposed into [d][slot] pages
  for (int h = h0; h < h0 + nh; ++h) {
    constexpr int V16 = 16 / sizeof(T);
    __syncthreads();
    for (int e = threadIdx.x; e < nt * (D / V16); e += THREADS) {
      const int j = e / (D / V16), c = (e % (D / V16)) * V16;
      *reinterpret_cast<uint4 *>(&vt[j][c]) =
          *reinterpret_cast<const uint4 *>(src + j * a.ld + static_cast<size_t>(a.nq + a.nkv + h) * D + c);
    }
    __syncthreads();
    // 16 consecutive threads cover one d-row's tokens (consecutive slots)
    for (int e = threadIdx.x; e < TT * D; e += THREADS) {
      const int d = e / TT, j = e % TT;
      const int pg = j < nt ? s_page[j] : -1;
      if (pg >= 0)
        static_cast<T *>(a.v)[((static_cast<size_t>(pg) * a.nkv + h) * D + d) * PAGE + s_pos[j] % PAGE] = vt[j][d];
    }
  }
}

// theta tables depend on (d, base) alone; 64 pow calls are most of a small
// call's host time, so the last table is kept
const RopeArgs &rope_of(int d, float base) {
  static thread_local RopeArgs tab;
  static thread_local int tab_d = 0;
  static thread_local float tab_base = 0.f;
  if (tab_d != d || tab_base != base) {
    tab = rope_table(d, base);
    tab_d = d;
    tab_base = base;
  }
  return tab;
}

}  // namespace

int check_heads(const char *who, const dflash_heads *hs) {
  if (!hs) return set_error(DFLASH_ERR_ARG, "%s: null heads", who);
  if (hs->dtype != DFLASH_BF16 && hs->dtype != DFLASH_F32)
    return set_error(DFLASH_ERR_ARG, "%s: dtype must be bf16 or fp32", who);
  if (hs->n_q_heads <= 0 || hs->n_kv_heads <= 0 || hs->n_q_heads % hs->n_kv_heads)
    return set_error(DFLASH_ERR_SHAPE, "%s: kv heads must divide q heads", who);
  if (hs->head_dim != 64 && hs->head_dim != 128)
    return set_error(DFLASH_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128", who);
  if (hs->n_q_heads / hs->n_kv_heads > 8 || hs->n_kv_heads > 1024)
    return set_error(DFLASH_ERR_UNSUPPORTED, "%s: at most 8 q heads per kv head and 1024 kv heads", who);
  return DFLASH_OK;
}

int check_target(const char *who, const dflash_heads *hs, const dflash_kv *kv, int layer, const void *rows,
                 long long row_stride, int row_elems, const int32_t *cu_new, int total_new, const int32_t *ctx_len,
                 int batch, const void *workspace, size_t workspace_bytes, size_t need) {
  if (!kv || !kv->k_cache || !kv->v_cache || !kv->page_table || !cu_new || !ctx_len || !workspace ||
      (total_new > 0 && !rows))
    return set_error(DFLASH_ERR_ARG, "%s: null argument", who);
  if (batch < 0 || batch > DFLASH_MAX_BATCH || total_new < 0 || layer < 0)
    return set_error(DFLASH_ERR_ARG, "%s: batch, total_new or layer out of range", who);
  if (kv->num_pages <= 0 || kv->max_pages <= 0 || kv->max_pages > (1 << 18))
    return set_error(DFLASH_ERR_SHAPE, "%s: num_pages must be positive and max_pages in 1..2^18", who);
  if (static_cast<unsigned long long>(kv->num_pages) * hs->n_kv_heads * 128 >= 0x7fffffffull)
    return set_error(DFLASH_ERR_SHAPE, "%s: num_pages x kv heads must stay below 2^24", who);
  const int size = elt_bytes(*hs);
  if (row_stride < row_elems) return set_error(DFLASH_ERR_SHAPE, "%s: row stride below the row's %d elements", who, row_elems);
  if ((row_stride * size) % 16 || (reinterpret_cast<uintptr_t>(rows) & 15) ||
      (reinterpret_cast<uintptr_t>(kv->k_cache) & 15) || (reinterpret_cast<uintptr_t>(kv->v_cache) & 15) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15))
    return set_error(DFLASH_ERR_ALIGN, "%s: rows, their stride, the cache and the workspace must be 16-byte aligned", who);
  if (workspace_bytes < need)
    return set_error(DFLASH_ERR_SHAPE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes, need);
  return DFLASH_OK;
}

int device_sms(int *sms) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = -1;
  if (int e = cuda_check(cudaGetDevice(&dev), "cudaGetDevice")) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < 64 && known[dev]) {
    *sms = known[dev];
    return DFLASH_OK;
  }
  if (int e = cuda_check(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev), "SM count")) return e;
  if (dev >= 0 && dev < 64) known[dev] = *sms;
  return DFLASH_OK;
}

}  // namespace dflash

extern "C" DFLASH_API int dflash_append_kv(const dflash_heads *hs, const dflash_kv *kv, int layer, const void *qkv,
                                           long long row_stride, const float *g_q, const float *g_k, float eps,
                                           float rope_base, const int32_t *cu_new, int total_new,
                                           const int32_t *ctx_len, int batch, void *q_out, void *workspace,
                                           size_t workspace_bytes, dflash_stream_t stream) {
  using namespace dflash;
  const char *who = "append_kv";
  if (int e = check_heads(who, hs)) return e;
  const int nq = hs->n_q_heads, nkv = hs->n_kv_heads, d = hs->head_dim;
  if (int e = check_target(who, hs, kv, layer, qkv, row_stride, (nq + 2 * nkv) * d, cu_new, total_new, ctx_len, batch,
                           workspace, workspace_bytes, 256))
    return e;
  if ((g_q == nullptr) != (g_k == nullptr)) return set_error(DFLASH_ERR_ARG, "append_kv: g_q and g_k, both or neither");
  if (!(eps >= 0.f) || !(rope_base == 0.f || (rope_base > 1.f && rope_base < 3.0e38f)))
    return set_error(DFLASH_ERR_ARG, "append_kv: eps / rope_base out of range");
  if (reinterpret_cast<uintptr_t>(q_out) & 15) return set_error(DFLASH_ERR_ALIGN, "append_kv: q_out not 16-byte aligned");
  if (batch == 0 || total_new == 0) return DFLASH_OK;
  int sms = 0;
  if (int e = device_sms(&sms)) return e;
  const size_t off = layer_offset(*hs, *kv, layer) * elt_bytes(*hs);
  AppendArgs a = {};
  a.qkv = qkv;
  a.ld = row_stride;
  a.g_q = g_q;
  a.g_k = g_k;
  a.eps = eps;
  a.rotate = rope_base != 0.f;
  a.cu_new = cu_new;
  a.ctx_len = ctx_len;
  a.page_table = kv->page_table;
  a.B = batch;
  a.total = total_new;
  a.max_pages = kv->max_pages;
  a.num_pages = kv->num_pages;
  a.nq = nq;
  a.nkv = nkv;
  a.g = nq / nkv;
  a.k = static_cast<char *>(kv->k_cache) + off;
  a.v = static_cast<char *>(kv->v_cache) + off;
  a.q_out = q_out;
  a.status = static_cast<int *>(workspace);
  const int tiles = (total_new + TT - 1) / TT;
  a.hpc = 1;
  const dim3 grid(tiles, (nkv + a.hpc - 1) / a.hpc);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RopeArgs &rp = rope_of(d, a.rotate ? rope_base : 1e6f);
  if (hs->dtype == DFLASH_F32)
    launch_pdl(d == 64 ? append_kernel<float, 64> : append_kernel<float, 128>, grid, dim3(THREADS), 0, s, a, rp);
  else
    launch_pdl(d == 64 ? append_kernel<__nv_bfloat16, 64> : append_kernel<__nv_bfloat16, 128>, grid, dim3(THREADS), 0,
               s, a, rp);
  return cuda_check(cudaGetLastError(), "append_kv launch");
}
