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

namespace dflash {
namespace {

constexpr int TT = 16;        // tokens per CTA at most
constexpr int THREADS = 256;
constexpr int MAX_HPC = 4;    // kv heads per CTA

struct AppendArgs {
  const void *qkv;
  long long ld;               // elements
  const float *g_q, *g_k;     // null: no norm
  float eps;
  int rotate;
  const int32_t *cu_new, *ctx_len, *page_table;
  int B, total, max_pages, num_pages;
  int nq, nkv, g, hpc, tt;    // kv heads (with their q heads) and tokens per CTA
  void *k, *v, *q_out;
  int *status;
};

// 4 consecutive values of a row, as they lie in memory and as fp32
template <typename T> struct Four;
template <> struct Four<float> {
  using Raw = uint4;
  static __device__ __forceinline__ void unpack(const uint4 &u, float *x) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <> struct Four<__nv_bfloat16> {
  using Raw = uint2;
  static __device__ __forceinline__ void unpack(const uint2 &u, float *x) {
    x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
  }
  static __device__ __forceinline__ uint2 pack(const float *x) {
    return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  }
};

// A kernel parameter's element by its generic address: lanes that read
// neighbours share one access, where the constant bank takes one per address
// (walking the table uniformly took 2 us of a CTA).
__device__ __forceinline__ float param_at(const float *p) {
  float v;
  asm volatile("ld.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// The last b < B with cu[b] <= t, for both of a warp's tokens at once.  Up to
// 256 requests every entry is loaded side by side (one dependent load, where a
// binary search takes eight); more are searched 32 ways first.
__device__ __forceinline__ void requests_of(const int32_t *cu, int B, int t0, int t1, int lane, int &b0, int &b1) {
  int base = 0, n = B;
  while (n > 256) {   // the answers are in [base, base + n); t0 <= t1 lie in one tile
    const int step = (n + 31) / 32, i = lane * step;
    const unsigned m0 = __ballot_sync(0xffffffffu, i < n && cu[base + i] <= t0);
    const unsigned m1 = __ballot_sync(0xffffffffu, i < n && cu[base + i] <= t1);
    const int k0 = m0 ? 31 - __clz(m0) : 0, k1 = m1 ? 31 - __clz(m1) : 0;
    base += k0 * step;
    const int m = min(n - k0 * step, (k1 - k0 + 1) * step);
    if (m >= n) break;   // the two answers lie far apart (many empty requests)
    n = m;
  }
  int c0 = 0, c1 = 0;
  for (int i = lane; i < n; i += 32) {
    const int v = cu[base + i];
    c0 += v <= t0;
    c1 += v <= t1;
  }
  b0 = base + max(__reduce_add_sync(0xffffffffu, c0) - 1, 0);
  b1 = base + max(__reduce_add_sync(0xffffffffu, c1) - 1, 0);
}

// CTA (4 to 16 tokens, up to 4 kv heads with their q heads).  A row (one head of
// one token) is D / 8 lanes; lane l holds values 4l..4l+3 of both halves, so
// that the rotation's pairs are its own (with 8 consecutive values per lane
// the exchange and the rotation table made shared memory the bound: 159 us
// for 23 040 prompt tokens of 32 + 16 heads, where this takes 95).  The first
// rows' loads and the V rows' copies into shared memory do not depend on where
// the tokens belong, so they are under way while each token's request, page
// and rotation are looked up (three dependent loads).  The rotation of the
// tile's tokens is tabulated once and shared by the heads.  V leaves transposed.
template <typename T, int D>
__global__ void __launch_bounds__(THREADS) append_kernel(const AppendArgs a, const __grid_constant__ RopeArgs rp) {
  constexpr int LPR = D / 8, HALF = D / 2, ROWS = THREADS / LPR, V16 = 16 / sizeof(T);
  using F = Four<T>;
  __shared__ __align__(16) float2 cs[TT][HALF];      // pairs 4l + 2q, 4l + 2q + 1 as float4 number q LPR + l
  __shared__ __align__(16) T vt[MAX_HPC][TT][D + V16];
  __shared__ __align__(16) float gains[2][D];
  __shared__ int s_page[TT], s_pos[TT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * a.tt, h0 = blockIdx.y * a.hpc, nh = min(a.hpc, a.nkv - h0);
  const int rows = min(a.tt, a.total - t0);            // rows of the buffer; the batch may end before
  const int sh = rows > 8 ? 4 : rows > 4 ? 3 : rows > 2 ? 2 : rows > 1 ? 1 : 0;   // a power of two of tokens
  const int nqh = a.q_out ? nh * a.g : 0, items = (nqh + nh) << sh;               // rows (head, token): q heads, then k
  const int slot = threadIdx.x / LPR, l = threadIdx.x % LPR;                      // this thread's row of a pass, its lane in it
  float th_hi[HALF / 32], th_lo[HALF / 32];
  if (a.rotate) {
#pragma unroll
    for (int i = 0; i < HALF / 32; ++i) {
      th_hi[i] = param_at(rp.th_hi + lane + 32 * i);
      th_lo[i] = param_at(rp.th_lo + lane + 32 * i);
    }
  }
  pdl_start();
  if (a.g_q && threadIdx.x < D) {
    gains[0][threadIdx.x] = a.g_q[threadIdx.x];
    gains[1][threadIdx.x] = a.g_k[threadIdx.x];
  }
  const T *src = static_cast<const T *>(a.qkv) + static_cast<size_t>(t0) * a.ld;
  for (int e = threadIdx.x; e < nh * rows * (D / V16); e += THREADS) {
    const int c = (e % (D / V16)) * V16, hj = e / (D / V16), h = hj / rows, j = hj - h * rows;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&vt[h][j][c])),
                 "l"(src + j * a.ld + static_cast<size_t>(a.nq + a.nkv + h0 + h) * D + c)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  constexpr int U = 4;   // rows in flight per thread
  typename F::Raw raw[U][2];
  auto load = [&](int it0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = it0 + u * ROWS, j = it & ((1 << sh) - 1), hh = it >> sh;
      if (it < items && j < rows) {
        const T *row = src + j * a.ld + static_cast<size_t>(hh < nqh ? h0 * a.g + hh : a.nq + h0 + hh - nqh) * D + 4 * l;
        raw[u][0] = *reinterpret_cast<const typename F::Raw *>(row);
        raw[u][1] = *reinterpret_cast<const typename F::Raw *>(row + HALF);
      }
    }
  };
  load(slot);
  // ---- where the tokens go: warp w looks up tokens w and w + 8
  const int end = a.cu_new[a.B], total = min(a.total, end), nt = min(a.tt, total - t0);
  const int begin = a.cu_new[0], j0 = begin > t0 ? begin - t0 : 0;   // rows before the first request's: left alone
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && (end > a.total || end < 0))
    report(a.status, DFLASH_ERR_DEVICE);
  {
    int bb[2];
    requests_of(a.cu_new, a.B, t0 + warp, t0 + warp + 8, lane, bb[0], bb[1]);
    int pos[2], pg[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = t0 + warp + 8 * k, first = a.cu_new[bb[k]], c = a.ctx_len[bb[k]];
      const long long at = static_cast<long long>(c) + t - first;
      const bool in = first >= 0 && first <= t && c >= 0 && at < static_cast<long long>(a.max_pages) * PAGE;
      pos[k] = in ? static_cast<int>(at) : -1;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      pg[k] = pos[k] >= 0 && warp + 8 * k < nt ? a.page_table[static_cast<size_t>(bb[k]) * a.max_pages + pos[k] / PAGE] : -1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = warp + 8 * k;
      if (j >= nt) continue;
      const bool ok = pg[k] >= 0 && pg[k] < a.num_pages;
      if (lane == 0) {
        if (!ok && j >= j0) report(a.status, DFLASH_ERR_DEVICE);
        s_page[j] = ok ? pg[k] : -1;
        s_pos[j] = max(pos[k], 0);
      }
#pragma unroll
      for (int i = 0; i < HALF / 32; ++i) {
        float co = 1.f, si = 0.f;
        if (a.rotate) rope_cs(max(pos[k], 0), th_hi[i], th_lo[i], co, si);
        const int pair = lane + 32 * i;
        cs[j][((pair >> 1 & 1) * LPR + (pair >> 2)) * 2 + (pair & 1)] = make_float2(co, si);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  if (nt <= 0) return;
  // ---- v heads, transposed into [d][slot] pages.  Consecutive lanes take a
  // d-row's consecutive slots: what costs here is the number of sectors each
  // store instruction touches (lanes along d took 7 times as long)
  {
    const int pg = s_page[0], sl = s_pos[0] % PAGE;
    const bool packed = nt == a.tt && nt >= V16 && pg >= 0 && s_page[nt - 1] == pg && sl % V16 == 0 &&
                        s_pos[nt - 1] % PAGE == sl + nt - 1;
    T *vc = static_cast<T *>(a.v);
    if (packed) {   // the tile is consecutive slots of one page, on 16-byte boundaries
      const int gs = sh - (V16 == 8 ? 3 : 2);   // log2 of a d-row's 16-byte groups
      for (int e = threadIdx.x; e < nh * D << gs; e += THREADS) {
        const int grp = e & ((1 << gs) - 1), d = (e >> gs) % D, h = (e >> gs) / D;
        __align__(16) T w[V16];
#pragma unroll
        for (int i = 0; i < V16; ++i) w[i] = vt[h][grp * V16 + i][d];
        *reinterpret_cast<uint4 *>(vc + ((static_cast<size_t>(pg) * a.nkv + h0 + h) * D + d) * PAGE + sl + grp * V16) =
            *reinterpret_cast<const uint4 *>(w);
      }
    } else {
      for (int e = threadIdx.x; e < nh * D << sh; e += THREADS) {
        const int j = e & ((1 << sh) - 1), d = (e >> sh) % D, h = (e >> sh) / D;
        if (j < nt && s_page[j] >= 0)
          vc[((static_cast<size_t>(s_page[j]) * a.nkv + h0 + h) * D + d) * PAGE + s_pos[j] % PAGE] = vt[h][j][d];
      }
    }
  }
  // ---- q and k heads
  const unsigned mine = max(nt - j0, 0);
  for (int it0 = slot; it0 - slot < items; it0 += ROWS * U) {   // uniform trip count
    if (it0 != slot) load(it0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (it0 - slot + u * ROWS >= items) break;   // uniform
      const int it = it0 + u * ROWS, j = it & ((1 << sh) - 1), hh = it >> sh;
      const bool live = it < items && static_cast<unsigned>(j - j0) < mine, isq = hh < nqh;
      float x[8], y[8];
      F::unpack(raw[u][0], x);
      F::unpack(raw[u][1], x + 4);
      if (a.g_q) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss / D + a.eps);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 w = *reinterpret_cast<const float4 *>(&gains[isq ? 0 : 1][(i >> 2) * HALF + 4 * l]);
          x[i] *= r * w.x, x[i + 1] *= r * w.y, x[i + 2] *= r * w.z, x[i + 3] *= r * w.w;
        }
      }
      const float4 *c4 = reinterpret_cast<const float4 *>(cs[live ? j : 0]);
      const float4 ca = c4[l], cb = c4[LPR + l];
      const float co[4] = {ca.x, ca.z, cb.x, cb.z}, si[4] = {ca.y, ca.w, cb.y, cb.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = fmaf(-si[i], x[4 + i], x[i] * co[i]);
        y[4 + i] = fmaf(si[i], x[i], x[4 + i] * co[i]);
      }
      T *dst = nullptr;
      if (live && isq)
        dst = static_cast<T *>(a.q_out) + (static_cast<size_t>(t0 + j) * a.nq + h0 * a.g + hh) * D;
      else if (live && s_page[j] >= 0)
        dst = static_cast<T *>(a.k) + ((static_cast<size_t>(s_page[j]) * a.nkv + h0 + hh - nqh) * PAGE + s_pos[j] % PAGE) * D;
      if (dst) {
        *reinterpret_cast<typename F::Raw *>(dst + 4 * l) = F::pack(y);
        *reinterpret_cast<typename F::Raw *>(dst + HALF + 4 * l) = F::pack(y + 4);
      }
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
  if (!kv || !kv->k_cache || !kv->v_cache || !workspace ||
      (batch > 0 && (!kv->page_table || !cu_new || !ctx_len)) || (total_new > 0 && batch > 0 && !rows))
    return set_error(DFLASH_ERR_ARG, "%s: null argument", who);
  if (batch < 0 || batch > DFLASH_MAX_BATCH || total_new < 0 || total_new > (1 << 30) || layer < 0)
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
  if (off_words(cu_new, ctx_len, kv->page_table))
    return set_error(DFLASH_ERR_ALIGN, "%s: index arrays must be aligned to their elements", who);
  if (workspace_bytes < need)
    return set_error(DFLASH_ERR_SHAPE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes, need);
  return DFLASH_OK;
}

int current_device(Device *d) {
  static std::atomic<int> known[64] = {};
  if (int e = cuda_check(cudaGetDevice(&d->index), "cudaGetDevice")) return e;
  const bool slot = d->index >= 0 && d->index < 64;
  d->sms = slot ? known[d->index].load(std::memory_order_relaxed) : 0;
  if (d->sms) return DFLASH_OK;
  if (int e = cuda_check(cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->index), "SM count"))
    return e;
  if (slot) known[d->index].store(d->sms, std::memory_order_relaxed);
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
  if (off_words(g_q, g_k)) return set_error(DFLASH_ERR_ALIGN, "append_kv: g_q and g_k must be aligned to their elements");
  if (batch == 0 || total_new == 0) return DFLASH_OK;
  Device dev;
  if (int e = current_device(&dev)) return e;
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
  // as many kv heads per CTA as leave two CTAs per SM, then as many tokens as
  // leave four (64 requests x 16 tokens, 8 kv heads: 10.9 us in 1024 CTAs of 8
  // tokens, 12.8 in 512 of 16; 64 x 1: 4.1 in tiles of 4 tokens, 6.6 of 16)
  a.tt = TT;
  a.hpc = MAX_HPC;
  auto ctas = [&] { return static_cast<long long>((total_new + a.tt - 1) / a.tt) * ((nkv + a.hpc - 1) / a.hpc); };
  while (a.hpc > 1 && ctas() < 2LL * dev.sms) a.hpc /= 2;
  while (a.tt > 4 && ctas() < 4LL * dev.sms) a.tt /= 2;
  const dim3 grid((total_new + a.tt - 1) / a.tt, (nkv + a.hpc - 1) / a.hpc);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RopeArgs &rp = rope_of(d, a.rotate ? rope_base : 1e6f);
  if (hs->dtype == DFLASH_F32)
    launch_pdl(d == 64 ? append_kernel<float, 64> : append_kernel<float, 128>, grid, dim3(THREADS), 0, s, a, rp);
  else
    launch_pdl(d == 64 ? append_kernel<__nv_bfloat16, 64> : append_kernel<__nv_bfloat16, 128>, grid, dim3(THREADS), 0,
               s, a, rp);
  return cuda_check(cudaGetLastError(), "append_kv launch");
}
