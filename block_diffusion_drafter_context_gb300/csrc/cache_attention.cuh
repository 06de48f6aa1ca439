// What the kernels of dflash_cache_attention share: the call's parameters, the
// list of pages they cut into runs, and the join of partial results.
#pragma once

#include "common.cuh"
#include "target.h"

#include <float.h>
#include <math.h>

namespace dflash {

constexpr float LOG2E_F = 1.4426950408889634f, LN2_F = 0.6931471805599453f;
constexpr float RESCALE_LOG2 = 8.f;        // a row's maximum is moved when it grows by more than 2^8
constexpr unsigned long long WAIT_NS = 2000000000ull;
constexpr size_t HEADER_BYTES = 256;
constexpr size_t PART_BYTES = 22u << 20;   // workspace for partials: (max, sum, O) of up to two tiles per CTA
constexpr size_t PART_TOTAL = PART_BYTES / sizeof(float);

struct Params {
  const void *q;
  long long ldq;
  void *out;
  float *lse;
  const void *k, *v;                       // this layer (read through tensor maps)
  const int32_t *page_table, *cu_new, *ctx_len;
  int max_pages, num_pages;
  int B, nkv, g, total, max_new, window;
  int tiles;                               // row tiles of a (request, kv head) at most (bf16: 1)
  int min_chunks;
  int cs;                                  // cluster form: CTAs per tile
  float scale_log2;
  int *counters;
  float *partials;
  int *status;
};

// One request's place: rows row0 .. row0+n-1, ctx tokens before them, pages
// p0 .. p0+np-1 hold every position any of its tokens sees.
struct Req {
  int row0, n, ctx, p0, np;
};

__device__ __forceinline__ Req make_request(const Params &p, int row0, int next, int ctx, bool tell) {
  Req r;
  r.row0 = row0;
  const long long n = static_cast<long long>(next) - row0;
  r.ctx = ctx;
  const bool ok = r.row0 >= 0 && n >= 0 && n <= p.max_new && r.row0 + n <= p.total && r.ctx >= 0 &&
                  r.ctx + n <= static_cast<long long>(p.max_pages) * PAGE;
  if (!ok && tell) report(p.status, DFLASH_ERR_DEVICE);
  r.n = ok ? static_cast<int>(n) : 0;
  r.p0 = 0;
  r.np = 0;
  if (r.n > 0) {
    const int lo = p.window > 0 ? max(0, r.ctx - p.window + 1) : 0;
    r.p0 = lo / PAGE;
    r.np = (r.ctx + r.n - 1) / PAGE - r.p0 + 1;
  }
  return r;
}

__device__ __forceinline__ Req request(const Params &p, int b, bool tell) {
  return make_request(p, p.cu_new[b], p.cu_new[b + 1], p.ctx_len[b], tell);
}
// Pages of requests b0 .. b1-1, each as often as it has row tiles; four
// requests' loads at a time (one by one, 4096 requests took 45 us).
template <typename Tiles>
__device__ __forceinline__ long long sum_pages(const Params &p, int b0, int b1, bool tell, Tiles tiles_of) {
  long long sum = 0;
  for (int b = b0; b < b1; b += 4) {
    int row0[5], ctx[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) row0[i] = p.cu_new[min(b + i, p.B)];
#pragma unroll
    for (int i = 0; i < 4; ++i) ctx[i] = p.ctx_len[min(b + i, p.B - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i < b1) {
        const Req r = make_request(p, row0[i], row0[i + 1], ctx[i], tell);
        sum += static_cast<long long>(r.np) * tiles_of(r);
      }
  }
  return sum;
}

// How the list of `total` pages is shared out: G CTAs take runs of `base` pages,
// the first `rem` of them one more.  64-bit divisions are some 150 cycles
// each, so lists below 2^32 (all but absurd ones) divide in 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}
struct Runs {
  long long total, base;
  int G, rem;
  __device__ __forceinline__ void cut(long long n, int min_chunks, int ctas) {
    total = n;
    const long long want = quotient(n + min_chunks - 1, min_chunks);
    G = static_cast<int>(want < ctas ? (want < 1 ? 1 : want) : ctas);
    base = quotient(n, G);
    rem = static_cast<int>(n - base * G);
  }
  __device__ __forceinline__ long long lo(int c) const { return c * base + min(c, rem); }
  __device__ __forceinline__ int owner(long long x) const {   // the CTA whose run holds page x
    const long long big = rem * (base + 1);
    return static_cast<int>(x < big ? quotient(x, base + 1) : rem + quotient(x - big, base));
  }
};

// What the consumers need to know of a chunk, written by the producer beside
// the chunk's data.
struct Chunk {
  int b, h, rt, page;        // request, kv head, row tile, page of the request
  int row0, n, ctx, flags;   // FIRST / LAST of this CTA's part, BAD page, WHOLE: no other CTA has a part
  int cf, cl, slot0, slot;   // contributors cf..cl; whether cf's part is its first; this part's slot
};
enum { FIRST = 1, LAST = 2, BAD = 4, WHOLE = 8 };

// a number as a type, for lambdas
template <int N>
struct Count {
  static constexpr int value = N;
};

// Where a tile's rows go.  By value: a reference to the kernel's parameters
// would move them out of the constant bank.
struct Dest {
  void *out;
  float *lse;
  int row0, h, nkv, g;     // the request's first row, the kv head
  int base;                // the tile's first query row
};
__device__ __forceinline__ Dest dest_of(const Params &p, int row0, int h, int base = 0) {
  return {p.out, p.lse, row0, h, p.nkv, p.g, base};
}

// A share's maximum as it goes into a join: +inf where its sum is NaN (a NaN
// score; maxima pass over NaN), which makes the joined row NaN too.
__device__ __forceinline__ float join_max(float m, float l) { return l == l ? m : INFINITY; }

// A row's maximum is -inf only where it sees no position; a row that sees some,
// all with scores of -inf (an infinite query, an overflow), has LOWEST.  With a
// sum of 0 the first is out = 0, lse = -inf, the second 0 / 0 = NaN.
constexpr float LOWEST = -FLT_MAX;
__device__ __forceinline__ float inverse_sum(float M, float L) {   // L NaN: so is the row
  return L != 0.f ? 1.f / L : M == -INFINITY ? 0.f : NAN;
}
__device__ __forceinline__ float log_sum(float M, float L) {
  return L != 0.f ? (M + log2f(L)) * LN2_F : M == -INFINITY ? -INFINITY : NAN;
}

// Row `row` of the tile: output columns c4 .. c4 + 3, and its log-sum-exp.
template <typename T, int D>
__device__ __forceinline__ void write_row(const Dest &p, int row, int c4, float4 o, float M, float L) {
  row += p.base;
  const size_t at = static_cast<size_t>(p.row0 + row / p.g) * (p.nkv * p.g) + p.h * p.g + row % p.g;
  const float inv = inverse_sum(M, L);
  T *dst = static_cast<T *>(p.out) + at * D + c4;
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4 *>(dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  else
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (p.lse && c4 == 0) p.lse[at] = log_sum(M, L);
}

// The join of a tile cut over several CTAs, by the last of them to arrive: np
// partials (O [tile_rows][D], maxima [tile_rows], sums [tile_rows], at
// src(0..np-1)), in that order.  The partials sit in L2, so the time is its
// latency: NV float4 columns and B partials per thread are in flight.
template <typename T, int D, int NV, int B, typename Src>
__device__ __forceinline__ void join_tile(const Dest &p, Src src, int np, int tile_rows, int rows, int tid, int nthr) {
  constexpr int PER = D / 4 / NV;   // items per row
  for (int e = tid; e < rows * PER; e += nthr) {
    const int r = e / PER, c = (e % PER) * 4;   // columns c + 4 PER k
    float M = -INFINITY, L = 0.f;
    float4 acc[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < np; i += B) {
      float m[B], l[B];
      float4 v[B][NV];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const float *pp = src(min(i + u, np - 1));
        m[u] = __ldcg(pp + tile_rows * D + r);
        l[u] = __ldcg(pp + tile_rows * D + tile_rows + r);
#pragma unroll
        for (int k = 0; k < NV; ++k) v[u][k] = __ldcg(reinterpret_cast<const float4 *>(pp + r * D + c + 4 * PER * k));
      }
      float mn = M;
#pragma unroll
      for (int u = 0; u < B; ++u) {
        if (i + u >= np) m[u] = -INFINITY;
        mn = fmaxf(mn, m[u]);
      }
      if (mn == -INFINITY) continue;
      const float f = fast_exp2(M - mn);
      M = mn;
      L *= f;
#pragma unroll
      for (int k = 0; k < NV; ++k) acc[k].x *= f, acc[k].y *= f, acc[k].z *= f, acc[k].w *= f;
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const float w = fast_exp2(m[u] - mn);
        L = fmaf(w, l[u], L);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          acc[k].x = fmaf(w, v[u][k].x, acc[k].x);
          acc[k].y = fmaf(w, v[u][k].y, acc[k].y);
          acc[k].z = fmaf(w, v[u][k].z, acc[k].z);
          acc[k].w = fmaf(w, v[u][k].w, acc[k].w);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) write_row<T, D>(p, r, c + 4 * PER * k, acc[k], M, L);
  }
}
// the same for the runs' partials: np contributors from CTA cf on, a tile's
// slot at (CTA * 2 + slot) * stride.  Not inlined: the kernels' main loops have
// no registers to spare for it.
template <typename T, int D>
__device__ __noinline__ void join_parts(Dest p, const float *partials, int cf, int np, int slot0, int stride, int tile_rows,
                                        int rows, int tid, int nthr) {
  auto src = [&](int i) { return partials + (static_cast<size_t>(cf + i) * 2 + (i > 0 || slot0 ? 0 : 1)) * stride; };
  if (rows * (D / 4) <= 2 * nthr)
    join_tile<T, D, 1, 8>(p, src, np, tile_rows, rows, tid, nthr);
  else if (np > 4)
    join_tile<T, D, 4, 8>(p, src, np, tile_rows, rows, tid, nthr);
  else
    join_tile<T, D, 4, 4>(p, src, np, tile_rows, rows, tid, nthr);
}

// 17..128 query rows per (request, kv head) on tcgen05 (cache_attention_tc.cu).
int launch_verify(const dflash_heads &hs, const dflash_kv &kv, Params &p, const Device &dev, cudaStream_t s);

}  // namespace dflash
