// What the kernels of dflash_cache_attention share: the call's parameters, the
// list of pages they cut into runs, and the join of partial results.
#pragma once

#include "common.cuh"
#include "target.h"

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
  const void *k, *v;                       // this layer (fp32 path; the bf16 path goes through tensor maps)
  const int32_t *page_table, *cu_new, *ctx_len;
  int max_pages, num_pages;
  int B, nkv, g, total, max_new, window;
  int tiles;                               // row tiles of a (request, kv head) at most: counter stride
  int min_chunks;
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

__device__ __forceinline__ Req request(const Params &p, int b, bool tell) {
  Req r;
  r.row0 = p.cu_new[b];
  const long long n = static_cast<long long>(p.cu_new[b + 1]) - r.row0;
  r.ctx = p.ctx_len[b];
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

// the runs: CTA c of G takes list positions [run_lo(c), run_lo(c + 1))
__device__ __forceinline__ long long run_lo(int c, long long total, int G) {
  return static_cast<long long>(c) * total / G;
}
__device__ __forceinline__ int run_owner(long long x, long long total, int G) {
  return static_cast<int>(((x + 1) * G + total - 1) / total) - 1;
}

// What the consumers need to know of a chunk, written by the producer beside
// the chunk's data.
struct Chunk {
  int b, h, rt, page;        // request, kv head, row tile, page of the request
  int row0, n, ctx, flags;   // FIRST / LAST of this CTA's part, BAD page, WHOLE: no other CTA has a part
  int cf, cl, slot0, slot;   // contributors cf..cl; whether cf's part is its first; this part's slot
  int nrow0, nn, nh, pad;    // the tile after this one, where this CTA has a part of it: its rows and kv head (nn 0: none)
};
enum { FIRST = 1, LAST = 2, BAD = 4, WHOLE = 8 };


// The partials of one tile: O rows [rows][D], maxima [rows], sums [rows], a
// tile's slot at (CTA * 2 + slot) * stride.  The last contributor to arrive
// joins contributors c.cf..c.cl in order and writes rows 0..rows-1 (of the
// tile starting at query row row_base); `tid` of `nthr` threads.
template <int D>
__device__ __forceinline__ void join_parts(const Params &p, const Chunk &c, int stride, int tile_rows, int rows,
                                           int row_base, int tid, int nthr) {
  auto src = [&](int cc) -> const float * {
    return p.partials + (static_cast<size_t>(cc) * 2 + (cc > c.cf || c.slot0 ? 0 : 1)) * stride;
  };
  for (int e = tid; e < rows * (D / 4); e += nthr) {
    const int r = e / (D / 4), c4 = (e % (D / 4)) * 4;
    float M = -INFINITY, L = 0.f;
#pragma unroll 8
    for (int cc = c.cf; cc <= c.cl; ++cc) M = fmaxf(M, __ldcg(src(cc) + tile_rows * D + r));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int cc = c.cf; cc <= c.cl; ++cc) {
      const float *pp = src(cc);
      const float mw = __ldcg(pp + tile_rows * D + r), lw = __ldcg(pp + tile_rows * D + tile_rows + r);
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(pp + r * D + c4));
      const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
      L = fmaf(f, lw, L);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    const int row = row_base + r, tok = c.row0 + row / p.g, hq = c.h * p.g + row % p.g;
    const float inv = L > 0.f ? 1.f / L : 0.f;
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) +
                               (static_cast<size_t>(tok) * (p.nkv * p.g) + hq) * D + c4) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (p.lse && c4 == 0)
      p.lse[static_cast<size_t>(tok) * (p.nkv * p.g) + hq] = L > 0.f ? (M + log2f(L)) * LN2_F : -INFINITY;
  }
}

// Query rows > 32 per (request, kv head) on tcgen05 (cache_attention_tc.cu).
int launch_verify(const dflash_heads &hs, const dflash_kv &kv, Params &p, const Device &dev, cudaStream_t s);

}  // namespace dflash
