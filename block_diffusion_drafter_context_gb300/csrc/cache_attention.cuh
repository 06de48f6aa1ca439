// What the kernels of dflash_cache_attention and dflash_shared_attention share:
// the call's parameters, the list of pages they cut into runs, and the join of
// partial results.
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

// dflash_shared_attention is two launches.  The first takes the prefix that the
// batch shares for one request: its "requests" are runs of `tile_tokens` tokens,
// whosever they are, that see every position of the prefix, and a row's
// (O, maximum, sum) go to `rows`.  The second takes each request's own pages,
// and joins them where it writes a row.  Where the prefix is short, one launch
// reads it once for each request, from the first request's row of the table.
enum Form { PREFIX, OWN, ONE };
struct Prefix {
  float *rows;         // [row_cap][nq][D] O, then [row_cap][nq] (maximum, sum); row 0 is the batch's first
  int row_cap;         // rows a valid batch has at most
  int pages;           // of the prefix
  Form form;
  int tile_tokens;     // PREFIX: tokens per run
  int batch;           // requests (Params.B counts runs in PREFIX)
  int cost;            // of a tile beside its pages, in pages: see Start
};

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
  Prefix pre;                              // dflash_shared_attention
};

// One request's place: rows row0 .. row0+n-1, ctx tokens before them, pages
// p0 .. p0+np-1 hold every position any of its tokens sees.
struct Req {
  int row0, n, ctx, p0, np;
};

// PRE in all of the following: a launch of dflash_shared_attention.
template <bool PRE>
__device__ __forceinline__ Req make_request(const Params &p, int row0, int next, int ctx, bool tell) {
  Req r;
  r.row0 = row0;
  const long long n = static_cast<long long>(next) - row0;
  r.ctx = ctx;
  bool ok = r.row0 >= 0 && n >= 0 && n <= p.max_new && r.row0 + n <= p.total && r.ctx >= 0 &&
            r.ctx + n <= static_cast<long long>(p.max_pages) * PAGE;
  if (PRE) {   // behind the prefix, and among the rows that have a share of it
    const int begin = p.cu_new[0];
    ok = ok && begin >= 0 && row0 >= begin && next - begin <= p.pre.row_cap && (n == 0 || ctx >= p.pre.pages * PAGE);
  }
  if (!ok && tell) report(p.status, DFLASH_ERR_DEVICE);
  r.n = ok ? static_cast<int>(n) : 0;
  r.p0 = 0;
  r.np = 0;
  if (r.n > 0) {
    const int lo = p.window > 0 ? max(0, r.ctx - p.window + 1) : 0;
    r.p0 = !PRE ? lo / PAGE : p.pre.form == OWN ? p.pre.pages : 0;
    r.np = (r.ctx + r.n - 1) / PAGE - r.p0 + 1;
  }
  return r;
}

// Run j of PREFIX: the prefix lies before all of its tokens.
__device__ __forceinline__ Req prefix_run(const Params &p, int j) {
  const int begin = min(max(0, p.cu_new[0]), p.total);
  const int end = min(p.cu_new[p.pre.batch], begin + min(p.total - begin, p.pre.row_cap));   // `rows` holds no more
  Req r;
  r.row0 = begin + j * p.pre.tile_tokens;
  r.n = max(0, min(p.pre.tile_tokens, end - r.row0));
  r.ctx = p.pre.pages * PAGE;
  r.p0 = 0;
  r.np = r.n > 0 ? p.pre.pages : 0;
  return r;
}
template <bool PRE>
__device__ __forceinline__ Req request(const Params &p, int b, bool tell) {
  if (PRE && p.pre.form == PREFIX) return prefix_run(p, b);
  return make_request<PRE>(p, p.cu_new[b], p.cu_new[b + 1], p.ctx_len[b], tell);
}
// page k of request b: the first request's row of the table holds the prefix
template <bool PRE>
__device__ __forceinline__ int page_of(const Params &p, int b, int k) {
  return p.page_table[k + (PRE && k < p.pre.pages ? 0 : static_cast<size_t>(b) * p.max_pages)];
}
// A tile's length in the list that is shared out.
template <bool PRE>
__device__ __forceinline__ long long tile_units(const Params &p, const Req &r) {
  return PRE && r.np > 0 ? r.np + p.pre.cost : r.np;
}
// Pages (and `cost` for each tile that has some) of requests b0 .. b1-1, each as
// often as it has row tiles; four requests' loads at a time (one by one, 4096
// requests took 45 us).
template <bool PRE, typename Tiles>
__device__ __forceinline__ long long sum_pages(const Params &p, int b0, int b1, bool tell, Tiles tiles_of) {
  long long sum = 0;
  if (PRE && p.pre.form == PREFIX) {
    for (int b = b0; b < b1; ++b) {
      const Req r = prefix_run(p, b);
      sum += tile_units<PRE>(p, r) * tiles_of(r);
    }
    return sum;
  }
  for (int b = b0; b < b1; b += 4) {
    int row0[5], ctx[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) row0[i] = p.cu_new[min(b + i, p.B)];
#pragma unroll
    for (int i = 0; i < 4; ++i) ctx[i] = p.ctx_len[min(b + i, p.B - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i < b1) {
        const Req r = make_request<PRE>(p, row0[i], row0[i + 1], ctx[i], tell);
        sum += tile_units<PRE>(p, r) * tiles_of(r);
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

// A CTA's run: n pages, the first of them k of tile (b, h, rt), which begins at x0
// in the list.  Each tile is its pages, behind `cost` units that stand for what
// the tile takes beside them: queries, join, output.  The launch behind a
// prefix has a cost (short own parts: 64 requests of 2..32 pages; without it
// the run with the shortest lists took twice the mean), the others 0.
struct Start {
  long long x0;
  int n, b, h, rt, k;
};
// The lane whose slice b0 .. b1-1 of the requests, at `pre` in the list, holds
// the run's first unit lo.
template <bool PRE, typename Tiles>
__device__ __forceinline__ void find_start(const Params &p, int b0, int b1, long long pre, long long lo, long long hi,
                                           Tiles tiles_of, Start *s) {
  for (int b = b0; b < b1; ++b) {
    Req r = request<PRE>(p, b, false);
    const long long tile = tile_units<PRE>(p, r), head = tile * tiles_of(r), span = head * p.nkv;
    if (lo >= pre + span) {
      pre += span;
      continue;
    }
    const long long h = quotient(lo - pre, head), rt = quotient(lo - pre - h * head, tile), off = lo - pre - h * head - rt * tile;
    const int cost = PRE ? p.pre.cost : 0;
    s->b = b;
    s->h = static_cast<int>(h);
    s->rt = static_cast<int>(rt);
    s->x0 = lo - off;
    s->k = static_cast<int>(off > cost ? off - cost : 0);
    long long n = hi - lo;
    if (PRE && cost > 0) {   // pages alone
      n = 0;
      long long x = lo - off, left = (p.nkv - h) * tiles_of(r) - rt;   // a tile's beginning; tiles of the request from there on
      while (x < hi) {
        const long long t = tile_units<PRE>(p, r), from = x + cost > lo ? x + cost : lo, to = x + t < hi ? x + t : hi;
        if (to > from) n += to - from;
        x += t;
        if (--left == 0 && x < hi) {
          do r = request<PRE>(p, ++b, false);   // another request with work follows
          while (r.np == 0 && b + 1 < p.B);
          left = static_cast<long long>(p.nkv) * tiles_of(r);
        }
      }
    }
    s->n = static_cast<int>(n);
    return;
  }
}

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
  float *share;            // PRE: the prefix's share of the request's first row, its maximum and sum
  float2 *share_ml;
  Form form;               // PRE
};
template <bool PRE>
__device__ __forceinline__ Dest dest_of(const Params &p, int D, int row0, int h, int base = 0) {
  Dest d = {p.out, p.lse, row0, h, p.nkv, p.g, base, nullptr, nullptr, OWN};
  if (PRE) {
    const size_t nq = static_cast<size_t>(p.nkv) * p.g, at = (row0 - max(0, p.cu_new[0])) * nq;
    d.share = p.pre.rows + at * D;
    d.share_ml = reinterpret_cast<float2 *>(p.pre.rows + static_cast<size_t>(p.pre.row_cap) * nq * D) + at;
    d.form = p.pre.form;
  }
  return d;
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

// (M, L) joined with the prefix's share: the factors of both O.  A row of
// nothing (M = -inf) has 0 in both.
struct Join2 {
  float own, pre;
};
__device__ __forceinline__ Join2 join_prefix(float &M, float &L, float2 pre) {
  const float m = fmaxf(M, pre.x);
  Join2 f = {0.f, 0.f};
  if (m != -INFINITY) {
    f.own = fast_exp2(M - m);
    f.pre = fast_exp2(pre.x - m);
  }
  M = m;
  L = f.own * L + f.pre * pre.y;
  return f;
}

// The prefix's share of row `row` of the tile: columns c4 .. c4 + 3, its maximum
// and sum.  Read before the parts that it joins, whose loads do not wait for it.
struct Share {
  float4 o;
  float2 ml;
};
template <int D>
__device__ __forceinline__ size_t share_index(const Dest &p, int row) {
  row += p.base;
  return static_cast<size_t>(row / p.g) * (p.nkv * p.g) + p.h * p.g + row % p.g;
}
template <int D, bool PRE>
__device__ __forceinline__ Share share_of(const Dest &p, int row, int c4) {
  Share s = {make_float4(0.f, 0.f, 0.f, 0.f), make_float2(-INFINITY, 0.f)};
  if (PRE && p.form == OWN) {
    const size_t i = share_index<D>(p, row);
    s.o = __ldcg(reinterpret_cast<const float4 *>(p.share + i * D + c4));
    s.ml = __ldcg(p.share_ml + i);
  }
  return s;
}

// Row `row` of the tile: output columns c4 .. c4 + 3, and its log-sum-exp.
template <typename T, int D, bool PRE>
__device__ __forceinline__ void write_row(const Dest &p, int row, int c4, float4 o, float M, float L, const Share &share) {
  if (PRE) {
    if (p.form == PREFIX) {
      const size_t i = share_index<D>(p, row);
      __stcg(reinterpret_cast<float4 *>(p.share + i * D + c4), o);
      if (c4 == 0) __stcg(p.share_ml + i, make_float2(M, L));
      return;
    }
    const Join2 f = join_prefix(M, L, share.ml);
    o.x = f.own * o.x + f.pre * share.o.x;
    o.y = f.own * o.y + f.pre * share.o.y;
    o.z = f.own * o.z + f.pre * share.o.z;
    o.w = f.own * o.w + f.pre * share.o.w;
  }
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
template <typename T, int D, bool PRE, int NV, int B, typename Src>
__device__ __forceinline__ void join_tile(const Dest &p, Src src, int np, int tile_rows, int rows, int tid, int nthr) {
  constexpr int PER = D / 4 / NV;   // items per row
  for (int e = tid; e < rows * PER; e += nthr) {
    const int r = e / PER, c = (e % PER) * 4;   // columns c + 4 PER k
    Share share[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) share[k] = share_of<D, PRE>(p, r, c + 4 * PER * k);
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
    for (int k = 0; k < NV; ++k) write_row<T, D, PRE>(p, r, c + 4 * PER * k, acc[k], M, L, share[k]);
  }
}
// the same for the runs' partials: np contributors from CTA cf on, a tile's
// slot at (CTA * 2 + slot) * stride.  Not inlined: the kernels' main loops have
// no registers to spare for it.
template <typename T, int D, bool PRE>
__device__ __noinline__ void join_parts(Dest p, const float *partials, int cf, int np, int slot0, int stride, int tile_rows,
                                        int rows, int tid, int nthr) {
  auto src = [&](int i) { return partials + (static_cast<size_t>(cf + i) * 2 + (i > 0 || slot0 ? 0 : 1)) * stride; };
  if (rows * (D / 4) <= 2 * nthr)
    join_tile<T, D, PRE, 1, 8>(p, src, np, tile_rows, rows, tid, nthr);
  else if (np > 4)
    join_tile<T, D, PRE, 4, 8>(p, src, np, tile_rows, rows, tid, nthr);
  else
    join_tile<T, D, PRE, 4, 4>(p, src, np, tile_rows, rows, tid, nthr);
}

// x = hi + lo, hi of 11 significant bits (to nearest, in integer arithmetic:
// the conversion instruction runs at a quarter of its rate); the product reads
// 11 bits of lo
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t &hi, uint32_t &lo) {
  hi = (x + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d += A B from split operands, the small terms in dl (may be d itself).  The
// tensor cores cut their sums off instead of rounding them, so sums that go on
// for long are kept short here and added up outside: with O accumulated over
// all pages the outputs came out 5e-6 too small at 32k positions.
__device__ __forceinline__ void mma_split(float (&d)[4], float (&dl)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                          uint32_t b0, uint32_t b1) {
  uint32_t h0, l0, h1, l1;
  split_tf32(b0, h0, l0);
  split_tf32(b1, h1, l1);
  mma_tf32(dl, al, h0, h1);
  mma_tf32(dl, ah, l0, l1);
  mma_tf32(d, ah, h0, h1);
}

// 17..128 query rows per (request, kv head) on tcgen05 (cache_attention_tc.cu).
// `pages`: the longest list of a (request, kv head) that the call may have.
int launch_verify(const dflash_heads &hs, const dflash_kv &kv, Params &p, int pages, const Device &dev, cudaStream_t s);

// The first launch of dflash_shared_attention, bf16 and more than 16 rows per kv
// head (shared_prefix.cu).  Its partials lie behind the shares in `rows`.
constexpr size_t PREFIX_PART_BYTES = 42u << 20;
int launch_prefix(const dflash_heads &hs, const dflash_kv &kv, const Params &p, const Device &dev, cudaStream_t s);

}  // namespace dflash
