// The prefix's part of dflash_shared_attention for bf16 calls of more than 16
// query rows per kv head, on the 5th-generation tensor cores.
//
// All rows of the batch (token, head of the group) see the same positions, so
// this is a matrix product with a softmax in the middle: 4 d operations per row
// and position on 4 d bytes a position, bound by the tensor cores from some 300
// rows on and by HBM below.  Nothing is masked.
//
// A CTA takes 256 rows as two tiles of 128 (one tensor-memory lane a row) that
// share every K and V^T page of the ring:
//   warps 0-3, 4-7   softmax of tile 0 and 1: one row per thread, online in the
//               exp2 domain, P in bf16 over the page's S;
//   warp 8      feeds the ring by TMA;
//   warps 9, 10   issue the products, one warp for each tile: S = Q K^T of a page
//               into one of two buffers, then O += P V of the page before, so that
//               the next scores are there when a page's probabilities are done.
// Tensor memory is full: two S (64 columns) and an O (128) for each tile; Q lies
// in shared memory.
// For 1024 tokens x 40 heads on 32768 positions (128 positions are 2048 cycles
// of products for both tiles): 850 us with Q in tensor memory, one S and the
// products issued by a thread on a branch of its own; 582 with blocks of 128
// positions; 513 with a converged warp that issues; 475 with two S, which take
// a tile's products out of the chain from its scores to the next ones; 450 with a
// wait for every page's P V (pv_done.h).
//
// Tiles of a (kv head, 256 rows) go out whole while every CTA gets one, in the
// order of the heads, so that the CTAs of a head sweep its pages together and
// L2 serves all but the first; what is left over is cut into equal runs of
// pages, whose (O, maximum, sum) partials a second kernel joins row by row over
// the whole GPU, in the order of the pages: the same bits on every call.
#include "cache_attention.cuh"
#include "pv_done.h"

namespace dflash {
namespace {

constexpr int MROWS = 128, TILE = 2 * MROWS;
constexpr int SOFT = 8, NTHR = 32 * (SOFT + 3);   // softmax warps, then the producer and the MMA issuers
template <int D>
struct PShape {
  static constexpr int SLOT = PAGE * D * 2;                     // K of a page, [D / 64][64][64], or its V^T, [D][64]
  static constexpr int ST = D == 128 ? 10 : 16;                 // ring depth
  static constexpr int QB = MROWS * D * 2;                      // a tile's Q, [D / 64][128][64]
  static constexpr int SMEM = 1024 + ST * SLOT + 2 * QB + 1024;
  static constexpr int PART = TILE * (D + 2);                   // O, then (maximum, sum) of each row
};
constexpr uint32_t S_COL = 0, O_COL = 256;                      // of tile w: + 128 w; S of odd pages: + 64

struct PrefixArgs {
  const __nv_bfloat16 *q;
  long long ldq;
  const int32_t *pages, *cu_new;   // the first request's row of the page table
  Prefix pre;
  int num_pages, total, nkv, g;
  uint32_t over_g;                 // 2^32 / g, rounded up: see token_of
  float scale_log2;
  float *partials;                 // [CTA][2][PART]
  int *status;
};

// r / g for r < 2^20 (65536 tokens of up to 8 heads), g = 1..8: the product is
// off by r times less than 8 / 2^32, below 1 / g.
__device__ __forceinline__ int token_of(const PrefixArgs &a, int r) { return a.g == 1 ? r : static_cast<int>(__umulhi(r, a.over_g)); }

// The rows of the batch and how their tiles go out to the CTAs.
struct Plan {
  int begin, rows;                 // first token; rows per kv head
  int per_head, whole, left;       // tiles of a head; of all that go out whole; that are cut up
  Runs runs;                       // of their pages
  __device__ __forceinline__ void make(const PrefixArgs &a, int ctas) {
    begin = min(max(0, a.cu_new[0]), a.total);
    const int end = min(a.cu_new[a.pre.batch], begin + min(a.total - begin, a.pre.row_cap));   // `rows` holds no more
    rows = max(0, end - begin) * a.g;
    per_head = (rows + TILE - 1) / TILE;
    const int tiles = per_head * a.nkv;
    whole = tiles / ctas * ctas;
    left = tiles - whole;
    runs.cut(static_cast<long long>(left) * a.pre.pages, 2, ctas);
  }
};
// A CTA's segments: its whole tiles, then the stretches of tiles in its run.
struct Seg {
  int tile, page, n;               // pages page .. page + n - 1
  int slot;                        // of the partial; -1: the tile is this CTA's alone
};
struct Segs {
  int c, ctas, at;                 // whole tiles given out so far
  long long x, end;
  __device__ __forceinline__ void start(const Plan &p, int cta, int n_ctas) {
    c = cta, ctas = n_ctas, at = cta;
    const bool in = p.left > 0 && c < p.runs.G;
    x = in ? p.runs.lo(c) : 0;
    end = in ? p.runs.lo(c + 1) : 0;
  }
  __device__ __forceinline__ bool next(const Plan &p, int pages, Seg &s) {
    if (at < p.whole) {
      s = {at, 0, pages, -1};
      at += ctas;
      return true;
    }
    if (x >= end) return false;
    const int t = static_cast<int>(quotient(x, pages));
    const long long x0 = static_cast<long long>(t) * pages;
    s.tile = p.whole + t;
    s.page = static_cast<int>(x - x0);
    s.n = static_cast<int>(min(end - x, x0 + pages - x));
    s.slot = s.n == pages ? -1 : x == p.runs.lo(c) ? 0 : 1;
    x += s.n;
    return true;
  }
};

struct __align__(16) PCtrl {
  uint64_t full[16], empty[16];                    // a slot's data; both tiles' products are done with it
  uint64_t qfull[2], sfull[2][2], pfull[2][2], oempty[2], drain[2];   // [2]: of a tile; [2][2]: and of an S
  uint64_t pdone[2][PV_BARS];                      // P V of a tile's page (pv_done.h)
  uint32_t tmem;
  int abort_flag;
  int bad[16];                                     // the slot's page is not there
};
static_assert(sizeof(PCtrl) <= 1024, "shared memory");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int D>
__global__ void __launch_bounds__(NTHR, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PrefixArgs a) {
  using S = PShape<D>;
  constexpr int ST = S::ST, SLOT = S::SLOT;
  static_assert(S::SMEM <= 232448 && ST <= 16, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sq = ring + ST * SLOT;
  PCtrl *ct = reinterpret_cast<PCtrl *>(sq + 2 * S::QB);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: uniform to the compiler
  volatile int *abort_flag = &ct->abort_flag;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&ct->full[i], 1);
      mbar_init(&ct->empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ct->qfull[i], 4);
      mbar_init(&ct->sfull[i][0], 1);
      mbar_init(&ct->sfull[i][1], 1);
      mbar_init(&ct->pfull[i][0], 4);
      mbar_init(&ct->pfull[i][1], 4);
      for (int k = 0; k < PV_BARS; ++k) mbar_init(&ct->pdone[i][k], 1);
      mbar_init(&ct->oempty[i], 4);
      mbar_init(&ct->drain[i], 1);
    }
    ct->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == SOFT) {
    tmem_alloc(&ct->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ct->tmem;
  pdl_start();
  const int pages = a.pre.pages;
  Plan plan;
  plan.make(a, gridDim.x);
  Segs segs;
  segs.start(plan, blockIdx.x, gridDim.x);
  Seg sg;
  // Whether any of the prefix's pages is missing: only then do the warps ask of each block.
  int missing = 0;
  for (int i = threadIdx.x; i < pages; i += NTHR) {
    const int page = a.pages[i];
    missing |= page < 0 || page >= a.num_pages;
  }
  const bool any_bad = __syncthreads_or(missing) != 0;
  // the rows of tile w of a segment
  auto rows_of = [&](const Seg &s, int w) { return plan.rows - (s.tile % plan.per_head) * TILE - w * MROWS; };

  // A segment's slots in the ring: K of page 0; K of page p, V of page p - 1; V of the last.
  if (warp == SOFT) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bool ok = true;
      int i = 0;
      while (ok && segs.next(plan, pages, sg)) {
        const int h = sg.tile / plan.per_head;
        for (int k = 0; k < 2 * sg.n; ++k, ++i) {
          const bool v = k > 0 && (k == 2 * sg.n - 1 || !(k & 1));
          const int page = a.pages[sg.page + (k == 2 * sg.n - 1 ? sg.n - 1 : v ? k / 2 - 1 : (k + 1) / 2)], st = i % ST;
          const bool bad = page < 0 || page >= a.num_pages;
          ok = mbar_wait(&ct->empty[st], static_cast<uint32_t>(((i / ST) & 1) ^ 1), abort_flag, WAIT_NS);
          if (!ok) break;
          if (bad) report(a.status, DFLASH_ERR_DEVICE);
          ct->bad[st] = bad;
          mbar_arrive_expect_tx(&ct->full[st], bad ? 0 : SLOT);
          if (bad) continue;
          uint8_t *dst = ring + st * SLOT;
          if (v)
            tma_load_2d(dst, &tmV, &ct->full[st], 0, (page * a.nkv + h) * D);
          else
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
              tma_load_2d(dst + half * (PAGE * 128), &tmK, &ct->full[st], half * 64, (page * a.nkv + h) * PAGE);
        }
      }
      if (!ok) {
        report(a.status, DFLASH_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // every issued copy lands before the shared memory goes away
      for (int j = max(0, i - ST); j < i; ++j)
        mbar_wait(&ct->full[j % ST], static_cast<uint32_t>((j / ST) & 1), nullptr, WAIT_NS);
    }
  } else if (warp > SOFT) {
    // ------------------------------------------------------------ MMA issuers
    // the whole warp, converged; one lane of it issues
    constexpr uint32_t idesc_s = idesc_bf16_f32(MROWS, PAGE), idesc_o = idesc_bf16_f32(MROWS, D);
    const int w = warp - SOFT - 1;
    const uint32_t s_col = tmem + S_COL + 128 * w, o_col = tmem + O_COL + 128 * w, q0 = smem_u32(sq + w * S::QB);
    const uint32_t ring0 = smem_u32(ring);
    bool ok = true, any = false;
    int n_tile = 0, n_s = 0, n_p = 0;              // tiles of this half of the CTA, pages' S and P V issued
    int st = 0;                                    // the next slot of the ring, and its parity
    uint32_t ph = 0;
    auto wait = [&](uint64_t *bar, uint32_t n) { return mbar_wait(bar, n & 1, abort_flag, WAIT_NS); };
    auto all = [](bool fine) { return !__any_sync(0xffffffffu, !fine); };
    auto step = [&] {
      if (++st == ST) {
        st = 0;
        ph ^= 1;
      }
    };
    while (ok && segs.next(plan, pages, sg)) {
      if (rows_of(sg, w) <= 0) {                   // the tile is not there: its slots are free as they come
        for (int i = 0; i < 2 * sg.n && ok; ++i, step()) {
          ok = all(wait(&ct->full[st], ph));
          if (ok && lane == 0) mbar_arrive(&ct->empty[st]);
        }
        continue;
      }
      any = true;
      bool started = false;                        // O holds something of the tile
      // S of the next page; one that is not there gives columns that nobody reads
      auto scores = [&] {
        const uint32_t k0 = ring0 + st * SLOT, d = s_col + 64 * (n_s & 1);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_bf16_elect(d, sdesc_k_sw128(q0 + (kk >> 2) * (MROWS * 128) + (kk & 3) * 32),
                          sdesc_k_sw128(k0 + (kk >> 2) * (PAGE * 128) + (kk & 3) * 32), idesc_s, kk > 0 ? 1u : 0u);
        umma_commit_elect(&ct->sfull[w][n_s & 1]);
        umma_commit_elect(&ct->empty[st]);
        ++n_s;
        step();
      };
      if (!(ok = all(wait(&ct->full[st], ph) && wait(&ct->qfull[w], n_tile++)))) break;
      tc_fence_after();
      scores();
      for (int k = 0; k < sg.n; ++k) {             // S of page k + 1, O += P V of page k
        if (k + 1 < sg.n) {                        // its buffer is free: P V of page k - 1 was issued before
          if (!(ok = all(wait(&ct->full[st], ph)))) break;
          tc_fence_after();
          scores();
        }
        ok = wait(&ct->full[st], ph);
        // the first P V of a tile: the O of the tile before has been read
        if (k == 0 && n_tile > 1) ok = ok && wait(&ct->oempty[w], n_tile);
        ok = ok && wait(&ct->pfull[w][n_p & 1], n_p >> 1);
        if (!(ok = all(ok))) break;
        tc_fence_after();
        if (!any_bad || !ct->bad[st]) {
          const uint32_t v0 = ring0 + st * SLOT, p0 = s_col + 64 * (n_p & 1);
#pragma unroll
          for (int kk = 0; kk < PAGE / 16; ++kk)
            umma_bf16_ts_elect(o_col, p0 + static_cast<uint32_t>(kk * 8), sdesc_k_sw128(v0 + kk * 32), idesc_o,
                               kk > 0 || started ? 1u : 0u);
          started = true;
        }
        umma_commit_elect(&ct->pdone[w][pv_bar(n_p)]);
        umma_commit_elect(&ct->empty[st]);
        ++n_p;
        step();
      }
    }
    if (!ok && lane == 0) {
      report(a.status, DFLASH_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    __syncwarp();
    if (any) {
      umma_commit_elect(&ct->drain[w]);   // every issued MMA retires before TMEM is released
      mbar_wait(&ct->drain[w], 0, nullptr, WAIT_NS);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2, quad = warp & 3, row = quad * 32 + lane;   // tile; TMEM lane = query row
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t my_s = lane_base + S_COL + 128 * w, my_o = lane_base + O_COL + 128 * w;
    const int nq = a.nkv * a.g;
    bool ok = true;
    int np = 0;                      // pages this tile had
    float m = -INFINITY, l = 0.f;    // maximum (scaled, log2) and sum of this row
    auto waitw = [&](uint64_t *bar, int n) -> bool {   // warp-uniform bounded wait
      const bool done = mbar_wait(bar, static_cast<uint32_t>(n & 1), abort_flag, WAIT_NS);
      return !__any_sync(0xffffffffu, !done);
    };
    // the first of this warp's 32 rows of a segment, among the rows of its head
    auto first_row = [&](const Seg &s) { return (s.tile % plan.per_head) * TILE + w * MROWS + quad * 32; };
    // This warp's part of the query rows in shared memory: 32 rows of 128 bytes for
    // each 64 dims, 16-byte chunks XORed by the row as TMA would.
    auto q_part = [&](int half) { return sq + w * S::QB + half * (MROWS * 128) + quad * (32 * 128); };
    // Where it pays to be short: code that runs once a tile comes from the
    // instruction memory, 5 us for this with its loops unrolled and g divided by.
    auto load_q = [&](const Seg &s) {   // whole rows, 16 bytes a lane
      constexpr int LPR = D / 8, RPI = 32 / LPR, U = 8;
      const int c = lane % LPR, h = s.tile / plan.per_head;
#pragma unroll 1
      for (int t0 = 0; t0 < 32; t0 += U * RPI) {
        uint4 u[U];
#pragma unroll
        for (int t = 0; t < U; ++t) {
          const int r = first_row(s) + t0 + t * RPI + lane / LPR, tok = token_of(a, r);
          u[t] = make_uint4(0u, 0u, 0u, 0u);
          if (r < plan.rows)
            u[t] = __ldg(reinterpret_cast<const uint4 *>(a.q + (plan.begin + tok) * a.ldq + (h * a.g + r - tok * a.g) * D) + c);
        }
#pragma unroll
        for (int t = 0; t < U; ++t) {
          const int r = t0 + t * RPI + lane / LPR;
          *reinterpret_cast<uint4 *>(q_part(c >> 3) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = u[t];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct->qfull[w]);
    };
    // on to the next segment that has rows for this tile
    auto advance = [&](Seg &s) -> bool {
      while (segs.next(plan, pages, s)) {
        if (rows_of(s, w) > 0) return true;
      }
      return false;
    };
    bool more = advance(sg);
    if (more) load_q(sg);
    while (more && ok) {
      for (int k = 0; k < sg.n; ++k, ++np) {
        const uint32_t sp = my_s + 64 * (np & 1);
        if (!(ok = waitw(&ct->sfull[w][np & 1], np >> 1))) break;
        // no phase of P V goes by unseen: the waits below rest on it (pv_done.h)
        if (np > 1 && !(ok = waitw(&ct->pdone[w][pv_bar(np - 2)], pv_phase(np - 2)))) break;
        tc_fence_after();
        bool bad = false;
        if (any_bad) {
          const int page = a.pages[sg.page + k];
          bad = page < 0 || page >= a.num_pages;
        }
        uint32_t x[4][16];
#pragma unroll
        for (int t = 0; t < 4; ++t) tmem_ld16_nw(sp + 16 * t, x[t]);
        tmem_wait_ld();
        float x0 = -INFINITY, x1 = x0, x2 = x0, x3 = x0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          tmem_regs_ready(x[t]);
          if (any_bad)   // what a page that is not there left in its columns
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (bad) x[t][e] = __float_as_uint(-INFINITY);
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            x0 = max3(x0, __uint_as_float(x[t][e]), __uint_as_float(x[t][e + 1]));
            x1 = max3(x1, __uint_as_float(x[t][e + 2]), __uint_as_float(x[t][e + 3]));
            x2 = max3(x2, __uint_as_float(x[t][e + 4]), __uint_as_float(x[t][e + 5]));
            x3 = max3(x3, __uint_as_float(x[t][e + 6]), __uint_as_float(x[t][e + 7]));
          }
        }
        const float mx = fmaxf(fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) * a.scale_log2, bad ? -INFINITY : LOWEST);
        const bool need = mx > m + RESCALE_LOG2;
        if (k == 0) {
          m = mx;
          l = 0.f;
        } else if (__any_sync(0xffffffffu, need)) {   // wait for the P V of the page before, rescale O in TMEM
          if (!(ok = waitw(&ct->pdone[w][pv_bar(np - 1)], pv_phase(np - 1)))) break;
          tc_fence_after();
          const float f = need ? fast_exp2(m - mx) : 1.f;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t ov[16];
            tmem_ld16_nw(my_o + c0, ov);
            tmem_wait_ld();
            tmem_regs_ready(ov);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
            tmem_st16_nw(my_o + c0, ov);
          }
          tmem_wait_st();
          if (need) {
            l *= f;
            m = mx;
          }
        }
        // P, rounded to bf16, over the page's S; the sum keeps fp32
        const float nm = m == -INFINITY ? 0.f : -m;
        const uint64_t sc2 = pair(a.scale_log2, a.scale_log2), nm2 = pair(nm, nm);
        uint64_t sum0 = pair(0.f, 0.f), sum1 = sum0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const uint32_t *y = &x[2 * c + (e >> 4)][e & 15];
            const float2 y0 = unpair(fma2(pair(__uint_as_float(y[0]), __uint_as_float(y[1])), sc2, nm2));
            const float2 y1 = unpair(fma2(pair(__uint_as_float(y[2]), __uint_as_float(y[3])), sc2, nm2));
            const float p0 = fast_exp2(y0.x), p1 = fast_exp2(y0.y), p2 = fast_exp2(y1.x), p3 = fast_exp2(y1.y);
            sum0 = add2(sum0, pair(p0, p1));
            sum1 = add2(sum1, pair(p2, p3));
            pk[e >> 1] = pack_bf16(p0, p1);
            pk[(e >> 1) + 1] = pack_bf16(p2, p3);
          }
          tmem_st16_nw(sp + 16 * c, pk);
        }
        const float2 s0 = unpair(add2(sum0, sum1));
        l += s0.x + s0.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct->pfull[w][np & 1]);
      }
      if (!ok) break;
      // ---- the tile's rows, as shares or partials, through this warp's part of
      // the query rows (the last S of the tile is complete, so they are not needed
      // any more): 32 rows straight from their threads took 4 us of stores a tile
      const Seg last = sg;
      if (!(ok = waitw(&ct->pdone[w][pv_bar(np - 1)], pv_phase(np - 1)))) break;   // and with it every P V before
      tc_fence_after();
      const int head = last.tile / plan.per_head * a.g;
      float *part = last.slot < 0 ? nullptr : a.partials + (static_cast<size_t>(blockIdx.x) * 2 + last.slot) * S::PART;
      auto place = [&](int rr) -> size_t {           // of row rr of the warp's 32 among the shares
        const int r = first_row(last) + rr, tok = token_of(a, r);
        return static_cast<size_t>(tok) * nq + head + r - tok * a.g;
      };
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint8_t *stage = q_part(c0 / 32 % (D / 64));
#pragma unroll
        for (int u = 0; u < 32; u += 16) {
          uint32_t ov[16];
          tmem_ld16_nw(my_o + c0 + u, ov);
          tmem_wait_ld();
          tmem_regs_ready(ov);
#pragma unroll
          for (int t = 0; t < 4; ++t) {            // sum 0: O may never have been written
            uint4 v = make_uint4(ov[4 * t], ov[4 * t + 1], ov[4 * t + 2], ov[4 * t + 3]);
            if (l == 0.f) v = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(stage + lane * 128 + (((u / 4 + t) ^ (lane & 7)) << 4)) = v;
          }
        }
        __syncwarp();
#pragma unroll 4
        for (int t = 0; t < 8; ++t) {
          const int rr = 4 * t + (lane >> 3), c = lane & 7;
          const uint4 v = *reinterpret_cast<const uint4 *>(stage + rr * 128 + ((c ^ (rr & 7)) << 4));
          float *dst = part ? part + (w * MROWS + quad * 32 + rr) * D : a.pre.rows + place(rr) * D;
          if (first_row(last) + rr < plan.rows) __stcg(reinterpret_cast<uint4 *>(dst + c0 + 4 * c), v);
        }
        __syncwarp();
      }
      if (first_row(last) + lane < plan.rows) {
        float *ml = part ? part + TILE * D + 2 * (w * MROWS + row)
                         : a.pre.rows + static_cast<size_t>(a.pre.row_cap) * nq * D + 2 * place(lane);
        __stcg(reinterpret_cast<float2 *>(ml), make_float2(join_max(m, l), l));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct->oempty[w]);
      more = advance(sg);
      if (more) load_q(sg);
    }
    if (!ok) {
      report(a.status, DFLASH_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == SOFT) tmem_dealloc(tmem, 512);
}

// The rows of the tiles that were cut up: D / 4 threads a row, the partials of
// up to 8 CTAs in flight.
constexpr int JOIN_THREADS = 256;
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) prefix_join_kernel(const PrefixArgs a, int ctas) {
  constexpr int PER = D / 4, ROWS = JOIN_THREADS / PER, PART = PShape<D>::PART;
  pdl_start();
  Plan plan;
  plan.make(a, ctas);
  const int item = blockIdx.x * ROWS + threadIdx.x / PER, c4 = threadIdx.x % PER * 4;
  const int t = item / TILE, tr = item % TILE, tile = plan.whole + t;
  if (t >= plan.left) return;
  const int h = tile / plan.per_head, r = (tile % plan.per_head) * TILE + tr, nq = a.nkv * a.g, pages = a.pre.pages;
  const long long x0 = static_cast<long long>(t) * pages;
  const int cf = plan.runs.owner(x0), np = plan.runs.owner(x0 + pages - 1) - cf + 1;
  if (r >= plan.rows || np == 1) return;     // one CTA: it wrote the share itself
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < np; i += 8) {
    float2 ml[8];
    float4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = cf + min(i + u, np - 1);
      const float *part = a.partials + (static_cast<size_t>(c) * 2 + (plan.runs.lo(c) < x0 ? 1 : 0)) * PART;
      ml[u] = __ldcg(reinterpret_cast<const float2 *>(part + TILE * D) + tr);
      v[u] = __ldcg(reinterpret_cast<const float4 *>(part + tr * D + c4));
    }
    float mn = M;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (i + u >= np) ml[u] = make_float2(-INFINITY, 0.f);
      mn = fmaxf(mn, ml[u].x);
    }
    if (mn == -INFINITY) continue;
    const float f = fast_exp2(M - mn);
    M = mn;
    L *= f;
    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float e = fast_exp2(ml[u].x - mn);
      L = fmaf(e, ml[u].y, L);
      acc.x = fmaf(e, v[u].x, acc.x);
      acc.y = fmaf(e, v[u].y, acc.y);
      acc.z = fmaf(e, v[u].z, acc.z);
      acc.w = fmaf(e, v[u].w, acc.w);
    }
  }
  const int tok = token_of(a, r);
  const size_t at = static_cast<size_t>(tok) * nq + h * a.g + r - tok * a.g;
  __stcg(reinterpret_cast<float4 *>(a.pre.rows + at * D + c4), acc);
  if (c4 == 0) __stcg(reinterpret_cast<float2 *>(a.pre.rows + static_cast<size_t>(a.pre.row_cap) * nq * D) + at, make_float2(M, L));
}

template <int D>
int launch(const dflash_heads &hs, const dflash_kv &kv, const Params &p, const Device &dev, cudaStream_t s) {
  using S = PShape<D>;
  auto *kernel = prefix_kernel<D>;
  static std::atomic<uint64_t> smem_set;
  if (int e = allow_smem(smem_set, dev, kernel, S::SMEM)) return e;
  const uint64_t pages = static_cast<uint64_t>(kv.num_pages) * hs.n_kv_heads;
  CUtensorMap tk, tv;
  if (int e = make_tmap_2d(&tk, p.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, D, pages * PAGE, D * 2, 64, PAGE)) return e;
  if (int e = make_tmap_2d(&tv, p.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, PAGE, pages * D, PAGE * 2, 64, D)) return e;
  PrefixArgs a = {};
  a.q = static_cast<const __nv_bfloat16 *>(p.q);
  a.ldq = p.ldq;
  a.pages = p.page_table;
  a.cu_new = p.cu_new;
  a.pre = p.pre;
  a.num_pages = p.num_pages;
  a.total = p.total;
  a.nkv = p.nkv;
  a.g = p.g;
  a.over_g = static_cast<uint32_t>((0x100000000ull + p.g - 1) / p.g);
  a.scale_log2 = p.scale_log2;
  a.status = p.status;
  const size_t nq = static_cast<size_t>(p.nkv) * p.g;
  a.partials = p.pre.rows + (p.pre.row_cap * nq * (D + 2) + 3) / 4 * 4;
  const int most = static_cast<int>(PREFIX_PART_BYTES / (2 * S::PART * sizeof(float))), ctas = dev.sms < most ? dev.sms : most;
  if (int e = cuda_check(launch_pdl(kernel, dim3(ctas), dim3(NTHR), S::SMEM, s, tk, tv, a), "shared_attention launch")) return e;
  // as many tiles as may be left over
  const long long tiles = (static_cast<long long>(p.pre.row_cap) * p.g + TILE - 1) / TILE * p.nkv;
  const int rows = static_cast<int>(tiles < ctas ? tiles : ctas - 1) * TILE, per = JOIN_THREADS / (D / 4);
  return cuda_check(launch_pdl(prefix_join_kernel<D>, dim3(rows / per), dim3(JOIN_THREADS), 0, s, a, ctas),
                    "shared_attention join launch");
}

}  // namespace

int launch_prefix(const dflash_heads &hs, const dflash_kv &kv, const Params &p, const Device &dev, cudaStream_t s) {
  return hs.head_dim == 64 ? launch<64>(hs, kv, p, dev, s) : launch<128>(hs, kv, p, dev, s);
}

}  // namespace dflash
