// The prefix's part of dflash_shared_attention for bf16 calls of more than 16
// query rows per kv head, on the 5th-generation tensor cores.
//
// All rows of the batch (token, head of the group) see the same positions, so
// this is a matrix product with a softmax in the middle: 4 d operations per row
// and position on 4 d bytes a position, bound by the tensor cores from some 300
// rows on and by HBM below.  Nothing is masked.
//
// A CTA takes 256 rows as two tiles of 128 (one tensor-memory lane a row) that
// share every block of 128 positions (two pages) in the ring:
//   warp 0      feeds the ring by TMA, a block's K, then its V^T;
//   warp 1      issues, block by block, for each tile O += P V of the block before
//               and S = Q K^T of this one, so that one tile's products run while
//               the other's scores turn into probabilities;
//   warps 4-7, 8-11   softmax of tile 0 and 1: one row per thread, online in the
//               exp2 domain, P in bf16 over the block's S.
// Tensor memory is full: S (128 columns) and O (128) twice; Q lies in shared
// memory.  At 64 positions a block, Q in tensor memory, a block's fixed times
// (barriers, loads, votes) were as long as its work: 1024 tokens x 40 heads on
// 32768 positions took 850 us.
//
// Tiles of a (kv head, 256 rows) go out whole while every CTA gets one, in the
// order of the heads, so that the CTAs of a head sweep its pages together and
// L2 serves all but the first; what is left over is cut into equal runs of
// pages, whose (O, maximum, sum) partials a second kernel joins row by row over
// the whole GPU, in the order of the pages: the same bits on every call.
#include "cache_attention.cuh"

namespace dflash {
namespace {

constexpr int MROWS = 128, TILE = 2 * MROWS;
constexpr int NTHR = 384;
template <int D>
struct PShape {
  static constexpr int SLOT = 2 * PAGE * D * 2;                 // K of two pages, [D / 64][128][64], or their V^T, [2][D][64]
  static constexpr int ST = D == 128 ? 5 : 10;                  // ring depth
  static constexpr int QB = MROWS * D * 2;                      // a tile's Q, [D / 64][128][64]
  static constexpr int SMEM = 1024 + ST * SLOT + 2 * QB + 1024;
  static constexpr int PART = TILE * (D + 2);                   // O, then (maximum, sum) of each row
};
constexpr uint32_t S_COL = 0, O_COL = 256;                      // of tile w: + 128 w

struct PrefixArgs {
  const __nv_bfloat16 *q;
  long long ldq;
  const int32_t *pages, *cu_new;   // the first request's row of the page table
  Prefix pre;
  int num_pages, total, nkv, g;
  float scale_log2;
  float *partials;                 // [CTA][2][PART]
  int *status;
};

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
  uint64_t full[10], empty[10];                    // a slot's data; its last reader (the second tile's product) is done
  uint64_t qfull[2], sfull[2], pfull[2], pdone[2], oempty[2], drain;   // [2]: of a tile
  uint32_t tmem;
  int abort_flag;
  int bad[10];                                     // pages of the slot that are not there, a bit each
};
static_assert(sizeof(PCtrl) <= 1024, "shared memory");

// packed pairs of fp32
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int D>
__global__ void __launch_bounds__(NTHR, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PrefixArgs a) {
  using S = PShape<D>;
  constexpr int ST = S::ST, SLOT = S::SLOT;
  static_assert(S::SMEM <= 232448 && ST <= 10, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sq = ring + ST * SLOT;
  PCtrl *ct = reinterpret_cast<PCtrl *>(sq + 2 * S::QB);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort_flag = &ct->abort_flag;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&ct->full[i], 1);
      mbar_init(&ct->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ct->qfull[i], 4);
      mbar_init(&ct->sfull[i], 1);
      mbar_init(&ct->pfull[i], 4);
      mbar_init(&ct->pdone[i], 1);
      mbar_init(&ct->oempty[i], 4);
    }
    mbar_init(&ct->drain, 1);
    ct->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
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
  // the rows of tile w of a segment; its blocks of two pages (the last one may have one)
  auto rows_of = [&](const Seg &s, int w) { return plan.rows - (s.tile % plan.per_head) * TILE - w * MROWS; };
  auto blocks_of = [](const Seg &s) { return (s.n + 1) / 2; };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bool ok = true;
      int i = 0;                   // slots: K of block j is 2 j, V 2 j + 1
      while (ok && segs.next(plan, pages, sg)) {
        const int h = sg.tile / plan.per_head;
        for (int k = 0; k < blocks_of(sg) && ok; ++k) {
          const int have = min(2, sg.n - 2 * k);
          int page[2], bad = have < 2 ? 2 : 0;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            page[u] = u < have ? a.pages[sg.page + 2 * k + u] : 0;
            if (page[u] < 0 || page[u] >= a.num_pages) {
              bad |= 1 << u;
              report(a.status, DFLASH_ERR_DEVICE);
            }
          }
          for (int v = 0; v < 2; ++v, ++i) {
            const int st = i % ST;
            ok = mbar_wait(&ct->empty[st], static_cast<uint32_t>(((i / ST) & 1) ^ 1), abort_flag, WAIT_NS);
            if (!ok) break;
            ct->bad[st] = bad;
            mbar_arrive_expect_tx(&ct->full[st], (2 - __popc(bad)) * (SLOT / 2));
            uint8_t *dst = ring + st * SLOT;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (bad >> u & 1) continue;
              if (v)
                tma_load_2d(dst + u * (SLOT / 2), &tmV, &ct->full[st], 0, (page[u] * a.nkv + h) * D);
              else
#pragma unroll
                for (int half = 0; half < D / 64; ++half)
                  tma_load_2d(dst + half * (MROWS * 128) + u * (PAGE * 128), &tmK, &ct->full[st], half * 64,
                              (page[u] * a.nkv + h) * PAGE);
            }
          }
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
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(MROWS, 2 * PAGE), idesc_o = idesc_bf16_f32(MROWS, D);
      bool ok = true, any = false;
      int j = 0;                                     // block of the CTA
      int n_tile[2] = {0, 0}, n_block[2] = {0, 0};   // tiles and blocks a tile of the CTA had
      bool started[2] = {false, false};              // O holds something of the tile
      auto wait = [&](uint64_t *bar, int n) { return mbar_wait(bar, static_cast<uint32_t>(n & 1), abort_flag, WAIT_NS); };
      // O += P V of block b of the CTA
      auto pv = [&](int w, int b, bool frees) -> bool {
        const int i = 2 * b + 1, st = i % ST;
        if (!wait(&ct->full[st], i / ST) || !wait(&ct->pfull[w], n_block[w] - 1)) return false;
        tc_fence_after();
        const int bad = ct->bad[st];
        const uint32_t pt = tmem + S_COL + 128 * w, v0 = smem_u32(ring + st * SLOT);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (bad >> u & 1) continue;
#pragma unroll
          for (int kk = 0; kk < PAGE / 16; ++kk)
            umma_bf16_ts(tmem + O_COL + 128 * w, pt + static_cast<uint32_t>(32 * u + kk * 8),
                         sdesc_k_sw128(v0 + u * (SLOT / 2) + kk * 32), idesc_o, kk > 0 || started[w] ? 1u : 0u);
          started[w] = true;
        }
        umma_commit(&ct->pdone[w]);
        if (frees) umma_commit(&ct->empty[st]);
        return true;
      };
      // S = Q K^T of block b; a page that is not there gives columns that nobody reads
      auto qk = [&](int w, int b, bool frees) {
        const int st = 2 * b % ST;
        const uint32_t k0 = smem_u32(ring + st * SLOT), q0 = smem_u32(sq + w * S::QB);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_bf16(tmem + S_COL + 128 * w, sdesc_k_sw128(q0 + (kk >> 2) * (MROWS * 128) + (kk & 3) * 32),
                    sdesc_k_sw128(k0 + (kk >> 2) * (MROWS * 128) + (kk & 3) * 32), idesc_s, kk > 0 ? 1u : 0u);
        umma_commit(&ct->sfull[w]);
        if (frees) umma_commit(&ct->empty[st]);
        ++n_block[w];
      };
      while (ok && segs.next(plan, pages, sg)) {
        const int both = rows_of(sg, 1) > 0 ? 2 : 1, blocks = blocks_of(sg);
        any = true;
        for (int k = 0; k <= blocks && ok; ++k) {    // the scores of block k, and P V of the block before
          if (k < blocks) ok = wait(&ct->full[2 * j % ST], 2 * j / ST);
          for (int w = 0; w < both && ok; ++w) {
            if (k == 1) {                            // the tile's first P V: the O of the tile before has been read
              started[w] = false;
              if (n_tile[w]++ > 0) ok = wait(&ct->oempty[w], n_tile[w]);
            }
            if (ok && k > 0) ok = pv(w, j - 1, w == both - 1);
            if (ok && k == 0) ok = wait(&ct->qfull[w], n_tile[w]);   // the first S of a tile wants its query rows
            if (ok && k < blocks) qk(w, j, w == both - 1);
          }
          if (k < blocks) ++j;
        }
      }
      if (!ok) {
        report(a.status, DFLASH_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (any) {
        umma_commit(&ct->drain);   // every issued MMA retires before TMEM is released
        mbar_wait(&ct->drain, 0, nullptr, WAIT_NS);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int w = (warp >> 2) - 1, quad = warp & 3, row = quad * 32 + lane;   // TMEM lane = query row
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t my_s = lane_base + S_COL + 128 * w, my_o = lane_base + O_COL + 128 * w;
    const int nq = a.nkv * a.g;
    bool ok = true;
    int nb = 0, j = 0;               // blocks this tile had; block of the CTA
    float m = -INFINITY, l = 0.f;    // maximum (scaled, log2) and sum of this row
    auto waitw = [&](uint64_t *bar, int n) -> bool {   // warp-uniform bounded wait
      const bool done = mbar_wait(bar, static_cast<uint32_t>(n & 1), abort_flag, WAIT_NS);
      return !__any_sync(0xffffffffu, !done);
    };
    // this row's query into shared memory, 16-byte chunks XORed by the row as TMA would
    auto load_q = [&](const Seg &s) {
      const int r = (s.tile % plan.per_head) * TILE + w * MROWS + row;
      const bool live = r < plan.rows;
      const uint4 *src = reinterpret_cast<const uint4 *>(a.q + static_cast<size_t>(plan.begin + (live ? r / a.g : 0)) * a.ldq +
                                                         static_cast<size_t>(s.tile / plan.per_head * a.g + r % a.g) * D);
      uint4 u[D / 8];
#pragma unroll
      for (int t = 0; t < D / 8; ++t) u[t] = live ? __ldg(src + t) : make_uint4(0u, 0u, 0u, 0u);
      uint8_t *dst = sq + w * S::QB + row * 128;
#pragma unroll
      for (int t = 0; t < D / 8; ++t)
        *reinterpret_cast<uint4 *>(dst + (t >> 3) * (MROWS * 128) + (((t & 7) ^ (row & 7)) << 4)) = u[t];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct->qfull[w]);
    };
    // on to the next segment that has rows for this tile; j moves past the others' blocks
    auto advance = [&](Seg &s) -> bool {
      while (segs.next(plan, pages, s)) {
        if (rows_of(s, w) > 0) return true;
        j += blocks_of(s);
      }
      return false;
    };
    bool more = advance(sg);
    if (more) load_q(sg);
    while (more && ok) {
      const int blocks = blocks_of(sg);
      for (int k = 0; k < blocks; ++k, ++j, ++nb) {
        // V's slot and its `bad` stay until this block's P V
        const int vs = (2 * j + 1) % ST;
        if (!(ok = waitw(&ct->sfull[w], nb) && waitw(&ct->full[vs], (2 * j + 1) / ST))) break;
        tc_fence_after();
        const int bad = ct->bad[vs];
        // ---- the row's maximum over the block
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (bad >> c & 1) continue;
          uint32_t r[4][16];
#pragma unroll
          for (int t = 0; t < 4; ++t) tmem_ld16_nw(my_s + 64 * c + 16 * t, r[t]);
          tmem_wait_ld();
          float x0 = -INFINITY, x1 = x0, x2 = x0, x3 = x0;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            tmem_regs_ready(r[t]);
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              x0 = fmaxf(fmaxf(x0, __uint_as_float(r[t][e])), __uint_as_float(r[t][e + 1]));
              x1 = fmaxf(fmaxf(x1, __uint_as_float(r[t][e + 2])), __uint_as_float(r[t][e + 3]));
              x2 = fmaxf(fmaxf(x2, __uint_as_float(r[t][e + 4])), __uint_as_float(r[t][e + 5]));
              x3 = fmaxf(fmaxf(x3, __uint_as_float(r[t][e + 6])), __uint_as_float(r[t][e + 7]));
            }
          }
          mx = fmaxf(mx, fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)));
        }
        mx = fmaxf(mx * a.scale_log2, bad == 3 ? -INFINITY : LOWEST);
        if (k == 0) {
          m = mx;
          l = 0.f;
        } else {
          const bool need = mx > m + RESCALE_LOG2;
          if (__any_sync(0xffffffffu, need)) {   // wait for the P V of the block before, rescale O in TMEM
            if (!(ok = waitw(&ct->pdone[w], nb - 1))) break;
            tc_fence_after();
            const float f = need ? fast_exp2(m - mx) : 1.f;
#pragma unroll
            for (int c0 = 0; c0 < D / 16; c0 += 2) {
              uint32_t ov[2][16];
#pragma unroll
              for (int u = 0; u < 2; ++u) tmem_ld16_nw(my_o + (c0 + u) * 16, ov[u]);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                tmem_regs_ready(ov[u]);
#pragma unroll
                for (int e = 0; e < 16; ++e) ov[u][e] = __float_as_uint(__uint_as_float(ov[u][e]) * f);
                tmem_st16_nw(my_o + (c0 + u) * 16, ov[u]);
              }
            }
            tmem_wait_st();
            if (need) {
              l *= f;
              m = mx;
            }
          }
        }
        // ---- P over the block's S, rounded to bf16; the sum keeps fp32.  32
        // columns at a time, read again; their P takes the first half of the columns read before.
        const float nm = m == -INFINITY ? 0.f : -m;
        const uint64_t sc2 = pair(a.scale_log2, a.scale_log2), nm2 = pair(nm, nm);
        uint64_t sum0 = pair(0.f, 0.f), sum1 = sum0;
        uint32_t r[2][2][16];
        tmem_ld16_nw(my_s, r[0][0]);
        tmem_ld16_nw(my_s + 16, r[0][1]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c == 2 && (bad & 2)) break;        // the second page is not there: no P V reads it
          tmem_wait_ld();
          tmem_regs_ready(r[c & 1][0]);
          tmem_regs_ready(r[c & 1][1]);
          if (c < 3 && !(c == 1 && (bad & 2))) {
            tmem_ld16_nw(my_s + 32 * (c + 1), r[(c + 1) & 1][0]);
            tmem_ld16_nw(my_s + 32 * (c + 1) + 16, r[(c + 1) & 1][1]);
          }
          if (c < 2 && (bad & 1)) continue;
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const uint32_t *x = &r[c & 1][e >> 4][e & 15];
            const float2 y0 = unpair(fma2(pair(__uint_as_float(x[0]), __uint_as_float(x[1])), sc2, nm2));
            const float2 y1 = unpair(fma2(pair(__uint_as_float(x[2]), __uint_as_float(x[3])), sc2, nm2));
            const float p0 = fast_exp2(y0.x), p1 = fast_exp2(y0.y), p2 = fast_exp2(y1.x), p3 = fast_exp2(y1.y);
            sum0 = add2(sum0, pair(p0, p1));
            sum1 = add2(sum1, pair(p2, p3));
            pk[e >> 1] = pack_bf16(p0, p1);
            pk[(e >> 1) + 1] = pack_bf16(p2, p3);
          }
          tmem_st16_nw(my_s + 16 * c, pk);
        }
        const float2 s0 = unpair(add2(sum0, sum1));
        l += s0.x + s0.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct->pfull[w]);
      }
      if (!ok) break;
      const Seg last = sg;
      const int r = (last.tile % plan.per_head) * TILE + w * MROWS + row;
      more = advance(sg);
      if (more) load_q(sg);      // the last S of this tile is complete: its query rows are not needed any more
      // ---- the tile's row, as a share or a partial
      if (!(ok = waitw(&ct->pdone[w], nb - 1))) break;
      tc_fence_after();
      const bool live = r < plan.rows;
      const size_t at = static_cast<size_t>(live ? r / a.g : 0) * nq + last.tile / plan.per_head * a.g + r % a.g;
      float *dst, *ml;
      if (last.slot < 0) {
        dst = a.pre.rows + at * D;
        ml = a.pre.rows + static_cast<size_t>(a.pre.row_cap) * nq * D + 2 * at;
      } else {
        float *part = a.partials + (static_cast<size_t>(blockIdx.x) * 2 + last.slot) * S::PART;
        dst = part + (w * MROWS + row) * D;
        ml = part + TILE * D + 2 * (w * MROWS + row);
      }
#pragma unroll
      for (int c0 = 0; c0 < D / 16; c0 += 2) {
        uint32_t ov[2][16];
#pragma unroll
        for (int u = 0; u < 2; ++u) tmem_ld16_nw(my_o + (c0 + u) * 16, ov[u]);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          tmem_regs_ready(ov[u]);
          if (!live) continue;
#pragma unroll
          for (int t = 0; t < 4; ++t) {   // sum 0: O may never have been written
            const float4 v = make_float4(__uint_as_float(ov[u][4 * t]), __uint_as_float(ov[u][4 * t + 1]),
                                         __uint_as_float(ov[u][4 * t + 2]), __uint_as_float(ov[u][4 * t + 3]));
            __stcg(reinterpret_cast<float4 *>(dst + (c0 + u) * 16 + 4 * t), l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : v);
          }
        }
      }
      if (live) __stcg(reinterpret_cast<float2 *>(ml), make_float2(join_max(m, l), l));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct->oempty[w]);
    }
    if (!ok) {
      report(a.status, DFLASH_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
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
  const size_t at = static_cast<size_t>(r / a.g) * nq + h * a.g + r % a.g;
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
