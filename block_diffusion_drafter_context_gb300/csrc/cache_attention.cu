// Causal attention of the newest 1..16 tokens of each request over its paged
// cache, which already holds their own keys and values
// (dflash_cache_attention): decode steps and verification passes.
//
// For query head q of token i (position p = ctx + i) and its kv head's keys:
//   s_t = scale q.k_t over p - window < t <= p,
//   out = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m),  lse = m + log sum.
// One pass over the pages with a running maximum and sum; a kv head's pages
// are read once for all its g query heads and all new tokens (rows r = i g +
// query head, R = n g of them).  At 2 d bf16 values a token and 4 d R
// operations on them the pass is bound by HBM, and the work is the flat list
// of pages over (request, kv head), cut into equal runs, one persistent CTA
// each, so that ragged batches and a single long request both fill the GPU.
// A (request, kv head) cut by a run boundary leaves (max, sum, O) partials, and
// the last contributor to arrive joins them in contributor order: the same bits
// on every call.
#include "cache_attention.cuh"

namespace dflash {
namespace {

// ------------------------------------------------------------------ tiles of 16 query rows: warp MMAs
// bf16 calls with up to 16 rows per (request, kv head), and every fp32 call in
// tiles of 16.  One tile on mma.sync: with so few rows the tensor work is a
// fraction of the HBM time whichever way it is issued, and register
// accumulators keep a page's path short.  (Two tiles of 16 rows per warp,
// tried for 17..32 bf16 rows, left one CTA per SM at 255 registers: 149 us
// against 103 of the tcgen05 form, 95 by now, for 5 tokens x 4 heads at 128k.)
//
// Warp 0 produces: the K page as 128-byte-wide swizzled column blocks, the V^T
// page (fp32: as two blocks of 32 slots), and for a new tile its query rows,
// into a ring of NST stages.  Warps 1-4 each take 16 tokens of every page with
// a maximum, sum and O of their own (no exchange per page) and meet when the
// tile ends, in the last page's stage.
//
// fp32 operands go through the tensor cores as sums of two tf32 parts, x = hi
// + lo with hi rounded to 11 bits and lo the exact rest: hi hi + hi lo + lo hi
// leaves out lo lo and the bits of lo past 11, each about 2^-24 of a product,
// so it is good to about fp32's own rounding.  On CUDA cores the same
// products took two to five times as long (a value from shared memory served 4
// rows).
constexpr int ROWS = 16;
template <typename T, int D>
struct Shape {
  static constexpr int SIZE = sizeof(T);
  static constexpr int KB = PAGE * D * SIZE, STAGE = 2 * KB;
  static constexpr int QP = D * SIZE + 16, QB = ROWS * QP;                 // query rows at a padded pitch
  static constexpr int NST = D * SIZE == 128 ? 6 : 3;
  static constexpr int CTAS = D * SIZE == 512 ? 1 : 2;                     // per SM
  static constexpr int SMEM = 1024 + NST * (STAGE + QB) + 1024;
  static constexpr int PART = ROWS * (D + 2);                              // floats of a partial
};

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

struct __align__(16) Ctrl {
  uint64_t full[6], empty[6], cons;
  long long lo;
  Runs runs;
  int n_mine, b, h, rt, k;                 // the run's first page: k of tile (b, h, rt)
  int abort_flag, merge;
  Chunk chunk[6];
};

// CL: few tiles over short capacities.  One cluster of
// p.cs CTAs per tile shares its pages out evenly, with no list to scan, and
// the shares meet in distributed shared memory: on a request of 2 048 tokens
// the partials' way through L2 and its counter took 5 of 15 us.
template <typename T, int D, bool CL>
__global__ void __launch_bounds__(160, Shape<T, D>::CTAS)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p) {
  using S = Shape<T, D>;
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int NST = S::NST, KB = S::KB, NT = D / 8, KS = D * S::SIZE / 32;   // k-steps of 32 bytes
  static_assert(sizeof(Ctrl) <= 1024 && S::SMEM <= 232448 / S::CTAS, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = base + NST * S::STAGE;
  Ctrl *ct = reinterpret_cast<Ctrl *>(sQ + NST * S::QB);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&ct->full[i], 1);
      mbar_init(&ct->empty[i], 4);
    }
    mbar_init(&ct->cons, 4);
    ct->abort_flag = 0;
    fence_mbar_init();
  }
  volatile int *abort_flag = &ct->abort_flag;
  auto tiles_of = [&](const Req &r) { return F32 ? (r.n * p.g + ROWS - 1) / ROWS : r.n > 0; };
  pdl_start();
  if (CL) {
    if (threadIdx.x == 0) {
      const int list = blockIdx.x / p.cs, rank = blockIdx.x % p.cs, head = list / p.tiles;
      ct->b = head / p.nkv;
      ct->h = head % p.nkv;
      ct->rt = list % p.tiles;
      const Req r = request(p, ct->b, rank == 0 && ct->h == 0 && ct->rt == 0);
      const int np = ct->rt < tiles_of(r) ? r.np : 0;
      ct->k = rank * np / p.cs;
      ct->n_mine = (rank + 1) * np / p.cs - ct->k;
    }
  } else if (warp == 0) {
    // Lane i sums the pages of a contiguous slice of the requests; a warp
    // scan gives the list length and the slice holding this CTA's start.
    const int per = (p.B + 31) / 32, b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
    const long long sum = sum_pages(p, b0, b1, blockIdx.x == 0, tiles_of);
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    const long long total = __shfl_sync(0xffffffffu, inc, 31) * p.nkv;
    Runs runs;
    runs.cut(total, p.min_chunks, gridDim.x);
    const int c = blockIdx.x;
    const long long lo = c < runs.G ? runs.lo(c) : 0, hi = c < runs.G ? runs.lo(c + 1) : 0;
    const long long ex = (inc - sum) * p.nkv, in = inc * p.nkv;
    if (lane == 0) {
      ct->n_mine = static_cast<int>(hi - lo);
      ct->lo = lo;
      ct->runs = runs;
    }
    if (hi > lo && lo >= ex && lo < in) {   // exactly one lane
      long long pre = ex;
      for (int b = b0; b < b1; ++b) {
        const Req r = request(p, b, false);
        const long long np = r.np, head = np * tiles_of(r), span = head * p.nkv;
        if (lo < pre + span) {
          const long long h = quotient(lo - pre, head), rt = quotient(lo - pre - h * head, np);
          ct->b = b;
          ct->h = static_cast<int>(h);
          ct->rt = static_cast<int>(rt);
          ct->k = static_cast<int>(lo - pre - h * head - rt * np);
          break;
        }
        pre += span;
      }
    }
  }
  __syncthreads();
  const int n = ct->n_mine;
  if (warp == 0) {
    // ------------------------------------------------------------ producer (the whole warp walks)
    if (!CL && n == 0) return;
    const T *q = static_cast<const T *>(p.q);
    const uint64_t pol = policy_evict_first();
    const Runs runs = ct->runs;
    int cf = 0, cl = 0;
    int b = ct->b, h = ct->h, rt = ct->rt, k = ct->k;
    long long x = ct->lo;
    Req r = request(p, b, false);
    int issued = 0;
    bool ok = true;
    for (int i = 0; i < n; ++i, ++x) {
      const int st = i % NST;
      ok = mbar_wait(&ct->empty[st], static_cast<uint32_t>(((i / NST) & 1) ^ 1), abort_flag, WAIT_NS);
      ok = !__any_sync(0xffffffffu, !ok);
      if (!ok) break;
      const bool first = i == 0 || (!CL && k == 0), last = i == n - 1 || (!CL && k == r.np - 1);
      const int page = p.page_table[static_cast<size_t>(b) * p.max_pages + r.p0 + k];
      const bool bad = page < 0 || page >= p.num_pages;
      const int live = first ? min(ROWS, r.n * p.g - rt * ROWS) : 0;   // query rows to load
      if (lane == 0) {
        if (bad) report(p.status, DFLASH_ERR_DEVICE);
        if (!CL && first) {
          cf = runs.owner(x - k);
          cl = runs.owner(x - k + r.np - 1);
        }
        Chunk c;
        c.b = b, c.h = h, c.rt = rt, c.page = r.p0 + k, c.row0 = r.row0, c.n = r.n, c.ctx = r.ctx;
        c.flags = (first ? FIRST : 0) | (last ? LAST : 0) | (bad ? BAD : 0) | (!CL && cf == cl ? WHOLE : 0);
        c.cf = cf, c.cl = cl, c.slot0 = runs.lo(cf) == x - k, c.slot = i - k <= 0 ? 0 : 1;
        ct->chunk[st] = c;
        mbar_arrive_expect_tx(&ct->full[st], (bad ? 0 : S::STAGE) + live * D * S::SIZE);
      }
      __syncwarp();
      if (lane < live) {
        const int row = rt * ROWS + lane;
        bulk_load(sQ + st * S::QB + lane * S::QP,
                  q + static_cast<size_t>(r.row0 + row / p.g) * p.ldq + static_cast<size_t>(h * p.g + row % p.g) * D,
                  D * S::SIZE, &ct->full[st]);
      }
      if (lane == 0 && !bad) {
        uint8_t *dk = base + st * S::STAGE;
        const int rowk = (page * p.nkv + h) * PAGE, rowv = (page * p.nkv + h) * D;
        constexpr int W = 128 / S::SIZE;   // elements of a block's width
#pragma unroll
        for (int i = 0; i < D / W; ++i)
          tma_load_2d_hint(dk + i * (PAGE * 128), &tmK, &ct->full[st], i * W, rowk, pol);
#pragma unroll
        for (int i = 0; i < PAGE / W; ++i)
          tma_load_2d_hint(dk + KB + i * (D * 128), &tmV, &ct->full[st], i * W, rowv, pol);
      }
      issued = i + 1;
      if (++k == r.np && !CL) {
        k = 0;
        if (++rt == tiles_of(r)) {
          rt = 0;
          if (++h == p.nkv && i + 1 < n) {
            h = 0;
            do r = request(p, ++b, false);   // i + 1 < n: another request with work follows
            while (r.np == 0 && b + 1 < p.B);
          }
        }
      }
    }
    if (!ok && lane == 0) {
      report(p.status, DFLASH_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    // every issued copy lands before the shared memory goes away
    for (int i = max(0, issued - NST); i < issued; ++i)
      mbar_wait(&ct->full[i % NST], static_cast<uint32_t>((i / NST) & 1), nullptr, WAIT_NS);
    if (!CL) return;
  }
  // -------------------------------------------------------------- consumers
  const int cw = warp - 1, ctid = static_cast<int>(threadIdx.x) - 32;
  // CL: the CTA's share after its last page, in the stage behind that page's:
  // O [ROWS][D], (maximum, sum) [ROWS]
  auto share = [&](int st) { return reinterpret_cast<float *>(base + ((st + 1) % NST) * S::STAGE); };
  auto share_stage = [&](int np, int rank) {
    const int k = (rank + 1) * np / p.cs - rank * np / p.cs;
    return k > 0 ? (k - 1) % NST : 0;
  };
  static_assert(S::STAGE >= ROWS * (D + 2) * 4, "share");
  uint32_t cphase = 0;
  auto waitw = [&](uint64_t *bar, uint32_t par) -> bool {   // warp-uniform bounded wait
    const bool ok = mbar_wait(bar, par, abort_flag, WAIT_NS);
    return !__any_sync(0xffffffffu, !ok);
  };
  auto csync = [&]() -> bool {   // the four consumer warps meet
    __syncwarp();
    if (lane == 0) mbar_arrive(&ct->cons);
    const bool ok = waitw(&ct->cons, cphase & 1);
    ++cphase;
    return ok;
  };
  uint32_t qf[KS][4];
  float o[NT][4], m[2], l[2];                 // rows lane / 4 and lane / 4 + 8
  int top[2];                                 // the last position a row sees
  // Also at the end of a tile, where nothing of it is live any more: the join
  // is a call, and would otherwise save all of this around it.
  auto clear = [&]() {
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) qf[kk][e] = 0u;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    top[0] = top[1] = 0;
  };
  clear();
  bool ok = true;
  const int n_use = CL && warp == 0 ? 0 : n;   // CL: the producer waits for the cluster at the end
  for (int i = 0; i < n_use && ok; ++i) {
    const int st = i % NST;
    ok = waitw(&ct->full[st], static_cast<uint32_t>((i / NST) & 1));
    if (!ok) break;
    const Chunk &c = ct->chunk[st];   // stays until the stage is released: no registers for it
    uint8_t *stage = base + st * S::STAGE;
    if (c.flags & FIRST) {
      const uint32_t qa = smem_u32(sQ + st * S::QB) + ((lane & 7) + (lane & 8)) * S::QP + (lane >> 4) * 16;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) ldmatrix_x4(qa + kk * 32, qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // rows past the tile's are zeros, whatever the slot held: they have
        // a say in when the warp moves its maxima
        const int row = c.rt * ROWS + e * 8 + (lane >> 2);
        if (row >= c.n * p.g)
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) qf[kk][e] = qf[kk][2 + e] = 0u;
        top[e] = c.ctx + min(c.n - 1, row / p.g);
      }
    }
    const int t0 = c.page * PAGE + cw * 16;   // this warp's 16 positions
    const int newest = c.ctx + c.n - 1, oldest = p.window > 0 ? c.ctx - p.window + 1 : 0;
    if (!(c.flags & BAD) && t0 <= newest && t0 + 15 >= oldest) {
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      float sl[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};   // fp32: the small terms
      const int ktok = cw * 16 + (lane >> 4) * 8 + (lane & 7);
      const uint32_t ka = smem_u32(stage) + ktok * 128;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        uint32_t b0, b1, b2, b3;   // 8 tokens x 16 bytes each: tokens 0-7, then 8-15
        const int ch = (kk & 3) * 2 + ((lane >> 3) & 1);
        ldmatrix_x4(ka + (kk >> 2) * (PAGE * 128) + ((ch ^ (ktok & 7)) << 4), b0, b1, b2, b3);
        if constexpr (F32) {
          uint32_t qh[4], ql[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split_tf32(qf[kk][e], qh[e], ql[e]);
          mma_split(s[0], sl[0], qh, ql, b0, b1);
          mma_split(s[1], sl[1], qh, ql, b2, b3);
        } else {
          mma_bf16_16816(s[0], qf[kk], b0, b1);
          mma_bf16_16816(s[1], qf[kk], b2, b3);
        }
      }
      if constexpr (F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e >> 2][e & 3] += sl[e >> 2][e & 3];
      }
      // positions a row does not see (whatever their slots hold)
      const bool edge = t0 + 15 > c.ctx || (p.window > 0 && t0 < newest - p.window + 1);
      float low[2] = {LOWEST, LOWEST};   // -inf where a row sees none of the 16
      if (edge) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (t0 > top[e] || (p.window > 0 && t0 + 15 <= top[e] - p.window)) low[e] = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int pos = t0 + t * 8 + (lane & 3) * 2 + (e & 1), hi = top[e >> 1];
            if (pos > hi || (p.window > 0 && pos <= hi - p.window)) s[t][e] = -INFINITY;
          }
      }
      float mx[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1])) * p.scale_log2;
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        mx[e] = fmaxf(v, low[e]);
      }
      const bool need = mx[0] > m[0] + RESCALE_LOG2 || mx[1] > m[1] + RESCALE_LOG2;
      if (__any_sync(0xffffffffu, need)) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[e], mx[e]);
          f[e] = mn == -INFINITY ? 1.f : fast_exp2(m[e] - mn);
          m[e] = mn;
          l[e] *= f[e];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] *= f[e >> 1];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float nm = m[e] == -INFINITY ? 0.f : -m[e];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int u = 0; u < 2; ++u) s[t][2 * e + u] = fast_exp2(fmaf(s[t][2 * e + u], p.scale_log2, nm));
        l[e] += (s[0][2 * e] + s[0][2 * e + 1]) + (s[1][2 * e] + s[1][2 * e + 1]);
      }
      // slots past the newest token may hold anything: their V becomes 0
      const bool stale = t0 + 15 > newest;
      const int mine = t0 + (lane & 3) * 2;   // this lane's tokens: mine, mine + 1, mine + 8, mine + 9
      const uint32_t va = smem_u32(stage + KB);
      if constexpr (F32) {
        // the accumulators of 8 tokens are an A operand whose k index t stands
        // for token 2t and t + 4 for 2t + 1; V's lanes read the same pairs
        uint32_t ph[2][4], pl[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          split_tf32(__float_as_uint(s[t][0]), ph[t][0], pl[t][0]);
          split_tf32(__float_as_uint(s[t][2]), ph[t][1], pl[t][1]);
          split_tf32(__float_as_uint(s[t][1]), ph[t][2], pl[t][2]);
          split_tf32(__float_as_uint(s[t][3]), ph[t][3], pl[t][3]);
        }
        const uint32_t vb = va + (cw >> 1) * (D * 128) + (lane >> 2) * 128 + (lane & 1) * 8;
        const int ch = (cw & 1) * 4 + ((lane & 3) >> 1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int u = 0; u < 2; ++u) {   // 8 tokens per step
            uint32_t b0, b1;
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(b0), "=r"(b1)
                         : "r"(vb + t * 1024 + (((ch + 2 * u) ^ (lane >> 2)) << 4)));
            if (stale) {
              if (mine + 8 * u > newest) b0 = 0u;
              if (mine + 8 * u + 1 > newest) b1 = 0u;
            }
            mma_split(d, d, ph[u], pl[u], b0, b1);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] += d[e];
        }
      } else {
        // P rounded to bf16, the type its product with V takes; the sum keeps
        // fp32.  A second product with the rounding's rest would make P exact
        // to 2^-16 for 1 to 3 % of the time (32 x 1 at 1k..8k: 95.9 us, 96.6
        // with it), but out's own rounding is as large and the verification
        // form pays 12 % for it: both keep the one product.
        const uint32_t pa[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]), pack_bf16(s[1][0], s[1][1]),
                                pack_bf16(s[1][2], s[1][3])};
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (stale) {
          keep0 = mine + 1 <= newest ? 0xffffffffu : mine <= newest ? 0xffffu : 0u;
          keep1 = mine + 9 <= newest ? 0xffffffffu : mine + 8 <= newest ? 0xffffu : 0u;
        }
        const int dr = (lane >> 4) * 8 + (lane & 7), vch = cw * 2 + ((lane >> 3) & 1);
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          uint32_t b0, b1, b2, b3;
          ldmatrix_x4(va + (t * 8 + dr) * 128 + ((vch ^ (dr & 7)) << 4), b0, b1, b2, b3);
          if (stale) b0 &= keep0, b1 &= keep1, b2 &= keep0, b3 &= keep1;
          mma_bf16_16816(o[t], pa, b0, b1);
          mma_bf16_16816(o[t + 1], pa, b2, b3);
        }
      }
    }
    if (!(c.flags & LAST)) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct->empty[st]);
      continue;
    }
    // ---- the end of this CTA's part of the tile: the four warps' shares are
    // joined in the stage this page occupied, O as [warp][row][D] with the
    // columns XORed by the row (no bank conflicts)
    const bool whole = c.flags & WHOLE;
    float *part = p.partials + (static_cast<size_t>(blockIdx.x) * 2 + c.slot) * S::PART;
    const int rows = min(ROWS, c.n * p.g - c.rt * ROWS);
    float *so = reinterpret_cast<float *>(stage);
    float *sm = reinterpret_cast<float *>(sQ + st * S::QB);   // [4][16] maxima, then sums (the Q slot is consumed)
    static_assert(S::QB >= 4 * 16 * 2 * 4 && S::STAGE >= 4 * 16 * D * 4, "join scratch");
    if (!(ok = csync())) break;   // every warp has read the stage
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = l[e];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      const int row = (lane >> 2) + e * 8;
      if ((lane & 3) == 0) {
        sm[cw * 16 + row] = join_max(m[e], s);
        sm[64 + cw * 16 + row] = s;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int col = (t * 8 + (lane & 3) * 2) ^ ((row & 7) << 3);
        *reinterpret_cast<float2 *>(so + (cw * 16 + row) * D + col) = make_float2(o[t][2 * e], o[t][2 * e + 1]);
      }
    }
    if (!(ok = csync())) break;
    for (int e = ctid; e < rows * (D / 4); e += 128) {
      const int row = e / (D / 4), c4 = (e % (D / 4)) * 4;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, sm[w * 16 + row]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float mw = sm[w * 16 + row], f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
        const float4 v = *reinterpret_cast<const float4 *>(so + (w * 16 + row) * D + (c4 ^ ((row & 7) << 3)));
        L = fmaf(f, sm[64 + w * 16 + row], L);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (CL) {   // this CTA's share, in a stage that holds nothing any more
        float *xo = share(st);
        *reinterpret_cast<float4 *>(xo + row * D + c4) = acc;
        if (c4 == 0) *reinterpret_cast<float2 *>(xo + ROWS * D + 2 * row) = make_float2(M, L);
      } else if (whole) {
        write_row<T, D>(dest_of(p, c.row0, c.h, c.rt * ROWS), row, c4, acc, M, L);
      } else {
        __stcg(reinterpret_cast<float4 *>(part + row * D + c4), acc);
        if (c4 == 0) {
          __stcg(part + ROWS * D + row, M);
          __stcg(part + ROWS * D + ROWS + row, L);
        }
      }
    }
    if (!ok || CL) break;
    if (!whole) {
      __threadfence();
      if (!(ok = csync())) break;
      if (ctid == 0) {
        int *ctr = p.counters + (static_cast<size_t>(c.b) * p.nkv + c.h) * p.tiles + c.rt;
        const int old = atomicAdd(ctr, 1), done = old == c.cl - c.cf;
        if (done) atomicExch(ctr, 0);
        __threadfence();
        ct->merge = done;
      }
      if (!(ok = csync())) break;
      if (ct->merge)
        join_parts<T, D>(dest_of(p, c.row0, c.h, c.rt * ROWS), p.partials, c.cf, c.cl - c.cf + 1, c.slot0, S::PART, ROWS,
                         rows, ctid, 128);
    } else if (!(ok = csync())) {   // the join's reads of the stage are done
      break;
    }
    fence_proxy_async_smem();   // the stage was written by plain stores: before the next bulk copy into it
    __syncwarp();
    if (lane == 0) mbar_arrive(&ct->empty[st]);
    clear();
  }
  if (!ok) {
    report(p.status, DFLASH_ERR_TIMEOUT);
    *abort_flag = 1;
  }
  if constexpr (CL) {
    // ---- the cluster's shares: every CTA finishes a part of the tile's columns
    const Req r = request(p, ct->b, false);
    const int rows = min(ROWS, r.n * p.g - ct->rt * ROWS), rank = static_cast<int>(cluster_ctarank());
    float *xo = share(share_stage(rows > 0 ? r.np : 0, rank));
    if (n == 0 || !ok)   // nothing to add
      for (int i = ctid; i >= 0 && i < ROWS; i += 128) *reinterpret_cast<float2 *>(xo + ROWS * D + 2 * i) = make_float2(-INFINITY, 0.f);
    __syncwarp();
    cluster_sync();
    // Each CTA an equal part, all of a column's shares in flight: left to
    // the first CTAs, in two rounds, it took 5200 cycles for 4 rows of 16 shares.
    const int items = rows * (D / 4), per = (items + p.cs - 1) / p.cs, end = min(items, (rank + 1) * per);
    auto join = [&](auto in_flight) {
      constexpr int N = decltype(in_flight)::value;
      for (int e = rank * per + ctid; ctid >= 0 && e < end; e += 128) {
        const int row = e / (D / 4), c4 = (e % (D / 4)) * 4;
        float2 ml[N];
        float4 v[N];
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int u = 0; u < N; ++u) {   // the shares' places differ by how many pages a CTA had
          const int k = min(u, p.cs - 1);
          const float *xk = share(share_stage(r.np, k));
          ml[u] = ld_dsmem_f2(dsmem_addr(xk + ROWS * D + 2 * row, k));
          v[u] = ld_dsmem_f4(dsmem_addr(xk + row * D + c4, k));
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
          if (u >= p.cs) ml[u] = make_float2(-INFINITY, 0.f);
          M = fmaxf(M, ml[u].x);
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < N; ++u) {
          if (ml[u].y == 0.f) continue;   // a share of nothing was never written
          const float w = fast_exp2(ml[u].x - M);
          L = fmaf(w, ml[u].y, L);
          acc.x = fmaf(w, v[u].x, acc.x);
          acc.y = fmaf(w, v[u].y, acc.y);
          acc.z = fmaf(w, v[u].z, acc.z);
          acc.w = fmaf(w, v[u].w, acc.w);
        }
        write_row<T, D>(dest_of(p, r.row0, ct->h, ct->rt * ROWS), row, c4, acc, M, L);
      }
    };
    if (p.cs > 8)
      join(Count<16>());
    else if (p.cs > 2)
      join(Count<8>());
    else
      join(Count<2>());
    __syncwarp();
    cluster_sync();   // no CTA leaves while its share is read
  }
}

// ------------------------------------------------------------------ host
// row tiles of a (request, kv head) at most
int row_tiles(const dflash_heads &h, int max_new) {
  return h.dtype == DFLASH_F32 ? (max_new * (h.n_q_heads / h.n_kv_heads) + ROWS - 1) / ROWS : 1;
}

template <typename T, int D, bool CL>
int launch_decode(const dflash_heads &hs, const dflash_kv &kv, Params &p, const Device &dev, cudaStream_t s) {
  using S = Shape<T, D>;
  auto *kernel = decode_kernel<T, D, CL>;
  static std::atomic<uint64_t> smem_set, wide_set;
  if (int e = allow_smem(smem_set, dev, kernel, S::SMEM)) return e;
  if (CL && p.cs > 8)
    if (int e = allow_wide_clusters(wide_set, dev, kernel)) return e;
  const uint64_t pages = static_cast<uint64_t>(kv.num_pages) * hs.n_kv_heads;
  CUtensorMap tk, tv;
  constexpr auto type = S::SIZE == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr int W = 128 / S::SIZE;
  if (int e = make_tmap_2d(&tk, p.k, type, S::SIZE, D, pages * PAGE, D * S::SIZE, W, PAGE)) return e;
  if (int e = make_tmap_2d(&tv, p.v, type, S::SIZE, PAGE, pages * D, PAGE * S::SIZE, W, D)) return e;
  p.min_chunks = 2;
  const int most = static_cast<int>(PART_TOTAL / (2 * S::PART));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL ? static_cast<unsigned>(p.B * p.nkv * p.tiles * p.cs) : static_cast<unsigned>(min(dev.sms * S::CTAS, most)));
  cfg.blockDim = dim3(160);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL ? p.cs : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL ? 2 : 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, kernel, tk, tv, p), "cache_attention launch");
}

// one per (request, kv head, row tile)
size_t counter_count(const dflash_heads &h, int batch, int max_new) {
  return static_cast<size_t>(batch) * h.n_kv_heads * row_tiles(h, max_new);
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" {

DFLASH_API size_t dflash_target_workspace_bytes(const dflash_heads *hs, int max_batch, int max_new) {
  if (check_heads("target_workspace_bytes", hs)) return 0;
  if (max_batch < 1 || max_batch > DFLASH_MAX_BATCH || max_new < 1 || max_new > TARGET_MAX_NEW) {
    set_error(DFLASH_ERR_ARG, "target_workspace_bytes: max_batch must be 1..%d and max_new 1..%d", DFLASH_MAX_BATCH,
              TARGET_MAX_NEW);
    return 0;
  }
  return HEADER_BYTES + PART_BYTES + (counter_count(*hs, max_batch, max_new) * sizeof(int) + 255) / 256 * 256;
}

DFLASH_API int dflash_cache_attention(const dflash_heads *hs, const dflash_kv *kv, int layer, const void *q,
                                      long long q_stride, const int32_t *cu_new, int total_new,
                                      const int32_t *ctx_len, int batch, int max_new, int window, float scale,
                                      void *out, float *lse, void *workspace, size_t workspace_bytes,
                                      dflash_stream_t stream) {
  const char *who = "cache_attention";
  if (int e = check_heads(who, hs)) return e;
  if (max_new < 1 || max_new > TARGET_MAX_NEW)
    return set_error(DFLASH_ERR_ARG, "cache_attention: max_new must be 1..%d", TARGET_MAX_NEW);
  const int nq = hs->n_q_heads, nkv = hs->n_kv_heads, d = hs->head_dim;
  const size_t need = HEADER_BYTES + PART_BYTES + counter_count(*hs, batch > 0 ? batch : 0, max_new) * sizeof(int);
  if (int e = check_target(who, hs, kv, layer, q, q_stride, nq * d, cu_new, total_new, ctx_len, batch, workspace,
                           workspace_bytes, need))
    return e;
  if (total_new > 0 && !out) return set_error(DFLASH_ERR_ARG, "cache_attention: null out");
  if (reinterpret_cast<uintptr_t>(out) & 15) return set_error(DFLASH_ERR_ALIGN, "cache_attention: out not 16-byte aligned");
  if (off_words(lse)) return set_error(DFLASH_ERR_ALIGN, "cache_attention: lse not aligned to its elements");
  if (window < 0 || !(scale > 0.f) || !(scale < 2.0e38f))   // its product with log2(e) is finite
    return set_error(DFLASH_ERR_ARG, "cache_attention: window must be >= 0 and scale positive and below 2e38");
  if (batch == 0 || total_new == 0) return DFLASH_OK;
  Device dev;
  if (int e = current_device(&dev)) return e;
  const size_t off = layer_offset(*hs, *kv, layer) * elt_bytes(*hs);
  Params p = {};
  p.q = q;
  p.ldq = q_stride;
  p.out = out;
  p.lse = lse;
  p.k = static_cast<const char *>(kv->k_cache) + off;
  p.v = static_cast<const char *>(kv->v_cache) + off;
  p.page_table = kv->page_table;
  p.cu_new = cu_new;
  p.ctx_len = ctx_len;
  p.max_pages = kv->max_pages;
  p.num_pages = kv->num_pages;
  p.B = batch;
  p.nkv = nkv;
  p.g = nq / nkv;
  p.total = total_new;
  p.max_new = max_new;
  p.window = window;
  p.scale_log2 = scale * LOG2E_F;
  p.partials = reinterpret_cast<float *>(static_cast<char *>(workspace) + HEADER_BYTES);
  p.counters = reinterpret_cast<int *>(static_cast<char *>(workspace) + HEADER_BYTES + PART_BYTES);
  p.status = static_cast<int *>(workspace);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = hs->dtype == DFLASH_F32;
  p.tiles = row_tiles(*hs, max_new);
  if (!f32 && max_new * p.g > ROWS) return launch_verify(*hs, *kv, p, dev, s);
  // Clusters of up to 16 CTAs per tile while one CTA per SM holds them all (8,
  // and three quarters of the SMs, where a CTA fills its SM), down to a CTA per
  // tile while all are resident, and while the capacity leaves a CTA 16 pages
  // at most: beyond that the balanced runs over the whole GPU are faster
  // (32 x 8 tiles of 1..4 pages: 8.5 us on a CTA each, 14 in runs; 64 x 8 the
  // same either way, 256 x 8 51 and 39).
  const long long lists = static_cast<long long>(batch) * nkv * p.tiles;
  p.cs = 1;
  const bool big = f32 && d == 128;
  while (p.cs < (big ? 8 : 16) && lists * p.cs * 2 <= (big ? dev.sms * 3 / 4 : dev.sms)) p.cs *= 2;
  const bool cl = kv->max_pages <= 16 * p.cs && lists <= (big ? dev.sms : 2 * dev.sms);
#define DECODE(T_, D_) \
  return cl ? launch_decode<T_, D_, true>(*hs, *kv, p, dev, s) : launch_decode<T_, D_, false>(*hs, *kv, p, dev, s)
  if (f32 && d == 64) DECODE(float, 64);
  if (f32) DECODE(float, 128);
  if (d == 64) DECODE(__nv_bfloat16, 64);
  DECODE(__nv_bfloat16, 128);
#undef DECODE
}

}  // extern "C"
