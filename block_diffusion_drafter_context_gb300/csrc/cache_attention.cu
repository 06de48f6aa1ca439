// Causal attention of the newest 1..16 tokens of each request over its paged
// cache, which already holds their own keys and values
// (dflash_cache_attention): decode steps and verification passes; and the same
// behind a prefix that the requests share (dflash_shared_attention).
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

struct __align__(16) Ctrl {
  uint64_t full[6], empty[6], cons;
  Runs runs;
  Start run;
  int abort_flag, merge;
  Chunk chunk[6];
};

// CL: few tiles over short capacities.  One cluster of
// p.cs CTAs per tile shares its pages out evenly, with no list to scan, and
// the shares meet in distributed shared memory: on a request of 2 048 tokens
// the partials' way through L2 and its counter took 5 of 15 us.
template <typename T, int D, bool CL, bool PRE>
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
      ct->run.b = head / p.nkv;
      ct->run.h = head % p.nkv;
      ct->run.rt = list % p.tiles;
      const Req r = request<PRE>(p, ct->run.b, rank == 0 && ct->run.h == 0 && ct->run.rt == 0);
      const int np = ct->run.rt < tiles_of(r) ? r.np : 0;
      ct->run.k = rank * np / p.cs;
      ct->run.n = (rank + 1) * np / p.cs - ct->run.k;
    }
  } else if (warp == 0) {
    // Lane i sums the pages of a contiguous slice of the requests; a warp
    // scan gives the list length and the slice holding this CTA's start.
    const int per = (p.B + 31) / 32, b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
    const long long sum = sum_pages<PRE>(p, b0, b1, blockIdx.x == 0, tiles_of);
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
      if (hi == lo) ct->run.n = 0;
      ct->runs = runs;
    }
    if (hi > lo && lo >= ex && lo < in)   // exactly one lane
      find_start<PRE>(p, b0, b1, ex, lo, hi, tiles_of, &ct->run);
  }
  __syncthreads();
  const int n = ct->run.n;
  if (warp == 0) {
    // ------------------------------------------------------------ producer (the whole warp walks)
    if (!CL && n == 0) return;
    const T *q = static_cast<const T *>(p.q);
    const uint64_t pol = PRE && p.pre.form == PREFIX ? policy_evict_last() : policy_evict_first();
    const Runs runs = ct->runs;
    int cf = 0, cl = 0;
    int b = ct->run.b, h = ct->run.h, rt = ct->run.rt, k = ct->run.k;
    long long x0 = ct->run.x0;   // the tile's beginning in the list
    const int cost = PRE ? p.pre.cost : 0;
    Req r = request<PRE>(p, b, false);
    int issued = 0;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int st = i % NST;
      ok = mbar_wait(&ct->empty[st], static_cast<uint32_t>(((i / NST) & 1) ^ 1), abort_flag, WAIT_NS);
      ok = !__any_sync(0xffffffffu, !ok);
      if (!ok) break;
      const bool first = i == 0 || (!CL && k == 0), last = i == n - 1 || (!CL && k == r.np - 1);
      const int page = page_of<PRE>(p, b, r.p0 + k);
      const bool bad = page < 0 || page >= p.num_pages;
      const int live = first ? min(ROWS, r.n * p.g - rt * ROWS) : 0;   // query rows to load
      if (lane == 0) {
        if (bad) report(p.status, DFLASH_ERR_DEVICE);
        if (!CL && first) {
          cf = runs.owner(x0 + cost);
          cl = runs.owner(x0 + cost + r.np - 1);
        }
        Chunk c;
        c.b = b, c.h = h, c.rt = rt, c.page = r.p0 + k, c.row0 = r.row0, c.n = r.n, c.ctx = r.ctx;
        c.flags = (first ? FIRST : 0) | (last ? LAST : 0) | (bad ? BAD : 0) | (!CL && cf == cl ? WHOLE : 0);
        c.cf = cf, c.cl = cl, c.slot0 = runs.lo(cf) >= x0, c.slot = i - k <= 0 ? 0 : 1;
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
        x0 += tile_units<PRE>(p, r);
        if (++rt == tiles_of(r)) {
          rt = 0;
          if (++h == p.nkv && i + 1 < n) {
            h = 0;
            do r = request<PRE>(p, ++b, false);   // i + 1 < n: another request with work follows
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
        // With a shared prefix the rest has its product: over few rows the error
        // of a call's outputs was up to 1.57 times that of their own rounding
        // (1.37 over many rows), and is 1.0 times with it; 64 x 1 on 8k 63.4 us
        // without, 64.6 with it.
        uint32_t pr[4];
        if constexpr (PRE) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            pr[i] = pack_bf16(s[i >> 1][(i & 1) * 2] - __uint_as_float(pa[i] << 16),
                              s[i >> 1][(i & 1) * 2 + 1] - __uint_as_float(pa[i] & 0xffff0000u));
        }
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
          if constexpr (PRE) {
            mma_bf16_16816(o[t], pr, b0, b1);
            mma_bf16_16816(o[t + 1], pr, b2, b3);
          }
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
    const Dest dest = dest_of<PRE>(p, D, c.row0, c.h, c.rt * ROWS);
    for (int e = ctid; e < rows * (D / 4); e += 128) {
      const int row = e / (D / 4), c4 = (e % (D / 4)) * 4;
      Share pre;
      if (!CL && whole) pre = share_of<D, PRE>(dest, row, c4);
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
        write_row<T, D, PRE>(dest, row, c4, acc, M, L, pre);
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
        join_parts<T, D, PRE>(dest, p.partials, c.cf, c.cl - c.cf + 1, c.slot0,
                              S::PART, ROWS, rows, ctid, 128);
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
    const Req r = request<PRE>(p, ct->run.b, false);
    const int rows = min(ROWS, r.n * p.g - ct->run.rt * ROWS), rank = static_cast<int>(cluster_ctarank());
    float *xo = share(share_stage(rows > 0 ? r.np : 0, rank));
    if (n == 0 || !ok)   // nothing to add
      for (int i = ctid; i >= 0 && i < ROWS; i += 128) *reinterpret_cast<float2 *>(xo + ROWS * D + 2 * i) = make_float2(-INFINITY, 0.f);
    __syncwarp();
    cluster_sync();
    // Each CTA an equal part, all of a column's shares in flight: left to
    // the first CTAs, in two rounds, it took 5200 cycles for 4 rows of 16 shares.
    const int items = rows * (D / 4), per = (items + p.cs - 1) / p.cs, end = min(items, (rank + 1) * per);
    const Dest dest = dest_of<PRE>(p, D, r.row0, ct->run.h, ct->run.rt * ROWS);
    auto join = [&](auto in_flight) {
      constexpr int N = decltype(in_flight)::value;
      for (int e = rank * per + ctid; ctid >= 0 && e < end; e += 128) {
        const int row = e / (D / 4), c4 = (e % (D / 4)) * 4;
        const Share pre = share_of<D, PRE>(dest, row, c4);
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
        write_row<T, D, PRE>(dest, row, c4, acc, M, L, pre);
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

template <typename T, int D, bool CL, bool PRE>
int launch_decode(const dflash_heads &hs, const dflash_kv &kv, Params &p, const Device &dev, cudaStream_t s) {
  using S = Shape<T, D>;
  auto *kernel = decode_kernel<T, D, CL, PRE>;
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

template <typename T, int D>
int launch_tiles(const dflash_heads &hs, const dflash_kv &kv, Params &p, bool cl, const Device &dev, cudaStream_t s) {
  if (p.pre.pages > 0)
    return cl ? launch_decode<T, D, true, true>(hs, kv, p, dev, s) : launch_decode<T, D, false, true>(hs, kv, p, dev, s);
  return cl ? launch_decode<T, D, true, false>(hs, kv, p, dev, s) : launch_decode<T, D, false, false>(hs, kv, p, dev, s);
}

// One launch over p.B requests of at most `rows` query rows per kv head and
// `pages` pages.
int launch_attention(const dflash_heads &hs, const dflash_kv &kv, Params &p, long long rows, int pages, const Device &dev,
                     cudaStream_t s) {
  const bool f32 = hs.dtype == DFLASH_F32;
  const int d = hs.head_dim;
  if (!f32 && rows > ROWS) return launch_verify(hs, kv, p, pages, dev, s);
  // Clusters of up to 16 CTAs per tile while one CTA per SM holds them all (8,
  // and three quarters of the SMs, where a CTA fills its SM), down to a CTA per
  // tile while all are resident, and while the capacity leaves a CTA 16 pages
  // at most: beyond that the balanced runs over the whole GPU are faster
  // (32 x 8 tiles of 1..4 pages: 8.5 us on a CTA each, 14 in runs; 64 x 8 the
  // same either way, 256 x 8 51 and 39).
  const long long lists = static_cast<long long>(p.B) * p.nkv * p.tiles;
  p.cs = 1;
  const bool big = f32 && d == 128;
  while (p.cs < (big ? 8 : 16) && lists * p.cs * 2 <= (big ? dev.sms * 3 / 4 : dev.sms)) p.cs *= 2;
  const bool cl = pages <= 16 * p.cs && lists <= (big ? dev.sms : 2 * dev.sms);
  if (f32) return d == 64 ? launch_tiles<float, 64>(hs, kv, p, cl, dev, s) : launch_tiles<float, 128>(hs, kv, p, cl, dev, s);
  return d == 64 ? launch_tiles<__nv_bfloat16, 64>(hs, kv, p, cl, dev, s)
                 : launch_tiles<__nv_bfloat16, 128>(hs, kv, p, cl, dev, s);
}

// The arguments that both entry points share, checked and taken over; p.B == 0:
// nothing to do.
int take(const char *who, const dflash_heads *hs, const dflash_kv *kv, int layer, const void *q, long long q_stride,
         const int32_t *cu_new, int total_new, const int32_t *ctx_len, int batch, int max_new, float scale, void *out,
         float *lse, void *workspace, size_t workspace_bytes, Params &p) {
  if (int e = check_heads(who, hs)) return e;
  if (max_new < 1 || max_new > TARGET_MAX_NEW)
    return set_error(DFLASH_ERR_ARG, "%s: max_new must be 1..%d", who, TARGET_MAX_NEW);
  const int nq = hs->n_q_heads, nkv = hs->n_kv_heads, d = hs->head_dim;
  const size_t need = HEADER_BYTES + PART_BYTES + counter_count(*hs, batch > 0 ? batch : 0, max_new) * sizeof(int);
  if (int e = check_target(who, hs, kv, layer, q, q_stride, nq * d, cu_new, total_new, ctx_len, batch, workspace,
                           workspace_bytes, need))
    return e;
  if (total_new > 0 && !out) return set_error(DFLASH_ERR_ARG, "%s: null out", who);
  if (reinterpret_cast<uintptr_t>(out) & 15) return set_error(DFLASH_ERR_ALIGN, "%s: out not 16-byte aligned", who);
  if (off_words(lse)) return set_error(DFLASH_ERR_ALIGN, "%s: lse not aligned to its elements", who);
  if (!(scale > 0.f) || !(scale < 2.0e38f))   // its product with log2(e) is finite
    return set_error(DFLASH_ERR_ARG, "%s: scale must be positive and below 2e38", who);
  p = Params();
  if (batch == 0 || total_new == 0) return DFLASH_OK;
  const size_t off = layer_offset(*hs, *kv, layer) * elt_bytes(*hs);
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
  p.scale_log2 = scale * LOG2E_F;
  p.tiles = row_tiles(*hs, max_new);
  p.partials = reinterpret_cast<float *>(static_cast<char *>(workspace) + HEADER_BYTES);
  p.counters = reinterpret_cast<int *>(static_cast<char *>(workspace) + HEADER_BYTES + PART_BYTES);
  p.status = static_cast<int *>(workspace);
  return DFLASH_OK;
}

std::atomic<int> forced_launches{0};   // dflash_debug_shared_launches

// rows of a valid batch: each of its requests has at most max_new
int row_cap(int total_new, int batch, int max_new) {
  const long long most = static_cast<long long>(batch) * max_new;
  return static_cast<int>(most < total_new ? most : total_new);
}
size_t share_bytes(const dflash_heads &h, int rows) {
  const size_t shares = static_cast<size_t>(rows) * h.n_q_heads * (h.head_dim + 2) * sizeof(float);
  return (shares + 15) / 16 * 16 + (h.dtype == DFLASH_F32 ? 0 : PREFIX_PART_BYTES);
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
  if (window < 0) return set_error(DFLASH_ERR_ARG, "cache_attention: window must be >= 0");
  Params p;
  if (int e = take("cache_attention", hs, kv, layer, q, q_stride, cu_new, total_new, ctx_len, batch, max_new, scale, out,
                   lse, workspace, workspace_bytes, p))
    return e;
  if (p.B == 0) return DFLASH_OK;
  Device dev;
  if (int e = current_device(&dev)) return e;
  p.window = window;
  return launch_attention(*hs, *kv, p, static_cast<long long>(max_new) * p.g, kv->max_pages, dev,
                          reinterpret_cast<cudaStream_t>(stream));
}

DFLASH_API size_t dflash_shared_rows_bytes(const dflash_heads *hs, int max_batch, int max_new) {
  if (check_heads("shared_rows_bytes", hs)) return 0;
  if (max_batch < 1 || max_batch > DFLASH_MAX_BATCH || max_new < 1 || max_new > TARGET_MAX_NEW) {
    set_error(DFLASH_ERR_ARG, "shared_rows_bytes: max_batch must be 1..%d and max_new 1..%d", DFLASH_MAX_BATCH,
              TARGET_MAX_NEW);
    return 0;
  }
  return share_bytes(*hs, max_batch * max_new);
}

DFLASH_API int dflash_debug_shared_launches(int n) {
  if (n < 0 || n > 2) return set_error(DFLASH_ERR_ARG, "debug_shared_launches: 0, 1 or 2");
  forced_launches.store(n, std::memory_order_relaxed);
  return DFLASH_OK;
}

DFLASH_API int dflash_shared_attention(const dflash_heads *hs, const dflash_kv *kv, int layer, const void *q,
                                       long long q_stride, const int32_t *cu_new, int total_new,
                                       const int32_t *ctx_len, int batch, int max_new, int shared_len, float scale,
                                       void *out, float *lse, void *rows, size_t rows_bytes, void *workspace,
                                       size_t workspace_bytes, dflash_stream_t stream) {
  const char *who = "shared_attention";
  Params p;
  if (int e = take(who, hs, kv, layer, q, q_stride, cu_new, total_new, ctx_len, batch, max_new, scale, out, lse, workspace,
                   workspace_bytes, p))
    return e;
  if (shared_len < 0 || shared_len % PAGE || shared_len / PAGE >= kv->max_pages)
    return set_error(DFLASH_ERR_SHAPE, "shared_attention: shared_len must be whole pages of %d, fewer than max_pages", PAGE);
  if (p.B == 0) return DFLASH_OK;
  const int most = row_cap(total_new, batch, max_new);
  if (shared_len > 0) {
    if (!rows) return set_error(DFLASH_ERR_ARG, "shared_attention: null rows");
    if (reinterpret_cast<uintptr_t>(rows) & 15) return set_error(DFLASH_ERR_ALIGN, "shared_attention: rows not 16-byte aligned");
    if (rows_bytes < share_bytes(*hs, most))
      return set_error(DFLASH_ERR_SHAPE, "shared_attention: rows of %zu bytes, %zu needed", rows_bytes, share_bytes(*hs, most));
  }
  Device dev;
  if (int e = current_device(&dev)) return e;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int pages = shared_len / PAGE;
  const bool f32 = hs->dtype == DFLASH_F32;
  const long long rows_each = static_cast<long long>(max_new) * p.g, all = static_cast<long long>(most) * p.g;
  p.pre.rows = static_cast<float *>(rows);
  p.pre.row_cap = most;
  p.pre.pages = pages;
  p.pre.batch = batch;
  // One launch while what it reads of the prefix beyond two launches is little:
  // once per request (fp32: per tile of 16 rows) instead of once (per 16 of all
  // rows).  Two launches against one, us, at
  //   32 / 8 heads x 1 token, 4 requests on 1024: 15.9, 10.1; 16 on 1024 (60 MB):
  //     21.5, 19.4; 32 on 1024 (130 MB): 22.3, 26.4;
  //   40 / 8 heads x 16 tokens, 8 on 4096 (117 MB): 47, 45; 16 on 4096 (250 MB): 58, 61.5;
  //   fp32, 16 / 8 heads x 1 token, 16 on 256 (29 MB): 23, 21; 64 on 256 (115 MB): 59, 65.
  const long long tiles_each = f32 ? (rows_each + ROWS - 1) / ROWS : 1;
  const long long passes = batch * tiles_each - (f32 ? (all + ROWS - 1) / ROWS : 1);
  const long long again = passes * hs->n_kv_heads * pages * 2 * PAGE * hs->head_dim * elt_bytes(*hs);
  const int forced = forced_launches.load(std::memory_order_relaxed);
  if (pages == 0 || (forced ? forced == 1 : again <= (f32 ? 48ll << 20 : rows_each > ROWS ? 192ll << 20 : 96ll << 20))) {
    p.pre.form = ONE;
    return launch_attention(*hs, *kv, p, rows_each, kv->max_pages, dev, s);
  }
  // The prefix.  fp32, or no more than 16 rows: one request with every row, in
  // tiles of 16, whose counters are at most batch * row_tiles(max_new) for each
  // kv head, as many as the second launch has.
  if (f32 || all <= ROWS) {
    Params x = p;
    x.B = 1;
    x.pre.form = PREFIX;
    x.pre.tile_tokens = most;
    x.tiles = static_cast<int>((all + ROWS - 1) / ROWS);
    if (int e = launch_attention(*hs, *kv, x, all, pages, dev, s)) return e;
  } else if (int e = launch_prefix(*hs, *kv, p, dev, s)) {
    return e;
  }
  // What a tile takes beside its pages, in pages (a call of 64 requests: 16 new
  // tokens of 5 heads on 2..32 own pages behind 2048 positions 206 us at 0, 147 at 8,
  // 145 at 12, 147 at 16; one token of 4 heads on 1..16 pages behind 8192 67.2 at 0,
  // 63.3 at 3, 65.0 at 8).
  p.pre.form = OWN;
  p.pre.cost = !f32 && rows_each > ROWS ? 14 : 3;
  return launch_attention(*hs, *kv, p, rows_each, kv->max_pages - pages, dev, s);
}

}  // extern "C"
