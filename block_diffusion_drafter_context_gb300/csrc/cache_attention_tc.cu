// The verification form of dflash_cache_attention: 17..128 query rows per
// (request, kv head), bf16, on the 5th-generation tensor cores.
//
// At 80 rows (5 heads x 16 tokens) a 64-token page is 2.6 MFLOP of products on
// 32 KB: 0.55 PFLOP/s at HBM speed, past what warp-level MMAs reach, so S = Q
// K^T and O += P V are tcgen05.mma with M = 128 rows (the tile's, padded), S
// and O in tensor memory, and Q and P as A operands from tensor memory too:
// the shared memory then holds nothing but a ring of K / V^T pages.  One
// persistent CTA per SM with a warp per duty:
//   warp 0      walks the CTA's run of pages and feeds the ring by TMA;
//   warp 1      issues S = Q K^T (N = 64, K = D) into one of the S buffers;
//   warp 2      issues O += P V (N = D, K = the page's tokens rounded to 16);
//   warps 4-7   softmax of the run's even pages, warps 8-11 of the odd ones: one
//               tensor-memory lane (= query row) per thread: mask, online
//               softmax in the exp2 domain, P in bf16 over the page's S.
// A page's softmax alone is as long as its share of HBM's time at D = 128 and
// twice as long at D = 64, hence two groups (64 requests x 16 tokens x 5 heads
// at 16k..32k: 1021 us with one, 940 with two, the copy rate).  Each has its
// own O, maximum and sum; O is rescaled only when a row's maximum grows by 2^8.
// The group with a tile's last page joins the two and writes, while the other
// begins the next tile: it writes that tile's query rows as soon as the last S
// of this one is there.
// Row r of a tile is token r / g, query head r % g of the group.
#include "cache_attention.cuh"

namespace dflash {
namespace {

constexpr int MROWS = 128;
constexpr int NTHR = 384;
constexpr uint32_t TMEM_COLS = 512;
// Tensor memory: S buffers of 64 columns (P takes the first half of each), Q,
// two O of D columns: 512 columns at D = 128.
template <int D>
struct Shape {
  static constexpr int KB = PAGE * D * 2, STAGE = 2 * KB;       // K page as halves of [64][64], then V^T [D][64]
  static constexpr int ST = D == 128 ? 6 : 12;                  // ring depth
  static constexpr int NSB = D == 128 ? 3 : 4;                  // S buffers
  static constexpr uint32_t Q_COL = NSB * PAGE, O_COL = D == 128 ? 256 : 384;   // O of group w at O_COL + w D
  static constexpr int SMEM = 1024 + ST * STAGE + 4096;
  static constexpr int PART = MROWS * (D + 2);
  static_assert(Q_COL + D / 2 <= O_COL && O_COL + 2 * D <= TMEM_COLS, "tensor memory");
};
constexpr int MAX_ST = 12, MAX_SB = 4;

// What the other warps need to know of a page, written by the producer beside
// the page's data.  The tile's part in this CTA's run is pages i0 .. i1 of it.
struct Page {
  int b, h, page, row0, n, ctx;
  int flags;                 // BAD page, WHOLE: no other CTA has a part of the tile
  int cf, cl, slot0, slot;   // as in Chunk
  int i0, i1, pad;
};
struct __align__(16) Ctrl {
  uint64_t full[MAX_ST], empty[MAX_ST];    // a page's data; its last reader (the PV) is done
  uint64_t sfull[MAX_SB], pfull[MAX_SB], pdone[MAX_SB];   // S written; P written; PV done, the buffer is free
  uint64_t qfull, oempty[2], ml[2], cons[2], drain;       // [2]: of a softmax group
  long long lo;
  Runs runs;
  int n_mine, b, h, k;                                   // the run's first page: k of (b, h)
  uint32_t tmem;
  int abort_flag, merge[2];
  float2 helper[2][MROWS];                 // (maximum, sum) of the group without the tile's last page
  Page page[MAX_ST];
};
static_assert(sizeof(Ctrl) <= 4096, "shared memory");

// CL: few (request, kv head)s over short capacities: one cluster of p.cs CTAs
// per tile, joined in distributed shared memory.
template <int D, bool CL>
__global__ void __launch_bounds__(NTHR, 1)
    verify_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p) {
  using S = Shape<D>;
  constexpr int ST = S::ST, KB = S::KB, STAGE = S::STAGE, NSB = S::NSB;
  static_assert(S::SMEM <= 232448, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctrl *ct = reinterpret_cast<Ctrl *>(ring + ST * STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = p.g;
  volatile int *abort_flag = &ct->abort_flag;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&ct->full[i], 1);
      mbar_init(&ct->empty[i], 1);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&ct->sfull[i], 1);
      mbar_init(&ct->pfull[i], 4);
      mbar_init(&ct->pdone[i], 1);
    }
    mbar_init(&ct->qfull, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ct->oempty[i], 4);
      mbar_init(&ct->ml[i], 4);
      mbar_init(&ct->cons[i], 4);
    }
    mbar_init(&ct->drain, 2);   // both MMA issuers
    ct->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ct->tmem, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ct->tmem;
  pdl_start();
  if (CL) {
    if (threadIdx.x == 0) {
      const int list = blockIdx.x / p.cs, rank = blockIdx.x % p.cs;
      ct->b = list / p.nkv;
      ct->h = list % p.nkv;
      const int np = request(p, ct->b, rank == 0 && ct->h == 0).np;
      ct->k = rank * np / p.cs;
      ct->n_mine = (rank + 1) * np / p.cs - ct->k;
    }
  } else if (warp == 0) {
    // Lane i sums the pages of a contiguous slice of the requests; a warp
    // scan gives the list length and the slice holding this CTA's start.
    const int per = (p.B + 31) / 32, b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
    const long long sum = sum_pages(p, b0, b1, blockIdx.x == 0, [](const Req &) { return 1; });
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
        const long long np = request(p, b, false).np, span = np * p.nkv;
        if (lo < pre + span) {
          ct->b = b;
          const long long h = quotient(lo - pre, np);
          ct->h = static_cast<int>(h);
          ct->k = static_cast<int>(lo - pre - h * np);
          break;
        }
        pre += span;
      }
    }
  }
  __syncthreads();
  const int n = ct->n_mine;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (n > 0) {
      const uint64_t pol = policy_evict_first();
      const Runs runs = ct->runs;
      int cf = 0, cl = 0, i0 = 0, i1 = 0;
      int b = ct->b, h = ct->h, k = ct->k, issued = 0;
      long long x = ct->lo;
      Req r = request(p, b, false);
      bool ok = true, fresh = true;
      for (int i = 0; i < n; ++i, ++x) {
        const int st = i % ST;
        if (fresh) {
          i0 = i;
          i1 = CL ? n - 1 : min(n - 1, i + r.np - 1 - k);
        }
        ok = mbar_wait(&ct->empty[st], static_cast<uint32_t>(((i / ST) & 1) ^ 1), abort_flag, WAIT_NS);
        ok = !__any_sync(0xffffffffu, !ok);
        if (!ok) break;
        const int page = p.page_table[static_cast<size_t>(b) * p.max_pages + r.p0 + k];
        const bool bad = page < 0 || page >= p.num_pages;
        if (lane == 0) {
          if (bad) report(p.status, DFLASH_ERR_DEVICE);
          if (!CL && fresh) {
            cf = runs.owner(x - k);
            cl = runs.owner(x - k + r.np - 1);
          }
          Page c;
          c.b = b, c.h = h, c.page = r.p0 + k, c.row0 = r.row0, c.n = r.n, c.ctx = r.ctx;
          c.flags = (bad ? BAD : 0) | (!CL && cf == cl ? WHOLE : 0);
          c.cf = cf, c.cl = cl, c.slot0 = runs.lo(cf) == x - k, c.slot = i - k <= 0 ? 0 : 1;
          c.i0 = i0, c.i1 = i1, c.pad = 0;
          ct->page[st] = c;
          mbar_arrive_expect_tx(&ct->full[st], bad ? 0 : STAGE);
          if (!bad) {
            uint8_t *dk = ring + st * STAGE;
            const int rowk = (page * p.nkv + h) * PAGE, rowv = (page * p.nkv + h) * D;
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
              tma_load_2d_hint(dk + half * (PAGE * 128), &tmK, &ct->full[st], half * 64, rowk, pol);
            tma_load_2d_hint(dk + KB, &tmV, &ct->full[st], 0, rowv, pol);
          }
        }
        __syncwarp();
        issued = i + 1;
        fresh = false;
        if (++k == r.np && !CL) {
          k = 0;
          fresh = true;
          if (++h == p.nkv && i + 1 < n) {
            h = 0;
            do r = request(p, ++b, false);   // i + 1 < n: another request with work follows
            while (r.np == 0 && b + 1 < p.B);
          }
        }
      }
      if (!ok && lane == 0) {
        report(p.status, DFLASH_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // every issued copy lands before the shared memory goes away
      for (int i = max(0, issued - ST); i < issued; ++i)
        mbar_wait(&ct->full[i % ST], static_cast<uint32_t>((i / ST) & 1), nullptr, WAIT_NS);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ QK issuer
    if (lane == 0 && n > 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(MROWS, PAGE);
      int seg = 0;
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int st = i % ST, sb = i % NSB;
        ok = mbar_wait(&ct->full[st], static_cast<uint32_t>((i / ST) & 1), abort_flag, WAIT_NS);
        if (!ok) break;
        const Page &c = ct->page[st];
        const bool bad = c.flags & BAD;
        if (i == c.i0) ok = mbar_wait(&ct->qfull, static_cast<uint32_t>(seg++ & 1), abort_flag, WAIT_NS);
        ok = ok && mbar_wait(&ct->pdone[sb], static_cast<uint32_t>(((i / NSB) & 1) ^ 1), abort_flag, WAIT_NS);
        if (!ok) break;
        tc_fence_after();
        if (!bad) {
          const uint32_t k0 = smem_u32(ring + st * STAGE), qa = tmem + S::Q_COL;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)   // 16 dims = 8 columns of Q per k-step
            umma_bf16_ts(tmem + sb * PAGE, qa + static_cast<uint32_t>(kk * 8),
                         sdesc_k_sw128(k0 + (kk >> 2) * (PAGE * 128) + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
        }
        umma_commit(&ct->sfull[sb]);
      }
      if (!ok) {
        report(p.status, DFLASH_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      umma_commit(&ct->drain);   // every issued MMA retires before TMEM is released
      mbar_wait(&ct->drain, 0, nullptr, WAIT_NS);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ PV issuer
    if (lane == 0 && n > 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(MROWS, D);
      int uses[2] = {0, 0};              // tiles in which an O had a part
      bool ok = true, started[2] = {false, false};   // O holds something of this tile
      for (int i = 0; i < n && ok; ++i) {
        const int st = i % ST, sb = i % NSB, w = i & 1;
        ok = mbar_wait(&ct->full[st], static_cast<uint32_t>((i / ST) & 1), abort_flag, WAIT_NS) &&
             mbar_wait(&ct->pfull[sb], static_cast<uint32_t>((i / NSB) & 1), abort_flag, WAIT_NS);
        if (!ok) break;
        const Page &c = ct->page[st];
        if (i <= c.i0 + 1) {   // the O's first page of this tile
          started[w] = false;
          if (uses[w]++ > 0) ok = mbar_wait(&ct->oempty[w], static_cast<uint32_t>(uses[w] & 1), abort_flag, WAIT_NS);
          if (!ok) break;
        }
        tc_fence_after();
        // only the 16-token steps that hold tokens of the request
        const int left = c.ctx + c.n - c.page * PAGE, steps = (c.flags & BAD) ? 0 : (min(left, PAGE) + 15) / 16;
        const uint32_t pt = tmem + static_cast<uint32_t>(sb * PAGE), v0 = smem_u32(ring + st * STAGE + KB);
#pragma unroll
        for (int kk = 0; kk < PAGE / 16; ++kk)
          if (kk < steps)
            umma_bf16_ts(tmem + S::O_COL + w * D, pt + static_cast<uint32_t>(kk * 8), sdesc_k_sw128(v0 + kk * 32), idesc,
                         (kk > 0 || started[w]) ? 1u : 0u);
        started[w] = started[w] || steps > 0;
        umma_commit(&ct->pdone[sb]);
        umma_commit(&ct->empty[st]);   // PV is the last reader of the stage
      }
      if (!ok) {
        report(p.status, DFLASH_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      umma_commit(&ct->drain);
      mbar_wait(&ct->drain, 0, nullptr, WAIT_NS);
    }
  } else if (warp >= 4 && n > 0) {
    // ------------------------------------------------------------ softmax
    // (all four warps of a group, with query rows or not: the joins want the threads)
    const int wg = (warp >> 2) - 1, quad = warp & 3, row = quad * 32 + lane, tid = row;   // TMEM lane = query row
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t my_o = lane_base + S::O_COL + wg * D, its_o = lane_base + S::O_COL + (wg ^ 1) * D;
    const int tok = row / g, head = row % g;
    uint32_t cphase = 0;
    int uses = 0, helped = 0;       // tiles this group had a part in; those of them it closed with the other's help
    bool ok = true;
    float m = -INFINITY, l = 0.f;   // maximum (scaled, log2) and sum of this row over the group's pages of the tile
    auto waitw = [&](uint64_t *bar, uint32_t par) -> bool {   // warp-uniform bounded wait
      const bool done = mbar_wait(bar, par, abort_flag, WAIT_NS);
      return !__any_sync(0xffffffffu, !done);
    };
    auto csync = [&]() -> bool {   // the group's warps meet
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct->cons[wg]);
      const bool done = waitw(&ct->cons[wg], cphase & 1);
      ++cphase;
      return done;
    };
    for (int i = wg; i < n && ok; i += 2) {
      const int st = i % ST, sb = i % NSB;
      if (!(ok = waitw(&ct->full[st], static_cast<uint32_t>((i / ST) & 1)))) break;
      const Page &c = ct->page[st];   // stays until this page's PV, which waits for this group
      const bool first = i <= c.i0 + 1;
      if (first) ++uses;
      if (i == c.i0) {
        // the tile's query rows, this lane's: column c holds dims 2c and 2c +
        // 1.  Q is free once the last S of the tile before is complete.
        const bool live = tok < c.n;
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) +
                                                           static_cast<size_t>(c.row0 + (live ? tok : 0)) * p.ldq +
                                                           static_cast<size_t>(c.h * g + head) * D);
        uint4 u[D / 8];
#pragma unroll
        for (int t = 0; t < D / 8; ++t) u[t] = live ? __ldg(src + t) : make_uint4(0u, 0u, 0u, 0u);
        if (i > 0 && !(ok = waitw(&ct->sfull[(i - 1) % NSB], static_cast<uint32_t>(((i - 1) / NSB) & 1)))) break;
        tc_fence_after();
#pragma unroll
        for (int c4 = 0; c4 < D / 32; ++c4) {
          uint32_t w[16];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            w[4 * t] = u[4 * c4 + t].x;
            w[4 * t + 1] = u[4 * c4 + t].y;
            w[4 * t + 2] = u[4 * c4 + t].z;
            w[4 * t + 3] = u[4 * c4 + t].w;
          }
          tmem_st16_nw(lane_base + S::Q_COL + static_cast<uint32_t>(16 * c4), w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct->qfull);
      }
      if (!(ok = waitw(&ct->sfull[sb], static_cast<uint32_t>((i / NSB) & 1)))) break;
      tc_fence_after();
      const int t0 = c.page * PAGE, newest = c.ctx + c.n - 1;
      const bool bad = c.flags & BAD;
      // In a cluster a warp without query rows leaves its lanes of P as they
      // are: they only reach their own rows of O (8 requests of 900..1000
      // positions, 32 rows: 17 us, 18 without; in runs of many short tiles it
      // was 4 % slower).
      if (!CL || quad * 32 < c.n * g) {
        float x[PAGE];
        {
          uint32_t r[4][16];   // the four loads in flight together
#pragma unroll
          for (int t = 0; t < 4; ++t) tmem_ld16_nw(lane_base + sb * PAGE + 16 * t, r[t]);
          tmem_wait_ld();
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            tmem_regs_ready(r[t]);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[16 * t + e] = __uint_as_float(r[t][e]);
          }
        }
        // positions this row does not see (whatever their slots hold)
        const bool edge = bad || t0 + PAGE - 1 > c.ctx || (p.window > 0 && t0 < newest - p.window + 1);
        float low = LOWEST;   // -inf where the row sees nothing of the page
        if (edge) {
          const int top = c.ctx + min(c.n - 1, tok);
          const int hi = bad ? -1 : top - t0, lo = p.window > 0 ? top - p.window + 1 - t0 : 0;
          if (hi < 0 || lo >= PAGE) low = -INFINITY;
#pragma unroll
          for (int e = 0; e < PAGE; ++e)
            if (e > hi || e < lo) x[e] = -INFINITY;
        }
        float mx;
        {
          float a0 = x[0], a1 = x[1], a2 = x[2], a3 = x[3];
#pragma unroll
          for (int e = 4; e < PAGE; e += 4) {
            a0 = fmaxf(a0, x[e]);
            a1 = fmaxf(a1, x[e + 1]);
            a2 = fmaxf(a2, x[e + 2]);
            a3 = fmaxf(a3, x[e + 3]);
          }
          mx = fmaxf(fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * p.scale_log2, low);
        }
        if (first) {
          m = mx;
          l = 0.f;
        } else {
          const bool need = mx > m + RESCALE_LOG2;
          if (__any_sync(0xffffffffu, need)) {   // O holds the group's pages up to i - 2: wait for that PV, rescale in TMEM
            if (!(ok = waitw(&ct->pdone[(i - 2) % NSB], static_cast<uint32_t>(((i - 2) / NSB) & 1)))) break;
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
        const float nm = m == -INFINITY ? 0.f : -m;
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int e = 0; e < PAGE; e += 4) {
          x[e] = fast_exp2(fmaf(x[e], p.scale_log2, nm));
          x[e + 1] = fast_exp2(fmaf(x[e + 1], p.scale_log2, nm));
          x[e + 2] = fast_exp2(fmaf(x[e + 2], p.scale_log2, nm));
          x[e + 3] = fast_exp2(fmaf(x[e + 3], p.scale_log2, nm));
          s0 += x[e];
          s1 += x[e + 1];
          s2 += x[e + 2];
          s3 += x[e + 3];
        }
        l += (s0 + s1) + (s2 + s3);
        {   // P over this page's S, rounded to bf16 (with a second product for the rest of each
            // value the S buffers come round too late: 64 x 16 at 16k..32k 1065 us, 949 without)
          uint32_t w0[16], w1[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            w0[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
            w1[j] = pack_bf16(x[32 + 2 * j], x[32 + 2 * j + 1]);
          }
          tmem_st16_nw(lane_base + sb * PAGE, w0);
          tmem_st16_nw(lane_base + sb * PAGE + 16, w1);
          tmem_wait_st();
        }
      }
      // slots past the newest token may hold anything: in the 16-token step
      // that the PV reads with them, V becomes 0
      const int held = newest - t0 + 1;
      if (held < PAGE && (held & 15) && !bad) {
        const int ch = held >> 3, kept = held & 7;   // the 8-slot chunk with the first such slot
        for (int dr = tid; dr < D; dr += 4 * 32) {
          uint4 *v = reinterpret_cast<uint4 *>(ring + st * STAGE + KB + dr * 128);
          uint4 w = v[ch ^ (dr & 7)];
          uint32_t *e = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] &= 2 * j + 1 < kept ? 0xffffffffu : 2 * j < kept ? 0xffffu : 0u;
          v[ch ^ (dr & 7)] = w;
          if (!(ch & 1)) v[(ch + 1) ^ (dr & 7)] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      const Page last = c;   // the stage may go once P is handed over
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct->pfull[sb]);
      if (i + 1 < last.i1) continue;
      if (i + 1 == last.i1) {
        // the other group closes the tile: this one's maxima and sums for it,
        // once it has read those of the tile before
        if (uses > 1 && !(ok = waitw(&ct->oempty[wg], static_cast<uint32_t>(uses & 1)))) break;
        ct->helper[wg][row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct->ml[wg]);
        continue;
      }

      // ---- the end of this CTA's part of the tile, i == i1
      const bool two = last.i1 > last.i0;   // the other group has a part
      float2 its = make_float2(-INFINITY, 0.f);
      if (two) {
        if (!(ok = waitw(&ct->ml[wg ^ 1], static_cast<uint32_t>(helped++ & 1)))) break;
        its = ct->helper[wg ^ 1][row];
      }
      if (!(ok = waitw(&ct->pdone[sb], static_cast<uint32_t>((i / NSB) & 1)))) break;   // and with it every PV before
      tc_fence_after();
      m = join_max(m, l);
      its.x = join_max(its.x, its.y);
      const float M = fmaxf(m, its.x);
      const float f0 = l == 0.f ? 0.f : fast_exp2(m - M), f1 = its.y == 0.f ? 0.f : fast_exp2(its.x - M);
      const float L = f0 * l + f1 * its.y;
      const bool whole = last.flags & WHOLE, live = tok < last.n;
      float *xo = reinterpret_cast<float *>(ring);   // CL: this CTA's share, in the ring, idle now
      const int rows = last.n * g;
      const size_t at = static_cast<size_t>(last.row0 + (live ? tok : 0)) * (p.nkv * g) + last.h * g + head;
      float *part = p.partials + (static_cast<size_t>(blockIdx.x) * 2 + last.slot) * S::PART;
      const float inv = inverse_sum(M, L);
#pragma unroll
      for (int c0 = 0; c0 < D / 16; c0 += 2) {
        uint32_t a[2][16], b[2][16];
#pragma unroll
        for (int u = 0; u < 2; ++u) tmem_ld16_nw(my_o + (c0 + u) * 16, a[u]);
        if (two)
#pragma unroll
          for (int u = 0; u < 2; ++u) tmem_ld16_nw(its_o + (c0 + u) * 16, b[u]);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          tmem_regs_ready(a[u]);
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = l == 0.f ? 0.f : f0 * __uint_as_float(a[u][e]);   // sum 0: O was never written
          if (two) {
            tmem_regs_ready(b[u]);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = its.y == 0.f ? v[e] : fmaf(f1, __uint_as_float(b[u][e]), v[e]);
          }
          if (!live) continue;
          if (CL) {   // float4s XORed by the row: no bank conflicts
#pragma unroll
            for (int t = 0; t < 4; ++t)
              *reinterpret_cast<float4 *>(xo + row * D + ((((c0 + u) * 4 + t) ^ (row & (D / 4 - 1))) << 2)) =
                  make_float4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]);
          } else if (whole) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack_bf16(v[2 * e] * inv, v[2 * e + 1] * inv);
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at * D + (c0 + u) * 16);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
          } else {
            float4 *dst = reinterpret_cast<float4 *>(part + row * D + (c0 + u) * 16);
#pragma unroll
            for (int t = 0; t < 4; ++t) __stcg(dst + t, make_float4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]));
          }
        }
      }
      tc_fence_before();
      if (CL) {
        if (live) *reinterpret_cast<float2 *>(xo + MROWS * D + 2 * row) = make_float2(M, L);
        break;
      }
      __syncwarp();
      if (lane == 0) {   // the next tiles may overwrite the O
        mbar_arrive(&ct->oempty[wg]);
        if (two) mbar_arrive(&ct->oempty[wg ^ 1]);
      }
      if (whole) {
        if (live && p.lse) p.lse[at] = log_sum(M, L);
        continue;
      }
      if (live) {
        __stcg(part + MROWS * D + row, M);
        __stcg(part + MROWS * D + MROWS + row, L);
      }
      __threadfence();
      if (!(ok = csync())) break;
      if (tid == 0) {
        int *ctr = p.counters + static_cast<size_t>(last.b) * p.nkv + last.h;
        const int old = atomicAdd(ctr, 1), done = old == last.cl - last.cf;
        if (done) atomicExch(ctr, 0);
        __threadfence();
        ct->merge[wg] = done;
      }
      if (!(ok = csync())) break;
      if (ct->merge[wg])
        join_parts<__nv_bfloat16, D>(dest_of(p, last.row0, last.h), p.partials, last.cf, last.cl - last.cf + 1, last.slot0,
                                     S::PART, MROWS, rows, tid, 4 * 32);
    }
    if (!ok) {
      report(p.status, DFLASH_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }
  // all duties done: TMEM and the ring are free
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
  if constexpr (CL) {
    // ---- the cluster's shares: every CTA finishes a part of the tile's columns
    const Req r = request(p, ct->b, false);
    const int rows = r.n * g, rank = static_cast<int>(cluster_ctarank());
    float *xo = reinterpret_cast<float *>(ring);
    if (n == 0 || ct->abort_flag)   // nothing to add
      for (int i = threadIdx.x; i < MROWS; i += NTHR) *reinterpret_cast<float2 *>(xo + MROWS * D + 2 * i) = make_float2(-INFINITY, 0.f);
    __syncwarp();
    cluster_sync();
    const Dest dest = dest_of(p, r.row0, ct->h);
    const int items = rows * (D / 4), per = (items + p.cs - 1) / p.cs, end = min(items, (rank + 1) * per);
    for (int e = rank * per + threadIdx.x; e < end; e += NTHR) {
      const int row = e / (D / 4), c = e % (D / 4);
      const float *at = xo + row * D + ((c ^ (row & (D / 4 - 1))) << 2), *ml_at = xo + MROWS * D + 2 * row;
      float2 ml[8];
      float4 v[8];
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = min(u, p.cs - 1);
        ml[u] = ld_dsmem_f2(dsmem_addr(ml_at, k));
        v[u] = ld_dsmem_f4(dsmem_addr(at, k));
        if (u >= p.cs) ml[u] = make_float2(-INFINITY, 0.f);
        M = fmaxf(M, ml[u].x);
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (ml[u].y == 0.f) continue;   // a share of nothing was never written
        const float w = fast_exp2(ml[u].x - M);
        L = fmaf(w, ml[u].y, L);
        acc.x = fmaf(w, v[u].x, acc.x);
        acc.y = fmaf(w, v[u].y, acc.y);
        acc.z = fmaf(w, v[u].z, acc.z);
        acc.w = fmaf(w, v[u].w, acc.w);
      }
      write_row<__nv_bfloat16, D>(dest, row, c * 4, acc, M, L);
    }
    __syncwarp();
    cluster_sync();   // no CTA leaves while its share is read
  }
}

}  // namespace

template <int D, bool CL>
static int launch(const dflash_heads &hs, const dflash_kv &kv, Params &p, const Device &dev, cudaStream_t s) {
  using S = Shape<D>;
  auto *kernel = verify_kernel<D, CL>;
  static std::atomic<uint64_t> smem_set;
  if (int e = allow_smem(smem_set, dev, kernel, S::SMEM)) return e;
  const uint64_t pages = static_cast<uint64_t>(kv.num_pages) * hs.n_kv_heads;
  CUtensorMap tk, tv;
  if (int e = make_tmap_2d(&tk, p.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, D, pages * PAGE, D * 2, 64, PAGE)) return e;
  if (int e = make_tmap_2d(&tv, p.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, PAGE, pages * D, PAGE * 2, 64, D)) return e;
  p.min_chunks = 4;
  const int most = static_cast<int>(PART_TOTAL / (2 * S::PART));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL ? static_cast<unsigned>(p.B * p.nkv * p.cs) : static_cast<unsigned>(dev.sms < most ? dev.sms : most));
  cfg.blockDim = dim3(NTHR);
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

int launch_verify(const dflash_heads &hs, const dflash_kv &kv, Params &p, const Device &dev, cudaStream_t s) {
  // the rule of the narrower tiles: clusters while the SMs hold them all (three
  // quarters of them: a cluster stays within a GPC, and 16 of 8 CTAs that fill
  // an SM each took two waves, 14 us against 9), a CTA per tile while all are
  // resident, 16 pages per CTA at most
  const long long lists = static_cast<long long>(p.B) * p.nkv;
  p.cs = 1;
  while (p.cs < 8 && lists * p.cs * 2 <= dev.sms * 3 / 4) p.cs *= 2;
  const bool cl = kv.max_pages <= 16 * p.cs && lists <= dev.sms;
  if (hs.head_dim == 64) return cl ? launch<64, true>(hs, kv, p, dev, s) : launch<64, false>(hs, kv, p, dev, s);
  return cl ? launch<128, true>(hs, kv, p, dev, s) : launch<128, false>(hs, kv, p, dev, s);
}

}  // namespace dflash
