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
// A (request, kv head) cut by a run boundary leaves (max, sum, O) partials, and the last contributor to arrive joins them in
// contributor order: the same bits on every call.
#include "cache_attention.cuh"

namespace dflash {
namespace {

// ------------------------------------------------------------------ bf16, up to 16 query rows per (request, kv head): warp MMAs
// One 16-row tile on mma.sync: with so few rows the tensor work is a fraction
// of the HBM time whichever way it is issued, and register accumulators keep a
// page's path short.  (Two tiles of 16 rows per warp, tried for 17..32 rows,
// left one CTA per SM at 255 registers: 149 us against 103 of the tcgen05 form
// for 5 tokens x 4 heads at 128k.)  Warp 0
// produces: K page as 128-byte-swizzled 64-column halves, V^T page, and for a
// new tile its query rows, into a ring of NST stages.  Warps 1-4 each take 16
// tokens of every page with a maximum, sum and O of their own (no exchange
// per page) and meet when the tile ends, in the last page's stage.
constexpr int ROWS = 16;
template <int D>
struct Shape {
  static constexpr int KB = PAGE * D * 2, STAGE = 2 * KB;
  static constexpr int QP = D * 2 + 16, QB = ROWS * QP;                    // query rows at a padded pitch
  static constexpr int NST = D == 64 ? 6 : 3;
  static constexpr int CTAS = 2;                                           // per SM
  static constexpr int SMEM = 1024 + NST * (STAGE + QB) + 1024;
  static constexpr int PART = ROWS * (D + 2);                              // floats of a partial
};

struct __align__(16) Ctrl {
  uint64_t full[6], empty[6], cons;
  long long lo;
  Runs runs;
  int n_mine, b, h, k;                     // the run's first page: k of (b, h)
  int abort_flag, merge;
  Chunk chunk[6];
};

// CL: few (request, kv head)s over short capacities.  One cluster of
// p.cs CTAs per tile shares its pages out evenly, with no list to scan, and
// the shares meet in distributed shared memory: on a request of 2 048 tokens
// the partials' way through L2 and its counter took 5 of 15 us.
template <int D, bool CL>
__global__ void __launch_bounds__(160, Shape<D>::CTAS)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p) {
  using S = Shape<D>;
  constexpr int NST = S::NST, KB = S::KB, NT = D / 8, KS = D / 16;
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
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += request(p, b, blockIdx.x == 0).np;
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
          const long long h = quotient(lo - pre, np);
          ct->b = b;
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
    // ------------------------------------------------------------ producer (the whole warp walks)
    if (!CL && n == 0) return;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q);
    const uint64_t pol = policy_evict_first();
    const Runs runs = ct->runs;
    int cf = 0, cl = 0;
    int b = ct->b, h = ct->h, k = ct->k;
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
      const int live = first ? r.n * p.g : 0;   // query rows to load
      if (lane == 0) {
        if (bad) report(p.status, DFLASH_ERR_DEVICE);
        if (!CL && first) {
          cf = runs.owner(x - k);
          cl = runs.owner(x - k + r.np - 1);
        }
        Chunk c;
        c.b = b, c.h = h, c.page = r.p0 + k, c.row0 = r.row0, c.n = r.n, c.ctx = r.ctx;
        c.flags = (first ? FIRST : 0) | (last ? LAST : 0) | (bad ? BAD : 0) | (!CL && cf == cl ? WHOLE : 0);
        c.cf = cf, c.cl = cl, c.slot0 = runs.lo(cf) == x - k, c.slot = i - k <= 0 ? 0 : 1;
        c.nrow0 = c.nn = c.nh = c.pad = c.pad2 = 0;
        ct->chunk[st] = c;
        mbar_arrive_expect_tx(&ct->full[st], (bad ? 0 : S::STAGE) + live * D * 2);
      }
      __syncwarp();
      if (lane < live) {
        bulk_load(sQ + st * S::QB + lane * S::QP,
                  q + static_cast<size_t>(r.row0 + lane / p.g) * p.ldq + static_cast<size_t>(h * p.g + lane % p.g) * D, D * 2,
                  &ct->full[st]);
      }
      if (lane == 0 && !bad) {
        uint8_t *dk = base + st * S::STAGE;
        const int rowk = (page * p.nkv + h) * PAGE, rowv = (page * p.nkv + h) * D;
#pragma unroll
        for (int half = 0; half < D / 64; ++half)
          tma_load_2d_hint(dk + half * (PAGE * 128), &tmK, &ct->full[st], half * 64, rowk, pol);
        tma_load_2d_hint(dk + KB, &tmV, &ct->full[st], 0, rowv, pol);
      }
      issued = i + 1;
      if (++k == r.np && !CL) {
        k = 0;
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
        const int row = e * 8 + (lane >> 2);
        if (row >= c.n * p.g)
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) qf[kk][e] = qf[kk][2 + e] = 0u;
        m[e] = -INFINITY;
        l[e] = 0.f;
        top[e] = c.ctx + min(c.n - 1, row / p.g);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    }
    const int t0 = c.page * PAGE + cw * 16;   // this warp's 16 positions
    const int newest = c.ctx + c.n - 1, oldest = p.window > 0 ? c.ctx - p.window + 1 : 0;
    if (!(c.flags & BAD) && t0 <= newest && t0 + 15 >= oldest) {
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int ktok = cw * 16 + (lane >> 4) * 8 + (lane & 7);
      const uint32_t ka = smem_u32(stage) + ktok * 128;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        uint32_t b0, b1, b2, b3;
        const int ch = (kk & 3) * 2 + ((lane >> 3) & 1);
        ldmatrix_x4(ka + (kk >> 2) * (PAGE * 128) + ((ch ^ (ktok & 7)) << 4), b0, b1, b2, b3);
        mma_bf16_16816(s[0], qf[kk], b0, b1);
        mma_bf16_16816(s[1], qf[kk], b2, b3);
      }
      // positions a row does not see (whatever their slots hold)
      const bool edge = t0 + 15 > c.ctx || (p.window > 0 && t0 < newest - p.window + 1);
      if (edge) {
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
        mx[e] = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
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
      // P rounded to bf16, the type its product with V takes; the sum keeps fp32
      uint32_t pa[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float nm = m[e] == -INFINITY ? 0.f : -m[e];
        const float p0 = fast_exp2(fmaf(s[0][2 * e], p.scale_log2, nm));
        const float p1 = fast_exp2(fmaf(s[0][2 * e + 1], p.scale_log2, nm));
        const float p2 = fast_exp2(fmaf(s[1][2 * e], p.scale_log2, nm));
        const float p3 = fast_exp2(fmaf(s[1][2 * e + 1], p.scale_log2, nm));
        l[e] += (p0 + p1) + (p2 + p3);
        pa[e] = pack_bf16(p0, p1);
        pa[2 + e] = pack_bf16(p2, p3);
      }
      // slots past the newest token may hold anything: their V becomes 0
      const bool stale = t0 + 15 > newest;
      uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
      if (stale) {
        const int pos = t0 + (lane & 3) * 2;
        keep0 = pos + 1 <= newest ? 0xffffffffu : pos <= newest ? 0xffffu : 0u;
        keep1 = pos + 9 <= newest ? 0xffffffffu : pos + 8 <= newest ? 0xffffu : 0u;
      }
      const uint32_t va = smem_u32(stage + KB);
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
    const int rows = c.n * p.g;
    float *so = reinterpret_cast<float *>(stage);
    float *sm = reinterpret_cast<float *>(sQ + st * S::QB);   // [4][16] maxima, then sums (the Q slot is consumed)
    static_assert(S::QB >= 4 * 16 * 2 * 4 && S::STAGE == 4 * 16 * D * 4, "join scratch");
    if (!(ok = csync())) break;   // every warp has read the stage
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = l[e];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      const int row = (lane >> 2) + e * 8;
      if ((lane & 3) == 0) {
        sm[cw * 16 + row] = m[e];
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
        write_row<__nv_bfloat16, D>(dest_of(p, c.row0, c.h), row, c4, acc, M, L);
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
        int *ctr = p.counters + static_cast<size_t>(c.b) * p.nkv + c.h;
        const int old = atomicAdd(ctr, 1), done = old == c.cl - c.cf;
        if (done) atomicExch(ctr, 0);
        __threadfence();
        ct->merge = done;
      }
      if (!(ok = csync())) break;
      if (ct->merge)
        join_parts<D>(dest_of(p, c.row0, c.h), p.partials, c.cf, c.cl - c.cf + 1, c.slot0, S::PART, ROWS, rows, ctid,
                      128);
    } else if (!(ok = csync())) {   // the join's reads of the stage are done
      break;
    }
    fence_proxy_async_smem();   // the stage was written by plain stores: before the next bulk copy into it
    __syncwarp();
    if (lane == 0) mbar_arrive(&ct->empty[st]);
  }
  if (!ok) {
    report(p.status, DFLASH_ERR_TIMEOUT);
    *abort_flag = 1;
  }
  if constexpr (CL) {
    // ---- the cluster's shares: every CTA finishes a part of the tile's columns
    const Req r = request(p, ct->b, false);
    const int rows = r.n * p.g, rank = static_cast<int>(cluster_ctarank());
    float *xo = share(share_stage(r.np, rank));
    if (n == 0 || !ok)   // nothing to add
      for (int i = ctid; i >= 0 && i < ROWS; i += 128) *reinterpret_cast<float2 *>(xo + ROWS * D + 2 * i) = make_float2(-INFINITY, 0.f);
    __syncwarp();
    cluster_sync();
    for (int e = rank * 128 + ctid; ctid >= 0 && e < rows * (D / 4); e += p.cs * 128) {
      const int row = e / (D / 4), c4 = (e % (D / 4)) * 4;
      float M = -INFINITY, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k0 = 0; k0 < p.cs; k0 += 8) {
        float2 ml[8];
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {   // the shares' places differ by how many pages a CTA had
          const int k = min(k0 + u, p.cs - 1);
          const float *xk = share(share_stage(r.np, k));
          ml[u] = ld_dsmem_f2(dsmem_addr(xk + ROWS * D + 2 * row, k));
          v[u] = ld_dsmem_f4(dsmem_addr(xk + row * D + c4, k));
        }
        float mn = M;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (k0 + u >= p.cs) ml[u] = make_float2(-INFINITY, 0.f);
          mn = fmaxf(mn, ml[u].x);
        }
        if (mn == -INFINITY) continue;
        const float f = fast_exp2(M - mn);
        M = mn;
        L *= f;
        acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (ml[u].y == 0.f) continue;   // a share of nothing was never written
          const float w = fast_exp2(ml[u].x - mn);
          L = fmaf(w, ml[u].y, L);
          acc.x = fmaf(w, v[u].x, acc.x);
          acc.y = fmaf(w, v[u].y, acc.y);
          acc.z = fmaf(w, v[u].z, acc.z);
          acc.w = fmaf(w, v[u].w, acc.w);
        }
      }
      write_row<__nv_bfloat16, D>(dest_of(p, r.row0, ct->h), row, c4, acc, M, L);
    }
    __syncwarp();
    cluster_sync();   // no CTA leaves while its share is read
  }
}

// ------------------------------------------------------------------ fp32
// CUDA cores (tensor-core formats would round the inputs).  One CTA takes a
// share of the pages of a tile of 8 query rows of one (request, kv head):
// thread t scores token t % 64 for rows 4 (t / 64) .., then sums column t
// (of D) of P V for all 8 rows, so a K or V value read from shared memory
// serves 4 or 8 rows.  Shares are joined by the last CTA to arrive.
constexpr int F_ROWS = 8, F_THREADS = 128;

template <int D>
__global__ void __launch_bounds__(F_THREADS) decode_f32_kernel(const Params p) {
  constexpr int KP = D + 4, VP = PAGE + 4, NC = D == 128 ? 1 : 2;   // NC threads share a column at D = 64
  extern __shared__ float4 smem4[];
  float *sk = reinterpret_cast<float *>(smem4);      // [2][64][KP]
  float *sv = sk + 2 * PAGE * KP;                    // [2][D][VP]
  float *sq = sv + 2 * D * VP;                       // [8][D]
  float *sp = sq + F_ROWS * D;                       // [8][64] scores, then probabilities
  float *st = sp + F_ROWS * PAGE;                    // [3][8] maximum, sum, factor
  __shared__ int last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_start();
  const int rt = blockIdx.x % p.tiles, h = blockIdx.x / p.tiles % p.nkv, b = blockIdx.x / (p.tiles * p.nkv);
  const Req r = request(p, b, blockIdx.y == 0 && rt == 0 && h == 0 && tid == 0);
  const int rows = min(F_ROWS, r.n * p.g - rt * F_ROWS);
  if (rows <= 0) return;
  const int k0 = static_cast<int>(static_cast<long long>(blockIdx.y) * r.np / gridDim.y);
  const int k1 = static_cast<int>(static_cast<long long>(blockIdx.y + 1) * r.np / gridDim.y);
  const float *kc = static_cast<const float *>(p.k), *vc = static_cast<const float *>(p.v);
  const float *q = static_cast<const float *>(p.q);
  auto page_of = [&](int k) {
    const int pg = p.page_table[static_cast<size_t>(b) * p.max_pages + r.p0 + k];
    return pg >= 0 && pg < p.num_pages ? pg : -1;
  };
  auto load = [&](int k, int buf) {   // 16-byte asynchronous copies, rows at a padded pitch
    const int pg = page_of(k);
    if (pg >= 0) {
      const float *gk = kc + (static_cast<size_t>(pg) * p.nkv + h) * PAGE * D;
      const float *gv = vc + (static_cast<size_t>(pg) * p.nkv + h) * PAGE * D;
      for (int e = tid; e < PAGE * D / 4; e += F_THREADS) {
        const uint32_t dk = smem_u32(sk + buf * PAGE * KP + (e / (D / 4)) * KP + (e % (D / 4)) * 4);
        const uint32_t dv = smem_u32(sv + buf * D * VP + (e / (PAGE / 4)) * VP + (e % (PAGE / 4)) * 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dk), "l"(gk + 4 * e) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dv), "l"(gv + 4 * e) : "memory");
      }
    } else if (tid == 0) {
      report(p.status, DFLASH_ERR_DEVICE);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (k0 < k1) load(k0, 0);
  for (int e = tid; e < F_ROWS * D; e += F_THREADS) {
    const int row = rt * F_ROWS + e / D;
    sq[e] = e / D < rows ? q[static_cast<size_t>(r.row0 + row / p.g) * p.ldq +
                             static_cast<size_t>(h * p.g + row % p.g) * D + e % D]
                         : 0.f;
  }
  if (tid < F_ROWS) {
    st[tid] = -INFINITY;
    st[8 + tid] = 0.f;
  }
  float acc[F_ROWS];
#pragma unroll
  for (int i = 0; i < F_ROWS; ++i) acc[i] = 0.f;
  const int tok = tid % PAGE, rg = (tid / PAGE) * 4;       // scores: token, rows rg .. rg + 3
  const int col = tid % D, part_t = NC == 2 ? (tid / D) * (PAGE / 2) : 0;
  const int newest = r.ctx + r.n - 1;
  for (int k = k0; k < k1; ++k) {
    const int buf = (k - k0) & 1;
    if (k + 1 < k1) {
      load(k + 1, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const bool have = page_of(k) >= 0;
    const float *kr = sk + buf * PAGE * KP + tok * KP;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (have) {
#pragma unroll 8
      for (int c = 0; c < D; c += 4) {
        const float4 kv = *reinterpret_cast<const float4 *>(kr + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 qv = *reinterpret_cast<const float4 *>(sq + (rg + i) * D + c);
          s[i] = fmaf(kv.x, qv.x, s[i]);
          s[i] = fmaf(kv.y, qv.y, s[i]);
          s[i] = fmaf(kv.z, qv.z, s[i]);
          s[i] = fmaf(kv.w, qv.w, s[i]);
        }
      }
    }
    const int pos = (r.p0 + k) * PAGE + tok;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int hi = r.ctx + min(r.n - 1, (rt * F_ROWS + rg + i) / p.g);
      const bool see = have && pos <= hi && (p.window <= 0 || pos > hi - p.window);
      sp[(rg + i) * PAGE + tok] = see ? s[i] * p.scale_log2 : -INFINITY;
    }
    __syncthreads();
    // running maximum and sum: warp w serves rows 2 w, 2 w + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = warp * 2 + i;
      const float a = sp[row * PAGE + lane], c = sp[row * PAGE + 32 + lane];
      const float mo = st[row], mn = fmaxf(mo, warp_max(fmaxf(a, c)));
      const float nm = mn == -INFINITY ? 0.f : -mn;
      const float pa = exp2f(a + nm), pc = exp2f(c + nm), f = mn == -INFINITY ? 1.f : exp2f(mo - mn);
      const float sum = warp_sum(pa + pc);
      sp[row * PAGE + lane] = pa;
      sp[row * PAGE + 32 + lane] = pc;
      __syncwarp();
      if (lane == 0) {
        st[row] = mn;
        st[8 + row] = st[8 + row] * f + sum;
        st[16 + row] = f;
      }
    }
    __syncthreads();
    if (have) {
      const float *vr = sv + buf * D * VP + col * VP + part_t;
      const int left = newest - (r.p0 + k) * PAGE - part_t;   // slots past the newest token may hold anything
#pragma unroll
      for (int i = 0; i < F_ROWS; ++i) acc[i] *= st[16 + i];
#pragma unroll 4
      for (int c = 0; c < PAGE / NC; c += 4) {
        float4 vv = *reinterpret_cast<const float4 *>(vr + c);
        if (left < PAGE) {
          if (c > left) vv.x = 0.f;
          if (c + 1 > left) vv.y = 0.f;
          if (c + 2 > left) vv.z = 0.f;
          if (c + 3 > left) vv.w = 0.f;
        }
#pragma unroll
        for (int i = 0; i < F_ROWS; ++i) {
          const float4 pv = *reinterpret_cast<const float4 *>(sp + i * PAGE + part_t + c);
          acc[i] = fmaf(pv.x, vv.x, acc[i]);
          acc[i] = fmaf(pv.y, vv.y, acc[i]);
          acc[i] = fmaf(pv.z, vv.z, acc[i]);
          acc[i] = fmaf(pv.w, vv.w, acc[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < F_ROWS; ++i) acc[i] *= st[16 + i];
    }
    __syncthreads();
  }
  if (NC == 2) {   // the two halves of a column's tokens
    __syncthreads();
    if (tid >= D)
#pragma unroll
      for (int i = 0; i < F_ROWS; ++i) sk[i * D + col] = acc[i];
    __syncthreads();
    if (tid < D)
#pragma unroll
      for (int i = 0; i < F_ROWS; ++i) acc[i] += sk[i * D + col];
  }
  __syncthreads();
  const bool writer = tid < D;
  auto write = [&](int i, float o, float M, float L) {
    const int row = rt * F_ROWS + i, t = r.row0 + row / p.g, hq = h * p.g + row % p.g;
    const size_t at = static_cast<size_t>(t) * (p.nkv * p.g) + hq;
    static_cast<float *>(p.out)[at * D + col] = L > 0.f ? o / L : 0.f;
    if (p.lse && col == 0) p.lse[at] = L > 0.f ? (M + log2f(L)) * LN2_F : -INFINITY;
  };
  if (gridDim.y == 1) {
    if (writer)
#pragma unroll
      for (int i = 0; i < F_ROWS; ++i)
        if (i < rows) write(i, acc[i], st[i], st[8 + i]);
    return;
  }
  constexpr int FP = F_ROWS * (D + 2);
  float *part = p.partials + (static_cast<size_t>(blockIdx.x) * gridDim.y + blockIdx.y) * FP;
  if (writer)
#pragma unroll
    for (int i = 0; i < F_ROWS; ++i) __stcg(part + i * D + col, acc[i]);
  if (tid < F_ROWS) {
    __stcg(part + F_ROWS * D + tid, st[tid]);
    __stcg(part + F_ROWS * D + F_ROWS + tid, st[8 + tid]);
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    int *ctr = p.counters + blockIdx.x;
    const int old = atomicAdd(ctr, 1);
    last = old == static_cast<int>(gridDim.y) - 1;
    if (last) atomicExch(ctr, 0);
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  const float *all = p.partials + static_cast<size_t>(blockIdx.x) * gridDim.y * FP;
  join_tile<float, D, 1, 8>(dest_of(p, r.row0, h, rt * F_ROWS), [&](int i) { return all + i * FP; }, gridDim.y, F_ROWS, rows, tid, F_THREADS);
}

// ------------------------------------------------------------------ host
int row_tiles(const dflash_heads &h, int max_new, int tile_rows) {
  return (max_new * (h.n_q_heads / h.n_kv_heads) + tile_rows - 1) / tile_rows;
}

template <int D, bool CL>
int launch_decode(const dflash_heads &hs, const dflash_kv &kv, Params &p, const Device &dev, cudaStream_t s) {
  using S = Shape<D>;
  auto *kernel = decode_kernel<D, CL>;
  static std::atomic<uint64_t> smem_set, wide_set;
  if (int e = allow_smem(smem_set, dev, kernel, S::SMEM)) return e;
  if (CL && p.cs > 8)
    if (int e = allow_wide_clusters(wide_set, dev, kernel)) return e;
  const uint64_t pages = static_cast<uint64_t>(kv.num_pages) * hs.n_kv_heads;
  CUtensorMap tk, tv;
  if (int e = make_tmap_2d(&tk, p.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, D, pages * PAGE, D * 2, 64, PAGE)) return e;
  if (int e = make_tmap_2d(&tv, p.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, PAGE, pages * D, PAGE * 2, 64, D)) return e;
  p.min_chunks = 2;
  const int most = static_cast<int>(PART_TOTAL / (2 * S::PART));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL ? static_cast<unsigned>(p.B * p.nkv * p.cs) : static_cast<unsigned>(min(dev.sms * S::CTAS, most)));
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

template <int D>
int launch_f32(const Params &p, const Device &dev, cudaStream_t s) {
  constexpr int SMEM = (2 * PAGE * (D + 4) + 2 * D * (PAGE + 4) + F_ROWS * D + F_ROWS * PAGE + 24) * 4;
  auto *kernel = decode_f32_kernel<D>;
  static std::atomic<uint64_t> smem_set;
  if (int e = allow_smem(smem_set, dev, kernel, SMEM)) return e;
  // few (request, kv head, row tile)s: their pages split over several CTAs
  const long long items = static_cast<long long>(p.B) * p.nkv * p.tiles;
  const long long cap = static_cast<long long>(PART_BYTES / (F_ROWS * (D + 2) * 4)) / items;
  long long split = (3LL * dev.sms + items - 1) / items;
  split = split > (p.max_pages + 1) / 2 ? (p.max_pages + 1) / 2 : split;
  split = split > cap ? cap : split;
  split = split < 1 ? 1 : split;
  launch_pdl(kernel, dim3(static_cast<unsigned>(items), static_cast<unsigned>(split)), dim3(F_THREADS), SMEM, s, p);
  return cuda_check(cudaGetLastError(), "cache_attention launch");
}

// counters: one per (request, kv head, row tile), of the narrowest tile any path uses
size_t counter_count(const dflash_heads &h, int batch, int max_new) {
  return static_cast<size_t>(batch) * h.n_kv_heads * row_tiles(h, max_new, F_ROWS);
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
  if (window < 0 || !(scale > 0.f) || !(scale < 3.0e38f))
    return set_error(DFLASH_ERR_ARG, "cache_attention: window must be >= 0 and scale positive and finite");
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
  if (hs->dtype == DFLASH_F32) {
    p.tiles = row_tiles(*hs, max_new, F_ROWS);
    return d == 64 ? launch_f32<64>(p, dev, s) : launch_f32<128>(p, dev, s);
  }
  if (max_new * p.g > ROWS) return launch_verify(*hs, *kv, p, dev, s);
  // Clusters of up to 16 CTAs per (request, kv head) while one CTA per SM holds
  // them all, and the capacity leaves a CTA 16 pages at most: beyond that the
  // balanced runs over the whole GPU are faster.
  const long long lists = static_cast<long long>(batch) * nkv;
  p.cs = 1;
  while (p.cs < 16 && lists * p.cs * 2 <= dev.sms) p.cs *= 2;
  const bool cl = p.cs > 1 && kv->max_pages <= 16 * p.cs;
  if (d == 64) return cl ? launch_decode<64, true>(*hs, *kv, p, dev, s) : launch_decode<64, false>(*hs, *kv, p, dev, s);
  return cl ? launch_decode<128, true>(*hs, *kv, p, dev, s) : launch_decode<128, false>(*hs, *kv, p, dev, s);
}

}  // extern "C"
