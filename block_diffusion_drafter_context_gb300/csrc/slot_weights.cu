// The attention weight that each cached token receives from the newest tokens,
// added up per kv head (dflash_add_weights), the measure by which a cache that
// outgrew its budget is cut down (evict.cu).
//
// For the key t of a (request, kv head), rows r = (committed token i, head of
// the group) with t <= ctx + i, and the row's log-sum-exp from the attention:
//   w[t] += sum_r exp(scale q_r.k_t - lse_r);
// a key that is itself new begins at 0.  A pass over K alone, 2 d values of
// operations R = tokens x heads times a key of 2 d bytes (bf16): bound by HBM.
//
// The sum runs over rows and each key has its own, so the scores are computed
// transposed, S^T = K Q^T: keys are the 128 rows of tcgen05.mma, two pages at a
// time, the query rows (N = R rounded up to 16) its columns.  In tensor memory
// a lane is then a key, and its sum is a thread's own over its columns: no
// exchange between threads, no maximum (lse is known), no atomics, the same
// bits on every call.  The list of page pairs over (request, kv head) is cut
// into equal runs, a persistent CTA each.
#include "cache_attention.cuh"

namespace dflash {
namespace {

constexpr int PAIR = 2 * PAGE;   // keys of a chunk

struct WeightArgs {
  const void *q;
  long long ldq;
  const float *lse;
  const int32_t *page_table, *cu_new, *ctx_len, *pos, *commit;   // pos, commit: may be null
  float *weights;
  int32_t *positions;      // this layer's
  long long row_len;       // capacity
  int max_pages, num_pages;
  int B, nkv, g, total, max_new, first;
  float scale_log2;
  int *status;
};

// Committed tokens m of request b: keys first .. ctx + m - 1, in chunks of
// `width` keys from page p0 on.
struct WReq {
  int row0, m, ctx, p0, np, chunks;
};
__device__ __forceinline__ WReq weight_request(const WeightArgs &a, int row0, int next, int ctx, int m, int width, bool tell) {
  const long long n = static_cast<long long>(next) - row0;
  const bool ok = row0 >= 0 && n >= 0 && n <= a.max_new && row0 + n <= a.total && ctx >= 0 &&
                  ctx + n <= static_cast<long long>(a.max_pages) * PAGE && m >= 0 && m <= n;
  if (!ok && tell) report(a.status, DFLASH_ERR_DEVICE);
  WReq r = {row0, ok && m > 0 ? m : 0, ctx, a.first / PAGE, 0, 0};
  if (r.m > 0 && ctx + r.m > a.first) {
    r.np = (ctx + r.m - 1) / PAGE - r.p0 + 1;
    r.chunks = (r.np * PAGE + width - 1) / width;
  }
  return r;
}
__device__ __forceinline__ WReq weight_request(const WeightArgs &a, int b, int width, bool tell) {
  const int row0 = a.cu_new[b], next = a.cu_new[b + 1];
  return weight_request(a, row0, next, a.ctx_len[b], a.commit ? a.commit[b] : next - row0, width, tell);
}

// A CTA's run of the list of chunks over (request, kv head).
struct Run {
  int n, b, h, k;          // chunks; the first is k of (b, h)
};
// By one warp: every lane sums the chunks of a slice of the requests.
__device__ __forceinline__ void find_run(const WeightArgs &a, int width, int least, int lane, Run *run) {
  const int per = (a.B + 31) / 32, b0 = min(a.B, lane * per), b1 = min(a.B, b0 + per);
  long long sum = 0;
  for (int b = b0; b < b1; b += 4) {   // four requests' loads at a time
    int row[5], ctx[4], m[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) row[i] = a.cu_new[min(b + i, a.B)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ctx[i] = a.ctx_len[min(b + i, a.B - 1)];
      m[i] = a.commit ? a.commit[min(b + i, a.B - 1)] : row[i + 1] - row[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i < b1) sum += weight_request(a, row[i], row[i + 1], ctx[i], m[i], width, blockIdx.x == 0).chunks;
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  Runs runs;
  runs.cut(__shfl_sync(0xffffffffu, inc, 31) * a.nkv, least, gridDim.x);
  const int c = blockIdx.x;
  const long long lo = c < runs.G ? runs.lo(c) : 0, hi = c < runs.G ? runs.lo(c + 1) : 0;
  const long long ex = (inc - sum) * a.nkv, in = inc * a.nkv;
  if (lane == 0) run->n = static_cast<int>(hi - lo);
  if (hi > lo && lo >= ex && lo < in) {   // exactly one lane
    long long pre = ex;
    for (int b = b0; b < b1; ++b) {
      const long long n = weight_request(a, b, width, false).chunks, span = n * a.nkv;
      if (lo < pre + span) {
        const long long h = quotient(lo - pre, n);
        run->b = b;
        run->h = static_cast<int>(h);
        run->k = static_cast<int>(lo - pre - h * n);
        break;
      }
      pre += span;
    }
  }
}
// Walks a run; i counts its chunks.
struct Walk {
  int i, b, h, k;
  bool fresh;              // the first chunk of (b, h) in this run
  WReq r;
  __device__ __forceinline__ void start(const WeightArgs &a, const Run &run, int width) {
    i = 0, b = run.b, h = run.h, k = run.k, fresh = true;
    if (run.n > 0) r = weight_request(a, b, width, false);
  }
  __device__ __forceinline__ void next(const WeightArgs &a, const Run &run, int width) {
    fresh = false;
    if (++i < run.n && ++k == r.chunks) {
      k = 0;
      fresh = true;
      if (++h == a.nkv) {
        h = 0;
        do r = weight_request(a, ++b, width, false);   // another request with work follows
        while (r.chunks == 0 && b + 1 < a.B);
      }
    }
  }
  // on to the next (b, h) of the run
  __device__ __forceinline__ void skip(const WeightArgs &a, const Run &run, int width) {
    i += r.chunks - k - 1;
    k = r.chunks - 1;
    next(a, run, width);
  }
};

// What a row's exp2 argument starts from: -lse in the exp2 domain.  A row that
// saw nothing (lse = -inf) gives no weight; a NaN lse makes the weights NaN.
__device__ __forceinline__ float row_bias(float lse) { return lse == -INFINITY ? -INFINITY : -lse * LOG2E_F; }

// ------------------------------------------------------------------ bf16: tcgen05
// warp 0 feeds the ring with page pairs by TMA, warp 1 issues S^T = K Q^T,
// warps 2-3 bring each tile's query rows (swizzled as TMA would) and biases
// into one of two buffers, warps 4-7 and 8-11 turn the scores of even and odd
// chunks into weights.  At 80 rows a chunk keeps four warps busy for as long as
// its share of HBM's time: 64 requests x 16 tokens x 5 heads at 16k..32k took 553
// us with four of them, 487 with eight (the copy rate).
constexpr int NTHR = 384;
constexpr int NSB = 4;           // S^T buffers of up to 128 columns: all of tensor memory
template <int D>
struct WShape {
  static constexpr int HALF = PAIR * 128;                 // 64 dims of a chunk
  static constexpr int STAGE = HALF * (D / 64);
  static constexpr int ST = D == 128 ? 4 : 8;
  static constexpr int QB = 128 * D * 2;
  static constexpr int SMEM = 1024 + ST * STAGE + 2 * QB + 4096;
};
struct WChunk {
  int b, h, t0, m, ctx, flags;   // t0: first key
  int seg;                       // tiles before this one in the run
  int rows;
};
enum { NEW_TILE = 1, END_TILE = 2, DROP0 = 4, DROP1 = 8, NEXT_END = 16 };   // DROP: a page that is not there; NEXT_END: the next chunk ends the tile
struct __align__(16) WCtrl {
  uint64_t full[8], empty[8], ready[NSB], sfull[NSB], sempty[NSB], qfull[2], qempty[2], drain;   // ready: sfull will come
  Run run;
  uint32_t tmem;
  int abort_flag;
  float bias[2][128];
  WChunk chunk[8 + NSB];         // chunk i at i % (ST + NSB): the producer is at most ST ahead of the MMAs, they NSB of the weights
};
static_assert(sizeof(WCtrl) <= 4096, "shared memory");

template <int D>
__global__ void __launch_bounds__(NTHR, 1) weights_kernel(const __grid_constant__ CUtensorMap tmK, const WeightArgs a) {
  using S = WShape<D>;
  constexpr int ST = S::ST, NI = ST + NSB;
  static_assert(S::SMEM <= 232448, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sq = ring + ST * S::STAGE;
  WCtrl *ct = reinterpret_cast<WCtrl *>(sq + 2 * S::QB);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: uniform to the compiler
  volatile int *abort_flag = &ct->abort_flag;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&ct->full[i], 1);
      mbar_init(&ct->empty[i], 1);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&ct->ready[i], 1);
      mbar_init(&ct->sfull[i], 1);
      mbar_init(&ct->sempty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ct->qfull[i], 2);
      mbar_init(&ct->qempty[i], 8);
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
  if (warp == 0) find_run(a, PAIR, 1, lane, &ct->run);
  __syncthreads();
  const Run run = ct->run;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (run.n > 0) {
      const uint64_t pol = policy_evict_first();
      Walk w;
      w.start(a, run, PAIR);
      bool ok = true;
      int issued = 0, seg = -1;
      for (; w.i < run.n; w.next(a, run, PAIR)) {
        const int i = w.i, st = i % ST;
        ok = mbar_wait(&ct->empty[st], static_cast<uint32_t>(((i / ST) & 1) ^ 1), abort_flag, WAIT_NS);
        ok = !__any_sync(0xffffffffu, !ok);
        if (!ok) break;
        // lanes 0 and 1: the chunk's pages
        const int pg = w.r.p0 + 2 * w.k + (lane & 1);
        const bool there = 2 * w.k + (lane & 1) < w.r.np;
        const int page = there ? a.page_table[static_cast<size_t>(w.b) * a.max_pages + pg] : -1;
        const bool bad = page < 0 || page >= a.num_pages;
        if (lane < 2 && there && bad) report(a.status, DFLASH_ERR_DEVICE);
        const unsigned drop = __ballot_sync(0xffffffffu, bad) & 3;
        const int page1 = __shfl_sync(0xffffffffu, page, 1);
        if (w.fresh) ++seg;
        if (lane == 0) {
          WChunk c;
          c.b = w.b, c.h = w.h, c.t0 = (w.r.p0 + 2 * w.k) * PAGE, c.m = w.r.m, c.ctx = w.r.ctx;
          const int left = min(run.n - i, w.r.chunks - w.k);   // of the tile, this one among them
          c.flags = (w.fresh ? NEW_TILE : 0) | (left == 1 ? END_TILE : left == 2 ? NEXT_END : 0) | static_cast<int>(drop) * DROP0;
          c.seg = seg, c.rows = w.r.m * a.g;
          ct->chunk[i % NI] = c;
          mbar_arrive_expect_tx(&ct->full[st], (2 - __popc(drop)) * (S::STAGE / 2));
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (!(drop >> u & 1))
#pragma unroll
              for (int half = 0; half < D / 64; ++half)
                tma_load_2d_hint(ring + st * S::STAGE + half * S::HALF + u * (PAGE * 128), &tmK, &ct->full[st], half * 64,
                                 ((u ? page1 : page) * a.nkv + w.h) * PAGE, pol);
        }
        __syncwarp();
        issued = i + 1;
      }
      if (!ok && lane == 0) {
        report(a.status, DFLASH_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // every issued copy lands before the shared memory goes away
      for (int i = max(0, issued - ST); i < issued; ++i)
        mbar_wait(&ct->full[i % ST], static_cast<uint32_t>((i / ST) & 1), nullptr, WAIT_NS);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // (the whole warp, converged; one lane of it issues)
    bool ok = true;
    int st = 0;
    uint32_t ph = 0;
    const uint32_t ring0 = smem_u32(ring), sq0 = smem_u32(sq);
    for (int i = 0; i < run.n; ++i) {
      const int sb = i % NSB;
      ok = mbar_wait(&ct->full[st], ph, abort_flag, WAIT_NS) &&
           mbar_wait(&ct->sempty[sb], static_cast<uint32_t>(((i / NSB) & 1) ^ 1), abort_flag, WAIT_NS);
      if (!(ok = !__any_sync(0xffffffffu, !ok))) break;
      const WChunk &c = ct->chunk[i % NI];
      const int qb = c.seg & 1, n = (c.rows + 15) & ~15;
      if (c.flags & NEW_TILE) {
        ok = mbar_wait(&ct->qfull[qb], static_cast<uint32_t>((c.seg >> 1) & 1), abort_flag, WAIT_NS);
        if (!(ok = !__any_sync(0xffffffffu, !ok))) break;
      }
      tc_fence_after();
      const uint32_t idesc = idesc_bf16_f32(PAIR, n), k0 = ring0 + st * S::STAGE, q0 = sq0 + qb * S::QB;
      // a page that is not there leaves what the stage held: its lanes are dropped
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_bf16_elect(tmem + sb * 128, sdesc_k_sw128(k0 + (kk >> 2) * S::HALF + (kk & 3) * 32),
                        sdesc_k_sw128(q0 + (kk >> 2) * (n * 128) + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
      umma_commit_elect(&ct->sfull[sb]);
      umma_commit_elect(&ct->empty[st]);
      if (lane == 0) mbar_arrive(&ct->ready[sb]);
      if (++st == ST) {
        st = 0;
        ph ^= 1;
      }
    }
    if (run.n > 0) {
      if (!ok && lane == 0) {
        report(a.status, DFLASH_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      __syncwarp();
      umma_commit_elect(&ct->drain);   // every issued MMA retires before TMEM is released
      mbar_wait(&ct->drain, 0, nullptr, WAIT_NS);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ query rows
    if (run.n > 0) {
      const int tid = threadIdx.x - 64;
      Walk w;
      w.start(a, run, PAIR);
      bool ok = true;
      for (int seg = 0; w.i < run.n; ++seg, w.skip(a, run, PAIR)) {
        const int qb = seg & 1, rows = w.r.m * a.g, n = (rows + 15) & ~15;
        ok = mbar_wait(&ct->qempty[qb], static_cast<uint32_t>(((seg >> 1) & 1) ^ 1), abort_flag, WAIT_NS);
        ok = !__any_sync(0xffffffffu, !ok);
        if (!ok) break;
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) + static_cast<size_t>(w.r.row0) * a.ldq +
                                   static_cast<size_t>(w.h) * a.g * D;
        uint8_t *dst = sq + qb * S::QB;
        constexpr int U = 4;
        for (int e0 = tid; e0 < n * (D / 8); e0 += 64 * U) {
          uint4 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int e = e0 + 64 * u, row = e / (D / 8), ch = e % (D / 8);
            v[u] = row < rows ? __ldg(reinterpret_cast<const uint4 *>(src + static_cast<size_t>(row / a.g) * a.ldq +
                                                                      (row % a.g) * D + ch * 8))
                              : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int e = e0 + 64 * u, row = e / (D / 8), ch = e % (D / 8);
            if (row < n)
              *reinterpret_cast<uint4 *>(dst + (ch >> 3) * (n * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = v[u];
          }
        }
        for (int r = tid; r < n; r += 64)
          ct->bias[qb][r] = r < rows ? row_bias(a.lse[static_cast<size_t>(w.r.row0 + r / a.g) * (a.nkv * a.g) + w.h * a.g +
                                                      r % a.g])
                                     : -INFINITY;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct->qfull[qb]);
      }
      if (!ok && lane == 0) {
        report(a.status, DFLASH_ERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else if (run.n > 0) {
    // ------------------------------------------------------------ weights
    const int wg = (warp >> 2) - 1, quad = warp & 3, key = quad * 32 + lane;   // TMEM lane = key of the chunk
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    bool ok = true;
    auto waitw = [&](uint64_t *bar, uint32_t par) -> bool {   // warp-uniform bounded wait
      const bool done = mbar_wait(bar, par, abort_flag, WAIT_NS);
      return !__any_sync(0xffffffffu, !done);
    };
    for (int i = wg; i < run.n; i += 2) {
      const int sb = i % NSB;
      // not on `full`: the ring may have come round by now
      if (!(ok = waitw(&ct->ready[sb], static_cast<uint32_t>((i / NSB) & 1)))) break;
      const WChunk c = ct->chunk[i % NI];
      const int t = c.t0 + key, end = c.ctx + c.m, n = (c.rows + 15) & ~15;
      const bool mine = t >= a.first && t < end && !(c.flags & (key < PAGE ? DROP0 : DROP1));
      const size_t at = (static_cast<size_t>(c.b) * a.nkv + c.h) * a.row_len + t;
      const float old = mine && t < c.ctx ? a.weights[at] : 0.f;   // under way while the scores are computed
      const int hidden = t > c.ctx ? (t - c.ctx) * a.g : 0;        // rows of tokens before this key
      const bool edge = c.t0 + PAIR - 1 > c.ctx;
      if (!(ok = waitw(&ct->sfull[sb], static_cast<uint32_t>((i / NSB) & 1)))) break;
      tc_fence_after();
      const float *bias = ct->bias[c.seg & 1];
      // 16 rows at a time, the next ones on their way
      const uint64_t sc2 = pair(a.scale_log2, a.scale_log2);
      uint64_t sum0 = pair(0.f, 0.f), sum1 = sum0;
      auto add = [&](const uint32_t (&r)[16], int c0) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 bi = *reinterpret_cast<const float4 *>(bias + c0 + e);
          const float2 y = unpair(fma2(pair(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), sc2, pair(bi.x, bi.y)));
          const float2 z = unpair(fma2(pair(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])), sc2, pair(bi.z, bi.w)));
          float p0 = fast_exp2(y.x), p1 = fast_exp2(y.y), p2 = fast_exp2(z.x), p3 = fast_exp2(z.y);
          if (edge) {
            if (c0 + e < hidden) p0 = 0.f;
            if (c0 + e + 1 < hidden) p1 = 0.f;
            if (c0 + e + 2 < hidden) p2 = 0.f;
            if (c0 + e + 3 < hidden) p3 = 0.f;
          }
          sum0 = add2(sum0, pair(p0, p1));
          sum1 = add2(sum1, pair(p2, p3));
        }
      };
      uint32_t r0[16], r1[16];
      tmem_ld16_nw(lane_base + sb * 128, r0);
      for (int c0 = 0; c0 < n; c0 += 32) {
        tmem_wait_ld();
        tmem_regs_ready(r0);
        if (c0 + 16 < n) tmem_ld16_nw(lane_base + sb * 128 + c0 + 16, r1);
        add(r0, c0);
        if (c0 + 16 >= n) break;
        tmem_wait_ld();
        tmem_regs_ready(r1);
        if (c0 + 32 < n) tmem_ld16_nw(lane_base + sb * 128 + c0 + 32, r0);
        add(r1, c0 + 16);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ct->sempty[sb]);
        // each group once a tile, at its last chunk of it; both at the only one
        if (c.flags & (END_TILE | NEXT_END)) mbar_arrive(&ct->qempty[c.seg & 1]);
        if ((c.flags & NEW_TILE) && (c.flags & END_TILE)) mbar_arrive(&ct->qempty[c.seg & 1]);
      }
      if (mine) {
        const float2 sum = unpair(add2(sum0, sum1));
        a.weights[at] = old + (sum.x + sum.y);
        if (t >= c.ctx) a.positions[at] = (a.pos ? a.pos[c.b] : c.ctx) + (t - c.ctx);
      }
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

// ------------------------------------------------------------------ fp32: warp MMAs
// The same transposed products as sums of two tf32 parts: a page per chunk, 16
// of its keys per warp as the MMA's rows, the query rows its columns; a key's
// sum is a thread's over its columns and then over the four lanes of its row.
template <int D>
struct FShape {
  static constexpr int STAGE = PAGE * D * 4, ST = 3, QP = D * 4 + 16;
  static constexpr int SMEM = 1024 + ST * STAGE + 128 * QP + 2048;
};
struct __align__(16) FCtrl {
  uint64_t full[4], empty[4], cons;
  Run run;
  int abort_flag;
  float bias[128];
};

template <int D>
__global__ void __launch_bounds__(160, 1) weights_f32_kernel(const __grid_constant__ CUtensorMap tmK, const WeightArgs a) {
  using S = FShape<D>;
  constexpr int ST = S::ST;
  static_assert(S::SMEM <= 232448 && sizeof(FCtrl) <= 2048, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sq = ring + ST * S::STAGE;
  FCtrl *ct = reinterpret_cast<FCtrl *>(sq + 128 * S::QP);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort_flag = &ct->abort_flag;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&ct->full[i], 1);
      mbar_init(&ct->empty[i], 4);
    }
    mbar_init(&ct->cons, 4);
    ct->abort_flag = 0;
    fence_mbar_init();
  }
  pdl_start();
  if (warp == 0) find_run(a, PAGE, 1, lane, &ct->run);
  __syncthreads();
  const Run run = ct->run;
  if (run.n == 0) return;
  Walk w;
  w.start(a, run, PAGE);
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = policy_evict_first();
    bool ok = true;
    int issued = 0;
    for (; w.i < run.n; w.next(a, run, PAGE)) {
      const int i = w.i, st = i % ST;
      ok = mbar_wait(&ct->empty[st], static_cast<uint32_t>(((i / ST) & 1) ^ 1), abort_flag, WAIT_NS);
      ok = !__any_sync(0xffffffffu, !ok);
      if (!ok) break;
      const int page = a.page_table[static_cast<size_t>(w.b) * a.max_pages + w.r.p0 + w.k];
      const bool bad = page < 0 || page >= a.num_pages;
      if (lane == 0) {
        if (bad) report(a.status, DFLASH_ERR_DEVICE);
        mbar_arrive_expect_tx(&ct->full[st], bad ? 0 : S::STAGE);
        if (!bad)
#pragma unroll
          for (int u = 0; u < D / 32; ++u)
            tma_load_2d_hint(ring + st * S::STAGE + u * (PAGE * 128), &tmK, &ct->full[st], u * 32, (page * a.nkv + w.h) * PAGE,
                             pol);
      }
      __syncwarp();
      issued = i + 1;
    }
    if (!ok && lane == 0) {
      report(a.status, DFLASH_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    // every issued copy lands before the shared memory goes away
    for (int i = max(0, issued - ST); i < issued; ++i)
      mbar_wait(&ct->full[i % ST], static_cast<uint32_t>((i / ST) & 1), nullptr, WAIT_NS);
    return;
  }
  const int cw = warp - 1, ctid = static_cast<int>(threadIdx.x) - 32;
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
  bool ok = true;
  for (; w.i < run.n; w.next(a, run, PAGE)) {
    const int i = w.i, st = i % ST, rows = w.r.m * a.g, n = (rows + 15) & ~15;
    if (w.fresh) {   // the tile's query rows
      if (!(ok = csync())) break;
      const float *src = static_cast<const float *>(a.q) + static_cast<size_t>(w.r.row0) * a.ldq +
                         static_cast<size_t>(w.h) * a.g * D;
      for (int e = ctid; e < n * (D / 4); e += 128) {
        const int row = e / (D / 4), ch = e % (D / 4);
        *reinterpret_cast<uint4 *>(sq + row * S::QP + ch * 16) =
            row < rows ? __ldg(reinterpret_cast<const uint4 *>(src + static_cast<size_t>(row / a.g) * a.ldq +
                                                               (row % a.g) * D + ch * 4))
                       : make_uint4(0u, 0u, 0u, 0u);
      }
      for (int r = ctid; r < n; r += 128)
        ct->bias[r] = r < rows ? row_bias(a.lse[static_cast<size_t>(w.r.row0 + r / a.g) * (a.nkv * a.g) + w.h * a.g + r % a.g])
                               : -INFINITY;
      if (!(ok = csync())) break;
    }
    const int page = a.page_table[static_cast<size_t>(w.b) * a.max_pages + w.r.p0 + w.k];
    const bool bad = page < 0 || page >= a.num_pages;
    const int t0 = (w.r.p0 + w.k) * PAGE + cw * 16, ctx = w.r.ctx, end = ctx + w.r.m;
    // this lane's keys t and t + 8 of the warp's 16
    const int t = t0 + (lane >> 2);
    const size_t at = (static_cast<size_t>(w.b) * a.nkv + w.h) * a.row_len + t;
    if (!(ok = waitw(&ct->full[st], static_cast<uint32_t>((i / ST) & 1)))) break;
    float sum[2] = {0.f, 0.f};
    if (!bad && t0 < end && t0 + 15 >= a.first) {
      const uint32_t ka = smem_u32(ring + st * S::STAGE);
      const int krow = cw * 16 + (lane & 15);                     // ldmatrix: keys 0-7, 8-15 of dims 0-3, then of dims 4-7
      const uint32_t qa = smem_u32(sq) + ((lane & 7) + (lane >> 4) * 8) * S::QP + ((lane >> 3) & 1) * 16;
      for (int r0 = 0; r0 < n; r0 += 16) {
        float s[2][4] = {}, sl[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 8; ++kk) {
          uint32_t x[4], kh[4], kl[4], q0, q1, q2, q3;
          const int ch = (kk & 3) * 2 + (lane >> 4);
          ldmatrix_x4(ka + (kk >> 2) * (PAGE * 128) + krow * 128 + ((ch ^ (krow & 7)) << 4), x[0], x[1], x[2], x[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) split_tf32(x[e], kh[e], kl[e]);
          ldmatrix_x4(qa + r0 * S::QP + kk * 32, q0, q1, q2, q3);   // rows 0-7 dims 0-3, 4-7, then rows 8-15
          mma_split(s[0], sl[0], kh, kl, q0, q1);
          mma_split(s[1], sl[1], kh, kl, q2, q3);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = r0 + 8 * u + (lane & 3) * 2 + (e & 1), tk = t + 8 * (e >> 1);
            const float p = fast_exp2(fmaf(s[u][e] + sl[u][e], a.scale_log2, ct->bias[row]));
            sum[e >> 1] += row < (tk - ctx) * a.g ? 0.f : p;   // rows of tokens before this key
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tk = t + 8 * e;
        if ((lane & 3) == 0 && tk >= a.first && tk < end) {
          a.weights[at + 8 * e] = (tk < ctx ? a.weights[at + 8 * e] : 0.f) + sum[e];
          if (tk >= ctx) a.positions[at + 8 * e] = (a.pos ? a.pos[w.b] : ctx) + (tk - ctx);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ct->empty[st]);
  }
  if (!ok) {
    report(a.status, DFLASH_ERR_TIMEOUT);
    *abort_flag = 1;
  }
}

// ------------------------------------------------------------------ host
template <int D>
int launch_bf16(const dflash_heads &hs, const dflash_kv &kv, const void *k, const WeightArgs &a, const Device &dev, cudaStream_t s) {
  auto *kernel = weights_kernel<D>;
  static std::atomic<uint64_t> smem_set;
  if (int e = allow_smem(smem_set, dev, kernel, WShape<D>::SMEM)) return e;
  CUtensorMap tk;
  const uint64_t rows = static_cast<uint64_t>(kv.num_pages) * hs.n_kv_heads * PAGE;
  if (int e = make_tmap_2d(&tk, k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, D, rows, D * 2, 64, PAGE)) return e;
  return cuda_check(launch_pdl(kernel, dim3(dev.sms), dim3(NTHR), WShape<D>::SMEM, s, tk, a), "add_weights launch");
}
template <int D>
int launch_f32(const dflash_heads &hs, const dflash_kv &kv, const void *k, const WeightArgs &a, const Device &dev, cudaStream_t s) {
  auto *kernel = weights_f32_kernel<D>;
  static std::atomic<uint64_t> smem_set;
  if (int e = allow_smem(smem_set, dev, kernel, FShape<D>::SMEM)) return e;
  CUtensorMap tk;
  const uint64_t rows = static_cast<uint64_t>(kv.num_pages) * hs.n_kv_heads * PAGE;
  if (int e = make_tmap_2d(&tk, k, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, D, rows, D * 4, 32, PAGE)) return e;
  return cuda_check(launch_pdl(kernel, dim3(dev.sms), dim3(160), FShape<D>::SMEM, s, tk, a), "add_weights launch");
}

}  // namespace

int check_slots(const char *who, const dflash_slots *sl, int batch) {
  if (!sl || !sl->weights || !sl->positions) return set_error(DFLASH_ERR_ARG, "%s: null slots", who);
  if (off_words(sl->weights, sl->positions))
    return set_error(DFLASH_ERR_ALIGN, "%s: weights and positions must be aligned to their elements", who);
  if (sl->capacity < 1 || sl->capacity > (1 << 24) || sl->batch_rows < batch || sl->batch_rows > DFLASH_MAX_BATCH)
    return set_error(DFLASH_ERR_SHAPE, "%s: capacity must be in 1..2^24 and batch_rows in batch..%d", who, DFLASH_MAX_BATCH);
  return DFLASH_OK;
}

}  // namespace dflash

extern "C" DFLASH_API int dflash_add_weights(const dflash_heads *hs, const dflash_kv *kv, const dflash_slots *slots, int layer,
                                             const void *q, long long q_stride, const float *lse, const int32_t *cu_new,
                                             int total_new, const int32_t *ctx_len, const int32_t *pos,
                                             const int32_t *n_commit, int batch, int max_new, int first, float scale,
                                             void *workspace, size_t workspace_bytes, dflash_stream_t stream) {
  using namespace dflash;
  const char *who = "add_weights";
  if (int e = check_heads(who, hs)) return e;
  if (max_new < 1 || max_new > TARGET_MAX_NEW)
    return set_error(DFLASH_ERR_ARG, "add_weights: max_new must be 1..%d", TARGET_MAX_NEW);
  const int nq = hs->n_q_heads, nkv = hs->n_kv_heads, d = hs->head_dim;
  if (int e = check_target(who, hs, kv, layer, q, q_stride, nq * d, cu_new, total_new, ctx_len, batch, workspace,
                           workspace_bytes, HEADER_BYTES))
    return e;
  if (int e = check_slots(who, slots, batch)) return e;
  if (slots->capacity < static_cast<long long>(kv->max_pages) * PAGE)
    return set_error(DFLASH_ERR_SHAPE, "add_weights: a capacity of %d, the page table's rows hold %lld", slots->capacity,
                     static_cast<long long>(kv->max_pages) * PAGE);
  if (total_new > 0 && batch > 0 && !lse) return set_error(DFLASH_ERR_ARG, "add_weights: null lse");
  if (off_words(lse, pos, n_commit))
    return set_error(DFLASH_ERR_ALIGN, "add_weights: lse, pos and n_commit must be aligned to their elements");
  if (first < 0 || !(scale > 0.f) || !(scale < 2.0e38f))   // its product with log2(e) is finite
    return set_error(DFLASH_ERR_ARG, "add_weights: first must be >= 0 and scale positive and below 2e38");
  if (batch == 0 || total_new == 0) return DFLASH_OK;
  Device dev;
  if (int e = current_device(&dev)) return e;
  const void *k = static_cast<const char *>(kv->k_cache) + layer_offset(*hs, *kv, layer) * elt_bytes(*hs);
  const size_t at = static_cast<size_t>(layer) * slots->batch_rows * nkv * slots->capacity;
  WeightArgs a = {};
  a.q = q;
  a.ldq = q_stride;
  a.lse = lse;
  a.page_table = kv->page_table;
  a.cu_new = cu_new;
  a.ctx_len = ctx_len;
  a.pos = pos;
  a.commit = n_commit;
  a.weights = slots->weights + at;
  a.positions = slots->positions + at;
  a.row_len = slots->capacity;
  a.max_pages = kv->max_pages;
  a.num_pages = kv->num_pages;
  a.B = batch;
  a.nkv = nkv;
  a.g = nq / nkv;
  a.total = total_new;
  a.max_new = max_new;
  a.first = first;
  a.scale_log2 = scale * LOG2E_F;
  a.status = static_cast<int *>(workspace);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (hs->dtype == DFLASH_F32)
    return d == 64 ? launch_f32<64>(*hs, *kv, k, a, dev, s) : launch_f32<128>(*hs, *kv, k, a, dev, s);
  return d == 64 ? launch_bf16<64>(*hs, *kv, k, a, dev, s) : launch_bf16<128>(*hs, *kv, k, a, dev, s);
}
