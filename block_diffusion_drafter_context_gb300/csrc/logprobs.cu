// Log probabilities of given tokens, with the row's entropy, the token's rank
// and the 16 most probable alternatives (dflash_token_logprobs).
//
// With y = x / T, m = max y and z = sum e^(y - m) over the vocabulary:
//   logprob = y_t - m - log z,   entropy = log z - sum e^(y - m) (y - m) / z,
//   rank = #{v : x_v > x_t, or x_v = x_t and v < t}.
// Everything comes from one pass over the logits: a running (m, z, w = sum
// e^(y-m) (y-m)) per thread, joined as m' = max, z' = z e^(m-m'),
// w' = e^(m-m') (w + z (m - m')); the rank is a count against the token's own
// logit, read first; the alternatives lie where a thread's maximum reaches the
// 16th largest of the threads' maxima, and only those pieces of the row are
// read again.  Bound by the logits' HBM bytes; a row is cut over a cluster of
// CTAs, which join through distributed shared memory, so that no workspace is
// needed.
#include "top16.cuh"
#include "target.h"

#include <math.h>

namespace dflash {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32, CTAS = 4;   // CTAS: resident per SM
constexpr int MAX_CLUSTER = 8;
constexpr float LOG2E_F = 1.4426950408889634f, LN2_F = 0.6931471805599453f;
// y - m in log2 units below which e^(y-m) is 0 in fp32: masked logits are kept
// here, so that 0 * (y - m) stays 0
constexpr float FAR = -1000.f;

struct Args {
  const void *x;
  long long ld;
  int V, n_top, cs;
  const int32_t *ids;
  float inv_t;               // 1 / temperature
  float *logprob, *entropy;
  int32_t *rank, *top_ids;
  float *top_lp;
};

// running maximum of the logits, sum of e^(y-m) and of e^(y-m) (y-m) log2(e).
// The maximum is subtracted before the scaling c = log2(e) / T: exact for a
// row of the type's lowest values too.
struct Stat {
  float m, z, w;
};

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// z and w of a share with maximum m, against a larger maximum
__device__ __forceinline__ void rebase(Stat &a, float m, float c) {
  const float d = a.m == m ? 0.f : fmaxf((a.m - m) * c, FAR), f = fast_exp2(d);
  a.w = f * fmaf(a.z, d, a.w);
  a.z *= f;
  a.m = m;
}
// the warp's shares joined, into every lane: the maximum first, so that each
// lane scales once and the sums are plain
__device__ __forceinline__ void warp_join(Stat &a, int &cnt, float c) {
  rebase(a, warp_max_nan(a.m), c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
  }
  cnt = __reduce_add_sync(0xffffffffu, cnt);
}

template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t NONE = 0xff800000u;      // -inf
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
  }
  template <int U>
  static __device__ __forceinline__ float maximum(const uint4 (&u)[U]) {
    float m[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      m[i] = max_nan(max_nan(__uint_as_float(u[i].x), __uint_as_float(u[i].y)), max_nan(__uint_as_float(u[i].z), __uint_as_float(u[i].w)));
#pragma unroll
    for (int i = 1; i < U; ++i) m[0] = max_nan(m[0], m[i]);
    return m[0];
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t NONE = 0xff80ff80u;      // two -inf
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  template <int U>
  static __device__ __forceinline__ float maximum(const uint4 (&u)[U]) {
    uint32_t m[U];
#pragma unroll
    for (int i = 0; i < U; ++i) m[i] = max2(max2(u[i].x, u[i].y), max2(u[i].z, u[i].w));
#pragma unroll
    for (int i = 1; i < U; ++i) m[0] = max2(m[0], m[i]);
    return max_nan(__uint_as_float(m[0] << 16), __uint_as_float(m[0] & 0xffff0000u));
  }
};

// ---- shared memory of a CTA: for each warp a ring of STAGES x 2 KB of logits
// (4 vectors per lane), then the struct below.  Two stages: 128 KB of rings for
// an SM's 4 CTAs; four stages were slower (123 against 114 us at 1024 fp32 rows
// of 151 936).  Where the grid leaves an SM two CTAs at most,
// four: a CTA's own round trips are the time there (64 such rows on 4 CTAs
// each: 20 us with two stages, 15 with four).
constexpr int WIDE = 2, DEEP = 4;                    // stages
constexpr int U = 4, SV = 32 * U;
constexpr int SEGS = 8;                              // parts of the stream whose maxima each thread keeps
constexpr int ring_bytes(int stages) { return WARPS * stages * SV * 16; }
constexpr int MIN_SHARE = 8192;                      // logits of a CTA at least, where a row is cut
constexpr int MAX_SHARE = 400 << 10;                 // bytes of a CTA at most, while there are CTAs for a row left
constexpr int LIST = 512;                            // candidates a CTA can list
constexpr unsigned long long WAIT_NS = 2000000000ull;
struct Shared {
  alignas(16) uint64_t list[LIST];                   // candidates for the 16 largest (value, id) keys, unordered
  uint64_t best[TOP_K];      // the 16 largest in order, 0 where there are fewer
  uint64_t full[WARPS][DEEP];
  alignas(16) uint64_t peer_keys[MAX_CLUSTER * TOP_K];   // rank 0: every CTA's best
  float4 peer_stat[MAX_CLUSTER];                         // rank 0: (m, z, w, count) of every CTA
  float4 warp_stat[WARPS];
  float warp_two[WARPS];
  float seg[SEGS][THREADS];  // the threads' maxima, by part
  uint16_t owners[SEGS * THREADS];   // the (part, thread) pairs whose maximum reaches the floor
  int listed, owned, failed;
};
constexpr int smem_bytes(int stages) { return ring_bytes(stages) + static_cast<int>(sizeof(Shared)) + 16; }
static_assert(smem_bytes(WIDE) + 1024 <= 233472 / CTAS && smem_bytes(DEEP) + 1024 <= 233472 / 2, "shared memory");

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// two fp32 values in one 64-bit register: one instruction for both
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t p, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// the smallest float above x
__device__ __forceinline__ float next_up(float x) {
  const uint32_t u = __float_as_uint(x);
  return x == 0.f ? __uint_as_float(1u) : __uint_as_float(u & 0x80000000u ? u - 1u : u + 1u);
}

// The 16 largest of n distinct keys, in order, into best (0 past n): a key's
// place is the number of keys above it, counted by four threads.  The whole
// CTA calls it, behind a barrier after the keys' writes; best is valid behind
// the next one.
__device__ __forceinline__ void pick16(const uint64_t *keys, int n, uint64_t *best) {
  if (threadIdx.x < TOP_K && static_cast<int>(threadIdx.x) >= n) best[threadIdx.x] = 0;
  for (int i0 = 0; i0 < n; i0 += THREADS / 4) {   // uniform trip count
    const int i = i0 + (threadIdx.x >> 2);
    const uint64_t mine = i < n ? keys[i] : 0;
    int above = 0;
    for (int j = threadIdx.x & 3; j < n; j += 4) above += keys[j] > mine;
    above += __shfl_xor_sync(0xffffffffu, above, 1);
    above += __shfl_xor_sync(0xffffffffu, above, 2);
    if (i < n && above < TOP_K && (threadIdx.x & 3) == 0) best[above] = mine;
  }
}

// One cluster per row.  The row's 16-byte-aligned vectors are cut evenly over
// its cs CTAs and their warps; the elements before and after them (a row may
// start at any element) go to rank 0's first warp.  Every warp streams its
// share through a ring of bulk copies of its own and meets nobody until the
// share is done.
//   Sums: d = (x - m) c and e = 2^d per logit, two logits per instruction
//   where the instruction set has it (subtract, scale, both sums; the maxima
//   of bf16 logits too: 86 us without, 80 with it at 1024 rows of 151 936).
//   Rank: counted only where a stage's maximum reaches the token's logit.
//   Alternatives: the stream keeps no list.  A thread's running maximum m is
//   also the maximum of what it saw; 16 threads reach the 16th largest of
//   these maxima, so the 16 largest logits reach it too, and they all lie
//   where a thread's maximum does.  The threads keep one maximum for each
//   eighth of the stream, so that only some 16 of the 2048 pieces are read
//   again.  (A list kept during the stream, with
//   votes, atomics and a meeting per stage, took 89 us where this takes 78 at
//   640 fp32 rows of 151 936.)  With fewer than 16 finite logits in a CTA's
//   share the floor is -inf, and all of the share is read again, some three
//   times: 520 us at 640 such rows.
// Each CTA sends its 16 keys and sums to rank 0.
template <typename T, int STAGES>
__global__ void __launch_bounds__(THREADS, CTAS) logprobs_kernel(const Args a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ uint4 ring_all[];
  Shared &sh = *reinterpret_cast<Shared *>(ring_all + ring_bytes(STAGES) / 16);
  const int cs = a.cs, row = blockIdx.x / cs, rank = blockIdx.x % cs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint4 *ring = ring_all + warp * STAGES * SV;
  uint64_t *full = sh.full[warp];
  if (lane == 0)
    for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
  if (tid == 0) {
    sh.listed = sh.owned = sh.failed = 0;
  }
  if (lane == 0) fence_mbar_init();
  pdl_start();
  const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.ld;
  const int id = a.ids[row], V = a.V;
  if (id < 0) {   // a skipped row (the whole cluster takes this branch)
    if (rank == 0) {
      if (tid == 0) {
        a.logprob[row] = 0.f;
        a.entropy[row] = 0.f;
        a.rank[row] = -1;
      }
      if (tid < a.n_top) {
        a.top_ids[static_cast<size_t>(row) * a.n_top + tid] = -1;
        a.top_lp[static_cast<size_t>(row) * a.n_top + tid] = 0.f;
      }
    }
    return;
  }
  const int head = min(V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / static_cast<int>(sizeof(T)));
  const int nv = (V - head) / N;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
  // This CTA's vectors, and this warp's pieces of SV of them: every WARPS-th,
  // so that the CTA as a whole reads on (8 streams a row cost a third of the
  // DRAM rate).
  constexpr int STEP = WARPS * SV;
  const int cta0 = static_cast<int>(static_cast<long long>(rank) * nv / cs);
  const int end = static_cast<int>(static_cast<long long>(rank + 1) * nv / cs), v0 = cta0 + warp * SV;
  const int ns = v0 < end ? (end - v0 + STEP - 1) / STEP : 0;
  auto fetch = [&](int s) {
    const int n = min(SV, end - v0 - s * STEP);
    mbar_arrive_expect_tx(&full[s % STAGES], n * 16);
    bulk_load(ring + (s % STAGES) * SV, xv + v0 + static_cast<size_t>(s) * STEP, n * 16, &full[s % STAGES]);
  };
  if (lane == 0)
    for (int s = 0; s < min(STAGES, ns); ++s) fetch(s);
  const bool known = id < V, want = a.n_top > 0;
  const float xt = known ? Elt<T>::ld(x + id) : INFINITY, xt_up = next_up(xt);
  const float c = a.inv_t * LOG2E_F;
  const uint64_t c2 = pack2(c, c);
  __syncthreads();                // barriers and counters are set up
  if (cs > 1) cluster_arrive();   // waited for before rank 0's shared memory is written
  float m = -INFINITY;
  uint64_t z2 = pack2(0.f, 0.f), w2 = z2;
  int cnt = 0;
  // the stages of the CTA's longest warp, in SEGS parts
  const int seg_len = ((end - cta0 + STEP - 1) / STEP + SEGS - 1) / SEGS;
  float seg = -INFINITY;
#pragma unroll
  for (int i = 0; i < SEGS; ++i) sh.seg[i][tid] = -INFINITY;
  bool ok = true;
  for (int s = 0, part = 0, left = seg_len; s < ns; ++s) {
    ok = mbar_wait(&full[s % STAGES], static_cast<uint32_t>((s / STAGES) & 1), nullptr, WAIT_NS);
    ok = !__any_sync(0xffffffffu, !ok);
    if (!ok) {   // a copy did not arrive: no answer; those under way land before the shared memory goes away
      sh.failed = 1;
      for (int t = s; t < min(ns, s + STAGES); ++t)
        mbar_wait(&full[t % STAGES], static_cast<uint32_t>((t / STAGES) & 1), nullptr, WAIT_NS / 8);
      break;
    }
    const int n = min(SV, end - v0 - s * STEP);
    uint4 raw[U];
    const uint4 *stage = ring + (s % STAGES) * SV + lane;
    if (n == SV) {
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = stage[u * 32];
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u] = make_uint4(Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE);
        if (u * 32 + lane < n) raw[u] = stage[u * 32];
      }
    }
    const float top = Vec<T>::maximum(raw);
    seg = max_nan(seg, top);
    const float mn = max_nan(m, seg);
    if (--left == 0 || s + 1 == ns) {
      sh.seg[part++][tid] = seg;
      seg = -INFINITY;
      left = seg_len;
    }
    // The vote needs every lane's maximum, so behind it the stage is in
    // registers and may be refilled.  (Behind a mere __syncwarp loads were
    // still on their way when the next copy's first bytes came.)
    if (__any_sync(0xffffffffu, mn != m)) {
      const float d = m == mn ? 0.f : fmaxf((m - mn) * c, FAR), f = fast_exp2(d);
      const uint64_t f2 = pack2(f, f);
      w2 = mul2(f2, fma2(z2, pack2(d, d), w2));
      z2 = mul2(f2, z2);
      m = mn;
    }
    if (lane == 0 && s + STAGES < ns) fetch(s + STAGES);
    const uint64_t neg2 = pack2(-mn, -mn);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[N];
      Vec<T>::unpack(raw[u], v);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        float d0, d1;
        unpack2(mul2(add2(pack2(v[k], v[k + 1]), neg2), c2), d0, d1);
        d0 = fmaxf(d0, FAR);   // -inf, and -inf less -inf
        d1 = fmaxf(d1, FAR);
        const uint64_t e2 = pack2(fast_exp2(d0), fast_exp2(d1));
        z2 = add2(z2, e2);
        w2 = fma2(e2, pack2(d0, d1), w2);
      }
    }
    if (top >= xt) {   // otherwise nothing to count: the token's own vector reaches its logit
      const int i0 = head + (v0 + s * STEP + lane) * N;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * 32 + lane >= n) continue;
        const int i = i0 + u * 32 * N;
        const float reach = i + N <= id ? xt : xt_up;   // before the token equal logits count too
        float v[N];
        Vec<T>::unpack(raw[u], v);
#pragma unroll
        for (int k = 0; k < N; ++k) cnt += v[k] >= reach;
        if (static_cast<unsigned>(id - i) < static_cast<unsigned>(N))   // the token's own vector
#pragma unroll
          for (int k = 0; k < N; ++k) cnt += i + k < id && v[k] == xt;
      }
    }
  }
  const float seen = m;   // the maximum of this thread's vectors
  Stat st;
  {
    float z0, z1, w0, w1;
    unpack2(z2, z0, z1);
    unpack2(w2, w0, w1);
    st = {m, z0 + z1, w0 + w1};
  }
  if (rank == 0 && warp == 0) {   // the elements outside of the vectors: < 2 N <= 16
    const int ends = head + (V - head - nv * N), i = lane < head ? lane : nv * N + lane;
    if (lane < ends) {
      const float v = Elt<T>::ld(x + i);
      if (v != -INFINITY) {
        rebase(st, max_nan(st.m, v), c);
        const float d = fmaxf((v - st.m) * c, FAR), e = fast_exp2(d);
        st.z += e;
        st.w = fmaf(e, d, st.w);
      }
      cnt += v > xt || (v == xt && i < id);
      sh.list[lane] = make_key(v, i);
    }
    if (lane == 0) sh.listed = ends;
  }
  // ---- the CTA's sums
  warp_join(st, cnt, c);
  if (lane == 0) sh.warp_stat[warp] = make_float4(st.m, st.z, st.w, __int_as_float(cnt));
  if (want) {
    // ---- a floor under the 16th largest of the threads' maxima: some 40
    // threads reach the smallest of the 8 warps' second largest
    const float one = warp_max_nan(seen);
    const int who = __ffs(__ballot_sync(0xffffffffu, seen == one)) - 1;   // -1: NaN
    const float two = warp_max_nan(lane == who ? -INFINITY : seen);
    if (lane == 0) sh.warp_two[warp] = two;
    __syncthreads();
    const int listed = sh.listed;
    float floor_v = sh.warp_two[0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) floor_v = fminf(floor_v, sh.warp_two[i]);
    // (their (maximum, thread) keys pass through the list behind the ends' keys;
    // with this floor itself 1024 rows took 85 us instead of 81: three times as
    // many pieces are read again)
    uint64_t *maxima = sh.list + TOP_K;
    if (seen >= floor_v) maxima[atomicAdd(&sh.owned, 1)] = make_key(seen, tid);
    __syncthreads();
    pick16(maxima, sh.owned, sh.best);
    __syncthreads();
    uint64_t floor_k = sh.best[TOP_K - 1];
    floor_v = floor_k ? key_value(floor_k) : -INFINITY;   // fewer than 16 threads hold anything comparable
    floor_k = 0;
    if (tid == 0) sh.owned = 0;
    __syncthreads();
    if (seen >= floor_v)
#pragma unroll
      for (int i = 0; i < SEGS; ++i)
        if (sh.seg[i][tid] >= floor_v) sh.owners[atomicAdd(&sh.owned, 1)] = static_cast<uint16_t>(i * THREADS + tid);
    __syncthreads();
    const int owned = sh.owned;
    // ---- their vectors again: keys at or above the floor into the list; an
    // overflow raises the floor to the 16th of what the list holds
    for (;;) {
      // item = (a piece's vector number, piece)
      const int items = owned * seg_len * U;
      constexpr int B = 4;   // loads in flight per thread
      for (int e0 = tid; e0 < items; e0 += THREADS * B) {
        uint4 raw[B];
        int at[B];
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const int e = e0 + u * THREADS;
          at[u] = -1;
          if (e < items) {
            const int k = e / owned, o = sh.owners[e - k * owned], t = o % THREADS;
            const int i = cta0 + ((o / THREADS) * seg_len + k / U) * STEP + (t >> 5) * SV + (k % U) * 32 + (t & 31);
            if (i < end) {
              at[u] = i;
              raw[u] = __ldg(xv + i);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < B; ++u) {
          if (at[u] < 0) continue;
          float v[N];
          Vec<T>::unpack(raw[u], v);
#pragma unroll
          for (int k = 0; k < N; ++k)
            if (v[k] >= floor_v) {
              const uint64_t key = make_key(v[k], head + at[u] * N + k);
              if (key >= floor_k) {
                const int to = atomicAdd(&sh.listed, 1);
                if (to < LIST) sh.list[to] = key;
              }
            }
        }
      }
      __syncthreads();
      const int total = sh.listed;
      pick16(sh.list, min(total, LIST), sh.best);
      __syncthreads();
      if (total <= LIST) break;
      floor_k = sh.best[TOP_K - 1];
      floor_v = key_value(floor_k);
      if (tid == 0) sh.listed = listed;
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  auto gather = [&](const float4 *of, int k) {   // a warp: the first k shares joined
    const float4 q = lane < k ? of[lane] : make_float4(-INFINITY, 0.f, 0.f, __int_as_float(0));
    st = {q.x, q.y, q.z};
    cnt = __float_as_int(q.w);
    warp_join(st, cnt, c);
  };
  if (warp == 0) {
    gather(sh.warp_stat, WARPS);
    if (sh.failed) st.m = NAN;
  }
  // ---- the cluster: every CTA's share into rank 0's shared memory
  if (cs > 1) {
    cluster_wait();
    if (warp == 0) {
      if (lane < TOP_K) st_dsmem_u64(dsmem_addr(&sh.peer_keys[rank * TOP_K + lane], 0), want ? sh.best[lane] : 0);
      if (lane == 31) st_dsmem_f4(dsmem_addr(&sh.peer_stat[rank], 0), make_float4(st.m, st.z, st.w, __int_as_float(cnt)));
    }
    // Every CTA gets here (its waits are bounded), and rank 0 stays until all
    // have: no share goes to shared memory that is not its own any more.
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    if (want) {   // a key's place is the number of keys above it (0: a CTA with fewer than 16)
      const int n = cs * TOP_K, i = tid >> 1;
      const uint64_t mine = i < n ? sh.peer_keys[i] : 0;
      const ulonglong2 *keys = reinterpret_cast<const ulonglong2 *>(sh.peer_keys);
      int above = 0;
#pragma unroll 8
      for (int j = tid & 1; j < n / 2; j += 2) {
        const ulonglong2 k = keys[j];
        above += (k.x > mine) + (k.y > mine);
      }
      above += __shfl_xor_sync(0xffffffffu, above, 1);
      if (mine && above < TOP_K && !(tid & 1)) sh.best[above] = mine;
      __syncthreads();
    }
    if (warp == 0) {
      gather(sh.peer_stat, cs);
    }
  }
  if (warp != 0) return;
  const bool empty = st.m == -INFINITY;      // nothing but -inf
  const float lz = log2f(st.z), lnz = lz * LN2_F;
  const float bad = st.m - st.m;             // NaN for a NaN or +inf maximum, else 0
  if (lane == 0) {
    a.logprob[row] = !known ? NAN : empty ? -INFINITY : fmaf(xt - st.m, a.inv_t, -lnz) + bad;
    a.entropy[row] = empty ? 0.f : (lz - st.w / st.z) * LN2_F + bad;
    a.rank[row] = known ? cnt : -1;
  }
  if (lane < a.n_top) {
    const uint64_t key = sh.best[lane];
    a.top_ids[static_cast<size_t>(row) * a.n_top + lane] = min(max(key_id(key), 0), V - 1);
    a.top_lp[static_cast<size_t>(row) * a.n_top + lane] = empty ? -INFINITY : fmaf(key_value(key) - st.m, a.inv_t, -lnz) + bad;
  }
}

}  // namespace
}  // namespace dflash

extern "C" DFLASH_API int dflash_token_logprobs(const void *logits, int dtype, int rows, int vocab, long long row_stride,
                                                const int32_t *token_ids, float temperature, int n_top,
                                                float *logprob, float *entropy, int32_t *rank, int32_t *top_ids,
                                                float *top_logprobs, dflash_stream_t stream) {
  using namespace dflash;
  if (dtype != DFLASH_BF16 && dtype != DFLASH_F32)
    return set_error(DFLASH_ERR_ARG, "token_logprobs: dtype must be bf16 or fp32");
  if (rows < 0 || vocab < 1 || n_top < 0 || n_top > TOP_K || n_top > vocab)
    return set_error(DFLASH_ERR_ARG, "token_logprobs: rows, vocab or n_top (0..16, <= vocab) out of range");
  if (row_stride < vocab) return set_error(DFLASH_ERR_SHAPE, "token_logprobs: row stride below the vocabulary");
  if (!(temperature >= 1e-4f) || !(temperature <= 1e4f))
    return set_error(DFLASH_ERR_ARG, "token_logprobs: temperature must be in 1e-4..1e4");
  if (rows == 0) return DFLASH_OK;
  if (!logits || !token_ids || !logprob || !entropy || !rank || (n_top > 0 && (!top_ids || !top_logprobs)))
    return set_error(DFLASH_ERR_ARG, "token_logprobs: null pointer");
  const int size = dtype == DFLASH_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size || off_words(token_ids, logprob, entropy, rank, top_ids, top_logprobs))
    return set_error(DFLASH_ERR_ALIGN, "token_logprobs: arrays must be aligned to their elements");
  if (rows > (1 << 27)) return set_error(DFLASH_ERR_SHAPE, "token_logprobs: at most 2^27 rows per call");
  Device dev;
  if (int e = current_device(&dev)) return e;
  Args a = {};
  a.x = logits;
  a.ld = row_stride;
  a.V = vocab;
  a.n_top = n_top;
  a.ids = token_ids;
  a.inv_t = 1.f / temperature;
  a.logprob = logprob;
  a.entropy = entropy;
  a.rank = rank;
  a.top_ids = top_ids;
  a.top_lp = top_logprobs;
  // One CTA per row where the rows fill a quarter of the resident CTAs, more
  // where they do not (64 fp32 rows of 151 936: 28 us on one CTA each, 15 on 4,
  // 23 on 8) and where a CTA's share is long against the tail of a wave of
  // them (640 such rows: 82 us on one, 79 on 2, 88 on 4).
  int cs = 1;
  while (cs < MAX_CLUSTER && ((4LL * rows * cs < CTAS * dev.sms && static_cast<long long>(cs) * MIN_SHARE < vocab) ||
                              static_cast<long long>(vocab) * size > static_cast<long long>(cs) * MAX_SHARE))
    cs *= 2;
  const bool f32 = dtype == DFLASH_F32, deep = static_cast<long long>(rows) * cs <= 2 * dev.sms;
  auto *kernel = deep ? (f32 ? logprobs_kernel<float, DEEP> : logprobs_kernel<__nv_bfloat16, DEEP>)
                      : (f32 ? logprobs_kernel<float, WIDE> : logprobs_kernel<__nv_bfloat16, WIDE>);
  const int smem = smem_bytes(deep ? DEEP : WIDE);
  static std::atomic<uint64_t> smem_set[4];
  if (int e = allow_smem(smem_set[f32 + 2 * deep], dev, kernel, smem)) return e;
  cudaLaunchConfig_t cfg = {};
  a.cs = cs;
  cfg.gridDim = dim3(static_cast<unsigned>(cs) * rows);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_check(cudaLaunchKernelEx(&cfg, kernel, a), "token_logprobs launch");
}
