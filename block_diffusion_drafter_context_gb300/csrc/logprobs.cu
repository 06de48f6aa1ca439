// Log probabilities of given tokens, with the row's entropy, the token's rank
// and the 16 most probable alternatives (dflash_token_logprobs).
//
// With y = x / T, m = max y and z = sum e^(y - m) over the vocabulary:
//   logprob = y_t - m - log z,   entropy = log z - sum e^(y - m) (y - m) / z,
//   rank = #{v : x_v > x_t, or x_v = x_t and v < t}.
// Everything comes from one pass over the logits: a running (m, z, w = sum
// e^(y-m) (y-m)) per thread, joined as m' = max, z' = z e^(m-m'),
// w' = e^(m-m') (w + z (m - m')); the rank is a count against the token's own
// logit, read first; the alternatives are a filtered top-16 scan.  Bound by
// the logits' HBM bytes; a row is cut over a cluster of CTAs, which join
// through distributed shared memory, so that no workspace is needed.
#include "top16.cuh"
#include "target.h"

#include <math.h>

namespace dflash {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32, CTAS = 3;   // CTAS: resident per SM
constexpr int MAX_CLUSTER = 16;
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
};

// ---- shared memory of a CTA: a ring of 64 KB of logits in stages of 32 logits
// per thread (fewer made the meetings dominate: 101 against 88 us at 640 fp32
// rows of 151 936), then
constexpr int PER_STAGE = 32 * THREADS, RING = 65536, MAX_STAGES = 4;
constexpr int LIST = 512;                            // candidates a CTA can list
constexpr int FOLD_FIRST = 24, FOLD = 96;            // the length above which the list is folded: first, then
constexpr unsigned long long WAIT_NS = 2000000000ull;
struct Shared {
  alignas(16) uint64_t list[LIST];                   // candidates for the 16 largest (value, id) keys, unordered
  uint64_t best[TOP_K];      // the 16 largest in order, 0 where there are fewer
  uint64_t full[MAX_STAGES], mail;
  alignas(16) uint64_t peer_keys[MAX_CLUSTER * TOP_K];   // rank 0: every CTA's best
  float4 peer_stat[MAX_CLUSTER];                         // rank 0: (m, z, w, count) of every CTA
  float4 warp_stat[WARPS];
  float warp_two[WARPS], warp_tau[WARPS];
  int listed;                // candidates offered
};
constexpr int SMEM = RING + static_cast<int>(sizeof(Shared)) + 16;

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
// its cs CTAs; the elements before and after them (a row may start at any
// element) go to rank 0's first warp.  A CTA streams its share through a ring
// of bulk copies, so the bytes in flight do not depend on how far the
// arithmetic is, and meets once per stage.
//   Sums: d = (x - m) c and e = 2^d per logit, two logits per instruction
//   where the instruction set has it (subtract, scale, both sums).
//   Rank: counted only in vectors whose maximum reaches the token's logit.
//   Alternatives: logits at or above a floor that at least 16 logits reach
//   (at first the smallest of the 8 warps' second largest lane maxima, which
//   some 40 of 8192 logits reach) go to a list: a lane collects the bits of
//   its hits, takes room for them at once and reads them back from the ring
//   (a vote or an atomic per logit took four times as long).  The list is
//   folded to its 16 largest once, which makes the floor the 16th of what was
//   seen, and again only if it grows long.  A stage that overflows the list
//   raises the floor to the 16th of what the list holds and is offered again.
// Each CTA sends its 16 keys and sums to rank 0.
template <typename T>
__global__ void __launch_bounds__(THREADS, CTAS) logprobs_kernel(const Args a) {
  constexpr int N = Vec<T>::N, U = 32 / N, SV = PER_STAGE / N;   // vectors per thread, and of a stage
  constexpr int STAGES = RING / 16 / SV;
  static_assert(STAGES >= 2 && STAGES <= MAX_STAGES, "ring");
  extern __shared__ uint4 ring[];
  Shared &sh = *reinterpret_cast<Shared *>(ring + RING / 16);
  const int cs = a.cs, row = blockIdx.x / cs, rank = blockIdx.x % cs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], 1);
    mbar_init(&sh.mail, cs);
    fence_mbar_init();
    sh.listed = 0;
  }
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
  __syncthreads();                // the barriers are set up
  if (cs > 1) cluster_arrive();   // waited for before a peer's mailbox is written
  const int head = min(V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / static_cast<int>(sizeof(T)));
  const int nv = (V - head) / N;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
  const int v0 = static_cast<int>(static_cast<long long>(rank) * nv / cs);
  const int mine = static_cast<int>(static_cast<long long>(rank + 1) * nv / cs) - v0;   // this CTA's vectors
  const int ns = (mine + SV - 1) / SV;
  auto fetch = [&](int s) {
    const int n = min(SV, mine - s * SV);
    mbar_arrive_expect_tx(&sh.full[s % STAGES], n * 16);
    bulk_load(ring + (s % STAGES) * SV, xv + v0 + static_cast<size_t>(s) * SV, n * 16, &sh.full[s % STAGES]);
  };
  if (tid == 0)
    for (int s = 0; s < min(STAGES, ns); ++s) fetch(s);
  const bool known = id < V, want = a.n_top > 0;
  const float xt = known ? Elt<T>::ld(x + id) : INFINITY, xt_up = next_up(xt);
  const float c = a.inv_t * LOG2E_F;
  const uint64_t c2 = pack2(c, c);
  float m = -INFINITY;
  uint64_t z2 = pack2(0.f, 0.f), w2 = z2;
  int cnt = 0;
  const int ends = rank == 0 ? head + (V - head - nv * N) : 0;   // < 2 N <= 16 elements outside of the vectors
  int listed = ends;              // keys in the list before the current stage
  if (rank == 0 && warp == 0) {
    const int i = lane < head ? lane : head + nv * N + (lane - head);
    if (lane < ends) {
      const float v = Elt<T>::ld(x + i);
      m = v;
      z2 = pack2(v == -INFINITY ? 0.f : 1.f, 0.f);
      cnt = v > xt || (v == xt && i < id);
      sh.list[lane] = make_key(v, i);
    }
    if (lane == 0) sh.listed = ends;
  }
  if (want && ends) __syncthreads();
  float floor_v = -INFINITY;   // at least 16 of the row's logits are at or above (floor_v, floor_k)
  uint64_t floor_k = 0;
  bool folded = false, ok = true;
  for (int s = 0; s < ns; ++s) {
    ok = ok && mbar_wait(&sh.full[s % STAGES], static_cast<uint32_t>((s / STAGES) & 1), nullptr, WAIT_NS);
    const int n = ok ? min(SV, mine - s * SV) : 0;
    const uint4 *st = ring + (s % STAGES) * SV;
    uint4 raw[U];
    float vmax[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      raw[u] = make_uint4(Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE);
      if (u * THREADS + tid < n) raw[u] = st[u * THREADS + tid];
    }
    float mx = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[N];
      Vec<T>::unpack(raw[u], v);
      vmax[u] = max_nan(max_nan(v[0], v[1]), max_nan(v[2], v[3]));
      if (N == 8) vmax[u] = max_nan(vmax[u], max_nan(max_nan(v[N - 4], v[N - 3]), max_nan(v[N - 2], v[N - 1])));
      mx = max_nan(mx, vmax[u]);
    }
    if (want && s == 0) {
      const float one = warp_max_nan(mx);
      const int who = __ffs(__ballot_sync(0xffffffffu, mx == one)) - 1;   // -1: NaN
      const float two = warp_max_nan(lane == who ? -INFINITY : mx);
      if (lane == 0) sh.warp_two[warp] = two;
      __syncthreads();
      floor_v = sh.warp_two[0];
#pragma unroll
      for (int i = 1; i < WARPS; ++i) floor_v = fminf(floor_v, sh.warp_two[i]);
      if (floor_v == -INFINITY) {   // a warp without two: 16 of one warp's lanes instead
        const float tau = warp_16th_largest(mx, lane);
        if (lane == 0) sh.warp_tau[warp] = tau;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WARPS; ++i) floor_v = fmaxf(floor_v, sh.warp_tau[i]);
      }
    }
    const float mn = max_nan(m, mx);
    if (mn != m) {
      const float d = fmaxf((m - mn) * c, FAR), f = fast_exp2(d);
      const uint64_t f2 = pack2(f, f);
      w2 = mul2(f2, fma2(z2, pack2(d, d), w2));
      z2 = mul2(f2, z2);
      m = mn;
    }
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
    const int i0 = head + (v0 + s * SV + tid) * N;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * THREADS * N;
      const float reach = i + N <= id ? xt : xt_up;   // before the token equal logits count too
      const bool own = static_cast<unsigned>(id - i) < static_cast<unsigned>(N);   // the token's own vector
      if ((vmax[u] >= reach || own) && u * THREADS + tid < n) {
        float v[N];
        Vec<T>::unpack(raw[u], v);
#pragma unroll
        for (int k = 0; k < N; ++k) cnt += v[k] >= reach;
        if (own)
#pragma unroll
          for (int k = 0; k < N; ++k) cnt += i + k < id && v[k] == xt;
      }
    }
    if (!want) {
      ok = __syncthreads_and(ok);
    } else {
      for (;;) {
        if (mx >= floor_v) {   // few lanes, once the floor is tight
          uint32_t hits = 0;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[N];
            Vec<T>::unpack(raw[u], v);
#pragma unroll
            for (int k = 0; k < N; ++k) hits |= v[k] >= floor_v ? 1u << (u * N + k) : 0u;
            if (u * THREADS + tid >= n) hits &= (1u << (u * N)) - 1;
          }
          auto key_of = [&](int e) {
            const int u = e / N, k = e % N;
            return make_key(Elt<T>::ld(reinterpret_cast<const T *>(st + u * THREADS + tid) + k), i0 + u * THREADS * N + k);
          };
          for (uint32_t left = floor_k ? hits : 0u; left; left &= left - 1) {   // equal values of higher ids: out
            const int e = __ffs(left) - 1;
            if (key_of(e) < floor_k) hits &= ~(1u << e);
          }
          for (int to = hits ? atomicAdd(&sh.listed, __popc(hits)) : 0; hits; hits &= hits - 1, ++to)
            if (to < LIST) sh.list[to] = key_of(__ffs(hits) - 1);
        }
        ok = __syncthreads_and(ok);
        const int total = sh.listed;
        __syncthreads();   // read by all before it changes
        if (total <= LIST && (s + 1 == ns || total <= (folded ? FOLD : FOLD_FIRST))) {
          listed = total;
          break;
        }
        pick16(sh.list, min(total, LIST), sh.best);
        __syncthreads();
        folded = true;
        floor_k = max(floor_k, sh.best[TOP_K - 1]);
        floor_v = floor_k ? key_value(floor_k) : -INFINITY;
        if (total <= LIST) {
          if (tid < TOP_K) sh.list[tid] = sh.best[tid];
          listed = min(total, TOP_K);
        }                      // else this stage again, above the new floor
        if (tid == 0) sh.listed = listed;
        __syncthreads();
        if (total <= LIST) break;
      }
    }
    if (tid == 0 && ok && s + STAGES < ns) fetch(s + STAGES);
  }
  if (!ok) {   // a copy did not arrive: no answer
    m = NAN;
    if (tid == 0)   // let every issued copy land before the shared memory goes away
      for (int s = 0; s < ns; ++s) mbar_wait(&sh.full[s % STAGES], static_cast<uint32_t>((s / STAGES) & 1), nullptr, WAIT_NS / 64);
  }
  // ---- the CTA's sums and its 16 keys
  Stat st;
  {
    float z0, z1, w0, w1;
    unpack2(z2, z0, z1);
    unpack2(w2, w0, w1);
    st = {m, z0 + z1, w0 + w1};
  }
  warp_join(st, cnt, c);
  if (lane == 0) {
    sh.warp_stat[warp] = make_float4(st.m, st.z, st.w, __int_as_float(cnt));
  }
  __syncthreads();
  if (want) pick16(sh.list, listed, sh.best);
  auto gather = [&](const float4 *of, int k) {   // a warp: the first k shares joined
    const float4 q = lane < k ? of[lane] : make_float4(-INFINITY, 0.f, 0.f, __int_as_float(0));
    st = {q.x, q.y, q.z};
    cnt = __float_as_int(q.w);
    warp_join(st, cnt, c);
  };
  if (warp == 0) gather(sh.warp_stat, WARPS);
  __syncthreads();   // best is complete
  // ---- the cluster: every CTA's share into rank 0's mailbox
  if (cs > 1) {
    cluster_wait();
    if (warp == 0) {
      if (lane < TOP_K) st_dsmem_u64(dsmem_addr(&sh.peer_keys[rank * TOP_K + lane], 0), want ? sh.best[lane] : 0);
      if (lane == 31) st_dsmem_f4(dsmem_addr(&sh.peer_stat[rank], 0), make_float4(st.m, st.z, st.w, __int_as_float(cnt)));
      fence_acq_rel_cluster();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(dsmem_addr(&sh.mail, 0));
    }
    if (rank != 0) return;
    const bool all = mbar_wait_cluster(&sh.mail, 0, nullptr, WAIT_NS);
    if (want) {   // keys below some CTA's 16th are out (0: a CTA with fewer)
      uint64_t floor = 1;
      for (int r = 0; r < cs; ++r) floor = max(floor, sh.peer_keys[r * TOP_K + TOP_K - 1]);
      if (tid == 0) sh.listed = 0;
      __syncthreads();
      if (tid < cs * TOP_K && sh.peer_keys[tid] >= floor) sh.list[atomicAdd(&sh.listed, 1)] = sh.peer_keys[tid];
      __syncthreads();
      pick16(sh.list, sh.listed, sh.best);
      __syncthreads();
    }
    if (warp == 0) {
      gather(sh.peer_stat, cs);
      if (!all) st.m = NAN;
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
  if (reinterpret_cast<uintptr_t>(logits) % size)
    return set_error(DFLASH_ERR_ALIGN, "token_logprobs: logits not aligned to their elements");
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
  // Rows enough for half of the resident CTAs take one CTA each; fewer are cut
  // over clusters until that many CTAs work, each with a stage at least (64
  // fp32 rows of 151 936: 42 us on one CTA, 25 on 4, 32 on 16; 640 rows: 101
  // on one, 129 on 4).
  int cs = 1;
  while (cs < MAX_CLUSTER && 2LL * rows * cs < CTAS * dev.sms && static_cast<long long>(cs) * PER_STAGE < vocab) cs *= 2;
  auto *kernel = dtype == DFLASH_F32 ? logprobs_kernel<float> : logprobs_kernel<__nv_bfloat16>;
  static std::atomic<uint64_t> smem_set[2], wide_set[2];
  const int which = dtype == DFLASH_F32;
  if (int e = allow_smem(smem_set[which], dev, kernel, SMEM)) return e;
  if (cs > 8)
    if (int e = allow_wide_clusters(wide_set[which], dev, kernel)) return e;
  cudaLaunchConfig_t cfg = {};
  a.cs = cs;
  cfg.gridDim = dim3(static_cast<unsigned>(cs) * rows);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
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
