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

constexpr int THREADS = 256, WARPS = THREADS / 32;
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

__device__ __forceinline__ void join(Stat &a, float m, float z, float w, float c) {
  const float mn = max_nan(a.m, m);
  const float da = a.m == mn ? 0.f : fmaxf((a.m - mn) * c, FAR), db = m == mn ? 0.f : fmaxf((m - mn) * c, FAR);
  const float fa = fast_exp2(da), fb = fast_exp2(db);
  a.w = fa * fmaf(a.z, da, a.w) + fb * fmaf(z, db, w);
  a.z = fa * a.z + fb * z;
  a.m = mn;
}

template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

struct Shared {
  uint64_t lists[WARPS][TOP_K];
  uint64_t top[TOP_K];       // this CTA's list
  float m[WARPS], z[WARPS], w[WARPS];
  int cnt[WARPS];
  float cm, cz, cw;          // this CTA's sums
  int ccnt;
};

__device__ __forceinline__ uint64_t ld_dsmem_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// cluster = one row, cs CTAs.  The row's 16-byte-aligned
// vectors are cut evenly over them; the elements before and after the
// vectors (a row may start at any element) go to rank 0's first warp.
template <typename T>
__global__ void __launch_bounds__(THREADS) logprobs_kernel(const Args a) {
  constexpr int N = Vec<T>::N, U = 32 / N;   // 32 logits per thread in flight
  __shared__ Shared sh;
  const int cs = a.cs, row = blockIdx.x / cs, rank = blockIdx.x % cs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_start();
  const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.ld;
  const int id = a.ids[row], V = a.V;
  if (id < 0) {   // a skipped row (the whole cluster takes this branch)
    if (rank == 0) {
      if (threadIdx.x == 0) {
        a.logprob[row] = 0.f;
        a.entropy[row] = 0.f;
        a.rank[row] = -1;
      }
      if (static_cast<int>(threadIdx.x) < a.n_top) {
        a.top_ids[static_cast<size_t>(row) * a.n_top + threadIdx.x] = -1;
        a.top_lp[static_cast<size_t>(row) * a.n_top + threadIdx.x] = 0.f;
      }
    }
    return;
  }
  const bool known = id < V;
  const float xt = known ? Elt<T>::ld(x + id) : 0.f;
  const float c = a.inv_t * LOG2E_F;
  const int head = min(V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / static_cast<int>(sizeof(T)));
  const int nv = (V - head) / N;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
  const int v0 = static_cast<int>(static_cast<long long>(rank) * nv / cs);
  const int v1 = static_cast<int>(static_cast<long long>(rank + 1) * nv / cs);
  Stat st = {-INFINITY, 0.f, 0.f};
  int cnt = 0;
  uint64_t list = 0, thr = 0;
  const bool want = a.n_top > 0;
  auto add = [&](float v) {   // one logit into the sums
    join(st, v, v == -INFINITY ? 0.f : 1.f, 0.f, c);
  };
  if (rank == 0 && warp == 0) {
    const int ends = head + (V - head - nv * N);   // < 2 N <= 32
    const int i = lane < head ? lane : head + nv * N + (lane - head);
    const bool in = lane < ends;
    const float v = in ? Elt<T>::ld(x + i) : -INFINITY;
    if (in) {
      add(v);
      if (v > xt || (v == xt && i < id)) ++cnt;
    }
    if (want) offer(list, thr, in ? make_key(v, i) : 0, lane);
  }
  for (int wb = v0 + warp * 32; wb < v1; wb += WARPS * 32 * U) {   // warp-uniform trip count
    uint4 raw[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = wb + u * WARPS * 32 + lane;
      in[u] = i < v1;
      if (in[u]) raw[u] = __ldcs(xv + i);
    }
    float bmax[U];   // per vector
    float mx = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bmax[u] = -INFINITY;
      if (in[u]) {
        float v[N];
        Vec<T>::unpack(raw[u], v);
        bmax[u] = v[0];
#pragma unroll
        for (int k = 1; k < N; ++k) bmax[u] = max_nan(bmax[u], v[k]);
      }
      mx = max_nan(mx, bmax[u]);
    }
    // ---- sums, against the maximum with this batch in it
    const float mn = max_nan(st.m, mx);
    if (mn != st.m) {
      const float d = fmaxf((st.m - mn) * c, FAR), f = fast_exp2(d);
      st.w = f * fmaf(st.z, d, st.w);
      st.z *= f;
      st.m = mn;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in[u]) continue;
      float v[N];
      Vec<T>::unpack(raw[u], v);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float d = fmaxf((v[k] - mn) * c, FAR), e = fast_exp2(d);   // -inf less -inf too: FAR
        st.z += e;
        st.w = fmaf(e, d, st.w);
      }
      // ---- rank: most vectors of a probable token's row hold nothing above it
      if (bmax[u] >= xt) {
        const int i0 = head + (wb + u * WARPS * 32 + lane) * N;
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (v[k] > xt || (v[k] == xt && i0 + k < id)) ++cnt;
      }
    }
    // ---- the 16 largest (value, id) keys: while the list fills, only values
    // at or above the 16th largest lane maximum can belong to it; after that
    // only those at or above the list's 16th
    if (want) {
      float lo_v = thr == 0 ? warp_16th_largest(mx, lane) : key_value(thr);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!__any_sync(0xffffffffu, in[u] && bmax[u] >= lo_v)) continue;
        float v[N];
        Vec<T>::unpack(raw[u], v);
        const int i0 = head + (wb + u * WARPS * 32 + lane) * N;
#pragma unroll
        for (int k = 0; k < N; ++k) offer(list, thr, in[u] && v[k] >= lo_v ? make_key(v[k], i0 + k) : 0, lane);
        if (thr != 0) lo_v = fmaxf(lo_v, key_value(thr));
      }
    }
  }
  // ---- the CTA's warps
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, st.m, o), z2 = __shfl_xor_sync(0xffffffffu, st.z, o),
                w2 = __shfl_xor_sync(0xffffffffu, st.w, o);
    join(st, m2, z2, w2, c);
    cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
  }
  if (lane < TOP_K) sh.lists[warp][lane] = list;
  if (lane == 0) {
    sh.m[warp] = st.m, sh.z[warp] = st.z, sh.w[warp] = st.w;
    sh.cnt[warp] = cnt;
  }
  __syncthreads();
  if (warp == 0) {
    if (want) {
      uint64_t l2 = 0, t2 = 0;
      const uint64_t *all = &sh.lists[0][0];
      for (int i = lane; i < WARPS * TOP_K; i += 32) offer(l2, t2, all[i], lane);
      if (lane < TOP_K) sh.top[lane] = l2;
    }
    if (lane == 0) {
      Stat s = {-INFINITY, 0.f, 0.f};
      int n = 0;
      for (int i = 0; i < WARPS; ++i) {
        join(s, sh.m[i], sh.z[i], sh.w[i], c);
        n += sh.cnt[i];
      }
      sh.cm = s.m, sh.cz = s.z, sh.cw = s.w;
      sh.ccnt = n;
    }
  }
  if (cs > 1) cluster_sync();
  else __syncthreads();
  // ---- the cluster's CTAs, in rank order
  if (rank == 0 && warp == 0) {
    Stat s = {-INFINITY, 0.f, 0.f};
    int n = 0;
    for (int r = 0; r < cs; ++r) {
      join(s, __uint_as_float(ld_dsmem_u32(dsmem_addr(&sh.cm, r))), __uint_as_float(ld_dsmem_u32(dsmem_addr(&sh.cz, r))),
           __uint_as_float(ld_dsmem_u32(dsmem_addr(&sh.cw, r))), c);
      n += static_cast<int>(ld_dsmem_u32(dsmem_addr(&sh.ccnt, r)));
    }
    uint64_t l3 = 0, t3 = 0;
    if (want)
      for (int i = lane; i < cs * TOP_K; i += 32)
        offer(l3, t3, ld_dsmem_u64(dsmem_addr(&sh.top[i % TOP_K], i / TOP_K)), lane);
    const bool empty = s.m == -INFINITY;     // nothing but -inf
    const float lz = log2f(s.z), lnz = lz * LN2_F;
    const float bad = s.m - s.m;             // NaN for a NaN or +inf maximum, else 0
    if (lane == 0) {
      a.logprob[row] = !known ? NAN : empty ? -INFINITY : fmaf(xt - s.m, a.inv_t, -lnz) + bad;
      a.entropy[row] = empty ? 0.f : (lz - s.w / s.z) * LN2_F + bad;
      a.rank[row] = known ? n : -1;
    }
    if (lane < a.n_top) {
      const float v = key_value(l3);
      a.top_ids[static_cast<size_t>(row) * a.n_top + lane] = min(max(key_id(l3), 0), V - 1);
      a.top_lp[static_cast<size_t>(row) * a.n_top + lane] = empty ? -INFINITY : fmaf(v - s.m, a.inv_t, -lnz) + bad;
    }
  }
  if (cs > 1) cluster_sync();   // no CTA leaves while its share is read
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
  int sms = 0;
  if (int e = device_sms(&sms)) return e;
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
  // a row over enough CTAs to fill the GPU, of at least a batch of loads each
  const int per = THREADS * 32;
  int cs = 1;
  while (cs < 8 && static_cast<long long>(rows) * cs < 8LL * sms && static_cast<long long>(cs) * per < vocab) cs *= 2;
  auto *kernel = dtype == DFLASH_F32 ? logprobs_kernel<float> : logprobs_kernel<__nv_bfloat16>;
  cudaLaunchConfig_t cfg = {};
  a.cs = cs;
  cfg.gridDim = dim3(static_cast<unsigned>(cs) * rows);
  cfg.blockDim = dim3(THREADS);
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
